// tree_attention.cu -- attention of the nodes of a tree of drafts over a paged cache and over each
// other (include/svd_tree.h).
//
// What bounds it: every cached key and value is read once (2 x 2 bytes x D per key head and token)
// and serves the n * Hq / Hkv query rows of its head.  Up to about 128 rows that is less than the
// tensor cores' rate over HBM's, so the kernel streams the cache through shared memory and does all
// arithmetic behind it, until the power cap lowers the clock (1965 MHz for one request, 1335 for 128 sequences of 500
// to 6000 tokens back to back, 1080 at 6000 each).  With more rows no unit is full: at 512 rows a key head of 64
// elements the exponentials (16 a clock and SM) are half of the time, the tensor pipe is active in 25% of the cycles
// and 41% of the issue slots are used; two softmax warps a scheduler, each reading S twice from TMEM, do not hide
// one another's waits.
//
// Work.  An item is one sequence and key head; its keys are tiles of 128: the cached ones, then one tile of
// the drafted nodes.  All tiles of all items form one line (with a few places for the start and end of
// each item) that is cut into equal parts, so ragged lengths balance by themselves and one long sequence
// spreads over the whole GPU.  A CTA takes one part for one group of 128 query rows (a row is a node and a
// query head); the CTAs of the same part and different groups run side by side and share the part's keys
// through L2.  A part that holds a whole item writes its result; otherwise it leaves the unnormalised sum with
// the row maxima and sums in the workspace, and a second kernel (a programmatic dependent, its launch hidden)
// joins the parts in a fixed order.
//
// Roles in a CTA.  Two warps load K and V tiles page by page by TMA (128-byte swizzle), each into a ring of
// its own.  Two warps issue tcgen05.mma: one S = Q K^T into the next of three TMEM slots as soon as it is
// free, one O += P V with P read from TMEM.  Two softmax warpgroups take the tiles in turn, thread = row, so
// the sums and maxima of a tile need no exchange.  A warpgroup reads S and moves the row's reference maximum
// only when a tile exceeds it by more than 2^8 (the sums and O share the stale reference, so the quotient is
// exact all the same, and O in TMEM is rescaled rarely), hands the reference to the other warpgroup, and
// writes P = exp2(S - m) over S in the tensors' type (that rounding, at most half a step of the type per
// weight, is what the matrix instruction takes; maxima and sums stay fp32).  In fp16 the weights carry a factor of
// 2^7, see kLift.  Where an item ends, Q of the next
// one is fetched behind the last tile's softmax, and its first S forms while O is written out.
//
// Why so (cycles a tile, heads of 128; a tile's bytes take 2800 at HBM's rate and 1965 MHz): one softmax
// warpgroup alone took 1850 to 2200 besides its waits, of which 1024 are exponentials, and two that split the
// columns lost as much to their exchange; one warp for all products was busy 2300, most of it with waits; one
// warp for all loads 3200 where pages have 16 tokens.  As it is a tile takes about 1200 to 1700, less than its
// bytes: 17 nodes over 6000 tokens of 128 sequences take 515 to 600 us, 5.3 to 6.2 TB/s (a copy reaches 6.5).
//
// The running maximum and sum are those of the online softmax (Milakov and Gimelshein, 2018); to move the reference
// only beyond a threshold is a published refinement of it.
//
// Masks.  Columns behind the cache length and nodes that are not ancestors get P = 0 whatever S
// holds.  0 * NaN would still reach O through the matrix product, so rows of V behind the length
// are zeroed in shared memory, and elements of drafted V that are not finite are taken out there and
// added back, in the epilogue, to the rows that do see their node.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "tc_device.cuh"
#include "tree_device.cuh"

namespace svd {

namespace {

constexpr int kCtas = 148;         // one per SM of a B200
constexpr int kTile = 128;         // keys per tile, rows per group
constexpr uint64_t kWaitNs = 1000000000ull;
// Places of an item on the line besides its tiles: what its start and end cost, in tiles.  With none the parts of
// many short items ended last.  us with 0 / 2 / 3 / 4 / 6 places, 17 nodes, 32/8 heads:
//   32 sequences of 1 to 4096 tokens, heads of 128, pages of 16     95 /  77 /  77 /  78 /  80
//   the same, pages of 128                                          80 /  71 /  68 /  67 /  67
//   the same, heads of 64, pages of 16                              76 /  62 /  57 /  57 /  59
//   the same, heads of 64, pages of 128                             80 /  67 /  63 /  61 /  62
//   128 of 500 to 6000, heads of 128, pages of 64                  336 / 320 / 313 / 308 / 304
//   the same, heads of 64, pages of 16                             256 / 244 / 242 / 244 / 245
//   64 of 0 to 300, heads of 128, pages of 16                       51 /  46 /  44 /  44 /  43
//   the same, heads of 64, pages of 64                              45 /  40 /  39 /  39 /  39
constexpr int kItemCost = 3;
constexpr int kCombineWarps = 8;
constexpr int kLens = 64;          // sequences of a part whose lengths are kept in shared memory

struct PartInfo {                  // what the combine kernel needs to know of the item that starts in a
    int b, hk, last;               // part and does not end there: last part it reaches, or -1
};

struct AttnWs {
    size_t info, ml, o, total;
};
// Row groups, the parts that the line is cut into at most, and CTAs (more than one per SM only where a
// key head has more than 148 row groups).  From 75 to 147 groups (9473 to 18816 rows a key head) there is one part,
// and up to half of the SMs have nothing to do.
__host__ __device__ inline int row_groups(int rows) { return (rows + kTile - 1) / kTile; }
__host__ __device__ inline int max_parts(int groups) { return groups >= kCtas ? 1 : kCtas / groups; }
inline AttnWs attn_ws(int rows, int D) {
    const size_t used = rows < kTile ? rows : kTile, groups = row_groups(rows);
    const size_t ctas = groups * max_parts(static_cast<int>(groups));
    AttnWs L;
    L.info = sizeof(WsHeader);
    L.ml = align256(L.info + sizeof(PartInfo) * ctas);
    L.o = align256(L.ml + sizeof(float2) * 2 * ctas * used);
    L.total = align256(L.o + sizeof(float) * 2 * ctas * used * static_cast<size_t>(D));
    return L;
}

struct alignas(64) AttnParams {
    CUtensorMap ck, cv, nk, nv;    // cache and drafted nodes
    svd_tree_attention_args a;
    int G, rows, used, NR;         // heads per key head, its query rows, rows kept per slot, row groups
    int page_rows, page_shift;     // rows per TMA box, log2(page_size)
    int nb;                        // columns of the drafted tile, a multiple of 16
    float c, thr;                  // |scale| log2(e); 8 / c
    int qflip, qzero;              // the sign of the scale goes to Q; a scale of 0 zeroes Q
    uint32_t* status;
    PartInfo* info;                // [CTAs]
    float2* ml;                    // [2 CTAs][used]: reference maximum (raw scores), sum
    float* o;                      // [2 CTAs][used][D]
};

// Tiles of sequence b: its cached ones and the drafted one.
__device__ __forceinline__ int cache_len_of(const AttnParams& p, int b) {
    const long long cap = static_cast<long long>(p.a.max_pages) << p.page_shift;
    const int len = p.a.n_pages > 0 ? __ldg(p.a.cache_len + b) : 0;
    return len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile + 1; }

// A run of tiles of one item within this CTA's part.
struct Segment {
    int b, hk, len;
    int tile0, tile1, tiles;
};
// Steps through the segments of the part [lo, hi) of the line; `base` is where sequence b begins.  On the
// line an item is kItemCost places, which stand for its start and end, and then its tiles.
struct Walker {
    long long start, hi;           // where the item begins, and the part ends
    int first;                     // sequence in which the part begins
    bool any;
    Segment s;
    __device__ Walker(const AttnParams& p, long long lo, long long end, long long base, int b) : hi(end), first(b), any(lo < end) {
        if (!any) return;
        s.b = b;
        s.len = cache_len_of(p, b);
        s.tiles = tiles_of(s.len);
        const int width = s.tiles + kItemCost;
        s.hk = static_cast<int>((lo - base) / width);
        start = base + static_cast<long long>(s.hk) * width;
        s.tile0 = s.tile1 = max(0, static_cast<int>(lo - start) - kItemCost);
    }
    __device__ __forceinline__ bool next(const AttnParams& p, const int* lens) {
        if (!any) return false;
        if (s.tile1 == s.tiles) {      // the item before is done
            start += s.tiles + kItemCost;
            if (start >= hi) return any = false;
            s.tile1 = 0;
            if (++s.hk == p.a.Hkv) {
                s.hk = 0;
                ++s.b;
                // (from shared memory: behind the busy memory system a load takes thousands of cycles)
                const int i = s.b - first;
                s.len = i < kLens ? lens[i] : cache_len_of(p, s.b);
                s.tiles = tiles_of(s.len);
            }
        }
        s.tile0 = s.tile1;
        const long long left = hi - start - kItemCost;
        s.tile1 = s.tiles <= left ? s.tiles : max(0, static_cast<int>(left));
        return any = s.tile1 > s.tile0;
    }
};

struct Control {
    uint64_t full[2][6], empty[2][6];   // of the K ring, of the V ring
    uint64_t s_full[3], p_full[3], pv_done[3], m_ready[4][2], pair[4], aux[2], q_full, o_free, drain[2];
    long long lo, hi, base, total, parts;
    unsigned long long poison[2];  // drafted nodes with a V element that is not finite (alternating)
    int b;
    uint32_t tmem;
    int abort;
    int lens[kLens];
    float ref[2][kTile];           // reference maxima after a tile, by its warpgroup
    float sum[2][kTile];           // sums of the warpgroups at a segment's end
};

template <bool FP16>
__device__ __forceinline__ float to_f32(uint16_t w) {
    return FP16 ? __half2float(__ushort_as_half(w)) : __uint_as_float(static_cast<uint32_t>(w) << 16);
}
// Weights are 2^kLift exp2(S - m), the factor with them in the sums and in O: it cancels in the quotient, and
// lse takes it back.  fp16 has no normal values below 2^-14 and none below 2^-24, so without it a weight below 2^-25 of the
// largest was lost in O but not in the sum: under one dominant key the share of 32768 others was off by 6% where they
// were e^-16 each, and lost whole from e^-17.5 on.  The stale reference lets weights grow by 2^8, to 2^15 < 65504.
// What is left is 2^-32 of the largest weight for each key, in sum half a step of fp16 at 2^21 keys.
template <bool FP16>
constexpr float kLift = FP16 ? 7.f : 0.f;
template <bool FP16>
constexpr float kUnlift = FP16 ? 0x1p-7f : 1.f;

template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (!FP16) return pack_bf16x2(lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The rare parts are kept out of line: with everything inlined the kernel was 120 KB of code, and its few
// busy warps waited for instructions.

// A wait that did not end at once.  One that runs out ends the call's work in this CTA, with the error
// recorded.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
    const bool done = !*abort && mbar_wait_bounded(bar, parity, kWaitNs);
    if (__all_sync(0xffffffffu, done)) return true;
    if (!*abort) set_device_error(status, SVD_ERR_TIMEOUT);
    *abort = 1;
    return false;
}

// Adds to columns [d0, d1) of a written row what was taken out of V: for every visible node with infinities
// or NaN, its weight times them.  `m` is the reference of the row's weights, `factor` what its sums were
// multiplied by.
template <bool FP16, class Out>
__device__ __noinline__ void add_not_finite(const AttnParams& p, unsigned long long nodes, int b, int hk, size_t qrow, float m,
                                            float factor, Out* to, int d0, int d1) {
    const svd_tree_attention_args& a = p.a;
    const uint16_t* qr = static_cast<const uint16_t*>(a.q) + qrow * a.D;
    for (; nodes; nodes &= nodes - 1) {
        const int i = __ffsll(static_cast<long long>(nodes)) - 1;
        const size_t at = ((static_cast<size_t>(b) * a.n + i) * a.Hkv + hk) * a.D;
        const uint16_t* kr = static_cast<const uint16_t*>(a.k_new) + at;
        const uint16_t* vr = static_cast<const uint16_t*>(a.v_new) + at;
        float dot = 0.f;
#pragma unroll 1
        for (int d = 0; d < a.D; ++d) dot += to_f32<FP16>(qr[d]) * to_f32<FP16>(kr[d]);
        dot = p.qzero ? 0.f : (p.qflip ? -dot : dot);
        // (a weight that underflows is not zero)
        const float w = fmaxf(fast_exp2((dot - m) * p.c + kLift<FP16>) * factor, 1e-30f);
#pragma unroll 1
        for (int d = d0; d < d1; ++d) {
            const float x = to_f32<FP16>(vr[d]);
            if (isfinite(x)) continue;
            if (sizeof(Out) == 4) {
                to[d] = static_cast<Out>(static_cast<float>(to[d]) + w * x);
            } else {
                const float y = to_f32<FP16>(static_cast<uint16_t>(to[d])) + w * x;
                to[d] = static_cast<Out>(pack2<FP16>(y, y) & 0xffffu);
            }
        }
    }
}

// Columns of S that do not count, 32 at `at`, become -inf.
__device__ __noinline__ void hide_columns(uint32_t at, uint32_t keep) {
    uint32_t x[32];
    tmem_ld32(at, x);
    tmem_wait_ld();
    tmem_pin(x);
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = keep >> e & 1u ? x[e] : 0xff800000u;
    tmem_st32(at, x);
    tmem_wait_st();
}

// DP: head size padded to 64 or 128.
template <bool FP16, int DP>
struct Shape {
    static constexpr int kHalves = DP / 64;
    static constexpr int kTileBytes = kTile * DP * 2;
    static constexpr int kStages = DP == 128 ? 3 : 6;   // of the K ring and of the V ring
    static constexpr int kSmem = (1 + 2 * kStages) * kTileBytes + static_cast<int>(sizeof(Control));
    static constexpr int kSoftmaxWarps = 8;
    static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
    static_assert(kStages <= 6 && kSmem <= 232448, "shared memory");
};

template <bool FP16, int DP>
__global__ void __launch_bounds__(Shape<FP16, DP>::kThreads, 1)
tree_attention_kernel(const __grid_constant__ AttnParams p) {
    using Sh = Shape<FP16, DP>;
    constexpr int kHalves = Sh::kHalves, NS = Sh::kStages, kHalfBytes = kTile * 128;
    // swizzled tiles begin at multiples of 1024 bytes; there is no static shared memory in front
    extern __shared__ __align__(1024) uint8_t dyn[];
    if (smem_addr(dyn) & 1023u) {
        if (threadIdx.x == 0) set_device_error(p.status, SVD_ERR_CUDA);
        return;
    }
    uint8_t* sm_q = dyn;
    uint8_t* sm_kv = dyn + Sh::kTileBytes;
    Control& ctl = *reinterpret_cast<Control*>(sm_kv + 2 * NS * Sh::kTileBytes);
    const svd_tree_attention_args& a = p.a;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    constexpr int kLoadK = Sh::kSoftmaxWarps, kMmaS = kLoadK + 1, kMmaO = kLoadK + 2, kLoadV = kLoadK + 3;
    const int part = blockIdx.x / p.NR, rg = blockIdx.x % p.NR;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == kMmaS) {
        if (lane == 0) {
            for (int i = 0; i < 2 * NS; ++i) {
                mbar_init(&ctl.full[i % 2][i / 2], 1);
                mbar_init(&ctl.empty[i % 2][i / 2], 1);
            }
            for (int i = 0; i < 3; ++i) {
                mbar_init(&ctl.s_full[i], 1);
                mbar_init(&ctl.p_full[i], 4);
                mbar_init(&ctl.pv_done[i], 1);
            }
            for (int i = 0; i < 4; ++i) {
                mbar_init(&ctl.m_ready[i][0], 1);
                mbar_init(&ctl.m_ready[i][1], 1);
                mbar_init(&ctl.pair[i], 2);
            }
            mbar_init(&ctl.aux[0], 1);
            mbar_init(&ctl.aux[1], 1);
            mbar_init(&ctl.q_full, 8);
            mbar_init(&ctl.o_free, 8);
            mbar_init(&ctl.drain[0], 1);
            mbar_init(&ctl.drain[1], 1);
            fence_mbar_init();
            ctl.abort = 0;
        }
        tmem_alloc(&ctl.tmem, 512);
    } else if (warp == kLoadK) {
        if (lane == 0) { prefetch_map(&p.ck); prefetch_map(&p.cv); prefetch_map(&p.nk); prefetch_map(&p.nv); }
    } else if (warp == 0) {
        // this CTA's part of the line of tiles, and the sequence in which it begins
        const long long HR = a.Hkv;
        long long total = 0;
        bool bad = false;
        for (int b = lane; b < a.B; b += 32) {
            total += tiles_of(cache_len_of(p, b)) + kItemCost;
            if (blockIdx.x == 0 && a.n_pages > 0) bad = bad || __ldg(a.cache_len + b) != cache_len_of(p, b);
            if (blockIdx.x == 0 && a.n_pages == 0) bad = bad || __ldg(a.cache_len + b) != 0;
        }
        if (bad) set_device_error(p.status, SVD_ERR_PAGE_RANGE);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        total *= HR;
        const long long most = max_parts(p.NR), parts = total < most ? total : most, me = part;
        const long long lo = me < parts ? me * total / parts : 0, hi = me < parts ? (me + 1) * total / parts : 0;
        long long base = 0;
        int b0 = 0;
        for (int bb = 0; bb < a.B; bb += 32) {
            const int b = bb + lane;
            long long w = b < a.B ? (tiles_of(cache_len_of(p, b)) + kItemCost) * HR : 0, x = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const unsigned in = __ballot_sync(0xffffffffu, base + x > lo && b < a.B);
            if (in) {
                const int l = __ffs(in) - 1;
                b0 = bb + l;
                base += __shfl_sync(0xffffffffu, x - w, l);
                break;
            }
            base += __shfl_sync(0xffffffffu, x, 31);
        }
        for (int i = lane; i < kLens; i += 32) ctl.lens[i] = b0 + i < a.B ? cache_len_of(p, b0 + i) : 0;
        if (lane == 0) {
            ctl.lo = lo;
            ctl.hi = hi;
            ctl.total = total;
            ctl.parts = parts;
            ctl.base = base;
            ctl.b = b0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    Walker wk(p, ctl.lo, ctl.hi, ctl.base, ctl.b);
    const Segment& s = wk.s;
    // Whole warps wait; the answer is the same in every lane.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u)) || wait_on(bar, parity & 1u, &ctl.abort, p.status);
    };

    if (warp == kLoadK || warp == kLoadV) {
        // ------------------------------------------------------------------ producer
        // one warp for K, one for V
        const int kv = warp == kLoadV ? 1 : 0;
        const CUtensorMap* const cached = kv ? &p.cv : &p.ck;
        const CUtensorMap* const fresh = kv ? &p.nv : &p.nk;
        uint64_t* const full = ctl.full[kv];
        const bool one = lane == 0;
        uint32_t u = 0;                 // tiles so far
        bool ok = true;
        PartInfo inf = {0, 0, -1};   // the item that starts here and goes on in later parts
        while (ok && wk.next(p, ctl.lens)) {
            if (s.tile0 == 0 && s.tile1 < s.tiles) {
                const long long end = wk.start + kItemCost + s.tiles;   // behind the item
                long long c = (end - 1) * ctl.parts / ctl.total;
                while ((c + 1) * ctl.total / ctl.parts < end) ++c;
                while (c * ctl.total / ctl.parts >= end) --c;
                inf = PartInfo{s.b, s.hk, static_cast<int>(c)};
            }
            const int pages_per_tile = kTile / p.page_rows;
            const int32_t* table = a.page_table + static_cast<size_t>(s.b) * a.max_pages;
            const int ctiles = s.tiles - 1;
            auto page_of = [&](int tile) {   // lane l: page of the tile's rows l * page_rows ..
                const int row = tile * kTile + lane * p.page_rows;
                if (tile >= ctiles || lane >= pages_per_tile || row >= s.len) return -1;
                int pg = __ldg(table + (row >> p.page_shift));
                if (pg < 0 || pg >= a.n_pages) {
                    set_device_error(p.status, SVD_ERR_PAGE_RANGE);
                    pg = 0;
                }
                return pg;
            };
            int pg = page_of(s.tile0);
            for (int tile = s.tile0; tile < s.tile1; ++tile, ++u) {
                const int next_pg = tile + 1 < s.tile1 ? page_of(tile + 1) : -1;
                const uint32_t st = u % NS;
                if (u >= NS) ok = wait(&ctl.empty[kv][st], u / NS - 1);
                if (!ok) break;
                uint8_t* dst = sm_kv + (kv * NS + st) * Sh::kTileBytes;
                if (tile < ctiles) {
                    // box by box in code that the warp runs together: issued lane by lane, the 16 boxes of a tile of
                    // 16-token pages took 1600 cycles
                    const uint32_t box = p.page_rows * 128u;
                    const int boxes = __popc(__ballot_sync(0xffffffffu, pg >= 0));
                    const int row = (tile * kTile) & (a.page_size - 1);   // (0 unless pages are longer than tiles)
                    if (one) mbar_arrive_expect_tx(&full[st], boxes * kHalves * box);
                    __syncwarp();
#pragma unroll 2
                    for (int i = 0; i < boxes; ++i) {
                        const int page = __shfl_sync(0xffffffffu, pg, i);
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
                            tma_load_4d(one, dst + h * kHalfBytes + i * box, cached, h * 64, s.hk, row, page, &full[st]);
                    }
                } else {
                    if (one) mbar_arrive_expect_tx(&full[st], kHalves * p.nb * 128u);
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) tma_load_4d(one, dst + h * kHalfBytes, fresh, h * 64, s.hk, 0, s.b, &full[st]);
                }
                __syncwarp();
                pg = next_pg;
            }
        }
        if (one && kv == 0) p.info[blockIdx.x] = inf;
        // after a wait that ran out: no copy of this CTA may be in flight when it ends
        if (!ok)
            for (uint32_t i = u > NS ? u - NS : 0; i < u; ++i) mbar_wait_bounded(&full[i % NS], (i / NS) & 1u, kWaitNs);
    } else if (warp == kMmaS) {
        // ------------------------------------------------------------------ S = Q K^T
        // Tiles are numbered through the part.  S of a tile is issued as soon as its K, its segment's Q and its
        // slot are there.  (One warp for both products was busy with its own waits for 2300 cycles a tile; the
        // products alone take 1060.)
        constexpr uint32_t kId = mma_desc(FP16, false, kTile, kTile);
        const uint32_t id_new = mma_desc(FP16, false, kTile, p.nb);
        const bool one = lane == 0;
        const uint64_t q_desc = mat_desc(smem_addr(sm_q), 16, 1024);
        uint32_t u = 0, seg = 0;
        bool ok = true;
        while (ok && wk.next(p, ctl.lens)) {
            ok = wait(&ctl.q_full, seg++);
            for (int kt = s.tile0; ok && kt < s.tile1; ++kt, ++u) {
                const uint32_t st = u % NS, slot = u % 3;
                if (u >= 3) ok = wait(&ctl.pv_done[slot], u / 3 - 1);
                ok = ok && wait(&ctl.full[0][st], u / NS);
                if (!ok) break;
                tc_fence_after();
                const uint64_t k_desc = mat_desc(smem_addr(sm_kv + st * Sh::kTileBytes), 16, 1024);
                const uint32_t id = kt == s.tiles - 1 ? id_new : kId;
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
                    const uint32_t off = ((kk / 4) * kHalfBytes + (kk % 4) * 32) >> 4;   // (of the address fields)
                    mma_ss(one, tmem + slot * kTile, q_desc + off, k_desc + off, id, kk > 0);
                }
                mma_commit(one, &ctl.s_full[slot]);
                mma_commit(one, &ctl.empty[0][st]);
                __syncwarp();
            }
        }
        // nothing may be in flight when TMEM is freed
        mma_commit(one, &ctl.drain[0]);
        __syncwarp();
        mbar_wait_bounded(&ctl.drain[0], 0, kWaitNs);
    } else if (warp == kMmaO) {
        // ------------------------------------------------------------------ O += P V
        constexpr uint32_t kId = mma_desc(FP16, true, kTile, DP);
        const bool one = lane == 0;
        uint32_t u = 0, naux = 0, seg = 0;
        bool ok = true;
        for (; ok && wk.next(p, ctl.lens); ++seg) {
            for (int kt = s.tile0; ok && kt < s.tile1; ++kt, ++u) {
                const uint32_t st = u % NS, slot = u % 3;
                uint8_t* v = sm_kv + (NS + st) * Sh::kTileBytes;
                const bool drafted = kt == s.tiles - 1;
                const int valid = drafted ? p.nb : min(kTile, s.len - kt * kTile);
                const int steps = (valid + 15) >> 4;
                ok = wait(&ctl.full[1][st], u / NS);
                // (S of a drafted tile: every warp has left the segment before last, whose note is replaced here)
                if (drafted) ok = ok && wait(&ctl.s_full[slot], u / 3);
                if (!ok) break;
                if (drafted) {
                    // rows of padding nodes become zero; elements that are not finite are taken out
                    // and their nodes noted (rows behind n came as zeros from the TMA unit)
                    const int used = a.n_nodes ? max(0, min(a.n, __ldg(a.n_nodes + s.b))) : a.n;
                    const uint32_t ex = FP16 ? 0x7c00u : 0x7f80u;
                    unsigned long long bad = 0;
#pragma unroll 2
                    for (int i = lane; i < a.n * (DP / 8); i += 32) {
                        const int row = i / (DP / 8), ch = i % (DP / 8);
                        uint4* at = reinterpret_cast<uint4*>(v + (ch >> 3) * kHalfBytes + row * 128 +
                                                             (((ch & 7) ^ (row & 7)) << 4));
                        uint4 x = *at;
                        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
                        bool hit = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool lo = (w[e] & ex) == ex, hi = (w[e] & (ex << 16)) == (ex << 16);
                            w[e] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
                            hit = hit || lo || hi;
                        }
                        if (row >= used) x = make_uint4(0, 0, 0, 0);
                        else if (hit) bad |= 1ull << row;
                        if (hit || row >= used) *at = x;
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
                    if (lane == 0) {
                        ctl.poison[naux & 1u] = bad;
                        mbar_arrive(&ctl.aux[naux & 1u]);
                    }
                    ++naux;
                    fence_async();
                    __syncwarp();
                } else if (valid < steps * 16) {
                    for (int i = lane; i < (steps * 16 - valid) * kHalves * 8; i += 32) {
                        const int row = valid + i / (kHalves * 8), ch = i % (kHalves * 8);
                        *reinterpret_cast<uint4*>(v + (ch >> 3) * kHalfBytes + row * 128 + ((ch & 7) << 4)) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_async();
                    __syncwarp();
                }
                ok = wait(&ctl.p_full[slot], u / 3);
                // (P comes from one warpgroup; the other may still be reading the O of the segment before)
                if (kt == s.tile0 && seg > 0) ok = ok && wait(&ctl.o_free, seg - 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t v_desc = mat_desc(smem_addr(v), kHalfBytes, 1024);
                auto step = [&](int kk) {
                    mma_ts(one, tmem + 3 * kTile, tmem + slot * kTile + kk * 8, v_desc + (kk * 2048 >> 4), kId,
                           kt > s.tile0 || kk > 0);
                };
                if (steps == kTile / 16) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk) step(kk);
                } else {
#pragma unroll 1
                    for (int kk = 0; kk < steps; ++kk) step(kk);
                }
                mma_commit(one, &ctl.pv_done[slot]);
                mma_commit(one, &ctl.empty[1][st]);
                __syncwarp();
            }
        }
        mma_commit(one, &ctl.drain[1]);
        __syncwarp();
        mbar_wait_bounded(&ctl.drain[1], 0, kWaitNs);
    } else {
        // ------------------------------------------------------------------ softmax: thread = row
        // warpgroup wg takes the tiles with number % 2 == wg, and half of O's columns at a segment's end
        const uint32_t wg = warp >> 2;
        const int quarter = warp & 3, trow = quarter * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t o_at = lane_base + 3 * kTile;
        const float c = p.c;
        const int row = rg * kTile + trow;                       // row of the key head: node * G + head
        const bool live = row < p.rows, warp_live = rg * kTile + quarter * 32 < p.rows;
        const int node = live ? row / p.G : 0, g_head = live ? row - node * p.G : 0;
        uint32_t u = 0, naux = 0, phase = 0;                     // tiles, drafted tiles, exchanges so far
        bool ok = true;
        auto q_row = [&](const Segment& g) { return (static_cast<size_t>(g.b) * a.n + node) * a.Hq + g.hk * p.G + g_head; };
        // Q rows of a segment into shared memory (this warpgroup: its half of the columns), completed by q_ready
        auto q_chunk = [&](int i) {
            const int ch = static_cast<int>(wg) * (DP / 16) + i;
            return sm_q + trow * 128 + (ch >> 3) * kHalfBytes + (((ch & 7) ^ (trow & 7)) << 4);
        };
        auto fetch_q = [&](const Segment& g) {
            const uint16_t* src = static_cast<const uint16_t*>(a.q) + q_row(g) * a.D;
#pragma unroll 1
            for (int i = 0; i < DP / 16; ++i) {
                const int ch = static_cast<int>(wg) * (DP / 16) + i;
                // (of zero bytes from global memory the rest is zeros)
                const uint32_t bytes = live && ch * 8 < a.D && !p.qzero ? 16u : 0u;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(q_chunk(i))), "l"(src + (bytes ? ch * 8 : 0)),
                             "r"(bytes)
                             : "memory");
            }
        };
        auto q_ready = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (p.qflip) {
#pragma unroll 1
                for (int i = 0; i < DP / 16; ++i) {
                    uint4* at = reinterpret_cast<uint4*>(q_chunk(i));
                    uint4 x = *at;
                    x.x ^= 0x80008000u; x.y ^= 0x80008000u; x.z ^= 0x80008000u; x.w ^= 0x80008000u;
                    *at = x;
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.q_full);
        };
        // `wk` is at the segment behind the current one
        bool more = wk.next(p, ctl.lens);
        if (more) {
            fetch_q(wk.s);
            q_ready();
        }
        int seq = -1, anc_seq = -1, used = a.n;   // sequences that `used` and `anc` belong to
        unsigned long long anc = 0;
        while (ok && more) {
            const Segment s = wk.s;
            more = wk.next(p, ctl.lens);
            if (a.n_nodes && s.b != seq) used = max(0, min(a.n, __ldg(a.n_nodes + s.b)));
            seq = s.b;
            // ancestors of this row's node, by shuffles of the sequence's parents
            const bool has_new = s.tile1 == s.tiles;
            if (has_new && warp_live && s.b != anc_seq) {
                const size_t at = static_cast<size_t>(s.b) * a.n;
                const int p0 = lane < used ? checked_parent(a.parent, at, lane, p.status) : -1;
                const int p1 = lane + 32 < used ? checked_parent(a.parent, at, lane + 32, p.status) : -1;
                int i = live && node < used ? node : -1;
                anc = 0;
                while (__any_sync(0xffffffffu, i >= 0)) {
                    if (i >= 0) anc |= 1ull << i;
                    const int q0 = __shfl_sync(0xffffffffu, p0, i & 31), q1 = __shfl_sync(0xffffffffu, p1, i & 31);
                    i = i < 0 ? -1 : (i < 32 ? q0 : q1);
                }
                anc_seq = s.b;
            }
            // m: the reference that this thread's l is relative to
            float m = -INFINITY, l = 0.f;
            const uint32_t u_end = u + static_cast<uint32_t>(s.tile1 - s.tile0);
            for (int kt = s.tile0; ok && kt < s.tile1; ++kt, ++u) {
                // A segment's last S is waited for by both warpgroups: Q is free for the next segment, and the wait on
                // pv_done[slot] below cannot pass on the phase before last (S of this tile was issued behind
                // the product of the tile that had the slot before).
                const bool last = kt + 1 == s.tile1, mine = (u & 1u) == wg;
                const uint32_t slot = u % 3;
                if (mine || last) ok = wait(&ctl.s_full[slot], u / 3);
                if (!ok) break;
                if (last && more) fetch_q(wk.s);
                if (mine && warp_live) {
                    tc_fence_after();
                    const uint32_t s_at = lane_base + slot * kTile;
                    // Chunks of 32 columns, two in each round of a loop that is kept short: with the tile
                    // unrolled the warps waited for instructions (2.9 of 8 stalled cycles an issue).
                    const bool drafted = kt == s.tiles - 1;
                    const int rounds = drafted ? 1 : 2, valid = s.len - kt * kTile;
                    if (drafted || valid < kTile) {
#pragma unroll 1
                        for (int q = 0; q < 2 * rounds; ++q) {
                            const int left = valid - 32 * q;
                            hide_columns(s_at + q * 32, drafted ? static_cast<uint32_t>(anc >> (32 * q))
                                                                : (left >= 32 ? ~0u : (left <= 0 ? 0u : (1u << left) - 1u)));
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    uint32_t x[2][32];
#pragma unroll 1
                    for (int q = 0; q < rounds; ++q) {
                        tmem_ld32(s_at + q * 64, x[0]);
                        tmem_ld32(s_at + q * 64 + 32, x[1]);
                        tmem_wait_ld();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            tmem_pin(x[h]);
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mx[k] = fmax3(mx[k], __uint_as_float(x[h][e + 2 * k]), __uint_as_float(x[h][e + 2 * k + 1]));
                        }
                    }
                    const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    // the first chunk comes back while the reference is settled
                    tmem_ld32(s_at, x[0]);
                    float mn = mt;
                    if (kt > s.tile0) {
                        const uint32_t prev = u - 1;
                        ok = wait(&ctl.m_ready[quarter][prev & 1u], prev >> 1);
                        const float mp = *const_cast<volatile float*>(&ctl.ref[prev & 1u][trow]);
                        const bool up = !(mt <= mp + p.thr);
                        mn = up ? fmaxf(mp, mt) : mp;
                        if (__any_sync(0xffffffffu, up)) {
                            // every product into O so far has to be complete
                            ok = ok && wait(&ctl.pv_done[prev % 3], prev / 3);
                            if (!ok) break;
                            tc_fence_after();
                            const float f = up ? fast_exp2((mp - mn) * c) : 1.f;
#pragma unroll 1
                            for (int q = 0; q < DP / 32; ++q) {
                                uint32_t o[32];
                                tmem_ld32(o_at + q * 32, o);
                                tmem_wait_ld();
                                tmem_pin(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st32(o_at + q * 32, o);
                            }
                        }
                    }
                    ctl.ref[wg][trow] = mn;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.m_ready[quarter][wg]);
                    if (__any_sync(0xffffffffu, m != mn)) l *= m == mn ? 1.f : fast_exp2((m - mn) * c);
                    m = mn;
                    const float mref = m == -INFINITY ? 0.f : kLift<FP16> - m * c;
                    const float2 c2 = make_float2(c, c), m2 = make_float2(mref, mref);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                    for (int q = 0; q < rounds; ++q) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            tmem_wait_ld();
                            tmem_pin(x[h]);
                            // the next chunk's load; P goes over columns that have been read
                            if (h == 0 || q + 1 < rounds) tmem_ld32(s_at + (2 * q + h + 1) * 32, x[h ^ 1]);
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float2 z = fma2(make_float2(__uint_as_float(x[h][2 * e]), __uint_as_float(x[h][2 * e + 1])), c2, m2);
                                z.x = fast_exp2(z.x);
                                z.y = fast_exp2(z.y);
                                sum[e & 1] = add2(sum[e & 1], z);
                                w[e] = pack2<FP16>(z.x, z.y);
                            }
                            tmem_st16(s_at + (2 * q + h) * 16, w);
                        }
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tmem_wait_st();
                    tc_fence_before();
                    if (!ok) break;
                }
                __syncwarp();
                if (mine && lane == 0) mbar_arrive(&ctl.p_full[slot]);
                if (last && more) q_ready();
            }
            if (!ok) break;
            // ---- the segment's end: this warpgroup's columns of O, normalised or as a part
            const uint32_t prev = u_end - 1;
            ok = wait(&ctl.pv_done[prev % 3], prev / 3);
            if (has_new) ok = ok && wait(&ctl.aux[naux & 1u], naux >> 1);
            if (!ok) break;
            tc_fence_after();
            const unsigned long long poison = has_new ? *const_cast<volatile unsigned long long*>(&ctl.poison[naux & 1u]) & anc : 0ull;
            if (has_new) ++naux;
            if (warp_live) {
                // both warpgroups' sums, relative to the last tile's reference
                ok = wait(&ctl.m_ready[quarter][prev & 1u], prev >> 1);
                const float mf = *const_cast<volatile float*>(&ctl.ref[prev & 1u][trow]);
                if (l != 0.f && m != mf) l *= fast_exp2((m - mf) * c);
                m = mf;
                ctl.sum[wg][trow] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.pair[quarter]);
                ok = wait(&ctl.pair[quarter], phase++) && ok;
                // (in this order in both warpgroups)
                l = *const_cast<volatile float*>(&ctl.sum[0][trow]) + *const_cast<volatile float*>(&ctl.sum[1][trow]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.pair[quarter]);   // read: may be overwritten
                ok = wait(&ctl.pair[quarter], phase++) && ok;
                if (!ok) break;
                const size_t qrow = q_row(s);
                const bool whole = s.tile0 == 0 && s.tile1 == s.tiles;
                const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (s.tile0 == 0 ? 1 : 0)) * p.used + trow;
                const bool pad = node >= used;
                const float inv = pad || l == 0.f ? 0.f : __fdiv_rn(1.f, l);
                float* to_part = p.o + slot * a.D;
                uint16_t* out = static_cast<uint16_t*>(a.out) + qrow * a.D;
#pragma unroll 1
                for (int q = 0; q < DP / 64; ++q) {
                    const int d0 = static_cast<int>(wg) * (DP / 2) + q * 32;
                    uint32_t o[32];
                    tmem_ld32(o_at + d0, o);
                    tmem_wait_ld();
                    tmem_pin(o);
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        const int d = d0 + e;
                        if (!live || d >= a.D) continue;
                        float y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = __uint_as_float(o[e + k]);
                        if (whole) {
                            uint4 v;
                            v.x = pad ? 0u : pack2<FP16>(y[0] * inv, y[1] * inv);
                            v.y = pad ? 0u : pack2<FP16>(y[2] * inv, y[3] * inv);
                            v.z = pad ? 0u : pack2<FP16>(y[4] * inv, y[5] * inv);
                            v.w = pad ? 0u : pack2<FP16>(y[6] * inv, y[7] * inv);
                            *reinterpret_cast<uint4*>(out + d) = v;
                        } else {
                            *reinterpret_cast<float4*>(to_part + d) = make_float4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<float4*>(to_part + d + 4) = make_float4(y[4], y[5], y[6], y[7]);
                        }
                    }
                    __syncwarp();
                }
                if (live && poison) {
                    const int d0 = static_cast<int>(wg) * (DP / 2), d1 = min(a.D, d0 + DP / 2);
                    if (whole) add_not_finite<FP16>(p, poison, s.b, s.hk, qrow, m, inv, out, d0, d1);
                    else add_not_finite<FP16>(p, poison, s.b, s.hk, qrow, m, 1.f, to_part, d0, d1);
                }
                __syncwarp();
                if (live && wg == 0) {
                    if (!whole) p.ml[slot] = make_float2(m, l);
                    else if (a.lse) a.lse[qrow] = pad ? -INFINITY : (m == -INFINITY ? 0.f : m * c * kLn2) + logf(l * kUnlift<FP16>);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.o_free);
        }
        // (a wait that ran out may have left some in flight)
        asm volatile("cp.async.wait_all;" ::: "memory");
        tmem_wait_ld();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaS) tmem_free(tmem, 512);
}

// What a part's sum and O are multiplied by for the row's maximum m; a part that saw nothing has the maximum -inf, the
// sum 0 and O = 0.
__device__ __forceinline__ float join_factor(const float2& ml, float m, float c) {
    return ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : fast_exp2((ml.x - m) * c);
}

// The sum over a row's parts once more, where it came out as NaN: an infinity of a visible node stays one where its part
// lies so far below the maximum that its factor is zero.  (Out of line and for such rows alone: with the choice
// in the loop a decode step took 16.2 us instead of 14.4.)
__device__ __noinline__ float4 join_not_finite(const AttnParams& p, size_t first, size_t second, size_t step, int parts, float m, int d) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i = 0; i < parts; ++i) {
        const size_t slot = i == 0 ? first : second + (i - 1) * step;
        const float f = join_factor(p.ml[slot], m, p.c);
        const float4 o = *reinterpret_cast<const float4*>(p.o + slot * p.a.D + d);
        acc.x += isinf(o.x) ? o.x : o.x * f;
        acc.y += isinf(o.y) ? o.y : o.y * f;
        acc.z += isinf(o.z) ? o.z : o.z * f;
        acc.w += isinf(o.w) ? o.w : o.w * f;
    }
    return acc;
}

// Joins the parts of the item that starts in part blockIdx.x and goes on: one warp per row, the parts
// in order, relative to the row's largest maximum.
template <bool FP16>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const __grid_constant__ AttnParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const svd_tree_attention_args& a = p.a;
    const PartInfo inf = p.info[blockIdx.x];
    if (inf.last < 0) return;
    const int lane = threadIdx.x & 31, rg = blockIdx.x % p.NR;
    const int in_group = blockIdx.y * kCombineWarps + (threadIdx.x >> 5);
    const int row = rg * kTile + in_group;
    if (in_group >= p.used || row >= p.rows) return;
    const int parts = inf.last - static_cast<int>(blockIdx.x) / p.NR + 1;
    auto slot = [&](int i) {
        return (2 * (static_cast<size_t>(blockIdx.x) + static_cast<size_t>(i) * p.NR) + (i == 0 ? 1 : 0)) * p.used + in_group;
    };
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool act = lane * 4 < a.D;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float2 ml = p.ml[slot(i)];
        const float f = join_factor(ml, m, p.c);
        l += ml.y * f;
        if (act) {
            const float4 o = *reinterpret_cast<const float4*>(p.o + slot(i) * a.D + lane * 4);
            acc.x += o.x * f; acc.y += o.y * f; acc.z += o.z * f; acc.w += o.w * f;
        }
    }
    if (act && (isnan(acc.x) || isnan(acc.y) || isnan(acc.z) || isnan(acc.w)))
        acc = join_not_finite(p, slot(0), slot(1), 2 * static_cast<size_t>(p.NR) * p.used, parts, m, lane * 4);
    const int node = row / p.G, head = inf.hk * p.G + row - node * p.G;
    const bool pad = a.n_nodes && node >= __ldg(a.n_nodes + inf.b);
    const float inv = pad || l == 0.f ? 0.f : __fdiv_rn(1.f, l);
    const size_t qrow = (static_cast<size_t>(inf.b) * a.n + node) * a.Hq + head;
    if (act) {
        uint2 w = make_uint2(pack2<FP16>(acc.x * inv, acc.y * inv), pack2<FP16>(acc.z * inv, acc.w * inv));
        if (pad) w = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + qrow * a.D + lane * 4) = w;
    }
    if (a.lse && lane == 0) a.lse[qrow] = pad ? -INFINITY : (m == -INFINITY ? 0.f : m * p.c * kLn2) + logf(l * kUnlift<FP16>);
}

// The driver's encoder, reached through the runtime so that the library does not link the driver.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// [outer][rows][Hkv][D] with boxes of `box_rows` rows of one head, 64 elements (128 bytes) wide.
// Elements behind D, and rows behind `rows`, arrive as zeros.
bool encode(CUtensorMap* map, bool fp16, const void* base, int D, int Hkv, int rows, int outer, int64_t outer_stride,
            int box_rows) {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(D) * Hkv * 2,
                                   static_cast<cuuint64_t>(outer_stride) * 2};
    const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(box_rows), 1}, step[4] = {1, 1, 1, 1};
    return encoder()(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
                     dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP16, int DP>
cudaError_t launch(const AttnParams& p, cudaStream_t st) {
    using Sh = Shape<FP16, DP>;
    cudaError_t e = cudaFuncSetAttribute(tree_attention_kernel<FP16, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = p.NR * max_parts(p.NR);
    tree_attention_kernel<FP16, DP><<<ctas, Sh::kThreads, Sh::kSmem, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(ctas, (p.used + kCombineWarps - 1) / kCombineWarps);
    cfg.blockDim = dim3(kCombineWarps * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_combine_kernel<FP16>, p);
}

template <bool FP16>
cudaError_t launch_type(const AttnParams& p, cudaStream_t st) {
    return p.a.D > 64 ? launch<FP16, 128>(p, st) : launch<FP16, 64>(p, st);
}

}  // namespace

size_t tree_attention_ws_bytes(int, int n, int Hq, int Hkv, int D) { return attn_ws(n * (Hq / Hkv), D).total; }

int launch_tree_attention(const svd_tree_attention_args& a, void* ws, void* stream) {
    AttnParams p;
    std::memset(&p, 0, sizeof p);
    p.a = a;
    p.G = a.Hq / a.Hkv;
    p.rows = a.n * p.G;
    p.used = p.rows < kTile ? p.rows : kTile;
    p.NR = row_groups(p.rows);
    p.page_rows = a.page_size < kTile ? a.page_size : kTile;
    while ((1 << p.page_shift) < a.page_size) ++p.page_shift;
    p.nb = (a.n + 15) / 16 * 16;
    p.qzero = a.scale == 0.f;
    p.qflip = a.scale < 0.f;
    p.c = p.qzero ? 1.f : fabsf(a.scale) * kLog2e;
    p.thr = 8.f / p.c;
    const AttnWs L = attn_ws(p.rows, a.D);
    char* base = static_cast<char*>(ws);
    p.status = reinterpret_cast<uint32_t*>(base);
    p.info = reinterpret_cast<PartInfo*>(base + L.info);
    p.ml = reinterpret_cast<float2*>(base + L.ml);
    p.o = reinterpret_cast<float*>(base + L.o);
    const bool fp16 = a.dtype == SVD_FP16;
    if (!encoder()) return static_cast<int>(cudaErrorNotSupported);
    const int64_t page = static_cast<int64_t>(a.page_size) * a.Hkv * a.D, tree = static_cast<int64_t>(a.n) * a.Hkv * a.D;
    bool ok = encode(&p.nk, fp16, a.k_new, a.D, a.Hkv, a.n, a.B, tree, p.nb) &&
              encode(&p.nv, fp16, a.v_new, a.D, a.Hkv, a.n, a.B, tree, p.nb);
    p.ck = p.nk;   // an empty cache is never read
    p.cv = p.nv;
    if (a.n_pages > 0 && a.max_pages > 0)
        ok = ok &&
             encode(&p.ck, fp16, a.cache_k, a.D, a.Hkv, a.page_size, a.n_pages, a.n_pages > 1 ? a.page_stride_k : page, p.page_rows) &&
             encode(&p.cv, fp16, a.cache_v, a.D, a.Hkv, a.page_size, a.n_pages, a.n_pages > 1 ? a.page_stride_v : page, p.page_rows);
    if (!ok) return static_cast<int>(cudaErrorInvalidValue);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return static_cast<int>(fp16 ? launch_type<true>(p, st) : launch_type<false>(p, st));
}

}  // namespace svd
