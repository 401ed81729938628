// tree_attention.cu -- attention of the nodes of a tree of drafts over a paged cache and over each
// other (include/svd_tree.h).
//
// What bounds it: every cached key and value is read once (2 x 2 bytes x D per key head and token)
// and serves the n * Hq / Hkv query rows of its head.  Up to about 128 rows that is less than the
// tensor cores' rate over HBM's, so the kernel streams the cache through shared memory and does all
// arithmetic behind it.
//
// Work.  An item is one sequence, key head and group of up to R * 128 query rows (a row is a node
// and a query head; R = 1 or 2 row tiles); its keys are tiles of 128: the cached ones, then one tile of
// the drafted nodes.  All tiles of all items form one line that is cut into equal parts, one per CTA
// (148, one per SM), so ragged lengths balance by themselves and one long sequence spreads over the
// whole GPU.  A part that holds a whole item writes its result; otherwise it leaves the unnormalised
// sum with the row maxima and sums in the workspace, and a second kernel (a programmatic dependent,
// its launch hidden) joins the parts in a fixed order.
//
// Roles in a CTA.  A producer warp loads K and V tiles page by page by TMA (128-byte swizzle) into a
// ring; one warp issues tcgen05.mma: S = Q K^T into TMEM, O += P V with P read from TMEM; one
// softmax warpgroup per row tile: thread = row, so maxima and sums need no exchange.  It reads S,
// keeps a running maximum that moves only when a tile exceeds it by more than 2^8 (the sum and O
// share the stale reference, so the quotient is exact all the same, and O in TMEM is rescaled
// rarely), and writes P = exp2(S - m) over S in the tensors' type (that rounding, at most half a step of
// the type per weight, is what the matrix instruction takes; maxima and sums stay fp32).  With one row
// tile S is double buffered, so the next tile's S forms while this tile's softmax runs; with two,
// the row tiles alternate.
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

constexpr int kCtas = 148;         // parts of the line of tiles: one per SM of a B200
constexpr int kTile = 128;         // keys per tile, rows per row tile
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kCombineWarps = 8;

struct PartInfo {                  // what the combine kernel needs to know of the item that starts in a
    int b, hk, rg, last;           // part and does not end there: last part it reaches, or -1
};

struct AttnWs {
    size_t info, ml, o, total;
};
__host__ __device__ inline int row_tiles(int rows) { return rows > kTile ? 2 : 1; }
inline AttnWs attn_ws(int rows, int D) {
    const int used = rows < row_tiles(rows) * kTile ? rows : row_tiles(rows) * kTile;
    AttnWs L;
    L.info = sizeof(WsHeader);
    L.ml = align256(L.info + sizeof(PartInfo) * kCtas);
    L.o = align256(L.ml + sizeof(float2) * 2 * kCtas * static_cast<size_t>(used));
    L.total = align256(L.o + sizeof(float) * 2 * kCtas * static_cast<size_t>(used) * static_cast<size_t>(D));
    return L;
}

struct alignas(64) AttnParams {
    CUtensorMap ck, cv, nk, nv;    // cache and drafted nodes
    svd_tree_attention_args a;
    int G, rows, used, NR;         // heads per key head, rows per item line, rows kept per slot, row groups
    int page_rows, page_shift;     // rows per TMA box, log2(page_size)
    int nb;                        // columns of the drafted tile, a multiple of 16
    float c, thr;                  // |scale| log2(e); 8 / c
    int qflip, qzero;              // the sign of the scale goes to Q; a scale of 0 zeroes Q
    uint32_t* status;
    PartInfo* info;
    float2* ml;                    // [2 kCtas][used]: running maximum (raw scores), sum
    float* o;                      // [2 kCtas][used][D]
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
    int b, hk, rg, len;
    int tile0, tile1, tiles;
};
struct Walker {
    long long pos, hi, base;
    int b;
    __device__ bool next(const AttnParams& p, Segment& s) {
        if (pos >= hi) return false;
        while (true) {
            s.len = cache_len_of(p, b);
            s.tiles = tiles_of(s.len);
            const long long w = static_cast<long long>(s.tiles) * p.a.Hkv * p.NR;
            if (pos < base + w) break;
            base += w;
            ++b;
        }
        const long long r = pos - base;
        const int it = static_cast<int>(r / s.tiles);
        s.b = b;
        s.hk = it / p.NR;
        s.rg = it - s.hk * p.NR;
        s.tile0 = static_cast<int>(r - static_cast<long long>(it) * s.tiles);
        const long long left = hi - pos;
        s.tile1 = s.tiles - s.tile0 <= left ? s.tiles : s.tile0 + static_cast<int>(left);
        pos += s.tile1 - s.tile0;
        return true;
    }
};

struct Control {
    uint64_t full[16], empty[16];
    uint64_t s_full[2], p_full[2], pv_done[2], q_full[2], aux, drain;
    long long lo, hi, base, total, parts;
    unsigned long long poison;     // drafted nodes with a V element that is not finite
    int b;
    uint32_t tmem;
    int abort;
};

template <bool FP16>
__device__ __forceinline__ float to_f32(uint16_t w) {
    return FP16 ? __half2float(__ushort_as_half(w)) : __uint_as_float(static_cast<uint32_t>(w) << 16);
}
template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (!FP16) return pack_bf16x2(lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// DP: head size padded to 64 or 128; R: row tiles per item; NS: stages of the ring (a K or a V tile each).
template <bool FP16, int DP, int R>
struct Shape {
    static constexpr int kHalves = DP / 64;
    static constexpr int kTileBytes = kTile * DP * 2;
    static constexpr int kStages = R == 1 ? (DP == 128 ? 6 : 12) : (DP == 128 ? 5 : 10);
    static constexpr int kSmem = R * kTileBytes + kStages * kTileBytes + 1024 + static_cast<int>(sizeof(Control));
    static constexpr int kSoftmaxWarps = 4 * R;
    static constexpr int kThreads = 32 * (kSoftmaxWarps + 2);
    static_assert(kStages <= 16 && kSmem <= 232448, "shared memory");
};

template <bool FP16, int DP, int R>
__global__ void __launch_bounds__(Shape<FP16, DP, R>::kThreads, 1)
tree_attention_kernel(const __grid_constant__ AttnParams p) {
    using Sh = Shape<FP16, DP, R>;
    constexpr int kHalves = Sh::kHalves, NS = Sh::kStages, kHalfBytes = kTile * 128;
    extern __shared__ uint8_t dyn[];
    uint8_t* sm = dyn + ((1024u - (smem_addr(dyn) & 1023u)) & 1023u);
    uint8_t* sm_q = sm;
    uint8_t* sm_kv = sm + R * Sh::kTileBytes;
    Control& ctl = *reinterpret_cast<Control*>(sm_kv + NS * Sh::kTileBytes);
    const svd_tree_attention_args& a = p.a;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    constexpr int kProducer = Sh::kSoftmaxWarps, kMma = Sh::kSoftmaxWarps + 1;
    volatile int* abort = &ctl.abort;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == kMma) {
        if (lane == 0) {
            for (int i = 0; i < NS; ++i) { mbar_init(&ctl.full[i], 1); mbar_init(&ctl.empty[i], 1); }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&ctl.s_full[i], 1);
                mbar_init(&ctl.p_full[i], 4);
                mbar_init(&ctl.pv_done[i], 1);
                mbar_init(&ctl.q_full[i], 4);
            }
            mbar_init(&ctl.aux, 1);
            mbar_init(&ctl.drain, 1);
            fence_mbar_init();
            ctl.abort = 0;
            ctl.poison = 0;
        }
        tmem_alloc(&ctl.tmem, 512);
    } else if (warp == kProducer) {
        if (lane == 0) { prefetch_map(&p.ck); prefetch_map(&p.cv); prefetch_map(&p.nk); prefetch_map(&p.nv); }
    } else if (warp == 0) {
        // this CTA's part of the line of tiles, and the sequence in which it begins
        const long long HR = static_cast<long long>(a.Hkv) * p.NR;
        long long total = 0;
        bool bad = false;
        for (int b = lane; b < a.B; b += 32) {
            total += tiles_of(cache_len_of(p, b));
            if (blockIdx.x == 0 && a.n_pages > 0) bad = bad || __ldg(a.cache_len + b) != cache_len_of(p, b);
            if (blockIdx.x == 0 && a.n_pages == 0) bad = bad || __ldg(a.cache_len + b) != 0;
        }
        if (bad) set_device_error(p.status, SVD_ERR_PAGE_RANGE);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        total *= HR;
        const long long parts = total < static_cast<long long>(gridDim.x) ? total : gridDim.x;
        const long long me = blockIdx.x;
        const long long lo = me < parts ? me * total / parts : 0, hi = me < parts ? (me + 1) * total / parts : 0;
        long long base = 0;
        int b0 = 0;
        for (int bb = 0; bb < a.B; bb += 32) {
            const int b = bb + lane;
            long long w = b < a.B ? tiles_of(cache_len_of(p, b)) * HR : 0, x = w;
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
    Walker wk = {ctl.lo, ctl.hi, ctl.base, ctl.b};
    Segment s;
    // Whole warps wait; the answer is the same in every lane.  A wait that runs out ends the call's
    // work in this CTA with the error recorded.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool done = !*abort && mbar_wait_bounded(bar, parity & 1u, kWaitNs);
        if (__all_sync(0xffffffffu, done)) return true;
        if (!*abort) set_device_error(p.status, SVD_ERR_TIMEOUT);
        *abort = 1;
        return false;
    };

    if (warp == kProducer) {
        // ------------------------------------------------------------------ producer
        uint32_t cnt = 0;   // tiles put into the ring
        bool ok = true;
        PartInfo inf = {0, 0, 0, -1};   // the item that starts here and goes on in later parts
        while (ok && wk.next(p, s)) {
            if (s.tile0 == 0 && s.tile1 < s.tiles) {
                const long long end = wk.pos + (s.tiles - s.tile1);   // first tile behind the item
                long long c = (end - 1) * ctl.parts / ctl.total;
                while ((c + 1) * ctl.total / ctl.parts < end) ++c;
                while (c * ctl.total / ctl.parts >= end) --c;
                inf = PartInfo{s.b, s.hk, s.rg, static_cast<int>(c)};
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
            for (int tile = s.tile0; ok && tile < s.tile1; ++tile) {
                const int next_pg = tile + 1 < s.tile1 ? page_of(tile + 1) : -1;
                const int boxes = __popc(__ballot_sync(0xffffffffu, pg >= 0));
                for (int kv = 0; kv < 2; ++kv, ++cnt) {
                    const int st = cnt % NS;
                    if (cnt >= NS) ok = wait(&ctl.empty[st], cnt / NS - 1);
                    if (!ok) break;
                    uint8_t* dst = sm_kv + st * Sh::kTileBytes;
                    if (tile < ctiles) {
                        const uint32_t box = p.page_rows * 128u;
                        if (lane == 0) mbar_arrive_expect_tx(&ctl.full[st], boxes * kHalves * box);
                        __syncwarp();
                        if (pg >= 0) {
                            const int row = (tile * kTile + lane * p.page_rows) & (a.page_size - 1);
#pragma unroll
                            for (int h = 0; h < kHalves; ++h)
                                tma_load_4d(dst + h * kHalfBytes + lane * box, kv ? &p.cv : &p.ck, h * 64, s.hk, row, pg,
                                            &ctl.full[st]);
                        }
                    } else if (lane == 0) {
                        mbar_arrive_expect_tx(&ctl.full[st], kHalves * p.nb * 128u);
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
                            tma_load_4d(dst + h * kHalfBytes, kv ? &p.nv : &p.nk, h * 64, s.hk, 0, s.b, &ctl.full[st]);
                    }
                    __syncwarp();
                }
                pg = next_pg;
            }
        }
        if (lane == 0) p.info[blockIdx.x] = inf;
        // after a wait that ran out: no copy of this CTA may be in flight when it ends
        if (*abort)
            for (uint32_t i = cnt > NS ? cnt - NS : 0; i < cnt; ++i)
                mbar_wait_bounded(&ctl.full[i % NS], (i / NS) & 1u, kWaitNs);
    } else if (warp == kMma) {
        // ------------------------------------------------------------------ matrix instructions
        constexpr uint32_t kIdS = mma_desc(FP16, false, kTile, kTile), kIdO = mma_desc(FP16, true, kTile, DP);
        const uint32_t id_new = mma_desc(FP16, false, kTile, p.nb);
        uint32_t tg = 0, unit = 0, seg = 0, naux = 0;   // tiles, units (tile x row tile), segments so far
        bool ok = true;
        while (ok && wk.next(p, s)) {
            const int nt = s.tile1 - s.tile0, nu = nt * R;
            const uint32_t u0 = unit, t0 = tg;
            auto issue_s = [&](uint32_t u) {   // u: unit within the segment
                const uint32_t slot = (u0 + u) & 1u, r = R == 2 ? (u & 1u) : 0u, tile = u / R;
                const uint32_t cnt = 2 * (t0 + tile), st = cnt % NS;
                if (u0 + u >= 2) ok = ok && wait(&ctl.pv_done[slot], (u0 + u - 2) >> 1);
                if (r == 0) ok = ok && wait(&ctl.full[st], cnt / NS);
                if (tile == 0) ok = ok && wait(&ctl.q_full[r], seg);
                if (!ok) return;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t q = smem_addr(sm_q + r * Sh::kTileBytes), k = smem_addr(sm_kv + st * Sh::kTileBytes);
                    const uint32_t id = s.tile0 + static_cast<int>(tile) == s.tiles - 1 ? id_new : kIdS;
#pragma unroll
                    for (int kk = 0; kk < DP / 16; ++kk) {
                        const uint32_t off = (kk / 4) * kHalfBytes + (kk % 4) * 32;
                        mma_ss(tmem + slot * kTile, mat_desc(q + off, 16, 1024), mat_desc(k + off, 16, 1024), id, kk > 0);
                    }
                    mma_commit(&ctl.s_full[slot]);
                    if (r == R - 1) mma_commit(&ctl.empty[st]);
                }
                __syncwarp();
            };
            issue_s(0);
            for (uint32_t u = 0; ok && u < static_cast<uint32_t>(nu); ++u) {
                if (u + 1 < static_cast<uint32_t>(nu)) issue_s(u + 1);
                if (!ok) break;
                const uint32_t slot = (u0 + u) & 1u, r = R == 2 ? (u & 1u) : 0u, tile = u / R;
                const uint32_t cnt = 2 * (t0 + tile) + 1, st = cnt % NS;
                uint8_t* v = sm_kv + st * Sh::kTileBytes;
                const int kt = s.tile0 + static_cast<int>(tile);
                const bool drafted = kt == s.tiles - 1;
                const int valid = drafted ? p.nb : min(kTile, s.len - kt * kTile);
                const int steps = (valid + 15) >> 4;
                if (r == 0) {
                    ok = wait(&ctl.full[st], cnt / NS);
                    if (!ok) break;
                    if (drafted) {
                        // rows of padding nodes become zero; elements that are not finite are taken out
                        // and their nodes noted (rows behind n came as zeros from the TMA unit)
                        const int used = a.n_nodes ? max(0, min(a.n, __ldg(a.n_nodes + s.b))) : a.n;
                        const uint32_t ex = FP16 ? 0x7c00u : 0x7f80u;
                        unsigned long long bad = 0;
                        for (int i = lane; i < a.n * (DP / 8); i += 32) {
                            const int row = i / (DP / 8), ch = i % (DP / 8);
                            uint4* at = reinterpret_cast<uint4*>(v + (ch >> 3) * kHalfBytes + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
                            if (row >= used) {
                                *at = make_uint4(0, 0, 0, 0);
                                continue;
                            }
                            uint4 x = *at;
                            uint32_t* w = reinterpret_cast<uint32_t*>(&x);
                            bool hit = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((w[e] & ex) == ex) { w[e] &= 0xffff0000u; hit = true; }
                                if ((w[e] & (ex << 16)) == (ex << 16)) { w[e] &= 0x0000ffffu; hit = true; }
                            }
                            if (hit) {
                                *at = x;
                                bad |= 1ull << row;
                            }
                        }
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
                        if (lane == 0) {
                            ctl.poison = bad;
                            mbar_arrive(&ctl.aux);
                        }
                        ++naux;
                        fence_async();
                        __syncwarp();
                    } else if (valid < steps * 16) {
                        for (int i = lane; i < (steps * 16 - valid) * kHalves * 8; i += 32) {
                            const int row = valid + i / (kHalves * 8), ch = i % (kHalves * 8);
                            *reinterpret_cast<uint4*>(v + (ch >> 3) * kHalfBytes + row * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
                        }
                        fence_async();
                        __syncwarp();
                    }
                }
                ok = wait(&ctl.p_full[slot], (u0 + u) >> 1);
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t vb = smem_addr(v);
                    for (int kk = 0; kk < steps; ++kk)
                        mma_ts(tmem + 256 + r * DP, tmem + slot * kTile + kk * 8, mat_desc(vb + kk * 2048, kHalfBytes, 1024), kIdO,
                               tile > 0 || kk > 0);
                    mma_commit(&ctl.pv_done[slot]);
                    if (r == R - 1) mma_commit(&ctl.empty[st]);
                }
                __syncwarp();
            }
            unit += nu;
            tg += nt;
            ++seg;
        }
        // nothing may be in flight when TMEM is freed
        if (lane == 0) mma_commit(&ctl.drain);
        mbar_wait_bounded(&ctl.drain, 0, kWaitNs);
        (void)naux;
    } else {
        // ------------------------------------------------------------------ softmax: thread = row
        const int rt = warp >> 2, trow = (warp & 3) * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t o_at = lane_base + 256 + rt * DP;
        const float c = p.c;
        uint32_t unit = rt, seg = 0, naux = 0;
        bool ok = true;
        while (ok && wk.next(p, s)) {
            const int in_item = rt * kTile + trow;                   // row within the item
            const int row = s.rg * R * kTile + in_item;              // row of the key head: node * G + head
            const bool live = row < p.rows;
            const bool warp_live = s.rg * R * kTile + rt * kTile + (warp & 3) * 32 < p.rows;
            const int node = live ? row / p.G : 0;
            const int head = s.hk * p.G + (live ? row - node * p.G : 0);
            const int used = a.n_nodes ? max(0, min(a.n, __ldg(a.n_nodes + s.b))) : a.n;
            const size_t qrow = (static_cast<size_t>(s.b) * a.n + node) * a.Hq + head;
            if (warp_live) {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + qrow * a.D);
                uint8_t* dst = sm_q + rt * Sh::kTileBytes + trow * 128;
                uint4 x[DP / 8];
#pragma unroll
                for (int ch = 0; ch < DP / 8; ++ch)
                    x[ch] = live && ch * 8 < a.D && !p.qzero ? __ldg(src + ch) : make_uint4(0, 0, 0, 0);
                const uint32_t flip = p.qflip ? 0x80008000u : 0u;
#pragma unroll
                for (int ch = 0; ch < DP / 8; ++ch) {
                    x[ch].x ^= flip; x[ch].y ^= flip; x[ch].z ^= flip; x[ch].w ^= flip;
                    *reinterpret_cast<uint4*>(dst + (ch >> 3) * kHalfBytes + (((ch & 7) ^ (trow & 7)) << 4)) = x[ch];
                }
                fence_async();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.q_full[rt]);
            // ancestors of this row's node, by shuffles of the sequence's parents
            unsigned long long anc = 0;
            const bool has_new = s.tile1 == s.tiles;
            if (has_new && warp_live) {
                const size_t at = static_cast<size_t>(s.b) * a.n;
                const int p0 = lane < a.n ? checked_parent(a.parent, at, lane, p.status) : -1;
                const int p1 = lane + 32 < a.n ? checked_parent(a.parent, at, lane + 32, p.status) : -1;
                int i = live && node < used ? node : -1;
                while (__any_sync(0xffffffffu, i >= 0)) {
                    if (i >= 0) anc |= 1ull << i;
                    const int q0 = __shfl_sync(0xffffffffu, p0, i & 31), q1 = __shfl_sync(0xffffffffu, p1, i & 31);
                    i = i < 0 ? -1 : (i < 32 ? q0 : q1);
                }
            }
            float m = -INFINITY, l = 0.f;
            for (int kt = s.tile0; ok && kt < s.tile1; ++kt, unit += R) {
                const uint32_t slot = unit & 1u;
                ok = wait(&ctl.s_full[slot], unit >> 1);
                if (!ok) break;
                if (warp_live) {
                    tc_fence_after();
                    const uint32_t s_at = lane_base + slot * kTile;
                    auto tile = [&](auto nch_tag, auto mask) {
                        constexpr int NC = decltype(nch_tag)::value;   // chunks of 32 columns
                        uint32_t x[NC][32];
#pragma unroll
                        for (int q = 0; q < NC; ++q) tmem_ld32(s_at + q * 32, x[q]);
                        tmem_wait_ld();
                        mask(x);
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int q = 0; q < NC; ++q)
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mx[k] = fmax3(mx[k], __uint_as_float(x[q][e + 2 * k]), __uint_as_float(x[q][e + 2 * k + 1]));
                        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        if (kt == s.tile0) {
                            m = mt;
                        } else {
                            const bool up = !(mt <= m + p.thr);
                            if (__any_sync(0xffffffffu, up)) {
                                // the last product into this O has to be complete
                                const uint32_t prev = unit - R;
                                ok = wait(&ctl.pv_done[prev & 1u], prev >> 1);
                                if (!ok) return;
                                tc_fence_after();
                                const float mn = up ? fmaxf(m, mt) : m;
                                const float f = up ? fast_exp2((m - mn) * c) : 1.f;
                                m = mn;
                                l *= f;
#pragma unroll 1
                                for (int q = 0; q < DP / 32; ++q) {
                                    uint32_t o[32];
                                    tmem_ld32(o_at + q * 32, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                    tmem_st32(o_at + q * 32, o);
                                }
                            }
                        }
                        const float mref = m == -INFINITY ? 0.f : -m * c;
                        const float2 c2 = make_float2(c, c), m2 = make_float2(mref, mref);
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int q = 0; q < NC; ++q) {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float2 y = fma2(make_float2(__uint_as_float(x[q][2 * e]), __uint_as_float(x[q][2 * e + 1])), c2, m2);
                                y.x = fast_exp2(y.x);
                                y.y = fast_exp2(y.y);
                                sum[e & 1] = add2(sum[e & 1], y);
                                w[e] = pack2<FP16>(y.x, y.y);
                            }
                            tmem_st16(s_at + q * 16, w);
                        }
                        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                        tmem_wait_st();
                        tc_fence_before();
                    };
                    if (kt == s.tiles - 1) {
                        tile(std::integral_constant<int, 2>{}, [&](uint32_t (&x)[2][32]) {
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const uint32_t bits = static_cast<uint32_t>(anc >> (32 * q));
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(bits >> e & 1u)) x[q][e] = 0xff800000u;
                            }
                        });
                    } else {
                        const int valid = s.len - kt * kTile;
                        tile(std::integral_constant<int, 4>{}, [&](uint32_t (&x)[4][32]) {
                            if (valid < kTile) {
#pragma unroll
                                for (int q = 0; q < 4; ++q)
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (q * 32 + e >= valid) x[q][e] = 0xff800000u;
                            }
                        });
                    }
                    if (!ok) break;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_full[slot]);
            }
            if (!ok) break;
            // ---- the segment's end: O of this row, normalised or as a part
            const uint32_t prev = unit - R;
            ok = wait(&ctl.pv_done[prev & 1u], prev >> 1);
            if (has_new) ok = ok && wait(&ctl.aux, naux);
            if (!ok) break;
            tc_fence_after();
            const unsigned long long poison = has_new ? *reinterpret_cast<volatile unsigned long long*>(&ctl.poison) & anc : 0ull;
            if (has_new) ++naux;
            if (warp_live) {
                const bool whole = s.tile0 == 0 && s.tile1 == s.tiles;
                const int slot = 2 * blockIdx.x + (s.tile0 == 0 ? 1 : 0);
                const bool pad = node >= used;
                const float inv = whole ? (pad || l == 0.f ? 0.f : __fdiv_rn(1.f, l)) : 1.f;
                float* part = p.o + (static_cast<size_t>(slot) * p.used + in_item) * a.D;
                uint16_t* out = static_cast<uint16_t*>(a.out) + qrow * a.D;
#pragma unroll 1
                for (int q = 0; q < DP / 32; ++q) {
                    uint32_t o[32];
                    tmem_ld32(o_at + q * 32, o);
                    tmem_wait_ld();
                    for (unsigned long long bits = poison; bits; bits &= bits - 1) {
                        // a visible node with infinities or NaN: its weight, and what was taken out of its V
                        const int i = __ffsll(static_cast<long long>(bits)) - 1;
                        const size_t at = ((static_cast<size_t>(s.b) * a.n + i) * a.Hkv + s.hk) * a.D;
                        const uint16_t* kr = static_cast<const uint16_t*>(a.k_new) + at;
                        const uint16_t* vr = static_cast<const uint16_t*>(a.v_new) + at;
                        const uint16_t* qr = static_cast<const uint16_t*>(a.q) + qrow * a.D;
                        float dot = 0.f;
                        for (int d = 0; d < a.D; ++d) dot += to_f32<FP16>(qr[d]) * to_f32<FP16>(kr[d]);
                        dot = p.qzero ? 0.f : (p.qflip ? -dot : dot);
                        const float w = fmaxf(fast_exp2((dot - m) * c), 1e-30f);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int d = q * 32 + e;
                            const float x = d < a.D ? to_f32<FP16>(vr[d]) : 0.f;
                            if (!isfinite(x)) o[e] = __float_as_uint(__uint_as_float(o[e]) + w * x);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        const int d = q * 32 + e;
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
                            *reinterpret_cast<float4*>(part + d) = make_float4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<float4*>(part + d + 4) = make_float4(y[4], y[5], y[6], y[7]);
                        }
                    }
                    __syncwarp();
                }
                if (live) {
                    if (!whole) p.ml[static_cast<size_t>(slot) * p.used + in_item] = make_float2(m, l);
                    else if (a.lse) a.lse[qrow] = pad ? -INFINITY : (m == -INFINITY ? 0.f : m * c * kLn2) + logf(l);
                }
            }
            tc_fence_before();
            __syncwarp();
            ++seg;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMma) tmem_free(tmem, 512);
}

// Joins the parts of the item that starts in part blockIdx.x and goes on: one warp per row, the parts
// in order, relative to the row's largest maximum.
template <bool FP16>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const __grid_constant__ AttnParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const svd_tree_attention_args& a = p.a;
    const PartInfo inf = p.info[blockIdx.x];
    if (inf.last < 0) return;
    const int lane = threadIdx.x & 31;
    const int in_item = blockIdx.y * kCombineWarps + (threadIdx.x >> 5);
    const int row = inf.rg * row_tiles(p.rows) * kTile + in_item;
    if (in_item >= p.used || row >= p.rows) return;
    const int first = blockIdx.x, parts = inf.last - first + 1;
    auto slot = [&](int i) { return static_cast<size_t>(2 * (first + i) + (i == 0 ? 1 : 0)) * p.used + in_item; };
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
        // a part that saw nothing has the maximum -inf, the sum 0 and O = 0
        const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : fast_exp2((ml.x - m) * p.c);
        l += ml.y * f;
        if (act) {
            const float4 o = *reinterpret_cast<const float4*>(p.o + slot(i) * a.D + lane * 4);
            acc.x += o.x * f; acc.y += o.y * f; acc.z += o.z * f; acc.w += o.w * f;
        }
    }
    const int node = row / p.G, head = inf.hk * p.G + row - node * p.G;
    const bool pad = a.n_nodes && node >= __ldg(a.n_nodes + inf.b);
    const float inv = pad || l == 0.f ? 0.f : __fdiv_rn(1.f, l);
    const size_t qrow = (static_cast<size_t>(inf.b) * a.n + node) * a.Hq + head;
    if (act) {
        uint2 w = make_uint2(pack2<FP16>(acc.x * inv, acc.y * inv), pack2<FP16>(acc.z * inv, acc.w * inv));
        if (pad) w = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + qrow * a.D + lane * 4) = w;
    }
    if (a.lse && lane == 0) a.lse[qrow] = pad ? -INFINITY : (m == -INFINITY ? 0.f : m * p.c * kLn2) + logf(l);
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

template <bool FP16, int DP, int R>
cudaError_t launch(const AttnParams& p, cudaStream_t st) {
    using Sh = Shape<FP16, DP, R>;
    cudaError_t e = cudaFuncSetAttribute(tree_attention_kernel<FP16, DP, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    tree_attention_kernel<FP16, DP, R><<<kCtas, Sh::kThreads, Sh::kSmem, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(kCtas, (p.used + kCombineWarps - 1) / kCombineWarps);
    cfg.blockDim = dim3(kCombineWarps * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_combine_kernel<FP16>, p);
}

template <bool FP16>
cudaError_t launch_type(const AttnParams& p, cudaStream_t st) {
    const bool wide = p.a.D > 64, two = row_tiles(p.rows) == 2;
    if (wide) return two ? launch<FP16, 128, 2>(p, st) : launch<FP16, 128, 1>(p, st);
    return two ? launch<FP16, 64, 2>(p, st) : launch<FP16, 64, 1>(p, st);
}

}  // namespace

size_t tree_attention_ws_bytes(int, int n, int Hq, int Hkv, int D) { return attn_ws(n * (Hq / Hkv), D).total; }

int launch_tree_attention(const svd_tree_attention_args& a, void* ws, void* stream) {
    AttnParams p;
    std::memset(&p, 0, sizeof p);
    p.a = a;
    p.G = a.Hq / a.Hkv;
    p.rows = a.n * p.G;
    const int group = row_tiles(p.rows) * kTile;
    p.used = p.rows < group ? p.rows : group;
    p.NR = (p.rows + group - 1) / group;
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
