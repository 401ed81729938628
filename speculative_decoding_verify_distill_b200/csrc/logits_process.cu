// logits_process.cu -- penalties, biases and grammar masks on the logits of a tree of drafts, and
// the gradient of that map (include/svd_tree.h).
//
// Per element the map reads a logit and writes one, so it is bound by HBM: 4 bytes and an eighth (the
// mask bit) per element, and nearly every element passes through unchanged or masked: only the ids
// that the sequence has seen, or that carry a bias, need arithmetic.  A CTA owns a chunk of ids of one
// sequence and all of its rows (or a group of them).  Once, it builds a table of its chunk in shared
// memory (one word per id: prompt flag, count in the generated history, index of the drafted nodes
// with this token, bias) and the list of the ids that the table has anything for ("touched").  Rows then
// stream through a two-stage ring of bulk copies, two rows a stage.  A warp owns 512 of the ids in every row (every
// eighth block of 64: touched ids crowd among the low ones) and works without the others: its lanes share the (row, touched id) pairs of a stage and change those
// elements in shared memory, and then every lane takes whole vectors: mask, store, maximum.
//
// The pairs are what makes the touched ids cheap.  They are few and anywhere, so nearly every warp's
// vectors hold one; worked on by the lane that holds its vector, they cost every warp the arithmetic
// for one or two lanes (130 us at 32 x 17 rows of 151936 with 1536 tokens of history).  Sharing them over the
// whole CTA took a barrier a stage (84 us); over a warp it takes none (79 us).
//
// Ancestors' tokens differ from row to row.  They need no per-row table: the table names, for an
// id that some node drafted, the set of nodes with that token (64 bits), and the row's count is
// popc(set & ancestors of the row).
//
// The arithmetic is fp32 with explicit rounding in the documented order and rounds once, so the
// rounded values (and the argmax taken over them) are fixed bit for bit.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "tree_device.cuh"

namespace svd {

namespace {

constexpr int kWarps = 8;                      // that work on rows; one more fills the stages
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kVecs = 2;                       // vectors of 8 ids per lane and row
constexpr int kWarpIds = 8 * 32 * kVecs;       // ids of a warp
constexpr int kChunk = kWarps * kWarpIds;      // ids per CTA
constexpr int kStages = 2;
constexpr int kStageBytes = 4 * kChunk;        // two rows of bf16 or one of fp32
constexpr int kFewCtas = 444;                  // three per SM
constexpr uint64_t kWaitNs = 1000000000ull;

// Table word of an id.
constexpr uint32_t kPrompt = 0x80000000u;      // seen in the prompt
constexpr int kSlotShift = 24;                 // 7 bits: 1 + lowest node with this token
constexpr uint32_t kHasBias = 1u << 23;        // the rest of the word is the index of a bias entry, which
                                               // holds the bias and the word
constexpr uint32_t kCountMask = kHasBias - 1;  // count in the generated history

struct Tables {
    unsigned long long anc[kTreeMaxNodes];     // ancestors of every node
    unsigned long long nodes[kTreeMaxNodes];   // nodes that share the token of their lowest one
    uint4 best[kWarps][kTreeMaxNodes];         // each warp's best vector of each row,
    int best_at[kWarps][kTreeMaxNodes];        // and its first id (-1: none)
    uint64_t full[kStages], empty[kStages];
    int scan[kWarps + 1];
    int start[kWarps + 1];                     // of each warp's part of the list
    int tok[kTreeMaxNodes];
    int8_t parent[kTreeMaxNodes];
    int last, repeated;
};

struct Dyn {                                   // dynamic shared memory
    uint8_t* stage;                            // [kStages][kStageBytes]
    uint32_t* tab;                             // [kChunk]
    uint32_t* touched;                         // [kChunk / 32]
    uint16_t* list;                            // [kChunk]: touched ids, by owning warp
    uint32_t* bias_word;                       // [n_bias]
    float* bias;                               // [n_bias]
};
constexpr size_t kDynBytes = kStages * kStageBytes + kChunk * 4 + kChunk / 8 + kChunk * 2;

// Fills the chunk's table, touched bits and the ancestor sets; every thread of the CTA calls it.
__device__ void build_tables(const LogitsParams& p, int b, int v0, int v1, int n_bias, Tables& s, const Dyn& d) {
    const svd_logits_process_args& a = p.a;
    const int t = threadIdx.x;
    for (int i = t; i < kChunk / 4; i += kThreads) reinterpret_cast<uint4*>(d.tab)[i] = make_uint4(0, 0, 0, 0);
    for (int i = t; i < kChunk / 32; i += kThreads) d.touched[i] = 0;
    if (t == 0) s.repeated = 0;
    if (t < kTreeMaxNodes) {
        s.nodes[t] = 0;
        s.tok[t] = -1;
        if (t < a.n && a.node_tok) {
            const size_t row = static_cast<size_t>(b) * a.n;
            s.parent[t] = static_cast<int8_t>(checked_parent(a.parent, row, t, p.status));
            const int tok = __ldg(a.node_tok + row + t);
            if (tok >= 0 && tok < a.V) s.tok[t] = tok;
            else if (tok != -1) set_device_error(p.status, SVD_ERR_TOKEN_RANGE);
        }
    }
    __syncthreads();
    auto touch = [&](int i) { atomicOr(&d.touched[i >> 5], 1u << (i & 31)); };
    const int32_t* bt = a.bias_tok + static_cast<size_t>(b) * a.n_bias;
    const float* bv = a.bias_val + static_cast<size_t>(b) * a.n_bias;
    if (n_bias > 0) {
        for (int i = t; i < n_bias; i += kThreads) {
            d.bias_word[i] = 0;
            const int tok = __ldg(bt + i);
            if (tok >= v0 && tok < v1) {
                d.bias[i] = __ldg(bv + i);
                if (atomicCAS(&d.tab[tok - v0], 0u, kHasBias | static_cast<uint32_t>(i)) != 0u) s.repeated = 1;
                touch(tok - v0);
            } else if (tok < -1 || tok >= a.V) {
                set_device_error(p.status, SVD_ERR_TOKEN_RANGE);
            }
        }
        __syncthreads();
        if (s.repeated) {
            // an id occurs more than once: its entry gets the sum of all of them, in list order
            for (int i = t; i < n_bias; i += kThreads) {
                const int tok = __ldg(bt + i);
                if (tok < v0 || tok >= v1 || (d.tab[tok - v0] & kCountMask) != static_cast<uint32_t>(i)) continue;
                float sum = 0.f;
                for (int k = 0; k < n_bias; ++k)
                    if (__ldg(bt + k) == tok) sum = __fadd_rn(sum, __ldg(bv + k));
                d.bias[i] = sum;
            }
        }
    }
    auto word = [&](int at) {
        const uint32_t w = n_bias > 0 ? d.tab[at] : 0u;
        return w & kHasBias ? &d.bias_word[w & kCountMask] : &d.tab[at];
    };
    if (a.history) {
        const int S = a.hist_stride;
        int hl = a.hist_len ? __ldg(a.hist_len + b) : S;
        hl = hl < 0 ? 0 : (hl > S ? S : hl);
        int pl = a.prompt_len ? __ldg(a.prompt_len + b) : 0;
        pl = pl < 0 ? 0 : (pl > hl ? hl : pl);
        const int32_t* h = a.history + static_cast<size_t>(b) * S;
#pragma unroll 8
        for (int i = t; i < hl; i += kThreads) {
            const int tok = __ldg(h + i);
            if (tok >= v0 && tok < v1) {
                if (i < pl) atomicOr(word(tok - v0), kPrompt);
                else atomicAdd(word(tok - v0), 1u);
                touch(tok - v0);
            } else if (tok < -1 || tok >= a.V) {
                set_device_error(p.status, SVD_ERR_TOKEN_RANGE);
            }
        }
    }
    if (a.node_tok && t < a.n) {
        s.anc[t] = ancestors_of(s.parent, t);
        const int tok = s.tok[t];
        if (tok >= v0 && tok < v1) {
            int low = 0;
            while (s.tok[low] != tok) ++low;
            atomicOr(&s.nodes[low], 1ull << t);
            if (low == t) {
                atomicOr(word(tok - v0), static_cast<uint32_t>(t + 1) << kSlotShift);
                touch(tok - v0);
            }
        }
    }
    __syncthreads();
}

// Count of an id among the generated tokens that row j sees.
__device__ __forceinline__ int row_count(uint32_t w, unsigned long long anc, const Tables& s) {
    const uint32_t slot = (w >> kSlotShift) & 127u;
    int c = static_cast<int>(w & kCountMask);
    if (slot) c += __popcll(s.nodes[slot - 1] & anc);
    return c;
}

// prmt with the selector's replicate-sign bits (__byte_perm takes three bits of each selector only).
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(a), "r"(sel));
    return r;
}
// Elements whose bit in `m` is clear become `fill` (two copies of 16 bits): each bit is spread to the
// sign of a byte, and the byte permutation replicates signs over 16 bits.
__device__ __forceinline__ uint4 mask16(const uint4& x, uint32_t m, uint32_t fill) {
    const uint32_t lo = ((m & 15u) * 0x00204081u & 0x01010101u) << 7, hi = ((m >> 4 & 15u) * 0x00204081u & 0x01010101u) << 7;
    const uint32_t k0 = prmt(lo, 0x9988), k1 = prmt(lo, 0xbbaa);
    const uint32_t k2 = prmt(hi, 0x9988), k3 = prmt(hi, 0xbbaa);
    return make_uint4((x.x & k0) | (fill & ~k0), (x.y & k1) | (fill & ~k1), (x.z & k2) | (fill & ~k2), (x.w & k3) | (fill & ~k3));
}
// Writes the first `left` (at most 8) elements of a vector where the rows are not aligned.
template <class T>
__device__ __forceinline__ void store_some(T* to, const T (&x)[8], int left) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < left) to[e] = x[e];
}

// GRAD: the gradient (dz -> dlogits), F32: dz and dlogits in fp32.
template <bool GRAD, bool F32, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 3) logits_process_kernel(LogitsParams p) {
    using T = typename std::conditional<F32, float, uint16_t>::type;
    constexpr int kRows = F32 ? 1 : 2;                    // rows per stage
    // Pairs per lane that are worked on at once, and whose raw logits the gradient loads ahead: as many as a dense
    // chunk's two rows need, but one row of fp32 has half of them.  us with 1 / 2 / 4 in fp32:
    //   6 x 16 rows of 128256, 700 / 4000 tokens of history   28.8 / 25.3 / 26.8,  45.4 / 40.7 / 39.7
    //   32 x 16, 1 x 64 and 64 x 1 rows of 151936             120.1 / 120.0 / 121.5,  30.1 / 28.4 / 27.4,  35.9 / 36.1 / 36.6
    //   4 x 8 rows of 32000                                   12.4 / 12.2 / 11.8
    // and with 2 / 4 in bf16: 8 x 64 rows of 151936 92.9 / 90.1, 32 x 16 rows 74.6 / 73.9.
    constexpr int kAhead = F32 ? 2 : 4;
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ Tables s;
    const svd_logits_process_args& a = p.a;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, b = blockIdx.x, V = a.V;
    const int v0 = blockIdx.y * kChunk, v1 = min(V, v0 + kChunk);
    const int j0 = blockIdx.z * p.rows_per_cta, j1 = min(a.n, j0 + p.rows_per_cta);
    const int n_bias = GRAD ? 0 : a.n_bias;
    Dyn d;
    d.stage = dyn;
    d.tab = reinterpret_cast<uint32_t*>(dyn + kStages * kStageBytes);
    d.touched = d.tab + kChunk;
    d.list = reinterpret_cast<uint16_t*>(d.touched + kChunk / 32);
    d.bias_word = reinterpret_cast<uint32_t*>(d.list + kChunk);
    d.bias = reinterpret_cast<float*>(d.bias_word + n_bias);

    const bool want_arg = !GRAD && a.argmax != nullptr;
    const size_t row0 = static_cast<size_t>(b) * a.n;
    const uint16_t* const raw = a.logits + row0 * V;
    const T* const src = GRAD ? static_cast<const T*>(a.dz) + row0 * V : reinterpret_cast<const T*>(raw);
    T* const dst = GRAD ? static_cast<T*>(a.dlogits) + row0 * V
                        : (a.out ? reinterpret_cast<T*>(a.out) + row0 * V : nullptr);
    // in place without a mask only the touched elements are read and written
    const bool sparse = src == dst && !want_arg && !a.mask;
    const int batches = sparse ? 0 : (j1 - j0 + kRows - 1) / kRows;

    // (one thread) rows of batch k into its stage
    auto fetch = [&](int k) {
        uint8_t* to = d.stage + (k % kStages) * kStageBytes;
        const int j = j0 + k * kRows, rows = min(kRows, j1 - j);
        const uint32_t bytes = static_cast<uint32_t>(v1 - v0) * sizeof(T);
        mbar_arrive_expect_tx(&s.full[k % kStages], rows * bytes);
        for (int r = 0; r < rows; ++r)
            bulk_load(to + r * kChunk * sizeof(T), src + static_cast<size_t>(j + r) * V + v0, bytes, &s.full[k % kStages]);
    };
    if (ALIGNED && warp == kWarps && lane == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], kWarps);
        }
        fence_mbar_init();
        // the first rows arrive while the table is built
        for (int k = 0; k < kStages && k < batches; ++k) fetch(k);
    }
    build_tables(p, b, v0, v1, n_bias, s, d);

    // the list of touched ids, warp by warp
    // thread t: word t % 16 of the ids of warp t / 16, so that each warp's part of the list is contiguous
    const int word = (((t & 15) >> 1) * kWarps + (t >> 4)) * 2 + (t & 1);
    const uint32_t tw = t < kChunk / 32 ? d.touched[word] : 0u;
    int n_touched;
    {
        const int mine = __popc(tw);
        int rank = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, rank, o);
            if (lane >= o) rank += y;
        }
        if (lane == 31) s.scan[warp] = rank;
        __syncthreads();
        n_touched = 0;
#pragma unroll
        for (int w = 0; w <= kWarps; ++w) {
            if (w < warp) rank += s.scan[w];
            n_touched += s.scan[w];
        }
        rank -= mine;
        if (t < kChunk / 32 && t % (kWarpIds / 32) == 0) s.start[t / (kWarpIds / 32)] = rank;
        if (t == 0) s.start[kWarps] = n_touched;
        for (uint32_t bits = tw; bits; bits &= bits - 1) d.list[rank++] = static_cast<uint16_t>(word * 32 + __ffs(bits) - 1);
    }
    __syncthreads();

    const float rep = a.repetition ? __ldg(a.repetition + b) : 1.f;
    const float freq = !GRAD && a.frequency ? __ldg(a.frequency + b) : 0.f;
    const float pres = !GRAD && a.presence ? __ldg(a.presence + b) : 0.f;
    auto f32 = [](uint16_t w) { return __uint_as_float(static_cast<uint32_t>(w) << 16); };
    // the new value of id v0 + at in row j: x is the raw logit, or dz with the sign of the raw logit
    auto changed = [&](float x, bool positive, int at, int j) {
        uint32_t w = d.tab[at], entry = 0;
        const bool has_bias = n_bias > 0 && (w & kHasBias);
        if (has_bias) {
            entry = w & kCountMask;
            w = d.bias_word[entry];
        }
        const int c = row_count(w, a.node_tok ? s.anc[j] : 0ull, s);
        if (c > 0 || (w & kPrompt)) x = positive ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
        if (!GRAD) {
            x = __fsub_rn(x, __fmul_rn(freq, static_cast<float>(c)));
            if (c > 0) x = __fsub_rn(x, pres);
            if (has_bias) x = __fadd_rn(x, d.bias[entry]);
        }
        return x;
    };
    auto as_f32 = [&](T x) { return F32 ? static_cast<float>(x) : f32(static_cast<uint16_t>(x)); };
    auto as_t = [&](float x) { return F32 ? static_cast<T>(x) : static_cast<T>(__bfloat16_as_ushort(__float2bfloat16_rn(x))); };

    if (sparse) {
        for (int i = t; i < n_touched * (j1 - j0); i += kThreads) {
            const int at = d.list[i % n_touched], j = j0 + i / n_touched;
            const size_t e = static_cast<size_t>(j) * V + v0 + at;
            const float x = as_f32(dst[e]);
            dst[e] = as_t(changed(x, GRAD ? f32(__ldg(raw + e)) > 0.f : x > 0.f, at, j));
        }
        return;
    }

    const size_t W4 = static_cast<size_t>((V + 31) / 32) * 4;
    const bool row_mask = a.mask && a.mask_rows != 1;
    const uint8_t* const mask = reinterpret_cast<const uint8_t*>(a.mask) + (row_mask ? row0 : static_cast<size_t>(b)) * W4;
    const uint32_t mval = __bfloat16_as_ushort(__float2bfloat16_rn(GRAD ? 0.f : a.mask_value));
    const uint32_t fill = mval | mval << 16;
    bool ok = true;
    if (warp == kWarps) {
        // refills a stage when every warp has left it
        for (int k = kStages; ALIGNED && ok && k < batches; ++k) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s.empty[k % kStages], (k / kStages - 1) & 1, kWaitNs)) != 0;
            if (ok && lane == 0) fetch(k);
            __syncwarp();
        }
    }
    const int mine = warp < kWarps ? batches : 0;
    // the lane's vectors: eight lanes take a block of 64 ids
    auto id8 = [&](int q) { return ((q * 4 + (lane >> 3)) * kWarps + warp) * 64 + (lane & 7) * 8; };
    const uint16_t* const list = d.list + (warp < kWarps ? s.start[warp] : 0);
    const int pairs = warp < kWarps ? (s.start[warp + 1] - s.start[warp]) * kRows : 0;
    // mask bytes of a batch, and the gradient's raw logits of this lane's first pairs, go out a batch ahead
    uint32_t ms[kRows][kVecs];
    uint16_t raws[kAhead] = {};
    auto prefetch = [&](int k) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int j = j0 + k * kRows + r;
#pragma unroll
            for (int q = 0; q < kVecs; ++q) {
                const int v = v0 + id8(q);
                if (a.mask && j < j1 && v < v1) ms[r][q] = __ldg(mask + (row_mask ? j * W4 : 0) + (v >> 3));
            }
        }
#pragma unroll
        for (int u = 0; GRAD && u < kAhead; ++u) {
            const int i = lane + u * 32, j = j0 + k * kRows + i % kRows;
            if (i < pairs && j < j1) raws[u] = __ldg(raw + static_cast<size_t>(j) * V + v0 + list[i / kRows]);
        }
    };
    if (mine) prefetch(0);

    for (int k = 0; k < mine; ++k) {
        T* const st = reinterpret_cast<T*>(d.stage + (k % kStages) * kStageBytes);
        const int jb = j0 + k * kRows;
        if (ALIGNED) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s.full[k % kStages], (k / kStages) & 1, kWaitNs)) != 0;
            if (!ok) break;
        } else {
            // each warp brings its own ids
            for (int r = 0; r < kRows && jb + r < j1; ++r)
                for (int i = lane; i < kWarpIds; i += 32) {
                    const int at = ((i >> 6) * kWarps + warp) * 64 + (i & 63);
                    if (v0 + at < v1) st[r * kChunk + at] = src[static_cast<size_t>(jb + r) * V + v0 + at];
                }
            __syncwarp();
        }
        // new value of pair i; behind the last one, any value
        auto value = [&](int i, uint16_t raw_logit) {
            const int c = min(i, pairs - 1), r = c % kRows, at = list[c / kRows];
            const float x = as_f32(st[r * kChunk + at]);
            return changed(x, GRAD ? f32(raw_logit) > 0.f : x > 0.f, at, min(jb + r, a.n - 1));
        };
        auto put = [&](int i, float x) {
            if (i < pairs && jb + i % kRows < j1) st[i % kRows * kChunk + list[i / kRows]] = as_t(x);
        };
        if (pairs <= 32) {
            if (pairs > 0) put(lane, value(lane, raws[0]));
        } else {
            // several at once: one alone waits through shared memory, the division and (behind the first
            // kAhead) the raw logit
#pragma unroll 1
            for (int i = lane; i - lane < pairs; i += 32 * kAhead) {
                float x[kAhead];
#pragma unroll
                for (int u = 0; GRAD && u < kAhead; ++u) {
                    const int c = min(i + u * 32, pairs - 1);
                    if (i != lane) raws[u] = __ldg(raw + static_cast<size_t>(min(jb + c % kRows, a.n - 1)) * V + v0 + list[c / kRows]);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) x[u] = value(i + u * 32, raws[u]);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) put(i + u * 32, x[u]);
            }
        }
        __syncwarp();
        uint32_t mk[kRows][kVecs];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int q = 0; q < kVecs; ++q) mk[r][q] = a.mask ? ms[r][q] : 0xffu;
        if (k + 1 < batches) prefetch(k + 1);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int j = jb + r;
            if (j >= j1) break;
            float best_m = __int_as_float(0x7fffffff);   // NaN: no vector yet
            uint4 best = make_uint4(0, 0, 0, 0);
            int best_at = -1;
#pragma unroll
            for (int q = 0; q < kVecs; ++q) {
                const int i8 = id8(q), v = v0 + i8;
                if (v >= v1) continue;
                const size_t off = static_cast<size_t>(j) * V + v;
                if (F32) {
                    const float4 lo = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(st) + i8);
                    const float4 hi = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(st) + i8 + 4);
                    float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = mk[r][q] >> e & 1u ? x[e] : 0.f;
                    float* to = reinterpret_cast<float*>(dst) + off;
                    if (ALIGNED) {
                        __stcs(reinterpret_cast<float4*>(to), make_float4(x[0], x[1], x[2], x[3]));
                        __stcs(reinterpret_cast<float4*>(to) + 1, make_float4(x[4], x[5], x[6], x[7]));
                    } else {
                        store_some(to, x, V - v);
                    }
                    continue;
                }
                uint4 x = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(st) + r * kChunk + i8);
                if (a.mask) x = mask16(x, mk[r][q], fill);
                if (dst) {
                    uint16_t* to = reinterpret_cast<uint16_t*>(dst) + off;
                    if (ALIGNED) {
                        __stcs(reinterpret_cast<uint4*>(to), x);
                    } else {
                        const uint16_t w[8] = {static_cast<uint16_t>(x.x), static_cast<uint16_t>(x.x >> 16),
                                               static_cast<uint16_t>(x.y), static_cast<uint16_t>(x.y >> 16),
                                               static_cast<uint16_t>(x.z), static_cast<uint16_t>(x.z >> 16),
                                               static_cast<uint16_t>(x.w), static_cast<uint16_t>(x.w >> 16)};
                        store_some(to, w, V - v);
                    }
                }
                if (want_arg) {
                    if (!ALIGNED && v + 8 > V) {   // what lies behind V becomes NaN: no candidate
                        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (v + e >= V) w[e >> 1] |= 0x7fffu << (16 * (e & 1));
                        x = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    const float m = max8_bf16(x);
                    if (m > best_m || best_m != best_m) {
                        best = x;
                        best_m = m;
                        best_at = v;
                    }
                }
            }
            if (want_arg) {
                // the warp's best vector; of equal ones the lowest ids: first by q, then by lane
                const bool num = best_m == best_m;
                const float top = redux_max_f32(num ? best_m : -INFINITY);
                const unsigned win = __ballot_sync(0xffffffffu, num && best_m == top);
                const unsigned low = __ballot_sync(0xffffffffu, num && best_m == top && best_at == v0 + id8(0));
                if (lane == (win ? __ffs(low ? low : win) - 1 : 0)) {
                    s.best[warp][j - j0] = best;
                    s.best_at[warp][j - j0] = win ? best_at : -1;
                }
            }
        }
        if (ALIGNED) {
            fence_async();      // the stage is written by copies again
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.empty[k % kStages]);
        } else {
            __syncwarp();
        }
    }
    ok = __syncthreads_and(ok) != 0;
    if (!ok) {   // a copy did not arrive in time: record it, and leave no copy in flight
        if (t == 0) {
            set_device_error(p.status, SVD_ERR_TIMEOUT);
            for (int i = 0; i < kStages; ++i) mbar_wait_bounded(&s.full[i], 0, kWaitNs), mbar_wait_bounded(&s.full[i], 1, kWaitNs);
        }
    }
    if (!want_arg) return;
    // one atomic maximum per row and CTA (a maximum does not depend on the order); the last CTA of
    // the sequence turns the keys into ids and leaves the workspace zero, behind a time-out too
    if (ok && t < j1 - j0) {
        unsigned long long key = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (s.best_at[w][t] < 0) continue;
            const uint4 x = s.best[w][t];
            const float m = max8_bf16(x);
            key = max(key, argmax_key(m, s.best_at[w][t] + first_pos(x, m)));
        }
        if (key) atomicMax(&p.key[row0 + j0 + t], key);
        __threadfence();
    }
    __syncthreads();
    if (t == 0) s.last = atomicAdd(&p.ticket[b], 1u) == gridDim.y * gridDim.z - 1;
    __syncthreads();
    if (!s.last) return;
    __threadfence();
    if (t < a.n) {
        a.argmax[row0 + t] = argmax_id(__ldcg(&p.key[row0 + t]));
        p.key[row0 + t] = 0ull;
    }
    if (t == 0) p.ticket[b] = 0u;
}

template <bool GRAD, bool F32, bool ALIGNED>
cudaError_t launch(const LogitsParams& in, cudaStream_t st) {
    LogitsParams p = in;
    const int chunks = (p.a.V + kChunk - 1) / kChunk;
    // Every split of the rows builds the chunk's table again.  They are split so far that no SM is without
    // work, and into groups of eight or more to give two rounds of CTAs, behind which a chunk with many touched ids
    // does not stand alone (8 x 64 rows of 151936: 100 us with one round, 82 us with two).
    const int ctas = chunks * p.a.B, fill = kFewCtas / ctas, rounds = std::min((2 * kFewCtas + ctas - 1) / ctas, p.a.n / 8);
    int splits = std::min(p.a.n, std::max(1, std::max(fill, rounds)));
    p.rows_per_cta = (p.a.n + splits - 1) / splits;
    // low ids, which have the most touched ones, start first and do not end up in the tail
    const dim3 grid(p.a.B, chunks, (p.a.n + p.rows_per_cta - 1) / p.rows_per_cta);
    const size_t bytes = kDynBytes + (GRAD ? 0 : 8 * static_cast<size_t>(p.a.n_bias));
    const cudaError_t e = cudaFuncSetAttribute(logits_process_kernel<GRAD, F32, ALIGNED>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kDynBytes + 8 * 4096));
    if (e != cudaSuccess) return e;
    logits_process_kernel<GRAD, F32, ALIGNED><<<grid, kThreads, bytes, st>>>(p);
    return cudaGetLastError();
}

template <bool GRAD, bool F32>
cudaError_t launch_al(const LogitsParams& p, cudaStream_t st) {
    return p.aligned ? launch<GRAD, F32, true>(p, st) : launch<GRAD, F32, false>(p, st);
}

}  // namespace

int launch_logits_process(const LogitsParams& p, bool grad, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (!grad) e = launch_al<false, false>(p, st);
    else if (p.a.grad_fp32) e = launch_al<true, true>(p, st);
    else e = launch_al<true, false>(p, st);
    return static_cast<int>(e);
}

}  // namespace svd
