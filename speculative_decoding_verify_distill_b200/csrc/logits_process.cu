// logits_process.cu -- penalties, biases and grammar masks on the logits of a tree of drafts, and
// the gradient of that map (include/svd_tree.h).
//
// Per element the map reads a logit and writes one, so it is bound by HBM: 4 bytes and an eighth
// (the mask bit) per element, and nearly every element passes through unchanged or masked: only the
// ids that the sequence has seen, or that carry a bias, need arithmetic.  A CTA owns a chunk of ids
// of one sequence and all of its rows (or a group of them): it builds, once, a table of its chunk in
// shared memory (one word per id: prompt flag, count in the generated history, index of the
// drafted nodes with this token), and a bit per id that says whether the table has anything.  Each
// thread keeps the bits of its own vectors in a register for all rows, so the common vector costs
// a load, a mask byte and a store.
//
// Ancestors' tokens differ from row to row.  They need no per-row table: the table names, for an
// id that some node drafted, the set of nodes with that token (64 bits), and the row's count is
// popc(set & ancestors of the row).
//
// The arithmetic is fp32 with explicit rounding in the documented order and rounds once, so the
// rounded values (and the argmax taken over them) are fixed bit for bit.
#include <cuda_runtime.h>

#include <cmath>

#include "tree_device.cuh"

namespace svd {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kPrompt = 0x80000000u;   // table word: seen in the prompt
constexpr int kSlotShift = 24;              // 7 bits: 1 + lowest node with this token
constexpr uint32_t kCountMask = 0x00ffffffu;

template <bool ALIGNED>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int v, int V) {
    if (ALIGNED) return __ldcs(reinterpret_cast<const uint4*>(row + v));
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = v + e < V ? __ldg(row + v + e) : 0x7fffu;   // NaN: never an argmax
    return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}
template <bool ALIGNED>
__device__ __forceinline__ void store8(uint16_t* row, int v, int V, const uint4& x) {
    if (ALIGNED) {
        __stcs(reinterpret_cast<uint4*>(row + v), x);
        return;
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (v + e < V) row[v + e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
}
template <bool ALIGNED>
__device__ __forceinline__ void load8(const float* row, int v, int V, float (&x)[8]) {
    if (ALIGNED) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(row + v));
        const float4 b = __ldcs(reinterpret_cast<const float4*>(row + v) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v + e < V ? row[v + e] : 0.f;
}
template <bool ALIGNED>
__device__ __forceinline__ void store8(float* row, int v, int V, const float (&x)[8]) {
    if (ALIGNED) {
        __stcs(reinterpret_cast<float4*>(row + v), make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4*>(row + v) + 1, make_float4(x[4], x[5], x[6], x[7]));
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (v + e < V) row[v + e] = x[e];
}

struct Tables {
    unsigned long long anc[kTreeMaxNodes];    // ancestors of every node
    unsigned long long nodes[kTreeMaxNodes];  // nodes that share the token of their lowest one
    unsigned long long key[kWarps][kTreeMaxNodes];
    int tok[kTreeMaxNodes];
    int8_t parent[kTreeMaxNodes];
    int last;
};

// Fills the chunk's table, touched bits and the ancestor sets; every thread of the CTA calls it.
__device__ void build_tables(const LogitsParams& p, int b, int v0, int v1, bool grad, Tables& s,
                             uint32_t* tab, float* bias, uint32_t* touched) {
    const svd_logits_process_args& a = p.a;
    const int t = threadIdx.x, ch = p.chunk;
    const bool has_bias = !grad && a.n_bias > 0;
    for (int i = t; i < ch / 4; i += kThreads) reinterpret_cast<uint4*>(tab)[i] = make_uint4(0, 0, 0, 0);
    if (has_bias)
        for (int i = t; i < ch / 4; i += kThreads) reinterpret_cast<float4*>(bias)[i] = make_float4(0, 0, 0, 0);
    for (int i = t; i < ch / 32; i += kThreads) touched[i] = 0;
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
    auto touch = [&](int i) { atomicOr(&touched[i >> 5], 1u << (i & 31)); };
    if (a.history) {
        const int S = a.hist_stride;
        int hl = a.hist_len ? __ldg(a.hist_len + b) : S;
        hl = hl < 0 ? 0 : (hl > S ? S : hl);
        int pl = a.prompt_len ? __ldg(a.prompt_len + b) : 0;
        pl = pl < 0 ? 0 : (pl > hl ? hl : pl);
        const int32_t* h = a.history + static_cast<size_t>(b) * S;
        for (int i = t; i < hl; i += kThreads) {
            const int tok = __ldg(h + i);
            if (tok >= v0 && tok < v1) {
                if (i < pl) atomicOr(&tab[tok - v0], kPrompt);
                else atomicAdd(&tab[tok - v0], 1u);
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
                atomicOr(&tab[tok - v0], static_cast<uint32_t>(t + 1) << kSlotShift);
                touch(tok - v0);
            }
        }
    }
    if (has_bias) {
        const int32_t* bt = a.bias_tok + static_cast<size_t>(b) * a.n_bias;
        const float* bv = a.bias_val + static_cast<size_t>(b) * a.n_bias;
        for (int i = t; i < a.n_bias; i += kThreads) {
            const int tok = __ldg(bt + i);
            if (tok >= v0 && tok < v1) {
                // the first entry of an id adds all of them, in list order
                bool first = true;
                for (int k = 0; k < i; ++k) first = first && __ldg(bt + k) != tok;
                if (first) {
                    float sum = __ldg(bv + i);
                    for (int k = i + 1; k < a.n_bias; ++k)
                        if (__ldg(bt + k) == tok) sum = __fadd_rn(sum, __ldg(bv + k));
                    bias[tok - v0] = sum;
                    touch(tok - v0);
                }
            } else if (tok < -1 || tok >= a.V) {
                set_device_error(p.status, SVD_ERR_TOKEN_RANGE);
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

// GRAD: the gradient (dz -> dlogits), F32: dz and dlogits in fp32.  NV: vectors of 8 ids per thread.
template <bool GRAD, bool F32, bool ALIGNED, int NV>
__global__ void __launch_bounds__(kThreads) logits_process_kernel(LogitsParams p) {
    extern __shared__ __align__(16) uint32_t dyn[];
    __shared__ Tables s;
    const svd_logits_process_args& a = p.a;
    const int t = threadIdx.x, lane = t & 31, b = blockIdx.y, V = a.V;
    const int v0 = blockIdx.x * p.chunk, v1 = min(V, v0 + p.chunk);
    const int j0 = blockIdx.z * p.rows_per_cta, j1 = min(a.n, j0 + p.rows_per_cta);
    uint32_t* tab = dyn;
    uint32_t* touched = dyn + p.chunk;
    float* bias = reinterpret_cast<float*>(touched + p.chunk / 32);
    const bool has_bias = !GRAD && a.n_bias > 0;
    build_tables(p, b, v0, v1, GRAD, s, tab, bias, touched);

    const float rep = a.repetition ? __ldg(a.repetition + b) : 1.f;
    const float freq = !GRAD && a.frequency ? __ldg(a.frequency + b) : 0.f;
    const float pres = !GRAD && a.presence ? __ldg(a.presence + b) : 0.f;
    const bool want_arg = !GRAD && a.argmax != nullptr;
    // in place, a vector that nothing changes needs neither its load nor its store
    const bool in_place = GRAD ? a.dz == a.dlogits : a.logits == a.out;
    const bool may_skip = in_place && !want_arg;
    const size_t W = static_cast<size_t>((V + 31) / 32);

    int vv[NV];
    uint32_t tb[NV], mb1[NV];
    const uint8_t* mask = reinterpret_cast<const uint8_t*>(a.mask);
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        vv[q] = v0 + (q * kThreads + t) * 8;
        tb[q] = vv[q] < v1 ? reinterpret_cast<const uint8_t*>(touched)[(vv[q] - v0) >> 3] : 0u;
        mb1[q] = 0xffu;
        if (mask && a.mask_rows == 1 && vv[q] < v1) mb1[q] = __ldg(mask + b * W * 4 + (vv[q] >> 3));
    }
    const uint16_t mval = __bfloat16_as_ushort(__float2bfloat16_rn(GRAD ? 0.f : a.mask_value));

    for (int j = j0; j < j1; ++j) {
        const size_t row = static_cast<size_t>(b) * a.n + j;
        const size_t off = row * V;
        const unsigned long long anc = a.node_tok ? s.anc[j] : 0ull;
        uint4 best = make_uint4(0, 0, 0, 0);
        float best_m = -INFINITY;
        int best_at = -1;
        uint4 xs[NV];
        uint32_t ms[NV];
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            ms[q] = mb1[q];
            if (mask && a.mask_rows != 1 && vv[q] < v1) ms[q] = __ldg(mask + row * W * 4 + (vv[q] >> 3));
            if (!F32 && vv[q] < v1 && !(may_skip && tb[q] == 0u && ms[q] == 0xffu))
                xs[q] = load8<ALIGNED>((GRAD ? static_cast<const uint16_t*>(a.dz) : a.logits) + off, vv[q], V);
        }
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int v = vv[q];
            if (v >= v1 || (may_skip && tb[q] == 0u && ms[q] == 0xffu)) continue;
            if (F32) {
                float d[8];
                load8<ALIGNED>(static_cast<const float*>(a.dz) + off, v, V, d);
                if (tb[q]) {
                    float x[8];
                    unpack8(load8<ALIGNED>(a.logits + off, v, V), x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t w = (tb[q] >> e & 1u) ? tab[v - v0 + e] : 0u;
                        if (w && ((w & kPrompt) || row_count(w, anc, s) > 0))
                            d[e] = x[e] > 0.f ? __fdiv_rn(d[e], rep) : __fmul_rn(d[e], rep);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!(ms[q] >> e & 1u)) d[e] = 0.f;
                store8<ALIGNED>(static_cast<float*>(a.dlogits) + off, v, V, d);
                continue;
            }
            uint4 x4 = xs[q];
            if (tb[q]) {
                float x[8], r[8];
                unpack8(x4, x);
                if (GRAD) unpack8(load8<ALIGNED>(a.logits + off, v, V), r);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (!(tb[q] >> e & 1u)) continue;
                    const uint32_t w = tab[v - v0 + e];
                    const int c = row_count(w, anc, s);
                    if (c > 0 || (w & kPrompt)) {
                        const bool pos = GRAD ? r[e] > 0.f : x[e] > 0.f;
                        x[e] = pos ? __fdiv_rn(x[e], rep) : __fmul_rn(x[e], rep);
                    }
                    if (!GRAD) {
                        x[e] = __fsub_rn(x[e], __fmul_rn(freq, static_cast<float>(c)));
                        if (c > 0) x[e] = __fsub_rn(x[e], pres);
                        if (has_bias) x[e] = __fadd_rn(x[e], bias[v - v0 + e]);
                    }
                }
                x4 = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                pack_bf16x2(x[6], x[7]));
            }
            if (ms[q] != 0xffu) {
                uint32_t w[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t keep = 0xffffu << (16 * (e & 1));
                    if (!(ms[q] >> e & 1u)) w[e >> 1] = (w[e >> 1] & ~keep) | (static_cast<uint32_t>(mval) << (16 * (e & 1)));
                }
                x4 = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (GRAD) {
                store8<ALIGNED>(static_cast<uint16_t*>(a.dlogits) + off, v, V, x4);
            } else {
                if (a.out) store8<ALIGNED>(a.out + off, v, V, x4);
                if (want_arg) {
                    if (!ALIGNED && v + 8 > V) {   // the mask wrote over the padding behind V
                        uint32_t w[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (v + e >= V) w[e >> 1] |= 0x7fffu << (16 * (e & 1));
                        x4 = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    const float m = max8_bf16(x4);
                    if (best_at < 0 || m > best_m || (best_m != best_m && m == m)) {
                        best = x4;
                        best_m = m;
                        best_at = v;
                    }
                }
            }
        }
        if (want_arg) {
            const unsigned long long key = warp_best_key(best_at >= 0, best, best_at);
            if (lane == 0) s.key[t >> 5][j - j0] = key;
        }
    }
    if (!want_arg) return;
    // one atomic maximum per row and CTA (a maximum does not depend on the order); the last CTA of
    // the sequence turns the keys into ids and leaves the workspace zero
    __syncthreads();
    if (t < j1 - j0) {
        unsigned long long key = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) key = max(key, s.key[w][t]);
        if (key) atomicMax(&p.key[static_cast<size_t>(b) * a.n + j0 + t], key);
        __threadfence();
    }
    __syncthreads();
    if (t == 0) s.last = atomicAdd(&p.ticket[b], 1u) == gridDim.x * gridDim.z - 1;
    __syncthreads();
    if (!s.last) return;
    __threadfence();
    if (t < a.n) {
        const size_t row = static_cast<size_t>(b) * a.n + t;
        a.argmax[row] = argmax_id(__ldcg(&p.key[row]));
        p.key[row] = 0ull;
    }
    if (t == 0) p.ticket[b] = 0u;
}

template <bool GRAD, bool F32, bool ALIGNED, int NV>
cudaError_t launch(const LogitsParams& p, dim3 grid, cudaStream_t st) {
    const size_t words = static_cast<size_t>(p.chunk) + p.chunk / 32 + (!GRAD && p.a.n_bias > 0 ? p.chunk : 0);
    logits_process_kernel<GRAD, F32, ALIGNED, NV><<<grid, kThreads, words * 4, st>>>(p);
    return cudaGetLastError();
}

template <bool GRAD, bool F32, int NV>
cudaError_t launch_al(const LogitsParams& p, dim3 grid, cudaStream_t st) {
    return p.aligned ? launch<GRAD, F32, true, NV>(p, grid, st) : launch<GRAD, F32, false, NV>(p, grid, st);
}

}  // namespace

int launch_logits_process(const LogitsParams& in, bool grad, void* stream) {
    LogitsParams p = in;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.chunk = 8 * kThreads;
    p.rows_per_cta = p.a.n;
    const dim3 grid((p.a.V + p.chunk - 1) / p.chunk, p.a.B, (p.a.n + p.rows_per_cta - 1) / p.rows_per_cta);
    cudaError_t e;
    if (!grad) e = launch_al<false, false, 1>(p, grid, st);
    else if (p.a.grad_fp32) e = launch_al<true, true, 1>(p, grid, st);
    else e = launch_al<true, false, 1>(p, grid, st);
    return static_cast<int>(e);
}

}  // namespace svd
