// tree_verify.cu -- greedy acceptance over a tree of drafts (include/svd_tree.h).
//
// One pass over the logits for the argmax of every node's row (bound by HBM, 2 bytes a logit),
// then the walk, by the last CTA of each sequence.  The walk is no loop over the depth: a node is
// accepted where it and every node above it, up to the root, matches the target's choice at its
// parent and is the lowest such child, so the accepted set is one test of each node's ancestor bits
// against the set of matching nodes.
#include <cuda_runtime.h>

#include <cmath>

#include "tree_device.cuh"

namespace svd {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kVec = 8;                      // vectors of 8 ids per thread and row
constexpr int kChunk = 8 * kThreads * kVec;

struct WalkSmem {
    int y[kTreeMaxNodes], tok[kTreeMaxNodes];
    int8_t parent[kTreeMaxNodes];
    unsigned match[2], taken[2];
};

__device__ __forceinline__ int nodes_in_use(const svd_tree_verify_args& a, int b) {
    const int m = a.n_nodes ? __ldg(a.n_nodes + b) : a.n;
    return m < 0 ? 0 : (m > a.n ? a.n : m);
}

// The walk of sequence b by threads 0..63 (t < 64); y is the target's choice after node t.  Every
// thread of the CTA calls it.
__device__ void walk(const VerifyParams& p, int b, int y, WalkSmem& s) {
    const svd_tree_verify_args& a = p.a;
    const int t = threadIdx.x, m = nodes_in_use(a, b);
    const size_t row = static_cast<size_t>(b) * a.n;
    if (t < kTreeMaxNodes) {
        int par = -1, tok = -1;
        if (t < m) {
            par = checked_parent(a.parent, row, t, p.status);
            if (t > 0) {
                tok = __ldg(a.node_tok + row + t);
                if (tok < -1 || (a.T && tok >= a.V)) {
                    if (a.T) set_device_error(p.status, SVD_ERR_TOKEN_RANGE);
                    tok = -1;
                }
            }
        }
        s.parent[t] = static_cast<int8_t>(par);
        s.tok[t] = tok;
        s.y[t] = y;
    }
    __syncthreads();
    if (t < kTreeMaxNodes) {
        bool ok = t == 0;
        if (t > 0 && t < m && s.parent[t] >= 0 && s.tok[t] >= 0 && s.tok[t] == s.y[s.parent[t]]) {
            ok = true;
            for (int i = 1; i < t; ++i) ok = ok && !(s.parent[i] == s.parent[t] && s.tok[i] == s.tok[t]);
        }
        const unsigned w = __ballot_sync(0xffffffffu, ok && t < m);
        if ((t & 31) == 0) s.match[t >> 5] = w;
    }
    __syncthreads();
    if (t < kTreeMaxNodes) {
        const unsigned long long match = s.match[0] | static_cast<unsigned long long>(s.match[1]) << 32;
        const unsigned long long anc = ancestors_of(s.parent, t);
        const unsigned w = __ballot_sync(0xffffffffu, t < m && (anc & 1ull) && (anc & ~match) == 0ull);
        if ((t & 31) == 0) s.taken[t >> 5] = w;
    }
    __syncthreads();
    if (t < a.n) {
        const unsigned long long taken = s.taken[0] | static_cast<unsigned long long>(s.taken[1]) << 32;
        const int count = __popcll(taken);
        if (taken >> t & 1ull) {
            const int at = __popcll(taken & ((1ull << t) - 1));
            a.path[row + at] = t;
            a.emitted[row + at] = s.y[t];   // the token of the next node on the path, or the last choice
        }
        if (t >= count) {
            a.path[row + t] = -1;
            a.emitted[row + t] = -1;
        }
        if (a.target_argmax) a.target_argmax[row + t] = t < m ? s.y[t] : -1;
        if (t == 0) {
            a.n_path[b] = count;
            a.n_emitted[b] = count;
            a.accept_len[b] = count > 0 ? count - 1 : 0;
        }
    }
}

template <bool ALIGNED>
__global__ void __launch_bounds__(kThreads) tree_verify_kernel(VerifyParams p) {
    __shared__ WalkSmem s;
    __shared__ unsigned long long s_key[kWarps];
    __shared__ int s_last;
    const svd_tree_verify_args& a = p.a;
    const int t = threadIdx.x, b = blockIdx.y, j = blockIdx.z, V = a.V;
    const int v0 = blockIdx.x * kChunk;
    const size_t row = static_cast<size_t>(b) * a.n + j;
    if (j < nodes_in_use(a, b)) {
        const uint16_t* src = a.T + row * V;
        uint4 x[kVec];
#pragma unroll
        for (int q = 0; q < kVec; ++q) {
            const int v = v0 + (q * kThreads + t) * 8;
            if (ALIGNED) {
                x[q] = v < V ? __ldcs(reinterpret_cast<const uint4*>(src + v)) : make_uint4(~0u, ~0u, ~0u, ~0u);
            } else {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = v + e < V ? __ldg(src + v + e) : 0xffffu;   // NaN
                x[q] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
            }
        }
        uint4 best = x[0];
        float best_m = max8_bf16(x[0]);
        int best_at = v0 + t * 8;
#pragma unroll
        for (int q = 1; q < kVec; ++q) {
            const float m = max8_bf16(x[q]);
            if (m > best_m || (best_m != best_m && m == m)) {
                best = x[q];
                best_m = m;
                best_at = v0 + (q * kThreads + t) * 8;
            }
        }
        const unsigned long long key = warp_best_key(true, best, best_at);
        if ((t & 31) == 0) s_key[t >> 5] = key;
        __syncthreads();
        if (t == 0) {
            unsigned long long k = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) k = max(k, s_key[w]);
            if (k) atomicMax(&p.key[row], k);
        }
    }
    if (t == 0) {
        __threadfence();
        s_last = atomicAdd(&p.ticket[b], 1u) == gridDim.x * gridDim.z - 1;
        __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
    int y = -1;
    if (t < a.n) {
        unsigned long long* k = &p.key[static_cast<size_t>(b) * a.n + t];
        y = argmax_id(__ldcg(k));
        *k = 0ull;
    }
    if (t == 0) p.ticket[b] = 0u;
    walk(p, b, y, s);
}

// The target's choices are given: the walk alone.
__global__ void __launch_bounds__(kTreeMaxNodes) tree_walk_kernel(VerifyParams p) {
    __shared__ WalkSmem s;
    const int b = blockIdx.x, t = threadIdx.x;
    walk(p, b, t < p.a.n ? __ldg(p.a.target_tok + static_cast<size_t>(b) * p.a.n + t) : -1, s);
}

}  // namespace

int launch_tree_verify(const VerifyParams& p, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!p.a.T) {
        tree_walk_kernel<<<p.a.B, kTreeMaxNodes, 0, st>>>(p);
    } else {
        const dim3 grid((p.a.V + kChunk - 1) / kChunk, p.a.B, p.a.n);
        if (p.aligned) tree_verify_kernel<true><<<grid, kThreads, 0, st>>>(p);
        else tree_verify_kernel<false><<<grid, kThreads, 0, st>>>(p);
    }
    return static_cast<int>(cudaGetLastError());
}

}  // namespace svd
