// tree_attention.cu -- attention of the nodes of a tree of drafts over a paged cache and over each
// other (include/svd_tree.h).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "tree_device.cuh"

namespace svd {

namespace {

constexpr int kThreads = 128;

template <bool FP16>
__device__ __forceinline__ void load4(const void* base, size_t at, float (&x)[4]) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
    if (FP16) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
        x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    } else {
        x[0] = bf_lo(w.x); x[1] = bf_hi(w.x); x[2] = bf_lo(w.y); x[3] = bf_hi(w.y);
    }
}

// One warp per row (b, j, h): a pass over the keys with the running maximum and sum; lane l holds
// elements 4 l .. 4 l + 3 of the head.
template <bool FP16>
__global__ void __launch_bounds__(kThreads) tree_attention_rows(svd_tree_attention_args a, uint32_t* status) {
    const int lane = threadIdx.x & 31;
    const long long r = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (r >= static_cast<long long>(a.B) * a.n * a.Hq) return;
    const int h = static_cast<int>(r % a.Hq), j = static_cast<int>(r / a.Hq % a.n);
    const int b = static_cast<int>(r / a.Hq / a.n), hk = h / (a.Hq / a.Hkv);
    const bool act = lane * 4 < a.D;
    float q[4] = {0, 0, 0, 0}, o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.f;
    if (act) load4<FP16>(a.q, static_cast<size_t>(r) * a.D + lane * 4, q);
    auto key = [&](const void* kb, const void* vb, size_t ak, size_t av) {
        float k[4] = {0, 0, 0, 0}, v[4] = {0, 0, 0, 0};
        if (act) { load4<FP16>(kb, ak + lane * 4, k); load4<FP16>(vb, av + lane * 4, v); }
        const float s = warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]) * a.scale;
        const float mn = fmaxf(m, s), c = m > -INFINITY ? __expf(m - mn) : 0.f, p = __expf(s - mn);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = o[e] * c + p * v[e];
        m = mn;
    };
    const int used = a.n_nodes ? a.n_nodes[b] : a.n;
    if (j < used) {
        const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
        long long len = a.cache_len[b];
        if (len < 0 || len > cap) { set_device_error(status, SVD_ERR_PAGE_RANGE); len = len < 0 ? 0 : cap; }
        if (a.n_pages == 0) len = 0;
        for (int t = 0; t < len; ++t) {
            int pg = a.page_table[static_cast<size_t>(b) * a.max_pages + t / a.page_size];
            if (pg < 0 || pg >= a.n_pages) { set_device_error(status, SVD_ERR_PAGE_RANGE); pg = 0; }
            const size_t in = (static_cast<size_t>(t % a.page_size) * a.Hkv + hk) * a.D;
            key(a.cache_k, a.cache_v, static_cast<size_t>(pg) * a.page_stride_k + in,
                static_cast<size_t>(pg) * a.page_stride_v + in);
        }
        for (int i = j; i >= 0; i = checked_parent(a.parent, static_cast<size_t>(b) * a.n, i, status)) {
            const size_t at = ((static_cast<size_t>(b) * a.n + i) * a.Hkv + hk) * a.D;
            key(a.k_new, a.v_new, at, at);
        }
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    if (act) {
        uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<size_t>(r) * a.D + lane * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            out[e] = FP16 ? __half_as_ushort(__float2half_rn(o[e] * inv)) : __bfloat16_as_ushort(__float2bfloat16_rn(o[e] * inv));
    }
    if (a.lse && lane == 0) a.lse[r] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t tree_attention_ws_bytes(int, int, int, int, int) { return sizeof(WsHeader); }

int launch_tree_attention(const svd_tree_attention_args& a, void* ws, void* stream) {
    const long long rows = static_cast<long long>(a.B) * a.n * a.Hq;
    const int per = kThreads / 32;
    const unsigned grid = static_cast<unsigned>((rows + per - 1) / per);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a.dtype == SVD_FP16) tree_attention_rows<true><<<grid, kThreads, 0, st>>>(a, static_cast<uint32_t*>(ws));
    else tree_attention_rows<false><<<grid, kThreads, 0, st>>>(a, static_cast<uint32_t*>(ws));
    return static_cast<int>(cudaGetLastError());
}

}  // namespace svd
