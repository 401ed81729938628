// cache_append.cu -- append of new keys and values to the paged cache (include/svd_tree.h).
//
// A copy of 16-bit rows to the slots that the page table names: every byte is read once and written
// once.  One warp per entry copies its K and its V row in 16-byte vectors.
#include <cuda_runtime.h>

#include "tree_device.cuh"

namespace svd {

namespace {

constexpr int kThreads = 128;
constexpr int kEntries = kThreads / 32;   // per CTA

__global__ void __launch_bounds__(kThreads) cache_append_kernel(AppendParams p) {
    const svd_cache_append_args& a = p.a;
    const int b = blockIdx.y, t = threadIdx.x, lane = t & 31;
    const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
    // volatile: new_len may be cache_len itself, written by the sequence's last CTA
    const int len0 = *(const volatile int32_t*)(a.cache_len + b);
    const int cnt0 = *(const volatile int32_t*)(a.count + b);
    const int cnt = cnt0 < 0 ? 0 : (cnt0 > a.n ? a.n : cnt0);
    const long long len = len0 < 0 ? 0 : (len0 > cap ? cap : len0);
    const bool fits = len + cnt <= cap;
    if (t == 0 && blockIdx.x == 0) {
        if (len != len0 || !fits) set_device_error(p.status, SVD_ERR_PAGE_RANGE);
        if (cnt != cnt0) set_device_error(p.status, SVD_ERR_TREE);
    }
    const int i = blockIdx.x * kEntries + (t >> 5);
    if (i < cnt && len + i < cap) {
        int node = a.path ? __ldg(a.path + static_cast<size_t>(b) * a.n + i) : i;
        const int pos = static_cast<int>(len + i);
        const int page = __ldg(a.page_table + static_cast<size_t>(b) * a.max_pages + pos / a.page_size);
        if (node < 0 || node >= a.n) {
            if (lane == 0) set_device_error(p.status, SVD_ERR_TREE);
        } else if (page < 0 || page >= a.n_pages) {
            if (lane == 0) set_device_error(p.status, SVD_ERR_PAGE_RANGE);
        } else {
            const int vecs = a.Hkv * a.D / 8;
            const size_t src = (static_cast<size_t>(b) * a.n + node) * vecs;
            const size_t in_page = static_cast<size_t>(pos % a.page_size) * vecs;
            const uint4* ks = static_cast<const uint4*>(a.k_new) + src;
            const uint4* vs = static_cast<const uint4*>(a.v_new) + src;
            uint4* kd = static_cast<uint4*>(a.cache_k) + static_cast<size_t>(page) * (a.page_stride_k / 8) + in_page;
            uint4* vd = static_cast<uint4*>(a.cache_v) + static_cast<size_t>(page) * (a.page_stride_v / 8) + in_page;
            // eight loads in flight before the first store (the stores could alias, so the compiler keeps order)
            for (int c0 = lane; c0 < vecs; c0 += 128) {
                uint4 x[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c0 + 32 * i < vecs) {
                        x[i] = __ldcs(ks + c0 + 32 * i);
                        y[i] = __ldcs(vs + c0 + 32 * i);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c0 + 32 * i < vecs) {
                        kd[c0 + 32 * i] = x[i];
                        vd[c0 + 32 * i] = y[i];
                    }
            }
        }
    }
    if (!a.new_len) return;
    // the sequence's last CTA writes the length, when every CTA has read the old one
    __syncthreads();
    if (t == 0) {
        __threadfence();
        if (atomicAdd(&p.ticket[b], 1u) == gridDim.x - 1) {
            p.ticket[b] = 0u;
            a.new_len[b] = static_cast<int32_t>(fits ? len + cnt : cap);
        }
    }
}

}  // namespace

int launch_cache_append(const AppendParams& p, void* stream) {
    const dim3 grid((p.a.n + kEntries - 1) / kEntries, p.a.B);
    cache_append_kernel<<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace svd
