// tree_device.cuh -- device-side pieces shared by the operators on a tree of drafts.
#pragma once

#include "svd_device.cuh"
#include "tree_internal.h"

namespace svd {

// Ancestor sets (node j's own bit included) of the n <= 64 nodes of one sequence, by threads
// t < n: each walks up its own chain, which ends because a parent lies below its node.  `s_parent`
// holds the checked parents and must be visible to the caller's warps already.
__device__ __forceinline__ unsigned long long ancestors_of(const int8_t* s_parent, int j) {
    unsigned long long m = 0;
    for (int i = j; i >= 0; i = s_parent[i]) m |= 1ull << i;
    return m;
}

// Parent of node j as the call gave it: in [-1, j), else -1 with the error recorded.
__device__ __forceinline__ int checked_parent(const int32_t* parent, size_t row, int j,
                                              uint32_t* status) {
    const int p = parent ? __ldg(parent + row + j) : j - 1;
    if (p >= -1 && p < j) return p;
    set_device_error(status, SVD_ERR_TREE);
    return -1;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Generic-proxy accesses to shared memory before this are ordered before the async proxy's after it.
__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// A key that orders bf16 values (no NaN; -0 is taken as +0) and, among equal ones, lower ids first.
__device__ __forceinline__ unsigned long long argmax_key(float v, int id) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return (static_cast<unsigned long long>(o) << 32) | static_cast<uint32_t>(~id);
}
// 0 (no value but NaN was seen) gives id 0.
__device__ __forceinline__ int argmax_id(unsigned long long key) {
    return key == 0ull ? 0 : static_cast<int>(~static_cast<uint32_t>(key));
}

// Warp-wide: the key of the warp's best value over the vectors (`best`, ids from `at`) that its
// lanes hold; 0 if there is none.  `has` is false for lanes without a vector.
__device__ __forceinline__ unsigned long long warp_best_key(bool has, const uint4& best, int at) {
    const float m = has ? max8_bf16(best) : -INFINITY;
    const bool num = has && m == m;
    const unsigned any = __ballot_sync(0xffffffffu, num);
    if (any == 0u) return 0ull;
    const float top = redux_max_f32(num ? m : -INFINITY);
    const bool win = num && m == top;
    const uint32_t id = win ? static_cast<uint32_t>(at + first_pos(best, top)) : 0xffffffffu;
    return argmax_key(top, static_cast<int>(redux_min_u32(id)));
}

}  // namespace svd
