// tree_api.cu -- C ABI of include/svd_tree.h: argument checks, workspace carving, launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "tree_internal.h"

using namespace svd;

namespace {

constexpr int kMaxV = 327680;
constexpr int kMaxBias = 4096;
constexpr int kMaxHistory = 1 << 23;   // counts are kept in 23 bits
constexpr int kMaxGridYZ = 65535;
constexpr int64_t kMaxTokens = 1 << 30;        // of one sequence's page table
constexpr int64_t kMaxStride = 1ll << 39;      // elements: a tensor map's strides stay below 2^40 bytes

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
svd_status from_cuda(int err) { return err == 0 ? SVD_OK : SVD_ERR_CUDA; }

svd_status check_ws(void* ws, size_t ws_bytes, size_t need) {
    if (ws == nullptr) return SVD_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return SVD_ERR_ALIGNMENT;
    if (ws_bytes < need) return SVD_ERR_WORKSPACE;
    return SVD_OK;
}

template <class T>
T* at(void* ws, size_t off) {
    return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// Checks the lists that the processing and its gradient share.
svd_status check_lists(const svd_logits_process_args* a) {
    if (a->B < 0 || a->n < 1 || a->n > kTreeMaxNodes || a->V < 1) return SVD_ERR_INVALID_ARG;
    if (a->V > kMaxV || a->B > kMaxGridYZ) return SVD_ERR_UNSUPPORTED;
    if (a->history && (a->hist_stride < 0 || a->hist_stride >= kMaxHistory)) return SVD_ERR_INVALID_ARG;
    if (a->bias_tok && (!a->bias_val || a->n_bias < 0 || a->n_bias > kMaxBias)) return SVD_ERR_INVALID_ARG;
    if (a->mask && a->mask_rows != 1 && a->mask_rows != a->n) return SVD_ERR_INVALID_ARG;
    return SVD_OK;
}

svd_status run_logits(const svd_logits_process_args* a, bool grad, bool aligned, void* ws,
                      size_t ws_bytes, void* stream) {
    const LogitsWs L = logits_ws(a->B, a->n);
    const svd_status s = check_ws(ws, ws_bytes, L.total);
    if (s != SVD_OK) return s;
    LogitsParams p;
    std::memset(&p, 0, sizeof p);
    p.a = *a;
    if (!p.a.history) p.a.hist_stride = 0;
    if (!p.a.bias_tok) p.a.n_bias = 0;
    p.aligned = aligned ? 1 : 0;
    p.status = at<uint32_t>(ws, 0);
    p.key = at<unsigned long long>(ws, L.key);
    p.ticket = at<uint32_t>(ws, L.ticket);
    return from_cuda(launch_logits_process(p, grad, stream));
}

// Page geometry shared by attention and append (the page table of no sequences is empty).
bool bad_pages(int B, int n_pages, int page_size, int max_pages, const void* ck, const void* cv,
               const int32_t* table, int64_t sk, int64_t sv, int64_t page_elems) {
    if (n_pages < 0 || max_pages < 0 || page_size < 1) return true;
    if (static_cast<int64_t>(max_pages) * page_size > kMaxTokens) return true;
    if (B > 0 && max_pages > 0 && !table) return true;
    if (n_pages > 0 && (!ck || !cv)) return true;
    // pages that overlap or lie backwards make no cache
    if (n_pages > 1 && (sk < page_elems || sv < page_elems)) return true;
    return false;
}

}  // namespace

extern "C" {

size_t svd_tree_attention_workspace_bytes(int B, int n, int Hq, int Hkv, int D) {
    if (B < 0 || n < 1 || n > kTreeMaxNodes || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || D < 1) return 0;
    return tree_attention_ws_bytes(B, n, Hq, Hkv, D);
}

svd_status svd_tree_attention(const svd_tree_attention_args* a, void* ws, size_t ws_bytes,
                              void* stream) {
    if (!a) return SVD_ERR_INVALID_ARG;
    if (a->B < 0 || a->n < 1 || a->n > kTreeMaxNodes || a->Hkv < 1 || a->Hq < 1 || a->Hq % a->Hkv != 0 || a->D < 1)
        return SVD_ERR_INVALID_ARG;
    if (a->dtype != SVD_BF16 && a->dtype != SVD_FP16) return SVD_ERR_INVALID_ARG;
    if (!(std::fabs(a->scale) <= 0x1p127f)) return SVD_ERR_INVALID_ARG;   // scale * log2(e) stays finite
    if (bad_pages(a->B, a->n_pages, a->page_size, a->max_pages, a->cache_k, a->cache_v, a->page_table,
                  a->page_stride_k, a->page_stride_v,
                  static_cast<int64_t>(a->page_size) * a->Hkv * a->D))
        return SVD_ERR_INVALID_ARG;
    if (a->page_stride_k >= kMaxStride || a->page_stride_v >= kMaxStride ||
        static_cast<int64_t>(a->page_size) * a->Hkv * a->D >= kMaxStride)
        return SVD_ERR_UNSUPPORTED;
    if (a->D > 128 || a->D % 8 != 0 || a->Hq > 1024 || a->page_size < 8 || (a->page_size & (a->page_size - 1)) != 0)
        return SVD_ERR_UNSUPPORTED;
    if (a->B == 0) return SVD_OK;
    if (!a->q || !a->k_new || !a->v_new || !a->cache_len || !a->out) return SVD_ERR_INVALID_ARG;
    if (!aligned16(a->q) || !aligned16(a->k_new) || !aligned16(a->v_new) || !aligned16(a->out) ||
        !aligned16(a->cache_k) || !aligned16(a->cache_v) || a->page_stride_k % 8 != 0 || a->page_stride_v % 8 != 0)
        return SVD_ERR_ALIGNMENT;
    const svd_status s = check_ws(ws, ws_bytes, tree_attention_ws_bytes(a->B, a->n, a->Hq, a->Hkv, a->D));
    if (s != SVD_OK) return s;
    return from_cuda(launch_tree_attention(*a, ws, stream));
}

size_t svd_logits_process_workspace_bytes(int B, int n) {
    return B < 0 || n < 1 || n > kTreeMaxNodes ? 0 : logits_ws(B, n).total;
}

svd_status svd_logits_process(const svd_logits_process_args* a, void* ws, size_t ws_bytes, void* stream) {
    if (!a) return SVD_ERR_INVALID_ARG;
    const svd_status s = check_lists(a);
    if (s != SVD_OK) return s;
    if (std::isnan(a->mask_value)) return SVD_ERR_INVALID_ARG;
    if (a->B == 0) return SVD_OK;
    if (!a->logits || (!a->out && !a->argmax)) return SVD_ERR_INVALID_ARG;
    return run_logits(a, false, a->V % 8 == 0 && aligned16(a->logits) && aligned16(a->out), ws, ws_bytes, stream);
}

svd_status svd_logits_process_grad(const svd_logits_process_args* a, void* ws, size_t ws_bytes, void* stream) {
    if (!a) return SVD_ERR_INVALID_ARG;
    const svd_status s = check_lists(a);
    if (s != SVD_OK) return s;
    if (a->grad_fp32 != 0 && a->grad_fp32 != 1) return SVD_ERR_INVALID_ARG;
    if (a->B == 0) return SVD_OK;
    if (!a->logits || !a->dz || !a->dlogits) return SVD_ERR_INVALID_ARG;
    return run_logits(a, true, a->V % 8 == 0 && aligned16(a->logits) && aligned16(a->dz) && aligned16(a->dlogits), ws,
                      ws_bytes, stream);
}

size_t svd_tree_verify_workspace_bytes(int B, int n) { return svd_logits_process_workspace_bytes(B, n); }

svd_status svd_tree_verify(const svd_tree_verify_args* a, void* ws, size_t ws_bytes, void* stream) {
    if (!a) return SVD_ERR_INVALID_ARG;
    if (a->B < 0 || a->n < 1 || a->n > kTreeMaxNodes || (a->T && a->V < 1)) return SVD_ERR_INVALID_ARG;
    if ((a->T && a->V > kMaxV) || a->B > kMaxGridYZ) return SVD_ERR_UNSUPPORTED;
    if (a->T && a->target_tok) return SVD_ERR_INVALID_ARG;
    if (a->B == 0) return SVD_OK;
    if ((!a->T && !a->target_tok) || !a->node_tok || !a->path || !a->n_path || !a->accept_len || !a->emitted ||
        !a->n_emitted)
        return SVD_ERR_INVALID_ARG;
    const LogitsWs L = logits_ws(a->B, a->n);
    const svd_status s = check_ws(ws, ws_bytes, L.total);
    if (s != SVD_OK) return s;
    VerifyParams p;
    std::memset(&p, 0, sizeof p);
    p.a = *a;
    p.aligned = a->T && a->V % 8 == 0 && aligned16(a->T) ? 1 : 0;
    p.status = at<uint32_t>(ws, 0);
    p.key = at<unsigned long long>(ws, L.key);
    p.ticket = at<uint32_t>(ws, L.ticket);
    return from_cuda(launch_tree_verify(p, stream));
}

size_t svd_cache_append_workspace_bytes(int B) {
    return B < 0 ? 0 : align256(sizeof(WsHeader) + sizeof(uint32_t) * static_cast<size_t>(B));
}

svd_status svd_cache_append(const svd_cache_append_args* a, void* ws, size_t ws_bytes, void* stream) {
    if (!a) return SVD_ERR_INVALID_ARG;
    if (a->B < 0 || a->n < 1 || a->Hkv < 1 || a->D < 1) return SVD_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(a->Hkv) * a->D;
    if (row > (1 << 24) || row % 8 != 0 || a->B > kMaxGridYZ) return SVD_ERR_UNSUPPORTED;
    if (bad_pages(a->B, a->n_pages, a->page_size, a->max_pages, a->cache_k, a->cache_v, a->page_table,
                  a->page_stride_k, a->page_stride_v, a->page_size * row))
        return SVD_ERR_INVALID_ARG;
    if (a->B == 0) return SVD_OK;
    if (!a->k_new || !a->v_new || !a->cache_len || !a->count) return SVD_ERR_INVALID_ARG;
    if (!aligned16(a->k_new) || !aligned16(a->v_new) || !aligned16(a->cache_k) || !aligned16(a->cache_v) ||
        a->page_stride_k % 8 != 0 || a->page_stride_v % 8 != 0)
        return SVD_ERR_ALIGNMENT;
    const svd_status s = check_ws(ws, ws_bytes, svd_cache_append_workspace_bytes(a->B));
    if (s != SVD_OK) return s;
    AppendParams p;
    std::memset(&p, 0, sizeof p);
    p.a = *a;
    p.status = at<uint32_t>(ws, 0);
    p.ticket = at<uint32_t>(ws, sizeof(WsHeader));
    return from_cuda(launch_cache_append(p, stream));
}

}  // extern "C"
