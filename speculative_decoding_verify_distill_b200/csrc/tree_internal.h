// tree_internal.h -- kernel parameter blocks, workspace layouts and launch entry points of the
// operators in include/svd_tree.h.
#pragma once

#include "../../include/svd_tree.h"
#include "svd_internal.h"

namespace svd {

constexpr int kTreeMaxNodes = SVD_TREE_MAX_NODES;

// ------------------------------------------------------------------------------------------
// logits processing and acceptance: a key per logit row (ordered value << 32 | ~id), a ticket per
// sequence, both back at zero after the call
// ------------------------------------------------------------------------------------------
struct LogitsWs {
    size_t key, ticket, total;
};
__host__ __device__ inline LogitsWs logits_ws(int B, int n) {
    LogitsWs L;
    L.key = sizeof(WsHeader);
    L.ticket = align256(L.key + sizeof(unsigned long long) * (size_t)B * (size_t)n);
    L.total = align256(L.ticket + sizeof(uint32_t) * (size_t)B);
    return L;
}

struct LogitsParams {
    svd_logits_process_args a;
    int aligned;       // 16-byte vectors; 0: element loads and stores
    int rows_per_cta;
    uint32_t* status;
    unsigned long long* key;   // [B, n]
    uint32_t* ticket;          // [B]
};
int launch_logits_process(const LogitsParams& p, bool grad, void* stream);

struct VerifyParams {
    svd_tree_verify_args a;
    int aligned;
    uint32_t* status;
    unsigned long long* key;
    uint32_t* ticket;
};
int launch_tree_verify(const VerifyParams& p, void* stream);

// ------------------------------------------------------------------------------------------
// cache append: a ticket per sequence
// ------------------------------------------------------------------------------------------
struct AppendParams {
    svd_cache_append_args a;
    uint32_t* status;
    uint32_t* ticket;
};
int launch_cache_append(const AppendParams& p, void* stream);

// ------------------------------------------------------------------------------------------
// tree attention
// ------------------------------------------------------------------------------------------
size_t tree_attention_ws_bytes(int B, int n, int Hq, int Hkv, int D);
int launch_tree_attention(const svd_tree_attention_args& a, void* ws, void* stream);

}  // namespace svd
