/* svd_tree.h -- C ABI of the operators around the verification of a TREE of drafted tokens: the
 * target's attention for the drafted nodes over a paged cache, the processing of the logits before
 * the decision (penalties, biases, grammar masks) with its gradient, the acceptance over the tree,
 * and the append of the accepted path to the cache.
 *
 * A chain of k drafts is the tree with n = k + 1 nodes 0 -> 1 -> ... -> k, which is what
 * svd_verify (svd.h) decides from D, T; the pages that describe the method verify chains, and
 * the tree is this library's extension of them.
 *
 * The tree of one sequence
 *   - n <= SVD_TREE_MAX_NODES nodes; parent[b, j] is the parent of node j: -1 (none) or a node
 *     below j.  parent == NULL means the chain parent[b, j] = j - 1.
 *   - anc(j) is node j and every node on the way up from it.  Node 0 is the root: the token that
 *     was emitted last and is not yet in the cache.  Row j of the logits is the target's
 *     distribution after node j.
 *   - n_nodes[b] <= n nodes are in use (NULL: all n); the others are padding.
 *   - A parent outside [-1, j) of a node in use counts as -1 and records SVD_ERR_TREE; parents of
 *     padding nodes are not read.  (The processing of logits has no n_nodes: all its nodes are in use.)
 *
 * The paged cache
 *   - cache_k and cache_v hold n_pages pages of page_size tokens, [page_size, Hkv, D] each,
 *     page_stride_k / page_stride_v elements apart (page_size * Hkv * D when pages are
 *     contiguous; twice that where K and V pages alternate in one buffer).
 *   - Token t of sequence b is row t % page_size of page page_table[b, t / page_size].
 *   - cache_len[b] tokens are in the cache.  Lengths outside [0, max_pages * page_size] are
 *     clamped, and page ids outside [0, n_pages) are read as page 0 (attention) or skipped
 *     (append); both record SVD_ERR_PAGE_RANGE.
 *   - Rows of a page behind cache_len are never used, whatever they hold.
 *   - max_pages * page_size <= 2^30.
 *
 * Conventions as in svd.h: device pointers, row-major and contiguous unless a stride is given,
 * every call enqueues on `stream` and never synchronizes, argument errors are returned before any
 * launch, device errors go to the workspace's status word (svd_get_device_error).  The current
 * device must be the one that holds the tensors.  A workspace must be zero before its first use
 * and is left ready for the next call, after a device error too; calls that share one must not
 * overlap on the GPU, so two captured graphs that may run at the same time need two.  Outputs lie
 * apart from inputs and from each other, except where a call says that they may be the same.
 */
#ifndef SVD_TREE_H
#define SVD_TREE_H

#include "svd.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SVD_TREE_MAX_NODES 64

typedef enum svd_dtype {
    SVD_BF16 = 0,
    SVD_FP16 = 1
} svd_dtype;

/* ---------------------------------------------------------------------------------------------
 * Attention of the drafted nodes over the cache and over each other.
 *   s_t = scale * q[b, j, h] . K_t  over the cached tokens t < cache_len[b] and the nodes of anc(j)
 *   out[b, j, h] = sum_t softmax(s)_t V_t,   lse[b, j, h] = log sum_t exp(s_t)
 * Query head h reads key head h / (Hq / Hkv).  With n = 1 it is the attention of a decode step.
 * The nodes' own keys and values are k_new, v_new: they need not be in the cache, and a node that
 * is not in anc(j) has no influence on row j, whatever it holds.  Rows of padding nodes get
 * out = 0 and lse = -inf.
 * Scores, maxima, sums, lse and accumulators are fp32.  The softmax weights are rounded once to the
 * tensors' 16-bit type for the product with V, as out is: on random inputs the two roundings leave
 * 2.3e-3 of the result's norm in bf16 where out's alone leaves 1.7e-3, in fp16 2.9e-4 and 2.1e-4.
 * fp16 weights keep the type's precision down to 2^-21 of the row's largest, and are off by at most
 * 2^-32 of it below.  A visible element of v_new that is infinite or NaN makes its element of out
 * so, however small its weight; one of the cache is multiplied as it is (0 * inf is NaN).
 * Limits: 1 <= n <= 64, Hq % Hkv == 0, Hq <= 1024, D % 8 == 0, 8 <= D <= 128, page_size a power
 * of two >= 8; pointers 16-byte aligned, page strides multiples of 8 elements.
 * --------------------------------------------------------------------------------------------- */
typedef struct svd_tree_attention_args {
    const void* q;              /* [B, n, Hq, D]                                               */
    const void* k_new;          /* [B, n, Hkv, D]                                              */
    const void* v_new;          /* [B, n, Hkv, D]                                              */
    const void* cache_k;        /* pages, see above; may be NULL when n_pages == 0             */
    const void* cache_v;
    int64_t page_stride_k;      /* elements                                                    */
    int64_t page_stride_v;
    const int32_t* page_table;  /* [B, max_pages]; may be NULL when max_pages == 0             */
    const int32_t* cache_len;   /* [B]                                                         */
    const int32_t* parent;      /* [B, n] or NULL (chain)                                      */
    const int32_t* n_nodes;     /* [B] or NULL (all n)                                         */
    int B, n, Hq, Hkv, D;
    int n_pages, page_size, max_pages;
    svd_dtype dtype;            /* of q, k_new, v_new, the cache and out                       */
    float scale;                /* at most 2^127 in size                                       */
    void* out;                  /* [B, n, Hq, D]                                               */
    float* lse;                 /* [B, n, Hq] or NULL                                          */
} svd_tree_attention_args;

size_t svd_tree_attention_workspace_bytes(int B, int n, int Hq, int Hkv, int D);

svd_status svd_tree_attention(const svd_tree_attention_args* args, void* ws, size_t ws_bytes,
                              void* stream);

/* ---------------------------------------------------------------------------------------------
 * Logits processing for every row j of every sequence: with x a raw logit of id v,
 *   c    = how often v is among the generated tokens history[b, prompt_len .. hist_len) and the
 *          tokens node_tok[b, i], i in anc(j)
 *   seen = c > 0, or v is in the prompt history[b, 0 .. prompt_len)
 *   x1 = seen ? (x > 0 ? x / repetition[b] : x * repetition[b]) : x
 *   z  = x1 - frequency[b] * c - (c > 0 ? presence[b] : 0) + (sum of bias_val[b, i] with bias_tok[b, i] == v)
 *   out = mask bit of v is set (or mask == NULL) ? z : mask_value
 * evaluated in this order in fp32 and rounded once to bf16; argmax[b, j] is the lowest id of the
 * largest rounded value (0 if every value is NaN).  out may be logits itself (in place).
 * Ids of -1 in history, node_tok and bias_tok are padding; other ids outside [0, V) are left out
 * and record SVD_ERR_TOKEN_RANGE.  svd_verify and svd_verify_distill want finite logits: give them
 * a finite mask_value (SVD_MASK_VALUE).  A row whose mask leaves nothing is all mask_value.
 * Penalties and biases are finite.
 * The gradient with respect to the raw logits, with the counts and the mask of the same lists:
 *   dlogits = masked ? 0 : seen ? (x > 0 ? dz / repetition : dz * repetition) : dz
 * dlogits may be dz itself.
 * Lengths outside [0, hist_stride], and a prompt longer than the history, are clamped.
 * Limits: B <= 65535, 1 <= n <= 64, 1 <= V <= 327680, hist_stride < 2^23, n_bias <= 4096, n_bias ids of one
 * sequence may repeat (their values add in list order).  V % 8 == 0 with 16-byte aligned logits,
 * out, dz and dlogits takes the fast path.
 * --------------------------------------------------------------------------------------------- */
#define SVD_MASK_VALUE (-32768.0f)

typedef struct svd_logits_process_args {
    const uint16_t* logits;     /* [B, n, V] bf16                                              */
    int B, n, V;
    const int32_t* history;     /* [B, hist_stride] or NULL                                    */
    int hist_stride;
    const int32_t* prompt_len;  /* [B] or NULL (0)                                             */
    const int32_t* hist_len;    /* [B] or NULL (hist_stride)                                   */
    const int32_t* node_tok;    /* [B, n] or NULL                                              */
    const int32_t* parent;      /* [B, n] or NULL (chain)                                      */
    const float* repetition;    /* [B] > 0, or NULL (1)                                        */
    const float* frequency;     /* [B] or NULL (0)                                             */
    const float* presence;      /* [B] or NULL (0)                                             */
    const int32_t* bias_tok;    /* [B, n_bias] or NULL                                         */
    const float* bias_val;      /* [B, n_bias]                                                 */
    int n_bias;
    const uint32_t* mask;       /* [B, mask_rows, ceil(V / 32)] or NULL: bit v % 32 of word v / 32 */
    int mask_rows;              /* 1 (one mask for the sequence's rows) or n                   */
    float mask_value;           /* not NaN                                                     */
    uint16_t* out;              /* [B, n, V] bf16, or NULL when only argmax is wanted          */
    int32_t* argmax;            /* [B, n] or NULL                                              */
    const void* dz;             /* gradient call: [B, n, V] bf16 or fp32                       */
    void* dlogits;              /* gradient call: the same type                                */
    int grad_fp32;              /* gradient call: 0 bf16, 1 fp32                               */
} svd_logits_process_args;

size_t svd_logits_process_workspace_bytes(int B, int n);

svd_status svd_logits_process(const svd_logits_process_args* args, void* ws, size_t ws_bytes,
                              void* stream);

/* Uses logits, the lists, repetition, parent, mask, dz, dlogits and grad_fp32. */
svd_status svd_logits_process_grad(const svd_logits_process_args* args, void* ws, size_t ws_bytes,
                                   void* stream);

/* ---------------------------------------------------------------------------------------------
 * Greedy acceptance over a tree.  y_j = argmax T[b, j] (lowest id on ties), or target_tok[b, j] where
 * the caller has the target's choice already (svd_logits_process's argmax, a sampler's draw).
 * From node 0: while some child c of the current node has node_tok[b, c] == y of that node, step to
 * the lowest such child; path lists the nodes stepped on, node 0 first.
 *   n_path = nodes on the path, accept_len = n_path - 1 drafts accepted (0 if n_path is 0),
 *   emitted = the accepted drafts' tokens, then y of the last node; n_emitted = n_path.
 * path and emitted are padded with -1.  Sequences with n_nodes[b] = 0 have an empty path.  On a
 * chain the result is that of svd_verify with b_k = k, kt = k + 1.  node_tok ids outside [0, V) other
 * than -1 match nothing and, where T is given, record SVD_ERR_TOKEN_RANGE; node 0's is not read.
 * Limits: B <= 65535, 1 <= n <= 64, 1 <= V <= 327680.  Sampled acceptance is the caller's: draw target_tok.
 * --------------------------------------------------------------------------------------------- */
typedef struct svd_tree_verify_args {
    const uint16_t* T;          /* [B, n, V] bf16, or NULL with target_tok                     */
    const int32_t* target_tok;  /* [B, n] or NULL with T                                       */
    const int32_t* node_tok;    /* [B, n]                                                      */
    const int32_t* parent;      /* [B, n] or NULL (chain)                                      */
    const int32_t* n_nodes;     /* [B] or NULL (all n)                                         */
    int B, n, V;                /* V is not used with target_tok                               */
    int32_t* target_argmax;     /* [B, n] or NULL: y                                           */
    int32_t* path;              /* [B, n]                                                      */
    int32_t* n_path;            /* [B]                                                         */
    int32_t* accept_len;        /* [B]                                                         */
    int32_t* emitted;           /* [B, n]                                                      */
    int32_t* n_emitted;         /* [B]                                                         */
} svd_tree_verify_args;

size_t svd_tree_verify_workspace_bytes(int B, int n);

svd_status svd_tree_verify(const svd_tree_verify_args* args, void* ws, size_t ws_bytes,
                           void* stream);

/* ---------------------------------------------------------------------------------------------
 * Append of new keys and values to the paged cache: entry i < count[b] of sequence b is node
 * path[b, i] of k_new, v_new (node i where path is NULL, as for a prompt) and becomes token
 * cache_len[b] + i.  new_len[b] = cache_len[b] + count[b] (at most the capacity); new_len may be
 * cache_len itself.  The elements are 16 bits wide and are copied as they are.  Entries whose node,
 * page or position is out of range are skipped and recorded (SVD_ERR_TREE, SVD_ERR_PAGE_RANGE).
 * No slot may be named twice by one call (pages shared by sequences end in front of cache_len).
 * Limits: B <= 65535, n >= 1, page_size >= 1, Hkv * D % 8 == 0; pointers 16-byte aligned, page strides multiples
 * of 8 elements.
 * --------------------------------------------------------------------------------------------- */
typedef struct svd_cache_append_args {
    const void* k_new;          /* [B, n, Hkv, D]                                              */
    const void* v_new;
    void* cache_k;
    void* cache_v;
    int64_t page_stride_k;
    int64_t page_stride_v;
    const int32_t* page_table;  /* [B, max_pages]                                              */
    const int32_t* cache_len;   /* [B]                                                         */
    const int32_t* count;       /* [B]; clamped to [0, n]                                      */
    const int32_t* path;        /* [B, n] or NULL                                              */
    int B, n, Hkv, D;
    int n_pages, page_size, max_pages;
    int32_t* new_len;           /* [B] or NULL                                                 */
} svd_cache_append_args;

size_t svd_cache_append_workspace_bytes(int B);

svd_status svd_cache_append(const svd_cache_append_args* args, void* ws, size_t ws_bytes,
                            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SVD_TREE_H */
