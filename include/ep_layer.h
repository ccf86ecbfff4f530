/*
 * ep_layer.h -- the operators around dispatch and combine in a transformer
 * layer (same library, libep.so):
 *
 *   ep_router_topk           the router's logits -> topk_idx, topk_weights,
 *                            the inputs of ep_layout and ep_combine
 *   ep_router_topk_backward  gradient of those weights back to the logits
 *                            (ep_combine_backward's grad_topk_weights in)
 *   ep_kv_append             rotate queries and keys by position and append
 *                            keys and values to a paged cache
 *   ep_paged_attention       attention of one new token per sequence over
 *                            that cache
 *   ep_expert_w4             the experts' products on dispatched rows with
 *                            4-bit weights and group scales
 *
 * The conventions of ep.h hold: device pointers owned by the caller, work
 * enqueued on `stream` and asynchronous, arguments checked on the host before
 * anything is enqueued, every kernel launched as a programmatic dependent of
 * the one before it, no allocation and no host synchronisation, so every call
 * can be captured into a CUDA graph. None of these calls takes a handle; calls
 * on different streams or from different host threads are independent as long
 * as their outputs and workspaces are. Strides and leading dimensions count
 * elements.
 */
#ifndef EP_GB300_EP_LAYER_H
#define EP_GB300_EP_LAYER_H

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- router */

typedef enum {
    EP_SCORE_SOFTMAX = 0,      /* p = softmax over the E logits              */
    EP_SCORE_SIGMOID = 1       /* p = 1 / (1 + exp(-logit)), expert by expert */
} ep_score_t;

/* Options of the router; an all-zero struct means bf16 logits, softmax
 * scores, weights p * 0: set `scale`. */
typedef struct {
    int logits_dtype;   /* EP_DTYPE_BF16, EP_DTYPE_FP16 or EP_DTYPE_FP32       */
    int score;          /* ep_score_t                                          */
    int renormalize;    /* 0: w = scale * p; 1: w = scale * p / (sum of the
                           token's chosen p)                                   */
    float scale;        /* factor on every weight                              */
    int num_groups;     /* 0 or 1: no groups; else experts form num_groups equal
                           contiguous groups (num_groups <= 32)                */
    int topk_groups;    /* with groups: a token's experts come from this many
                           groups, those with the largest group score          */
    int group_top;      /* 0 or 1: group score = its largest key; 2: the sum of
                           its two largest keys                                */
} ep_router_config_t;

/*
 * ep_router_topk -- each token's K experts and their weights.
 *
 *  logits         device, [T, E] rows logits_ld apart (>= E). NaN and
 *                 -infinity mark an expert that the token cannot use.
 *  bias           device, fp32 [E], or NULL: added to the score for the
 *                 selection only, never to the weights.
 *  T, E, K        tokens, experts, experts per token; 1 <= E <=
 *                 EP_MAX_EXPERTS, 1 <= K <= EP_MAX_TOPK, T >= 0.
 *  topk_idx       device, int64 [T, K]: the K usable experts with the largest
 *                 keys, largest first, equal keys in ascending expert order.
 *                 The key is the logit itself; with a bias, or with group_top
 *                 2, it is p (+ bias) in fp32. Places left over (fewer usable
 *                 experts than K) hold -1, ep_layout's unused slot.
 *  topk_weights   device, fp32 [T, K]: the weights above, 0 where topk_idx is
 *                 -1. Computed in fp32; a renormalised weight is a ratio of
 *                 scores whose common factor has been taken out, so it is
 *                 defined for all finite logits.
 */
EP_API ep_status_t ep_router_topk(const void* logits, int64_t logits_ld, const float* bias, int T, int E, int K,
                                  const ep_router_config_t* config, int64_t* topk_idx, float* topk_weights,
                                  void* stream);

/*
 * ep_router_topk_backward -- grad_logits of a loss with gradient grad_weights
 * [T, K] (fp32) at topk_weights, for the experts in topk_idx ([T, K], rows
 * topk_ld >= K apart: a slice of a full sort serves). (The selection
 * itself is not differentiated; an id outside [0, E), or of an expert whose
 * logit is NaN or -infinity, contributes nothing.)
 * With g = scale * grad_weights and the scores p of the same logits:
 *   softmax                   p_j ([j chosen] g_j - sum_k g_k p_k), all j
 *   softmax, renormalised     q_j (g_j - sum_k g_k q_k), chosen j, else 0
 *   sigmoid                   g_j p_j (1 - p_j), chosen j, else 0
 *   sigmoid, renormalised     q_j (1 - p_j) (g_j - sum_k g_k q_k), chosen j
 * where q = p / (sum of chosen p). An expert named twice gets both terms, in
 * ascending k. grad_logits has the logits' type, rows grad_ld apart; every
 * element [T, E] is written. Of the config: logits_dtype, score, renormalize
 * and scale.
 */
EP_API ep_status_t ep_router_topk_backward(const void* logits, int64_t logits_ld, const int64_t* topk_idx,
                                           int64_t topk_ld, const float* grad_weights, int T, int E, int K,
                                           const ep_router_config_t* config, void* grad_logits, int64_t grad_ld,
                                           void* stream);

/* ----------------------------------------------------------- paged cache */

/*
 * A paged cache holds num_pages pages of page_size slots; slot s is page
 * s / page_size, place s % page_size. Element (page, place, head, i) of the
 * keys is at page * k_page_stride + place * k_slot_stride + head *
 * k_head_stride + i, the values likewise, so pages may be laid out slot by
 * slot or head by head. Rows (head_dim elements) must start on 16 bytes: base
 * pointers 16-byte aligned, strides and head_dim * element size multiples of
 * 16 bytes.
 */
typedef struct {
    int dtype;              /* of the cache: EP_DTYPE_BF16, EP_DTYPE_FP16 or
                               EP_DTYPE_FP8_E4M3                               */
    int page_size;          /* >= 1                                            */
    int64_t num_pages;      /* num_pages * page_size < 2^40                     */
    int64_t k_page_stride, k_slot_stride, k_head_stride;
    int64_t v_page_stride, v_slot_stride, v_head_stride;
    float k_scale, v_scale; /* e4m3 only: the stored code stands for code *
                               scale; finite and > 0                           */
} ep_cache_t;

typedef struct {
    int dtype;              /* q, k, v, q_out: EP_DTYPE_BF16 or EP_DTYPE_FP16    */
    int num_heads;          /* query heads; 0: no queries (q, q_out unused)    */
    int num_kv_heads;
    int head_dim;           /* multiple of 8 (16 for an e4m3 cache), <= 1024    */
    int rotary_dim;         /* even, 0 .. head_dim: the leading values that turn */
    int interleaved;        /* 0: pairs (i, i + rotary_dim/2); 1: (2i, 2i + 1)   */
    int64_t q_ld, k_ld, v_ld, q_out_ld;  /* elements from one token to the next */
    int64_t max_position;   /* rows of cos_sin                                   */
} ep_append_config_t;

/*
 * ep_kv_append -- for each of T tokens: turn the leading rotary_dim values of
 * every query and key head by the token's position, write the queries to
 * q_out, and the keys and the (unturned) values to the token's cache slot.
 *
 *  q, k, v        device, [T, heads, head_dim], heads dense, tokens *_ld apart
 *                 (>= heads * head_dim): slices of one fused projection serve.
 *                 16-byte aligned rows.
 *  positions      device, int64 [T], each in [0, max_position).
 *  slots          device, int64 [T], each in [0, num_pages * page_size), or -1:
 *                 the token's queries are turned but nothing is cached (a
 *                 padding token). Two tokens must not name the same slot.
 *  cos_sin        device, fp32 [max_position, rotary_dim]: the cosines of the
 *                 rotary_dim/2 angles of a position, then their sines. NULL is
 *                 allowed when rotary_dim is 0.
 *  q_out          device, [T, num_heads, head_dim]; may be q itself.
 *  device_error   device, int32 [1] or NULL: set to 0, or to
 *                 EP_ERR_INVALID_ARG if a slot or a position was out of range.
 *                 Such a token is not cached; with a bad position its q_out
 *                 rows are zero.
 * A pair (a, b) becomes (a cos - b sin, b cos + a sin), in fp32, rounded once
 * to the output type. An e4m3 cache stores round-to-nearest-even of
 * value * (1 / scale), saturating at +-448, NaN kept; a scale whose reciprocal
 * is not finite in fp32 is refused.
 */
EP_API ep_status_t ep_kv_append(const void* q, const void* k, const void* v, const int64_t* positions,
                                const int64_t* slots, const float* cos_sin, int T,
                                const ep_append_config_t* config, void* q_out, void* k_cache, void* v_cache,
                                const ep_cache_t* cache, int32_t* device_error, void* stream);

/* ------------------------------------------------------------- attention */

typedef struct {
    int dtype;              /* q and out: EP_DTYPE_BF16 or EP_DTYPE_FP16; a 16-bit
                               cache has the same type                          */
    int num_heads;          /* query heads, a multiple of num_kv_heads          */
    int num_kv_heads;       /* query head h reads cache head
                               h / (num_heads / num_kv_heads)                   */
    int head_dim;           /* multiple of 8 (16 for an e4m3 cache), 8 .. 256    */
    int max_pages;          /* columns of block_table                          */
    int64_t q_ld, out_ld;   /* elements from one sequence to the next           */
    int64_t table_ld;       /* entries from one sequence's pages to the next's  */
    float scale;            /* factor on q . k                                  */
    int window;             /* 0: all keys; else the last `window` keys only    */
} ep_attention_config_t;

/*
 * ep_paged_attention -- out[b, h] = sum_i softmax_i(scale * q[b, h] . key_i) *
 * value_i over the keys i = 0 .. seq_lens[b] - 1 of sequence b (its new
 * token's own among them: append first), key i in page
 * block_table[b, i / page_size], place i % page_size.
 *
 *  q, out         device, [B, num_heads, head_dim], 16-byte aligned rows.
 *  block_table    device, int32 [B, max_pages]. Entries past a sequence's end
 *                 (or before its window) are not read as pages. A page id
 *                 outside [0, num_pages) masks its keys out.
 *  seq_lens       device, int32 [B]; taken as 0 when negative and as
 *                 max_pages * page_size when larger.
 *  lse            device, fp32 [B, num_heads] or NULL: the natural logarithm of
 *                 the sum of exp(scale * q . key_i), -infinity for no keys.
 *  workspace      device, 16-byte aligned, ep_paged_attention_workspace bytes;
 *                 contents need no initialising and are not kept.
 * A sequence with no keys (length 0, every page masked) gives zeros. What lies
 * in the cache behind a sequence's end, NaN included, does not matter.
 * Scores, softmax statistics and sums are fp32. A softmax weight enters the
 * products as the sum of two 16-bit numbers: within 2^-16 of itself over a bf16
 * cache, within 2^-22 of itself or 2^-36 of the sequence's largest weight,
 * whichever is more, over an fp16 or e4m3 cache. B * num_heads < 2^31.
 */
EP_API ep_status_t ep_paged_attention(const void* q, const void* k_cache, const void* v_cache,
                                      const ep_cache_t* cache, const int32_t* block_table,
                                      const int32_t* seq_lens, int B, const ep_attention_config_t* config, void* out,
                                      float* lse, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that ep_paged_attention needs for these sizes on the
 * current device; -1 for invalid sizes or a CUDA error. */
EP_API int64_t ep_paged_attention_workspace(int B, int num_heads, int num_kv_heads, int head_dim);

/* ------------------------------------------------------- 4-bit experts */

typedef enum {
    EP_ACT_NONE = 0,
    EP_ACT_SWIGLU = 1          /* y = silu(gate) * up                          */
} ep_activation_t;

typedef struct {
    int dtype;              /* x, scales and y: EP_DTYPE_BF16 or EP_DTYPE_FP16   */
    int group_size;         /* 32, 64 or 128 inputs share a scale              */
    int activation;         /* ep_activation_t                                 */
    int64_t x_ld, y_ld;     /* elements from one row to the next                */
} ep_w4_config_t;

/*
 * ep_expert_w4 -- y[n] = W_e x[n] for the rows n of each expert e, with
 *   W_e[o, i] = scales[e, i / group_size, o] * (code[e, o, i] - zero),
 * meant for the few rows per expert of decoding (it is right for any number).
 *
 *  x              device, [rows, I]; rows in ep_dispatch's order. I a multiple
 *                 of group_size. 16-byte aligned rows.
 *  weights        device, uint8 [E, O, I/2], dense, 16-byte aligned: byte j of
 *                 a row holds the codes of inputs 2j (low four bits) and 2j + 1.
 *  scales         device, [E, I/group_size, O], dense.
 *  zeros          device, uint8 [E, I/group_size, O] (0 .. 15), or NULL: 8.
 *  expert_offsets device, int32 [E + 1], as every ep_layout* writes it: expert
 *                 e owns rows [expert_offsets[e], expert_offsets[e + 1]). NULL
 *                 with E = 1: all rows.
 *  expert_counts  device, int32 [E], or NULL: only the first expert_counts[e]
 *                 of them are real (num_tokens_per_expert of an aligned or a
 *                 strided layout). The others' y is not written.
 *  E, O           experts and weight rows; O even with EP_ACT_SWIGLU, whose y
 *                 has O/2 columns: gate = weight row j, up = row O/2 + j.
 *  y              device, [rows, O or O/2].
 *  workspace      device, 16-byte aligned, ep_expert_w4_workspace bytes;
 *                 contents need no initialising and are not kept.
 * Each input is taken to within 2^-24 of the largest of the group (of
 * group_size inputs) that it is in; products and sums are fp32, a
 * group's scale multiplies the group's sum, and y is rounded once, after the
 * activation. An infinite input makes its row of y NaN. Offsets are taken as
 * at most `rows`; rows, I and O are at most 2^31 - 512.
 */
EP_API ep_status_t ep_expert_w4(const void* x, int64_t rows, int I, const uint8_t* weights, const void* scales,
                                const uint8_t* zeros, const int32_t* expert_offsets, const int32_t* expert_counts,
                                int E, int O, const ep_w4_config_t* config, void* y, void* workspace,
                                int64_t workspace_bytes, void* stream);

/* Bytes of workspace that ep_expert_w4 needs; -1 for invalid sizes. */
EP_API int64_t ep_expert_w4_workspace(int64_t rows, int I, int group_size, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* EP_GB300_EP_LAYER_H */
