/*
 * hs_heads.h -- C ABI of the operators on pages of grouped heads, held in 8 bits.
 *
 *   hs_append_heads   quantises the keys and values of new tokens into the pool's pages.
 *   hs_read_heads     reads tokens of requests back, in 16 or 32 bits.
 *   hs_attend_heads   attention of grouped query heads over the pages: single tokens, verify positions,
 *                     prompt chunks and prompts.
 *
 * A pool is bytes to the resolver's neighbours: block tables, the residency manager (hs_residency.h) and
 * hs_offload_pages move pages whatever they hold.  These operators are for the attention layers whose keys and
 * values are heads of their own (dense layers beside the sparse ones, the layer that drafts the verify
 * positions), as hs_latent.h is for latent rows.  Formats and formulas are this library's; the source pages
 * ("vLLM GLM 5.3 Optimizations: Hybrid HiSparse Offloading") speak of pages only.
 *
 * Pages.  page_size is HS_HEADS_PAGE tokens; head_dim is 64 or 128; row_bytes = 2 * kv_heads * head_dim + 16.
 * A page is, for each head of keys and values,
 *     head_dim / 64 blocks of [64 tokens][64 dims] key codes, then
 *     head_dim / 64 blocks of [64 dims][64 tokens] value codes (both e4m3, a byte each),
 * and behind the last head fp32 scales: one for the keys of each head, then one for the values of each head; the
 * rest of the page (1024 - 8 * kv_heads bytes) is not used.  value = code * scale.  All of a page, its scales
 * included, moves with it.  A page has no rows of its own: hs_resolve_topk and hs_gather_rows are not for such
 * pools.  A pool knows its row_bytes only, not what its pages hold: that 128 dimensions were written as such, and not as
 * twice the heads of 64, or that rows of 656 bytes are 5 heads of 64 and not latent rows (hs_latent.h), is the caller's to keep.
 *
 * Scales are positive; hs_append_heads writes powers of two, the reading calls take any positive normal number.
 *
 * Conventions: those of hs.h and hs_latent.h (memory, streams, status words, strides in elements, alignment to 16
 * bytes, the pool's device current, shared workspaces on one stream).
 *
 * Requests.  Token j of request r lies at place j % 64 of page block_table[r][j / 64]; max_pages * 64 is at most 2^30.  The tokens of ragged
 * tensors are cu[r] .. cu[r + 1] - 1 for request r; with cu == NULL every request has the same number, n / R.  cu
 * ascends within 0 .. n; where it does not, the status is HS_ERR_ID_RANGE and the call does nothing (hs_attend_heads:
 * all results are zero and -infinity).
 */
#ifndef HS_HEADS_H_
#define HS_HEADS_H_

#include "hs.h"
#include "hs_latent.h" /* hs_dtype */

#ifdef __cplusplus
extern "C" {
#endif

#define HS_HEADS_PAGE 64
#define HS_MAX_KV_HEADS 128

/* row_bytes of a pool for these heads; 0 when there is none (head_dim other than 64 or 128, kv_heads outside
 * 1..HS_MAX_KV_HEADS). */
int32_t hs_heads_row_bytes(int32_t kv_heads, int32_t head_dim);

/* New tokens: the last cu[r + 1] - cu[r] of the ctx_len[r] tokens that request r then has.  (A page that they continue was begun
 * by this call: its scales are powers of two.)  For each page, head and side (keys or values) that they touch:
 *   need  = the smallest power of two, at least 2^-126, with |x| <= 448 * need for all finite new values x
 *   scale = need where the new tokens begin the page (what it held before counts for nothing), and the larger of
 *           need and the page's scale where they continue it; where that raises the scale, the codes of the
 *           page's earlier tokens become e4m3(code * old scale / scale)
 *   code  = e4m3(x / scale), ties to even; the NaN code for an x that is infinite or NaN.
 * Places behind the last new token keep their bytes.  Appending a token again, with the page's later tokens gone or
 * appended with it, is allowed (a verify step's rejected tokens); the scale never falls until a page begins anew. */
typedef struct {
  int32_t kv_heads, head_dim;
  int32_t dtype;              /* hs_dtype of k and v                                                  */
  int32_t R, max_pages;
  int64_t n;                  /* new tokens of all requests                                           */
  const int32_t* block_table; /* device [R][max_pages]; no page that is written to occurs twice       */
  const int32_t* ctx_len;     /* device [R]                                                           */
  const int32_t* cu;          /* device [R + 1], or NULL: n / R tokens each                           */
  const void* k;              /* device [n][kv_heads][head_dim]                                       */
  int64_t k_token_stride, k_head_stride;
  const void* v;              /* device [n][kv_heads][head_dim]                                       */
  int64_t v_token_stride, v_head_stride;
  int32_t* status;            /* optional device word: HS_ERR_ID_RANGE where cu does not ascend, or a request
                                 has more new tokens than ctx_len (nothing of it is written);
                                 HS_ERR_TABLE_RANGE for a needed table entry outside [0, num_gpu_blocks) or past
                                 max_pages (those tokens are not written)                             */
} hs_heads_append;

hs_status hs_append_heads(const hs_pool* pool, int32_t layer, const hs_heads_append* a, hs_stream_t stream);

/* Tokens start[r] .. start[r] + (cu[r + 1] - cu[r]) - 1 of every request into rows cu[r] .. of k and v: code * scale,
 * rounded once.  Rows that no request has keep what they hold. */
typedef struct {
  int32_t kv_heads, head_dim;
  int32_t dtype;              /* hs_dtype of k and v                                                  */
  int32_t R, max_pages;
  int64_t n;                  /* rows of k and v                                                      */
  const int32_t* block_table; /* device [R][max_pages]                                                */
  const int32_t* start;       /* device [R], or NULL: 0                                               */
  const int32_t* cu;          /* device [R + 1], or NULL: n / R tokens each                           */
  void* k;                    /* device [n][kv_heads][head_dim]                                       */
  int64_t k_token_stride, k_head_stride;
  void* v;                    /* device [n][kv_heads][head_dim]                                       */
  int64_t v_token_stride, v_head_stride;
  int32_t* status;            /* optional device word: HS_ERR_ID_RANGE where cu does not ascend, or start is
                                 negative (nothing of that request is read); HS_ERR_TABLE_RANGE as above
                                 (those tokens are zero)                                              */
} hs_heads_read;

hs_status hs_read_heads(const hs_pool* pool, int32_t layer, const hs_heads_read* a, hs_stream_t stream);

/* Query tokens cu_q[r] .. cu_q[r + 1] - 1 of request r, with n = cu_q[r + 1] - cu_q[r], over its first ctx_len[r]
 * tokens; with causal != 0 they are the last tokens of the context, and the i-th of them sees the first
 * ctx_len[r] - n + 1 + i.  Query head h reads head h / (q_heads / kv_heads) of the pages:
 *   s[j] = scale * q[t][h] . k[j]     out[t][h] = sum_j softmax(s)[j] v[j]     lse[t][h] = log sum_j exp(s[j])
 * over the tokens j that it sees.  A query that sees none, or that no request has, gets zeros and -infinity.
 * Products are in fp16 with fp32 sums.  e4m3 codes are exact there; a query (of one head) is divided by a power of
 * two and keeps the bits of values down to 2^-15 of its largest; a token's weight times its page's value scale is
 * rounded to 11 bits and keeps them down to 2^-21 of the largest such product, and is zero below 2^-32 of it.  The
 * value scales that one query sees may differ by up to 2^100.  lse and the sum of the weights are fp32 throughout.
 * What a query does not see has no part in its result, whatever it holds.  A NaN value that it sees makes that element
 * of out NaN.  Scores that are not finite in fp32 (NaN keys; queries that hold NaN or an infinity) enter as the
 * formulas say: a NaN among those that it sees makes out and lse NaN, +infinity out NaN and lse +infinity, and where all
 * are -infinity, out is NaN and lse -infinity. */
typedef struct {
  int32_t kv_heads, head_dim;
  int32_t q_heads;            /* a multiple of kv_heads, at most HS_MAX_HEADS                         */
  int32_t dtype;              /* hs_dtype of q and out: HS_BF16 or HS_FP16                            */
  int32_t causal;
  float scale;                /* of either sign, at most 2^127 in magnitude                           */
  int32_t R, max_pages;
  int64_t n;                  /* query tokens; n * q_heads is below 2^31                              */
  const int32_t* block_table; /* device [R][max_pages]                                                */
  const int32_t* ctx_len;     /* device [R]                                                           */
  const int32_t* cu_q;        /* device [R + 1], or NULL: n / R tokens each                           */
  const void* q;              /* device [n][q_heads][head_dim]                                        */
  int64_t q_token_stride, q_head_stride;
  void* out;                  /* device [n][q_heads][head_dim]                                        */
  int64_t out_token_stride, out_head_stride;
  float* lse;                 /* device fp32 [n][q_heads], or NULL                                    */
  int32_t* status;            /* optional device word: HS_ERR_ID_RANGE where cu_q does not ascend; HS_ERR_TABLE_RANGE for a needed table entry
                                 outside [0, num_gpu_blocks) or a context past max_pages (those tokens are
                                 skipped); HS_ERR_TIMEOUT: a bounded wait inside the kernel gave up (results are
                                 then undefined), after about two seconds, which contexts beyond 2^26
                                 tokens may take                                                      */
} hs_heads_attend;

/* Bytes of device workspace (16-byte aligned) that hs_attend_heads needs at most on the current device, whatever the
 * call's shape.  0 when there is no device. */
size_t hs_heads_workspace_bytes(void);

hs_status hs_attend_heads(const hs_pool* pool, int32_t layer, const hs_heads_attend* a, void* workspace,
                          size_t workspace_bytes, hs_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* HS_HEADS_H_ */
