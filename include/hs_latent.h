/*
 * hs_latent.h -- C ABI of the operators that write and read the latent rows of the paged KV pool.
 *
 *   hs_append_rows      writes the rows of new tokens: the position rotation of the key part, the
 *                       quantisation of the latent part and the store into the pool, in one launch;
 *                       rotates the queries' position part in the same launch.
 *   hs_read_rows        reads rows back by id, in 16 or 32 bits: a prefix's latents, to be expanded.
 *   hs_attend_rows      absorbed latent attention over row ids, as hs_resolve_topk hands them back.
 *   hs_attend_pages     absorbed latent attention over whole contexts through a block table (requests
 *                       whose pages are all GPU-resident).
 *   hs_attend_expanded  attention over keys and values expanded from the latents to every head, with
 *                       one rotated key part shared by the heads: prompts and prompt chunks.
 *
 * The source pages describe the cache these read and write (FP8 KV of a sparse-MLA model, "vLLM GLM 5.3
 * Optimizations: Hybrid HiSparse Offloading", benchmark section) and an attention kernel that sees hot
 * pages as ordinary pages (Japanese article, section "必要な時にスパーシティを活用する"); its arithmetic is
 * not on the pages.  The formulas below are this library's.
 *
 * Rows.  The pool's row_bytes says how its rows are kept:
 *   HS_ROW_BYTES_FP8  (656)   512 latent values as e4m3 codes | 4 fp32 scales, one per 128 values |
 *                             64 rotated key values in bf16.  value = code * scale.
 *   HS_ROW_BYTES_BF16 (1152)  512 latent values in bf16 | 64 rotated key values in bf16.
 * Pools of other row sizes are refused (HS_ERR_INVALID_ARG).  hs_append_rows writes scales that are
 * powers of two, so that code * scale is exact in bf16; the attention calls read any finite scale and
 * round code * scale to bf16.  They multiply fp8 rows in fp16, rows and query columns divided by powers of two:
 *   within a row, values (rotated ones included) keep their bits down to 2^-29 of the largest that the row's
 *   scales and rotated part cover, and are zero below 2^-40 of it;
 *   within a query (of one head), values keep their bits down to 2^-15 of its largest;
 *   between rows, a weight times the row's size keeps its bits down to 2^-21 of the largest such product, and is
 *   zero below 2^-32 of it.  The rows that one token sees may differ in size by up to 2^100.
 * A group of zeros has no size, whatever its scale.
 *
 * Conventions: those of hs.h.  The caller owns all memory and streams; calls validate what the host can
 * see, launch on the given stream and return; data errors go to an optional device status word, which is
 * written only when there is one.  Strides are in elements; the innermost dimension is contiguous; tensor
 * pointers and strides are multiples of 16 bytes; the rows of a tensor that is written must not overlap, while
 * one that is read may repeat them (stride 0; hs_attend_expanded takes a stride of 0 between heads, not between
 * tokens).  The current device must be the pool's (for hs_attend_expanded: the one that holds the tensors).
 * Calls that share a workspace must be ordered on one stream.
 */
#ifndef HS_LATENT_H_
#define HS_LATENT_H_

#include "hs.h"

#ifdef __cplusplus
extern "C" {
#endif

#define HS_LATENT_DIM 512
#define HS_ROPE_DIM 64
#define HS_SCALE_GROUP 128
#define HS_NOPE_DIM 128  /* expanded form: per-head key values without position */
#define HS_VALUE_DIM 128 /* expanded form: per-head values                      */
#define HS_ROW_BYTES_FP8 656
#define HS_ROW_BYTES_BF16 1152
#define HS_MAX_HEADS 1024
#define HS_MAX_QUERY_POSITIONS 1024

typedef enum { HS_BF16 = 0, HS_FP16 = 1, HS_FP32 = 2 } hs_dtype;

/* New tokens of one layer.  For token t with row id rows[t]:
 *   (a, b) -> (a cos - b sin, b cos + a sin) for the 32 pairs of the key part, in fp32, rounded once;
 *   pairs are elements (i, i + 32), or (2i, 2i + 1) with interleaved != 0; cos and sin are
 *   rotation[positions[t]][i] and [32 + i].
 *   fp8 rows: per group of 128 latent values, scale = the smallest power of two (at least 2^-126) with
 *   max |finite value| <= 448 * scale, 1 for a group of zeros; code = e4m3(value / scale), ties to even;
 *   a value that is infinite or NaN becomes the NaN code.  bf16 rows: each value rounded to bf16. */
typedef struct {
  int64_t n;                /* tokens                                                                 */
  const int32_t* rows;      /* device [n]: pool row ids, distinct; -1 writes no row.  Where two tokens
                               name one row, either may win                                           */
  const int32_t* positions; /* device [n]                                                             */
  const float* rotation;    /* device [num_positions][64]: 32 cosines, then 32 sines                  */
  int32_t num_positions;
  int32_t interleaved;
  int32_t dtype;            /* hs_dtype of latent, rope, q_rope and q_out                             */
  int32_t heads;            /* query heads to rotate, 0 for none (q_rope and q_out may be NULL)       */
  const void* latent;       /* device [n][512]                                                        */
  int64_t latent_stride;
  const void* rope;         /* device [n][64]                                                         */
  int64_t rope_stride;
  const void* q_rope;       /* device [n][heads][64]                                                  */
  int64_t q_token_stride, q_head_stride;
  void* q_out;              /* device [n][heads][64]; may be q_rope itself (same strides)             */
  int64_t q_out_token_stride, q_out_head_stride;
  int32_t* status;          /* optional device word: HS_ERR_ID_RANGE when a row id lies outside
                               [-1, num_gpu_blocks * page_size) (that row is not written) or a position
                               outside [0, num_positions) (the token's row is not written and its
                               rotated queries are zero)                                              */
} hs_append;

hs_status hs_append_rows(const hs_pool* pool, int32_t layer, const hs_append* a, hs_stream_t stream);

/* Rows by id: latent[t] = code * scale (fp8 rows; bf16 rows: the value) and rope[t] = the rotated key values, each
 * rounded once to the tensors' type.  An id of -1 gives zeros. */
typedef struct {
  int64_t n;                /* rows                                                                   */
  const int32_t* rows;      /* device [n]: pool row ids, in any order; an id may occur more than once */
  int32_t dtype;            /* hs_dtype of latent and rope                                            */
  void* latent;             /* device [n][512]                                                        */
  int64_t latent_stride;
  void* rope;               /* device [n][64]                                                         */
  int64_t rope_stride;
  int32_t* status;          /* optional device word: HS_ERR_ID_RANGE when a row id lies outside
                               [-1, num_gpu_blocks * page_size) (its row of the tensors is zero)      */
} hs_read_latent;

hs_status hs_read_rows(const hs_pool* pool, int32_t layer, const hs_read_latent* a, hs_stream_t stream);

/* Queries and results of an absorbed attention call.  For query token t, head h and the visible rows k
 * with latent c[k] (fp32 of the stored value, rounded to bf16) and rotated key r[k]:
 *   s[k] = scale * (q_latent[t][h] . c[k] + q_rope[t][h] . r[k])
 *   out[t][h] = sum_k softmax(s)[k] c[k]        lse[t][h] = log sum_k exp(s[k])
 * Sums and softmax statistics are fp32; softmax weights are rounded to bf16 (fp8 rows: to fp16) before their
 * product with the latents; out is rounded once.  A token that sees no row gets zeros and lse = -infinity.
 * A row that a token does not see has no part in its result, whatever the row holds; a NaN in one that it sees makes
 * its result NaN, and an infinity there makes it NaN or leaves out the infinite value where the row's weight is zero. */
typedef struct {
  int32_t heads;            /* 1..HS_MAX_HEADS                                                        */
  float scale;
  const void* q_latent;     /* device bf16 [tokens][heads][512]                                       */
  int64_t ql_token_stride, ql_head_stride;
  const void* q_rope;       /* device bf16 [tokens][heads][64]                                        */
  int64_t qr_token_stride, qr_head_stride;
  void* out;                /* device bf16 [tokens][heads][512]                                       */
  int64_t out_token_stride, out_head_stride;
  float* lse;               /* device fp32 [tokens][heads], or NULL                                   */
  int32_t* status;          /* optional device word, see the calls; HS_ERR_TIMEOUT: a bounded wait
                               inside the kernel gave up (results are then undefined)                 */
} hs_attend;

/* Bytes of device workspace (16-byte aligned) that hs_attend_rows and hs_attend_pages need at most on the
 * current device, whatever the call's shape: partial results of contexts that several CTAs share.  0 when
 * there is no device. */
size_t hs_attend_workspace_bytes(void);

/* tokens queries, query t over the rows rows[t][0..K): device int32 [tokens][K], the layout of
 * hs_resolve_topk's out_rows for one layer (tokens = R * P).  -1 entries are skipped; an id that occurs
 * twice counts twice.  K is at most 2^30.  status: HS_ERR_ID_RANGE for an id outside
 * [-1, num_gpu_blocks * page_size), which is skipped. */
hs_status hs_attend_rows(const hs_pool* pool, int32_t layer, const int32_t* rows, int64_t tokens, int32_t K,
                         const hs_attend* a, void* workspace, size_t workspace_bytes, hs_stream_t stream);

/* R requests of P query positions each (tokens = R * P, token r * P + p): the context of request r is the
 * tokens 0 .. ctx_len[r] - 1, the last P of them the query positions, and position p sees the first
 * ctx_len[r] - P + 1 + p of them.  Token j lives in row block_table[r][j / page_size] * page_size +
 * j % page_size.
 *   block_table  device int32 [R][max_pages]
 *   ctx_len      device int32 [R]
 * max_pages * page_size is at most 2^30, and (max_pages * page_size / 64 + 1) * (P * heads / 64 + 1) below 2^31.
 * status: HS_ERR_TABLE_RANGE for a needed entry outside [0, num_gpu_blocks) or a context longer than
 * max_pages pages; the tokens concerned are skipped. */
hs_status hs_attend_pages(const hs_pool* pool, int32_t layer, const int32_t* block_table, const int32_t* ctx_len,
                          int32_t R, int32_t P, int32_t max_pages, const hs_attend* a, void* workspace,
                          size_t workspace_bytes, hs_stream_t stream);

/* Ragged sequences: queries cu_q[b] .. cu_q[b+1] - 1 of sequence b over its keys cu_k[b] .. cu_k[b+1] - 1.
 *   s[i][j] = scale * (q_nope[i][h] . k_nope[j][h] + q_rope[i][h] . k_rope[j])
 *   out[i][h] = sum_j softmax(s)[i][j] v[j][h]      lse[i][h] = log sum_j exp(s[i][j])
 * With causal != 0 the queries are the last tokens of the sequence: query i (counted within it) sees the
 * keys j <= i + keys - queries.  Rounding (bf16 weights) and empty rows as in hs_attend.  Keys that a query does not
 * see have no part in its result, whatever they and their values hold.  Query tokens that no sequence has (cu_q leaves
 * them out, or the sequence's offsets are bad) get zeros and -infinity. */
typedef struct {
  int32_t seqs, heads;
  int32_t causal;
  float scale;
  int64_t q_tokens, k_tokens; /* rows of the tensors below; cu_q and cu_k are clamped to them          */
  const int32_t* cu_q;        /* device [seqs + 1], ascending from 0                                   */
  const int32_t* cu_k;        /* device [seqs + 1]                                                     */
  const void* q_nope;         /* device bf16 [q_tokens][heads][128]                                    */
  int64_t qn_token_stride, qn_head_stride;
  const void* q_rope;         /* device bf16 [q_tokens][heads][64]                                     */
  int64_t qr_token_stride, qr_head_stride;
  const void* k_nope;         /* device bf16 [k_tokens][heads][128]                                    */
  int64_t kn_token_stride, kn_head_stride;
  const void* k_rope;         /* device bf16 [k_tokens][64]                                            */
  int64_t kr_token_stride;
  const void* v;              /* device bf16 [k_tokens][heads][128]                                    */
  int64_t v_token_stride, v_head_stride;
  void* out;                  /* device bf16 [q_tokens][heads][128]                                    */
  int64_t out_token_stride, out_head_stride;
  float* lse;                 /* device fp32 [q_tokens][heads], or NULL                                */
  int32_t* status;            /* optional device word: HS_ERR_ID_RANGE when cu_q or cu_k do not ascend
                                 within their tensors (those sequences are treated as empty);
                                 HS_ERR_TIMEOUT as in hs_attend                                        */
} hs_expanded;

hs_status hs_attend_expanded(const hs_expanded* a, hs_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* HS_LATENT_H_ */
