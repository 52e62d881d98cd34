// C ABI of the latent-row operators: argument validation and launches (see include/hs_latent.h).
#include "latent.cuh"

namespace {

bool aligned(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }
// A stride in elements of `size` bytes: a multiple of 16 bytes that byte offsets up to `count` fit in 62 bits.
bool stride_ok(int64_t stride, int64_t size, int64_t count) {
  if (stride < 0 || (stride * size) % 16) return false;
  return count <= 1 || stride <= (int64_t(1) << 60) / size / count;
}
// The same for a tensor that is written: no two of its `width`-element rows may overlap.
bool out_stride_ok(int64_t stride, int64_t size, int64_t count, int64_t width) {
  return stride_ok(stride, size, count) && (count <= 1 || stride >= width);
}
bool on_device(int dev) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return cur == dev;
}
hs_status status_of(cudaError_t e) { return e == cudaSuccess ? HS_OK : HS_ERR_CUDA; }

bool row_format(int32_t row_bytes) { return row_bytes == HS_ROW_BYTES_FP8 || row_bytes == HS_ROW_BYTES_BF16; }

// Fills what the two absorbed calls share; `tokens` query tokens.
hs_status prepare_attend(const hs_pool* pool, int32_t layer, const hs_attend* a, int64_t tokens, void* workspace,
                         size_t workspace_bytes, hs::AttendParams& p, hs::LayerView& v) {
  if (!a || !hs::pool_layer(pool, layer, &v) || !row_format(v.row_bytes)) return HS_ERR_INVALID_ARG;
  if (a->heads < 1 || a->heads > HS_MAX_HEADS || !(a->scale == a->scale)) return HS_ERR_INVALID_ARG;
  if (tokens == 0) return HS_OK;
  if (!aligned(a->q_latent) || !aligned(a->q_rope) || !aligned(a->out)) return HS_ERR_INVALID_ARG;
  if (!stride_ok(a->ql_token_stride, 2, tokens) || !stride_ok(a->ql_head_stride, 2, a->heads) ||
      !stride_ok(a->qr_token_stride, 2, tokens) || !stride_ok(a->qr_head_stride, 2, a->heads) ||
      !out_stride_ok(a->out_token_stride, 2, tokens, hs::kLatent) ||
      !out_stride_ok(a->out_head_stride, 2, a->heads, hs::kLatent))
    return HS_ERR_INVALID_ARG;
  if (!on_device(v.device)) return HS_ERR_INVALID_ARG;
  if (v.sms <= 0) return HS_ERR_CUDA;
  if (!aligned(workspace) || workspace_bytes < hs::attend_workspace_bytes(v.sms)) return HS_ERR_INVALID_ARG;
  p = hs::AttendParams{};
  p.base = v.base;
  p.row_bytes = v.row_bytes;
  p.page_size = v.page_size;
  p.num_blocks = v.num_blocks;
  p.num_rows = v.num_rows;
  p.heads = a->heads;
  p.q_latent = static_cast<const __nv_bfloat16*>(a->q_latent);
  p.ql_tok = a->ql_token_stride;
  p.ql_head = a->ql_head_stride;
  p.q_rope = static_cast<const __nv_bfloat16*>(a->q_rope);
  p.qr_tok = a->qr_token_stride;
  p.qr_head = a->qr_head_stride;
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.out_tok = a->out_token_stride;
  p.out_head = a->out_head_stride;
  p.lse = a->lse;
  p.scale_log2 = a->scale * hs::kLog2e;
  p.status = a->status;
  p.workspace = static_cast<float*>(workspace);
  return HS_OK;
}

}  // namespace

extern "C" {

hs_status hs_append_rows(const hs_pool* pool, int32_t layer, const hs_append* a, hs_stream_t stream) {
  HS_RANGE("hs_append_rows");
  hs::LayerView v;
  if (!a || !hs::pool_layer(pool, layer, &v) || !row_format(v.row_bytes)) return HS_ERR_INVALID_ARG;
  if (a->n < 0 || a->n > INT32_MAX || a->heads < 0 || a->heads > HS_MAX_HEADS || a->num_positions < 1 ||
      a->dtype < HS_BF16 || a->dtype > HS_FP32)
    return HS_ERR_INVALID_ARG;
  if (a->n == 0) return HS_OK;
  const int64_t size = a->dtype == HS_FP32 ? 4 : 2;
  if (!a->rows || !a->positions || !aligned(a->rotation) || !aligned(a->latent) || !aligned(a->rope))
    return HS_ERR_INVALID_ARG;
  if (!stride_ok(a->latent_stride, size, a->n) || !stride_ok(a->rope_stride, size, a->n)) return HS_ERR_INVALID_ARG;
  if (a->heads > 0 &&
      (!aligned(a->q_rope) || !aligned(a->q_out) || !stride_ok(a->q_token_stride, size, a->n) ||
       !stride_ok(a->q_head_stride, size, a->heads) || !out_stride_ok(a->q_out_token_stride, size, a->n, hs::kRope) ||
       !out_stride_ok(a->q_out_head_stride, size, a->heads, hs::kRope)))
    return HS_ERR_INVALID_ARG;
  if (!on_device(v.device)) return HS_ERR_INVALID_ARG;
  if (v.sms <= 0) return HS_ERR_CUDA;
  hs::AppendParams p{*a, v.base, v.num_rows, v.row_bytes};
  return status_of(hs::launch_append(p, v.sms, stream));
}

size_t hs_attend_workspace_bytes(void) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  const int sms = hs::device_sms(dev);
  return sms > 0 ? hs::attend_workspace_bytes(sms) : 0;
}

hs_status hs_attend_rows(const hs_pool* pool, int32_t layer, const int32_t* rows, int64_t tokens, int32_t K,
                         const hs_attend* a, void* workspace, size_t workspace_bytes, hs_stream_t stream) {
  HS_RANGE("hs_attend_rows");
  if (tokens < 0 || tokens > INT32_MAX || K < 0 || K > (1 << 30)) return HS_ERR_INVALID_ARG;
  hs::AttendParams p;
  hs::LayerView v;
  const hs_status st = prepare_attend(pool, layer, a, tokens, workspace, workspace_bytes, p, v);
  if (st != HS_OK || tokens == 0) return st;
  if (K > 0 && !rows) return HS_ERR_INVALID_ARG;
  p.rows = rows;
  p.K = K;
  p.items = (int32_t)tokens;
  p.P = 1;
  p.cols = a->heads;
  return status_of(hs::launch_attend(p, v.device, v.sms, stream));
}

hs_status hs_attend_pages(const hs_pool* pool, int32_t layer, const int32_t* block_table, const int32_t* ctx_len,
                          int32_t R, int32_t P, int32_t max_pages, const hs_attend* a, void* workspace,
                          size_t workspace_bytes, hs_stream_t stream) {
  HS_RANGE("hs_attend_pages");
  if (R < 0 || P < 1 || P > HS_MAX_QUERY_POSITIONS || max_pages < 0) return HS_ERR_INVALID_ARG;
  hs::AttendParams p;
  hs::LayerView v;
  const int64_t tokens = (int64_t)R * P;
  if (tokens > INT32_MAX) return HS_ERR_INVALID_ARG;
  const hs_status st = prepare_attend(pool, layer, a, tokens, workspace, workspace_bytes, p, v);
  if (st != HS_OK || tokens == 0) return st;
  if (!ctx_len || (max_pages > 0 && !block_table) || (int64_t)max_pages * v.page_size > (1 << 30))
    return HS_ERR_INVALID_ARG;
  // the kernel counts a request's tiles (64 keys x 64 columns) in 32 bits
  if (((int64_t)max_pages * v.page_size / 64 + 1) * ((int64_t)P * a->heads / 64 + 1) > INT32_MAX) return HS_ERR_INVALID_ARG;
  p.paged = 1;
  p.table = block_table;
  p.ctx_len = ctx_len;
  p.max_pages = max_pages;
  p.items = R;
  p.P = P;
  p.cols = P * a->heads;
  return status_of(hs::launch_attend(p, v.device, v.sms, stream));
}

hs_status hs_attend_expanded(const hs_expanded* a, hs_stream_t stream) {
  HS_RANGE("hs_attend_expanded");
  if (!a || a->seqs < 0 || a->heads < 1 || a->heads > HS_MAX_HEADS || a->q_tokens < 0 || a->k_tokens < 0 ||
      a->q_tokens > INT32_MAX || a->k_tokens > INT32_MAX || !(a->scale == a->scale))
    return HS_ERR_INVALID_ARG;
  if (a->q_tokens == 0) return HS_OK;
  if (!a->cu_q || !a->cu_k || !aligned(a->q_nope) || !aligned(a->q_rope) || !aligned(a->out)) return HS_ERR_INVALID_ARG;
  if (a->k_tokens > 0 && (!aligned(a->k_nope) || !aligned(a->k_rope) || !aligned(a->v))) return HS_ERR_INVALID_ARG;
  const int64_t q = a->q_tokens, k = a->k_tokens, h = a->heads;
  if (!stride_ok(a->qn_token_stride, 2, q) || !stride_ok(a->qn_head_stride, 2, h) ||
      !stride_ok(a->qr_token_stride, 2, q) || !stride_ok(a->qr_head_stride, 2, h) ||
      !stride_ok(a->kn_token_stride, 2, k) || !stride_ok(a->kn_head_stride, 2, h) ||
      !stride_ok(a->kr_token_stride, 2, k) || !stride_ok(a->v_token_stride, 2, k) ||
      !stride_ok(a->v_head_stride, 2, h) || !out_stride_ok(a->out_token_stride, 2, q, hs::kValue) ||
      !out_stride_ok(a->out_head_stride, 2, h, hs::kValue))
    return HS_ERR_INVALID_ARG;
  if ((q > 1 && (a->qn_token_stride == 0 || a->qr_token_stride == 0)) ||
      (k > 1 && (a->kn_token_stride == 0 || a->kr_token_stride == 0 || a->v_token_stride == 0)))
    return HS_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return HS_ERR_CUDA;
  }
  const int sms = hs::device_sms(dev);
  if (sms <= 0) return HS_ERR_CUDA;
  return status_of(hs::launch_expanded(*a, dev, sms, stream));
}

}  // extern "C"
