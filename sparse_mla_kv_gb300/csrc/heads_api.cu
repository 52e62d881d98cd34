// C ABI of the operators on pages of grouped heads: argument validation and launches (see include/hs_heads.h).
#include <math.h>

#include "heads.cuh"

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

// Whether the pool's pages hold these heads, and the tokens of R requests are what cu (or n / R each) says; fills the views.
template <typename Args>
bool geometry(const hs_pool* pool, int32_t layer, const Args& a, const int32_t* cu, hs::LayerView* v, hs::HeadPages* pages,
              hs::Ragged* ragged) {
  if (!hs::pool_layer(pool, layer, v)) return false;
  const int32_t row_bytes = hs_heads_row_bytes(a.kv_heads, a.head_dim);
  if (row_bytes == 0 || v->row_bytes != row_bytes || v->page_size != HS_HEADS_PAGE) return false;
  if (a.n < 0 || a.n > INT32_MAX || a.R < 0 || a.max_pages < 0 || (int64_t)a.max_pages * HS_HEADS_PAGE > (1 << 30)) return false;
  if (!cu && (a.R == 0 ? a.n > 0 : a.n % a.R != 0)) return false;
  if (a.R > 0 && a.max_pages > 0 && !a.block_table) return false;
  *pages = hs::HeadPages{v->base, (int64_t)v->row_bytes * v->page_size, v->num_blocks, a.kv_heads, a.max_pages, a.block_table};
  *ragged = hs::Ragged{cu, a.R, cu || a.R == 0 ? 0 : (int32_t)(a.n / a.R), a.n};
  return true;
}

}  // namespace

extern "C" {

int32_t hs_heads_row_bytes(int32_t kv_heads, int32_t head_dim) {
  if ((head_dim != 64 && head_dim != 128) || kv_heads < 1 || kv_heads > HS_MAX_KV_HEADS) return 0;
  return 2 * kv_heads * head_dim + 16;
}

hs_status hs_append_heads(const hs_pool* pool, int32_t layer, const hs_heads_append* a, hs_stream_t stream) {
  HS_RANGE("hs_append_heads");
  hs::LayerView v;
  hs::HeadsAppendParams p;
  if (!a || a->dtype < HS_BF16 || a->dtype > HS_FP32 || !geometry(pool, layer, *a, a->cu, &v, &p.pages, &p.ragged))
    return HS_ERR_INVALID_ARG;
  if (a->n == 0) return HS_OK;
  const int64_t size = a->dtype == HS_FP32 ? 4 : 2;
  if ((a->R > 0 && !a->ctx_len) || !aligned(a->k) || !aligned(a->v)) return HS_ERR_INVALID_ARG;
  if (!stride_ok(a->k_token_stride, size, a->n) || !stride_ok(a->k_head_stride, size, a->kv_heads) ||
      !stride_ok(a->v_token_stride, size, a->n) || !stride_ok(a->v_head_stride, size, a->kv_heads))
    return HS_ERR_INVALID_ARG;
  if (!on_device(v.device)) return HS_ERR_INVALID_ARG;
  p.a = *a;
  return status_of(hs::launch_append_heads(p, stream));
}

hs_status hs_read_heads(const hs_pool* pool, int32_t layer, const hs_heads_read* a, hs_stream_t stream) {
  HS_RANGE("hs_read_heads");
  hs::LayerView v;
  hs::HeadsReadParams p;
  if (!a || a->dtype < HS_BF16 || a->dtype > HS_FP32 || !geometry(pool, layer, *a, a->cu, &v, &p.pages, &p.ragged))
    return HS_ERR_INVALID_ARG;
  if (a->n == 0) return HS_OK;
  const int64_t size = a->dtype == HS_FP32 ? 4 : 2;
  if (!aligned(a->k) || !aligned(a->v)) return HS_ERR_INVALID_ARG;
  if (!out_stride_ok(a->k_token_stride, size, a->n, a->head_dim) ||
      !out_stride_ok(a->k_head_stride, size, a->kv_heads, a->head_dim) ||
      !out_stride_ok(a->v_token_stride, size, a->n, a->head_dim) ||
      !out_stride_ok(a->v_head_stride, size, a->kv_heads, a->head_dim))
    return HS_ERR_INVALID_ARG;
  if (!on_device(v.device)) return HS_ERR_INVALID_ARG;
  p.a = *a;
  return status_of(hs::launch_read_heads(p, stream));
}

size_t hs_heads_workspace_bytes(void) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  const int sms = hs::device_sms(dev);
  return sms > 0 ? hs::heads_workspace_bytes(sms) : 0;
}

hs_status hs_attend_heads(const hs_pool* pool, int32_t layer, const hs_heads_attend* a, void* workspace,
                          size_t workspace_bytes, hs_stream_t stream) {
  HS_RANGE("hs_attend_heads");
  hs::LayerView v;
  hs::HeadsAttendParams p;
  if (!a || (a->dtype != HS_BF16 && a->dtype != HS_FP16) || !geometry(pool, layer, *a, a->cu_q, &v, &p.pages, &p.ragged))
    return HS_ERR_INVALID_ARG;
  if (a->q_heads < a->kv_heads || a->q_heads > HS_MAX_HEADS || a->q_heads % a->kv_heads || !(fabsf(a->scale) <= 0x1p127f) ||
      a->n * a->q_heads > INT32_MAX)
    return HS_ERR_INVALID_ARG;
  if (a->n == 0) return HS_OK;
  if ((a->R > 0 && !a->ctx_len) || !aligned(a->q) || !aligned(a->out)) return HS_ERR_INVALID_ARG;
  if (!stride_ok(a->q_token_stride, 2, a->n) || !stride_ok(a->q_head_stride, 2, a->q_heads) ||
      !out_stride_ok(a->out_token_stride, 2, a->n, a->head_dim) || !out_stride_ok(a->out_head_stride, 2, a->q_heads, a->head_dim))
    return HS_ERR_INVALID_ARG;
  if (!on_device(v.device)) return HS_ERR_INVALID_ARG;
  if (v.sms <= 0) return HS_ERR_CUDA;
  if (!aligned(workspace) || workspace_bytes < hs::heads_workspace_bytes(v.sms)) return HS_ERR_INVALID_ARG;
  p.a = *a;
  p.group = a->q_heads / a->kv_heads;
  p.scale_log2 = a->scale * hs::kLog2e;
  p.workspace = static_cast<float*>(workspace);
  return status_of(hs::launch_attend_heads(p, v.device, v.sms, stream));
}

}  // extern "C"
