// Internal declarations of the latent-row operators (append, absorbed and expanded attention).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_once.cuh"
#include "hs_internal.cuh"
#include "hs_latent.h"

namespace hs {

constexpr int kLatent = HS_LATENT_DIM;
constexpr int kRope = HS_ROPE_DIM;
constexpr int kNope = HS_NOPE_DIM;
constexpr int kValue = HS_VALUE_DIM;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One layer of a pool, as these operators see it.
struct LayerView {
  uint8_t* base;
  int32_t row_bytes, page_size, num_blocks;
  int64_t num_rows;
  int device, sms;
};
// Fills v for a layer of the pool; false when the layer or the pool is not there.
bool pool_layer(const hs_pool* pool, int32_t layer, LayerView* v);
int device_sms(int dev);

struct AppendParams {
  hs_append a;
  uint8_t* base;
  int64_t num_rows;
  int32_t row_bytes;
};
cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t s);

struct ReadRowsParams {
  hs_read_latent a;
  const uint8_t* base;
  int64_t num_rows;
  int32_t row_bytes;
};
cudaError_t launch_read_rows(const ReadRowsParams& p, cudaStream_t s);

// Absorbed attention.  An item is what shares keys: a token of a rows call (cols = heads), a request of a
// pages call (cols = positions * heads; column c is position c / heads, head c % heads).
struct AttendParams {
  const uint8_t* base;
  int32_t row_bytes, page_size, num_blocks;
  int64_t num_rows;
  int32_t paged;             // 1: a pages call, 0: a rows call
  const int32_t* rows;       // rows call: [items][K] (may be null when K = 0)
  int32_t K;
  const int32_t* table;      // pages call: [items][max_pages]
  const int32_t* ctx_len;
  int32_t max_pages;
  int32_t items, P, heads, cols;
  const __nv_bfloat16* q_latent;
  int64_t ql_tok, ql_head;
  const __nv_bfloat16* q_rope;
  int64_t qr_tok, qr_head;
  __nv_bfloat16* out;
  int64_t out_tok, out_head;
  float* lse;
  float scale_log2;          // scale * log2(e)
  int32_t* status;
  float* workspace;
};
// dev: the current device, sms its number of SMs.
cudaError_t launch_attend(const AttendParams& p, int dev, int sms, cudaStream_t s);
size_t attend_workspace_bytes(int sms);

cudaError_t launch_expanded(const hs_expanded& a, int dev, int sms, cudaStream_t s);

// Records a data error: the status word keeps the largest code seen.
__device__ __forceinline__ void report(int32_t* status, int32_t code) {
  if (status) atomicMax(status, code);
}

}  // namespace hs
