// Internal declarations of the operators on pages of grouped heads (append, read, attention).
#pragma once

#include "hs_heads.h"
#include "latent.cuh"

namespace hs {

constexpr int kHeadsPage = HS_HEADS_PAGE;

// The pages of one layer.
struct HeadPages {
  uint8_t* base;
  int64_t page_bytes;
  int32_t num_blocks, kv_heads, max_pages;
  const int32_t* table;  // [R][max_pages]

  // Codes of a head's keys in a page; its values' follow `dim` * 64 bytes later.
  __device__ __forceinline__ uint8_t* codes(int32_t block, int head, int dim) const {
    return base + (int64_t)block * page_bytes + (int64_t)head * (2 * dim * kHeadsPage);
  }
  // The scale of a head's keys (values: kv_heads further).
  __device__ __forceinline__ float* scale(int32_t block, int head, int dim) const {
    return reinterpret_cast<float*>(base + (int64_t)block * page_bytes + (int64_t)kv_heads * (2 * dim * kHeadsPage)) + head;
  }
};

// The tokens of request r in a ragged tensor of n tokens: [t0, t0 + count).  False (and none) where the offsets do not ascend.
struct Ragged {
  const int32_t* cu;  // or nullptr: `each` tokens a request
  int32_t R, each;
  int64_t n;
  __device__ __forceinline__ bool tokens(int r, int64_t* t0, int* count) const {
    if (!cu) {
      *t0 = (int64_t)r * each;
      *count = each;
      return true;
    }
    const int a = __ldg(cu + r), b = __ldg(cu + r + 1);
    const bool ok = a >= 0 && b >= a && b <= n;
    *t0 = ok ? a : 0;
    *count = ok ? b - a : 0;
    return ok;
  }
};

struct HeadsAppendParams {
  hs_heads_append a;
  HeadPages pages;
  Ragged ragged;
};
struct HeadsReadParams {
  hs_heads_read a;
  HeadPages pages;
  Ragged ragged;
};
cudaError_t launch_append_heads(const HeadsAppendParams& p, cudaStream_t s);
cudaError_t launch_read_heads(const HeadsReadParams& p, cudaStream_t s);

struct HeadsAttendParams {
  hs_heads_attend a;
  HeadPages pages;
  Ragged ragged;
  int32_t group;     // query heads of a head of keys and values
  float scale_log2;  // scale * log2(e)
  float* workspace;
};
cudaError_t launch_attend_heads(const HeadsAttendParams& p, int dev, int sms, cudaStream_t s);
size_t heads_workspace_bytes(int sms);
// Requests of more than `limit` columns (query tokens x group); launch_attend_heads takes the others by itself.
cudaError_t launch_heads_prompt(const HeadsAttendParams& p, int limit, int dev, int sms, cudaStream_t s);
size_t heads_prompt_workspace_bytes(int sms);

}  // namespace hs
