// Absorbed latent attention over the rows of the paged pool.
//
// First form: one CTA per (query token, head), a warp per key in turn, running maximum and sum per warp.
#include "latent.cuh"

namespace hs {
namespace {

constexpr int kWarps = 4;

// Row of key k of item i, or -1.
__device__ __forceinline__ int64_t key_row(const AttendParams& p, int i, int k) {
  if (!p.paged) {
    const int r = __ldg(p.rows + (int64_t)i * p.K + k);
    if (r >= 0 && r < p.num_rows) return r;
    if (r != -1) report(p.status, HS_ERR_ID_RANGE);
    return -1;
  }
  const int page = k / p.page_size;
  const int b = __ldg(p.table + (int64_t)i * p.max_pages + page);
  if (b >= 0 && b < p.num_blocks) return (int64_t)b * p.page_size + (k - page * p.page_size);
  report(p.status, HS_ERR_TABLE_RANGE);
  return -1;
}

__device__ __forceinline__ float bf16_round(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

__global__ void __launch_bounds__(32 * kWarps) attend_kernel(const AttendParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.x, col = blockIdx.y;
  const int pos = col / p.heads, head = col - pos * p.heads;
  const int64_t tok = (int64_t)item * p.P + pos;
  int keys = p.K;
  if (p.paged) {
    const int64_t room = (int64_t)p.max_pages * p.page_size;
    int len = __ldg(p.ctx_len + item);
    if (len > room) report(p.status, HS_ERR_TABLE_RANGE);
    keys = max(0, min((int)room, len - p.P + 1 + pos));
  }
  // lane: latent values 16*lane .. +15, rope values 2*lane, 2*lane+1
  float q[16], qr[2], acc[16];
  for (int i = 0; i < 16; ++i) {
    q[i] = __bfloat162float(p.q_latent[tok * p.ql_tok + head * p.ql_head + 16 * lane + i]);
    acc[i] = 0.f;
  }
  for (int i = 0; i < 2; ++i) qr[i] = __bfloat162float(p.q_rope[tok * p.qr_tok + head * p.qr_head + 2 * lane + i]);
  float m = -INFINITY, l = 0.f;
  for (int k = warp; k < keys; k += kWarps) {
    const int64_t row = key_row(p, item, k);
    if (row < 0) continue;
    const uint8_t* src = p.base + row * p.row_bytes;
    float c[16];
    const __nv_bfloat16* rope;
    if (p.row_bytes == HS_ROW_BYTES_FP8) {
      const float scale = reinterpret_cast<const float*>(src + kLatent)[lane >> 3];
      const uint4 v = reinterpret_cast<const uint4*>(src)[lane];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      for (int i = 0; i < 8; ++i) {
        uint32_t h;
        const uint16_t two = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        c[2 * i] = bf16_round(f.x * scale);
        c[2 * i + 1] = bf16_round(f.y * scale);
      }
      rope = reinterpret_cast<const __nv_bfloat16*>(src + kLatent + 16);
    } else {
      const __nv_bfloat16* lat = reinterpret_cast<const __nv_bfloat16*>(src);
      for (int i = 0; i < 16; ++i) c[i] = __bfloat162float(lat[16 * lane + i]);
      rope = lat + kLatent;
    }
    float s = 0.f;
    for (int i = 0; i < 16; ++i) s += q[i] * c[i];
    for (int i = 0; i < 2; ++i) s += qr[i] * __bfloat162float(rope[2 * lane + i]);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= p.scale_log2;
    const float top = fmaxf(m, s);
    const float keep = m == -INFINITY ? 0.f : exp2f(m - top), w = exp2f(s - top);
    l = l * keep + w;
    for (int i = 0; i < 16; ++i) acc[i] = acc[i] * keep + w * c[i];
    m = top;
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kLatent];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int i = 0; i < 16; ++i) so[warp][16 * lane + i] = acc[i];
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  float total = 0.f, f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - top);
    total += f[w] * sl[w];
  }
  const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
  for (int d = threadIdx.x; d < kLatent; d += 32 * kWarps) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w) o += f[w] * so[w][d];
    p.out[tok * p.out_tok + head * p.out_head + d] = __float2bfloat16_rn(o * inv);
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[tok * p.heads + head] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
}

}  // namespace

size_t attend_workspace_bytes(int sms) { return (size_t)sms * 2 * 64 * (kLatent + 4) * sizeof(float); }

cudaError_t launch_attend(const AttendParams& p, int sms, cudaStream_t s) {
  (void)sms;
  if (p.cols > 65535) return cudaErrorInvalidValue;
  attend_kernel<<<dim3((unsigned)p.items, (unsigned)p.cols), 32 * kWarps, 0, s>>>(p);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hs
