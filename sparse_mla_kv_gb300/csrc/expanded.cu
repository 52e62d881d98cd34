// Attention over keys and values expanded to every head: prompts and prompt chunks.
//
// First form: one warp per (query, head), running maximum and sum.
#include "latent.cuh"

namespace hs {
namespace {

__global__ void __launch_bounds__(128) expanded_kernel(const hs_expanded a, float scale_log2) {
  const int lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (u >= a.q_tokens * a.heads) return;
  if (u == 0 && lane == 0)
    for (int s = 0; s < a.seqs; ++s) {
      const int x0 = __ldg(a.cu_q + s), x1 = __ldg(a.cu_q + s + 1), y0 = __ldg(a.cu_k + s), y1 = __ldg(a.cu_k + s + 1);
      if (x0 < 0 || x1 < x0 || x1 > a.q_tokens || y0 < 0 || y1 < y0 || y1 > a.k_tokens) report(a.status, HS_ERR_ID_RANGE);
    }
  const int64_t i = u / a.heads;
  const int h = (int)(u - i * a.heads);
  int b = -1, q0 = 0, q1 = 0;
  for (int s = 0; s < a.seqs; ++s) {
    q0 = __ldg(a.cu_q + s), q1 = __ldg(a.cu_q + s + 1);
    if (i >= q0 && i < q1) {
      b = s;
      break;
    }
  }
  if (b < 0) return;
  const int k0 = __ldg(a.cu_k + b), k1 = __ldg(a.cu_k + b + 1);
  if (q0 < 0 || q1 > a.q_tokens || k0 < 0 || k1 < k0 || k1 > a.k_tokens) return;
  int64_t keys = k1 - k0;
  if (a.causal) keys = min(keys, (i - q0) + 1 + keys - (q1 - q0));
  const __nv_bfloat16* qn = static_cast<const __nv_bfloat16*>(a.q_nope) + i * a.qn_token_stride + h * a.qn_head_stride;
  const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q_rope) + i * a.qr_token_stride + h * a.qr_head_stride;
  float q[6], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  for (int x = 0; x < 4; ++x) q[x] = __bfloat162float(qn[4 * lane + x]);
  for (int x = 0; x < 2; ++x) q[4 + x] = __bfloat162float(qr[2 * lane + x]);
  for (int64_t j = k0; j < k0 + keys; ++j) {
    const __nv_bfloat16* kn = static_cast<const __nv_bfloat16*>(a.k_nope) + j * a.kn_token_stride + h * a.kn_head_stride;
    const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(a.k_rope) + j * a.kr_token_stride;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + j * a.v_token_stride + h * a.v_head_stride;
    float s = 0.f;
    for (int x = 0; x < 4; ++x) s += q[x] * __bfloat162float(kn[4 * lane + x]);
    for (int x = 0; x < 2; ++x) s += q[4 + x] * __bfloat162float(kr[2 * lane + x]);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= scale_log2;
    const float top = fmaxf(m, s);
    const float keep = m == -INFINITY ? 0.f : exp2f(m - top), w = exp2f(s - top);
    l = l * keep + w;
    for (int x = 0; x < 4; ++x) acc[x] = acc[x] * keep + w * __bfloat162float(v[4 * lane + x]);
    m = top;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + i * a.out_token_stride + h * a.out_head_stride;
  for (int x = 0; x < 4; ++x) o[4 * lane + x] = __float2bfloat16_rn(acc[x] * inv);
  if (lane == 0 && a.lse) a.lse[i * a.heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

cudaError_t launch_expanded(const hs_expanded& a, int sms, cudaStream_t s) {
  (void)sms;
  const int64_t blocks = (a.q_tokens * a.heads + 3) / 4;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  expanded_kernel<<<(unsigned)blocks, 128, 0, s>>>(a, a.scale * kLog2e);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hs
