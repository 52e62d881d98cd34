// Appending rows to the paged pool: rotation, quantisation and store in one launch, with the rotation of
// the queries' position part.
//
// Mathematics.  Rotation: 32 pairs (a, b) -> (a cos - b sin, b cos + a sin) in fp32, one rounding.
// Quantisation: e4m3 has its own exponent, so a group's scale only places the group inside the type's range
// (2^-9 .. 448): a power of two does that as well as amax / 448, at the cost of at most one binade of range
// at the low end, and in return value / scale and code * scale are exact shifts of the exponent, so that
// readers can hold the dequantised value in bf16 without a second rounding.  From amax = m * 2^e,
// m in [0.5, 1): 448 = 0.875 * 2^9, so the smallest k with amax <= 448 * 2^k is e - 9, or e - 8 when m > 0.875.
//
// Bound: HBM.  A bf16 token is 1152 B in, 656 B out, 256 B of the rotation table, and 256 B per query head.
// Split: a warp takes one token's row (16 latent values a lane, a group's maximum over 8 lanes by shuffles;
// lanes 0..3 also rotate the key), or kHeads heads of a token's queries (4 lanes a head, 8 pairs a lane; the table's
// values stay in registers over the heads).  Rows and queries are separate units so that a decode step of few tokens
// still spreads over the SMs.  Measured (fp8 rows): 64 tokens x 64 heads 2.1 us; 32768 tokens x 16 heads 40 us, 5.0 TB/s,
// x 64 heads 102 us, 5.9 TB/s.  More resident warps with fewer registers (10 or 12 blocks an SM) took 43 and 54 us.
#include "latent.cuh"
#include "vec8.cuh"

HS_CHECK_WORD

namespace hs {
namespace {

constexpr int kThreads = 128;

// The 8 pairs of quarter j of a 64-vector: x[0..7] and x[8..15] hold the elements at offsets lo(j) and hi(j).
__device__ __forceinline__ int lo(int j, bool inter) { return inter ? 16 * j : 8 * j; }
__device__ __forceinline__ int hi(int j, bool inter) { return inter ? 16 * j + 8 : 32 + 8 * j; }

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float u = a * c - b * s;
  b = b * c + a * s;
  a = u;
}
__device__ __forceinline__ void rotate(float* x, const float* c, const float* s, bool inter) {
  if (inter) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x[i], x[8 + i], c[i], s[i]);
  }
}

// kHeads: heads of a query unit.  blockIdx.y is the unit of a token: 0 its row, then its queries.  Everything that does not
// depend on another load is loaded first.
template <typename T, int kHeads>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
  const hs_append& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.n) return;
  const bool inter = a.interleaved != 0;
  const int pos = __ldg(a.positions + t);
  const int j = lane & 3;
  bool pos_ok;
  float c[8], s[8];
  auto table = [&]() {
    pos_ok = pos >= 0 && pos < a.num_positions;
    const float* cs = a.rotation + (int64_t)(pos_ok ? pos : 0) * kRope;
    Vec8<float> x, y;
    x.load(cs + 8 * j);
    y.load(cs + 32 + 8 * j);
    x.values(c);
    y.values(s);
  };
  if (blockIdx.y > 0) {
    const T* q = static_cast<const T*>(a.q_rope) + t * a.q_token_stride;
    T* o = static_cast<T*>(a.q_out) + t * a.q_out_token_stride;
    const int h0 = (blockIdx.y - 1) * kHeads + (lane >> 2);
    Vec8<T> in[kHeads / 8][2];
#pragma unroll
    for (int i = 0; i < kHeads / 8; ++i) {
      const int h = min(h0 + 8 * i, a.heads - 1);
      in[i][0].load(q + h * a.q_head_stride + lo(j, inter));
      in[i][1].load(q + h * a.q_head_stride + hi(j, inter));
    }
    table();
#pragma unroll
    for (int i = 0; i < kHeads / 8; ++i) {
      const int h = h0 + 8 * i;
      float x[16];
      in[i][0].values(x);
      in[i][1].values(x + 8);
      rotate(x, c, s, inter);
      if (!pos_ok)
        for (int e = 0; e < 16; ++e) x[e] = 0.f;
      if (h < a.heads) {
        Vec8<T>::store(o + h * a.q_out_head_stride + lo(j, inter), x);
        Vec8<T>::store(o + h * a.q_out_head_stride + hi(j, inter), x + 8);
      }
    }
    return;
  }
  const int row = __ldg(a.rows + t);
  const T* src = static_cast<const T*>(a.latent) + t * a.latent_stride + 16 * lane;
  Vec8<T> in[2], key[2];
  in[0].load(src);
  in[1].load(src + 8);
  if (lane < 4) {
    const T* k = static_cast<const T*>(a.rope) + t * a.rope_stride;
    key[0].load(k + lo(j, inter));
    key[1].load(k + hi(j, inter));
  }
  float r[16];
  pos_ok = pos >= 0 && pos < a.num_positions;
  if (lane < 4) {
    table();
    key[0].values(r);
    key[1].values(r + 8);
    rotate(r, c, s, inter);
  }
  const bool row_ok = row >= 0 && row < p.num_rows;
  if (lane == 0 && ((row != -1 && !row_ok) || !pos_ok)) report(a.status, HS_ERR_ID_RANGE);
  if (!row_ok || !pos_ok || !HS_CHECK((int64_t)row * p.row_bytes + p.row_bytes <= p.num_rows * p.row_bytes, kChkPoolRow)) return;
  uint8_t* dst = p.base + (int64_t)row * p.row_bytes;
  float x[16];
  in[0].values(x);
  in[1].values(x + 8);
  int rope_at;
  if (p.row_bytes == HS_ROW_BYTES_FP8) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float m = fabsf(x[i]);
      if (m <= 3.402823466e38f) amax = fmaxf(amax, m);  // finite values only
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    const float scale = group_scale(amax);
    const float inv = 1.f / scale;  // an exact power of two: scale is in [2^-126, 2^120]
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fabsf(x[i]) <= 3.402823466e38f ? x[i] * inv : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = e4m3x2(x[4 * i], x[4 * i + 1]) | e4m3x2(x[4 * i + 2], x[4 * i + 3]) << 16;
    *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    if ((lane & 7) == 0) reinterpret_cast<float*>(dst + kLatent)[lane >> 3] = scale;
    rope_at = kLatent + 16;
  } else {
    Vec8<__nv_bfloat16>::store(reinterpret_cast<__nv_bfloat16*>(dst) + 16 * lane, x);
    Vec8<__nv_bfloat16>::store(reinterpret_cast<__nv_bfloat16*>(dst) + 16 * lane + 8, x + 8);
    rope_at = 2 * kLatent;
  }
  if (lane < 4) {
    __nv_bfloat16* k = reinterpret_cast<__nv_bfloat16*>(dst + rope_at);
    Vec8<__nv_bfloat16>::store(k + lo(j, inter), r);
    Vec8<__nv_bfloat16>::store(k + hi(j, inter), r + 8);
  }
}

template <int kHeads>
void launch_heads(const AppendParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.a.n + kThreads / 32 - 1) / (kThreads / 32)), 1 + (p.a.heads + kHeads - 1) / kHeads);
  if (p.a.dtype == HS_BF16)
    append_kernel<__nv_bfloat16, kHeads><<<grid, kThreads, 0, s>>>(p);
  else if (p.a.dtype == HS_FP16)
    append_kernel<__half, kHeads><<<grid, kThreads, 0, s>>>(p);
  else
    append_kernel<float, kHeads><<<grid, kThreads, 0, s>>>(p);
}

}  // namespace

uint32_t check_take_append() {
#if HS_CHECKED
  unsigned v = 0u, z = 0u;
  if (cudaMemcpyFromSymbol(&v, hs_check_word_, sizeof(v)) != cudaSuccess ||
      cudaMemcpyToSymbol(hs_check_word_, &z, sizeof(z)) != cudaSuccess) {
    cudaGetLastError();
    return 0xFFFFFFFFu;
  }
  return v;
#else
  return 0u;
#endif
}

cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t s) {
  // few tokens are spread further (512 x 64 heads: 2.9 us with 8 heads a warp and 3.4 with 16); many take fewer reads of the
  // table (32768 x 64: 102 us with 16, 106 with 8)
  if (p.a.n * (1 + p.a.heads / 16) < 64 * (int64_t)sms)
    launch_heads<8>(p, s);
  else
    launch_heads<16>(p, s);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hs
