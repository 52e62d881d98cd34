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
// lanes 0..3 also rotate the key), or up to kHeadsPerUnit heads of a token's queries (4 lanes a head, 8 pairs
// a lane; the table's values stay in registers over the heads).  Rows and queries are separate units so that a
// decode step of few tokens still spreads over the SMs.
#include "latent.cuh"

namespace hs {
namespace {

constexpr int kThreads = 128;

template <typename T>
struct Vec8;  // 8 values of T <-> 8 floats
template <>
struct Vec8<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<__half> {
  static __device__ __forceinline__ void load(const __half* p, float* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void store(__half* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<float> {
  static __device__ __forceinline__ void load(const float* p, float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = reinterpret_cast<const float4*>(p)[i];
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  }
  static __device__ __forceinline__ void store(float* p, const float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
};

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

// Power-of-two scale of a group whose largest finite magnitude is amax (see the head of this file).
__device__ __forceinline__ float group_scale(float amax) {
  if (amax == 0.f) return 1.f;
  const uint32_t b = __float_as_uint(amax);
  const int field = (int)(b >> 23);  // 0 for subnormal amax: its scale is the smallest one
  int k = -126;
  if (field > 0) {
    const uint32_t mant = b & 0x7FFFFFu;           // amax = (1 + mant / 2^23) * 2^(field - 127)
    k = field - 126 - 9 + (mant > 0x600000u ? 1 : 0);  // frexp exponent e = field - 126; 0.875 = 1.75 / 2
    k = max(k, -126);
  }
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo_value, float hi_value) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi_value), "f"(lo_value));
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p, int units_per_token,
                                                          int heads_per_unit, int64_t units) {
  const hs_append& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (u >= units) return;
  const int64_t t = u / units_per_token;
  const int part = (int)(u - t * units_per_token);
  const bool inter = a.interleaved != 0;
  const int pos = __ldg(a.positions + t);
  const bool pos_ok = pos >= 0 && pos < a.num_positions;
  const float* cs = a.rotation + (int64_t)(pos_ok ? pos : 0) * kRope;
  const int j = lane & 3;
  float c[8], s[8];
  if (part > 0 || lane < 4) {
    Vec8<float>::load(cs + 8 * j, c);
    Vec8<float>::load(cs + 32 + 8 * j, s);
  }
  if (part > 0) {
    const T* q = static_cast<const T*>(a.q_rope) + t * a.q_token_stride;
    T* o = static_cast<T*>(a.q_out) + t * a.q_out_token_stride;
    const int h0 = (part - 1) * heads_per_unit;
    const int h1 = min(a.heads, h0 + heads_per_unit);
    for (int h = h0 + (lane >> 2); h < h1; h += 8) {
      float x[16];
      Vec8<T>::load(q + h * a.q_head_stride + lo(j, inter), x);
      Vec8<T>::load(q + h * a.q_head_stride + hi(j, inter), x + 8);
      rotate(x, c, s, inter);
      if (!pos_ok)
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
      Vec8<T>::store(o + h * a.q_out_head_stride + lo(j, inter), x);
      Vec8<T>::store(o + h * a.q_out_head_stride + hi(j, inter), x + 8);
    }
    return;
  }
  const int row = __ldg(a.rows + t);
  const bool row_ok = row >= 0 && row < p.num_rows;
  if (lane == 0 && ((row != -1 && !row_ok) || !pos_ok)) report(a.status, HS_ERR_ID_RANGE);
  if (!row_ok || !pos_ok) return;
  uint8_t* dst = p.base + (int64_t)row * p.row_bytes;
  const T* src = static_cast<const T*>(a.latent) + t * a.latent_stride + 16 * lane;
  float x[16];
  Vec8<T>::load(src, x);
  Vec8<T>::load(src + 8, x + 8);
  float r[16];
  if (lane < 4) {
    const T* k = static_cast<const T*>(a.rope) + t * a.rope_stride;
    Vec8<T>::load(k + lo(j, inter), r);
    Vec8<T>::load(k + hi(j, inter), r + 8);
    rotate(r, c, s, inter);
  }
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

}  // namespace

cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t s) {
  const int heads_per_unit = 8;
  const int upt = 1 + (p.a.heads + heads_per_unit - 1) / heads_per_unit;
  const int64_t units = p.a.n * upt;
  const int64_t blocks = (units + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  (void)sms;
  if (p.a.dtype == HS_BF16)
    append_kernel<__nv_bfloat16><<<(unsigned)blocks, kThreads, 0, s>>>(p, upt, heads_per_unit, units);
  else if (p.a.dtype == HS_FP16)
    append_kernel<__half><<<(unsigned)blocks, kThreads, 0, s>>>(p, upt, heads_per_unit, units);
  else
    append_kernel<float><<<(unsigned)blocks, kThreads, 0, s>>>(p, upt, heads_per_unit, units);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hs
