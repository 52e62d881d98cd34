// Eight values at a time, in any of the element types, and the quantisation of values to e4m3 codes with a power-of-two scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace hs {

template <typename T>
struct Vec8;  // 8 values of T as they lie in memory <-> 8 floats
template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void values(float* x) const {
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
  uint4 v;
  __device__ __forceinline__ void load(const __half* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void values(float* x) const {
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
  float4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = reinterpret_cast<const float4*>(p)[0];
    v[1] = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void values(float* x) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) x[4 * i] = v[i].x, x[4 * i + 1] = v[i].y, x[4 * i + 2] = v[i].z, x[4 * i + 3] = v[i].w;
  }
  static __device__ __forceinline__ void store(float* p, const float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
};

// The smallest power of two, at least 2^-126, with amax <= 448 times it.  From amax = m * 2^e, m in [0.5, 1): 448 = 0.875 * 2^9,
// so it is 2^(e - 9), or 2^(e - 8) when m > 0.875.
__device__ __forceinline__ float power_scale(float amax) {
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
// The scale of a group of latent values: 1 for a group of zeros.
__device__ __forceinline__ float group_scale(float amax) { return amax == 0.f ? 1.f : power_scale(amax); }

// Larger of amax and |x|, x finite; a value that is infinite or NaN does not count.
__device__ __forceinline__ float max_finite(float amax, float x) {
  const float m = fabsf(x);
  return m <= 3.402823466e38f ? fmaxf(amax, m) : amax;
}
// x / scale as what is to be encoded: NaN for a value that is not finite.
__device__ __forceinline__ float scaled_finite(float x, float inv) {
  return fabsf(x) <= 3.402823466e38f ? x * inv : __uint_as_float(0x7FC00000u);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo_value, float hi_value) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi_value), "f"(lo_value));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) { return e4m3x2(a, b) | e4m3x2(c, d) << 16; }

// 4 e4m3 codes -> 4 fp16 (exact)
__device__ __forceinline__ uint2 half_of_codes(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}
// 4 e4m3 codes -> 4 floats
__device__ __forceinline__ void float_of_codes(uint32_t w, float* x) {
  const uint2 h = half_of_codes(w);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

}  // namespace hs
