// What the attention kernels over pages of grouped heads share.
#pragma once

#include "heads.cuh"
#include "tc.cuh"
#include "vec8.cuh"

namespace hs {
namespace heads {

// Log2 units.  A new reference R puts the largest t at kTop above it, and moves when a t passes it by kLazy: fp16 weights are
// normal from 2^-14 to 2^16.  kFar: see heads_attend.cu.
constexpr float kTop = 7.f, kLazy = 15.f, kFar = 60.f;
// Scores beyond kLarge, in log2 units, are taken from an anchor of their own first: added to log2(sv) as they are, they would
// swallow it, and a product that is not rounded could pass the rounded largest by far.
constexpr float kLarge = 65536.f;

// Scores that are not finite.  Maxima pass NaN over; the sums of weights have it, whatever the reference.  The largest of the scores that
// a row sees in a page is at most kMost: a row that sees +infinity has its anchor there, weights of +infinity and no others, and so
// has l.  A row that has seen a token has an m of kLowest at least, also where all its scores are -infinity and l is zero: with
// m = -infinity and l = 0 it has seen none.
constexpr float kMost = 3.402823466e38f, kLowest = -kMost;
__device__ __forceinline__ bool saw_none(float m, float l) { return m == -INFINITY && l == 0.f; }
// What a row's weighted sums are multiplied by, one factor after the other: 2^(ref - m) / l, by halves; zeros for a row that saw no
// token, NaN where the weights' sum is zero, infinite or NaN.
__device__ __forceinline__ float2 result_factors(float ref, float m, float l) {
  if (saw_none(m, l)) return make_float2(0.f, 0.f);
  const float up = exp2f(0.5f * (ref - m));
  return make_float2(up, l > 0.f && l < INFINITY ? up / l : __uint_as_float(0x7FC00000u));
}
__device__ __forceinline__ float result_lse(float anchor, float m, float l) { return (anchor + (m + log2f(l))) * kLn2; }

// A call's work is numbered in tiles, and a run of them is what one worker takes.
struct RunHeader {
  int64_t run, total;  // tiles of a worker, of the call
};
struct RunRecord {
  int64_t begin, end;        // tiles of the unit that begins in this run and is cut by its end; begin == end: none
  int64_t t0;                // first query token of its request
  int32_t head, group, cols, unused[3];
};
static_assert(sizeof(RunHeader) == 16 && sizeof(RunRecord) == 48, "the parts stay aligned to 16 bytes");

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts_u(uint32_t a, uint32_t x) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory"); }
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack(bool f16, float lo, float hi) { return f16 ? pack_half(lo, hi) : tc::pack_bf16(lo, hi); }
// 0x80 in every byte that is the NaN code
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Waits, and tells the whole warp when one of its lanes gave up.
__device__ __forceinline__ void await(tc::Waiter& w, uint32_t bar, uint32_t parity) {
  w.wait(bar, parity);
  w.dead = __any_sync(0xFFFFFFFFu, w.dead);
}
// a / b, neither negative: in 32 bits where that does (a division in 64 is a long chain).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The cut units, for the kernels that join their parts: numbers of the records in two lists (units of more than `few` parts are in
// the second), by the whole block of kThreads threads.  kMax: records at most.
template <int kThreads, int kMax>
struct CutLists {
  uint16_t at[2][kMax];
  static constexpr int kRounds = kMax / kThreads, kWarps = kThreads / 32, kCounts = kRounds * kWarps, kPer = (kCounts + 31) / 32;
  uint16_t counts[2][32 * kPer];  // of a round's warps, rounds one after the other
  __device__ __forceinline__ void build(const RunRecord* records, int n, int64_t run, int few, int (&total)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t begin[kRounds], end[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int i = k * kThreads + threadIdx.x;
      begin[k] = end[k] = 0;
      if (i < n) begin[k] = records[i].begin, end[k] = records[i].end;
    }
    unsigned those[2][kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const bool is = end[k] > begin[k], many = is && end[k] > (k * kThreads + (int)threadIdx.x + few) * run;
      those[0][k] = __ballot_sync(0xFFFFFFFFu, is && !many), those[1][k] = __ballot_sync(0xFFFFFFFFu, many);
      if (lane == 0) counts[0][k * kWarps + warp] = __popc(those[0][k]), counts[1][k * kWarps + warp] = __popc(those[1][k]);
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      // each warp adds all counts up, kPer a lane
      int count[kPer], mine = 0;
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        count[x] = lane * kPer + x < kCounts ? counts[y][lane * kPer + x] : 0;
        mine += count[x];
      }
      int upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int z = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += z;
      }
      total[y] = __shfl_sync(0xFFFFFFFFu, upto, 31);
      int before[kPer];
      before[0] = upto - mine;
#pragma unroll
      for (int x = 1; x < kPer; ++x) before[x] = before[x - 1] + count[x - 1];
#pragma unroll
      for (int k = 0; k < kRounds; ++k) {
        const int c = k * kWarps + warp;
        int first = 0;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          const int z = __shfl_sync(0xFFFFFFFFu, before[x], c / kPer);
          if (c % kPer == x) first = z;
        }
        if (those[y][k] >> lane & 1) at[y][first + __popc(those[y][k] & ((1u << lane) - 1))] = (uint16_t)(k * kThreads + threadIdx.x);
      }
    }
    __syncthreads();
  }
};

// What parts of a column's (or row's) results have been joined so far: the references, the sum of weights.  A part's statistics are
// (ref, m, l, anchor); those of a row that has seen no token are left out.
struct Joined {
  float anchor = -INFINITY, ref = -INFINITY, m = -INFINITY, l = 0.f;
  // Joins a part; returns what the results so far, and the part's, are to be multiplied by.
  __device__ __forceinline__ float2 join(float4 st) {
    if (saw_none(st.y, st.z)) return make_float2(1.f, 0.f);
    const float to = fmaxf(anchor, st.w), here = st.w - to;
    if (to != anchor) ref += anchor - to, m += anchor - to, anchor = to;
    const float now = fmaxf(ref, st.x + here), now_m = fmaxf(m, st.y + here);
    const float2 f = make_float2(ref == now ? 1.f : exp2f(ref - now), st.x == -INFINITY ? 0.f : exp2f(st.x + here - now));
    l = l * (m == now_m ? 1.f : exp2f(m - now_m)) + st.z * (st.y + here == now_m ? 1.f : exp2f(st.y + here - now_m));
    ref = now, m = now_m;
    return f;
  }
};

// What the queries take of the scale; the rest is a factor of the scores, kept above zero.
__device__ __forceinline__ float scale_sign(float scale) { return scale < 0.f ? -1.f : scale > 0.f ? 1.f : 0.f; }
// The exponent field e of a power of two that brings a query's largest magnitude into fp16's range, by division: left as they
// are (127) when it is in 2^-2 .. 2^15, where fp16 keeps all but what is 2^-23 of it.
__device__ __forceinline__ int query_field(float top) {
  const int e = (int)(__float_as_uint(top) >> 23);
  return top == 0.f || (e >= 125 && e < 142) ? 127 : min(max(e - 14, 1), 240);
}
__device__ __forceinline__ float power_of_field(int e) { return __uint_as_float((uint32_t)e << 23); }

}  // namespace heads
}  // namespace hs
