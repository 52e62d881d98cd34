// Reading latent rows back by id.
//
// Mathematics.  value = code * scale in fp32, rounded once to the output's type: exact in bf16 for the powers of two that
// hs_append_rows writes.
//
// Bound: HBM.  An fp8 row is 656 B in and 1152 B out in 16 bits.  Split: a warp takes kRows rows and loads all of them before
// it converts any; a lane has 8 consecutive values of every 256, so that a warp's stores are whole lines.  131072 fp8 rows in bf16:
// 38 us, 6.2 TB/s; 1024 rows 2.2 us.
#include "latent.cuh"
#include "vec8.cuh"

HS_CHECK_WORD

namespace hs {
namespace {

constexpr int kThreads = 128, kRows = 2;

template <typename T, bool kF8>
__global__ void __launch_bounds__(kThreads) read_rows_kernel(const ReadRowsParams p) {
  const hs_read_latent& a = p.a;
  constexpr int kRowBytes = kF8 ? HS_ROW_BYTES_FP8 : HS_ROW_BYTES_BF16;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kRows;
  if (t0 >= a.n) return;
  const int32_t mine = lane < kRows && t0 + lane < a.n ? __ldg(a.rows + t0 + lane) : -1;
  const bool bad = mine < -1 || mine >= p.num_rows;
  if (bad) report(a.status, HS_ERR_ID_RANGE);
  const int32_t valid = bad ? -1 : mine;
  uint2 codes[kRows][2];
  float scale[kRows][2];
  uint4 wide[kRows][2], rope[kRows];
  int row[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    row[i] = __shfl_sync(0xFFFFFFFFu, valid, i);
    if (row[i] < 0) continue;
    if (!HS_CHECK((int64_t)row[i] < p.num_rows, kChkPoolRow)) row[i] = 0;
    const uint8_t* src = p.base + (int64_t)row[i] * kRowBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (kF8) {
        codes[i][h] = __ldg(reinterpret_cast<const uint2*>(src + 256 * h) + lane);
        scale[i][h] = __ldg(reinterpret_cast<const float*>(src + kLatent) + 2 * h + (lane >> 4));
      } else {
        wide[i][h] = __ldg(reinterpret_cast<const uint4*>(src + 512 * h) + lane);
      }
    }
    if (lane < 8) rope[i] = __ldg(reinterpret_cast<const uint4*>(src + kRowBytes - 2 * kRope) + lane);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (t0 + i >= a.n) return;
    T* latent = static_cast<T*>(a.latent) + (t0 + i) * a.latent_stride;
    T* out_rope = static_cast<T*>(a.rope) + (t0 + i) * a.rope_stride;
    float x[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (row[i] < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
      } else if constexpr (kF8) {
        float_of_codes(codes[i][h].x, x);
        float_of_codes(codes[i][h].y, x + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= scale[i][h];
      } else {
        Vec8<__nv_bfloat16>{wide[i][h]}.values(x);
      }
      Vec8<T>::store(latent + 256 * h + 8 * lane, x);
    }
    if (lane < 8) {
      if (row[i] < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
      } else {
        Vec8<__nv_bfloat16>{rope[i]}.values(x);
      }
      Vec8<T>::store(out_rope + 8 * lane, x);
    }
  }
}

template <typename T>
void launch(const ReadRowsParams& p, cudaStream_t s) {
  constexpr int kPer = kThreads / 32 * kRows;
  const unsigned grid = (unsigned)((p.a.n + kPer - 1) / kPer);
  if (p.row_bytes == HS_ROW_BYTES_FP8)
    read_rows_kernel<T, true><<<grid, kThreads, 0, s>>>(p);
  else
    read_rows_kernel<T, false><<<grid, kThreads, 0, s>>>(p);
}

}  // namespace

uint32_t check_take_read_rows() {
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

cudaError_t launch_read_rows(const ReadRowsParams& p, cudaStream_t s) {
  if (p.a.dtype == HS_BF16)
    launch<__nv_bfloat16>(p, s);
  else if (p.a.dtype == HS_FP16)
    launch<__half>(p, s);
  else
    launch<float>(p, s);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hs
