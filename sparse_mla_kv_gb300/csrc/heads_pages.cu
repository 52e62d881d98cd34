// Pages of grouped heads: quantising new keys and values into them, and reading tokens back.
//
// Mathematics.  The scale of a page's keys (or values) of a head is the smallest power of two that brings them into e4m3's
// range, so that x / scale, code * scale and, when a later token raises the scale, code * old / new are exact but for e4m3's
// own rounding.  A scale only rises while a page fills: a token rounded once is rounded again only when the page's largest
// value passes a power of two.
//
// Layout.  Keys lie token by token and values dimension by dimension, in blocks of 64 x 64 codes: as the attention's products
// read them.  The values are turned on the way, four tokens x eight dimensions a thread, in registers.
//
// Split: a block takes one page of one head, keys and values.  A page is found by a number that grows faster than the pages
// can: request r's pages start at cu[r] / 64 + 2 r, since n tokens touch at most (n - 2) / 64 + 2 pages.
// Bound: HBM for prompts (an element is 2 B in and 1 B out), latency for single tokens: offsets, table, scale, codes.
#include "heads.cuh"
#include "vec8.cuh"

HS_CHECK_WORD

namespace hs {
namespace {

// One page of a request: tokens at its places [lo, hi), of which the first is row `row` of the ragged tensor.
struct PageWork {
  int32_t request, page, lo, hi;
  int64_t row;
};

// The page with number i, found by the whole block; false where there is none or cu does not ascend.  first(r, count) is the
// position of request r's first token, negative where the request has none to give.  Block 0 reports.
template <typename First>
__device__ __forceinline__ bool find_page(const Ragged& g, int64_t i, bool reports, int32_t* status, First first, PageWork* w) {
  __shared__ PageWork found;
  if (threadIdx.x == 0) found.request = -1;
  __syncthreads();
  bool bad = false;
  for (int r = threadIdx.x; r < g.R; r += blockDim.x) {
    int64_t t0;
    int count;
    bad |= !g.tokens(r, &t0, &count);
    const int64_t base = t0 / kHeadsPage + 2 * (int64_t)r;
    const int from = first(r, count);
    if (count > 0 && from < 0 && reports) report(status, HS_ERR_ID_RANGE);
    if (count <= 0 || from < 0 || i < base) continue;
    const int64_t page = from / kHeadsPage + (i - base), at = page * kHeadsPage;
    if (at >= (int64_t)from + count) continue;
    found.page = (int32_t)page;
    found.lo = (int32_t)(from > at ? from - at : 0);
    found.hi = (int32_t)min((int64_t)kHeadsPage, (int64_t)from + count - at);
    found.row = t0 + at + found.lo - from;
    found.request = r;
  }
  bad = __syncthreads_or(bad);
  if (bad && reports && threadIdx.x == 0) report(status, HS_ERR_ID_RANGE);
  *w = found;
  return !bad && w->request >= 0;
}

// The pool block of a page, or -1 (and a report) where the table has none.
__device__ __forceinline__ int block_of(const HeadPages& p, const PageWork& w, int32_t* status) {
  int b = -1;
  if (w.page < p.max_pages) b = __ldg(p.table + (int64_t)w.request * p.max_pages + w.page);
  if (b >= 0 && b < p.num_blocks) return b;
  if (threadIdx.x == 0) report(status, HS_ERR_TABLE_RANGE);
  return -1;
}

// Who has what of a page, for blocks of 2 D threads.  Keys: the 8 dimensions of chunk key_chunk, tokens key_token + 16 i.
// Values: chunk value_chunk, tokens 4 quad .. 4 quad + 3.
template <int D>
struct Place {
  static constexpr int kChunks = D / 8;
  int key_chunk, key_token, value_chunk, quad;
  __device__ __forceinline__ Place() {
    const int t = threadIdx.x, lane = t & 31;
    key_chunk = t % kChunks;
    key_token = t / kChunks;
    value_chunk = 2 * (t >> 5) + (lane & 1);
    quad = lane >> 1;
  }
  __device__ __forceinline__ int key_at(int token) const { return (key_chunk >> 3) * 4096 + token * 64 + (key_chunk & 7) * 8; }
  __device__ __forceinline__ int value_at(int e) const {
    const int d = 8 * value_chunk + e;
    return (d >> 6) * 4096 + (d & 63) * 64 + 4 * quad;
  }
};

// blockIdx.z: 0 the keys, 1 the values.
template <typename T, int D>
__global__ void __launch_bounds__(2 * D) append_heads_kernel(const HeadsAppendParams p) {
  const hs_heads_append& a = p.a;
  const bool reports = blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
  PageWork w;
  auto first = [&](int r, int count) {
    const int ctx = __ldg(a.ctx_len + r);
    return ctx < count ? -1 : ctx - count;
  };
  if (!find_page(p.ragged, blockIdx.x, reports, a.status, first, &w)) return;
  const int head = blockIdx.y;
  const bool values = blockIdx.z == 1;
  const Place<D> at;
  auto is_new = [&](int token) { return token >= w.lo && token < w.hi; };
  // tokens of this thread: key_token + 16 i, or 4 quad + i
  const int token0 = values ? 4 * at.quad : at.key_token, step = values ? 1 : 16;
  // everything that the page's place does not decide is loaded first
  Vec8<T> in[4];
  const T* src = values ? static_cast<const T*>(a.v) + (w.row - w.lo) * a.v_token_stride + head * a.v_head_stride + 8 * at.value_chunk
                        : static_cast<const T*>(a.k) + (w.row - w.lo) * a.k_token_stride + head * a.k_head_stride + 8 * at.key_chunk;
  const int64_t stride = values ? a.v_token_stride : a.k_token_stride;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (is_new(token0 + step * i)) in[i].load(src + (token0 + step * i) * stride);
  const int block = block_of(p.pages, w, a.status);
  if (block < 0 || !HS_CHECK(block < p.pages.num_blocks && head < p.pages.kv_heads, kChkPoolRow)) return;
  uint8_t* codes = p.pages.codes(block, head, D) + (values ? D * kHeadsPage : 0);
  float* scale_at = p.pages.scale(block, head, D) + (values ? p.pages.kv_heads : 0);
  const float old = w.lo > 0 ? *scale_at : 0.f;

  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!is_new(token0 + step * i)) continue;
    float x[8];
    in[i].values(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max_finite(top, x[e]);
  }
  __shared__ uint32_t tops[2 * D / 32];
  const uint32_t warp_top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));  // (not negative: ordered as their bits)
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = warp_top;
  __syncthreads();
  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < 2 * D / 32; ++i) all = max(all, tops[i]);
  const float scale = fmaxf(power_scale(__uint_as_float(all)), old), inv = 1.f / scale;
  const bool grown = w.lo > 0 && scale > old;
  const float shrink = old * inv;
  if (threadIdx.x == 0) *scale_at = scale;  // (all threads have read it)

  if (!values) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int token = token0 + 16 * i;
      uint2* to = reinterpret_cast<uint2*>(codes + at.key_at(token));
      float x[8];
      if (is_new(token)) {
        in[i].values(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = scaled_finite(x[e], inv);
      } else if (grown && token < w.lo) {
        const uint2 c = *to;
        float_of_codes(c.x, x);
        float_of_codes(c.y, x + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= shrink;
      } else {
        continue;
      }
      *to = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
    }
    return;
  }
  // values: four tokens of a dimension are a word; one that has other tokens too keeps those
  const bool whole = token0 >= w.lo && token0 + 4 <= w.hi, some = token0 < w.hi && token0 + 4 > w.lo, older = grown && token0 < w.lo;
  if (!some && !older) return;
  uint32_t word[8];
  if (!whole) {
#pragma unroll
    for (int e = 0; e < 8; ++e) word[e] = *reinterpret_cast<const uint32_t*>(codes + at.value_at(e));
  }
  float x[4][8];
  uint32_t fresh = 0, grow = 0;  // bytes of a word that are new, and that are rescaled
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (is_new(token0 + i)) {
      in[i].values(x[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = scaled_finite(x[i][e], inv);
      fresh |= 0xFFu << (8 * i);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
      if (older && token0 + i < w.lo) grow |= 0xFFu << (8 * i);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t c = e4m3x4(x[0][e], x[1][e], x[2][e], x[3][e]);
    if (!whole) {
      float y[4];
      float_of_codes(word[e], y);
      const uint32_t smaller = e4m3x4(y[0] * shrink, y[1] * shrink, y[2] * shrink, y[3] * shrink);
      c = (c & fresh) | (smaller & grow) | (word[e] & ~(fresh | grow));
    }
    *reinterpret_cast<uint32_t*>(codes + at.value_at(e)) = c;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(2 * D) read_heads_kernel(const HeadsReadParams p) {
  const hs_heads_read& a = p.a;
  const bool reports = blockIdx.x == 0 && blockIdx.y == 0;
  PageWork w;
  // (positions past 2^31 are past any table: the request is refused like one that starts below zero)
  auto first = [&](int r, int count) {
    const int s = a.start ? __ldg(a.start + r) : 0;
    return s > INT32_MAX - count ? -1 : s;
  };
  if (!find_page(p.ragged, blockIdx.x, reports, a.status, first, &w)) return;
  const int head = blockIdx.y;
  const Place<D> at;
  const int block = block_of(p.pages, w, a.status);
  const bool there = block >= 0 && HS_CHECK(block < p.pages.num_blocks && head < p.pages.kv_heads, kChkPoolRow);
  uint2 key[4] = {};
  uint32_t word[8] = {};
  float scale_k = 0.f, scale_v = 0.f;
  const int q0 = 4 * at.quad;
  auto asked = [&](int token) { return token >= w.lo && token < w.hi; };
  if (there) {
    const uint8_t* codes = p.pages.codes(block, head, D);
    const float* scales = p.pages.scale(block, head, D);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (asked(at.key_token + 16 * i)) key[i] = *reinterpret_cast<const uint2*>(codes + at.key_at(at.key_token + 16 * i));
    if (q0 < w.hi && q0 + 4 > w.lo) {
#pragma unroll
      for (int e = 0; e < 8; ++e) word[e] = *reinterpret_cast<const uint32_t*>(codes + D * kHeadsPage + at.value_at(e));
    }
    scale_k = scales[0], scale_v = scales[p.pages.kv_heads];
  }
  T* k = static_cast<T*>(a.k) + (w.row - w.lo) * a.k_token_stride + head * a.k_head_stride + 8 * at.key_chunk;
  T* v = static_cast<T*>(a.v) + (w.row - w.lo) * a.v_token_stride + head * a.v_head_stride + 8 * at.value_chunk;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int token = at.key_token + 16 * i;
    if (!asked(token)) continue;
    float x[8];
    float_of_codes(key[i].x, x);
    float_of_codes(key[i].y, x + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= scale_k;
    Vec8<T>::store(k + token * a.k_token_stride, x);
  }
  float x[4][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float y[4];
    float_of_codes(word[e], y);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i][e] = y[i] * scale_v;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (asked(q0 + i)) Vec8<T>::store(v + (q0 + i) * a.v_token_stride, x[i]);
}

// Pages that n tokens of R requests touch at most, by their numbers.
dim3 page_grid(int64_t n, int R, int heads) { return dim3((unsigned)(n / kHeadsPage + 2 * (int64_t)R), (unsigned)heads); }

template <typename T>
void launch_append_type(const HeadsAppendParams& p, dim3 grid, cudaStream_t s) {
  if (p.a.head_dim == 64)
    append_heads_kernel<T, 64><<<grid, 128, 0, s>>>(p);
  else
    append_heads_kernel<T, 128><<<grid, 256, 0, s>>>(p);
}
template <typename T>
void launch_read_type(const HeadsReadParams& p, dim3 grid, cudaStream_t s) {
  if (p.a.head_dim == 64)
    read_heads_kernel<T, 64><<<grid, 128, 0, s>>>(p);
  else
    read_heads_kernel<T, 128><<<grid, 256, 0, s>>>(p);
}

}  // namespace

uint32_t check_take_heads_pages() {
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

cudaError_t launch_append_heads(const HeadsAppendParams& p, cudaStream_t s) {
  dim3 grid = page_grid(p.a.n, p.a.R, p.a.kv_heads);
  grid.z = 2;
  if (p.a.dtype == HS_BF16)
    launch_append_type<__nv_bfloat16>(p, grid, s);
  else if (p.a.dtype == HS_FP16)
    launch_append_type<__half>(p, grid, s);
  else
    launch_append_type<float>(p, grid, s);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_read_heads(const HeadsReadParams& p, cudaStream_t s) {
  const dim3 grid = page_grid(p.a.n, p.a.R, p.a.kv_heads);
  if (p.a.dtype == HS_BF16)
    launch_read_type<__nv_bfloat16>(p, grid, s);
  else if (p.a.dtype == HS_FP16)
    launch_read_type<__half>(p, grid, s);
  else
    launch_read_type<float>(p, grid, s);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hs
