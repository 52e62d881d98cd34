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
// Split: a block takes one page of one head, its keys or its values (reading: both); the heads of a page follow one another, so
// that a token's row of the tensors is read (or written) at about one time.  A page is found by a number that grows faster
// than the pages can: request r's pages start at cu[r] / 64 + 2 r, since n tokens touch at most (n - 2) / 64 + 2 pages, or,
// where that is less in all, at cu[r], since they touch at most n.
// Bound: HBM for prompts (an element is 2 B in and 1 B out): 5 chunks of up to 8192 tokens, 8 heads of 128 dimensions, 46 us, 4.7 TB/s;
// reading 16 prefixes of up to 8000 tokens back, 65 us, 6.4 TB/s.  Latency for single tokens, offsets, table, scale, codes:
// 64 requests 5.3 us; reading three short prefixes 3.8 us.  Blocks of 128 threads: with 256 a page and side 50 and 7.9 us.
#include "heads.cuh"
#include "vec8.cuh"

HS_CHECK_WORD

namespace hs {
namespace {

__host__ __device__ __forceinline__ bool numbered_by_token(int64_t n, int R) { return n <= n / kHeadsPage + 2 * (int64_t)R; }

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
  const bool by_token = numbered_by_token(g.n, g.R);
  bool bad = false;
  for (int r = threadIdx.x; r < g.R; r += blockDim.x) {
    int64_t t0;
    int count;
    bad |= !g.tokens(r, &t0, &count);
    const int64_t base = by_token ? t0 : t0 / kHeadsPage + 2 * (int64_t)r;
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

// Who has what of a page, in blocks of kThreads.  Keys: the 8 dimensions of chunk key_chunk, tokens key_token + kKeyStep i.
// Values: of kTiles tiles t, the 8 dimensions of chunk value_chunk + 8 t, tokens 4 quad .. 4 quad + 3.
constexpr int kThreads = 128;
template <int D>
struct Place {
  static constexpr int kChunks = D / 8, kKeyStep = kThreads / kChunks, kKeys = kHeadsPage / kKeyStep, kTiles = D / 64;
  int key_chunk, key_token, value_chunk, quad;
  __device__ __forceinline__ Place() {
    const int t = threadIdx.x, lane = t & 31;
    key_chunk = t % kChunks;
    key_token = t / kChunks;
    value_chunk = 2 * (t >> 5) + (lane & 1);
    quad = lane >> 1;
  }
  __device__ __forceinline__ int key_at(int token) const { return (key_chunk >> 3) * 4096 + token * 64 + (key_chunk & 7) * 8; }
  __device__ __forceinline__ int value_at(int tile, int e) const { return tile * 4096 + (8 * value_chunk + e) * 64 + 4 * quad; }
};

// Blocks are numbered by head, then keys or values, then page.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_heads_kernel(const HeadsAppendParams p) {
  using At = Place<D>;
  constexpr int kVecs = At::kKeys;  // (a thread has as many of values)
  static_assert(At::kTiles * 4 == kVecs);
  const hs_heads_append& a = p.a;
  const bool reports = blockIdx.x == 0;
  const int heads = p.pages.kv_heads, head = blockIdx.x % heads;
  const bool values = blockIdx.x / heads % 2 == 1;
  PageWork w;
  auto first = [&](int r, int count) {
    const int ctx = __ldg(a.ctx_len + r);
    return ctx < count ? -1 : ctx - count;
  };
  if (!find_page(p.ragged, blockIdx.x / heads / 2, reports, a.status, first, &w)) return;
  const At at;
  auto is_new = [&](int token) { return token >= w.lo && token < w.hi; };
  auto token_of = [&](int i) { return values ? 4 * at.quad + (i & 3) : at.key_token + At::kKeyStep * i; };
  // everything that the page's place does not decide is loaded first
  Vec8<T> in[kVecs];
  if (values) {
    const T* v = static_cast<const T*>(a.v) + (w.row - w.lo + 4 * at.quad) * a.v_token_stride + head * a.v_head_stride + 8 * at.value_chunk;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (is_new(token_of(i))) in[i].load(v + (i & 3) * a.v_token_stride + 64 * (i >> 2));
  } else {
    const T* k = static_cast<const T*>(a.k) + (w.row - w.lo + at.key_token) * a.k_token_stride + head * a.k_head_stride + 8 * at.key_chunk;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (is_new(token_of(i))) in[i].load(k + At::kKeyStep * i * a.k_token_stride);
  }
  const int block = block_of(p.pages, w, a.status);
  if (block < 0 || !HS_CHECK(block < p.pages.num_blocks && head < p.pages.kv_heads, kChkPoolRow)) return;
  uint8_t* codes = p.pages.codes(block, head, D) + (values ? D * kHeadsPage : 0);
  float* scale_at = p.pages.scale(block, head, D) + (values ? p.pages.kv_heads : 0);
  const float old = w.lo > 0 ? *scale_at : 0.f;

  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (!is_new(token_of(i))) continue;
    float x[8];
    in[i].values(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max_finite(top, x[e]);
  }
  __shared__ uint32_t tops[kThreads / 32];
  const uint32_t warp_top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));  // (not negative: ordered as their bits)
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = warp_top;
  __syncthreads();
  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) all = max(all, tops[i]);
  const float scale = fmaxf(power_scale(__uint_as_float(all)), old), inv = 1.f / scale;
  const bool grown = w.lo > 0 && scale > old;
  const float shrink = old * inv;
  if (threadIdx.x == 0) *scale_at = scale;  // (all threads have read it)

  if (!values) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int token = token_of(i);
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
  const int token0 = 4 * at.quad;
  const bool whole = token0 >= w.lo && token0 + 4 <= w.hi, some = token0 < w.hi && token0 + 4 > w.lo, older = grown && token0 < w.lo;
  if (!some && !older) return;
  uint32_t fresh = 0, grow = 0;  // bytes of a word that are new, and that are rescaled
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (is_new(token0 + i))
      fresh |= 0xFFu << (8 * i);
    else if (older && token0 + i < w.lo)
      grow |= 0xFFu << (8 * i);
  }
#pragma unroll
  for (int t = 0; t < At::kTiles; ++t) {
    float x[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (is_new(token0 + i)) {
        in[4 * t + i].values(x[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = scaled_finite(x[i][e], inv);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t* to = reinterpret_cast<uint32_t*>(codes + at.value_at(t, e));
      uint32_t c = e4m3x4(x[0][e], x[1][e], x[2][e], x[3][e]);
      if (!whole) {
        const uint32_t word = *to;
        float y[4];
        float_of_codes(word, y);
        const uint32_t smaller = e4m3x4(y[0] * shrink, y[1] * shrink, y[2] * shrink, y[3] * shrink);
        c = (c & fresh) | (smaller & grow) | (word & ~(fresh | grow));
      }
      *to = c;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_heads_kernel(const HeadsReadParams p) {
  using At = Place<D>;
  const hs_heads_read& a = p.a;
  const bool reports = blockIdx.x == 0;
  const int heads = p.pages.kv_heads, head = blockIdx.x % heads;
  PageWork w;
  // (positions past 2^31 are past any table: the request is refused like one that starts below zero)
  auto first = [&](int r, int count) {
    const int s = a.start ? __ldg(a.start + r) : 0;
    return s > INT32_MAX - count ? -1 : s;
  };
  if (!find_page(p.ragged, blockIdx.x / heads, reports, a.status, first, &w)) return;
  const At at;
  const int block = block_of(p.pages, w, a.status);
  const bool there = block >= 0 && HS_CHECK(block < p.pages.num_blocks && head < p.pages.kv_heads, kChkPoolRow);
  uint2 key[At::kKeys] = {};
  uint32_t word[At::kTiles][8] = {};
  float scale_k = 0.f, scale_v = 0.f;
  const int token0 = 4 * at.quad;
  auto asked = [&](int token) { return token >= w.lo && token < w.hi; };
  if (there) {
    const uint8_t* codes = p.pages.codes(block, head, D);
    const float* scales = p.pages.scale(block, head, D);
#pragma unroll
    for (int i = 0; i < At::kKeys; ++i) {
      const int token = at.key_token + At::kKeyStep * i;
      if (asked(token)) key[i] = *reinterpret_cast<const uint2*>(codes + at.key_at(token));
    }
    if (token0 < w.hi && token0 + 4 > w.lo) {
#pragma unroll
      for (int t = 0; t < At::kTiles; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) word[t][e] = *reinterpret_cast<const uint32_t*>(codes + D * kHeadsPage + at.value_at(t, e));
    }
    scale_k = scales[0], scale_v = scales[p.pages.kv_heads];
  }
  T* k = static_cast<T*>(a.k) + (w.row - w.lo) * a.k_token_stride + head * a.k_head_stride + 8 * at.key_chunk;
  T* v = static_cast<T*>(a.v) + (w.row - w.lo) * a.v_token_stride + head * a.v_head_stride + 8 * at.value_chunk;
#pragma unroll
  for (int i = 0; i < At::kKeys; ++i) {
    const int token = at.key_token + At::kKeyStep * i;
    if (!asked(token)) continue;
    float x[8];
    float_of_codes(key[i].x, x);
    float_of_codes(key[i].y, x + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= scale_k;
    Vec8<T>::store(k + token * a.k_token_stride, x);
  }
#pragma unroll
  for (int t = 0; t < At::kTiles; ++t) {
    float x[4][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float y[4];
      float_of_codes(word[t][e], y);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i][e] = y[i] * scale_v;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (asked(token0 + i)) Vec8<T>::store(v + (token0 + i) * a.v_token_stride + 64 * t, x[i]);
  }
}

// Blocks for the pages that n tokens of R requests touch at most, by their numbers, `each` for a page; 0: too many for a grid.
unsigned blocks(int64_t n, int R, int each) {
  const int64_t pages = numbered_by_token(n, R) ? n : n / kHeadsPage + 2 * (int64_t)R;
  return pages <= INT32_MAX / each ? (unsigned)(pages * each) : 0;
}

template <typename T>
void launch_append_type(const HeadsAppendParams& p, unsigned grid, cudaStream_t s) {
  if (p.a.head_dim == 64)
    append_heads_kernel<T, 64><<<grid, kThreads, 0, s>>>(p);
  else
    append_heads_kernel<T, 128><<<grid, kThreads, 0, s>>>(p);
}
template <typename T>
void launch_read_type(const HeadsReadParams& p, unsigned grid, cudaStream_t s) {
  if (p.a.head_dim == 64)
    read_heads_kernel<T, 64><<<grid, kThreads, 0, s>>>(p);
  else
    read_heads_kernel<T, 128><<<grid, kThreads, 0, s>>>(p);
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
  if (p.a.R == 0) return cudaSuccess;  // no request has any of the tokens
  const unsigned grid = blocks(p.a.n, p.a.R, 2 * p.a.kv_heads);
  if (grid == 0) return cudaErrorInvalidConfiguration;
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
  if (p.a.R == 0) return cudaSuccess;  // no request has any of the tokens
  const unsigned grid = blocks(p.a.n, p.a.R, p.a.kv_heads);
  if (grid == 0) return cudaErrorInvalidConfiguration;
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
