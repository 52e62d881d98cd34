// Attention over pages of grouped heads in 8 bits, for many query columns a head of keys: prompts and prompt chunks, on the
// tensor cores.
//
// Mathematics.  As in heads_attend.cu: codes are multiplied in fp16, a page's value scale is part of its weights, the reference R
// of the weights follows the largest product of weight and scale, and the sum of the weights has a reference m of its own.  Here a
// query row is a thread's, and so are R, m and the sum.
//
// Layout.  A work item is (request, head of keys and values, 256 columns): two tiles of 128 columns (query token x query head of
// the group, token by token) over the same key tiles of 128 tokens (two pages), so that a page widened serves 256 rows.  The
// key tiles of all items are numbered (with something added for each item), and every CTA takes an equal run of them, whatever the
// contexts' lengths and the causal mask leave; items that are cut leave partial results in the workspace, which prompt_join_kernel
// joins in a fixed order.
// 16 warps, one CTA per SM (the warpgroups trade registers):
//   warps 0-3, 4-7   softmax and results of query tile 0 and 1, a row a thread;
//   warps 8, 9       issue the products of query tile 0 and 1;
//   warp 10          copies codes into staging (a key tile's keys or values at a time) and reads the pages' scales;
//   warp 11          finds the run's items and hands them to the others, two at a time;
//   warps 12-15      widen the codes to fp16, into the operands' places, and bring the queries there.
// Shared memory: queries, two key tiles and two value tiles in fp16 (64 KB each for 128 dimensions), and the codes of the next key
// tile (of the next two for 64 dimensions).  Tensor memory: S and O of both query tiles, and P, in fp16, the left operand of the
// second product: in S's place for 128 dimensions, in one of its own for 64.
// A value's NaN must not reach rows that do not see its token, and a weight of zero does not keep it from them: where a key tile
// is not seen whole by all rows, the widening warps put zero for it and note, by dimension, the first such token; rows that see
// it get their NaN at the end.
//
// What bounds it.  The products, 512 D operations a row and key tile, would take 291 us for 8192 tokens with 8 x 4 heads of 128
// dimensions at 1887 TFLOP/s, the reads nothing to speak of; measured 481 us, 1144 TFLOP/s (1290 for 4 chunks of 512 over 16000).
// A key tile takes 3500 cycles of the SM or less: 2160 of products, 3100 of shared memory's bandwidth (both operands of the scores are
// read for each page, the values for each query tile, the widened codes written once), 1024 of exponentials.  An item costs about
// 7 us beside its key tiles: queries brought and converted, masked tiles, results, instructions fetched anew (so that short code
// counts there: 16 values unrolled instead of whole rows took 14 us of 522).  For 64 dimensions the exponentials weigh twice as
// much and the chain of a key tile is longer than its products: 355 us for the same prompt, 775 TFLOP/s.  The smallest prompts
// (100 tokens, 2 x 4 heads) take 18 us.
#include "heads_device.cuh"

HS_CHECK_WORD

namespace hs {
namespace {

using namespace heads;

constexpr int kQRows = 128, kKeys = 128, kBlock = 2 * kQRows;
constexpr int kThreads = 16 * 32, kMmaWarp = 8, kLoadWarp = 10, kWalkWarp = 11, kWidenWarp = 12;
constexpr int kTakers = 15;  // warps that the items are handed to
constexpr int kRegsLaunch = 128;
// Registers after the trade, of the softmax warps and of the others.  12000 tokens, 4 x 3 heads of 64 dimensions: 317 us with 208 and
// 48, 288 us with 200 and 56, 284 us with 192 and 64.  For 128 dimensions, a page at a time, all from 136 and 120 to 168 and 88 do
// (8192 tokens, 8 x 4 heads: 483, 480 and 482 us with 136, 152 and 168; 486 us with 184).
template <int D>
struct Regs {
  static constexpr int kSoftmax = D == 64 ? 192 : 152, kOther = D == 64 ? 64 : 104;
  static_assert(2 * kSoftmax + 2 * kOther <= 4 * kRegsLaunch, "more registers than the launch has");
};
constexpr int kScales = 8;  // key tiles whose scales are kept
// What an item costs beside its key tiles, in these (12000 tokens, 4 x 3 heads of 64: 293 us with 2, 284 us with 3, 278 us with 4; 8192
// tokens, 8 x 4 heads of 128: 514, 480 and 453 us; 3 is of the time when 128 dimensions went by key tiles), and the least of a run: fewer would be mostly set-up and joining (64 tokens
// behind 16000, 1 x 2 heads: 31 us with 2, 25 us with 4 and 6), and with more, small calls leave CTAs without any (100 tokens, 2 x 4
// heads: 17.5 us with 4, 25 us with 6).
constexpr int kItemCost = 3, kMinRun = 4;
// (four: of query tile 0 and 1, for a key tile's first part, then for its second)
enum Bar { kStFull = 0, kStEmpty = kStFull + 4, kKFull = kStEmpty + 4, kKEmpty = kKFull + 2, kVFull = kKEmpty + 2,
           kVEmpty = kVFull + 2, kQFull = kVEmpty + 2, kQEmpty = kQFull + 2, kSFull = kQEmpty + 2, kPReady = kSFull + 4,
           kODone = kPReady + 4, kSFree = kODone + 4, kItem = kSFree + 4, kItemDone = kItem + 2, kDrain = kItemDone + 2,
           kBars = kDrain + 2 };

// Workspace: header, a record a CTA, statistics [CTA][2][256][4], results [CTA][2][D / 4][256][4].
__host__ __device__ constexpr size_t ws_stats_offset(int ctas) { return sizeof(RunHeader) + (size_t)ctas * sizeof(RunRecord); }
__host__ __device__ constexpr size_t ws_parts_offset(int ctas) { return ws_stats_offset(ctas) + (size_t)ctas * 2 * kBlock * 16; }
__host__ __device__ constexpr size_t ws_bytes(int ctas, int dim) { return ws_parts_offset(ctas) + (size_t)ctas * 2 * kBlock * dim * 4; }

// What a call has of one request: `blocks` is 0 where it has no queries, or at most `limit` columns.
struct Request {
  int64_t t0;
  int n, ctx, keys, blocks;
  __device__ __forceinline__ void load(const HeadsAttendParams& p, int r, int limit) {
    p.ragged.tokens(r, &t0, &n);
    ctx = __ldg(p.a.ctx_len + r);
    keys = max(0, min(ctx, p.a.max_pages * kHeadsPage));
    const int cols = n * p.group;
    blocks = cols > limit ? (cols - 1) / kBlock + 1 : 0;  // (cols may be all of 31 bits)
  }
  // tokens that column c sees
  __device__ __forceinline__ int sees(const HeadsAttendParams& p, int c) const {
    return p.a.causal ? max(0, min(keys, ctx - n + 1 + c / p.group)) : keys;
  }
  // key tiles of block b
  __device__ __forceinline__ int tiles(const HeadsAttendParams& p, int b) const {
    return max(1, (sees(p, min(n * p.group - 1, b * kBlock + (kBlock - 1))) + kKeys - 1) / kKeys);
  }
};
// Units of a request's blocks (of one head), by the whole warp.
__device__ __forceinline__ int64_t request_units(const HeadsAttendParams& p, const Request& q) {
  int64_t s = 0;
  for (int b = threadIdx.x & 31; b < q.blocks; b += 32) s += kItemCost + q.tiles(p, b);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  return s;
}

// Where a run begins: `in` units into an item.  An item is kItemCost units and one for each of its key tiles.
struct Start {
  int r, head, block, in;
  int64_t at, left;  // in units
};

// One item, or this run's part of it: key tiles [k0, k1) of `tiles`.  In shared memory, two of them; everything else that belongs
// to an item is kept twice too.
struct Item {
  int64_t t0;          // the request's first query token
  int64_t begin;       // the item's first key tile among the call's units
  int32_t request, head, col0, rows;  // the item's first column of (request, head), and how many
  int32_t k0, k1, tiles;
  int32_t end[2];      // the query tile's part of the run ends here (at k0: it has none)
  int32_t keys, shift, past;  // column c sees the first c / group + shift tokens, at most keys; past: of more than the table has room for
  int32_t part;        // which of the run's two places for partial results is its
  int32_t none;        // no item: the run has ended
};
static_assert(sizeof(Item) % 8 == 0, "alignment of what follows");

template <int D>
struct Smem {
  static constexpr int kUnits = D / 64, kUnit = 128 * 128;  // a unit: 128 rows of 64 fp16
  // Of a key tile, the pages that are taken together from scores to weights to results, and the number of such parts.  For 128
  // dimensions a page at a time: its products run while the other page's weights are made (4 chunks of 512 behind 16000 tokens, 4 x 8
  // heads: 313 us; 357 us by key tiles).  For 64 both: the products are short, and hand-overs cost more (227 us; 291 us by pages).
  static constexpr int kPages = D == 64 ? 2 : 1, kParts = 2 / kPages;
  // Tensor memory, for each query tile: S, 64 columns a page; D columns of O; and P, 32 columns a page: where there is room, of its
  // own, so that the next scores are made while the weights are; else in the place of the page's S.
  static constexpr bool kApart = D == 64;
  static constexpr uint32_t kTo = kApart ? 384 : 256, kTp = kApart ? 256 : 0, kToStep = D, kTpStep = kApart ? 64 : 128, kTpPage = kApart ? 32 : 64;
  static constexpr int kStage = D * kHeadsPage;
  static constexpr int kQ = 0, kK = kQ + 2 * kUnits * kUnit, kV = kK + 2 * kUnits * kUnit, kVPage = D * 128;
  // Staged key tiles: of each, the keys of its two pages, then their values.  Barriers: keys and values of the even ones, of the
  // odd ones.
  static constexpr int kDepth = D == 64 ? 2 : 1, kTileStage = 4 * kStage;
  static constexpr int kStages = kV + 4 * kVPage, kMisc = kStages + kDepth * kTileStage;
  // query scales (exponent fields, a byte each) [2][256], first NaNs (ints) [2][D], floats: page scales [kScales][8]
  static constexpr int kNan = kMisc + 2 * kBlock, kPage = kNan + 2 * D * 4, kFlag = kPage + kScales * 32, kItems = kFlag + 16, kBar = kItems + 2 * sizeof(Item);
  static constexpr int kBytes = kBar + kBars * 8;
  static_assert(kBytes <= 232448, "shared memory");
};

// tokens that column c of the item's request and head sees
__device__ __forceinline__ int item_sees(const HeadsAttendParams& p, const Item& it, int c) {
  return p.a.causal ? max(0, min(it.keys, c / p.group + it.shift)) : it.keys;
}

// Hands the run's items to the others (one warp).
template <int D>
__device__ __forceinline__ void walk_items(const HeadsAttendParams& p, Start at, int limit, uint8_t* raw, uint32_t bars) {
  using L = Smem<D>;
  Item* items = reinterpret_cast<Item*>(raw + L::kItems);
  const int lane = threadIdx.x & 31;
  tc::Waiter w;
  const int64_t first = at.at;
  Request q{};
  if (at.left > 0) q.load(p, at.r, limit);
#pragma unroll 1
  for (uint32_t k = 0;; ++k) {
    Item it{};
    it.none = 1;
    while (at.left > 0 && it.none) {
      if (at.block == q.blocks) {
        at.block = 0;
        if (++at.head == p.pages.kv_heads) {
          at.head = 0;
          do q.load(p, ++at.r, limit);
          while (q.blocks == 0 && at.r + 1 < p.a.R);
        }
      }
      it.tiles = q.tiles(p, at.block);
      const int units = (int)min((int64_t)(kItemCost + it.tiles - at.in), at.left);
      it.begin = at.at - at.in + kItemCost;
      it.part = it.begin > first;
      it.k0 = max(0, at.in - kItemCost);
      it.k1 = at.in + units - kItemCost;
      if (it.k1 > it.k0) {  // (a run that ends before an item's first key tile leaves it to the next)
        it.none = 0;
        it.t0 = q.t0, it.request = at.r, it.head = at.head, it.col0 = at.block * kBlock;
        it.rows = min(kBlock, q.n * p.group - it.col0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int last = min(it.rows, (t + 1) * kQRows) - 1;
          const int mine = last < t * kQRows ? 0 : (q.sees(p, it.col0 + last) + kKeys - 1) / kKeys;
          it.end[t] = max(it.k0, min(it.k1, mine));
        }
        it.keys = q.keys, it.shift = q.ctx - q.n + 1, it.past = q.ctx > q.keys;
      }
      at.left -= units;
      at.at += units;
      at.in = 0;
      ++at.block;
    }
    if (k >= 2) await(w, bars + 8 * (kItemDone + (k & 1)), (k / 2 - 1) & 1);
    if (w.dead) break;
    for (int i = lane; i < D; i += 32) reinterpret_cast<int*>(raw + L::kNan)[(k & 1) * D + i] = INT_MAX;
    if (lane == 0) reinterpret_cast<int*>(raw + L::kFlag)[k & 1] = 0;
    __syncwarp();
    if (lane == 0) {
      items[k & 1] = it;
      tc::mbar_arrive(bars + 8 * (kItem + (k & 1)));
    }
    __syncwarp();
    if (it.none) break;
  }
  if (w.dead) report(p.a.status, HS_ERR_TIMEOUT);
}
// The next item, for each of the others; null at the run's end, or after a wait that gave up.
__device__ __forceinline__ const Item* take_item(const Item* items, uint32_t k, uint32_t bars, tc::Waiter& w) {
  await(w, bars + 8 * (kItem + (k & 1)), k / 2 & 1);
  const Item* it = items + (k & 1);
  return w.dead || it->none ? nullptr : it;
}
__device__ __forceinline__ void done_with_item(uint32_t k, uint32_t bars) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bars + 8 * (kItemDone + (k & 1)));
}

// ---- copies (one warp) ----
template <int D>
__device__ __forceinline__ void load_items(const HeadsAttendParams& p, const Item* items, uint32_t smem) {
  using L = Smem<D>;
  const uint32_t bars = smem + L::kBar;
  const int lane = threadIdx.x & 31;
  tc::Waiter w;
  uint32_t tile = 0, part = 0;  // key tiles so far; of the next one, what has been announced (a bit for keys, one for values)
#pragma unroll 1
  for (uint32_t k = 0;; ++k) {
    const Item* item = take_item(items, k, bars, w);
    if (!item) break;
    const int request = item->request, head = item->head, keys = item->keys, k1 = item->k1;
    const bool past = item->past;
    int cached = -1, cached_at = -1;  // table entries: a page a lane
#pragma unroll 1
    for (int j = item->k0; j < k1; ++j, ++tile) {
      const int page0 = 2 * j;
      if (cached_at != (page0 & ~31)) {
        cached_at = page0 & ~31;
        const int page = cached_at + lane;
        cached = -1;
        if (page * kHeadsPage < keys && HS_CHECK(request < p.a.R && page < p.a.max_pages, kChkTablePage))
          cached = __ldg(p.pages.table + (int64_t)request * p.a.max_pages + page);
      }
      int block[2];
      bool there[2];
      bool bad = past;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        block[i] = __shfl_sync(0xFFFFFFFFu, cached, (page0 + i) & 31);
        there[i] = block[i] >= 0 && block[i] < p.pages.num_blocks;
        bad |= (page0 + i) * kHeadsPage < keys && !there[i];
      }
      if (bad && lane == 0) report(p.a.status, HS_ERR_TABLE_RANGE);
      // lanes 0..3: the scales of keys and values of both pages
      const int b = lane & 1 ? block[1] : block[0];
      const bool is = lane & 1 ? there[1] : there[0];
      float scale = 1.f;
      if (lane < 4 && is) scale = *p.pages.scale(b, head + (lane >> 1) * p.pages.kv_heads, D);
      if (lane >= 2 && lane < 4) scale = log2f(scale);
      const uint32_t scales = smem + L::kPage + tile % kScales * 32;
      __syncwarp();
      const uint32_t slot = tile % L::kDepth, use = tile / L::kDepth;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const uint32_t bar = bars + 8 * (kStFull + 2 * slot + side);
        if (use > 0) {
          await(w, bars + 8 * (kStEmpty + 2 * slot + side), (use - 1) & 1);
          // (complete by then, unless another warp's wait gave up: nothing is announced before the copy before has landed)
          await(w, bar, (use - 1) & 1);
        }
        if (w.dead) break;
        if (side == 0) {
          if (lane < 4) sts_u(scales + 4 * lane, __float_as_uint(scale));
          if (lane < 2) sts_u(scales + 16 + 4 * lane, is);
          __syncwarp();
        }
        if (lane == 0) {
          if (there[0] || there[1]) {
            tc::mbar_expect(bar, (there[0] + there[1]) * L::kStage);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (there[i])
                bulk_copy(smem + L::kStages + slot * L::kTileStage + (2 * side + i) * L::kStage,
                          p.pages.codes(block[i], head, D) + side * L::kStage, L::kStage, bar);
          } else {
            tc::mbar_arrive(bar);
          }
        }
        part |= 1u << side;
        __syncwarp();
      }
      if (w.dead) break;
      part = 0;
    }
    done_with_item(k, bars);
  }
  // no copy is in flight when the CTA ends
  tc::Drain drain;
#pragma unroll 1
  for (int i = 0; i < 2 * L::kDepth; ++i) {
    const uint32_t n = (tile + (part >> (i & 1) & 1) + L::kDepth - 1 - (i >> 1)) / L::kDepth;
    if (n > 0) drain.wait(bars + 8 * (kStFull + i), (n - 1) & 1);
  }
  if (w.dead) report(p.a.status, HS_ERR_TIMEOUT);
}

// ---- operands (four warps) ----

// Queries of query tile t.  First all of them are copied to their places as they are, asynchronously, a row by D / 8 lanes; then
// each thread turns a row into fp16 in place.
template <int D>
__device__ __forceinline__ void copy_queries(const HeadsAttendParams& p, const Item* it, int t, uint32_t smem) {
  using L = Smem<D>;
  constexpr int kLanes = D / 8, kRows = 128 / kLanes;
  const int thread = threadIdx.x & 127, piece = thread % kLanes;
  const int rows = it->rows - t * kQRows;
  int row = thread / kLanes, c = it->col0 + t * kQRows + row, token = c / p.group;
  // from row to row the column moves on by kRows: `tokens` of them and `heads` of the group, or one token more
  const int tokens = kRows / p.group, heads = kRows - tokens * p.group;
  const int64_t step = tokens * p.a.q_token_stride + heads * p.a.q_head_stride, wrap = p.a.q_token_stride - p.group * p.a.q_head_stride;
  int in_group = c - token * p.group;
  const uint16_t* from = static_cast<const uint16_t*>(p.a.q) + (it->t0 + token) * p.a.q_token_stride +
                         (it->head * p.group + in_group) * p.a.q_head_stride + 8 * piece;
  uint32_t to = smem + L::kQ + (t * L::kUnits + (piece >> 3)) * L::kUnit + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
#pragma unroll 2
  for (; row < kQRows; row += kRows, to += kRows * 128) {  // (kRows is a multiple of 8: the swizzle stays)
    const bool there = row < rows;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(there ? from : static_cast<const uint16_t*>(p.a.q)),
                 "r"(there ? 16 : 0)
                 : "memory");
    from += step;
    in_group += heads;
    if (in_group >= p.group) in_group -= p.group, from += wrap;
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Larger magnitudes of two values of 16 bits each, in either type (NaN is passed over).
__device__ __forceinline__ uint32_t max_magnitudes(bool f16, uint32_t a, uint32_t b) {
  b &= 0x7FFF7FFFu;
  if (f16)
    asm("max.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  else
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}
// A thread's row.  The largest magnitude is found on the way; only where it wants the row divided (rare) is it read again.
template <int D>
__device__ __forceinline__ void convert_queries(const HeadsAttendParams& p, const Item* it, int t, uint32_t smem, uint32_t qs, float sign) {
  using L = Smem<D>;
  const int row = threadIdx.x & 127;
  const bool f16 = p.a.dtype == HS_FP16;
  const uint32_t at = smem + L::kQ + t * L::kUnits * L::kUnit + row * 128, flip = sign < 0.f ? 0x80008000u : 0u;
  auto place = [&](int piece) { return at + (piece >> 3) * L::kUnit + (((piece & 7) ^ (row & 7)) << 4); };
  uint32_t most[4] = {0, 0, 0, 0};
#pragma unroll 4
  for (int i = 0; i < D / 8; ++i) {
    const uint4 v = lds16(place(i));
    uint32_t w[4] = {v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      most[x] = max_magnitudes(f16, most[x], w[x]);
      if (!f16) w[x] = pack_half(__uint_as_float(w[x] << 16), __uint_as_float(w[x] & 0xFFFF0000u));
    }
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(place(i)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
  }
  most[0] = max_magnitudes(f16, max_magnitudes(f16, most[0], most[1]), max_magnitudes(f16, most[2], most[3]));
  float2 two;
  if (f16)
    two = __half22float2(*reinterpret_cast<const __half2*>(&most[0]));
  else
    two = make_float2(__uint_as_float(most[0] << 16), __uint_as_float(most[0] & 0xFFFF0000u));
  const int e = query_field(fmaxf(two.x, two.y));
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(qs + t * kQRows + row), "r"(e) : "memory");
  if (e == 127 || t * kQRows + row >= it->rows) return;
  const float f = sign * power_of_field(254 - e);
  const int c = it->col0 + t * kQRows + row, token = c / p.group;
  const uint16_t* from = static_cast<const uint16_t*>(p.a.q) + (it->t0 + token) * p.a.q_token_stride +
                         (it->head * p.group + c - token * p.group) * p.a.q_head_stride;
#pragma unroll 1
  for (int i = 0; i < D / 8; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(from) + i);
    float x[8];
    if (f16)
      Vec8<__half>{v}.values(x);
    else
      Vec8<__nv_bfloat16>{v}.values(x);
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(place(i)), "r"(pack_half(x[0] * f, x[1] * f)),
                 "r"(pack_half(x[2] * f, x[3] * f)), "r"(pack_half(x[4] * f, x[5] * f)), "r"(pack_half(x[6] * f, x[7] * f))
                 : "memory");
  }
}

// A staged page's keys or values to fp16.  Row r of block db (a token's 64 dimensions, or a dimension's 64 tokens) goes to row r
// of `to` + db * step.
template <int D>
__device__ __forceinline__ void widen(uint32_t from, uint32_t to, int step) {
  const int thread = threadIdx.x & 127, row = thread >> 2, piece = thread & 3;  // (and row + 32)
  const uint32_t at = row * 128 + (((2 * piece) ^ (row & 7)) << 4);               // the odd piece beside it: its bit 4 turned
  uint4 v[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) v[i] = lds16(from + i * 2048 + thread * 16);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t words[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint2 x = half_of_codes(words[2 * h]), y = half_of_codes(words[2 * h + 1]);
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + (h ? at ^ 16 : at) + (i >> 1) * step + (i & 1) * 4096), "r"(x.x),
                   "r"(x.y), "r"(y.x), "r"(y.y)
                   : "memory");
    }
  }
}
// Before that, where it is wanted, by the same threads for the same codes.  zero: the page is not there.  Else NaN codes of values
// become zero and are noted, see the head of this file.
template <int D>
__device__ __forceinline__ void clean_staged(uint32_t from, bool zero, int key0, int* nan_first, int* flag) {
  const int thread = threadIdx.x & 127;
#pragma unroll 1
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t at = from + i * 2048 + thread * 16;
    uint4 v = lds16(at);
    if (zero) {
      v = make_uint4(0, 0, 0, 0);
    } else {
      if (!(nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w))) continue;
      auto word = [&](uint32_t& w, int x) {
        const uint32_t is = nan_codes(w);
        if (!is) return;
        atomicMin(nan_first + i * 32 + (thread >> 2), key0 + 16 * (thread & 3) + 4 * x + ((__ffs(is) - 1) >> 3));
        w &= ~((is >> 7) * 0xFFu);
      };
      word(v.x, 0), word(v.y, 1), word(v.z, 2), word(v.w, 3);
      *flag = 1;
    }
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
  }
  tc::fence_async_smem();  // (the next copy goes to the same place)
}
// True when x is true for any of the widening warps' threads.
__device__ __forceinline__ bool any_of_wideners(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

template <int D>
__device__ __forceinline__ void widen_items(const HeadsAttendParams& p, const Item* items, uint32_t smem, uint8_t* raw) {
  using L = Smem<D>;
  const uint32_t bars = smem + L::kBar;
  const int lane = threadIdx.x & 31;
  const float sign = scale_sign(p.scale_log2);
  tc::Waiter w;
  uint32_t tile = 0, brought = 0, odd = 0;  // query tiles that have been brought, and an odd number of times
  auto arrive = [&](int bar) {
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bars + 8 * bar);
  };
#pragma unroll 1
  for (uint32_t k = 0;; ++k) {
    const Item* it = take_item(items, k, bars, w);
    if (any_of_wideners(w.dead)) {  // (all of them go on, or none: they have barriers of their own within an item)
      w.dead = true;
      break;
    }
    if (!it) break;
    int* nan_first = reinterpret_cast<int*>(raw + L::kNan) + (k & 1) * D;
    int* flag = reinterpret_cast<int*>(raw + L::kFlag) + (k & 1);
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      if (it->end[t] <= it->k0) continue;
      if (brought >> t & 1) await(w, bars + 8 * (kQEmpty + t), (odd >> t & 1) ^ 1);
      brought |= 1u << t;
      odd ^= 1u << t;
      copy_queries<D>(p, it, t, smem);
    }
    const int all_see = item_sees(p, *it, it->col0), k0 = it->k0, k1 = it->k1;
#pragma unroll 1
    for (int j = k0; j < k1; ++j, ++tile) {
      const uint32_t buf = tile & 1, scales = smem + L::kPage + tile % kScales * 32, slot = tile % L::kDepth;
      const bool clean = (j + 1) * kKeys > all_see;
#pragma unroll 1
      for (int side = 0; side < 2; ++side) {
        if (tile >= 2) await(w, bars + 8 * ((side ? kVEmpty : kKEmpty) + buf), (tile / 2 - 1) & 1);
        await(w, bars + 8 * (kStFull + 2 * slot + side), tile / L::kDepth & 1);
        const uint32_t from = smem + L::kStages + slot * L::kTileStage + 2 * side * L::kStage;
#pragma unroll 1
        for (int page = 0; page < 2; ++page) {
          const bool zero = lds_u(scales + 16 + 4 * page) == 0;
          if (zero || (clean && side)) clean_staged<D>(from + page * L::kStage, zero, j * kKeys + page * kHeadsPage, nan_first, flag);
        }
        // a page's keys: rows page * 64 .. of every 64 dimensions' unit; its values: a part of D rows of its own
        const uint32_t to = smem + (side ? L::kV + 2 * buf * L::kVPage : L::kK + buf * L::kUnits * L::kUnit);
        const int page_step = side ? L::kVPage : 8192, step = side ? 64 * 128 : L::kUnit;
        widen<D>(from, to, step);
        widen<D>(from + L::kStage, to + page_step, step);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bars + 8 * (kStEmpty + 2 * slot + side));
        arrive((side ? kVFull : kKFull) + buf);
        if (side == 0 && j == k0) {  // (the first keys were widened while the queries were on their way)
          asm volatile("cp.async.wait_group 0;\n\tbar.sync 1, 128;" ::: "memory");
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            if (it->end[t] <= k0) continue;
            convert_queries<D>(p, it, t, smem, smem + L::kMisc + (k & 1) * kBlock, sign);
            arrive(kQFull + t);
          }
        }
      }
    }
    done_with_item(k, bars);
  }
  if (w.dead) report(p.a.status, HS_ERR_TIMEOUT);
}

// ---- products (one warp a query tile) ----
// Both warps wait for every key tile's keys and values and release them, whether their query tile needs them or not.
template <int D>
__device__ __forceinline__ void issue_items(const HeadsAttendParams& p, const Item* list, int t, uint32_t smem, uint32_t tmem) {
  using L = Smem<D>;
  constexpr uint32_t kIdS = tc::idesc(true, 128, kHeadsPage * L::kPages, false, false);
  constexpr uint32_t kIdO = tc::idesc(true, 128, D, false, false);
  const uint32_t bars = smem + L::kBar;
  tc::Waiter w;
  const bool leader = tc::elect();
  const uint64_t dq = tc::desc(smem + L::kQ + t * L::kUnits * L::kUnit, 16, 1024, tc::kSwizzle128);
  const uint64_t dk = tc::desc(smem + L::kK, 16, 1024, tc::kSwizzle128);
  const uint64_t dv = tc::desc(smem + L::kV, 16, 1024, tc::kSwizzle128);
  auto wait = [&](int bar, uint32_t parity) {
    w.wait(bars + 8 * bar, parity);
    __syncwarp();
    tc::fence_after();
  };
  uint32_t base = 0, items = 0, phase = 0;  // key tiles before this item; items with work, key tiles done, of the query tile
#pragma unroll 1
  for (uint32_t number = 0;; ++number) {
    const Item* it = take_item(list, number, bars, w);
    if (!it) break;
    const int k0 = it->k0, k1 = it->k1, end = it->end[t];
    auto keys_there = [&](int j) {
      const uint32_t n = base + j - k0;
      wait(kKFull + (n & 1), n / 2 & 1);
    };
    auto scores = [&](int j, int part) {
      const uint32_t buf = (base + j - k0) & 1;
#pragma unroll
      for (int i = 0; i < L::kUnits; ++i) {
        const uint64_t da = dq + (uint32_t)(i * L::kUnit >> 4), db = dk + (uint32_t)(((buf * L::kUnits + i) * L::kUnit + part * 8192) >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc::mma_ss(tmem + t * 128 + part * 64, da + (k * 32 >> 4), db + (k * 32 >> 4), kIdS, i > 0 || k > 0, leader);
      }
      tc::commit(bars + 8 * (kSFull + 2 * part + t), leader);
      if (part == L::kParts - 1) {
        tc::commit(bars + 8 * (kKEmpty + buf), leader);
        if (j + 1 == end) tc::commit(bars + 8 * (kQEmpty + t), leader);
      }
    };
    if (end > k0) {
      keys_there(k0);
      wait(kQFull + t, items & 1);
      ++items;
#pragma unroll 1
      for (int part = 0; part < L::kParts; ++part) {
        if (phase > 0) wait((L::kApart ? kSFree : kODone) + 2 * part + t, (phase - 1) & 1);  // the item before: S's place is free
        scores(k0, part);
      }
    }
#pragma unroll 1
    for (int j = k0; j < end; ++j, ++phase) {
      const uint32_t n = base + j - k0, buf = n & 1;
#pragma unroll 1
      for (int part = 0; part < L::kParts; ++part) {
        if (part == 0 && j + 1 < end) keys_there(j + 1);
        if (L::kApart && j + 1 < end) {
          wait(kSFree + 2 * part + t, phase & 1);
          scores(j + 1, part);
        }
        if (part == 0) wait(kVFull + buf, n / 2 & 1);
        wait(kPReady + 2 * part + t, phase & 1);
#pragma unroll
        for (int i = 0; i < L::kPages; ++i) {
          const int page = part + i;
          const uint64_t db = dv + (uint32_t)((2 * buf + page) * L::kVPage >> 4);
          // P: 16 tokens are 8 columns
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_ts(tmem + L::kTo + t * L::kToStep, tmem + L::kTp + t * L::kTpStep + page * L::kTpPage + k * 8, db + (k * 32 >> 4), kIdO,
                       j > k0 || page > 0 || k > 0, leader);
        }
        tc::commit(bars + 8 * (kODone + 2 * part + t), leader);
        if (part == L::kParts - 1) tc::commit(bars + 8 * (kVEmpty + buf), leader);
        if (!L::kApart && j + 1 < end) {
          wait(kODone + 2 * part + t, phase & 1);  // P, in S's place, has been read
          scores(j + 1, part);
        }
      }
    }
#pragma unroll 1
    for (int j = end; j < k1; ++j) {  // what only the other query tile reads
      const uint32_t n = base + j - k0, buf = n & 1;
      wait(kKFull + buf, n / 2 & 1);
      tc::commit(bars + 8 * (kKEmpty + buf), leader);
      wait(kVFull + buf, n / 2 & 1);
      tc::commit(bars + 8 * (kVEmpty + buf), leader);
    }
    base += k1 - k0;
    done_with_item(number, bars);
  }
  tc::commit(bars + 8 * (kDrain + t), leader);
  tc::Drain drain;
  drain.wait(bars + 8 * (kDrain + t), 0);
  __syncwarp();
  if (w.dead) report(p.a.status, HS_ERR_TIMEOUT);
}

// ---- softmax and results (128 threads a query tile) ----
// 64 columns of tensor memory, a row a thread.
__device__ __forceinline__ void load64(uint32_t a, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(a));
}
template <int D>
__device__ __forceinline__ void softmax_items(const HeadsAttendParams& p, const Item* items, uint32_t smem, const uint8_t* raw, uint32_t tmem) {
  using L = Smem<D>;
  const uint32_t bars = smem + L::kBar;
  tc::Waiter w;
  const int t = threadIdx.x >> 7, lane = threadIdx.x & 31;
  const int row = threadIdx.x & 255;
  const uint32_t lanes = (uint32_t)(32 * ((threadIdx.x >> 5) & 3)) << 16;
  const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + L::kTo + t * L::kToStep, tp = tmem + lanes + L::kTp + t * L::kTpStep;
  const float scale = fabsf(p.scale_log2);
  uint32_t phase = 0, before = 0;  // key tiles of this query tile; of the CTA, in the items before
  auto record = [&]() {
    return reinterpret_cast<RunRecord*>(reinterpret_cast<uint8_t*>(p.workspace) + sizeof(RunHeader)) + blockIdx.x;
  };
  if (threadIdx.x == 0) *record() = RunRecord{};
#pragma unroll 1
  for (uint32_t k = 0;; ++k) {
    const Item* it = take_item(items, k, bars, w);
    if (!it) break;
    const int k0 = it->k0, end = it->end[t];
    const int sees = row < it->rows ? item_sees(p, *it, it->col0 + row) : 0;
    const int all_see = item_sees(p, *it, it->col0 + t * kQRows);  // (its first row sees least)
    int first = INT_MAX;  // token of the pages that are there
    float ref = -INFINITY, m = -INFINITY, l = 0.f, anchor = 0.f, qs = 0.f;
#pragma unroll 1
    for (int u = L::kParts * k0; u < L::kParts * end; ++u) {
      constexpr int kPages = L::kPages, kTokens = kPages * kHeadsPage;
      const uint32_t part = u % L::kParts, mine = 2 * part + t;
      const uint32_t scales = smem + L::kPage + (before + u / L::kParts - k0) % kScales * 32 + 4 * part;
      w.wait(bars + 8 * (kSFull + mine), phase & 1);
      __syncwarp();
      tc::fence_after();
      if (u == L::kParts * k0) qs = scale * power_of_field(raw[L::kMisc + (k & 1) * kBlock + row]);
      float s[kTokens], size[kPages], c[kPages], top[kPages];
      bool valid[kPages], all_valid = true;
#pragma unroll
      for (int i = 0; i < kPages; ++i) load64(ts + (part + i) * 64, s + 64 * i);
#pragma unroll
      for (int i = 0; i < kPages; ++i) {
        size[i] = lds_f(scales + 8 + 4 * i);
        c[i] = fminf(fmaxf(lds_f(scales + 4 * i) * qs, 1.17549435e-38f), 3.402823466e38f);
        valid[i] = lds_u(scales + 16 + 4 * i) != 0;
        all_valid &= valid[i];
      }
      tc::tmem_wait_ld();
      tc::touch<kTokens>(s);
      if constexpr (L::kApart) {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bars + 8 * (kSFree + mine));
      }
      if (!all_valid || (u + 1) * kTokens > all_see) {
#pragma unroll
        for (int i = 0; i < kPages; ++i) {
          const int left = valid[i] ? sees - u * kTokens - 64 * i : 0;
#pragma unroll
          for (int x = 0; x < 64; ++x)
            if (x >= left) s[64 * i + x] = -INFINITY;
        }
      }
      float most = -INFINITY, most_sized = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPages; ++i) {
        top[i] = fminf(__fmul_rn(tc::max_of<64>(s + 64 * i), c[i]), kMost);
        most = fmaxf(most, top[i]), most_sized = fmaxf(most_sized, top[i] + size[i]);
      }
      auto products_before = [&](uint32_t bar, uint32_t parity) {
        w.wait(bars + 8 * (kODone + bar), parity);
        __syncwarp();
        tc::fence_after();
      };
      if (L::kApart && phase > 0) products_before(mine, (phase - 1) & 1);  // have read P, and are in O
      // rare: scores beyond kLarge, or a reference that has to move (a page that is not seen has a top of -infinity and does not count)
      bool large = anchor != 0.f;
#pragma unroll
      for (int i = 0; i < kPages; ++i) large |= fabsf(top[i]) > kLarge && top[i] != -INFINITY;
      if (__any_sync(0xFFFFFFFFu, large || most_sized > ref + kLazy)) {
        if (__any_sync(0xFFFFFFFFu, large)) {
          if (fabsf(most) <= 3.402823466e38f && (most - anchor > kLarge || (ref == -INFINITY && fabsf(most) > kLarge))) {
            const float by = most - anchor;
            anchor = most;
            ref -= by, m -= by;
          }
#pragma unroll
          for (int x = 0; x < kTokens; ++x) s[x] = __fsub_rn(__fmul_rn(s[x], c[x >> 6]), anchor);  // (rounded as the tops are)
          most -= anchor, most_sized = -INFINITY;
#pragma unroll
          for (int i = 0; i < kPages; ++i) top[i] -= anchor, c[i] = 1.f, most_sized = fmaxf(most_sized, top[i] + size[i]);
        }
        const bool over = most_sized > ref + kLazy;
        const float now = over ? most_sized - kTop : ref;
        const float alpha = over ? exp2f(ref - now) : 1.f;
        ref = now;
        if (u > L::kParts * k0) {
          if constexpr (L::kParts == 2) products_before(mine ^ 2, (part ? phase : phase - 1) & 1);  // the page before is in O
#pragma unroll 1
          for (int x = 0; x < D; x += 16) {
            float o[16];
            tc::tmem_ld16(to + x, o);
            tc::tmem_wait_ld();
            tc::touch<16>(o);
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] *= alpha;
            tc::tmem_st16(to + x, o);
          }
          tc::tmem_wait_st();
        }
      }
      const float r = ref == -INFINITY ? 0.f : ref;
      if (most > m + kFar) {
        l *= tc::exp2_fast(m - most);
        m = most;
      }
#pragma unroll
      for (int i = 0; i < kPages; ++i) {
        float bias = size[i] - r;
        if (top[i] + size[i] < r - kFar) bias = top[i] < -2.f * kLarge ? -INFINITY : -kFar - top[i];
        const float2 c2 = make_float2(c[i], c[i]), b2 = make_float2(bias, bias);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
        uint32_t pk[32];
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          const float2 z = tc::fma2(make_float2(s[64 * i + 2 * y], s[64 * i + 2 * y + 1]), c2, b2);
          const float2 e = make_float2(tc::exp2_fast(z.x), tc::exp2_fast(z.y));
          if (y & 1)
            sum1 = tc::add2(sum1, e);
          else
            sum0 = tc::add2(sum0, e);
          pk[y] = pack_half(e.x, e.y);
        }
        tc::tmem_st16(tp + L::kTpPage * (part + i), reinterpret_cast<const float*>(pk));
        tc::tmem_st16(tp + L::kTpPage * (part + i) + 16, reinterpret_cast<const float*>(pk + 16));
        l += ((sum0.x + sum0.y) + (sum1.x + sum1.y)) * (bias == -INFINITY ? 0.f : tc::exp2_fast(-bias - m));  // (NaN stays)
      }
      tc::tmem_wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bars + 8 * (kPReady + mine));
#pragma unroll
      for (int i = 0; i < kPages; ++i)
        if (first == INT_MAX && valid[i]) first = u * kTokens + 64 * i;
      if (part == L::kParts - 1) ++phase;
    }
    if (sees > first) m = fmaxf(m, kLowest);
    // results
    const bool work = end > k0, whole = k0 == 0 && it->k1 == it->tiles;
    if (work) {
      w.wait(bars + 8 * (kODone + 2 * (L::kParts - 1) + t), (phase - 1) & 1);
      __syncwarp();
      tc::fence_after();
    }
    const int* nan_first = reinterpret_cast<const int*>(raw + L::kNan) + (k & 1) * D;
    const bool nans = work && *(reinterpret_cast<const volatile int*>(raw + L::kFlag) + (k & 1)) != 0;
    const bool there = row < it->rows;
    const bool f16 = p.a.dtype == HS_FP16;
    if (!whole) {
      uint8_t* ws = reinterpret_cast<uint8_t*>(p.workspace);
      const int64_t slot = (int64_t)blockIdx.x * 2 + it->part;
      float4* parts = reinterpret_cast<float4*>(ws + ws_parts_offset(gridDim.x)) + slot * (D / 4) * kBlock + row;
      if (work) {
#pragma unroll 1
        for (int x = 0; x < D; x += 16) {
          float o[16];
          tc::tmem_ld16(to + x, o);
          tc::tmem_wait_ld();
          tc::touch<16>(o);
#pragma unroll
          for (int y = 0; y < 16; y += 4) {
            if (nans) {
#pragma unroll
              for (int z = 0; z < 4; ++z)
                if (sees > nan_first[x + y + z]) o[y + z] = __uint_as_float(0x7FC00000u);
            }
            if (there) parts[(x + y) / 4 * kBlock] = make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
          }
        }
      }
      if (there)
        *(reinterpret_cast<float4*>(ws + ws_stats_offset(gridDim.x)) + slot * kBlock + row) = make_float4(ref, m, l, anchor);
      if (threadIdx.x == 0 && k0 == 0)
        *record() = RunRecord{it->begin, it->begin + it->tiles, it->t0, it->head, it->col0 / kBlock, it->rows};
    } else {
      const int c = it->col0 + row, token = c / p.group, head = it->head * p.group + c - token * p.group;
      const bool writes = there && HS_CHECK(it->t0 + token < p.a.n && head < p.a.q_heads, kChkOutPos);
      uint16_t* out = static_cast<uint16_t*>(p.a.out) + (it->t0 + token) * p.a.out_token_stride + head * p.a.out_head_stride;
      const bool some = work && !saw_none(m, l);
      const float2 by = result_factors(ref, m, l);
#pragma unroll 1
      for (int x = 0; x < D; x += 16) {
        float o[16];
        if (work) {
          tc::tmem_ld16(to + x, o);
          tc::tmem_wait_ld();
          tc::touch<16>(o);
        }
        if (nans) {
#pragma unroll
          for (int y = 0; y < 16; ++y)
            if (sees > nan_first[x + y]) o[y] = __uint_as_float(0x7FC00000u);
        }
        uint32_t v[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) v[y] = pack(f16, some ? o[2 * y] * by.x * by.y : 0.f, some ? o[2 * y + 1] * by.x * by.y : 0.f);
        if (writes) {
          *reinterpret_cast<uint4*>(out + x) = make_uint4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<uint4*>(out + x + 8) = make_uint4(v[4], v[5], v[6], v[7]);
        }
      }
      if (there && p.a.lse) {
        const int col = it->col0 + row, token = col / p.group;
        p.a.lse[(it->t0 + token) * p.a.q_heads + it->head * p.group + col - token * p.group] = result_lse(anchor, m, l);
      }
    }
    before += it->k1 - k0;
    tc::fence_before();
    done_with_item(k, bars);
  }
  if (w.dead) report(p.a.status, HS_ERR_TIMEOUT);
}

// Where this CTA's run begins; by all threads, before the roles part.  Scratch: shared memory that nothing else uses yet.
struct Scratch {
  int64_t sums[kThreads / 32];
  Start start;
};
__device__ __forceinline__ void find_start(const HeadsAttendParams& p, int limit, Scratch* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // units of the request of each thread
  auto units_of = [&](int r) {
    Request q{};
    if (r < p.a.R) q.load(p, r, limit);
    int64_t mine = 0;
    for (unsigned has = __ballot_sync(0xFFFFFFFFu, q.blocks > 0); has; has &= has - 1) {
      const int who = __ffs(has) - 1;
      Request x;
      x.t0 = 0;
      x.n = __shfl_sync(0xFFFFFFFFu, q.n, who), x.ctx = __shfl_sync(0xFFFFFFFFu, q.ctx, who);
      x.keys = __shfl_sync(0xFFFFFFFFu, q.keys, who), x.blocks = __shfl_sync(0xFFFFFFFFu, q.blocks, who);
      const int64_t n = request_units(p, x) * p.pages.kv_heads;
      if (lane == who) mine = n;
    }
    return mine;
  };
  // all units, and (in the last round) those of the requests before this thread's, in its chunk of kThreads requests
  bool bad = false;
  int64_t total = 0, mine = 0, first = 0;
  for (int r0 = 0; r0 < p.a.R; r0 += kThreads) {
    const int r = r0 + threadIdx.x;
    int64_t t0;
    int n;
    bool wrong = false;
    if (r < p.a.R) wrong = !p.ragged.tokens(r, &t0, &n);
    mine = units_of(r);
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += x;
    }
    if (lane == 31) s->sums[warp] = upto;
    bad |= __syncthreads_or(wrong);
    first = total + upto - mine;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) first += s->sums[i];
      total += s->sums[i];
    }
    if (r0 + kThreads < p.a.R) __syncthreads();
  }
  if (bad) total = 0;
  const int64_t run = max((int64_t)kMinRun, (total + gridDim.x - 1) / gridDim.x), begin = run * blockIdx.x;
  if (threadIdx.x == 0) {
    s->start.at = begin;
    s->start.left = begin < total ? min(run, total - begin) : 0;
    if (blockIdx.x == 0) *reinterpret_cast<RunHeader*>(p.workspace) = RunHeader{run, total};
  }
  // the warp whose requests the run begins in looks for the block
  auto look = [&](int r0) {
    const unsigned owner = __ballot_sync(0xFFFFFFFFu, begin >= first && begin < first + mine);
    if (!owner) return;
    const int who = __ffs(owner) - 1, r = r0 + warp * 32 + who;
    Request q;
    q.load(p, r, limit);
    const int64_t a_head = quotient(__shfl_sync(0xFFFFFFFFu, mine, who), p.pages.kv_heads), offset = begin - __shfl_sync(0xFFFFFFFFu, first, who);
    const int head = (int)quotient(offset, a_head);
    int64_t left = offset - head * a_head;  // (a head's units may pass 32 bits, those of 32 blocks do not)
    int block = -1, in = 0;
    for (int b0 = 0; block < 0; b0 += 32) {
      const int n = b0 + lane < q.blocks ? kItemCost + q.tiles(p, b0 + lane) : 0;
      int upto = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += x;
      }
      const unsigned here = __ballot_sync(0xFFFFFFFFu, left < upto);
      if (here) {
        const int w = __ffs(here) - 1;
        block = b0 + w;
        in = (int)left - (__shfl_sync(0xFFFFFFFFu, upto, w) - __shfl_sync(0xFFFFFFFFu, n, w));
      } else {
        left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
        if (b0 + 32 >= q.blocks) block = 0;  // (not reached: the offset lies within the head's units)
      }
    }
    if (lane == 0) s->start.r = r, s->start.head = head, s->start.block = block, s->start.in = in;
  };
  if (begin < total) {
    if (p.a.R <= kThreads) {
      look(0);
    } else {  // the chunks once more
      int64_t before = 0;
      for (int r0 = 0; r0 < p.a.R; r0 += kThreads) {
        mine = units_of(r0 + threadIdx.x);
        int64_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
          if (lane >= d) upto += x;
        }
        __syncthreads();
        if (lane == 31) s->sums[warp] = upto;
        __syncthreads();
        first = before + upto - mine;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
          if (i < warp) first += s->sums[i];
          before += s->sums[i];
        }
        look(r0);
      }
    }
  }
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const HeadsAttendParams p, int limit) {
  using L = Smem<D>;
  extern __shared__ __align__(1024) uint8_t raw[];  // (all of the block's shared memory: the operands' swizzle wants this alignment)
  asm volatile("griddepcontrol.launch_dependents;");  // prompt_join_kernel waits for this kernel's results by itself
  const uint32_t smem = tc::smem_u32(raw);
  const uint32_t bars = smem + L::kBar;
  const int warp = threadIdx.x >> 5;
  Scratch* scratch = reinterpret_cast<Scratch*>(raw + L::kMisc);
  static_assert(sizeof(Scratch) <= 2 * kBlock, "scratch");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(raw + L::kFlag) + 2;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) tc::mbar_init(bars + 8 * (kStFull + i), 1), tc::mbar_init(bars + 8 * (kStEmpty + i), 4);
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(bars + 8 * (kSFull + i), 1);
      tc::mbar_init(bars + 8 * (kPReady + i), 4);
      tc::mbar_init(bars + 8 * (kODone + i), 1);
      tc::mbar_init(bars + 8 * (kSFree + i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bars + 8 * (kKFull + i), 4);
      tc::mbar_init(bars + 8 * (kKEmpty + i), 2);
      tc::mbar_init(bars + 8 * (kVFull + i), 4);
      tc::mbar_init(bars + 8 * (kVEmpty + i), 2);
      tc::mbar_init(bars + 8 * (kQFull + i), 4);
      tc::mbar_init(bars + 8 * (kQEmpty + i), 1);
      tc::mbar_init(bars + 8 * (kItem + i), 1);
      tc::mbar_init(bars + 8 * (kItemDone + i), kTakers);
      tc::mbar_init(bars + 8 * (kDrain + i), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  find_start(p, limit, scratch);
  const Start start = scratch->start;
  if (warp == kMmaWarp) tc::tmem_alloc(tc::smem_u32(tmem_slot), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  Item* items = reinterpret_cast<Item*>(raw + L::kItems);
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<D>::kSoftmax));
    softmax_items<D>(p, items, smem, raw, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<D>::kOther));
    if (warp >= kWidenWarp)
      widen_items<D>(p, items, smem, raw);
    else if (warp == kWalkWarp)
      walk_items<D>(p, start, limit, raw, bars);
    else if (warp == kLoadWarp)
      load_items<D>(p, items, smem);
    else
      issue_items<D>(p, items, warp - kMmaWarp, smem, tmem);
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::tmem_free(tmem, 512);
  }
}

// Joins the parts of items that several runs share, two at a time, so that their loads are on their way together (2 x 4 positions
// behind 131000, 2 x 16 heads of 128: 62 us for the whole call with one at a time, 54.6 us with two, 56.4 us with four, which take
// registers that more blocks need).  A thread has D / 8 dimensions (its warp's) of a row.  A block takes 32 rows of a cut item; where
// there are more than kFewParts, 8 rows, whose parts its lanes share out (64 tokens behind 16000, 1 x 2 heads, 21 parts: 25 us, 37 us
// without; with 10 parts, 8 x 8 heads, 49 us so and 48 us without).
constexpr int kJoinThreads = 256, kJoinRows = 32, kJoinFewRows = 8, kJoinParts = 2, kFewParts = 16, kMaxCtas = 512;
template <int D>
struct JoinedRow {
  static constexpr int kVecs = D / 32;  // float4 a thread
  Joined all;
  float4 acc[kVecs];
  __device__ __forceinline__ void add(float4 st, const float4* y) {
    if (saw_none(st.y, st.z)) return;
    const float2 f = all.join(st);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      acc[v].x = acc[v].x * f.x + f.y * y[v].x, acc[v].y = acc[v].y * f.x + f.y * y[v].y;
      acc[v].z = acc[v].z * f.x + f.y * y[v].z, acc[v].w = acc[v].w * f.x + f.y * y[v].w;
    }
  }
  // Parts first, first + step, .. of the item whose parts are i .. last.
  __device__ __forceinline__ void join(const float4* stats, const float4* parts, int i, int slot0, int first, int step, int last,
                                       int row, int piece) {
    all = Joined{};
#pragma unroll
    for (int v = 0; v < kVecs; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = first; x0 <= last; x0 += kJoinParts * step) {
      float4 st[kJoinParts], y[kJoinParts][kVecs];
#pragma unroll
      for (int x = 0; x < kJoinParts; ++x) {
        const int part = x0 + x * step;
        if (part > last) continue;
        const int64_t slot = (int64_t)part * 2 + (part == i ? slot0 : 0);
        st[x] = stats[slot * kBlock + row];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) y[x][v] = parts[(slot * (D / 4) + piece * kVecs + v) * kBlock + row];
      }
#pragma unroll
      for (int x = 0; x < kJoinParts; ++x)
        if (x0 + x * step <= last) add(st[x], y[x]);
    }
  }
  __device__ __forceinline__ void store(const HeadsAttendParams& p, const RunRecord& rec, int row, int piece) const {
    const float2 by = result_factors(all.ref, all.m, all.l);
    const int col = rec.group * kBlock + row, in_token = col / p.group;
    const int64_t token = rec.t0 + in_token;
    const int head = rec.head * p.group + col - in_token * p.group;
    if (!HS_CHECK(token < p.a.n && head < p.a.q_heads, kChkOutPos)) return;
    const bool f16 = p.a.dtype == HS_FP16;
    uint16_t* out = static_cast<uint16_t*>(p.a.out) + token * p.a.out_token_stride + head * p.a.out_head_stride + piece * (D / 8);
#pragma unroll
    for (int v = 0; v < kVecs; v += 2)
      *reinterpret_cast<uint4*>(out + 4 * v) = make_uint4(
          pack(f16, acc[v].x * by.x * by.y, acc[v].y * by.x * by.y), pack(f16, acc[v].z * by.x * by.y, acc[v].w * by.x * by.y),
          pack(f16, acc[v + 1].x * by.x * by.y, acc[v + 1].y * by.x * by.y), pack(f16, acc[v + 1].z * by.x * by.y, acc[v + 1].w * by.x * by.y));
    if (piece == 0 && p.a.lse)
      p.a.lse[token * p.a.q_heads + head] = result_lse(all.anchor, all.m, all.l);
  }
};
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 2) prompt_join_kernel(const HeadsAttendParams p, int ctas) {
  __shared__ CutLists<kJoinThreads, kMaxCtas> cuts;
  const int lane = threadIdx.x & 31, piece = threadIdx.x >> 5;  // (of 8)
  asm volatile("griddepcontrol.wait;" ::: "memory");            // for the results of prompt_kernel
  const uint8_t* ws = reinterpret_cast<const uint8_t*>(p.workspace);
  const RunHeader header = *reinterpret_cast<const RunHeader*>(ws);
  const RunRecord* records = reinterpret_cast<const RunRecord*>(ws + sizeof(RunHeader));
  const float4* stats = reinterpret_cast<const float4*>(ws + ws_stats_offset(ctas));
  const float4* parts = reinterpret_cast<const float4*>(ws + ws_parts_offset(ctas));
  int n[2];
  cuts.build(records, ctas, header.run, kFewParts, n);
  JoinedRow<D> mine;
  constexpr int kGroups = kBlock / kJoinRows, kFewGroups = kBlock / kJoinFewRows;
  const int few = n[0] * kGroups;
#pragma unroll 1
  for (int item = blockIdx.x; item < few + n[1] * kFewGroups; item += gridDim.x) {
    const bool many = item >= few;
    const int rows = many ? kJoinFewRows : kJoinRows, groups = many ? kFewGroups : kGroups, x = many ? item - few : item;
    const int i = cuts.at[many][x / groups], row = x % groups * rows + lane % rows;
    const RunRecord rec = records[i];
    const bool there = row < rec.cols;
    mine.join(stats, parts, i, rec.begin > i * header.run ? 1 : 0, i + lane / rows, 32 / rows,
              there ? (int)((rec.end - 1) / header.run) : -1, row, piece);
    // the lanes' shares are joined two and two; what the upper lanes make of them is not used
#pragma unroll 1
    for (int d = rows; d < 32; d *= 2) {
      auto other = [&](float f) { return __shfl_xor_sync(0xFFFFFFFFu, f, d); };
      const float4 st = make_float4(other(mine.all.ref), other(mine.all.m), other(mine.all.l), other(mine.all.anchor));
      float4 y[JoinedRow<D>::kVecs];
#pragma unroll
      for (int v = 0; v < JoinedRow<D>::kVecs; ++v)
        y[v] = make_float4(other(mine.acc[v].x), other(mine.acc[v].y), other(mine.acc[v].z), other(mine.acc[v].w));
      mine.add(st, y);
    }
    if (there && lane < rows) mine.store(p, rec, row, piece);
  }
}

template <int D>
cudaError_t launch(const HeadsAttendParams& p, int limit, int dev, int sms, cudaStream_t s) {
  using L = Smem<D>;
  static DeviceOnce once;
  const cudaError_t ready = once.ready(dev, [] {
    cudaFuncAttributes f{};
    cudaError_t e = cudaFuncGetAttributes(&f, prompt_kernel<D>);
    // the register trade waits for ever if the launch has fewer than it hands out
    if (e == cudaSuccess && f.numRegs != kRegsLaunch) e = cudaErrorInvalidKernelImage;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    return e;
  });
  if (ready != cudaSuccess) return ready;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  prompt_kernel<D><<<ctas, kThreads, L::kBytes, s>>>(p, limit);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // its launch overlaps the end of the kernel before
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(sms * 4);
  c.blockDim = dim3(kJoinThreads);
  c.stream = s;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &early;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, prompt_join_kernel<D>, p, ctas);
  count_launch();
  return e;
}

}  // namespace

uint32_t check_take_heads_prompt() {
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

size_t heads_prompt_workspace_bytes(int sms) { return ws_bytes(sms < kMaxCtas ? sms : kMaxCtas, 128); }

cudaError_t launch_heads_prompt(const HeadsAttendParams& p, int limit, int dev, int sms, cudaStream_t s) {
  return p.a.head_dim == 64 ? launch<64>(p, limit, dev, sms, s) : launch<128>(p, limit, dev, sms, s);
}

}  // namespace hs
