// Attention over pages of grouped heads in 8 bits, for few query columns a head of keys: single tokens and verify positions.
//
// Mathematics.  The columns of a unit (request, head of keys and values) are its query tokens x the query heads that share the
// head.  Over the pages (64 tokens each), with page scales sk and sv, log2 units throughout:
//   S = Q K^T (codes),  c = |scale| log2(e) sk qs,  t = S c + log2(sv),  P = 2^(t - R),  O += P V (codes).
// A page enters the result as its weights times sv, so P, which is rounded to fp16, is that product, and the reference R
// follows its largest: it is placed kTop above the largest t, and moves (with O) only when a t passes it by kLazy.  The sum of
// the weights themselves, 2^(S c - m), follows a reference m of its own, a thread's: from P by one factor a page.  Where a page's
// largest t is more than 2^kFar below R (values that are all but zero, say), log2(sv) is raised for its P so far that these stay
// normal numbers in fp32 for that sum; in fp16 they are zero then.
// Codes are exact in fp16; a query column is divided by qs, a power of two (mostly 1) that brings it into fp16's range.
//
// Layout.  The products are on mma.sync: what bounds a call of few columns is reading the pages, and these fragments come from
// shared memory as the pages are, 16 bytes a lane, with no transposition, no barrier between warps and no tensor memory:
//   scores   queries are the 16 rows, keys the 8 columns of a product.  Products of sums do not care for the order of the
//            dimensions: lane (g, t) takes 16 consecutive dimensions 16 t.. of a key and the queries are loaded to match.  The
//            8 keys of product j are 16 (g / 2) + 2 j + g % 2, so that lane t ends with keys 16 t .. 16 t + 15 of a query row;
//   results  which is what the transposed product O^T = V^T P^T wants of its right operand, V^T being stored by dimension.
// A worker is W warps (16 columns each, or 8) and a ring of copies (cp.async.bulk, a page's keys or values of a head each);
// every worker of the grid takes an equal run of pages, whatever the contexts' lengths; units that are cut leave partial
// results in the workspace, which join_kernel joins in a fixed order.
//
// What bounds it.  64 requests of up to 16384 tokens, 8 x 8 heads of 128 dimensions: 221 us, 5.6 TB/s of the codes, the copies
// being ahead of the products.  With 32 columns (64 requests of up to 4004 tokens, 4 x 8 heads, four positions) the products are, 73 us:
// each of two warps widens all of a page's codes for its 16 columns.  4 requests of 4096 tokens, 8 x 4 heads: 18.5 us: 2 until
// the runs are found, 3 until the first page is there, 5 of two pages' chains, 5 of joining, and the launches.
#include <algorithm>

#include "heads_device.cuh"

HS_CHECK_WORD

namespace hs {
namespace {

using namespace heads;

constexpr int kRingBytes = 192 * 1024;
// Requests of more columns are left to heads_prompt.cu.  With 32 columns a request (4 positions, 4 x 8 heads of 128 dimensions) this takes
// 86 us for 64 requests of up to 4000 tokens with offsets, 52 us for four of 30000, 15 us for one of 3000; that 93, 52 and 21 us.  With
// 48 (3 positions, 4 x 16 heads) that takes 92, 45 and 21 us; a group of 64 columns here, which four warps would share, took half as long
// again for the first two and 16 us for the last, and is not built.
constexpr int kStepCols = 32;

// Workspace: header, a record a worker, statistics [worker][2][cols][4], results [worker][2][cols][D].
__host__ __device__ constexpr size_t ws_stats_offset(int workers) { return sizeof(RunHeader) + (size_t)workers * sizeof(RunRecord); }
__host__ __device__ constexpr size_t ws_parts_offset(int workers, int cols) {
  return ws_stats_offset(workers) + (size_t)workers * 2 * cols * 16;
}
__host__ __device__ constexpr size_t ws_bytes(int workers, int cols, int dim) {
  return ws_parts_offset(workers, cols) + (size_t)workers * 2 * cols * dim * 4;
}

// What a call has of one request.
struct Request {
  int64_t t0;          // its first query token
  int n, ctx, keys;    // query tokens; context; tokens of it that the table has room for
  int tiles, groups;   // pages (at least one), groups of columns; 0 where it has no queries, or more than `limit` columns
  __device__ __forceinline__ void load(const HeadsAttendParams& p, int r, int cols, int limit) {
    p.ragged.tokens(r, &t0, &n);
    ctx = __ldg(p.a.ctx_len + r);
    keys = max(0, min(ctx, p.a.max_pages * kHeadsPage));
    const int all = n * p.group;
    const bool mine = n > 0 && all <= limit;
    tiles = mine ? max(1, (keys + kHeadsPage - 1) / kHeadsPage) : 0;
    groups = mine ? (all + cols - 1) / cols : 0;
  }
  // tokens of the context that query token i (counted from t0) sees
  __device__ __forceinline__ int sees(const HeadsAttendParams& p, int i) const {
    return p.a.causal ? max(0, min(keys, ctx - n + 1 + i)) : keys;
  }
};

// A place in the call's tiles: of request r, a head and a group of columns, page `tile`.
struct Cursor {
  int r, head, group, tile;
  Request q;
  int64_t left;
  // to the next tile; true when it is in another unit (left == 0: there is none)
  __device__ __forceinline__ bool next(const HeadsAttendParams& p, int cols, int limit) {
    --left;
    if (++tile < q.tiles) return false;
    tile = 0;
    if (++group < q.groups) return true;
    group = 0;
    if (++head < p.pages.kv_heads) return true;
    head = 0;
    if (left <= 0) return true;
    do q.load(p, ++r, cols, limit);
    while (q.tiles == 0 && r + 1 < p.a.R);
    return true;
  }
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
  return x + __shfl_xor_sync(0xFFFFFFFFu, x, 2);
}
template <int D, int NC, int W>
struct Shape {
  static constexpr int kWarps = 8, kThreads = kWarps * 32;
  static constexpr int kCols = NC * W, kWorkers = kWarps / W;  // columns of a group, workers of a CTA
  static constexpr int kUnit = D * kHeadsPage;                 // bytes of a page's keys (or values) of a head
  // a slot: the codes, the 16 bytes that hold the scale, a word that says whether the page is there
  static constexpr int kSlot = kUnit + 32, kSlots = kRingBytes / kUnit / kWorkers;
  static constexpr int kBars = kWorkers * kSlots * kSlot, kNan = kBars + 2 * kWorkers * kSlots * 8;
  static constexpr int kBytes = kNan + kWarps * D * 4;
  static_assert(kSlots >= 3 && kBytes <= 232448 - 1024, "shared memory");
};

// Copies of a worker's pages, in order: keys, values, keys, ... (one warp of the worker).
template <int D, int NC, int W>
struct Producer {
  using L = Shape<D, NC, W>;
  Cursor at;
  uint32_t count = 0;  // copies so far
  int cached = -1, cached_request = -1, cached_tile = -1;  // a lane's table entry of request and 32 pages
  int block = 0;
  bool there = false;

  __device__ __forceinline__ void issue(const HeadsAttendParams& p, uint32_t ring, uint32_t full, uint32_t empty, int limit,
                                        tc::Waiter& w) {
    if (at.left <= 0 || w.dead) return;
    const int lane = threadIdx.x & 31;
    const uint32_t slot = count % L::kSlots;
    if (W > 1 && count >= L::kSlots) {
      await(w, empty + 8 * slot, (count / L::kSlots - 1) & 1);
      if (w.dead) return;
    }
    const bool values = count & 1;
    if (!values) {
      if (cached_request != at.r || cached_tile != (at.tile & ~31)) {
        cached_request = at.r, cached_tile = at.tile & ~31;
        const int page = cached_tile + lane;
        cached = -1;
        if (page * kHeadsPage < at.q.keys && HS_CHECK(at.r < p.a.R && page < p.a.max_pages, kChkTablePage))
          cached = __ldg(p.pages.table + (int64_t)at.r * p.a.max_pages + page);
      }
      block = __shfl_sync(0xFFFFFFFFu, cached, at.tile & 31);
      there = block >= 0 && block < p.pages.num_blocks;
      if (lane == 0 && (at.q.ctx > at.q.keys || (at.q.keys > 0 && !there))) report(p.a.status, HS_ERR_TABLE_RANGE);
      if (!there) block = 0;  // (copied and not used: the ring goes on as ever)
    }
    __syncwarp();
    if (lane == 0) {
      const int head = at.head, scale = values ? p.pages.kv_heads + head : head;
      const uint32_t to = ring + slot * L::kSlot, bar = full + 8 * slot;
      const uint8_t* codes = p.pages.codes(block, head, D) + (values ? L::kUnit : 0);
      sts_u(to + L::kUnit + 16, there);
      tc::mbar_expect(bar, L::kUnit + 16);
      bulk_copy(to, codes, L::kUnit, bar);
      bulk_copy(to + L::kUnit, p.pages.scale(block, scale & ~3, D), 16, bar);
    }
    ++count;
    if (values) at.next(p, L::kCols, limit);
  }
  // After the worker is done with `taken` copies: the next one, and another while the ring is not full yet.
  __device__ __forceinline__ void refill(const HeadsAttendParams& p, uint32_t ring, uint32_t full, uint32_t empty, int limit,
                                         uint32_t taken, tc::Waiter& w) {
    issue(p, ring, full, empty, limit, w);
    if (L::kSlots > 4 && count < taken + L::kSlots) issue(p, ring, full, empty, limit, w);
  }
};

template <int D, int NC, int W>
__global__ void __launch_bounds__(Shape<D, NC, W>::kThreads, 1) steps_kernel(const HeadsAttendParams p, int limit) {
  using L = Shape<D, NC, W>;
  constexpr int kWarps = L::kWarps, kThreads = L::kThreads;
  constexpr int kHalves = NC / 8, kBlocks = D / 64;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ Cursor starts[L::kWorkers];
  __shared__ int64_t sums[kWarps];
  asm volatile("griddepcontrol.launch_dependents;");  // join_kernel waits for this kernel's results by itself
  const uint32_t smem = tc::smem_u32(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int worker = warp / W, sub = warp % W;
  const int workers = L::kWorkers * gridDim.x;
  const int number = worker * gridDim.x + blockIdx.x;  // of this worker in the order of runs
  const uint32_t ring = smem + worker * L::kSlots * L::kSlot;
  const uint32_t full = smem + L::kBars + worker * L::kSlots * 8, empty = full + L::kWorkers * L::kSlots * 8;

  if (threadIdx.x < L::kWorkers * L::kSlots) {
    tc::mbar_init(smem + L::kBars + 8 * threadIdx.x, 1);
    tc::mbar_init(smem + L::kBars + 8 * (L::kWorkers * L::kSlots + threadIdx.x), W);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the call's tiles, and where each worker's run begins: those of kThreads requests at a time, looked through once for their sum
  // and, where there are more, once again
  bool bad = false;
  int64_t total = 0, run = 1;
  const int rounds = (p.a.R + kThreads - 1) / kThreads;
  int64_t before = 0;  // tiles of the rounds before
#pragma unroll 1
  for (int pass = 0, x = 0; rounds > 0; ++x) {
    if (x == rounds) {
      x = 0;
      if (++pass == 2 || rounds == 1) break;
      before = 0;
    }
    const int r = x * kThreads + threadIdx.x;
    Request q{};
    bool wrong = false;
    if (r < p.a.R) {
      int64_t t0;
      int n;
      wrong = !p.ragged.tokens(r, &t0, &n);
      q.load(p, r, L::kCols, limit);
    }
    const int64_t mine = (int64_t)p.pages.kv_heads * q.groups * q.tiles;
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += y;
    }
    if (lane == 31) sums[warp] = upto;
    bad |= __syncthreads_or(wrong);
    int64_t first = before + upto - mine;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) first += sums[i];
      before += sums[i];
    }
    __syncthreads();
    if (pass == 0 && x + 1 == rounds) {
      total = bad ? 0 : before;
      run = max((int64_t)1, (total + workers - 1) / workers);
    }
    if (total > 0 && (pass == 1 || rounds == 1)) {
      for (int k = 0; k < L::kWorkers; ++k) {
        const int64_t begin = run * (k * (int64_t)gridDim.x + blockIdx.x);
        if (begin >= first && begin < first + mine) {
          starts[k].r = r;
          starts[k].q = q;
          starts[k].left = begin - first;  // (from its first tile on; the worker itself finds head, group and tile)
        }
      }
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (bad) report(p.a.status, HS_ERR_ID_RANGE);
    *reinterpret_cast<RunHeader*>(p.workspace) = RunHeader{run, total};
  }
  // query tokens that no request has: zeros and -infinity
  if (p.ragged.cu) {
    const int64_t from = bad ? 0 : __ldg(p.ragged.cu), to = bad ? 0 : __ldg(p.ragged.cu + p.a.R);
    const int64_t none = from + (p.a.n - to), words = (int64_t)p.a.q_heads * (D / 8);
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < none * words; i += (int64_t)gridDim.x * kThreads) {
      const int64_t k = i / words, token = k < from ? k : to + (k - from);
      const int head = (int)(i % words) / (D / 8), piece = (int)(i % words) % (D / 8);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + token * p.a.out_token_stride + head * p.a.out_head_stride +
                                8 * piece) = make_uint4(0, 0, 0, 0);
      if (piece == 0 && p.a.lse) p.a.lse[token * p.a.q_heads + head] = -INFINITY;
    }
  }
  const int64_t begin = run * number;
  RunRecord* record = reinterpret_cast<RunRecord*>(reinterpret_cast<uint8_t*>(p.workspace) + sizeof(RunHeader)) + number;
  float4* stats = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(p.workspace) + ws_stats_offset(workers)) +
                  (int64_t)number * 2 * L::kCols;
  float* parts = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.workspace) + ws_parts_offset(workers, L::kCols)) +
                 (int64_t)number * 2 * L::kCols * D;
  if (begin >= total) {
    if (sub == 0 && lane == 0) *record = RunRecord{};
    return;
  }

  const bool f16 = p.a.dtype == HS_FP16;
  const float sign = scale_sign(p.scale_log2), scale = fabsf(p.scale_log2);
  tc::Waiter w;
  Producer<D, NC, W> producer;
  Cursor cur = starts[worker];
  const int64_t unit = quotient(cur.left, cur.q.tiles);
  cur.tile = (int)(cur.left - unit * cur.q.tiles);
  cur.head = (int)quotient(unit, cur.q.groups);
  cur.group = (int)(unit - (int64_t)cur.head * cur.q.groups);
  cur.left = min(run, total - begin);
  producer.at = cur;
  uint32_t taken = 0;  // copies that this warp is done with
  int* nan_first = reinterpret_cast<int*>(smem_raw + L::kNan) + warp * D;  // by dimension: the first token whose value is NaN
  int64_t place = begin;  // of the current tile in the call
  RunRecord cut{};

#pragma unroll 1
  while (cur.left > 0 && !w.dead) {
    // a unit, or this run's part of it
    const int head = cur.head, group = cur.group, tile0 = cur.tile;
    const int cols = min(L::kCols, cur.q.n * p.group - group * L::kCols) - sub * NC;  // of this warp
    const Request req = cur.q;
    const int64_t unit_begin = place - tile0;
    uint32_t q[kBlocks][4][kHalves][2];
    float qs[kHalves];
    int sees[kHalves];
    int64_t row[kHalves];  // token and head of the column, as their offset in lse
    bool any_nan = false;
    for (int i = lane; i < D; i += 32) nan_first[i] = INT_MAX;
    uint4 raw[kHalves][kBlocks][2];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int c = 8 * h + g, in_group = group * L::kCols + sub * NC + c;
      const bool there = c < cols;
      const int token = there ? in_group / p.group : 0, qh = head * p.group + (there ? in_group - token * p.group : 0);
      sees[h] = there ? req.sees(p, token) : INT_MAX;
      row[h] = (req.t0 + token) * p.a.q_heads + qh;
      const uint16_t* src =
          static_cast<const uint16_t*>(p.a.q) + (req.t0 + token) * p.a.q_token_stride + qh * p.a.q_head_stride + 16 * t;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          raw[h][b][i] = there ? __ldg(reinterpret_cast<const uint4*>(src + 64 * b) + i) : make_uint4(0, 0, 0, 0);
    }
    // (the first copies start while the queries are on their way)
    if (sub == 0 && producer.count == 0) {
#pragma unroll 1
      for (int i = 0; i < min(L::kSlots, 4); ++i) producer.issue(p, ring, full, empty, limit, w);
    }
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      float x[kBlocks][16], top = 0.f;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (f16)
            Vec8<__half>{raw[h][b][i]}.values(x[b] + 8 * i);
          else
            Vec8<__nv_bfloat16>{raw[h][b][i]}.values(x[b] + 8 * i);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[b][i]));
      }
      top = quad_max(top);
      const int e = query_field(top);
      const float f = sign * power_of_field(254 - e);
      qs[h] = scale * power_of_field(e);
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) q[b][i][h][k] = pack_half(x[b][4 * i + 2 * k] * f, x[b][4 * i + 2 * k + 1] * f);
    }
    __syncwarp();
    int all_see = sees[0];
    if constexpr (kHalves == 2) all_see = min(all_see, sees[1]);
    all_see = __reduce_min_sync(0xFFFFFFFFu, all_see);
    float ref[kHalves], m[kHalves], l[kHalves], anchor[kHalves], o[kHalves][D / 16][4];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      ref[h] = m[h] = -INFINITY;
      l[h] = anchor[h] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[h][i][k] = 0.f;
    }

    int first = INT_MAX;  // token of the pages that are there
    bool moved;
#pragma unroll 1
    do {
      const int key0 = cur.tile * kHeadsPage;
      // scores
      uint32_t slot = ring + taken % L::kSlots * L::kSlot, at = slot - smem;  // (also as an offset)
      await(w, full + 8 * (taken % L::kSlots), taken / L::kSlots & 1);
      const bool valid = lds_u(slot + L::kUnit + 16) != 0;
      const float sk = lds_f(slot + L::kUnit + 4 * (head & 3));
      float s[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
// (loads first, and products of eight sums in turn: each waits for its own sum's last)
        uint4 k[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          k[j] = *reinterpret_cast<const uint4*>(smem_raw + at + b * 4096 + (16 * (g >> 1) + 2 * j + (g & 1)) * 64 + 16 * t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint2 x = half_of_codes(i == 0 ? k[j].x : i == 1 ? k[j].y : i == 2 ? k[j].z : k[j].w);
            if constexpr (kHalves == 2)
              mma(s[j], q[b][i][0][0], q[b][i][1][0], q[b][i][0][1], q[b][i][1][1], x.x, x.y);
            else
              mma(s[j], q[b][i][0][0], 0u, q[b][i][0][1], 0u, x.x, x.y);
          }
        }
      }
      __syncwarp();
      ++taken;
      if (W > 1 && lane == 0) tc::mbar_arrive(empty + 8 * ((taken - 1) % L::kSlots));
      if (sub == 0) producer.refill(p, ring, full, empty, limit, taken, w);

      // weights
      slot = ring + taken % L::kSlots * L::kSlot, at = slot - smem;
      await(w, full + 8 * (taken % L::kSlots), taken / L::kSlots & 1);
      const float sv = lds_f(slot + L::kUnit + 4 * ((p.pages.kv_heads + head) & 3));
      const float size = valid ? log2f(sv) : 0.f;
      if (first == INT_MAX && valid) first = key0;
      const bool mixed = !valid || key0 + kHeadsPage > all_see;
      uint32_t pf[kHalves][4][2];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        if (mixed) {
          const int left = valid ? sees[h] - key0 - 16 * t : 0;
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (2 * j + e >= left) s[j][2 * h + e] = -INFINITY;
        }
        float top = s[0][2 * h];
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(fmaxf(top, s[j][2 * h]), s[j][2 * h + 1]);
        float c = fminf(fmaxf(sk * qs[h], 1.17549435e-38f), 3.402823466e38f);
        top = fminf(__fmul_rn(top, c), kMost);
        if (__any_sync(0xFFFFFFFFu, fabsf(top) > kLarge || anchor[h] != 0.f)) {
          const float most = quad_max(top);
          if (fabsf(most) <= 3.402823466e38f && (most - anchor[h] > kLarge || (ref[h] == -INFINITY && fabsf(most) > kLarge))) {
            const float by = most - anchor[h];
            anchor[h] = most;
            ref[h] -= by, m[h] -= by;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[j][2 * h + e] = __fsub_rn(__fmul_rn(s[j][2 * h + e], c), anchor[h]);  // (rounded as top is)
          top -= anchor[h];
          c = 1.f;
        }
        if (__any_sync(0xFFFFFFFFu, top + size > ref[h] + kLazy)) {
          const float most = quad_max(top + size);
          const float now = most > ref[h] + kLazy ? most - kTop : ref[h];
          const float alpha = now == ref[h] ? 1.f : exp2f(ref[h] - now);
          ref[h] = now;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = __shfl_sync(0xFFFFFFFFu, alpha, 4 * (2 * t + e));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[h][i][e] *= f, o[h][i][2 + e] *= f;
          }
        }
        const float r = ref[h] == -INFINITY ? 0.f : ref[h];
        float bias = size - r;
        if (top + size < r - kFar) bias = top < -2.f * kLarge ? -INFINITY : -kFar - top;  // (-infinity: no weight at all)
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = tc::exp2_fast(fmaf(s[j][2 * h], c, bias)), y = tc::exp2_fast(fmaf(s[j][2 * h + 1], c, bias));
          sum0 += x, sum1 += y;
          pf[h][j >> 1][j & 1] = pack_half(x, y);
        }
        if (top > m[h] + kFar) {
          l[h] *= exp2f(m[h] - top);
          m[h] = top;
        }
        l[h] += (sum0 + sum1) * (bias == -INFINITY ? 0.f : exp2f(-bias - m[h]));  // (NaN stays, whatever the factor)
      }

      // results
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        uint4 v[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            v[i][y] = *reinterpret_cast<const uint4*>(smem_raw + at + b * 4096 + (16 * i + 8 * y + g) * 64 + 16 * t);
        if (mixed) {  // a weight of zero does not cancel a NaN: who sees it is settled at the unit's end
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t words[4] = {v[i][y].x, v[i][y].y, v[i][y].z, v[i][y].w};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t is = nan_codes(words[x]);
                if (is) {
                  words[x] &= ~((is >> 7) * 0xFFu);
                  if (valid) atomicMin(nan_first + 64 * b + 16 * i + 8 * y + g, key0 + 16 * t + 4 * x + ((__ffs(is) - 1) >> 3));
                  any_nan = true;
                }
              }
              v[i][y] = make_uint4(words[0], words[1], words[2], words[3]);
            }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 c = half_of_codes(x == 0 ? v[i][0].x : x == 1 ? v[i][0].y : x == 2 ? v[i][0].z : v[i][0].w);
            const uint2 d = half_of_codes(x == 0 ? v[i][1].x : x == 1 ? v[i][1].y : x == 2 ? v[i][1].z : v[i][1].w);
#pragma unroll
            for (int h = 0; h < kHalves; ++h) mma(o[h][4 * b + i], c.x, d.x, c.y, d.y, pf[h][x][0], pf[h][x][1]);
          }
        }
      }
      __syncwarp();
      ++taken;
      if (W > 1 && lane == 0) tc::mbar_arrive(empty + 8 * ((taken - 1) % L::kSlots));
      if (sub == 0) producer.refill(p, ring, full, empty, limit, taken, w);
      ++place;
      moved = cur.next(p, L::kCols, limit);
    } while (!moved && cur.left > 0 && !w.dead);

    // the unit's results, or this run's part of them
    __syncwarp();
    any_nan = __any_sync(0xFFFFFFFFu, any_nan);
    const bool whole = tile0 == 0 && moved;
    const int part = unit_begin > begin ? 1 : 0;
    if (!moved && tile0 == 0)
      cut = RunRecord{unit_begin, unit_begin + req.tiles, req.t0, head, group, cols + sub * NC};
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      float most = quad_max(m[h]);
      const float sum_l = quad_sum(m[h] == most ? l[h] : l[h] * exp2f(m[h] - most));
      if (sees[h] > first) most = fmaxf(most, kLowest);
      const bool there = 8 * h + g < cols;
      if (any_nan) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int limit_key = __shfl_sync(0xFFFFFFFFu, sees[h], 4 * (2 * t + e));
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              if (limit_key > nan_first[16 * i + 8 * y + g]) o[h][i][2 * y + e] = __uint_as_float(0x7FC00000u);
        }
      }
      if (whole) {
        const float2 by = result_factors(ref[h], most, sum_l);
        float f0[2], f1[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f0[e] = __shfl_sync(0xFFFFFFFFu, by.x, 4 * (2 * t + e));
          f1[e] = __shfl_sync(0xFFFFFFFFu, by.y, 4 * (2 * t + e));
        }
        uint16_t* out = static_cast<uint16_t*>(p.a.out) + row[h] / p.a.q_heads * p.a.out_token_stride +
                        row[h] % p.a.q_heads * p.a.out_head_stride + 2 * t;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t x = transposed(pack(f16, o[h][i][2 * y] * f0[0] * f1[0], o[h][i][2 * y + 1] * f0[1] * f1[1]));
            if (there && HS_CHECK(row[h] < p.a.n * p.a.q_heads, kChkOutPos)) *reinterpret_cast<uint32_t*>(out + 16 * i + 8 * y) = x;
          }
        if (there && t == 0 && p.a.lse) p.a.lse[row[h]] = result_lse(anchor[h], most, sum_l);
      } else {
        const int at = part * L::kCols + sub * NC + 8 * h;
        if (t == 0) stats[at + g] = make_float4(ref[h], most, sum_l, anchor[h]);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) parts[(at + 2 * t + (k & 1)) * D + 16 * i + 8 * (k >> 1) + g] = o[h][i][k];
      }
    }
    __syncwarp();
  }
  if (sub == 0 && lane == 0) *record = cut;
  if (sub == 0) {  // no copy is in flight when the CTA ends
    tc::Drain drain;
    for (; taken < producer.count; ++taken) drain.wait(full + 8 * (taken % L::kSlots), taken / L::kSlots & 1);
  }
  if (w.dead) report(p.a.status, HS_ERR_TIMEOUT);
}

// Joins the parts of units that several runs share, a column a warp; where there are more than kFewParts, a column a block, whose
// warps take every eighth part each.  Four parts at a time, so that their loads are on their way together.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinParts = 4, kFewParts = 16, kMaxWorkers = 2048;

// Column c of a cut unit: parts x0, x0 + step, ... <= last.
template <int D>
__device__ __forceinline__ Joined join_parts(const float4* stats, const float* parts, int i, int slot0, int c, int group_cols, int x0,
                                             int step, int last, float (&acc)[D / 32]) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  Joined res;
  for (; x0 <= last; x0 += step * kJoinParts) {
    float4 st[kJoinParts];
    float v[kJoinParts][kPer];
#pragma unroll
    for (int y = 0; y < kJoinParts; ++y) {
      const int x = x0 + y * step;
      if (x > last) continue;
      const int64_t at = ((int64_t)x * 2 + (x == i ? slot0 : 0)) * group_cols + c;
      st[y] = stats[at];
      if constexpr (kPer == 4) {
        const float4 f = *reinterpret_cast<const float4*>(parts + at * D + 4 * lane);
        v[y][0] = f.x, v[y][1] = f.y, v[y][2] = f.z, v[y][3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(parts + at * D + 2 * lane);
        v[y][0] = f.x, v[y][1] = f.y;
      }
    }
#pragma unroll
    for (int y = 0; y < kJoinParts; ++y) {
      if (x0 + y * step > last || saw_none(st[y].y, st[y].z)) continue;
      const float2 f = res.join(st[y]);
#pragma unroll
      for (int d = 0; d < kPer; ++d) acc[d] = acc[d] * f.x + v[y][d] * f.y;
    }
  }
  return res;
}
template <int D>
__device__ __forceinline__ void store_joined(const HeadsAttendParams& p, const RunRecord& rec, int c, int group_cols, const Joined& all,
                                             const float (&out)[D / 32]) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const float2 by = result_factors(all.ref, all.m, all.l);
  const int in_unit = rec.group * group_cols + c;
  const int64_t token = rec.t0 + in_unit / p.group;
  const int qh = rec.head * p.group + in_unit % p.group;
  if (!HS_CHECK(token < p.a.n && qh < p.a.q_heads, kChkOutPos)) return;
  uint16_t* to = static_cast<uint16_t*>(p.a.out) + token * p.a.out_token_stride + qh * p.a.out_head_stride + lane * kPer;
#pragma unroll
  for (int d = 0; d < kPer; d += 2)
    *reinterpret_cast<uint32_t*>(to + d) = pack(p.a.dtype == HS_FP16, out[d] * by.x * by.y, out[d + 1] * by.x * by.y);
  if (lane == 0 && p.a.lse) p.a.lse[token * p.a.q_heads + qh] = result_lse(all.anchor, all.m, all.l);
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const HeadsAttendParams p, int workers, int group_cols) {
  constexpr int kPer = D / 32;
  __shared__ CutLists<kJoinThreads, kMaxWorkers> cuts;
  __shared__ float4 joined[kJoinWarps];
  __shared__ float sums[kJoinWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the results of steps_kernel
  const uint8_t* ws = reinterpret_cast<const uint8_t*>(p.workspace);
  const RunHeader header = *reinterpret_cast<const RunHeader*>(ws);
  const RunRecord* records = reinterpret_cast<const RunRecord*>(ws + sizeof(RunHeader));
  const float4* stats = reinterpret_cast<const float4*>(ws + ws_stats_offset(workers));
  const float* parts = reinterpret_cast<const float*>(ws + ws_parts_offset(workers, group_cols));
  int n[2];
  cuts.build(records, workers, header.run, kFewParts, n);
  for (int item = blockIdx.x * kJoinWarps + warp; item < n[0] * group_cols; item += gridDim.x * kJoinWarps) {
    const int i = cuts.at[0][item / group_cols], c = item % group_cols;
    const RunRecord rec = records[i];
    if (c >= rec.cols) continue;
    float acc[kPer] = {};
    const Joined all = join_parts<D>(stats, parts, i, rec.begin > i * header.run ? 1 : 0, c, group_cols, i, 1,
                                     (int)((rec.end - 1) / header.run), acc);
    store_joined<D>(p, rec, c, group_cols, all, acc);
  }
  for (int item = blockIdx.x; item < n[1] * group_cols; item += gridDim.x) {
    const int i = cuts.at[1][item / group_cols], c = item % group_cols;
    const RunRecord rec = records[i];
    if (c >= rec.cols) continue;
    float acc[kPer] = {};
    const Joined some = join_parts<D>(stats, parts, i, rec.begin > i * header.run ? 1 : 0, c, group_cols, i + warp, kJoinWarps,
                                      (int)((rec.end - 1) / header.run), acc);
    if (lane == 0) joined[warp] = make_float4(some.ref, some.m, some.l, some.anchor);
#pragma unroll
    for (int d = 0; d < kPer; ++d) sums[warp][lane * kPer + d] = acc[d];
    __syncthreads();
    if (warp == 0) {
      Joined all;
      float out[kPer] = {};
#pragma unroll
      for (int y = 0; y < kJoinWarps; ++y) {
        const float2 f = all.join(joined[y]);
#pragma unroll
        for (int d = 0; d < kPer; ++d) out[d] = out[d] * f.x + sums[y][lane * kPer + d] * f.y;
      }
      store_joined<D>(p, rec, c, group_cols, all, out);
    }
    __syncthreads();
  }
}

template <int D, int NC, int W>
cudaError_t launch_steps(const HeadsAttendParams& p, int limit, int dev, int sms, cudaStream_t s) {
  using L = Shape<D, NC, W>;
  static DeviceOnce once;
  const cudaError_t ready = once.ready(dev, [] {
    return cudaFuncSetAttribute(steps_kernel<D, NC, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  });
  if (ready != cudaSuccess) return ready;
  const int workers = sms * L::kWorkers;
  if (workers > kMaxWorkers) return cudaErrorInvalidConfiguration;
  steps_kernel<D, NC, W><<<sms, L::kThreads, L::kBytes, s>>>(p, limit);
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
  e = cudaLaunchKernelEx(&c, join_kernel<D>, p, workers, L::kCols);
  count_launch();
  return e;
}

template <int D>
cudaError_t launch_dim(const HeadsAttendParams& p, int limit, int dev, int sms, cudaStream_t s) {
  // Columns of a request, on average: a group takes them all, up to 32 (a ragged call's longer ones take several).  64 requests of up
  // to 4000 tokens, offsets given, in groups of 8, 16 and 32: with 8 columns (8 x 8 heads of 128) 75, 83 and 123 us; with 16 (4 x 16
  // heads) 66, 63 and 83 us; with 32 (4 positions, 4 x 8 heads) 98, 82 and 86 us, but 420 and 402 us in groups of 16 and 32 for 63 of up to
  // 16384, 8 x 8 heads.  The mean is all that the host knows of offsets, and the tokens of prompts are in it: 63 single tokens
  // beside a chunk of 512 (8 x 8 heads) run in groups of 32, 510 us, where groups of 8 would take 350.
  const int64_t cols = p.a.R > 0 ? (p.a.n + p.a.R - 1) / p.a.R * p.group : 1;
  if (cols <= 8) return launch_steps<D, 8, 1>(p, limit, dev, sms, s);
  if (cols <= 16) return launch_steps<D, 16, 1>(p, limit, dev, sms, s);
  return launch_steps<D, 16, 2>(p, limit, dev, sms, s);
}

}  // namespace

uint32_t check_take_heads_attend() {
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

size_t heads_workspace_bytes(int sms) {
  size_t most = heads_prompt_workspace_bytes(sms);
  auto shape = [&](int workers, int cols, int dim) { most = std::max(most, ws_bytes(sms * workers, cols, dim)); };
  shape(Shape<64, 8, 1>::kWorkers, 8, 64);
  shape(Shape<128, 8, 1>::kWorkers, 8, 128);
  shape(Shape<128, 16, 1>::kWorkers, 16, 128);
  shape(Shape<128, 16, 2>::kWorkers, 32, 128);
  return most;
}

cudaError_t launch_attend_heads(const HeadsAttendParams& p, int dev, int sms, cudaStream_t s) {
  // Without offsets all requests have as many columns.  With them the host does not know, and each kernel takes its own.
  const int64_t all = p.a.n * p.group;
  const int64_t most = p.ragged.cu ? all : all / p.a.R;
  if (p.ragged.cu || most <= kStepCols) {
    const cudaError_t e = p.a.head_dim == 64 ? launch_dim<64>(p, kStepCols, dev, sms, s) : launch_dim<128>(p, kStepCols, dev, sms, s);
    if (e != cudaSuccess) return e;
  }
  return most > kStepCols ? launch_heads_prompt(p, kStepCols, dev, sms, s) : cudaSuccess;
}

}  // namespace hs
