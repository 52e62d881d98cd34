// Absorbed latent attention over the rows of the paged pool, on the tensor cores.
//
// Mathematics.  One latent row serves all columns of an item (the heads of a token, or positions x heads of a
// request) as key and as value.  A tile is 128 keys; both products are computed transposed, so that the tile is
// the 128-row operand and a call with few columns wastes nothing:
//   S^T[128 keys][N]  = K[128][576] * Q^T[576][N]          (36 steps of 16)
//   O^T[512][N]      += V^T[512][128] * P^T[128][N]         (4 row blocks x 8 steps)
// V is the latent part of K: the same bytes, once read as a K-major and once as an M-major operand.  The softmax
// is online with a lazy reference: weights are exp2(s - m) with any m that keeps them in range, since fp32 sums
// and bf16 weights have the same relative precision at every magnitude.  m starts as the first tile's maximum and
// moves (with O and the sums rescaled) only when a score exceeds it by kLazy, so the maximum over 128 lanes is
// rarely needed.  Sums are kept per key lane and joined once per unit.
//
// Layout.  A unit is (item, group of N columns); units are cut into tiles, numbered in order, and every CTA takes
// an equal run of tiles; a unit that several CTAs share leaves partial results in the workspace, which
// combine_kernel joins in a fixed order.  One CTA per SM, 16 warps:
//   warps 0-7   producers: load the next tile's rows into registers while the current one is in use, and store
//               them (fp8 dequantised to bf16) into the 128-byte-swizzled tile as its parts become free;
//   warps 8-11  softmax and results (lane = key, later lane = latent dimension);
//   warp 12     issues the products.
// The warpgroups trade registers (kRegs*): the launch gives every thread 128.
// The tile (128 x 576 bf16, 144 KB) has one buffer, released in five parts (four 128-dimension blocks after their
// product with P, the key part after S, or after P when P takes its place).
#include "latent.cuh"
#include "tc.cuh"

namespace hs {
namespace {

constexpr int kTile = 128;
constexpr int kProducerWarps = 8;
constexpr int kThreads = 512;  // four warpgroups; warps 13-15 only take part in the set-up
constexpr int kMmaWarp = kProducerWarps + 4;
constexpr int kMaxCols = 64;
constexpr int kRegsLaunch = 128, kRegsProducer = 144, kRegsSoftmax = 168, kRegsMma = 56;
static_assert(2 * kRegsProducer + kRegsSoftmax + kRegsMma <= 4 * kRegsLaunch, "more registers than the launch has");
template <int kRegs>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }
constexpr int kSub = kTile * 128;  // bytes of a sub-tile: 128 keys x 64 bf16
constexpr float kLazy = 64.f;      // log2 units by which a score may exceed the reference

// Workspace: partial results [2 per CTA][kMaxCols][512], their log2 sums [2 per CTA][kMaxCols], run starts [CTA].
struct RunStart {
  int64_t total;        // tiles of the call
  int32_t item, off;    // first tile: item and tile number within it
  int32_t tiles, pad;   // tiles of one unit of the item
};
__host__ __device__ constexpr size_t ws_lse_offset(int sms) { return (size_t)sms * 2 * kMaxCols * kLatent * 4; }
__host__ __device__ constexpr size_t ws_run_offset(int sms) { return ws_lse_offset(sms) + (size_t)sms * 2 * kMaxCols * 4; }

__device__ __forceinline__ int item_keys(const AttendParams& p, int item) {
  if (!p.paged) return p.K;
  const int64_t room = (int64_t)p.max_pages * p.page_size;
  return max(0, (int)min(room, (int64_t)__ldg(p.ctx_len + item)));
}
__device__ __forceinline__ int tiles_of(int keys) { return max(1, (keys + kTile - 1) / kTile); }

// Where a role is in the CTA's run of tiles.
struct Cursor {
  int item, group, tile, tiles, keys;
  int64_t left;
  __device__ __forceinline__ void start(const AttendParams& p, const RunStart& r, int64_t run) {
    item = r.item;
    group = r.off / r.tiles;
    tile = r.off - group * r.tiles;
    tiles = r.tiles;
    left = run;
    keys = left > 0 ? item_keys(p, item) : 0;
  }
  // to the next tile; true when it belongs to another unit (left == 0: there is none)
  __device__ __forceinline__ bool next(const AttendParams& p, int groups) {
    --left;
    if (++tile < tiles) return false;
    tile = 0;
    if (++group == groups) {
      group = 0;
      ++item;
      if (left > 0) {
        keys = item_keys(p, item);
        tiles = tiles_of(keys);
      }
    }
    return true;
  }
};

// Row of key `k` of an item, or -1; bad (a data error) is set when the entry is not a valid one.
__device__ __forceinline__ int key_row(const AttendParams& p, int item, int k, int keys, bool& bad) {
  if (k >= keys) return -1;
  if (!p.paged) {
    const int r = __ldg(p.rows + (int64_t)item * p.K + k);
    if (r >= 0 && r < p.num_rows) return r;
    bad |= r != -1;
    return -1;
  }
  const int page = k / p.page_size;
  const int b = __ldg(p.table + (int64_t)item * p.max_pages + page);
  if (b >= 0 && b < p.num_blocks) return b * p.page_size + (k - page * p.page_size);
  bad = true;
  return -1;
}

template <int N>
struct Smem {
  static constexpr int kTileBytes = 9 * kSub;
  static constexpr int kQ = kTileBytes;
  static constexpr int kQBytes = 9 * N * 128;
  static constexpr bool kAlias = N == 64;  // no room for P of 64 columns: it takes the key part's place
  static constexpr int kP = kAlias ? 8 * kSub : kQ + kQBytes;
  static constexpr int kMisc = kQ + kQBytes + (kAlias ? 0 : kTile * N * 2);
  // misc: barriers, references, joined sums, column limits
  static constexpr int kBytes = kMisc + 1024 + 16 * N * 4 + 1024;  // + alignment of the base
};
enum Bar { kFull = 0, kEmpty = 5, kQFull = 10, kQEmpty, kSFull, kPReady, kOFull, kDrain, kBars };

template <int N>
constexpr int tmem_cols() { return N == 64 ? 512 : N == 32 ? 256 : 128; }

// Reduction of N values over the warp's 32 lanes by halving: lane l ends with the results of columns
// l * N / 32 .. (N = 16: column l / 2).
template <int N, typename F>
__device__ __forceinline__ void halve(float* v, int lane, F f) {
#pragma unroll
  for (int half = N / 2, d = 16; d; half >>= 1, d >>= 1) {
    if (half == 0) {  // N = 16: the two lanes of a column
      v[0] = f(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], d));
    } else {
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const bool up = lane & d;
        const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
        v[i] = f(keep, __shfl_xor_sync(0xFFFFFFFFu, send, d));
      }
    }
  }
}

__device__ __forceinline__ uint4 ldg_row(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void sts(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// 4 e4m3 codes times scale -> 4 bf16
__device__ __forceinline__ uint2 dequant4(uint32_t w, float scale) {
  uint32_t a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(w));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return make_uint2(tc::pack_bf16(x.x * scale, x.y * scale), tc::pack_bf16(y.x * scale, y.y * scale));
}

__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool any_softmax(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// ---------------------------------------------------------------------------------------------------------
// Producers

// Query tile of a unit: N columns x 576, zero for columns past the item's.
template <int N>
__device__ __forceinline__ void load_queries(const AttendParams& p, uint32_t q, int item, int group, int tid) {
  constexpr int kChunks = N * 72;  // 16-byte chunks: column-major over (column, chunk of the 576)
#pragma unroll 3
  for (int i = tid; i < kChunks; i += kProducerWarps * 32) {
    const int col = i / 72, j = i - col * 72;
    const int c = group * N + col;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c < p.cols) {
      const int pos = c / p.heads, head = c - pos * p.heads;
      const int64_t tok = (int64_t)item * p.P + pos;
      const __nv_bfloat16* src = j < 64 ? p.q_latent + tok * p.ql_tok + head * p.ql_head + 8 * j
                                        : p.q_rope + tok * p.qr_tok + head * p.qr_head + 8 * (j - 64);
      v = __ldg(reinterpret_cast<const uint4*>(src));
    }
    sts(q + (j >> 3) * (N * 128) + col * 128 + (((j & 7) ^ (col & 7)) << 4), v.x, v.y, v.z, v.w);
  }
}

template <int N>
__device__ __forceinline__ void produce_fp8(const AttendParams& p, uint32_t tile, uint32_t q, uint32_t bars, Cursor cur,
                                            int groups, tc::Waiter& w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int key0 = warp * 16 + (lane >> 3), j = lane & 7;  // this lane's keys key0 + 4 i, its 16-byte piece j
  uint4 lat[4][4], rope[4];
  float4 sc[4];
  const uint8_t* row[4];
  int ids[4];
  bool bad = false;  // reported by the softmax warps

  Cursor ahead = cur;  // the tile whose rows are fetched next
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int id = key_row(p, ahead.item, ahead.tile * kTile + key0 + 4 * i, ahead.keys, bad);
    row[i] = id < 0 ? nullptr : p.base + (int64_t)id * HS_ROW_BYTES_FP8;
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto fetch = [&](int c, int i) { lat[c][i] = row[i] ? ldg_row(row[i] + 128 * c + 16 * j) : zero; };
  auto fetch_rope = [&](int i) { rope[i] = row[i] ? ldg_row(row[i] + 528 + 16 * j) : zero; };
  auto fetch_scales = [&](int i) {
    const uint4 s = row[i] ? ldg_row(row[i] + 512) : zero;
    sc[i] = make_float4(__uint_as_float(s.x), __uint_as_float(s.y), __uint_as_float(s.z), __uint_as_float(s.w));
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) fetch_scales(i);
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) fetch(c, i);
#pragma unroll
  for (int i = 0; i < 4; ++i) fetch_rope(i);
  ahead.next(p, groups);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    ids[i] = ahead.left > 0 ? key_row(p, ahead.item, ahead.tile * kTile + key0 + 4 * i, ahead.keys, bad) : -1;

  bool fresh = true;
  uint32_t it = 0, seg = 0;
  while (cur.left > 0) {
    if (fresh) {
      if (seg > 0) w.wait(bars + 8 * kQEmpty, (seg - 1) & 1);
      load_queries<N>(p, q, cur.item, cur.group, threadIdx.x);
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bars + 8 * kQFull);
      ++seg;
    }
    // rows of the tile ahead; their ids arrived during the last tile
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = ids[i] < 0 ? nullptr : p.base + (int64_t)ids[i] * HS_ROW_BYTES_FP8;
    const bool more = ahead.left > 0;
    if (more) ahead.next(p, groups);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ids[i] = ahead.left > 0 ? key_row(p, ahead.item, ahead.tile * kTile + key0 + 4 * i, ahead.keys, bad) : -1;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (it > 0) w.wait(bars + 8 * (kEmpty + c), (it - 1) & 1);
      const uint32_t sub = tile + (2 * c + (j >> 2)) * kSub;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + 4 * i;
        const float s = c == 0 ? sc[i].x : c == 1 ? sc[i].y : c == 2 ? sc[i].z : sc[i].w;
        const uint2 a = dequant4(lat[c][i].x, s), b = dequant4(lat[c][i].y, s);
        const uint2 d = dequant4(lat[c][i].z, s), e = dequant4(lat[c][i].w, s);
        const uint32_t at = sub + key * 128;
        const int ch = (j & 3) * 2;
        // lanes of the upper sub-tile write their halves in the other order: no two lanes of a store share a bank
        const bool flip = j >> 2;
        sts(at + (((ch + flip) ^ (key & 7)) << 4), flip ? d.x : a.x, flip ? d.y : a.y, flip ? e.x : b.x, flip ? e.y : b.y);
        sts(at + (((ch + !flip) ^ (key & 7)) << 4), flip ? a.x : d.x, flip ? a.y : d.y, flip ? b.x : e.x, flip ? b.y : e.y);
        if (more) {
          fetch(c, i);
          if (c == 3) fetch_scales(i);
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bars + 8 * (kFull + c));
    }
    if (it > 0) w.wait(bars + 8 * (kEmpty + 4), (it - 1) & 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key0 + 4 * i;
      sts(tile + 8 * kSub + key * 128 + ((j ^ (key & 7)) << 4), rope[i].x, rope[i].y, rope[i].z, rope[i].w);
      if (more) fetch_rope(i);
    }
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bars + 8 * (kFull + 4));
    fresh = cur.next(p, groups);
    ++it;
  }
}

// bf16 rows need no conversion: 16-byte asynchronous copies straight into the swizzled tile, the next tile's rows
// prefetched into L2 meanwhile.
template <int N>
__device__ __forceinline__ void produce_bf16(const AttendParams& p, uint32_t tile, uint32_t q, uint32_t bars, Cursor cur,
                                             int groups, tc::Waiter& w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int key0 = warp * 16 + (lane >> 3), j = lane & 7;
  bool bad = false;
  bool fresh = true;
  uint32_t it = 0, seg = 0;
  int ids[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ids[i] = key_row(p, cur.item, cur.tile * kTile + key0 + 4 * i, cur.keys, bad);
  while (cur.left > 0) {
    if (fresh) {
      if (seg > 0) w.wait(bars + 8 * kQEmpty, (seg - 1) & 1);
      load_queries<N>(p, q, cur.item, cur.group, threadIdx.x);
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bars + 8 * kQFull);
      ++seg;
    }
    const uint8_t* row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = ids[i] < 0 ? nullptr : p.base + (int64_t)ids[i] * HS_ROW_BYTES_BF16;
    Cursor ahead = cur;
    fresh = ahead.next(p, groups);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ids[i] = ahead.left > 0 ? key_row(p, ahead.item, ahead.tile * kTile + key0 + 4 * i, ahead.keys, bad) : -1;
    auto copy = [&](int sub, int i) {
      const int key = key0 + 4 * i;
      const uint32_t dst = tile + sub * kSub + key * 128 + ((j ^ (key & 7)) << 4);
      const uint8_t* src = row[i] ? row[i] + 128 * sub + 16 * j : p.base;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(row[i] ? 16 : 0) : "memory");
    };
    // part c is signalled once the copies of part c + 1 have been issued
#pragma unroll
    for (int c = 0; c < 6; ++c) {
      if (c < 5) {
        if (it > 0) w.wait(bars + 8 * (kEmpty + c), (it - 1) & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (c < 4) {
            copy(2 * c, i);
            copy(2 * c + 1, i);
          } else {
            copy(8, i);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (c == 1) {  // the ids of the next tile have arrived by now
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (ids[i] >= 0) {
              const uint8_t* r = p.base + (int64_t)ids[i] * HS_ROW_BYTES_BF16;
              asm volatile("prefetch.global.L2 [%0];" ::"l"(r + 128 * j));
              if (j == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(r + 1024));
            }
        }
      }
      if (c > 0) {
        if (c < 5)
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bars + 8 * (kFull + c - 1));
      }
    }
    cur = ahead;
    ++it;
  }
}

// ---------------------------------------------------------------------------------------------------------
// Products (one thread)

template <int N>
__device__ __forceinline__ void issue_products(const AttendParams& p, uint32_t tile, uint32_t q, uint32_t pt, uint32_t bars,
                                               uint32_t tmem, Cursor cur, int groups, tc::Waiter& w) {
  using L = Smem<N>;
  constexpr uint32_t kIdS = tc::idesc_bf16(128, N, false, false);
  constexpr uint32_t kIdO = tc::idesc_bf16(128, N, true, true);
  constexpr uint64_t kPSwizzle = N == 64 ? tc::kSwizzle128 : N == 32 ? tc::kSwizzle64 : tc::kSwizzle32;
  bool fresh = true;
  uint32_t it = 0, seg = 0;
  while (cur.left > 0) {
    if (fresh) w.wait(bars + 8 * kQFull, seg & 1);
    const bool first = fresh;
#pragma unroll
    for (int c = 0; c < 5; ++c) {
      w.wait(bars + 8 * (kFull + c), it & 1);
      tc::fence_after();
#pragma unroll
      for (int k = 0; k < (c < 4 ? 8 : 4); ++k) {
        const int sub = 2 * c + (k >> 2), in = (k & 3) * 32;
        tc::mma_ss(tmem, tc::desc(tile + sub * kSub + in, 16, 1024, tc::kSwizzle128),
                   tc::desc(q + sub * (N * 128) + in, 16, 1024, tc::kSwizzle128), kIdS, c > 0 || k > 0);
      }
    }
    tc::commit(bars + 8 * kSFull);
    if (!L::kAlias) tc::commit(bars + 8 * (kEmpty + 4));
    fresh = cur.next(p, groups);
    const bool last = fresh || cur.left == 0;
    if (last) tc::commit(bars + 8 * kQEmpty);
    w.wait(bars + 8 * kPReady, it & 1);
    tc::fence_after();
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        tc::mma_ss(tmem + N + g * N, tc::desc(tile + 2 * g * kSub + k * 2048, kSub, 1024, tc::kSwizzle128),
                   tc::desc(pt + k * 16 * N * 2, 16, 8 * N * 2, kPSwizzle), kIdO, !first || k > 0);
      tc::commit(bars + 8 * (kEmpty + g));
    }
    if (L::kAlias) tc::commit(bars + 8 * (kEmpty + 4));
    if (last) {
      tc::commit(bars + 8 * kOFull);
      ++seg;
    }
    ++it;
  }
  // nothing of this CTA's products is in flight when the others leave
  tc::commit(bars + 8 * kDrain);
  tc::Waiter drain;
  drain.wait(bars + 8 * kDrain, 0);
}

// ---------------------------------------------------------------------------------------------------------
// Softmax and results (128 threads)

template <int N>
__device__ __forceinline__ void softmax(const AttendParams& p, uint32_t pt, uint32_t bars, uint32_t tmem, float* ref,
                                        float* red, Cursor cur, int groups, int sms, tc::Waiter& w) {
  const int tid = threadIdx.x - kProducerWarps * 32;
  const int lane = tid & 31, warp = tid >> 5;
  const uint32_t tm = tmem + ((uint32_t)(32 * warp) << 16);  // this warp's lanes
  float* alpha = ref + N;                                    // [N] rescale factors, then 1 / sum
  int* limit = reinterpret_cast<int*>(ref + 2 * N);          // [N] keys that a column sees
  bool fresh = true, at_start = false;
  bool first_run = true;  // this CTA's first segment
  uint32_t it = 0, seg = 0;
  float l[N];
  while (cur.left > 0) {
    const int item = cur.item, group = cur.group;
    const int ncols = min(N, p.cols - group * N);
    if (fresh) {
      at_start = cur.tile == 0;
      if (tid < N) {
        ref[tid] = -INFINITY;
        const int c = min(group * N + tid, p.cols - 1);
        limit[tid] = p.paged ? __ldg(p.ctx_len + item) - p.P + 1 + c / p.heads : p.K;
      }
#pragma unroll
      for (int c = 0; c < N; ++c) l[c] = 0.f;
      bar_softmax();
    }
    const int k = cur.tile * kTile + tid;
    bool bad = false;
    const bool there = key_row(p, item, k, cur.keys, bad) >= 0;
    if (bad && group == 0) report(p.status, p.paged ? HS_ERR_TABLE_RANGE : HS_ERR_ID_RANGE);
    // columns differ in what they see only in the last P - 1 keys
    const bool ragged = p.paged && p.P > 1 && (cur.tile + 1) * kTile > limit[0];
    const bool first = fresh;
    w.wait(bars + 8 * kSFull, it & 1);
    __syncwarp();
    tc::fence_after();
    float s[N];
    auto scores = [&]() {
#pragma unroll
      for (int c = 0; c < N; c += 16) tc::tmem_ld16(tm + c, s + c);
      tc::tmem_wait_ld();
      tc::touch<N>(s);
#pragma unroll
      for (int c = 0; c < N; ++c) {
        s[c] *= p.scale_log2;
        if (!there) s[c] = -INFINITY;
      }
      if (ragged) {
#pragma unroll
        for (int c = 0; c < N; ++c)
          if (k >= limit[c]) s[c] = -INFINITY;
      }
    };
    scores();
    bool over = false;
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const float4 m = *reinterpret_cast<const float4*>(ref + c);
      const float mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) over |= s[c + x] > mm[x] + kLazy;
    }
    if (any_softmax(over)) {
      // a new reference for every column: the maximum of the old one and this tile's scores
      halve<N>(s, lane, [](float a, float b) { return fmaxf(a, b); });
      if (N == 64) {
        red[warp * N + 2 * lane] = s[0];
        red[warp * N + 2 * lane + 1] = s[1];
      } else if (N == 32) {
        red[warp * N + lane] = s[0];
      } else {
        red[warp * N + (lane >> 1)] = s[0];
      }
      bar_softmax();
      if (tid < N) {
        const float old = ref[tid];
        const float top = fmaxf(fmaxf(fmaxf(red[tid], red[N + tid]), fmaxf(red[2 * N + tid], red[3 * N + tid])), old);
        ref[tid] = top;
        alpha[tid] = old == -INFINITY ? 0.f : exp2f(old - top);
      }
      bar_softmax();
#pragma unroll
      for (int c = 0; c < N; ++c) l[c] *= alpha[c];
      if (!first) {
        // the products of the tiles before have finished: they were committed before these scores
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
#pragma unroll
          for (int c = 0; c < N; c += 16) {
            float o[16];
            tc::tmem_ld16(tm + N + g * N + c, o);
            tc::tmem_wait_ld();
            tc::touch<16>(o);
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] *= alpha[c + x];
            tc::tmem_st16(tm + N + g * N + c, o);
          }
        }
        tc::tmem_wait_st();
      }
      scores();
    }
    // weights, their sums per lane, and P^T: [key][column], 2 N bytes a key, swizzled like the descriptor says
#pragma unroll
    for (int c = 0; c < N; c += 8) {
      uint32_t out[4];
#pragma unroll
      for (int x = 0; x < 8; x += 4) {
        const float4 m = *reinterpret_cast<const float4*>(ref + c + x);
        const float mm[4] = {m.x, m.y, m.z, m.w};
        float e[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float v = s[c + x + y];
          e[y] = v == -INFINITY ? 0.f : tc::exp2_fast(v - mm[y]);
          l[c + x + y] += e[y];
        }
        out[x / 2] = tc::pack_bf16(e[0], e[1]);
        out[x / 2 + 1] = tc::pack_bf16(e[2], e[3]);
      }
      const int sw = N == 64 ? (tid & 7) : N == 32 ? ((tid >> 1) & 3) : ((tid >> 2) & 1);
      sts(pt + tid * (2 * N) + (((c / 8) ^ sw) << 4), out[0], out[1], out[2], out[3]);
    }
    tc::fence_async_smem();
    tc::fence_before();
    tc::mbar_arrive(bars + 8 * kPReady);

    const int unit_tiles = cur.tiles, tile = cur.tile;
    fresh = cur.next(p, groups);
    ++it;
    if (!fresh && cur.left > 0) continue;

    // the segment ends: join the sums, then the results
    const bool whole = at_start && tile + 1 == unit_tiles;
    halve<N>(l, lane, [](float a, float b) { return a + b; });
    if (N == 64) {
      red[warp * N + 2 * lane] = l[0];
      red[warp * N + 2 * lane + 1] = l[1];
    } else if (N == 32) {
      red[warp * N + lane] = l[0];
    } else {
      red[warp * N + (lane >> 1)] = l[0];
    }
    bar_softmax();
    const int slot = 2 * blockIdx.x + (first_run && !at_start ? 0 : 1);
    first_run = false;
    if (tid < N) {
      const float sum = (red[tid] + red[N + tid]) + (red[2 * N + tid] + red[3 * N + tid]);
      const float lse2 = sum == 0.f ? -INFINITY : ref[tid] + log2f(sum);
      alpha[tid] = sum == 0.f ? 0.f : 1.f / sum;
      if (!whole) {
        float* z = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.workspace) + ws_lse_offset(sms));
        z[slot * kMaxCols + tid] = lse2;
      } else if (p.lse && tid < ncols) {
        const int c = group * N + tid;
        p.lse[(int64_t)item * p.cols + c] = lse2 * kLn2;
      }
    }
    bar_softmax();
    w.wait(bars + 8 * kOFull, seg & 1);
    __syncwarp();
    ++seg;
    tc::fence_after();
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
      float o[N];
#pragma unroll
      for (int c = 0; c < N; c += 16) tc::tmem_ld16(tm + N + g * N + c, o + c);
      tc::tmem_wait_ld();
      tc::touch<N>(o);
      const int dim = 128 * g + tid;
      if (!whole) {
        float* z = p.workspace + ((int64_t)slot * kMaxCols) * kLatent + dim;
#pragma unroll
        for (int c = 0; c < N; ++c)
          if (c < ncols) z[(int64_t)c * kLatent] = o[c] * alpha[c];
      } else {
        // pairs of lanes exchange so that each writes two neighbouring dimensions of one column
#pragma unroll
        for (int c = 0; c < N; c += 2) {
          const float a = o[c] * alpha[c], b = o[c + 1] * alpha[c + 1];
          const bool odd = lane & 1;
          const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1);
          const int mine = c + odd;
          if (mine < ncols) {
            const int gc = group * N + mine;
            const int pos = gc / p.heads, head = gc - pos * p.heads;
            __nv_bfloat16* dst = p.out + ((int64_t)item * p.P + pos) * p.out_tok + head * p.out_head + (dim - odd);
            *reinterpret_cast<uint32_t*>(dst) = odd ? tc::pack_bf16(got, b) : tc::pack_bf16(a, got);
          }
        }
      }
    }
    tc::fence_before();
  }
}

// Sum of v over the block's threads, and this thread's exclusive prefix (kThreads threads).
__device__ int64_t block_scan(int64_t v, int64_t* total, int64_t* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += scratch[i];
    all += scratch[i];
  }
  *total = all;
  return before + x - v;
}

__host__ __device__ __forceinline__ int64_t run_begin(int64_t total, int ctas, int b) { return total * b / ctas; }

template <int N, int kRowBytes>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const AttendParams p, int groups, int sms) {
  using L = Smem<N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~uintptr_t(1023));
  __shared__ RunStart start;
  __shared__ uint32_t tmem_slot;
  __shared__ int64_t scratch[kThreads / 32];
  const int warp = threadIdx.x >> 5;
  const uint32_t base = tc::smem_u32(smem);
  const uint32_t bars = base + L::kMisc;
  float* ref = reinterpret_cast<float*>(smem + L::kMisc + 256);  // references, factors, limits: 3 N; joins: 4 N
  float* red = ref + 4 * N;

  // The run of tiles of this CTA.
  int64_t total, begin, run = 0;
  int ctas = gridDim.x;
  if (!p.paged) {
    const int tiles = tiles_of(p.K);
    total = (int64_t)p.items * groups * tiles;
    if (total < ctas) ctas = (int)total;
    if ((int)blockIdx.x < ctas) {
      begin = run_begin(total, ctas, blockIdx.x);
      run = run_begin(total, ctas, blockIdx.x + 1) - begin;
      if (threadIdx.x == 0) {
        const int per_item = groups * tiles;
        start = RunStart{total, (int)(begin / per_item), (int)(begin % per_item), tiles, 0};
      }
    }
  } else {
    int64_t mine = 0;
    bool long_ctx = false;
    for (int i = threadIdx.x; i < p.items; i += kThreads) {
      mine += (int64_t)tiles_of(item_keys(p, i)) * groups;
      long_ctx |= __ldg(p.ctx_len + i) > (int64_t)p.max_pages * p.page_size;
    }
    if (long_ctx && blockIdx.x == 0) report(p.status, HS_ERR_TABLE_RANGE);
    block_scan(mine, &total, scratch);
    if (total < ctas) ctas = (int)total;
    if ((int)blockIdx.x < ctas) {
      begin = run_begin(total, ctas, blockIdx.x);
      run = run_begin(total, ctas, blockIdx.x + 1) - begin;
      int64_t passed = 0;
      for (int i0 = 0; i0 < p.items; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        const int tiles = i < p.items ? tiles_of(item_keys(p, i)) : 0;
        int64_t all;
        const int64_t at = passed + block_scan((int64_t)tiles * groups, &all, scratch);
        if (begin >= at && begin < at + (int64_t)tiles * groups) start = RunStart{total, i, (int)(begin - at), tiles, 0};
        passed += all;
        if (begin < passed) break;
      }
    }
  }
  if ((int)blockIdx.x >= ctas) return;

  if (threadIdx.x == 0) {
    for (int c = 0; c < 5; ++c) {
      tc::mbar_init(bars + 8 * (kFull + c), kProducerWarps);
      tc::mbar_init(bars + 8 * (kEmpty + c), 1);
    }
    tc::mbar_init(bars + 8 * kQFull, kProducerWarps);
    tc::mbar_init(bars + 8 * kQEmpty, 1);
    tc::mbar_init(bars + 8 * kSFull, 1);
    tc::mbar_init(bars + 8 * kPReady, 128);
    tc::mbar_init(bars + 8 * kOFull, 1);
    tc::mbar_init(bars + 8 * kDrain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tc::tmem_alloc(tc::smem_u32(&tmem_slot), tmem_cols<N>());
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  if (threadIdx.x == 0)
    reinterpret_cast<RunStart*>(reinterpret_cast<uint8_t*>(p.workspace) + ws_run_offset(sms))[blockIdx.x] = start;
  Cursor cur;
  cur.start(p, start, run);
  tc::Waiter w;
  if (warp < kProducerWarps) {
    more_registers<kRegsProducer>();
    if (kRowBytes == HS_ROW_BYTES_FP8)
      produce_fp8<N>(p, base, base + L::kQ, bars, cur, groups, w);
    else
      produce_bf16<N>(p, base, base + L::kQ, bars, cur, groups, w);
  } else if (warp < kMmaWarp) {
    more_registers<kRegsSoftmax>();
    softmax<N>(p, base + L::kP, bars, tmem, ref, red, cur, groups, sms, w);
  } else {
    fewer_registers<kRegsMma>();
    if (threadIdx.x == kMmaWarp * 32)
      issue_products<N>(p, base, base + L::kQ, base + L::kP, bars, tmem, cur, groups, w);
  }
  if (w.dead) report(p.status, HS_ERR_TIMEOUT);
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::tmem_free(tmem, tmem_cols<N>());
  }
}

// Joins the partial results of the units that run boundary b = blockIdx.x + 1 is the first to cut: the results are
// weighted by exp2 of their log2 sums, in the order of the runs.  128 threads: 4 dimensions each, kJoinCols columns.
constexpr int kJoinCols = 4;
__global__ void __launch_bounds__(128) combine_kernel(const AttendParams p, int groups, int n, int sms, int grid) {
  const uint8_t* ws = reinterpret_cast<const uint8_t*>(p.workspace);
  const RunStart* runs = reinterpret_cast<const RunStart*>(ws + ws_run_offset(sms));
  const float* lse = reinterpret_cast<const float*>(ws + ws_lse_offset(sms));
  const int b = blockIdx.x + 1;
  const int64_t total = runs[0].total;
  const int ctas = (int)min((int64_t)grid, total);
  if (b >= ctas) return;
  const RunStart r = runs[b];
  const int group = r.off / r.tiles, tile = r.off - group * r.tiles;
  if (tile == 0) return;
  const int64_t unit0 = run_begin(total, ctas, b) - tile, unit1 = unit0 + r.tiles;
  if (run_begin(total, ctas, b - 1) > unit0) return;  // an earlier boundary cuts this unit
  int last = b;  // runs b - 1 .. last hold parts of it
  while (last + 1 < ctas && run_begin(total, ctas, last + 1) < unit1) ++last;
  const int ncols = min(n, p.cols - group * n);
  const int c1 = min(ncols, (int)(blockIdx.y + 1) * kJoinCols);
  for (int c = blockIdx.y * kJoinCols; c < c1; ++c) {
    float top = -INFINITY;
    for (int i = b - 1; i <= last; ++i) top = fmaxf(top, lse[(2 * i + (i < b)) * kMaxCols + c]);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = b - 1; i <= last; ++i) {
      const int slot = 2 * i + (i < b);
      const float z = lse[slot * kMaxCols + c];
      const float f = z == -INFINITY ? 0.f : exp2f(z - top);
      const float4 v = reinterpret_cast<const float4*>(p.workspace + ((int64_t)slot * kMaxCols + c) * kLatent)[threadIdx.x];
      sum += f;
      acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int gc = group * n + c;
    const int pos = gc / p.heads, head = gc - pos * p.heads;
    __nv_bfloat16* dst = p.out + ((int64_t)r.item * p.P + pos) * p.out_tok + head * p.out_head + 4 * threadIdx.x;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(tc::pack_bf16(acc.x * inv, acc.y * inv), tc::pack_bf16(acc.z * inv, acc.w * inv));
    if (threadIdx.x == 0 && p.lse)
      p.lse[(int64_t)r.item * p.cols + gc] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

template <int N, int kRowBytes>
cudaError_t launch(const AttendParams& p, int sms, cudaStream_t s) {
  static const cudaError_t ready = [] {
    cudaFuncAttributes a{};
    cudaError_t e = cudaFuncGetAttributes(&a, attend_kernel<N, kRowBytes>);
    // the register trade waits for ever if the launch has fewer than it hands out
    if (e == cudaSuccess && a.numRegs != kRegsLaunch) e = cudaErrorInvalidKernelImage;
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(attend_kernel<N, kRowBytes>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<N>::kBytes);
    return e;
  }();
  if (ready != cudaSuccess) return ready;
  const int groups = (p.cols + N - 1) / N;
  // a rows call knows its tiles; a pages call learns them on the device
  int grid = sms;
  bool cut = true;  // whether a unit may be shared by CTAs
  if (!p.paged) {
    const int64_t tiles = p.K > 0 ? (p.K + kTile - 1) / kTile : 1;
    const int64_t units = (int64_t)p.items * groups;
    if (units * tiles < grid) grid = (int)(units * tiles);
    cut = tiles > 1 && units % grid != 0;
  }
  attend_kernel<N, kRowBytes><<<grid, kThreads, Smem<N>::kBytes, s>>>(p, groups, sms);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !cut || grid < 2) return e;
  combine_kernel<<<dim3(grid - 1, N / kJoinCols), 128, 0, s>>>(p, groups, N, sms, grid);
  count_launch();
  return cudaGetLastError();
}

template <int kRowBytes>
cudaError_t launch_cols(const AttendParams& p, int sms, cudaStream_t s) {
  if (p.cols <= 16) return launch<16, kRowBytes>(p, sms, s);
  if (p.cols <= 32) return launch<32, kRowBytes>(p, sms, s);
  return launch<64, kRowBytes>(p, sms, s);
}

}  // namespace

size_t attend_workspace_bytes(int sms) { return ws_run_offset(sms) + (size_t)sms * sizeof(RunStart); }

cudaError_t launch_attend(const AttendParams& p, int sms, cudaStream_t s) {
  return p.row_bytes == HS_ROW_BYTES_FP8 ? launch_cols<HS_ROW_BYTES_FP8>(p, sms, s)
                                         : launch_cols<HS_ROW_BYTES_BF16>(p, sms, s);
}

}  // namespace hs
