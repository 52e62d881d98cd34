// Absorbed latent attention over the rows of the paged pool, on the tensor cores.
//
// Mathematics.  One latent row serves all columns of an item (the heads of a token, or positions x heads of a
// request) as key and as value.  A tile is 64 keys; both products are computed transposed, so that the tile is
// the operand with 64 or 128 rows and a call with few columns wastes nothing:
//   S^T[64 keys][N]  = K[64][576] * Q^T[576][N]           (36 steps of 16)
//   O^T[512][N]     += V^T[512][64] * P^T[64][N]           (4 row blocks x 4 steps)
// V is the latent part of K: the same bytes, once read as a K-major and once as an M-major operand.  The softmax
// is online with a lazy reference: weights are exp2(t - m), t the scores in log2 units, with any m that keeps them in
// range, since fp32 sums have the same relative precision at every magnitude.  m starts kTop below the first tile's maximum
// and moves (with O and the sums rescaled) only when a score exceeds it by kLazy, so the maximum over a tile's keys is rarely
// needed.  Sums are kept per thread and joined once per unit.
//
// Types.  bf16 rows: both products in bf16.  The two operands of a product have one type, and bf16 values have fp32's
// range, so the weights are rounded to 8 bits: root mean square error 2.0e-3 of the results', against 1.7e-3 with 32 bits and
// one rounding.  fp8 rows: both in fp16 (1.67e-3 against 1.66e-3), because an e4m3 code becomes fp16 in one instruction for
// two and fp16's 11 bits hold it exactly, while its range is narrow: 2^-24 (with full precision 2^-14) to 2^16.  So every
// factor is brought into range by a power of two: a row by skey (its values are code * scale / skey, its rotated part divided
// by it too), a query column by qs; S = S' skey qs.  A row enters the result as its weight times skey, so what is rounded to
// fp16 is that product: t above is then the score in log2 units plus log2 skey, and the reference m follows the largest t.  A
// large row thus counts by its share of the result, and not at all where it has no weight.  The sum of the weights takes
// exp2(t - m) / skey in fp32; its common factor 2^m cancels in the result, and the log of the sum adds m again.
// What fp16's range costs: within a row, bits of what is below 2^-14 skey, that is 2^-29 of the largest value that skey
// covers (a code of 448, or the rotated part where that is larger), and all of what is below 2^-25 skey; between rows, bits of
// a weight times skey below 2^-21 of the largest, and all of one below 2^-32; within a query column, bits of what is below
// 2^-15 of its largest.
//
// Layout.  A unit is (item, group of N columns); units are cut into tiles, numbered in order, and every CTA takes
// an equal run of tiles; a unit that several CTAs share leaves partial results in the workspace, which
// combine_kernel joins in a fixed order.  One CTA per SM, 28 warps (the warpgroups trade registers, kRegs*):
//   warps 0-15   bring tiles into operand form.  A warp owns four keys of every tile: it copies their rows into the tile's
//                place (16-byte asynchronous copies) and widens fp8 codes there, so that no other warp has to be waited for;
//   warps 16-23  softmax and results; each of the two groups of four warps has half of the columns;
//   warp 24      issues the scores of every tile as soon as it is there;
//   warp 25      issues the results as soon as the weights are there, and zeroes what is not finite in rows that some of its
//                columns do not see (a weight of zero does not cancel it).
// Two tiles (64 x 576 in 16 bits, 72 KB each) and the queries (up to 72 KB) fill shared memory; the weights take the place
// of the tile's rotated part once the scores are done.
//
// N is 16, 32 or 64 (the smallest that holds the item's columns, 64 beyond): a product of 64 or 128 rows costs 39 to 64
// cycles from N = 16 to N = 64, so a call with few heads pays little for its empty columns, and more than 64 columns
// would leave no room for the second tile.
//
// What bounds it.  The producers' chain, not a unit of the SM: wait, copies, 1300 cycles until they land, reading, widening,
// 700 to 1100 until the stores are visible.  Measured, 608 tokens x 2048 fp8 rows: 16 heads 290 us (2.8 TB/s of rows), 32 heads
// 303 us, 64 heads 336 us (516 TFLOP/s), that is 4.3 to 5.1 thousand cycles a tile.  In this form a tile's copies, widening and
// operand reads move about 400 KB in shared memory, 3100 cycles at 128 B a cycle, against 2200 of products (N = 64).
// Taken back as slower, at 256 x 4 tokens of 64 heads (this form: 572 to 594 us; the tiles' number and form as given): one
// 128-key tile filled in parts by copy warps 671; rows gathered by the copy engine into a ring, one 64-key tile 862 (the
// engine takes 73 cycles a row and 80 for a gather of four, whatever their width); two tiles with copy warps of their own
// 668; the next tile's copies issued before (606) or within (663) the widening; two teams of producers on alternate tiles
// and both products issued by one warp 808; one warp for both products 639.  Where few columns leave room, staging the codes
// of the next tile gained nothing, and loading them to registers a tile ahead took 291 us at 16 heads, 377 at 32 and 624 at
// 64 (608 tokens, as above): what is in flight towards registers needs L1, which the tiles leave little of.
#include "latent.cuh"
#include "tc.cuh"

HS_CHECK_WORD

namespace hs {
namespace {

constexpr int kTile = 64;
constexpr int kProducerWarps = 16, kSoftmaxWarps = 8;
constexpr int kBufs = 2;  // tiles in shared memory
constexpr int kMmaWarp = kProducerWarps + kSoftmaxWarps;
constexpr int kThreads = (kMmaWarp + 4) * 32;
constexpr int kMaxCols = 64;
constexpr int kRegsLaunch = 72, kRegsProducer = 64, kRegsSoftmax = 96, kRegsMma = 56;
static_assert(kProducerWarps * kRegsProducer + kSoftmaxWarps * kRegsSoftmax + 4 * kRegsMma <=
                  kThreads / 32 * kRegsLaunch,
              "more registers than the launch has");
template <int kRegs>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }
constexpr int kSub = kTile * 128;    // bytes of a sub-tile: 64 keys x 64 values
constexpr int kTileBytes = 9 * kSub;  // of which the ninth holds the rotated parts, and later the weights
// In log2 units: where a new reference puts the largest score, and the most that a score may reach before it moves.
// fp16 weights are normal from 2^-14 to 2^16; bf16 weights have fp32's range, but so do the values that they multiply, and
// the sums of both are fp32 too: weights of up to 2^16 leave values of 2^90 room.
template <bool kF16>
struct Range {
  static constexpr float kTop = kF16 ? 7.f : 0.f, kLazy = kF16 ? 15.f : 16.f;
};
// skey of an fp8 row: 2^-112 .. 2^112, as the field of a float's exponent; at the ends, fp16 still holds all e4m3 codes of the
// smallest normal scale and all values below 2^128.  A row whose latents are all zero has no size: it gets at least 2^-60,
// small against the rows that have one, so that it does not draw the reference up, and large enough that its weight over
// skey stays in fp32's range beside rows of up to 2^40.
constexpr int kMinKey = 127 - 112, kMaxKey = 127 + 112, kZeroKey = 127 - 60;
// The sums of fp8 rows' weights are 2^-kSumShift of what they stand for: with skey over its whole range, they stay within fp32's.
constexpr int kSumShift = 14;
static_assert(254 - kSumShift - kMaxKey >= 1, "2^-kSumShift / skey is a normal number");

// Workspace: partial results [2 per CTA][kMaxCols][512], their log2 sums [2 per CTA][kMaxCols], run starts [CTA].
struct RunStart {
  int64_t total;        // tiles of the call
  int64_t begin;        // number of the run's first tile
  int32_t item, group;  // of that tile
  int32_t tile, tiles;  // its number in its unit, tiles of the unit
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
  int item, group, tile, tiles, keys, left;
  __device__ __forceinline__ void start(const AttendParams& p, const RunStart& r, int run) {
    item = r.item;
    group = r.group;
    tile = r.tile;
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

// What a list or a page table says of a key: loaded ahead of its use, so nothing here looks at the loaded value.
struct Entry {
  int value, in_page;
  bool there, counts;
  __device__ __forceinline__ void load(const AttendParams& p, const Cursor& cur, int key) {
    const int k = cur.tile * kTile + key;
    there = cur.left > 0 && k < cur.keys;
    counts = cur.group == 0;
    value = -1;
    in_page = 0;
    if (!there) return;
    if (p.paged) {
      const int page = k / p.page_size;
      in_page = k - page * p.page_size;
      if (HS_CHECK(cur.item < p.items && page < p.max_pages, kChkTablePage))
        value = __ldg(p.table + (int64_t)cur.item * p.max_pages + page);
    } else {
      if (HS_CHECK(cur.item < p.items && k < p.K, kChkTablePage)) value = __ldg(p.rows + (int64_t)cur.item * p.K + k);
    }
  }
  // The key's row, or -1; bad (a data error) is set when the entry is not a valid one.
  __device__ __forceinline__ int row(const AttendParams& p, bool& bad) const {
    const bool in = value >= 0 && value < (p.paged ? (int64_t)p.num_blocks : p.num_rows);
    bad |= there && counts && !in && (p.paged || value != -1);
    const int r = !in ? -1 : p.paged ? value * p.page_size + in_page : value;
    return HS_CHECK(r >= -1 && r < p.num_rows, kChkPoolRow) ? r : -1;
  }
};

template <int N>
struct Smem {
  static constexpr int kQ = kBufs * kTileBytes;
  static constexpr int kMisc = kQ + 9 * N * 128;
  // after the queries: barriers (128 B), scales of fp8 rows [tile][key][4], results' offsets [N] (64 bits), then floats:
  // references, factors, limits [N] each, joined values [4][N], query scales [3][N], key scales [tile][64]
  static constexpr int kScales = kMisc + 128;
  static constexpr int kOffsets = kScales + kBufs * kTile * 16;
  static constexpr int kRef = kOffsets + N * 8;
  static constexpr int kQScale = 7 * N, kKeyScale = 10 * N;
  static constexpr int kBytes = kRef + (10 * N + kBufs * kTile) * 4 + 1024;  // + alignment of the base
  static_assert(kBytes <= 232448, "shared memory");
};
enum Bar { kFull = 0, kEmpty = 2, kQFull = 4, kQEmpty = 5, kSFull = 6, kPReady = 8, kOFull = 10, kDrain, kBars = kDrain + 2 };
static_assert(kBars * 8 <= 128, "barriers");

template <int N>
constexpr int tmem_cols() { return N == 64 ? 512 : N == 32 ? 256 : 128; }

__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts4(uint32_t a, uint32_t x) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
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
// 16 bytes to shared memory, asynchronously; zeros when there is nothing to copy.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void sts(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// 4 e4m3 codes -> 4 fp16
__device__ __forceinline__ uint2 codes4(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2 bf16 times a power of two -> 2 fp16
__device__ __forceinline__ uint32_t bf16_to_half(uint32_t w, float f) {
  return pack_half(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
}
// 2 codes (as fp16) times a scale, rounded to bf16, times a power of two -> 2 fp16
__device__ __forceinline__ uint32_t scaled_half(uint32_t codes, float scale, float f) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&codes));
  return bf16_to_half(tc::pack_bf16(x.x * scale, x.y * scale), f);
}
// Largest magnitude of 8 bf16 (NaN is passed over).
__device__ __forceinline__ float max_bf16x8(uint4 v) {
  uint32_t a = v.x & 0x7FFF7FFFu, b = v.y & 0x7FFF7FFFu, c = v.z & 0x7FFF7FFFu, d = v.w & 0x7FFF7FFFu;
  asm("{\n\tmax.bf16x2 %0, %0, %1;\n\tmax.bf16x2 %2, %2, %3;\n\tmax.bf16x2 %0, %0, %2;\n\t}" : "+r"(a), "+r"(b), "+r"(c) : "r"(d));
  return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
}

__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool any_softmax(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// ---------------------------------------------------------------------------------------------------------
// Producers

// Query tile of a unit: N columns x 576, zero for columns past the item's; asynchronous copies, which the caller waits for.
template <int N>
__device__ __forceinline__ void copy_queries(const AttendParams& p, uint32_t q, int item, int group) {
  constexpr int kPer = kProducerWarps * 32 / N;  // threads of a column
  const int col = threadIdx.x / kPer, j0 = threadIdx.x % kPer;
  const int c = group * N + col;
  const int pos = p.P > 1 ? c / p.heads : 0, head = c - pos * p.heads;
  const int64_t tok = (int64_t)item * p.P + pos;
  const bool there = c < p.cols;
  const __nv_bfloat16* lat = there ? p.q_latent + tok * p.ql_tok + head * p.ql_head : p.q_latent;
  const __nv_bfloat16* rope = there ? p.q_rope + tok * p.qr_tok + head * p.qr_head : p.q_rope;
#pragma unroll 3
  for (int j = j0; j < 72; j += kPer)
    copy16(q + (j >> 3) * (N * 128) + col * 128 + (((j & 7) ^ (col & 7)) << 4), j < 64 ? lat + 8 * j : rope + 8 * (j - 64),
           there);
}

// The same in fp16 by plain loads: a column is divided by qs, a power of two (mostly 1) that brings it into
// fp16's range.
template <int N>
__device__ __forceinline__ void convert_queries(const AttendParams& p, uint32_t q, float* qs, int item, int group) {
  constexpr int kPer = kProducerWarps * 32 / N;  // threads of a column: neighbouring lanes
  const int col = threadIdx.x / kPer, j0 = threadIdx.x % kPer;
  const int c = group * N + col;
  const int pos = p.P > 1 ? c / p.heads : 0, head = c - pos * p.heads;
  const int64_t tok = (int64_t)item * p.P + pos;
  const bool there = c < p.cols;
  const __nv_bfloat16* lat = there ? p.q_latent + tok * p.ql_tok + head * p.ql_head : p.q_latent;
  const __nv_bfloat16* rope = there ? p.q_rope + tok * p.qr_tok + head * p.qr_head : p.q_rope;
  constexpr int kChunks = (72 + kPer - 1) / kPer;
  uint4 v[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int j = j0 + i * kPer;
    v[i] = make_uint4(0, 0, 0, 0);
    if (there && j < 72) v[i] = __ldg(reinterpret_cast<const uint4*>(j < 64 ? lat + 8 * j : rope + 8 * (j - 64)));
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) top = fmaxf(top, max_bf16x8(v[i]));
#pragma unroll
  for (int d = 1; d < kPer; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  // left as they are when their largest magnitude is in 2^-2 .. 2^15: fp16 then keeps all but what is 2^-23 of it
  const int b = (int)(__float_as_uint(top) >> 23);
  const int e = top == 0.f || (b >= 125 && b < 142) ? 127 : min(max(b - 14, 1), 240);
  const float f = __uint_as_float((uint32_t)(254 - e) << 23);
  if (j0 == 0) qs[col] = __uint_as_float((uint32_t)e << 23);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int j = j0 + i * kPer;
    if (j < 72)
      sts(q + (j >> 3) * (N * 128) + col * 128 + (((j & 7) ^ (col & 7)) << 4), bf16_to_half(v[i].x, f),
          bf16_to_half(v[i].y, f), bf16_to_half(v[i].z, f), bf16_to_half(v[i].w, f));
  }
}

// A warp owns four keys of every tile: it copies their rows, and widens fp8 codes in place (a part's codes land in the
// upper half of its place), with no other warp to wait for.
template <int N, bool kF16>
__device__ __forceinline__ void produce_tiles(const AttendParams& p, uint32_t base, float* qs, float* skey, uint32_t bars,
                                              Cursor cur, int groups, tc::Waiter& w) {
  using L = Smem<N>;
  constexpr int kRow = kF16 ? HS_ROW_BYTES_FP8 : HS_ROW_BYTES_BF16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane >> 3, j = lane & 7;  // copies: key 4 warp + sub, of each 128 bytes of its row the 16-byte piece j
  const int key = 4 * warp + sub, swz = key & 7;
  const int half = lane >> 4, q = lane & 15;  // widening: keys 4 warp + half and + 2, of each 128 codes the 8 at 8 q
  uint32_t to[2];  // where their 8 values go
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = 4 * warp + 2 * i + half;
    to[i] = (q >> 3) * kSub + k * 128 + (((q & 7) ^ (k & 7)) << 4);
  }
  auto signal = [&](int bar) {
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bars + 8 * bar);
  };
  bool fresh = true, bad = false;
  uint32_t seg = 0, it = 0;
  Entry entry;  // of key 4 warp + lane % 4
  entry.load(p, cur, 4 * warp + (lane & 3));
#pragma unroll 1
  while (cur.left > 0) {
    const uint32_t buf = it % kBufs, tile = base + buf * kTileBytes;
    const uint32_t scales = base + L::kScales + (buf * kTile + key) * 16;
    const int row = __shfl_sync(0xFFFFFFFFu, entry.row(p, bad), sub);
    const bool there = row >= 0;
    const uint8_t* src = p.base + (int64_t)max(row, 0) * kRow + 16 * j;
    if (it >= kBufs) w.wait(bars + 8 * (kEmpty + buf), (it / kBufs - 1) & 1);
    __syncwarp();
    // the rows, on their way into the tile: zeros for keys that have none
    if (kF16) {
      if (j == 0) copy16(scales, src + kLatent, there);
      copy16(tile + 8 * kSub + key * 128 + 16 * j, src + kRow - 128, there);
#pragma unroll
      for (int c = 0; c < 4; ++c) copy16(tile + (2 * c + 1) * kSub + key * 128 + 16 * j, src + 128 * c, there);
    } else {
#pragma unroll
      for (int c = 0; c < 9; ++c) copy16(tile + c * kSub + key * 128 + ((j ^ swz) << 4), src + 128 * c, there);
      if (j == 0) skey[buf * kTile + key] = there ? 1.f : 0.f;
    }
    if (fresh) {
      if (seg > 0) w.wait(bars + 8 * kQEmpty, (seg - 1) & 1);
      __syncwarp();
      if (kF16) {
        convert_queries<N>(p, base + L::kQ, qs + (seg % 3) * N, cur.item, cur.group);
      } else {
        copy_queries<N>(p, base + L::kQ, cur.item, cur.group);
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
      signal(kQFull);
      ++seg;
    }
    fresh = cur.next(p, groups);
    ++it;
    entry.load(p, cur, 4 * warp + (lane & 3));
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    if constexpr (kF16) {
      const uint32_t codes = tile + kSub + (4 * warp + half) * 128 + 8 * q;
      const uint4 rope = lds16(tile + 8 * kSub + key * 128 + 16 * j);
      float sc = lds_f(scales + 4 * (j & 3));  // lanes j and j + 4 of a key have its scale of group j
      // skey: 2^7 below the power of two that covers the largest scale (codes reach 448 * 2^7 < 65504), and so that the
      // rotated part stays below 2^15
      const uint32_t sb = __float_as_uint(sc) & 0x7FFFFFFFu;
      const bool exact = __all_sync(0xFFFFFFFFu, (sb & 0x7FFFFFu) == 0);  // every scale is a power of two
      const int from_scale = (int)(sb >> 23) + ((sb & 0x7FFFFFu) ? 1 : 0) - 7;
      const int from_rope = (int)(__float_as_uint(max_bf16x8(rope)) >> 23) + 1 - 15;
      uint32_t both = (uint32_t)from_scale << 16 | ((uint32_t)from_rope & 0xFFFFu);  // two maxima at once
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) both = __vmaxs2(both, __shfl_xor_sync(0xFFFFFFFFu, both, d));
      const int top_rope = (int16_t)both;
      int e = max((int)both >> 16, top_rope), least = kMinKey;
      // A group of zeros may have any scale, and has no size.  That is looked at only where a scale is far above the rotated
      // part, or the row is very small: elsewhere it costs the row's other values or the other rows 8 bits of the range.
      if (__any_sync(0xFFFFFFFFu, (int)both >> 16 > top_rope + 8 || e < kZeroKey)) {
        uint32_t set = 0;  // groups of the warp's keys that have values other than zero: bit 4 (key - 4 warp) + group
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint2 x = lds8(codes + 2 * c * kSub + 256 * i);
            if ((x.x | x.y) & 0x7F7F7F7Fu) set |= 1u << (8 * i + c);
          }
        set = __reduce_or_sync(0xFFFFFFFFu, set << (4 * half)) >> (4 * sub);
        const bool empty = !(set >> (j & 3) & 1);
        if (empty) sc = 0.f;
        e = empty ? 0 : from_scale;
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, d));
        e = max(e, top_rope);
        if (!(set & 15)) least = kZeroKey;
      }
      e = min(max(e, least), kMaxKey);
      uint2 v[4][2];  // (read here and not before: the registers are needed above)
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) v[c][i] = lds8(codes + 2 * c * kSub + 256 * i);
      const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
      const uint32_t ratio = pack_half(sc * inv, sc * inv);
      if (j == 0) skey[buf * kTile + key] = there ? __uint_as_float((uint32_t)e << 23) : 0.f;
      __syncwarp();  // the codes and the rotated parts are read before their places are written
      sts(tile + 8 * kSub + key * 128 + ((j ^ swz) << 4), bf16_to_half(rope.x, inv), bf16_to_half(rope.y, inv),
          bf16_to_half(rope.z, inv), bf16_to_half(rope.w, inv));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int from = (2 * i + half) * 8 + c;
          uint2 a = codes4(v[c][i].x), b = codes4(v[c][i].y);
          if (exact) {
            const uint32_t r = __shfl_sync(0xFFFFFFFFu, ratio, from);
            a.x = mul_half2(a.x, r), a.y = mul_half2(a.y, r), b.x = mul_half2(b.x, r), b.y = mul_half2(b.y, r);
          } else {
            const float z = __shfl_sync(0xFFFFFFFFu, sc, from), f = __shfl_sync(0xFFFFFFFFu, inv, from);
            a.x = scaled_half(a.x, z, f), a.y = scaled_half(a.y, z, f);
            b.x = scaled_half(b.x, z, f), b.y = scaled_half(b.y, z, f);
          }
          sts(tile + 2 * c * kSub + to[i], a.x, a.y, b.x, b.y);
        }
      }
    }
    signal(kFull + buf);
  }
  if (bad) report(p.status, p.paged ? HS_ERR_TABLE_RANGE : HS_ERR_ID_RANGE);
}

// ---------------------------------------------------------------------------------------------------------
// Products

// One warp issues the scores of every tile, another the results: each waits for one thing only, and a tile's scores are
// made while the softmax works on the tile before.  (A tile's place in tensor memory is free when its place in shared memory
// is: that is refilled after the results of the tile that had both.)
template <int N, bool kF16>
__device__ __forceinline__ void issue_scores(const AttendParams& p, uint32_t base, uint32_t bars, uint32_t tmem, Cursor cur,
                                             int groups, tc::Waiter& w) {
  constexpr uint32_t kIdS = tc::idesc(kF16, kTile, N, false, false);
  const uint64_t dk = tc::desc(base, 16, 1024, tc::kSwizzle128);  // tile as keys (K-major)
  const uint64_t dq = tc::desc(base + Smem<N>::kQ, 16, 1024, tc::kSwizzle128);
  const bool leader = tc::elect();
  bool fresh = true;
  uint32_t seg = 0;
#pragma unroll 1
  for (uint32_t it = 0; cur.left > 0; ++it) {
    const uint32_t buf = it % kBufs;
    if (fresh) w.wait(bars + 8 * kQFull, seg++ & 1);
    w.wait(bars + 8 * (kFull + buf), it / kBufs & 1);
    __syncwarp();
    tc::fence_after();
    const uint64_t a0 = dk + (uint32_t)(buf * kTileBytes >> 4);
    const uint32_t d = tmem + buf * N;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      tc::mma_ss(d, a0 + ((8 * kSub + k * 32) >> 4), dq + ((8 * N * 128 + k * 32) >> 4), kIdS, k > 0, leader);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      const uint64_t a = a0 + (uint32_t)(2 * c * kSub >> 4), b = dq + (uint32_t)(2 * c * (N * 128) >> 4);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        tc::mma_ss(d, a + (((k >> 2) * kSub + (k & 3) * 32) >> 4), b + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4), kIdS, true,
                   leader);
    }
    tc::commit(bars + 8 * (kSFull + buf), leader);
    fresh = cur.next(p, groups);
    if (fresh || cur.left == 0) tc::commit(bars + 8 * kQEmpty, leader);
  }
  // nothing of this CTA's products is in flight when the others leave
  tc::commit(bars + 8 * kDrain, leader);
  tc::Drain drain;
  drain.wait(bars + 8 * kDrain, 0);
  __syncwarp();
}

// Infinite and NaN values of the tile's keys from .. to - 1 become zeros (one warp): some columns do not see these keys, and
// a weight of zero would not cancel such a value.  Columns that see a NaN have it in their sums already, by its score.
template <bool kF16>
__device__ __forceinline__ void finite_values(uint32_t tile, int from, int to) {
  constexpr uint32_t kExponent = kF16 ? 0x7C00u : 0x7F80u;
#pragma unroll 1
  for (int i = from * 64 + (threadIdx.x & 31); i < to * 64; i += 32) {
    const uint32_t at = tile + (i & 7) * kSub + (i >> 6) * 128 + (i >> 3 & 7) * 16;  // 16 bytes of key i / 64
    const uint4 x = lds16(at);
    uint32_t w[4] = {x.x, x.y, x.z, x.w}, kept = ~0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t keep = ((w[k] & kExponent) == kExponent ? 0u : 0xFFFFu) |
                            ((w[k] >> 16 & kExponent) == kExponent ? 0u : 0xFFFF0000u);
      w[k] &= keep;
      kept &= keep;
    }
    if (~kept) sts(at, w[0], w[1], w[2], w[3]);
  }
  tc::fence_async_smem();
  __syncwarp();
}

template <int N, bool kF16>
__device__ __forceinline__ void issue_results(const AttendParams& p, uint32_t base, uint32_t bars, uint32_t tmem, Cursor cur,
                                              int groups, tc::Waiter& w) {
  constexpr uint32_t kIdO = tc::idesc(kF16, 128, N, true, true);
  constexpr uint64_t kPSwizzle = N == 64 ? tc::kSwizzle128 : N == 32 ? tc::kSwizzle64 : tc::kSwizzle32;
  const uint64_t dv = tc::desc(base, kSub, 1024, tc::kSwizzle128);  // tile as values (M-major)
  const uint64_t dp = tc::desc(base + 8 * kSub, 16, 8 * N * 2, kPSwizzle);
  const bool leader = tc::elect();
  bool first = true;
  int seen = INT32_MAX;  // keys that all of the group's columns see: what its first column does
#pragma unroll 1
  for (uint32_t it = 0; cur.left > 0; ++it) {
    const uint32_t buf = it % kBufs;
    if (first && p.paged && p.P > 1) seen = __ldg(p.ctx_len + cur.item) - p.P + 1 + cur.group * N / p.heads;
    w.wait(bars + 8 * (kPReady + buf), it / kBufs & 1);
    __syncwarp();
    if (cur.keys > seen) {
      const int from = max(0, seen - cur.tile * kTile), to = min(kTile, cur.keys - cur.tile * kTile);
      if (from < to) finite_values<kF16>(base + buf * kTileBytes, from, to);
    }
    tc::fence_after();
    const uint64_t a0 = dv + (uint32_t)(buf * kTileBytes >> 4), b = dp + (uint32_t)(buf * kTileBytes >> 4);
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
      const uint64_t a = a0 + (uint32_t)(2 * g * kSub >> 4);
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        tc::mma_ss(tmem + (2 + g) * N, a + (k * 2048 >> 4), b + ((k * 16 * N * 2) >> 4), kIdO, !first || k > 0, leader);
    }
    tc::commit(bars + 8 * (kEmpty + buf), leader);
    first = cur.next(p, groups);
    if (first || cur.left == 0) tc::commit(bars + 8 * kOFull, leader);
  }
  tc::commit(bars + 8 * (kDrain + 1), leader);
  tc::Drain drain;
  drain.wait(bars + 8 * (kDrain + 1), 0);
  __syncwarp();
}

// ---------------------------------------------------------------------------------------------------------
// Softmax and results

// Reduction over the eight lanes that have the same columns (lane % 4), of n values each.
template <int n, typename F>
__device__ __forceinline__ void over_keys(float* v, F f) {
#pragma unroll
  for (int d = 4; d < 32; d <<= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = f(v[i], __shfl_xor_sync(0xFFFFFFFFu, v[i], d));
}

template <int N, bool kF16>
__device__ __forceinline__ void softmax(const AttendParams& p, uint32_t base, uint32_t bars, uint32_t tmem, float* nref,
                                        int64_t* offsets, Cursor cur, int groups, int sms, tc::Waiter& w) {
  constexpr float kTop = Range<kF16>::kTop, kLazy = Range<kF16>::kLazy;
  constexpr int kW = N / 2, kBlocks = kW / 8;  // columns of this warp, in blocks of 8
  const int tid = threadIdx.x - kProducerWarps * 32;
  const int lane = tid & 31, warp = (tid >> 5) & 3;
  const int c0 = (tid >> 7) * kW;                                 // its first column
  // scores: keys key0 and key0 + 8, of each block the columns 2 (lane % 4) and the next
  const int key0 = 16 * warp + (lane >> 2);
  const int my = c0 + 2 * (lane & 3);
  const int dim = tid & 127;                                      // results: dimension of a block of 128
  const uint32_t tm = tmem + ((uint32_t)(32 * warp) << 16) + c0;  // its warp's lanes, its columns
  // nref: [N] the references, negated (+infinity: none yet)
  float* alpha = nref + N;                             // [N] rescale factors, then result factors
  int* limit = reinterpret_cast<int*>(nref + 2 * N);   // [N] keys that a column sees
  float* red = nref + 3 * N;                           // [4][N] the warps' maxima or sums
  const float* skey = nref + Smem<N>::kKeyScale;
  auto pair = [](const float* v) { return *reinterpret_cast<const float2*>(v); };
  auto leave = [&](const float2* v) {  // joined values of this warp's columns
    if (lane < 4) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) *reinterpret_cast<float2*>(red + warp * N + my + 8 * b) = v[b];
    }
  };
  bool fresh = true, at_start = false;
  bool first_run = true;  // this CTA's first segment
  bool scaled = false;    // some column of the unit has a qs other than 1
  uint32_t it = 0, seg = 0;
  float2 l[kBlocks];
#pragma unroll 1
  while (cur.left > 0) {
    const int item = cur.item, group = cur.group;
    const float* qs = nref + Smem<N>::kQScale + (seg % 3) * N;
    const uint32_t buf = it % kBufs, phase = it / kBufs & 1;
    if (fresh) {
      bar_softmax();  // every thread is done with the unit before
      at_start = cur.tile == 0;
      if (tid < N) {
        nref[tid] = INFINITY;
        const int c = min(group * N + tid, p.cols - 1);
        const int pos = p.P > 1 ? c / p.heads : 0;
        limit[tid] = p.paged ? __ldg(p.ctx_len + item) - p.P + 1 + pos : p.K;
        offsets[tid] = ((int64_t)item * p.P + pos) * p.out_tok + (c - pos * p.heads) * p.out_head;
      }
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) l[b] = make_float2(0.f, 0.f);
      bar_softmax();
    }
    const int k = cur.tile * kTile + key0;
    w.wait(bars + 8 * (kFull + buf), phase);  // makes skey and qs visible
    const float sk[2] = {skey[buf * kTile + key0], skey[buf * kTile + key0 + 8]};
    const bool there[2] = {sk[0] > 0.f, sk[1] > 0.f};
    // columns differ in what they see only in the last P - 1 keys
    const bool ragged = p.paged && p.P > 1 && (cur.tile + 1) * kTile > limit[0];
    const bool masks = !__all_sync(0xFFFFFFFFu, there[0] && there[1]) || ragged;
    const bool first = fresh;
    float mult[2], size[2];  // of a key: factor of its scores, log2 skey
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mult[i] = kF16 ? p.scale_log2 * sk[i] : p.scale_log2;
      size[i] = kF16 ? (float)((int)(__float_as_uint(sk[i]) >> 23) - 127) : 0.f;
    }
    if (kF16 && fresh) scaled = __any_sync(0xFFFFFFFFu, qs[c0 + lane % kW] != 1.f);
    w.wait(bars + 8 * (kSFull + buf), phase);
    __syncwarp();
    tc::fence_after();
    // this thread's scores in log2 units (plus log2 skey), less the references or not; -infinity where the key is hidden
    float2 s[kBlocks][2];
    auto scores = [&](bool relative) {
      float raw[4 * kBlocks];
      tc::tmem_ld_rows16<kBlocks>(tm + buf * N, raw);
      tc::tmem_wait_ld();
      tc::touch<4 * kBlocks>(raw);
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const float2 m = relative ? pair(nref + my + 8 * b) : make_float2(0.f, 0.f);
        const float2 z = kF16 && scaled ? pair(qs + my + 8 * b) : make_float2(1.f, 1.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 x = make_float2(raw[4 * b + 2 * i], raw[4 * b + 2 * i + 1]);
          float2 f = make_float2(mult[i], mult[i]);
          if (kF16 && scaled) f = tc::mul2(f, z);
          s[b][i] = tc::fma2(x, f, kF16 ? tc::add2(m, make_float2(size[i], size[i])) : m);
        }
      }
      if (masks) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!there[i] || (ragged && k + 8 * i >= limit[my + 8 * b])) s[b][i].x = -INFINITY;
            if (!there[i] || (ragged && k + 8 * i >= limit[my + 8 * b + 1])) s[b][i].y = -INFINITY;
          }
      }
    };
    // twice at most: with the references as they are, and again if one had to move
    bool moved = false;
#pragma unroll 1
    while (true) {
      scores(true);
      const float top = tc::max_of<4 * kBlocks>(&s[0][0].x);
      if (moved || !any_softmax(top > kLazy)) break;
      moved = true;
      // a new reference for every column, kTop below the maximum of the old one's and this tile's scores
      scores(false);
      float2 m[kBlocks];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) m[b] = make_float2(fmaxf(s[b][0].x, s[b][1].x), fmaxf(s[b][0].y, s[b][1].y));
      over_keys<2 * kBlocks>(&m[0].x, [](float a, float b) { return fmaxf(a, b); });
      leave(m);
      bar_softmax();
      if (tid < N) {
        const float old = -nref[tid];
        const float now = fmaxf(fmaxf(fmaxf(red[tid], red[N + tid]), fmaxf(red[2 * N + tid], red[3 * N + tid])) - kTop, old);
        nref[tid] = -now;
        alpha[tid] = old == -INFINITY ? 0.f : exp2f(old - now);
      }
      bar_softmax();
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) l[b] = tc::mul2(l[b], pair(alpha + my + 8 * b));
      if (!first) {
        // once the products of the tiles before have finished
        w.wait(bars + 8 * (kEmpty + (it - 1) % kBufs), (it - 1) / kBufs & 1);
        __syncwarp();
        tc::fence_after();
#pragma unroll 1
        for (int c = 0; c < 4 * kW; c += 8) {
          const int g = c / kW, x0 = c % kW;
          float o[8];
          tc::tmem_ld<8>(tm + (2 + g) * N + x0, o);
          tc::tmem_wait_ld();
          tc::touch<8>(o);
#pragma unroll
          for (int x = 0; x < 8; ++x) o[x] *= alpha[c0 + x0 + x];
          tc::tmem_st8(tm + (2 + g) * N + x0, o);
        }
        tc::tmem_wait_st();
      }
    }
    // weights, their sums per thread, and P^T: [key][column], 2 N bytes a key, swizzled like the descriptor says
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = key0 + 8 * i;
      // 2^-kSumShift / skey (a key that is not there has no weight)
      const float inv = __uint_as_float((uint32_t)(254 - kSumShift - (int)(__float_as_uint(sk[i]) >> 23)) << 23);
      const uint32_t to = base + buf * kTileBytes + 8 * kSub + key * (2 * N) + 4 * (lane & 3);
      const int sw = N == 64 ? (key & 7) : N == 32 ? ((key >> 1) & 3) : ((key >> 2) & 1);
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const float2 e = make_float2(tc::exp2_fast(s[b][i].x), tc::exp2_fast(s[b][i].y));
        l[b] = kF16 ? tc::fma2(e, make_float2(inv, inv), l[b]) : tc::add2(l[b], e);
        const uint32_t two = kF16 ? pack_half(e.x, e.y) : tc::pack_bf16(e.x, e.y);
        sts4(to + (((c0 / 8 + b) ^ sw) << 4), two);
      }
    }
    tc::fence_async_smem();
    tc::fence_before();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bars + 8 * (kPReady + buf));

    const int unit_tiles = cur.tiles, tile = cur.tile;
    fresh = cur.next(p, groups);
    ++it;
    if (!fresh && cur.left > 0) continue;

    // the segment ends: join the sums, then the results
    const bool whole = at_start && tile + 1 == unit_tiles;
    const int ncols = min(N, p.cols - group * N);
    over_keys<2 * kBlocks>(&l[0].x, [](float a, float b) { return a + b; });
    leave(l);
    bar_softmax();
    const int part = 2 * blockIdx.x + (first_run && !at_start ? 0 : 1);
    first_run = false;
    const bool in_place = HS_CHECK(item < p.items && group * N < p.cols && part < 2 * sms, kChkOutPos);
    if (tid < N) {
      const float sum = (red[tid] + red[N + tid]) + (red[2 * N + tid] + red[3 * N + tid]);
      const float lse2 = sum == 0.f ? -INFINITY : log2f(sum) - nref[tid] + (kF16 ? kSumShift : 0);
      alpha[tid] = sum == 0.f ? 0.f : (kF16 ? 1.f / (1 << kSumShift) : 1.f) / sum;
      if (!whole) {
        float* z = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.workspace) + ws_lse_offset(sms));
        if (in_place) z[part * kMaxCols + tid] = lse2;
      } else if (p.lse && tid < ncols && in_place) {
        p.lse[(int64_t)item * p.cols + group * N + tid] = lse2 * kLn2;
      }
    }
    bar_softmax();
    w.wait(bars + 8 * kOFull, seg & 1);
    __syncwarp();
    ++seg;
    tc::fence_after();
    const bool odd = lane & 1;
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
      float o[kW];
      tc::tmem_ld<kW>(tm + (2 + g) * N, o);
      tc::tmem_wait_ld();
      tc::touch<kW>(o);
#pragma unroll
      for (int c = 0; c < kW; c += 4) {
        const float4 f = *reinterpret_cast<const float4*>(alpha + c0 + c);
        o[c] *= f.x, o[c + 1] *= f.y, o[c + 2] *= f.z, o[c + 3] *= f.w;
      }
      if (!whole) {
        float* z = p.workspace + ((int64_t)part * kMaxCols + c0) * kLatent + 128 * g + dim;
#pragma unroll
        for (int c = 0; c < kW; ++c)
          if (in_place) z[c * kLatent] = o[c];
      } else {
        // pairs of lanes exchange so that each writes two neighbouring dimensions of one column
        __nv_bfloat16* dst = p.out + 128 * g + (dim - odd);
#pragma unroll
        for (int c = 0; c < kW; c += 2) {
          const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? o[c] : o[c + 1], 1);
          const uint32_t two = odd ? tc::pack_bf16(got, o[c + 1]) : tc::pack_bf16(o[c], got);
          if (c0 + c + odd < ncols && in_place) *reinterpret_cast<uint32_t*>(dst + offsets[c0 + c + odd]) = two;
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

// total * b / ctas (ctas is a few hundred, and a 64-bit division some hundred instructions)
__device__ __forceinline__ int64_t run_begin(int64_t total, int ctas, int b) {
  const int64_t q = total >> 32 ? total / ctas : (int64_t)((uint32_t)total / (uint32_t)ctas);
  return q * b + (int)(total - q * ctas) * b / ctas;
}

template <int N, int kRowBytes>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const AttendParams p, int groups, int sms) {
  constexpr bool kF16 = kRowBytes == HS_ROW_BYTES_FP8;
  using L = Smem<N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~uintptr_t(1023));
  __shared__ RunStart start;
  __shared__ uint32_t tmem_slot;
  __shared__ int64_t scratch[kThreads / 32];
  const int warp = threadIdx.x >> 5;
  const uint32_t base = tc::smem_u32(smem);
  const uint32_t bars = base + L::kMisc;
  float* nref = reinterpret_cast<float*>(smem + L::kRef);
  int64_t* offsets = reinterpret_cast<int64_t*>(smem + L::kOffsets);

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
        const int item = begin >> 32 ? (int)(begin / per_item) : (int)((uint32_t)begin / (uint32_t)per_item);
        const int off = (int)(begin - (int64_t)item * per_item);
        start = RunStart{total, begin, item, off / tiles, off % tiles, tiles};
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
        if (begin >= at && begin < at + (int64_t)tiles * groups) {
          const int off = (int)(begin - at);
          start = RunStart{total, begin, i, off / tiles, off % tiles, tiles};
        }
        passed += all;
        if (begin < passed) break;
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;");  // combine_kernel waits for this kernel's results by itself
  if ((int)blockIdx.x >= ctas) return;

  if (threadIdx.x == 0) {
    for (int c = 0; c < kBufs; ++c) {
      tc::mbar_init(bars + 8 * (kFull + c), kProducerWarps);
      tc::mbar_init(bars + 8 * (kEmpty + c), 1);
      tc::mbar_init(bars + 8 * (kSFull + c), 1);
      tc::mbar_init(bars + 8 * (kPReady + c), kSoftmaxWarps);
    }
    tc::mbar_init(bars + 8 * kQFull, kProducerWarps);
    tc::mbar_init(bars + 8 * kQEmpty, 1);
    tc::mbar_init(bars + 8 * kOFull, 1);
    tc::mbar_init(bars + 8 * kDrain, 1);
    tc::mbar_init(bars + 8 * (kDrain + 1), 1);
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
  cur.start(p, start, (int)run);
  tc::Waiter w;
  if (warp < kProducerWarps) {
    fewer_registers<kRegsProducer>();
    produce_tiles<N, kF16>(p, base, nref + L::kQScale, nref + L::kKeyScale, bars, cur, groups, w);
  } else if (warp < kMmaWarp) {
    more_registers<kRegsSoftmax>();
    softmax<N, kF16>(p, base, bars, tmem, nref, offsets, cur, groups, sms, w);
  } else {
    fewer_registers<kRegsMma>();
    if (warp == kMmaWarp)
      issue_scores<N, kF16>(p, base, bars, tmem, cur, groups, w);
    else if (warp == kMmaWarp + 1)
      issue_results<N, kF16>(p, base, bars, tmem, cur, groups, w);
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
// weighted by exp2 of their log2 sums, in the order of the runs.  128 threads a column, with 4 dimensions each.  Bound: the
// latency of its few dependent loads.  Two columns a block: with four, 32 bf16 contexts of 128 heads take 72 us instead of 70.
constexpr int kJoinCols = 2;
__global__ void __launch_bounds__(128 * kJoinCols) combine_kernel(const AttendParams p, int groups, int n, int sms, int grid) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for attend_kernel's results
  const uint8_t* ws = reinterpret_cast<const uint8_t*>(p.workspace);
  const RunStart* runs = reinterpret_cast<const RunStart*>(ws + ws_run_offset(sms));
  const float* lse = reinterpret_cast<const float*>(ws + ws_lse_offset(sms));
  const int b = blockIdx.x + 1;
  const int64_t total = runs[0].total;
  const int ctas = (int)min((int64_t)grid, total);
  if (b >= ctas) return;
  const RunStart r = runs[b];
  const int64_t before = runs[b - 1].begin;
  const int group = r.group;
  if (r.tile == 0) return;
  const int64_t unit0 = r.begin - r.tile, unit1 = unit0 + r.tiles;
  if (before > unit0) return;  // an earlier boundary cuts this unit
  // runs b - 1 .. last hold parts of it
  const int next = b + 1 + threadIdx.x;
  const int last = b + __syncthreads_count(next < ctas && runs[next].begin < unit1);
  const int c = blockIdx.y * kJoinCols + threadIdx.x / 128, d = threadIdx.x % 128;
  if (c >= min(n, p.cols - group * n)) return;
  if (!HS_CHECK(r.item >= 0 && r.item < p.items && 2 * last < 2 * sms, kChkOutPos)) return;
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = b - 1; i0 <= last; i0 += 4) {  // four parts at a time
    float z[4];
    float4 v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = i0 + x, slot = 2 * i + (i < b);
      z[x] = -INFINITY;
      v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i <= last) {
        z[x] = lse[slot * kMaxCols + c];
        v[x] = reinterpret_cast<const float4*>(p.workspace + ((int64_t)slot * kMaxCols + c) * kLatent)[d];
      }
    }
    const float now = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), top);
    const float old = top == -INFINITY ? 0.f : exp2f(top - now);
    sum *= old, acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float f = z[x] == -INFINITY ? 0.f : exp2f(z[x] - now);
      sum += f;
      acc.x += f * v[x].x, acc.y += f * v[x].y, acc.z += f * v[x].z, acc.w += f * v[x].w;
    }
    top = now;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int gc = group * n + c;
  const int pos = gc / p.heads, head = gc - pos * p.heads;
  __nv_bfloat16* dst = p.out + ((int64_t)r.item * p.P + pos) * p.out_tok + head * p.out_head + 4 * d;
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(tc::pack_bf16(acc.x * inv, acc.y * inv), tc::pack_bf16(acc.z * inv, acc.w * inv));
  if (d == 0 && p.lse) p.lse[(int64_t)r.item * p.cols + gc] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <int N, int kRowBytes>
cudaError_t launch(const AttendParams& p, int dev, int sms, cudaStream_t s) {
  static DeviceOnce once;
  const cudaError_t ready = once.ready(dev, [] {
    cudaFuncAttributes a{};
    cudaError_t e = cudaFuncGetAttributes(&a, attend_kernel<N, kRowBytes>);
    // the register trade waits for ever if the launch has fewer than it hands out
    if (e == cudaSuccess && a.numRegs != kRegsLaunch) e = cudaErrorInvalidKernelImage;
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(attend_kernel<N, kRowBytes>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<N>::kBytes);
    return e;
  });
  if (ready != cudaSuccess) return ready;
  const int groups = (p.cols + N - 1) / N;
  // a rows call knows its tiles; a pages call learns them on the device
  int grid = min(sms, 128 * kJoinCols);  // (a thread of combine_kernel for each)
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
  // its launch overlaps the end of the kernel before
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid - 1, N / kJoinCols);
  c.blockDim = dim3(128 * kJoinCols);
  c.stream = s;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &early;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, combine_kernel, p, groups, N, sms, grid);
  count_launch();
  return e;
}

template <int kRowBytes>
cudaError_t launch_cols(const AttendParams& p, int dev, int sms, cudaStream_t s) {
  if (p.cols <= 16) return launch<16, kRowBytes>(p, dev, sms, s);
  if (p.cols <= 32) return launch<32, kRowBytes>(p, dev, sms, s);
  return launch<64, kRowBytes>(p, dev, sms, s);
}

}  // namespace

uint32_t check_take_attend() {
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

size_t attend_workspace_bytes(int sms) { return ws_run_offset(sms) + (size_t)sms * sizeof(RunStart); }

cudaError_t launch_attend(const AttendParams& p, int dev, int sms, cudaStream_t s) {
  return p.row_bytes == HS_ROW_BYTES_FP8 ? launch_cols<HS_ROW_BYTES_FP8>(p, dev, sms, s)
                                         : launch_cols<HS_ROW_BYTES_BF16>(p, dev, sms, s);
}

}  // namespace hs
