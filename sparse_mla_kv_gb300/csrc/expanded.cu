// Attention over keys and values expanded to every head, on the tensor cores: prompts and prompt chunks.
//
// Mathematics.  A query row keeps a reference m, a sum l and an accumulator O over the key tiles:
//   S = Q K^T (192 = 128 of the head + 64 of the shared rotated part), P = exp2(S scale - m), l += sum P, O += P V.
// The reference is lazy: it starts as the first tile's maximum and moves (with l and O rescaled) only when a score exceeds
// it by kLazy.  bf16 weights have fp32's range, so nothing is lost at the low end, and 2^kLazy leaves values of up to 2^90
// room in the fp32 sums.  The weights are bf16 because the values are and both operands of a product have one type: root mean
// square error 2.1e-3 to 2.3e-3 of the results', against 1.6e-3 to 1.7e-3 with 32 bits and one rounding.  The rotated part of
// the keys is read where it is, once for each head, and never copied to every head.
//
// Layout.  A work item is (sequence, head, 256 queries): two tiles of 128 queries over the same key tiles of 128, so that
// a key or value loaded serves 256 queries (81 KB a key tile; one query tile alone would need 64 B a cycle from L2).
// 12 warps, one CTA per SM, items taken in a fixed stride:
//   warps 0-3, 4-7   softmax and results of query tile 0 and 1, a row a thread;
//   warps 8, 9       issue the products of query tile 0 and 1, so that neither waits for the other's softmax, and zero
//                    value rows past a sequence's end before their product (a weight of zero does not cancel a NaN there);
//   warp 10          loads by the copy engine;
//   warp 11          clears the results of query tokens that no sequence has.
// Shared memory: 96 KB of queries and a ring of eight 16 KB units (128 keys x 64 dimensions); a key tile is three units
// of keys, then two of values.  Tensor memory: S and O of both tiles, 4 x 128 columns; P, in bf16, takes S's place and is
// the left operand of the second product from there.
// Bound: the tensor pipe, 12 x 64 + 8 x 64 cycles for 128 queries x 128 keys.  Measured: 16384 causal tokens x 8 heads
// 489 us, 1.40 PFLOP/s (0.73 of a measured library product), about 4.3 thousand cycles for a pair of such tiles, the items'
// ends included, against 2.6 of products.  What is left is each query tile's own chain (scores, their weights, results,
// scores of the next key tile into the same place): tensor memory holds no second S.  Results begun when half of the weights
// are there took 511 us (the two tiles' products then interleave in smaller pieces), one warp issuing for both query tiles
// 522 us, and two threads a row 897 us (16 softmax warps leave each thread too few registers for its half of a row).  A
// called function in the softmax's loop takes the traded registers away: 530 us.
#include "latent.cuh"
#include "tc.cuh"

HS_CHECK_WORD

namespace hs {
namespace {

constexpr int kQRows = 128, kKeys = 128, kBlock = 2 * kQRows;
constexpr int kUnit = kKeys * 128;  // bytes of a unit
constexpr int kRing = 8, kUnitsK = 3, kUnitsV = 2, kUnits = kUnitsK + kUnitsV;
constexpr int kThreads = 12 * 32, kMmaWarp = 8, kLoadWarp = kMmaWarp + 2;
constexpr int kSmemBytes = 6 * kUnit + kRing * kUnit + 512 + 1024;
// the warpgroups trade registers
constexpr int kRegsLaunch = 168, kRegsSoftmax = 208, kRegsOther = 88;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * kRegsLaunch, "more registers than the launch has");
constexpr float kLazy = 16.f;
// The units of a key tile's keys arrive on one barrier, those of its values on another; a ring of eight units holds parts
// of at most four such groups.  Units are released one by one.
constexpr int kGroups = 4;
enum Bar { kFull = 0, kEmpty = kGroups, kQFull = kEmpty + kRing, kQEmpty, kSFull, kPReady = kSFull + 2, kODone = kPReady + 2,
           kDrain = kODone + 2, kBars = kDrain + 2 };
static_assert(kBars * 8 <= 512, "barriers");

struct Maps {
  CUtensorMap q_nope, q_rope, k_nope, k_rope, v;
  int32_t head_step[4];  // of q_nope, q_rope, k_nope, v: 0 where all heads read one
};

// One work item: rows [q0, q0 + rows) of the query tensors, keys [k0, k0 + keys).
struct Item {
  int head, q0, rows, k0, keys;
  int shift;  // query row r (counted from q0) sees the keys below r + shift (keys, where not causal)
  int tiles[2];  // key tiles of each query tile; -1: no such query tile
  bool causal;
  // keys that every row of query tile t sees: those below this one
  __device__ __forceinline__ int all_see(int t) const { return causal ? min(keys, t * kQRows + shift) : keys; }
  __device__ __forceinline__ int query_tiles() const { return rows > kQRows ? 2 : 1; }
  __device__ __forceinline__ int most() const { return max(tiles[0], tiles[1]); }
};

// Sequence s: its rows, or nothing where its offsets are not ascending within the tensors.
__device__ __forceinline__ bool sequence(const hs_expanded& a, int s, int* q0, int* q1, int* k0, int* k1) {
  *q0 = __ldg(a.cu_q + s), *q1 = __ldg(a.cu_q + s + 1), *k0 = __ldg(a.cu_k + s), *k1 = __ldg(a.cu_k + s + 1);
  return *q0 >= 0 && *q1 >= *q0 && *q1 <= a.q_tokens && *k0 >= 0 && *k1 >= *k0 && *k1 <= a.k_tokens;
}

// Hands a warp the work items by number, in ascending order.  Items are numbered by level, from the highest: a sequence of
// b blocks has one block (of each head) on each of the levels b - 1 .. 0, and with causal masks the block of a level is
// the longer the higher the level, so that long items come first whatever the mix of sequences.
struct Finder {
  int level, on_level;  // the current level and the sequences on it
  int64_t before;       // blocks on higher levels

  static __device__ __forceinline__ int blocks_of(const hs_expanded& a, int s, int* q0, int* q1, int* k0, int* k1) {
    return s < a.seqs && sequence(a, s, q0, q1, k0, k1) ? (*q1 - *q0 + kBlock - 1) / kBlock : 0;
  }
  __device__ __forceinline__ void start(const hs_expanded& a) {
    int most = 0, q0, q1, k0, k1;
    for (int s = threadIdx.x & 31; s < a.seqs; s += 32) most = max(most, blocks_of(a, s, &q0, &q1, &k0, &k1));
    level = __reduce_max_sync(0xFFFFFFFFu, most);
    on_level = 0;
    before = 0;
  }
  // Item number n, not below the last one asked for; false when there is none.
  __device__ __forceinline__ bool find(const hs_expanded& a, int64_t n, Item* it) {
    const int lane = threadIdx.x & 31;
    const int64_t block = n / a.heads;
    int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    while (block >= before + on_level) {
      before += on_level;
      if (--level < 0) return false;
      int c = 0;
      for (int s = lane; s < a.seqs; s += 32) c += blocks_of(a, s, &q0, &q1, &k0, &k1) > level;
      on_level = __reduce_add_sync(0xFFFFFFFFu, c);
    }
    int skip = (int)(block - before);  // the sequence wanted: this many on the level come before it
    for (int s0 = 0;; s0 += 32) {
      const bool here = blocks_of(a, s0 + lane, &q0, &q1, &k0, &k1) > level;
      const unsigned has = __ballot_sync(0xFFFFFFFFu, here);
      if (skip >= __popc(has)) {
        skip -= __popc(has);
        continue;
      }
      const int who = __fns(has, 0, skip + 1);
      q0 = __shfl_sync(0xFFFFFFFFu, q0, who), q1 = __shfl_sync(0xFFFFFFFFu, q1, who);
      k0 = __shfl_sync(0xFFFFFFFFu, k0, who), k1 = __shfl_sync(0xFFFFFFFFu, k1, who);
      break;
    }
    const int first = level * kBlock;
    it->head = (int)(n - block * a.heads);
    it->q0 = q0 + first;
    it->rows = min(kBlock, q1 - q0 - first);
    it->k0 = k0;
    it->keys = k1 - k0;
    it->causal = a.causal != 0;
    it->shift = a.causal ? first + 1 + (k1 - k0) - (q1 - q0) : 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int last = min(it->rows, (t + 1) * kQRows) - 1;  // the tile's last row sees most
      const int sees = a.causal ? min(it->keys, last + it->shift) : it->keys;
      it->tiles[t] = last < t * kQRows ? -1 : max(0, (sees + kKeys - 1) / kKeys);
    }
    return true;
  }
};

// This CTA's k-th item: passes over the grid in alternating directions, so that who had a long block first has a short one
// of the next pass.
__device__ __forceinline__ int64_t item_number(int k) {
  return (int64_t)k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

__device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// ---- loads (one lane) ----
// Bytes are announced only on a barrier whose phase before is complete.  In order that is so already (a part's barrier had its
// last use four parts ago, and units of later parts have been released since); the waits for it matter when another warp's
// wait gave up, which releases units early.  After a wait that gave up nothing more is announced.
struct Loader {
  tc::Waiter w;
  uint32_t u = 0, items = 0, parts = 0;  // units, items, parts (keys or values of a key tile) so far

  // One item's queries, keys and values; false after a wait that gave up.
  __device__ __forceinline__ bool load(const Maps& m, const Item& it, uint32_t q, uint32_t ring, uint32_t bars, bool leader) {
    if (items > 0) {
      w.wait(bars + 8 * kQEmpty, (items - 1) & 1);
      w.wait(bars + 8 * kQFull, (items - 1) & 1);
    }
    if (__any_sync(0xFFFFFFFFu, w.dead)) return false;
    ++items;
    const int hq = it.head * m.head_step[0], hr = it.head * m.head_step[1], hk = it.head * m.head_step[2],
              hv = it.head * m.head_step[3];
    if (leader) {
      tc::mbar_expect(bars + 8 * kQFull, it.query_tiles() * 3 * kUnit);
      for (int t = 0; t < it.query_tiles(); ++t) {
        const uint32_t to = q + t * 3 * kUnit;
        const int row = it.q0 + t * kQRows;
        load3(to, &m.q_nope, 0, hq, row, bars + 8 * kQFull);
        load3(to + kUnit, &m.q_nope, 64, hq, row, bars + 8 * kQFull);
        load3(to + 2 * kUnit, &m.q_rope, 0, hr, row, bars + 8 * kQFull);
      }
    }
    const int tiles = it.most();
#pragma unroll 1
    for (int j = 0; j < tiles; ++j) {
      const int row = it.k0 + j * kKeys;
#pragma unroll 1
      for (int i = 0; i < kUnits; ++i, ++u) {
        const uint32_t slot = u % kRing;
        if (u >= kRing) w.wait(bars + 8 * (kEmpty + slot), (u / kRing - 1) & 1);
        const bool begins = i == 0 || i == kUnitsK;
        if (begins) {
          if (parts >= kGroups) w.wait(bars + 8 * (kFull + parts % kGroups), (parts / kGroups - 1) & 1);
          if (__any_sync(0xFFFFFFFFu, w.dead)) return false;
          ++parts;
        }
        __syncwarp();
        if (leader) {
          const uint32_t bar = bars + 8 * (kFull + (parts - 1) % kGroups), to = ring + slot * kUnit;
          if (begins) tc::mbar_expect(bar, (i == 0 ? kUnitsK : kUnitsV) * kUnit);
          if (i < 2)
            load3(to, &m.k_nope, 64 * i, hk, row, bar);
          else if (i == 2)
            load3(to, &m.k_rope, 0, 0, row, bar);
          else
            load3(to, &m.v, 64 * (i - 3), hv, row, bar);
        }
      }
    }
    return true;
  }
};

__device__ __forceinline__ void load_items(const hs_expanded& a, const Maps& m, uint32_t q, uint32_t ring, uint32_t bars) {
  const bool leader = tc::elect();
  Loader l;
  Item it;
  Finder f;
  f.start(a);
  for (int k = 0; f.find(a, item_number(k), &it); ++k)
    if (it.most() > 0 && !l.load(m, it, q, ring, bars, leader)) break;
  // no copy is in flight when the CTA ends
  tc::Drain drain;
  for (uint32_t r = l.parts > kGroups ? l.parts - kGroups : 0; r < l.parts; ++r)
    drain.wait(bars + 8 * (kFull + r % kGroups), (r / kGroups) & 1);
  if (l.items > 0) drain.wait(bars + 8 * kQFull, (l.items - 1) & 1);
  if (l.w.dead) report(a.status, HS_ERR_TIMEOUT);
}

// ---- products (one warp a query tile) ----
// Both warps wait for every part of a key tile and release it, whether their query tile needs it or not.
__device__ __forceinline__ void issue_items(const hs_expanded& a, int t, uint32_t q, uint32_t ring, uint32_t bars,
                                            uint32_t tmem, volatile int* done) {
  constexpr uint32_t kIdS = tc::idesc(false, 128, kKeys, false, false);
  constexpr uint32_t kIdO = tc::idesc(false, 128, 64, false, true);
  tc::Waiter w;
  const bool leader = tc::elect();
  const uint64_t dq = tc::desc(q + t * 3 * kUnit, 16, 1024, tc::kSwizzle128);
  const uint64_t dk = tc::desc(ring, 16, 1024, tc::kSwizzle128);
  const uint64_t dv = tc::desc(ring, 16, 1024, tc::kSwizzle128);  // dimensions contiguous, 64 of them: one atom wide
  auto await = [&](int bar, uint32_t parity) {
    w.wait(bars + 8 * bar, parity);
    __syncwarp();
    tc::fence_after();
  };
  uint32_t base = 0, count = 0, group = 0;  // units, items and parts (keys or values of a key tile) so far
  uint32_t phase = 0;                       // key tiles done by the query tile
  Item it;
  Finder f;
  f.start(a);
  for (int k = 0; f.find(a, item_number(k), &it); ++k) {
    const int tiles = it.most(), mine = max(0, it.tiles[t]), whole = it.all_see(t);
    if (tiles <= 0) continue;
    auto arrived = [&]() {  // waits for the next part
      await(kFull + group % kGroups, (group / kGroups) & 1);
      ++group;
    };
    auto release = [&](int j, int from, int to) {  // units of key tile j, when all products so far have read them
      for (int i = from; i < to; ++i) tc::commit(bars + 8 * (kEmpty + (base + j * kUnits + i) % kRing), leader);
    };
    auto scores = [&](int j) {
      arrived();
#pragma unroll 1
      for (int i = 0; i < kUnitsK; ++i) {
        const uint32_t x = base + j * kUnits + i;
        const uint64_t da = dq + (uint32_t)(i * kUnit >> 4), db = dk + (uint32_t)((x % kRing) * kUnit >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) tc::mma_ss(tmem + t * 128, da + (k * 32 >> 4), db + (k * 32 >> 4), kIdS, i > 0 || k > 0, leader);
      }
      tc::commit(bars + 8 * (kSFull + t), leader);
      release(j, 0, kUnitsK);
      if (j + 1 == mine) tc::commit(bars + 8 * kQEmpty, leader);
    };
    await(kQFull, count & 1);
    ++count;
    if (mine > 0) {
      if (phase > 0) await(kODone + t, (phase - 1) & 1);  // the item before: its last P has been read
      scores(0);
    } else {
      tc::commit(bars + 8 * kQEmpty, leader);
    }
#pragma unroll 1
    for (int j = 0; j < mine; ++j, ++phase) {
      await(kPReady + t, phase & 1);
      arrived();
      const int valid = it.keys - j * kKeys;
      bool skip = false;  // this tile's results are in O already
      if ((j + 1) * kKeys > whole && done[t]) {
        skip = true;
        __syncwarp();
        done[t] = 0;
        __syncwarp();
      }
#pragma unroll 1
      for (int i = 0; i < kUnitsV && !skip; ++i) {
        const uint32_t x = base + j * kUnits + kUnitsK + i;
        if (valid < kKeys) {  // by both warps: they write the same
          for (int k = threadIdx.x & 31; k < (kKeys - valid) * 8; k += 32) {
            const uint32_t at = ring + (x % kRing) * kUnit + (valid + (k >> 3)) * 128 + (k & 7) * 16;
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0u) : "memory");
          }
          tc::fence_async_smem();
          __syncwarp();
        }
        const uint64_t db = dv + (uint32_t)((x % kRing) * kUnit >> 4);
        // P: 16 keys are 8 columns
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          tc::mma_ts(tmem + 256 + t * 128 + i * 64, tmem + t * 128 + k * 8, db + (k * 2048 >> 4), kIdO, j > 0 || k > 0, leader);
      }
      tc::commit(bars + 8 * (kODone + t), leader);
      release(j, kUnitsK, kUnits);
      if (j + 1 < mine) {
        await(kODone + t, phase & 1);  // P, in S's place, has been read
        scores(j + 1);
      }
    }
#pragma unroll 1
    for (int j = mine; j < tiles; ++j) {  // what only the other query tile reads
      arrived();
      release(j, 0, kUnitsK);
      arrived();
      release(j, kUnitsK, kUnits);
    }
    base += tiles * kUnits;
  }
  tc::commit(bars + 8 * (kDrain + t), leader);
  tc::Drain drain;
  drain.wait(bars + 8 * (kDrain + t), 0);
  __syncwarp();
  if (w.dead) report(a.status, HS_ERR_TIMEOUT);
}

// ---- softmax and results (128 threads a query tile) ----

// A value that is infinite or NaN must not reach the queries that the causal mask hides it from, and a weight of zero does
// not keep it from them.  So the values of a key tile that some rows do not see whole are looked through (by the softmax's
// threads, 256 bytes each, while they wait for the scores: 6 prompts of up to 2500 tokens x 16 heads 122 -> 124 us), and where
// one is not finite, these threads add that tile's results themselves, key by key.
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// Whether the values of keys from .. to - 1 in a unit are all finite, in this thread's part.
__device__ __forceinline__ bool finite_part(uint32_t unit, int from, int to) {
  uint32_t sum = 0;  // of the values times zero: NaN once one was not finite
#pragma unroll
  for (int n = 0; n < kKeys; n += 16) {  // 16 keys at a time
    const int i = n * 8 + (threadIdx.x & 127);
    if (i < from * 8 || i >= to * 8) continue;
    const uint4 x = lds16(unit + i * 16);
    asm("{\n\tfma.rn.bf16x2 %0, %1, %5, %0;\n\tfma.rn.bf16x2 %0, %2, %5, %0;\n\tfma.rn.bf16x2 %0, %3, %5, %0;\n\t"
        "fma.rn.bf16x2 %0, %4, %5, %0;\n\t}"
        : "+r"(sum)
        : "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(0u));
  }
  return (sum & 0x7F80u) != 0x7F80u && (sum & 0x7F800000u) != 0x7F800000u;
}
// True when x is true for any of a query tile's threads.
__device__ __forceinline__ bool any_of_tile(int t, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(1 + t)
      : "memory");
  return r != 0;
}
// O (+)= P V over the first `sees` keys of the tile, by a row's thread; P as it was left for the product.
__device__ __forceinline__ void add_results(uint32_t ts, uint32_t to, uint32_t unit0, uint32_t unit1, int sees, bool first) {
#pragma unroll 1
  for (int c = 0; c < 128; c += 16) {
    float o[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) o[x] = 0.f;
    if (!first) {
      tc::tmem_ld16(to + c, o);
      tc::tmem_wait_ld();
      tc::touch<16>(o);
    }
    const uint32_t v = c < 64 ? unit0 : unit1;
    const int piece = (c & 63) >> 3;  // 8 dimensions of a key's 64
#pragma unroll 1
    for (int k0 = 0; k0 < kKeys; k0 += 16) {
      float p[8];  // 2 weights each
      tc::tmem_ld<8>(ts + k0 / 2, p);
      tc::tmem_wait_ld();
      tc::touch<8>(p);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (k0 + k >= sees) continue;
        const uint32_t two = __float_as_uint(p[k / 2]);
        const float w = __uint_as_float(k & 1 ? two & 0xFFFF0000u : two << 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 x = lds16(v + (k0 + k) * 128 + (((piece + h) ^ (k & 7)) << 4));
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            o[8 * h + 2 * d] += w * __uint_as_float(y[d] << 16);
            o[8 * h + 2 * d + 1] += w * __uint_as_float(y[d] & 0xFFFF0000u);
          }
        }
      }
    }
    __syncwarp();
    tc::tmem_st16(to + c, o);
  }
  tc::tmem_wait_st();
}

__device__ __forceinline__ void softmax_items(const hs_expanded& a, float scale_log2, uint32_t ring, uint32_t bars, uint32_t tmem,
                                              volatile int* done) {
  tc::Waiter w;
  const int t = threadIdx.x >> 7, lane = threadIdx.x & 31;
  const int row_in_tile = threadIdx.x & 127;
  const uint32_t lanes = (uint32_t)(32 * ((threadIdx.x >> 5) & 3)) << 16;
  const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
  // a negative scale turns the scores round; a scale of zero becomes the smallest normal number, so that a hidden key's
  // -infinity stays one
  const bool negative = scale_log2 < 0.f;
  const float scale = fmaxf(fabsf(scale_log2), 1.17549435e-38f);
  uint32_t phase = 0, passed = 0;  // key tiles of this query tile; of the CTA, in the items before
  Item it;
  Finder f;
  f.start(a);
  for (int k = 0; f.find(a, item_number(k), &it); ++k) {
    const int tiles = it.tiles[t];
    const uint32_t before = passed;
    passed += max(0, it.most());
    if (tiles < 0) continue;
    const int row = t * kQRows + row_in_tile;
    const int sees = a.causal ? min(it.keys, row + it.shift) : it.keys;  // keys below this one are seen
    const int all_see = it.all_see(t);
    float m = -INFINITY;
    float2 la = make_float2(0.f, 0.f), lb = la;  // the sum, in four chains
#pragma unroll 1
    for (int j = 0; j < tiles; ++j, ++phase) {
      // (the values are looked through while the scores are on their way)
      const uint32_t u = (before + j) * kUnits + kUnitsK;
      const uint32_t unit0 = ring + u % kRing * kUnit, unit1 = ring + (u + 1) % kRing * kUnit;
      const int from = max(0, all_see - j * kKeys), end = min(kKeys, it.keys - j * kKeys);  // keys hidden from some rows
      bool finite = true;
      if (from < end) {
        const uint32_t part = 2 * (before + j) + 1;
        w.wait(bars + 8 * (kFull + part % kGroups), part / kGroups & 1);
        finite = finite_part(unit0, from, end) & finite_part(unit1, from, end);
        __syncwarp();
        finite = !any_of_tile(t, !finite);
      }
      w.wait(bars + 8 * (kSFull + t), phase & 1);
      __syncwarp();
      tc::fence_after();
      float s[128];
      tc::tmem_ld<128>(ts, s);
      tc::tmem_wait_ld();
      tc::touch<128>(s);
      if (negative) {
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = -s[c];
      }
      const bool hidden = (j + 1) * kKeys > all_see;
      if (hidden) {
        const int left = sees - j * kKeys;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= left) s[c] = -INFINITY;
      }
      const float top = tc::max_of<128>(s) * scale;
      const bool over = top > m + kLazy;  // (m = -infinity: on the first key seen)
      if (__any_sync(0xFFFFFFFFu, over)) {
        const float now = over ? top : m;
        const float alpha = over ? (m == -INFINITY ? 0.f : exp2f(m - now)) : 1.f;
        m = now;
        la.x *= alpha, la.y *= alpha, lb.x *= alpha, lb.y *= alpha;
        if (j > 0) {  // the products so far have finished: this tile's scores were issued after them
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            float o[16];
            tc::tmem_ld16(to + c, o);
            tc::tmem_wait_ld();
            tc::touch<16>(o);
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] *= alpha;
            tc::tmem_st16(to + c, o);
          }
          tc::tmem_wait_st();
        }
      }
      const float2 sc2 = make_float2(scale, scale), base2 = make_float2(m == -INFINITY ? 0.f : -m, m == -INFINITY ? 0.f : -m);
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        uint32_t p[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float2 y = tc::fma2(make_float2(s[c + 2 * x], s[c + 2 * x + 1]), sc2, base2);
          float2 e = make_float2(tc::exp2_fast(y.x), tc::exp2_fast(y.y));
          if (x & 1)
            lb = tc::add2(lb, e);
          else
            la = tc::add2(la, e);
          p[x] = tc::pack_bf16(e.x, e.y);
        }
        tc::tmem_st16(ts + c / 2, reinterpret_cast<const float*>(p));
      }
      tc::tmem_wait_st();
      if (!finite) {
        add_results(ts, to, unit0, unit1, sees - j * kKeys, j == 0);
        done[t] = 1;
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bars + 8 * (kPReady + t));
    }
    // results
    const float l = (la.x + la.y) + (lb.x + lb.y);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (tiles > 0) {
      w.wait(bars + 8 * (kODone + t), (phase - 1) & 1);
      __syncwarp();
      tc::fence_after();
    }
    const bool there = row < it.rows && HS_CHECK(it.q0 >= 0 && it.q0 + row < a.q_tokens && it.head < a.heads, kChkOutPos);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (int64_t)(it.q0 + (there ? row : 0)) * a.out_token_stride +
                         it.head * a.out_head_stride;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      float o[32];
      if (tiles > 0) {
        tc::tmem_ld<32>(to + c, o);
        tc::tmem_wait_ld();
        tc::touch<32>(o);
      }
#pragma unroll
      for (int x = 0; x < 32; ++x) o[x] = l == 0.f ? 0.f : o[x] * inv;
      if (there) {
#pragma unroll
        for (int x = 0; x < 32; x += 8)
          *reinterpret_cast<uint4*>(out + c + x) =
              make_uint4(tc::pack_bf16(o[x], o[x + 1]), tc::pack_bf16(o[x + 2], o[x + 3]), tc::pack_bf16(o[x + 4], o[x + 5]),
                         tc::pack_bf16(o[x + 6], o[x + 7]));
      }
    }
    if (there && a.lse)
      a.lse[(int64_t)(it.q0 + row) * a.heads + it.head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    tc::fence_before();
  }
  if (w.dead) report(a.status, HS_ERR_TIMEOUT);
}

// ---- query tokens of no sequence (one warp) ----
// Zeros and -infinity for the tokens that no sequence has (cu_q leaves some out, or a sequence's offsets are bad).  Offsets that
// are all right and span the tensor leave none; else every CTA looks at its share of the tokens.
__device__ __forceinline__ void clear_rest(const hs_expanded& a) {
  const int lane = threadIdx.x & 31;
  int q0, q1, k0, k1;
  bool spans = a.seqs > 0 && __ldg(a.cu_q) == 0 && __ldg(a.cu_q + a.seqs) == a.q_tokens;
  for (int s = lane; s < a.seqs; s += 32) spans &= sequence(a, s, &q0, &q1, &k0, &k1);
  if (__all_sync(0xFFFFFFFFu, spans)) return;
  for (int64_t t0 = 32 * (int64_t)blockIdx.x; t0 < a.q_tokens; t0 += 32 * (int64_t)gridDim.x) {
    bool rest = t0 + lane < a.q_tokens;
    for (int s = 0; s < a.seqs; ++s) rest &= !(sequence(a, s, &q0, &q1, &k0, &k1) && t0 + lane >= q0 && t0 + lane < q1);
    for (unsigned who = __ballot_sync(0xFFFFFFFFu, rest); who; who &= who - 1) {
      const int64_t t = t0 + __ffs(who) - 1;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + t * a.out_token_stride;
      for (int i = lane; i < a.heads * 16; i += 32)
        *reinterpret_cast<uint4*>(out + (i >> 4) * a.out_head_stride + (i & 15) * 8) = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int h = lane; h < a.heads; h += 32) a.lse[t * a.heads + h] = -INFINITY;
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1) expanded_kernel(const hs_expanded a, const __grid_constant__ Maps maps,
                                                               float scale_log2) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ int done[2];  // by query tile: the softmax has added a key tile's results itself
  const uint32_t q = (tc::smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t ring = q + 6 * kUnit, bars = ring + kRing * kUnit;
  const int warp = threadIdx.x >> 5;
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s < a.seqs; s += kThreads) {
      int q0, q1, k0, k1;
      if (!sequence(a, s, &q0, &q1, &k0, &k1)) report(a.status, HS_ERR_ID_RANGE);
    }
  if (threadIdx.x == 0) {
    done[0] = done[1] = 0;
    for (int i = 0; i < kGroups; ++i) tc::mbar_init(bars + 8 * (kFull + i), 1);
    for (int i = 0; i < kRing; ++i) tc::mbar_init(bars + 8 * (kEmpty + i), 2);
    tc::mbar_init(bars + 8 * kQFull, 1);
    tc::mbar_init(bars + 8 * kQEmpty, 2);
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(bars + 8 * (kSFull + t), 1);
      tc::mbar_init(bars + 8 * (kPReady + t), 4);
      tc::mbar_init(bars + 8 * (kODone + t), 1);
      tc::mbar_init(bars + 8 * (kDrain + t), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tc::tmem_alloc(tc::smem_u32(&tmem_slot), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax_items(a, scale_log2, ring, bars, tmem, done);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp < kLoadWarp)
      issue_items(a, warp - kMmaWarp, q, ring, bars, tmem, done);
    else if (warp == kLoadWarp)
      load_items(a, maps, q, ring, bars);
    else
      clear_rest(a);
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::tmem_free(tmem, 512);
  }
}

// Tensor map of [tokens][heads][dims] in bf16 for boxes of 128 tokens x 64 dimensions of a head.
bool make_map(CUtensorMap* map, const void* base, int64_t dims, int64_t heads, int64_t tokens, int64_t head_stride,
              int64_t token_stride) {
  if (!tc::encode_tiled()) return false;
  const cuuint64_t size[3] = {(cuuint64_t)dims, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? head_stride * 2 : 256), (cuuint64_t)(tokens > 1 ? token_stride * 2 : 256)};
  const cuuint32_t box[3] = {64, 1, 128}, steps[3] = {1, 1, 1};
  return tc::encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), size, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

uint32_t check_take_expanded() {
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

cudaError_t launch_expanded(const hs_expanded& a, int dev, int sms, cudaStream_t s) {
  static DeviceOnce once;
  const cudaError_t ready = once.ready(dev, [] {
    cudaFuncAttributes f{};
    cudaError_t e = cudaFuncGetAttributes(&f, expanded_kernel);
    // the register trade waits for ever if the launch has fewer than it hands out
    if (e == cudaSuccess && f.numRegs != kRegsLaunch) e = cudaErrorInvalidKernelImage;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(expanded_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    return e;
  });
  if (ready != cudaSuccess) return ready;
  Maps m;
  // a head stride of zero broadcasts one head: a map of one head, read at head 0
  const int64_t strides[4] = {a.qn_head_stride, a.qr_head_stride, a.kn_head_stride, a.v_head_stride};
  int64_t heads[4];
  for (int i = 0; i < 4; ++i) {
    m.head_step[i] = strides[i] > 0 ? 1 : 0;
    heads[i] = strides[i] > 0 ? a.heads : 1;
  }
  // no keys at all: the maps describe the queries, and nothing is read through them
  const bool keys = a.k_tokens > 0;
  if (!make_map(&m.q_nope, a.q_nope, kNope, heads[0], a.q_tokens, strides[0], a.qn_token_stride) ||
      !make_map(&m.q_rope, a.q_rope, kRope, heads[1], a.q_tokens, strides[1], a.qr_token_stride) ||
      (keys && (!make_map(&m.k_nope, a.k_nope, kNope, heads[2], a.k_tokens, strides[2], a.kn_token_stride) ||
                !make_map(&m.k_rope, a.k_rope, kRope, 1, a.k_tokens, 0, a.kr_token_stride) ||
                !make_map(&m.v, a.v, kValue, heads[3], a.k_tokens, strides[3], a.v_token_stride))))
    return cudaErrorInvalidValue;
  // at most this many items: every sequence may end in a block of its own
  const int64_t most = (a.q_tokens / kBlock + a.seqs) * a.heads;
  const int grid = (int)(most < 1 ? 1 : most < sms ? most : sms);
  expanded_kernel<<<grid, kThreads, kSmemBytes, s>>>(a, m, a.scale * kLog2e);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hs
