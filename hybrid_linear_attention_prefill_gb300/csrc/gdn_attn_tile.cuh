// Attention of prompts on the tensor cores (sm_103a; gdn_attn.cuh has the mathematics); one translation unit per 32
// columns of a head instantiates it.
//
// A row is a query of one head.  The heads that share a key head go into one tile, 128 / G tokens of G
// heads, so that a key is read once for all of them and a mask's edge crosses few keys.  A CTA works on
// two such tiles side by side: while the tensor core multiplies for one, eight warps take the other's
// scores to weights, two threads a row.
//
//   scores  S = Q K^T              128 x 128, operands from shared memory, into TMEM
//   weights P = exp2(c S - m)      in the place of S, bf16, as the next product's operand in TMEM
//   output  O += P V               128 x d in TMEM
//
// m is the row's running maximum, but an older one stays in use until the new one is 2^8 above it: the
// weights are then up to 2^8 and their sums as exact as before, and O is rescaled only now and then.
// Sums, maxima, scores and O are fp32.
//
// Roles, 20 warps: eight for each tile's weights and finished outputs; one for each tile that issues MMAs, one
// that issues copies, one that works out the items.  They meet on mbarriers.  A CTA takes an item (256 rows of a key
// head) after another, the items dealt out forwards and backwards in turn; the ring of key and value tiles runs on
// across items.
//
// What bounds it, measured on one GB300 (d = 128, clocks of an SM): a pair of key tiles takes 3,200 where its products
// take 2,048.  A tile's round is a chain: its scores into registers 330, maxima and the vote 550, the rest of the weights
// 350, the issuing warp's look at the barrier 300, the products 1,100 beside the other tile's, and the two tiles' chains
// fill the tensor core to 0.60 between them (16,381 tokens, 16 heads over 2: 787 us, 1,400 TFLOP/s, call after call,
// when the clock falls to 1.75 GHz; 745 with pauses).  An item costs another 10,000: its last product, the output's way
// out and the next one's first tile follow one another in the same warps, so a window of 1,024 (nine tiles an item) runs
// at 880 TFLOP/s.  Steps that brought it here, for 16,381 tokens with pauses: one thread a row and one issuing warp
// 1,025; scores held in registers, descriptors as constants, two issuing warps in turns 967; two threads a row 770; output
// through copies 760; what is seldom run out of the loops' way 750.
//
// A value that is not finite in a place that a row does not see would reach the row as 0 x infinity.
// So a finished row that is not finite is looked into, and worked out again from the keys it sees alone where the
// values that it sees do not explain it.
#pragma once

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "gdn_attn.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"
#include "gdn_tmap.cuh"

namespace gdn {

namespace {

using attn::PromptArgs;
using attn::Seen;
using attn::View;

constexpr int kThreads = 640;
constexpr int kMmaWarp = 16, kLoadWarp = 18, kItemWarp = 19;  // (17: the other tile's products)
constexpr int kKeys = 128;            // a tile
constexpr uint32_t kColS = 0, kColO = 256;  // TMEM columns: two score tiles of 128, two outputs of 128
constexpr int kItemSlots = 4;
constexpr long long kPatience = 1LL << 34;  // clocks of a wait, about eight seconds; then it gives up
// Where a CTA's dynamic shared memory starts in its window, behind the KiB that the system keeps: known here so that the
// descriptors of the products are constants, asked for by the host before a launch, and looked at by every CTA.
constexpr uint32_t kSmemBase = 1024;
constexpr float kLazy = 8.f;           // how far (log2) a maximum may be above the one in use

// Shared memory: two tiles of queries, a ring of tiles of keys and values, statistics, items, barriers.  A tile is
// 128 rows, in halves of 64 columns; products take the head's columns in 32s (past d they are zeros).
constexpr int kHalf = 16384;
template <int kQuarters>
struct Cfg {
  static constexpr int kHalves = (kQuarters + 1) / 2, kTile = kHalves * kHalf, kRing = kHalves == 2 ? 2 : 4;
  static constexpr int kOffQ = 0, kOffK = 2 * kTile, kOffV = kOffK + kRing * kTile;
  static constexpr int kOffStage = kOffV + kRing * kTile;  // 32 rows of 32 columns of output for each warp
  static constexpr int kOffStat = kOffStage + 16 * 2048;
  static constexpr int kStatBytes = 2 * 2 * 128 * 4;
  static constexpr int kOffItem = kOffStat + kStatBytes, kOffBar = kOffItem + kItemSlots * 128;
  static constexpr int kBars = 4 * kRing + 2 * kItemSlots + 2 * 8;
  static constexpr int kSmem = kOffBar + kBars * 8 + 16;
  static_assert(kSmem <= 227 * 1024 && kSmem > 116 * 1024, "one CTA an SM");
};
template <int N>
using Slot = std::integral_constant<int, N>;
// f with the ring's slot as a constant, which the products' operands are made of: an MMA whose descriptors are
// constants is issued in less than the 64 clocks that it takes, one whose are worked out in 110.
template <int kRing, class F>
__device__ __forceinline__ void in_slot(int slot, F f) {
  if (slot == 0) f(Slot<0>());
  else if (kRing == 2 || slot == 1) f(Slot<1>());
  else if (slot == 2) f(Slot<2 % kRing>());
  else f(Slot<3 % kRing>());
}

// The keys that an item's queries see, one list: the first `sink` of the sequence (sinks, rounded up to 16; none where
// the window reaches them), then those from `lo` on, where the first query's window starts.  A tile of keys is 128
// places of the list; the one with the seam is loaded in boxes of 16.
struct Item {
  int valid;
  int q0, n[2];  // first query (among all tokens), queries of either tile
  int p0;        // the first one's position
  int k0;        // the sequence's first key
  int hk;
  int sink, lo;
  int tiles;     // of keys
  int sinks;     // tiles of keys with sinks
  int a[2], z[2];  // tiles of keys [a, z) that either tile of queries sees otherwise
  int lo_all[2], hi_all[2];  // places from `lo` on that all of a tile's queries see
  __device__ __forceinline__ int count(int t) const { return z[t] > 0 ? sinks + z[t] - a[t] : 0; }
  __device__ __forceinline__ int place(int key) const { return key - lo + sink; }  // of a key from `lo` on
};
static_assert(sizeof(Item) <= 128, "a slot");

__device__ __forceinline__ void find_keys(Item& it, const View& view, int tpt) {
  const int first = it.n[0] > 0 && it.p0 + it.n[0] > 0 ? 0 : 1;  // the first tile that sees any
  it.lo = attn::seen_by(view, it.p0 + first * tpt).lo;
  it.sink = (min(view.sinks, it.lo) + 15) / 16 * 16;
  if (view.sinks == 0) it.sink = 0;
  else if (it.sink >= it.lo) it.sink = it.lo = 0;
  it.sinks = (it.sink + kKeys - 1) / kKeys;
  it.tiles = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int pa = it.p0 + t * tpt, pb = pa + it.n[t] - 1;
    it.a[t] = it.z[t] = 0;
    if (it.n[t] <= 0 || pb < 0) continue;
    const int lo = attn::seen_by(view, pa).lo;
    it.z[t] = (it.place(pb + 1) + kKeys - 1) / kKeys;
    it.a[t] = max(it.sinks, view.sinks > 0 && it.sink == 0 ? 0 : it.place(lo) / kKeys);
    it.tiles = max(it.tiles, it.z[t]);
    it.lo_all[t] = it.place(attn::seen_by(view, pb).lo);
    it.hi_all[t] = it.place(attn::seen_by(view, pa).hi);
  }
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

// The two warps of a row's threads at barrier `id`: together, and whether any thread of them has `x`.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;\n" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool any_of_pair(int id, bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\tbarrier.cta.red.or.pred p, %1, 64, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(any)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return any != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ void tmem_st16_start(uint32_t a, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(a),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// 32 columns of a warp's rows to the output; that the copies before have been read from shared memory, or are all done.
__device__ __forceinline__ void copy_out(const CUtensorMap* map, const void* from, int column, int head, int token) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(map),
               "r"(column), "r"(head), "r"(token), "r"(smem_u32(from))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}
__device__ __forceinline__ void copies_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Bits [lo, hi) of 32, of bounds that may lie outside.
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t below_lo = lo >= 32 ? ~0u : lo <= 0 ? 0u : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

// Which of four bf16 are not finite, as their signs' bits; that of the i-th, and whether it is a NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t two) { return ((two & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ bool not_finite(const uint2& x, int i) { return not_finite(i < 2 ? x.x : x.y) >> (i & 1 ? 31 : 15) & 1u; }
__device__ __forceinline__ bool is_nan(const uint2& x, int i) { return ((i < 2 ? x.x : x.y) >> (i & 1 ? 16 : 0) & 0x7fffu) > 0x7f80u; }

// What the two warps of 32 rows look into and work out again: queries and outputs from the tile's first token and head, keys
// and values from the sequence's first (`there` of them to the end of the tensor).
struct Rows {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* out;
  long long qs, ks, vs, os, there;
  int d, G, row0, pa;  // of the warp's first row; position of the tile's first query
  View view;
  float scale_log2;
  __device__ __forceinline__ Seen seen(int row) const { return attn::seen_by(view, pa + row / G); }
  __device__ __forceinline__ long long at(int row, long long stride) const { return row / G * stride + row % G * d; }
};

// Whether the lane's row, which is not finite where `odd`, has to be worked out again: where a column of it is not finite
// and the values that the row sees do not say why, or one that it does not see may have changed it.  A column is as it has
// to be where a NaN is seen in it, or a value that is not finite is and none that is not seen.
//
// Only tiles at a mask's edge hold values that some row does not see, so these are read first; the others are read until
// all columns are explained.  One such value early in a sequence makes every row behind it odd: 4,096 tokens of 32 heads
// with a NaN among the first values take 0.24 ms instead of 0.12 (85 when every such row was worked out again), with one
// among the last, which the rows before it in its tile do not see and have to be worked out without, 2.5.
__device__ __forceinline__ bool unexplained(const Rows& x, const Item& it, int t, bool odd) {
  const int lane = threadIdx.x & 31, off = it.sink - it.lo;
  const bool has = 4 * lane < x.d;  // four columns a lane: bit l of word i is column 4 l + i
  uint32_t bad[4] = {}, nan[4] = {}, known[4] = {}, apart[4] = {};
#pragma unroll 1
  for (unsigned rest = __ballot_sync(0xffffffffu, odd); rest != 0; rest &= rest - 1) {
    const int r = __ffs(rest) - 1;
    const uint2 y = has ? __ldcg(reinterpret_cast<const uint2*>(x.out + x.at(x.row0 + r, x.os) + 4 * lane)) : make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = __ballot_sync(0xffffffffu, not_finite(y, i));
      if (lane == r) bad[i] = w;
    }
  }
  const Seen seen = x.seen(x.row0 + lane);
  auto open = [&]() {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= bad[i] & ~(nan[i] | (known[i] & ~apart[i]));
    return w != 0;
  };
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int kt = it.sinks > 0 ? 0 : it.a[t]; kt < it.z[t]; kt = kt + 1 == it.sinks ? it.a[t] : kt + 1) {
      const int v0 = kt * kKeys;
      const bool edge = it.hi_all[t] < v0 + kKeys || (it.lo_all[t] > v0 && x.view.sinks < v0 + kKeys);
      if (edge == (pass == 1)) continue;
      if (pass == 1 && !__any_sync(0xffffffffu, open())) break;
#pragma unroll 1
      for (int x0 = v0; x0 < v0 + kKeys; x0 += 8) {
        uint2 y[8];
        uint32_t some = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int key = x0 + u < it.sink ? x0 + u : x0 + u - off;
          y[u] = has && key < x.there ? *reinterpret_cast<const uint2*>(x.v + key * x.vs + 4 * lane) : make_uint2(0, 0);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) some |= not_finite(y[u].x) | not_finite(y[u].y);
        if (!__any_sync(0xffffffffu, some != 0)) continue;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int key = x0 + u < it.sink ? x0 + u : x0 + u - off;
          const bool sees = key < seen.hi && (key < x.view.sinks || key >= seen.lo);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t odds = __ballot_sync(0xffffffffu, not_finite(y[u], i));
            const uint32_t nans = __ballot_sync(0xffffffffu, is_nan(y[u], i));
            nan[i] |= sees ? nans : 0u;
            known[i] |= sees ? odds : 0u;
            apart[i] |= sees ? 0u : odds;
          }
        }
      }
    }
  }
  return open();
}

// Eight rows of a warp (the set bits of `rows`, eight at most) from the keys that they see alone, eight keys at a time:
// scores by `mma.sync` (a lane has row g of the eight, and eight columns in a row of each 32 of queries and keys alike),
// weights and sums in fp32, of which a lane has four columns.
__device__ __forceinline__ void rows_again(const Rows& x, unsigned rows) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const bool has = 4 * lane < x.d;
  const unsigned all = rows;
  Seen mine = {0, 0, 0};
  int own = x.row0, sink_end = 0, lo = 0x7fffffff, hi = 0;
#pragma unroll 1
  for (int i = 0; rows != 0; ++i, rows &= rows - 1) {
    const int row = x.row0 + __ffs(rows) - 1;
    const Seen s = x.seen(row);
    sink_end = max(sink_end, s.sink_end);
    lo = min(lo, s.lo);
    hi = max(hi, s.hi);
    if (g == i) own = row, mine = s;
  }
  uint4 q[4];
  auto pieces = [&](const __nv_bfloat16* from, uint4 (&y)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = 32 * i + 8 * c < x.d ? *reinterpret_cast<const uint4*>(from + 32 * i + 8 * c) : make_uint4(0, 0, 0, 0);
  };
  pieces(x.q + x.at(own, x.qs), q);
  float2 o[8][2] = {};
  float m = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int begin = part == 0 ? 0 : lo, end = part == 0 ? sink_end : hi;
#pragma unroll 1
    for (int j0 = begin; j0 < end; j0 += 8) {
      uint4 k[4];
      uint2 v[8];
      pieces(x.k + min(j0 + g, end - 1) * x.ks, k);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = has && j0 + u < end ? *reinterpret_cast<const uint2*>(x.v + (j0 + u) * x.vs + 4 * lane) : make_uint2(0, 0);
      float s[4] = {0.f, 0.f, 0.f, 0.f};  // keys 2 c and 2 c + 1 in the first two
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t q0[4] = {q[i].x, 0u, q[i].y, 0u}, q1[4] = {q[i].z, 0u, q[i].w, 0u};
        mma_bf16(s, q0, k[i].x, k[i].y);
        mma_bf16(s, q1, k[i].z, k[i].w);
      }
      bool sees[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = j0 + 2 * c + i;
        sees[i] = part == 0 ? key < mine.sink_end : key >= mine.lo && key < mine.hi;
        s[i] = sees[i] ? s[i] * x.scale_log2 : -INFINITY;
      }
      float top = fmaxf(s[0], s[1]);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(m, fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)));
      const float base = top == -INFINITY ? 0.f : top, keep = exp2f(m - base);
      m = top;
      uint32_t some = 0;  // values that a weight of 0 does not keep out
#pragma unroll
      for (int u = 0; u < 8; ++u) some |= not_finite(v[u].x) | not_finite(v[u].y);
      const bool odd = __any_sync(0xffffffffu, some != 0);
      float w[2];
      l *= keep;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // (weights of 2^-32 at most: sums of fewer than 2^31 finite values stay finite)
        w[i] = sees[i] ? exp2f(s[i] - base) * 0x1p-32f : 0.f;
        l += w[i];
        if (odd && !sees[i]) w[i] = -1.f;
      }
      if (__any_sync(0xffffffffu, keep != 1.f)) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float f = __shfl_sync(0xffffffffu, keep, 4 * r);
          o[r][0] = mul2(o[r][0], make_float2(f, f));
          o[r][1] = mul2(o[r][1], make_float2(f, f));
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float2 a = widen2(v[u].x), b = widen2(v[u].y);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float f = __shfl_sync(0xffffffffu, w[u & 1], 4 * r + u / 2);
          if (odd && f < 0.f) continue;
          o[r][0] = fma2(a, make_float2(f, f), o[r][0]);
          o[r][1] = fma2(b, make_float2(f, f), o[r][1]);
        }
      }
    }
  }
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  rows = all;
#pragma unroll
  for (int r = 0; r < 8; ++r, rows &= rows - 1) {
    const float sum = __shfl_sync(0xffffffffu, l, 4 * r), inv = 1.f / sum;
    const float2 f[2] = {mul2(o[r][0], make_float2(inv, inv)), mul2(o[r][1], make_float2(inv, inv))};
    if (rows != 0 && has)
      *reinterpret_cast<uint2*>(x.out + x.at(x.row0 + __ffs(rows) - 1, x.os) + 4 * lane) =
          sum == 0.f ? make_uint2(0, 0) : narrow4(f);
  }
}

// The rows of an item that are not finite (`odd`: the lane's, whose other thread's told[128] is about), by both warps of
// theirs.  Apart from the kernel, whose registers and instructions it would take.
__device__ __noinline__ void odd_rows(const PromptArgs& a, const Item& it, int tpt, float scale_log2, bool odd, float* stat,
                                      int* busy) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = warp >> 3, hf = warp >> 2 & 1, quad = warp & 3;
  const int pair = 1 + 4 * t + quad, G = a.Hq / a.Hkv;
  float* const told = stat + t * 256 + 32 * quad + lane;
  if (lane == 0) {
    copies_done();  // rows that are looked at, and may be written again
    atomicAdd(busy, 1);
  }
  __syncwarp();
  Rows x;
  const long long tok = (long long)it.q0 + t * tpt;
  x.q = a.q + tok * a.qs + (long long)it.hk * G * a.d;
  x.k = a.k + (long long)it.k0 * a.ks + it.hk * a.d;
  x.v = a.v + (long long)it.k0 * a.vs + it.hk * a.d;
  x.out = a.out + (tok * a.Hq + (long long)it.hk * G) * a.d;
  x.qs = a.qs;
  x.ks = a.ks;
  x.vs = a.vs;
  x.os = (long long)a.Hq * a.d;
  x.there = (a.cu != nullptr ? (long long)a.Tk : (long long)a.B * a.Tk) - it.k0;
  x.d = a.d;
  x.G = G;
  x.row0 = 32 * quad;
  x.pa = it.p0 + t * tpt;
  x.view = a.view;
  x.scale_log2 = scale_log2;
  told[128 * hf] = odd ? 1.f : 0.f;
  pair_sync(pair);
  if (hf == 0) told[0] = unexplained(x, it, t, odd || told[128] != 0.f) ? 1.f : 0.f;
  pair_sync(pair);
  // the two warps take those rows in turn, eight at a time
  unsigned rest = __ballot_sync(0xffffffffu, told[0] != 0.f);
#pragma unroll 1
  for (int i = 0; rest != 0; ++i) {
    unsigned eight = 0;
    for (int n = 0; n < 8; ++n, rest &= rest - 1) eight |= rest & (0u - rest);
    if ((i & 1) == hf) rows_again(x, eight);
  }
  __syncwarp();
  if (lane == 0) atomicSub(busy, 1);
}

}  // namespace

template <int kQuarters>
__global__ void __launch_bounds__(kThreads, 1)
gdn_attn_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
                     const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ CUtensorMap tm_out,
                     const __grid_constant__ attn::PromptArgs a, int items, int tpt,
                     float scale_log2, int negate, int* __restrict__ err) {
  using C = Cfg<kQuarters>;
  constexpr int kTile = C::kTile, kHalves = C::kHalves, kRing = C::kRing;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw;
  float* stat = reinterpret_cast<float*>(sm + C::kOffStat);  // [tile][half][row]: what a row's threads tell each other
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  uint64_t *k_full = bars, *k_empty = k_full + kRing, *v_full = k_empty + kRing, *v_empty = v_full + kRing,
           *item_full = v_empty + kRing, *item_empty = item_full + kItemSlots, *q_full = item_empty + kItemSlots,
           *q_empty = q_full + 2, *s_full = q_empty + 2, *p_full = s_full + 2, *o_full = p_full + 2, *o_empty = o_full + 2, *turn = o_empty + 2, *drain = turn + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* busy = reinterpret_cast<int*>(tmem_slot + 2);  // warps that work rows out again, which others wait for in patience

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(k_full + i, 1);
      tc::mbar_init(v_full + i, 1);
      tc::mbar_init(k_empty + i, 2);  // by the warps of either tile
      tc::mbar_init(v_empty + i, 2);
    }
    for (int i = 0; i < kItemSlots; ++i) {
      tc::mbar_init(item_full + i, 1);
      tc::mbar_init(item_empty + i, 19);  // sixteen warps of weights, three that issue
    }
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(q_full + t, 1);
      tc::mbar_init(q_empty + t, 1);
      tc::mbar_init(s_full + t, 1);
      tc::mbar_init(p_full + t, 8);
      tc::mbar_init(o_full + t, 1);
      tc::mbar_init(o_empty + t, 8);
      tc::mbar_init(turn + t, 1);
      tc::mbar_init(drain + t, 1);
    }
    *abort_flag = 0;
    *busy = 0;
    tc::fence_mbar_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    tc::prefetch_tensormap(&tm_q);
    tc::prefetch_tensormap(&tm_k);
    tc::prefetch_tensormap(&tm_v);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;  // 0, since it is all of it

  auto give_up = [&](int bit) {
    *abort_flag = 1;
    atomicOr(err, bit);
  };
  if (smem_u32(smem_raw) != kSmemBase) give_up(1);
  // Whether a wait has run out (what it waits for may itself wait for rows that are worked out again).
  auto run_out = [&](long long& since) {
    if (clock64() - since <= kPatience) return false;
    since = clock64();
    return *static_cast<volatile int*>(busy) == 0;
  };
  // One thread's wait; false once this or another wait has run out.
  auto wait = [&](uint64_t* bar, uint32_t par, int bit) {
    if (tc::mbar_wait(bar, par, 1)) return true;
    long long since = clock64();
#pragma unroll 1
    while (!*abort_flag) {
      if (tc::mbar_wait(bar, par, 1)) return true;
      if (run_out(since)) give_up(bit);
    }
    return false;
  };
  // A warp's, which ends for its lanes together.
  auto warp_wait = [&](uint64_t* bar, uint32_t par, int bit) {
    return __all_sync(0xffffffffu, wait(bar, par, bit)) != 0;
  };
  // The n-th item of this CTA.
  auto item_at = [&](int n) { return reinterpret_cast<const Item*>(sm + C::kOffItem + (n % kItemSlots) * 128); };
  auto item_par = [](int n) { return (uint32_t)(n / kItemSlots) & 1u; };

  // The launch's 96 registers a thread are dealt out anew (16 warps x 104 + 4 x 64 = 20 x 96).
  if (warp >= kMmaWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
  if (warp == kItemWarp) {
    // ---- the items: those of one rank of the grid after another, forwards and backwards in turn, so that
    // the CTAs' sums are alike where the items' sizes fall steadily
    const int per = 2 * tpt;
    int b = 0, base = 0;  // of a packed batch: sequences and items (of a head) before
    const int nseq = a.cu == nullptr ? (a.T + per - 1) / per : 0;
    const int heads = a.Hkv;
    bool more = true;
    for (int n = 0; more; ++n) {
      const long long idx = (long long)n * gridDim.x + (n & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      int sb = -1, tile = 0, hk = 0;
      more = idx < items;
      if (more && a.cu == nullptr) {  // the last tiles, which see the most, first
        const uint32_t each = (uint32_t)a.B * heads;  // (no more than items)
        const int rest = (int)((uint32_t)idx % each);
        tile = nseq - 1 - (int)((uint32_t)idx / each);
        sb = rest / heads;
        hk = rest - sb * heads;
      } else if (more) {
        const int f = (int)((uint32_t)idx / (uint32_t)heads);
        hk = (int)idx - f * heads;
        while (b < a.B) {  // 32 sequences at a time
          const int c = b + lane < a.B ? (seq_bounds(a.cu, b + lane, a.T).len + per - 1) / per : 0;
          int sum = c;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, base + sum > f);
          if (hit != 0) {
            const int l = __ffs(hit) - 1;
            sb = b + l;
            tile = __shfl_sync(0xffffffffu, c, l) - 1 - (f - (base + __shfl_sync(0xffffffffu, sum - c, l)));
            break;
          }
          base += __shfl_sync(0xffffffffu, sum, 31);
          b += 32;
        }
        more = sb >= 0;
      }
      if (n >= kItemSlots && !warp_wait(item_empty + n % kItemSlots, item_par(n - kItemSlots), 1)) break;
      if (lane == 0) {
        Item it = {};
        it.valid = more;
        if (more) {
          const SeqChunk sq = seq_bounds(a.cu, sb, a.T), sk = seq_bounds(a.cuk, sb, a.Tk);
          const int first = tile * per;
          it.q0 = (int)sq.bos + first;
          it.n[0] = min(tpt, sq.len - first);
          it.n[1] = min(tpt, sq.len - first - tpt);
          it.p0 = first + sk.len - sq.len;
          it.k0 = (int)sk.bos;
          it.hk = hk;
          find_keys(it, a.view, tpt);
        }
        *reinterpret_cast<Item*>(sm + C::kOffItem + (n % kItemSlots) * 128) = it;
        arrive(item_full + n % kItemSlots);
      }
    }
  } else if (warp == kLoadWarp) {
    // ---- copies: an item's queries, then its tiles of keys and values in turn
    if (lane == 0) {
      long long loads = 0;  // tiles of keys, and of values
      int queries[2] = {0, 0};
      bool ok = true;
      // the list's places from v0 on into a slot
      auto tile_in = [&](const CUtensorMap* whole, const CUtensorMap* part, unsigned char* to, uint64_t* full,
                         uint64_t* empty, const Item& it, int v0) {
        if (loads >= kRing && !wait(empty, (uint32_t)(loads / kRing - 1) & 1u, 2)) return false;
        tc::mbar_arrive_expect_tx(full, kTile);
        if (v0 < it.sink && v0 + kKeys > it.sink) {
#pragma unroll 1
          for (int i = 0; i < kKeys; i += 16) {
            const int tok = it.k0 + (v0 + i < it.sink ? v0 + i : it.lo + v0 + i - it.sink);
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              tc::tma_load_3d(to + h * kHalf + i * 128, part, 64 * h, it.hk, tok, full);
          }
        } else {
          const int tok = it.k0 + (v0 < it.sink ? v0 : it.lo + v0 - it.sink);
#pragma unroll
          for (int h = 0; h < kHalves; ++h) tc::tma_load_3d(to + h * kHalf, whole, 64 * h, it.hk, tok, full);
        }
        return true;
      };
      for (int n = 0; ok; ++n) {
        if (!(ok = wait(item_full + n % kItemSlots, item_par(n), 2))) break;
        const Item it = *item_at(n);
        arrive(item_empty + n % kItemSlots);
        if (!it.valid) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || (n > 0 && !(ok = wait(q_empty + t, (n - 1) & 1, 2)))) break;
          ++queries[t];
          tc::mbar_arrive_expect_tx(q_full + t, kHalves * 128 * G * tpt);
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tc::tma_load_3d(sm + C::kOffQ + t * kTile + h * kHalf, &tm_q, 64 * h, it.hk * G, it.q0 + t * tpt,
                            q_full + t);
        }
        for (int kt = 0; ok && kt < it.tiles; ++kt) {
          const int slot = (int)(loads % kRing);
          ok = tile_in(&tm_k, &tm_k16, sm + C::kOffK + slot * kTile, k_full + slot, k_empty + slot, it, kt * kKeys) &&
               tile_in(&tm_v, &tm_v16, sm + C::kOffV + slot * kTile, v_full + slot, v_empty + slot, it, kt * kKeys);
          if (ok) ++loads;
        }
      }
      // what is in flight lands before the CTA ends, whoever gave up (bounded again; after a wait that gave up a
      // tile of keys may be one ahead of its values)
      auto land = [](uint64_t* bar, uint32_t par) {
#pragma unroll 1
        for (int i = 0; i < 1 << 14 && !tc::mbar_wait(bar, par, 1); ++i) {
        }
      };
#pragma unroll 1
      for (int i = 0; i < kRing; ++i)
        if (i < loads || !ok) {
          const uint32_t p = (uint32_t)((loads - 1 - i) / kRing) & 1u;
#pragma unroll 1
          for (uint32_t x = ok ? p : 0; x <= (ok ? p : 1); ++x) {
            land(k_full + i, x);
            land(v_full + i, x);
          }
        }
      for (int t = 0; t < 2; ++t)
        if (queries[t] > 0) land(q_full + t, (uint32_t)(queries[t] - 1) & 1u);
    }
    __syncwarp();
  } else {
    // ---- products, a warp for either tile of queries: the last weights' product, then the next scores in the weights'
    // place.  The two warps take turns, so that the tensor core works on one tile while the other's weights are made
    // (left to themselves they fall into step).  Looking at a barrier takes 200 clocks beside running products: a warp's
    // lanes look at all that a step waits for at once, and while the other warp has its turn.
    auto products = [&](auto tile) {
      constexpr int t = decltype(tile)::value;
      constexpr uint32_t id_o = tc::idesc_bf16(128, 32 * kQuarters, 0, 1), sb = kSmemBase;
      const uint32_t id_s = tc::idesc_bf16(128, kKeys, 0, 0) | (negate ? 1u << 13 : 0u);
      bool on = false, first = false, last = false;  // weights whose product is to come
      int seen_items = 0;                            // items so far that this tile sees any keys of
      uint32_t p_par = 0;
      uint32_t tiles = 0;  // of keys, in all: the ring's slot and phase, and the turn
      bool ok = true;
      // Until every lane's barrier (null: none) has passed its phase; false after giving up.
      auto look = [&](uint64_t* bar, uint32_t par) {
        bool done = bar == nullptr;
        long long since = 0;
        for (int i = 0;; ++i) {
          if (!done) done = tc::mbar_wait(bar, par, 1);
          if (__all_sync(0xffffffffu, done)) return true;
          if ((i & 255) == 255) {
            if (since == 0) since = clock64();
            if (lane == 0 && run_out(since)) give_up(1);
            if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
          }
        }
      };
      // A step is a tile of keys.  An item without any, and the end, are one too, for the product that is pending (in one
      // place all, since what is executed between two tiles has to fit the instruction cache).
      for (int n = 0;; ++n) {
        if (!(ok = warp_wait(item_full + n % kItemSlots, item_par(n), 1))) break;
        const Item* ip = item_at(n);
        const int valid = ip->valid, all = ip->tiles, sinks = ip->z[t] > 0 ? ip->sinks : 0, from = ip->a[t], to = ip->z[t];
        const int total = ip->count(t);
        __syncwarp();
        if (lane == 0) arrive(item_empty + n % kItemSlots);
        int left = total;
#pragma unroll 1
        for (int kt = 0; kt < (valid ? max(all, 1) : 1); ++kt) {
          const bool keys = valid && kt < all, some = keys && (kt < sinks || (kt >= from && kt < to));
          const int slot = (int)(tiles % kRing), before = (int)((tiles + kRing - 1) % kRing);
          // the pending product's values, weights and place; the keys (an item's first ones and the queries apart, so
          // that the last item's product does not wait for them); the turn
          uint64_t* bar = nullptr;
          uint32_t par = 0;
          if (lane == 0 && tiles > 0) bar = v_full + before, par = ((tiles - 1) / kRing) & 1u;
          if (lane == 1 && keys && kt > 0) bar = k_full + slot, par = (tiles / kRing) & 1u;
          if (lane == 2 && on) bar = p_full + t, par = p_par;
          // (the item's before; items that see nothing have no phase, so that neither side can be two ahead)
          if (lane == 3 && on && first && seen_items > 1) bar = o_empty + t, par = (uint32_t)seen_items & 1u;
          if (lane == 4 && keys && (t == 1 || tiles > 0)) bar = turn + t, par = t == 1 ? tiles & 1u : (tiles - 1) & 1u;
          if (!(ok = look(bar, par))) break;
          in_slot<kRing>(slot, [&](auto at) {
            constexpr int S = decltype(at)::value, kBefore = (S + kRing - 1) % kRing;
            if (on && lane == 0) {
              const uint64_t v = tc::sdesc(sb + C::kOffV + kBefore * kTile, kHalf, 1024, tc::kSw128);
              const uint32_t more = first ? 0u : 1u;
              tc::fence_after();
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                tc::mma_f16_ta(kColO + t * 128, kColS + t * 128 + 8 * k, v + ((k * 2048) >> 4), id_o, k > 0 ? 1u : more);
              if (last) tc::commit(o_full + t);
            }
            __syncwarp();
            if (__builtin_expect(valid && kt == 0, 0)) {
              bar = lane == 0 ? q_full + t : lane == 1 && keys ? k_full + S : nullptr;
              if (!(ok = look(bar, lane == 0 ? (uint32_t)n & 1u : (tiles / kRing) & 1u))) return;
            }
            if (lane == 0) {
              if (some) {
                const uint64_t q = tc::sdesc(sb + C::kOffQ + t * kTile, 16, 1024, tc::kSw128);
                const uint64_t k = tc::sdesc(sb + C::kOffK + S * kTile, 16, 1024, tc::kSw128);
                tc::fence_after();
#pragma unroll
                for (int i = 0; i < 2 * kQuarters; ++i) {
                  // (A constant number of steps.  With each under a condition of its own, i below a run-time count, those
                  // past the fourth were built to multiply an earlier step's queries; why is not known.)
                  const uint64_t off = (uint64_t)(((i >> 2) * kHalf + (i & 3) * 32) >> 4);
                  tc::mma_bf16(kColS + t * 128, q + off, k + off, id_s, i > 0);
                  // the other warp's turn, so that its products are there when these end
                  if (i == kQuarters - 1) arrive(turn + 1 - t);
                }
                tc::commit(s_full + t);
              } else if (keys) {
                arrive(turn + 1 - t);
              }
              if (valid && (total > 0 ? some && left == 1 : kt == 0)) tc::commit(q_empty + t);
              if (keys && tiles > 0) tc::commit(v_empty + kBefore);
              if (keys) tc::commit(k_empty + S);
            }
          });
          if (!ok) break;
          if (on) p_par ^= 1u;
          on = some;
          if (some) {
            first = left == total;
            last = --left == 0;
            seen_items += first;
          }
          __syncwarp();
          tiles += keys;
        }
        if (!ok || !valid) break;
      }
      if (lane == 0) {
        tc::commit(drain + t);
        if (!tc::mbar_wait(drain + t, 0, 1u << 16)) give_up(1);
      }
    };
    if (warp == kMmaWarp) products(Slot<0>());
    else products(Slot<1>());
    __syncwarp();
  }
  } else {
    // ---- weights, and a finished tile's outputs: two threads a row, each for 64 of a tile's keys (and every other 32
    // columns of the output), in two warps that meet at a barrier of their own
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");
    const int t = warp >> 3, hf = warp >> 2 & 1, quad = warp & 3, row = 32 * quad + lane, tr = row / G;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t s_at = tmem + lanes + kColS + t * 128 + 64 * hf, p_at = tmem + lanes + kColS + t * 128 + 32 * hf,
                   o_at = tmem + lanes + kColO + t * 128;
    const int pair = 1 + 4 * t + quad;  // the barrier: both warps of a row come to it every time, one that gave up too
    float* const told = stat + t * 256 + row;  // of half h: + 128 h
    unsigned char* const stage = sm + C::kOffStage + warp * 2048;
    uint32_t s_par = 0, o_par = 0;
    bool ok = warp_wait(item_full, 0, 1);
    bool stop = any_of_pair(pair, !ok);
    for (int n = 0; !stop; ++n) {
      const Item* ip = item_at(n);
      const int valid = ip->valid, pa = ip->p0 + t * tpt, off = ip->sink - ip->lo;
      const int sink_tiles = ip->z[t] > 0 ? ip->sinks : 0, from = ip->a[t], to = ip->z[t];
      const int lo_all = ip->lo_all[t], hi_all = ip->hi_all[t];
      if (!valid) break;
      float m = -INFINITY, l = 0.f;  // the maximum in use (log2), the weights' sum
      // places of the list that the row sees: [0, sinks) and [lo, hi), and what all the tile's rows see
      const Seen mine = attn::seen_by(a.view, pa + tr);
      const int lo = mine.lo + off, hi = mine.hi + off;
      for (int kt = sink_tiles > 0 ? 0 : from; kt < to; kt = kt + 1 == sink_tiles ? from : kt + 1) {
        ok = warp_wait(s_full + t, s_par, 1);
        s_par ^= 1u;
        tc::fence_after();
        __syncwarp();
        const int v0 = kt * kKeys;
        float s[64];
        tc::tmem_ld32x2(s_at, s_at + 32, s);
        if (__builtin_expect(hi_all < v0 + kKeys || (lo_all > v0 && a.view.sinks < v0 + kKeys), 0)) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            const int x = v0 + 64 * hf + c;
            const uint32_t see = (bits(0, a.view.sinks - x) | bits(lo - x, 32)) & bits(0, hi - x);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see >> i & 1u)) s[c + i] = -INFINITY;
          }
        }
        // The weights of 32 keys relative to the maximum in use; the first beside the search for the tile's own maximum.
        float2 sum = make_float2(0.f, 0.f);
        uint32_t w[16];
        auto weights = [&](int from32) {
          const float base = m == -INFINITY ? 0.f : -m;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = fma2(make_float2(s[from32 + 2 * i], s[from32 + 2 * i + 1]),
                                  make_float2(scale_log2, scale_log2), make_float2(base, base));
            const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
            sum = fma2(p, make_float2(1.f, 1.f), sum);
            w[i] = pack_bf16(p.x, p.y);
          }
        };
        weights(0);
        float top4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) top4[i] = fmaxf(s[i], s[i + 4]);
#pragma unroll
        for (int i = 8; i < 64; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) top4[k] = max3(top4[k], s[i + k], s[i + k + 4]);
        float top = scale_log2 * fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]);
        // (Both warps have their scores when they meet: the other's weights go in the place of some of them.)
        if (__builtin_expect(any_of_pair(pair, !ok || top > m + kLazy), 0)) {
          // a row's is far above: it takes its place, and those weights are made again
          told[128 * hf] = top;
          if ((stop = any_of_pair(pair, !ok))) break;
          top = fmaxf(top, told[128 * (1 - hf)]);
          const float next = top > m + kLazy ? top : m;
          if (__any_sync(0xffffffffu, m != -INFINITY)) {
            const float f = next == m ? 1.f : ex2_approx(m - next);
            l *= f;
#pragma unroll 1
            for (int c = 16 * hf; c < a.d; c += 32) {
              float r[16];
              tc::tmem_ld16(o_at + c, r);
              uint32_t x[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(r[i] * f);
              tmem_st16_start(o_at + c, x);
            }
          }
          m = next;
          sum = make_float2(0.f, 0.f);
          weights(0);
        }
        tmem_st16_start(p_at, w);  // in the scores' place
        weights(32);
        tmem_st16_start(p_at + 16, w);
        l += sum.x + sum.y;
        tmem_st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) arrive(p_full + t);
      }
      if (stop) break;
      // ---- outputs (what they take of the item is read here, so that the loop above has the registers)
      const int tok0 = ip->q0 + t * tpt, hk = ip->hk, nt = ip->n[t];
      pair_sync(pair);  // (the maxima there are read)
      told[128 * hf] = l;
      pair_sync(pair);
      l += told[128 * (1 - hf)];  // (the two in either order: the same)
      const bool some = to > 0;
      if (some) {
        ok = warp_wait(o_full + t, o_par, 1);
        o_par ^= 1u;
        tc::fence_after();
      }
      const bool live = tr < tpt && tr < nt;
      const long long tok = (long long)tok0 + tr;
      const int head = hk * G + row - tr * G;
      __nv_bfloat16* out = a.out + (tok * a.Hq + head) * a.d;
      // A warp's rows go out as one copy of 32 columns where all of them are there and are whole heads or tokens.  (Stores of
      // a row a lane, 16 bytes of 32 lines each, hold up what the SM's other warps read and wait for: an item took 4,000
      // clocks longer; 4,096 tokens 123.5 us against 117.4, 128 prompts of 256 233 against 218.)
      const bool by_copy = 128 % G == 0 && (32 * quad + 31) / G < nt;
      const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
      float2 zero = make_float2(0.f, 0.f);  // or NaN, once a value is not finite
#pragma unroll 1
      for (int c = 32 * hf; c < a.d; c += 64) {
        float r[32] = {};
        __syncwarp();  // the load wants the lanes together, which a store of some of them may part
        if (some) tc::tmem_ld32(o_at + c, r);
        uint4 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 f[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[k] = mul2(make_float2(r[8 * i + 2 * k], r[8 * i + 2 * k + 1]), make_float2(inv, inv));
            zero = fma2(f[k], make_float2(0.f, 0.f), zero);
          }
          y[i] = narrow8(f);
        }
        if (by_copy) {
          if (lane == 0) copies_read();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(stage + lane * 64 + 16 * (i ^ (lane >> 1 & 3))) = y[i];
          tc::fence_proxy_async();
          __syncwarp();
          if (lane == 0) copy_out(&tm_out, stage, c, hk * G + (G > 32 ? 32 * quad % G : 0), tok0 + 32 * quad / G);
        } else if (live) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + 8 * i < a.d) *reinterpret_cast<uint4*>(out + c + 8 * i) = y[i];
        }
      }
      if (live && hf == 0 && a.lse != nullptr)
        a.lse[tok * a.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * attn::kLn2;
      tc::fence_before();
      __syncwarp();
      if (some && lane == 0) arrive(o_empty + t);
      // rows that are not finite are looked into (but where the weights' sum is not: nothing else could be; a row that
      // sees nothing is among them where values beside it are not, 0 times their sum)
      bool odd = !(zero.x + zero.y == 0.f) && live && l <= FLT_MAX;
      ok = ok && warp_wait(item_full + (n + 1) % kItemSlots, item_par(n + 1), 1);
      if (__builtin_expect(any_of_pair(pair, odd || !ok), 0)) {
        if (any_of_pair(pair, !ok)) break;
        odd_rows(a, *ip, tpt, negate ? -scale_log2 : scale_log2, odd, stat, busy);
      }
      if (lane == 0) arrive(item_empty + n % kItemSlots);
    }
    if (lane == 0) copies_done();
    __syncwarp();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  __syncwarp();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

namespace {

bool head_map(CUtensorMap* m, const void* base, long long stride, int heads, int d, long long tokens, int box_heads,
              int box_tokens, int columns = 64) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)(tokens > 1 ? stride : (long long)heads * d) * 2};
  const cuuint32_t box[3] = {(cuuint32_t)columns, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  return make_map16(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 3, dims, strides, box,
                    columns == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace

template <int kQuarters>
cudaError_t launch_attn_tiles(const attn::PromptArgs& a, int* status, cudaStream_t st) {
  const bool packed = a.cu != nullptr;
  const long long nq = packed ? (long long)a.T : (long long)a.B * a.T;
  const long long nk = packed ? (long long)a.Tk : (long long)a.B * a.Tk;
  const int G = a.Hq / a.Hkv, tpt = 128 / G, per = 2 * tpt, sms = device_sms();
  if (sms == 0) return cudaErrorNoDevice;
  const long long tiles = ((long long)a.T + per - 1) / per;
  const long long items = (packed ? tiles + a.B : tiles * a.B) * a.Hkv;  // (packed: an upper bound)
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  CUtensorMap q, k, v, k16, v16, out;
  if (!head_map(&q, a.q, a.qs, a.Hq, a.d, nq, G, tpt)) return cudaErrorInvalidValue;
  // without keys nothing is loaded by these
  auto key_map = [&](CUtensorMap* m, const void* x, long long stride, int box) {
    return nk > 0 ? head_map(m, x, stride, a.Hkv, a.d, nk, 1, box) : head_map(m, a.q, a.qs, a.Hkv, a.d, nq, 1, box);
  };
  if (!key_map(&k, a.k, a.ks, kKeys) || !key_map(&v, a.v, a.vs, kKeys) || !key_map(&k16, a.k, a.ks, 16) ||
      !key_map(&v16, a.v, a.vs, 16))
    return cudaErrorInvalidValue;
  // (not used where a warp's rows are not whole heads or tokens)
  const int rows_heads = 128 % G != 0 ? 1 : G < 32 ? G : 32;
  if (!head_map(&out, a.out, (long long)a.Hq * a.d, a.Hq, a.d, nq, rows_heads, 32 / rows_heads, 32))
    return cudaErrorInvalidValue;
  cudaError_t e = set_smem_limit_once<gdn_attn_tile_kernel<kQuarters>>(Cfg<kQuarters>::kSmem);
  if (e != cudaSuccess) return e;
  int base = 0;
  if ((e = attn_smem_base(&base)) != cudaSuccess) return e;
  if (base != (int)kSmemBase) return cudaErrorNotSupported;
  float c = a.scale * attn::kLog2e;
  const int negate = c < 0.f;  // as the sign of the queries
  c = std::max(negate ? -c : c, 0x1p-126f);  // (unseen scores are minus infinity, and 0 times that would not do)
  gdn_attn_tile_kernel<kQuarters><<<(unsigned)std::min<long long>(items, sms), kThreads, Cfg<kQuarters>::kSmem, st>>>(
      q, k, v, k16, v16, out, a, (int)items, tpt, c, negate, status);
  return cudaGetLastError();
}

}  // namespace gdn
