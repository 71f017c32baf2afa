// Attention of prompts on the tensor cores (sm_103a; gdn_attn.cuh has the mathematics).
//
// A row is a query of one head.  The heads that share a key head go into one tile, 128 / G tokens of G
// heads, so that a key is read once for all of them and a mask's edge crosses few keys.  A CTA works on
// two such tiles side by side: while the tensor core multiplies for one, four warps take the other's
// scores to weights, a row a thread, so that a row's maximum and sum need no exchange.
//
//   scores  S = Q K^T              128 x 128, operands from shared memory, into TMEM
//   weights P = exp2(c S - m)      in the place of S, bf16, as the next product's operand in TMEM
//   output  O += P V               128 x d in TMEM
//
// m is the row's running maximum, but an older one stays in use until the new one is 2^8 above it: the
// weights are then up to 2^8 and their sums as exact as before, and O is rescaled only now and then.
// Sums, maxima, scores and O are fp32.
//
// Roles, 16 warps: four for each tile's weights; four that write finished tiles out while the next item's
// products run; one that issues MMAs, one that issues copies, one that works out the items.  They meet on
// mbarriers only.  A CTA takes an item (256 rows of a key head) after another; the ring of key and value
// tiles runs on across items.
//
// A value that is not finite in a place that a row does not see would reach the row as 0 x infinity.
// So a finished row that is not finite is worked out again from the keys it sees alone.
#include <algorithm>

#include "gdn_attn.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"
#include "gdn_tmap.cuh"

namespace gdn {

namespace {

using attn::PromptArgs;
using attn::Seen;
using attn::View;

constexpr int kThreads = 512;
constexpr int kOutWarp = 8, kMmaWarp = 12, kLoadWarp = 13, kItemWarp = 14;
constexpr int kKeys = 128;            // a tile
constexpr uint32_t kColS = 0, kColO = 256;  // TMEM columns: two score tiles of 128, two outputs of 128
constexpr int kItemSlots = 4;
constexpr uint32_t kPolls = 1u << 20;  // of a wait, 3.7 us each: about four seconds; then it gives up
constexpr float kLazy = 8.f;           // how far (log2) a maximum may be above the one in use

// Shared memory: two tiles of queries, a ring of tiles of keys and values, statistics, items, barriers.  A tile is
// 128 rows, in halves of 64 columns (one half where d is at most 64; columns past d are zeros).
constexpr int kHalf = 16384;
template <int kHalves>
struct Cfg {
  static constexpr int kTile = kHalves * kHalf, kStages = kHalves == 2 ? 5 : 8;
  static constexpr int kOffQ = 0, kOffKv = 2 * kTile, kOffStat = kOffKv + kStages * kTile;
  static constexpr int kOffItem = kOffStat + 2 * 128 * 8, kOffBar = kOffItem + kItemSlots * 128;
  static constexpr int kBars = 2 * kStages + 2 * kItemSlots + 2 * 7 + 1;
  static constexpr int kSmem = kOffBar + kBars * 8 + 16;
  static_assert(kSmem <= 227 * 1024 && kSmem > 116 * 1024, "one CTA an SM");
};

// Tiles of 128 keys that a tile of queries sees some of: [0, s) and [a, z).
struct Span {
  int s, a, z;
  __device__ __forceinline__ bool has(int kt) const { return kt < s || (kt >= a && kt < z); }
  __device__ __forceinline__ int count() const { return s + z - a; }
};

struct Item {
  int valid;
  int q0, n0, n1;  // first query (among all tokens), queries of either tile
  int p0;          // the first one's position
  int k0;          // the sequence's first key
  int hk;
  int ns, w0, w1;  // tiles of keys: [0, ns) and [w0, w1)
  Span t[2];
};
static_assert(sizeof(Item) <= 128, "a slot");

__device__ __forceinline__ Span span_of(const View& view, int p0, int n) {
  Span r = {0, 0, 0};
  const int pb = p0 + n - 1;
  if (n <= 0 || pb < 0) return r;
  const Seen lo = attn::seen_by(view, p0), hi = attn::seen_by(view, pb);
  r.a = lo.lo / kKeys;
  r.z = (hi.hi + kKeys - 1) / kKeys;
  r.s = min((hi.sink_end + kKeys - 1) / kKeys, r.a);
  return r;
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
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
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Bits [lo, hi) of 32, of bounds that may lie outside.
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t below_lo = lo >= 32 ? ~0u : lo <= 0 ? 0u : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

}  // namespace

template <int kHalves>
__global__ void __launch_bounds__(kThreads, 1)
gdn_attn_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const attn::PromptArgs a, int items, int tpt,
                     float scale_log2, int negate, int* __restrict__ err) {
  using C = Cfg<kHalves>;
  constexpr int kTile = C::kTile, kStages = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw;
  float2* stat = reinterpret_cast<float2*>(sm + C::kOffStat);  // [tile][row]: maximum in use (log2), sum
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  uint64_t *kv_full = bars, *kv_empty = kv_full + kStages, *item_full = kv_empty + kStages,
           *item_empty = item_full + kItemSlots, *q_full = item_empty + kItemSlots, *q_empty = q_full + 2,
           *s_full = q_empty + 2, *p_full = s_full + 2, *st_full = p_full + 2, *o_full = st_full + 2,
           *o_empty = o_full + 2, *drain = o_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(kv_full + i, 1);
      tc::mbar_init(kv_empty + i, 1);
    }
    for (int i = 0; i < kItemSlots; ++i) {
      tc::mbar_init(item_full + i, 1);
      tc::mbar_init(item_empty + i, 14);  // twelve warps of weights and outputs, two that issue
    }
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(q_full + t, 1);
      tc::mbar_init(q_empty + t, 1);
      tc::mbar_init(s_full + t, 1);
      tc::mbar_init(p_full + t, 4);
      tc::mbar_init(st_full + t, 4);
      tc::mbar_init(o_full + t, 1);
      tc::mbar_init(o_empty + t, 4);
    }
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
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
  const uint32_t tmem = *tmem_slot;

  auto give_up = [&](int bit) {
    *abort_flag = 1;
    atomicOr(err, bit);
  };
  // One thread's wait; false once this or another wait has run out.
  auto wait = [&](uint64_t* bar, uint32_t par, int bit) {
    for (uint32_t n = 0; n < kPolls; n += 64) {
      if (tc::mbar_wait(bar, par, 64)) return true;
      if (*abort_flag) return false;
    }
    give_up(bit);
    return false;
  };
  // A warp's, which ends for its lanes together.
  auto warp_wait = [&](uint64_t* bar, uint32_t par, int bit) {
    return __all_sync(0xffffffffu, wait(bar, par, bit)) != 0;
  };
  // The n-th item of this CTA (one thread of a warp waits for the others' sake where `alone`).
  auto item_at = [&](int n) { return reinterpret_cast<const Item*>(sm + C::kOffItem + (n % kItemSlots) * 128); };
  auto item_par = [](int n) { return (uint32_t)(n / kItemSlots) & 1u; };

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
        const int rest = (int)(idx % ((long long)a.B * heads));
        tile = nseq - 1 - (int)(idx / ((long long)a.B * heads));
        sb = rest / heads;
        hk = rest - sb * heads;
      } else if (more) {
        const int f = (int)(idx / heads);
        hk = (int)(idx - (long long)f * heads);
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
          it.n0 = min(tpt, sq.len - first);
          it.n1 = min(tpt, sq.len - first - tpt);
          it.p0 = first + sk.len - sq.len;
          it.k0 = (int)sk.bos;
          it.hk = hk;
          it.t[0] = span_of(a.view, it.p0, it.n0);
          it.t[1] = span_of(a.view, it.p0 + tpt, it.n1);
          const bool one = it.t[0].count() > 0, two = it.t[1].count() > 0;
          it.w0 = one && two ? min(it.t[0].a, it.t[1].a) : one ? it.t[0].a : it.t[1].a;
          it.w1 = max(it.t[0].z, it.t[1].z);
          it.ns = min(max(it.t[0].s, it.t[1].s), it.w0);
        }
        *reinterpret_cast<Item*>(sm + C::kOffItem + (n % kItemSlots) * 128) = it;
        arrive(item_full + n % kItemSlots);
      }
    }
  } else if (warp == kLoadWarp) {
    // ---- copies: an item's queries, then its tiles of keys and values in turn
    if (lane == 0) {
      int stage = 0;
      uint32_t par = 0;
      long long loads = 0;
      int queries[2] = {0, 0};
      bool ok = true;
      auto tile_in = [&](const CUtensorMap* m, int hk, int tok) {
        if (loads >= kStages && !wait(kv_empty + stage, par ^ 1u, 2)) return false;
        tc::mbar_arrive_expect_tx(kv_full + stage, kTile);
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          tc::tma_load_3d(sm + C::kOffKv + stage * kTile + h * kHalf, m, 64 * h, hk, tok, kv_full + stage);
        ++loads;
        if (++stage == kStages) stage = 0, par ^= 1u;
        return true;
      };
      int n = 0;
      for (; ok; ++n) {
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
        for (int kt = it.ns > 0 ? 0 : it.w0; ok && kt < it.w1; kt = kt + 1 == it.ns ? it.w0 : kt + 1)
          ok = tile_in(&tm_k, it.hk, it.k0 + kt * kKeys) && tile_in(&tm_v, it.hk, it.k0 + kt * kKeys);
      }
      // what is in flight lands before the CTA ends, whoever gave up (bounded again)
      for (int i = 0; i < kStages && i < loads; ++i)
        (void)tc::mbar_wait(kv_full + i, (uint32_t)((loads - 1 - i) / kStages) & 1u, 1u << 14);
      for (int t = 0; t < 2; ++t)
        if (queries[t] > 0) (void)tc::mbar_wait(q_full + t, (uint32_t)(queries[t] - 1) & 1u, 1u << 14);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---- products.  For each tile of queries in turn: the last weights' product, then the next scores (in
    // the weights' place), so that the tensor core works on one while the other's weights are made.
    if (lane == 0) {
      const uint32_t id_s = tc::idesc_bf16(128, kKeys, 0, 0) | (negate ? 1u << 13 : 0u);
      const int nv = (a.d + 15) / 16 * 16;
      const uint32_t id_o = tc::idesc_bf16(128, nv, 0, 1);
      const uint32_t sb = smem_u32(sm);
      int stage = 0;
      uint32_t par = 0;
      struct Pending {
        bool on, first, last;
        int stage;
        uint32_t par;
      } pend[2] = {};
      uint32_t p_par[2] = {0, 0};
      int owed = -1;  // the stage of values that both pending products read
      bool ok = true;
      int n = 0;
      int o_item[2] = {0, 0};  // the item of the pending product
      // the product of tile t's weights, if one is pending
      auto flush = [&](int t) {
        Pending& p = pend[t];
        if (!p.on) return true;
        p.on = false;
        if (!wait(kv_full + p.stage, p.par, 2) || !wait(p_full + t, p_par[t], 1)) return false;
        p_par[t] ^= 1u;
        if (p.first && o_item[t] > 0 && !wait(o_empty + t, (o_item[t] - 1) & 1, 1)) return false;
        tc::fence_after();
        const uint64_t v = tc::sdesc(sb + C::kOffKv + p.stage * kTile, kHalf, 1024, tc::kSw128);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          tc::mma_f16_ta(tmem + kColO + t * 128, tmem + kColS + t * 128 + 8 * k, v + ((k * 2048) >> 4), id_o,
                         !p.first || k > 0);
        if (p.last) tc::commit(o_full + t);
        return true;
      };
      auto settle = [&]() {  // the pending products' values may go
        if (owed >= 0) tc::commit(kv_empty + owed);
        owed = -1;
      };
      for (;; ++n) {
        if (!(ok = wait(item_full + n % kItemSlots, item_par(n), 1))) break;
        const Item it = *item_at(n);
        arrive(item_empty + n % kItemSlots);
        if (!it.valid) break;
        int cnt[2] = {0, 0};
        const int total[2] = {it.t[0].count(), it.t[1].count()};
        bool fresh = true;
        for (int kt = it.ns > 0 ? 0 : it.w0; ok && kt < it.w1; kt = kt + 1 == it.ns ? it.w0 : kt + 1) {
          const int ks = stage;
          const uint32_t kpar = par;
          if (++stage == kStages) stage = 0, par ^= 1u;
          const int vs = stage;
          const uint32_t vpar = par;
          if (++stage == kStages) stage = 0, par ^= 1u;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || !(ok = flush(t))) break;
            if (t == 1) settle();
            if (t == 0 && !(ok = wait(kv_full + ks, kpar, 2))) break;
            if (fresh && !(ok = wait(q_full + t, n & 1, 2))) break;
            if (it.t[t].has(kt)) {
              tc::fence_after();
              const uint64_t q = tc::sdesc(sb + C::kOffQ + t * kTile, 16, 1024, tc::kSw128);
              const uint64_t k = tc::sdesc(sb + C::kOffKv + ks * kTile, 16, 1024, tc::kSw128);
#pragma unroll
              for (int i = 0; i < 4 * kHalves; ++i) {  // (past d by zeros; a step under a run-time condition was compiled wrong)
                const uint64_t off = (uint64_t)(((i >> 2) * kHalf + (i & 3) * 32) >> 4);
                tc::mma_bf16(tmem + kColS + t * 128, q + off, k + off, id_s, i > 0);
              }
              tc::commit(s_full + t);
              pend[t].on = true;
              pend[t].first = cnt[t] == 0;
              pend[t].last = cnt[t] + 1 == total[t];
              pend[t].stage = vs;
              pend[t].par = vpar;
              o_item[t] = n;
              if (++cnt[t] == total[t]) tc::commit(q_empty + t);
            }
          }
          fresh = false;
          tc::commit(kv_empty + ks);
          owed = vs;
        }
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (ok && total[t] == 0) {  // nothing for this tile: its phases go by in order all the same
            ok = flush(t) && (!fresh || wait(q_full + t, n & 1, 2)) &&
                 (n == 0 || wait(o_empty + t, (n - 1) & 1, 1));
            tc::commit(q_empty + t);
          }
      }
      if (ok) ok = flush(0) && flush(1);
      settle();
      tc::commit(drain);
      if (!tc::mbar_wait(drain, 0, 1u << 16)) give_up(1);
    }
    __syncwarp();
  } else if (warp < kOutWarp) {
    // ---- weights: a row a thread
    const int t = warp >> 2, row = tid & 127, tr = row / G;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + lanes + kColS + t * 128, o_at = tmem + lanes + kColO + t * 128;
    uint32_t s_par = 0;
    for (int n = 0;; ++n) {
      if (!warp_wait(item_full + n % kItemSlots, item_par(n), 1)) break;
      const Item* ip = item_at(n);
      const int valid = ip->valid, p0 = ip->p0 + t * tpt, nt = t == 0 ? ip->n0 : ip->n1, ns = ip->ns, w0 = ip->w0,
                w1 = ip->w1;
      const Span span = ip->t[t];
      __syncwarp();
      if (lane == 0) arrive(item_empty + n % kItemSlots);
      if (!valid) break;
      float m = -INFINITY, l = 0.f;  // the maximum in use (log2), the weights' sum
      const int pr = p0 + tr;
      bool ok = true;
      for (int kt = ns > 0 ? 0 : w0; kt < w1; kt = kt + 1 == ns ? w0 : kt + 1) {
        if (!span.has(kt)) continue;
        if (!(ok = warp_wait(s_full + t, s_par, 1))) break;
        s_par ^= 1u;
        tc::fence_after();
        __syncwarp();
        const int j0 = kt * kKeys;
        const bool full = p0 >= j0 + kKeys - 1 &&
                          (a.view.window == 0 || p0 + nt - a.view.window <= j0 || j0 + kKeys <= a.view.sinks);
        // columns of the tile that the row sees: [0, hi) but [sink, lo)
        const int hi = pr + 1 - j0, lo = a.view.window > 0 ? pr + 1 - a.view.window - j0 : -1, sink = a.view.sinks - j0;
        auto seen = [&](int c) { return bits(0, hi - c) & ~bits(sink - c, lo - c); };
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float r[32];
          tc::tmem_ld32(s_at + 32 * c, r);
          if (!full) {
            const uint32_t see = seen(32 * c);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see >> i & 1u)) r[i] = -INFINITY;
          }
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = fmaxf(r[i], r[i + 4]);
#pragma unroll
          for (int i = 8; i < 32; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = max3(x[k], r[i + k], r[i + k + 4]);
          top = max3(top, max3(x[0], x[1], x[2]), x[3]);
        }
        top *= scale_log2;
        // a maximum far above the one in use takes its place
        if (__any_sync(0xffffffffu, top > m + kLazy)) {
          const float next = top > m + kLazy ? top : m;
          if (__any_sync(0xffffffffu, m != -INFINITY)) {
            const float f = next == m ? 1.f : ex2_approx(m - next);
            l *= f;
#pragma unroll 1
            for (int c = 0; c < a.d; c += 32) {
              float r[32];
              tc::tmem_ld32(o_at + c, r);
              uint32_t w[2][16];
#pragma unroll
              for (int i = 0; i < 32; ++i) w[i >> 4][i & 15] = __float_as_uint(r[i] * f);
              tmem_st16_start(o_at + c, w[0]);
              tmem_st16_start(o_at + c + 16, w[1]);
            }
          }
          m = next;
        }
        const float base = m == -INFINITY ? 0.f : -m;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float r[32];
          uint32_t w[16];
          tc::tmem_ld32(s_at + 32 * c, r);
          if (!full) {
            const uint32_t see = seen(32 * c);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see >> i & 1u)) r[i] = -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = fma2(make_float2(r[2 * i], r[2 * i + 1]),
                                  make_float2(scale_log2, scale_log2), make_float2(base, base));
            const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
            sum = fma2(p, make_float2(1.f, 1.f), sum);
            w[i] = pack_bf16(p.x, p.y);
          }
          tmem_st16_start(s_at + 16 * c, w);  // over scores that are used up
        }
        l += sum.x + sum.y;
        tmem_st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) arrive(p_full + t);
      }
      if (!ok || (n > 0 && !warp_wait(o_empty + t, (n - 1) & 1, 1))) break;
      stat[t * 128 + row] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) arrive(st_full + t);
    }
  } else if (warp < kMmaWarp) {
    // ---- outputs: a row a thread
    const int row = tid & 127, tr = row / G, hr = row - tr * G;
    const uint32_t o_at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kColO;
    uint32_t o_par[2] = {0, 0};
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!warp_wait(item_full + n % kItemSlots, item_par(n), 1)) break;
      const Item it = *item_at(n);
      __syncwarp();
      if (lane == 0) arrive(item_empty + n % kItemSlots);
      if (!it.valid) break;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!(ok = warp_wait(st_full + t, n & 1, 1))) break;
        const float2 s = stat[t * 128 + row];
        const bool some = it.t[t].count() > 0;
        if (some) {
          if (!(ok = warp_wait(o_full + t, o_par[t], 1))) break;
          o_par[t] ^= 1u;
          tc::fence_after();
        }
        const bool live = tr < tpt && tr < (t == 0 ? it.n0 : it.n1);
        const long long tok = it.q0 + t * tpt + tr;
        const int head = it.hk * G + hr;
        __nv_bfloat16* out = a.out + (tok * a.Hq + head) * a.d;
        const float inv = s.y == 0.f ? 0.f : 1.f / s.y;
        bool odd = false;
        for (int c = 0; c < a.d; c += 32) {
          float r[32] = {};
          __syncwarp();  // the load wants the lanes together, which a store of some of them may part
          if (some) tc::tmem_ld32(o_at + t * 128 + c, r);
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            if (c + i >= a.d) break;
            float2 f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              f[k] = s.y == 0.f ? make_float2(0.f, 0.f)
                                : make_float2(r[i + 2 * k] * inv, r[i + 2 * k + 1] * inv);
              odd |= !(fabsf(f[k].x) <= 3.4e38f) || !(fabsf(f[k].y) <= 3.4e38f);
            }
            if (live) *reinterpret_cast<uint4*>(out + c + i) = narrow8(f);
          }
        }
        if (live && a.lse != nullptr)
          a.lse[tok * a.Hq + head] = s.y == 0.f ? -INFINITY : (s.x + log2f(s.y)) * attn::kLn2;
        tc::fence_before();
        __syncwarp();
        if (lane == 0) arrive(o_empty + t);
        // rows that are not finite again, one after the other
        for (unsigned rest = __ballot_sync(0xffffffffu, odd && live); rest != 0; rest &= rest - 1) {
          const int r2 = 32 * (warp & 3) + __ffs(rest) - 1, tr2 = r2 / G;
          const long long tok2 = it.q0 + t * tpt + tr2;
          const int head2 = it.hk * G + r2 - tr2 * G;
          const __nv_bfloat16 *k = a.k + (long long)it.k0 * a.ks + it.hk * a.d, *v = a.v + (long long)it.k0 * a.vs + it.hk * a.d;
          const attn::RowSum sum = attn::row_sum(
              a.q + tok2 * a.qs + (long long)head2 * a.d, a.d, negate ? -scale_log2 : scale_log2,
              attn::seen_by(a.view, it.p0 + t * tpt + tr2), [&](int j) { return k + j * a.ks; },
              [&](int j) { return v + j * a.vs; }, attn::WidenBf16());
          attn::put_row(sum, a.d, a.out + (tok2 * a.Hq + head2) * a.d, nullptr, 1.f);
        }
        __syncwarp();
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  __syncwarp();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

namespace {

bool head_map(CUtensorMap* m, const void* base, long long stride, int heads, int d, long long tokens, int box_heads,
              int box_tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)(tokens > 1 ? stride : (long long)heads * d) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  return make_map16(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int kHalves>
cudaError_t launch_tiles(const attn::PromptArgs& a, void* ws, cudaStream_t st) {
  const bool packed = a.cu != nullptr;
  const long long nq = packed ? (long long)a.T : (long long)a.B * a.T;
  const long long nk = packed ? (long long)a.Tk : (long long)a.B * a.Tk;
  const int G = a.Hq / a.Hkv, tpt = 128 / G, per = 2 * tpt, sms = device_sms();
  if (sms == 0) return cudaErrorNoDevice;
  const long long tiles = ((long long)a.T + per - 1) / per;
  const long long items = (packed ? tiles + a.B : tiles * a.B) * a.Hkv;  // (packed: an upper bound)
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  CUtensorMap q, k, v;
  if (!head_map(&q, a.q, a.qs, a.Hq, a.d, nq, G, tpt)) return cudaErrorInvalidValue;
  // without keys nothing is loaded by these
  if (!head_map(&k, nk > 0 ? a.k : a.q, nk > 0 ? a.ks : a.qs, a.Hkv, a.d, nk > 0 ? nk : nq, 1, kKeys) ||
      !head_map(&v, nk > 0 ? a.v : a.q, nk > 0 ? a.vs : a.qs, a.Hkv, a.d, nk > 0 ? nk : nq, 1, kKeys))
    return cudaErrorInvalidValue;
  const cudaError_t e = set_smem_limit_once<gdn_attn_tile_kernel<kHalves>>(Cfg<kHalves>::kSmem);
  if (e != cudaSuccess) return e;
  float c = a.scale * attn::kLog2e;
  const int negate = c < 0.f;  // as the sign of the queries
  c = std::max(negate ? -c : c, 0x1p-126f);  // (unseen scores are minus infinity, and 0 times that would not do)
  gdn_attn_tile_kernel<kHalves><<<(unsigned)std::min<long long>(items, sms), kThreads, Cfg<kHalves>::kSmem, st>>>(
      q, k, v, a, (int)items, tpt, c, negate, static_cast<int*>(ws));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn(const attn::PromptArgs& a, void* ws, cudaStream_t st) {
  return a.d <= 64 ? launch_tiles<1>(a, ws, st) : launch_tiles<2>(a, ws, st);
}

}  // namespace gdn
