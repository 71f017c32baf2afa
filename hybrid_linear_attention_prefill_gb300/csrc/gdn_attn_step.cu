// Attention of one token of every sequence over a paged cache (sm_103a; gdn_attn.cuh has the mathematics).
//
// Every visible key and value is read once for two products with a handful of queries: bandwidth bounds it.  The
// products are `mma.sync` ones, whose operands a warp loads straight into registers: nothing passes through shared
// memory, and a block's place in the cache is looked up once for 16 tokens.
//
//   scores   S^T [16 keys x 8 heads] = K Q^T      a lane's 16 bytes of a key are two steps' operand, since the sum over
//                                                 columns may go in any order that Q's operand shares
//   outputs  O^T [16 columns x 8 heads] += V^T P  a lane's 8 columns of four keys are four products' operand, pairs of
//                                                 keys put together by byte permutes; the weights, keys by heads as the
//                                                 scores come, are transposed by `movmatrix`
//
// Work.  A unit is 64 keys, 16 for each warp of a CTA.  The units of all sequences and key heads, one after the
// other, are dealt out in equal runs to as many CTAs as are resident, whatever the lengths; a warp keeps its own
// maxima, sums and outputs, and the CTA joins its warps' where a sequence (or the run) ends.  A sequence that is cut
// leaves partial sums in the workspace; the CTA that finishes its last part joins them in the runs' order, so
// results do not depend on which that is.  More than 16 heads of a key head are taken 16 at a time.
//
// A running maximum stays in use until a score is 2^8 above it (as for prompts), so that a step needs a vote and no
// exchange.  With an 8-bit cache the products are of fp16: every e4m3 value is one; the queries are scaled by a power
// of two a head to fit; weights are rounded to 11 bits instead of 8.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "gdn_attn.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

using attn::Seen;
using attn::StepArgs;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kBlock = 16;                  // keys a warp takes at a time
constexpr int kLeast = 2;                   // units that a run has at least, where there are so many
constexpr int kMaxHeads = 16;               // of a key head at a time
constexpr float kLazy = 8.f;
constexpr int kBadPage = 64;                // GDN_STATUS_BAD_PAGE

// Partial sums of a run's two ends: [2 runs][heads][d], then maxima and sums [2 runs][heads].
struct Work {
  float* sums;
  float2* stats;
  int* counters;  // parts of a (sequence, key head) that are done; zero between calls
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load_once(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// Eight values of the cache: as they are held, and as four pairs of 16 bits.
template <bool E4M3>
struct Piece;
template <>
struct Piece<false> {
  using Raw = uint4;
  static constexpr int kBytes = 2;
  __device__ static __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
  __device__ static __forceinline__ void pairs(const Raw& r, uint32_t (&w)[4]) {
    w[0] = r.x;
    w[1] = r.y;
    w[2] = r.z;
    w[3] = r.w;
  }
};
template <>
struct Piece<true> {
  using Raw = uint2;
  static constexpr int kBytes = 1;
  __device__ static __forceinline__ Raw zero() { return make_uint2(0, 0); }
  __device__ static __forceinline__ void pairs(const Raw& r, uint32_t (&w)[4]) {
    const uint32_t v[2] = {r.x, r.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
      w[i] = (uint32_t)h.x | (uint32_t)h.y << 16;
    }
  }
};

// What a part's sums (maximum, sum of weights) are multiplied by to be relative to `top`: nothing of a part that has
// seen nothing (or NaN, where its sum is that).
__device__ __forceinline__ float share(const float2& part, float top) {
  return part.x == -INFINITY ? part.y : ex2_approx(part.x - top);
}
__device__ __forceinline__ float4 add(const float4& x, float f, const float4& y) {
  return make_float4(fmaf(f, y.x, x.x), fmaf(f, y.y, x.y), fmaf(f, y.z, x.z), fmaf(f, y.w, x.w));
}

// A sequence's blocks of 16 keys with something to see: [0, s) and [a, z); the last is count - 1.
struct Blocks {
  int n, s, a, count;
  Seen seen;
};
__device__ __forceinline__ Blocks blocks_of(const StepArgs& a, int b) {
  Blocks r;
  const long long most = (long long)a.W * a.page;
  const int n = a.lens[b];
  r.n = n < 0 ? 0 : n < most ? n : (int)most;
  r.seen = attn::seen_by(a.view, r.n - 1);
  r.a = r.seen.lo / kBlock;
  r.s = min((r.seen.sink_end + kBlock - 1) / kBlock, r.a);
  r.count = r.s + (r.n + kBlock - 1) / kBlock - r.a;
  return r;
}
// (one at least, so that every row is written)
__device__ __forceinline__ int units_of(int blocks) { return blocks > kWarps ? (blocks + kWarps - 1) / kWarps : 1; }

}  // namespace

// NT: heads in eights; NC: columns in 32s; parts: heads of a key head in groups of 8 NT.
template <int NT, int NC, bool E4M3>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
gdn_attn_step_kernel(const StepArgs a, int groups, int heads, float scale_log2, Work work, int* __restrict__ err) {
  using P = Piece<E4M3>;
  using Raw = typename P::Raw;
  constexpr int NV = (NC + 1) / 2, kHeads = 8 * NT, kRow = 32 * NC + 4;  // a head's row in shared memory, padded
  __shared__ __align__(16) float so[kWarps][kHeads][kRow];
  __shared__ float2 stat[kWarps][kHeads];  // maximum (log2) and sum
  __shared__ int last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int G = a.Hq / a.Hkv, per_seq = a.Hkv * groups;

  // this CTA's run of units [u0, u1), and the sequence that it begins in
  long long total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    int u = b0 + lane < a.B ? units_of(blocks_of(a, b0 + lane).count) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    total += u;
  }
  total *= per_seq;
  const long long runs = min((long long)gridDim.x, max(1LL, total / kLeast));
  if (blockIdx.x >= runs) return;
  long long u0 = blockIdx.x * total / runs;
  const long long u1 = (blockIdx.x + 1) * total / runs;
  int b = -1;
  long long before = 0;  // units of the sequences before b
  for (int b0 = 0; b < 0 && b0 < a.B; b0 += 32) {
    const int u = b0 + lane < a.B ? units_of(blocks_of(a, b0 + lane).count) : 0;
    int sum = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + (long long)sum * per_seq > u0);
    if (hit != 0) {
      const int l = __ffs(hit) - 1;
      b = b0 + l;
      before += (long long)__shfl_sync(0xffffffffu, sum - u, l) * per_seq;
    } else {
      before += (long long)__shfl_sync(0xffffffffu, sum, 31) * per_seq;
    }
  }
  Blocks blk = blocks_of(a, b);
  int units = units_of(blk.count);
  int item = (int)((u0 - before) / units), first = (int)((u0 - before) - (long long)item * units);

  while (u0 < u1) {
    const int todo = (int)min((long long)(units - first), u1 - u0);
    const int hk = item / groups, h0 = hk * G + (item - hk * groups) * heads;
    const int nh = min(heads, (hk + 1) * G - h0);  // heads of this item

    // queries: head g of each eight, the columns that this lane's pieces of a key have
    uint32_t q[NT][NC][4];
    float scale[NT][2];  // of heads 2 c and 2 c + 1
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const __nv_bfloat16* row = a.q + b * a.qs + (long long)(h0 + 8 * t + g) * a.d;
      uint4 raw[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int col = 32 * i + 8 * c;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (8 * t + g < nh && col < a.d) raw[i] = *reinterpret_cast<const uint4*>(row + col);
      }
      scale[t][0] = scale[t][1] = scale_log2;
      if constexpr (E4M3) {
        // to below 2 by a power of two, which the scale takes back
        float top = 0.f;
        float2 f[NC][4];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          widen8(raw[i], f[i]);
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(f[i][k].x), fabsf(f[i][k].y)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = (int)(__float_as_uint(top) >> 23) - 127;
        e = e > 127 ? 0 : min(max(e, -100), 126);  // (infinities stay)
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) q[t][i][k] = pack_f16(f[i][k].x * down, f[i][k].y * down);
        const float ks = a.kscale[hk];
        scale[t][0] *= ks * __shfl_sync(0xffffffffu, up, 8 * c);  // lane 4 h has head h's
        scale[t][1] *= ks * __shfl_sync(0xffffffffu, up, 8 * c + 4);
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) Piece<false>::pairs(raw[i], q[t][i]);
      }
    }

    float o[NT][NV][4][4] = {};
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.f;

    const int32_t* table = a.table + b * a.table_stride;
    // the first key of this warp's i-th block, -1 behind the last
    auto key_of = [&](int i) {
      const int n = (first + i) * kWarps + warp;
      return i < todo && n < blk.count ? kBlock * (n < blk.s ? n : blk.a + n - blk.s) : -1;
    };
    auto page_of = [&](int key) { return key >= 0 ? table[key / a.page] : -1; };
    // whether a block is there, and its first token's place
    auto place = [&](int key, int page, long long& at) {
      if (key < 0) return false;
      if (page < 0 || page >= a.blocks) {
        if (lane == 0) atomicOr(err, kBadPage);
        return false;
      }
      at = ((long long)hk * a.page + key % a.page) * a.d;
      return true;
    };
    auto sees = [&](int key) { return key < blk.n && (key >= blk.seen.lo || key < blk.seen.sink_end); };
    auto sees_all = [&](int key) {
      return key + kBlock <= blk.n && (key >= blk.seen.lo || key + kBlock <= blk.seen.sink_end);
    };
    Raw kr[NC][2], vr[NV][4];
    auto load_k = [&](long long at, int page) {
      const unsigned char* p = static_cast<const unsigned char*>(a.kc) + ((long long)page * a.kbs + at) * P::kBytes;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int col = 32 * i + 8 * c;
#pragma unroll
        for (int r = 0; r < 2; ++r)
          kr[i][r] = col < a.d ? load_once(reinterpret_cast<const Raw*>(p + ((g + 8 * r) * a.d + col) * P::kBytes))
                               : P::zero();
      }
    };
    auto load_v = [&](long long at, int page, int key, bool all) {
      const unsigned char* p = static_cast<const unsigned char*>(a.vc) + ((long long)page * a.vbs + at) * P::kBytes;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = 64 * i + 8 * g;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 2 * c + (r & 1) + 8 * (r >> 1);
          // a value that is not seen is not read: zero times it might not be zero
          vr[i][r] = col < a.d && (all || sees(key + row))
                         ? load_once(reinterpret_cast<const Raw*>(p + (row * a.d + col) * P::kBytes))
                         : P::zero();
        }
      }
    };

    int key = key_of(0), page = page_of(key);
    int next_key = key_of(1), next_page = page_of(next_key);
    long long at = 0;
    bool there = place(key, page, at), all = there && sees_all(key);
    if (there) {
      load_k(at, page);
      load_v(at, page, key, all);
    }
    for (int i = 0; i < todo; ++i) {
      const int after_key = key_of(i + 2), after_page = page_of(after_key);
      long long next_at = 0;
      const bool next_there = place(next_key, next_page, next_at), next_all = next_there && sees_all(next_key);
      uint32_t p[NT][2];
      if (there) {
        float s[NT][4] = {};
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          uint32_t w0[4], w1[4];
          P::pairs(kr[j][0], w0);
          P::pairs(kr[j][1], w1);
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const uint32_t ka[4] = {w0[2 * st], w1[2 * st], w0[2 * st + 1], w1[2 * st + 1]};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if constexpr (E4M3) mma_f16(s[t], ka, q[t][j][2 * st], q[t][j][2 * st + 1]);
              else mma_bf16(s[t], ka, q[t][j][2 * st], q[t][j][2 * st + 1]);
            }
          }
        }
        if (next_there) load_k(next_at, next_page);
        bool above = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[t][k] *= scale[t][k & 1];
            if (!all && !sees(key + g + 8 * (k >> 1))) s[t][k] = -INFINITY;
            above |= s[t][k] > m[t][k & 1] + kLazy;
          }
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float top = fmaxf(s[t][k], s[t][k + 2]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              if (top > m[t][k]) {
                const float f = ex2_approx(m[t][k] - top);  // (0 at first)
                m[t][k] = top;
                l[t][k] *= f;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                  for (int x = 0; x < 4; ++x) o[t][v][x][k] *= f, o[t][v][x][k + 2] *= f;
              }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[k] = ex2_approx(s[t][k] - (m[t][k & 1] == -INFINITY ? 0.f : m[t][k & 1]));
            l[t][k & 1] += w[k];
          }
          p[t][0] = transposed(E4M3 ? pack_f16(w[0], w[1]) : pack_bf16(w[0], w[1]));
          p[t][1] = transposed(E4M3 ? pack_f16(w[2], w[3]) : pack_bf16(w[2], w[3]));
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          uint32_t w[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) P::pairs(vr[v][r], w[r]);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t va[4] = {__byte_perm(w[0][x], w[1][x], 0x5410), __byte_perm(w[0][x], w[1][x], 0x7632),
                                    __byte_perm(w[2][x], w[3][x], 0x5410), __byte_perm(w[2][x], w[3][x], 0x7632)};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if constexpr (E4M3) mma_f16(o[t][v][x], va, p[t][0], p[t][1]);
              else mma_bf16(o[t][v][x], va, p[t][0], p[t][1]);
            }
          }
        }
      } else if (next_there) {
        load_k(next_at, next_page);
      }
      if (next_there) load_v(next_at, next_page, next_key, next_all);
      key = next_key;
      there = next_there;
      all = next_all;
      next_key = after_key;
      next_page = after_page;
    }

    // the warps' sums together
    __syncthreads();  // the item before's are read
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float sum = l[t][k];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int h = 8 * t + 2 * c + k;
        if (g == 0) stat[warp][h] = make_float2(m[t][k], sum);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (64 * v + 8 * g >= 32 * NC) continue;
          float4* to = reinterpret_cast<float4*>(&so[warp][h][64 * v + 8 * g]);
          to[0] = make_float4(o[t][v][0][k], o[t][v][0][k + 2], o[t][v][1][k], o[t][v][1][k + 2]);
          to[1] = make_float4(o[t][v][2][k], o[t][v][2][k + 2], o[t][v][3][k], o[t][v][3][k + 2]);
        }
      }
    __syncthreads();
    const bool whole = first == 0 && todo == units;
    const int slot = 2 * blockIdx.x + (first == 0 ? 1 : 0);
    const float vs = E4M3 ? a.vscale[hk] : 1.f;
    // a head's quotient to its row (four columns), and the log of its sum
    auto put = [&](int h, int col, const float4& x, float top, float sum) {
      const long long row = (long long)b * a.Hq + h0 + h;
      const float inv = sum == 0.f ? 0.f : vs / sum;
      const float2 f[2] = {{x.x * inv, x.y * inv}, {x.z * inv, x.w * inv}};
      *reinterpret_cast<uint2*>(a.out + row * a.d + col) = sum == 0.f ? make_uint2(0, 0) : narrow4(f);
      if (a.lse != nullptr && col == 0) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * attn::kLn2;
    };
    const int quads = a.d / 4;
    for (int x = tid; x < nh * quads; x += kThreads) {
      const int h = x / quads, col = 4 * (x - h * quads);
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w][h].x);
      float4 all4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 st = stat[w][h];
        const float f = share(st, top);
        const float4 y = *reinterpret_cast<const float4*>(&so[w][h][col]);
        sum = fmaf(f, st.y, sum);
        all4 = add(all4, f, y);
      }
      if (whole) {
        put(h, col, all4, top, sum);
      } else {
        *reinterpret_cast<float4*>(work.sums + ((long long)slot * kMaxHeads + h) * attn::kMaxDim + col) = all4;
        if (col == 0) work.stats[slot * kMaxHeads + h] = make_float2(top, sum);
      }
    }
    if (!whole) {
      // the run that finishes the last part joins them all
      const long long start = before + (long long)item * units, end = start + units;  // the item's units
      auto run_of = [&](long long u) { return (int)(((u + 1) * runs - 1) / total); };
      const int r0 = run_of(start), r1 = run_of(end - 1);
      int* counter = work.counters + (long long)b * per_seq + item;
      __threadfence();
      __syncthreads();
      if (tid == 0) last = atomicAdd(counter, 1) == r1 - r0;
      __syncthreads();
      if (last) {
        __threadfence();
        if (tid == 0) *counter = 0;
        for (int x = tid; x < nh * quads; x += kThreads) {
          const int h = x / quads, col = 4 * (x - h * quads);
          float top = -INFINITY, sum = 0.f;
          for (int r = r0; r <= r1; ++r) top = fmaxf(top, __ldcg(&work.stats[(2 * r + (r == r0)) * kMaxHeads + h]).x);
          float4 all4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int r = r0; r <= r1; ++r) {
            const int from = (2 * r + (r == r0)) * kMaxHeads + h;
            const float2 st = __ldcg(&work.stats[from]);
            const float4 y = __ldcg(reinterpret_cast<const float4*>(work.sums + (long long)from * attn::kMaxDim + col));
            const float f = share(st, top);
            sum = fmaf(f, st.y, sum);
            all4 = add(all4, f, y);
          }
          put(h, col, all4, top, sum);
        }
      }
    }

    u0 += todo;
    first = 0;
    if (++item == per_seq) {
      item = 0;
      before += (long long)units * per_seq;
      if (++b == a.B) break;
      blk = blocks_of(a, b);
      units = units_of(blk.count);
    }
  }
}

namespace {

int resident(int heads, int sms) { return sms * (heads <= 8 ? 3 : 2); }

// Workspace: [256 B status words][partial sums][their maxima and sums][counters].  The places do not depend on the
// call, so that the counters are zero whatever call came before.
struct Layout {
  size_t stats, counters, total;
};
Layout layout(int B, int Hq, int Hkv, int sms) {
  const int G = Hq / Hkv, groups = (G + kMaxHeads - 1) / kMaxHeads;
  const size_t slots = 2 * (size_t)resident(1, sms) * kMaxHeads;
  Layout l;
  l.stats = 256 + slots * attn::kMaxDim * 4;
  l.counters = l.stats + slots * 8;
  l.total = l.counters + ((size_t)B * Hkv * groups * 4 + 255) / 256 * 256;
  return l;
}

template <int NT, bool E4M3>
void launch_step(const StepArgs& a, int nc, int groups, int heads, unsigned grid, Work w, int* err, cudaStream_t st) {
  const float c = a.scale * attn::kLog2e;
  switch (nc) {
    case 1: return gdn_attn_step_kernel<NT, 1, E4M3><<<grid, kThreads, 0, st>>>(a, groups, heads, c, w, err);
    case 2: return gdn_attn_step_kernel<NT, 2, E4M3><<<grid, kThreads, 0, st>>>(a, groups, heads, c, w, err);
    case 3: return gdn_attn_step_kernel<NT, 3, E4M3><<<grid, kThreads, 0, st>>>(a, groups, heads, c, w, err);
    default: return gdn_attn_step_kernel<NT, 4, E4M3><<<grid, kThreads, 0, st>>>(a, groups, heads, c, w, err);
  }
}

}  // namespace

size_t attn_step_workspace(int B, int Hq, int Hkv, int d) {
  const int sms = device_sms();
  return layout(B, Hq, Hkv, sms > 0 ? sms : 256).total;  // (without a device: enough for any)
}

cudaError_t launch_attn_step(const StepArgs& a, bool e4m3, void* ws, cudaStream_t st) {
  const int sms = device_sms();
  if (sms == 0) return cudaErrorNoDevice;
  const int G = a.Hq / a.Hkv, groups = (G + kMaxHeads - 1) / kMaxHeads, heads = (G + groups - 1) / groups;
  if ((long long)a.B * a.Hkv * groups > 0x3fffffffLL) return cudaErrorInvalidValue;
  const Layout l = layout(a.B, a.Hq, a.Hkv, sms);
  unsigned char* p = static_cast<unsigned char*>(ws);
  Work w = {reinterpret_cast<float*>(p + 256), reinterpret_cast<float2*>(p + l.stats),
            reinterpret_cast<int*>(p + l.counters)};
  int* err = static_cast<int*>(ws);
  const int nc = (a.d + 31) / 32;
  const unsigned grid = (unsigned)resident(heads, sms);
  auto run = [&](auto launch) { launch(a, nc, groups, heads, grid, w, err, st); };
  if (heads <= 8) e4m3 ? run(launch_step<1, true>) : run(launch_step<1, false>);
  else e4m3 ? run(launch_step<2, true>) : run(launch_step<2, false>);
  return cudaGetLastError();
}

}  // namespace gdn
