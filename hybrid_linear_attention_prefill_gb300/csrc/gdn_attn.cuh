// Attention: what the kernels for prompts and for single tokens share.
//
//   o = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale q.k_j),   over the keys j that the query sees
//
// A query at position p of its sequence sees j <= p and, with a window, of those the last `window` and
// the first `sinks`: two ranges, [0, sink_end) and [lo, hi).  Sums and weights are taken relative to the
// running maximum, in base 2 (scale log2(e) in the exponent).  A query that sees nothing, or nothing but
// weights of zero, gives 0 and a log of the sum of minus infinity.
#pragma once

#include "gdn_common.cuh"
#include "gdn_vec.cuh"

namespace gdn {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxDim = 128;  // of a head

struct View {
  int window, sinks;  // window 0: everything
};

// What the query at position p (below 0: nothing) sees.
struct Seen {
  int sink_end, lo, hi;
};
__host__ __device__ __forceinline__ Seen seen_by(const View& view, int p) {
  Seen s;
  s.hi = p + 1 > 0 ? p + 1 : 0;
  s.lo = view.window > 0 && s.hi > view.window ? s.hi - view.window : 0;
  s.sink_end = view.sinks < s.lo ? view.sinks : s.lo;
  return s;
}

// Operands of a prompt.  Dense: B sequences of T queries and Tk keys each; packed: T and Tk in all.
struct PromptArgs {
  const __nv_bfloat16 *q, *k, *v;
  long long qs, ks, vs;  // distances between tokens in elements
  const int32_t *cu, *cuk;
  __nv_bfloat16* out;
  float* lse;
  int B, T, Tk, Hq, Hkv, d;
  View view;
  float scale;
};

// Operands of a token of each of B sequences over the paged cache: pages of `page` tokens, a head's
// tokens of a page one after the other.
struct StepArgs {
  const __nv_bfloat16* q;
  long long qs;
  const void *kc, *vc;         // bf16 or e4m3 [blocks, Hkv, page, d]
  long long kbs, vbs;          // distances between blocks in elements
  const float *kscale, *vscale;  // e4m3: of each head
  const int32_t* table;
  long long table_stride;
  const int32_t* lens;
  __nv_bfloat16* out;
  float* lse;
  int B, Hq, Hkv, d, page, blocks, W;
  View view;
  float scale;
};

// One query by a warp, in fp32 throughout: `key(j)` and `value(j)` give the addresses of a visible
// token's d values, `widen(p, i, f)` eight of them from the i-th.  q: the query's values in global memory.
// Lane l ends with columns 4 l .. 4 l + 3 of the sum, and every lane with the maximum and the weights' sum.
struct RowSum {
  float o[4], m, l;
};
template <class Key, class Value, class Widen>
__device__ __forceinline__ RowSum row_sum(const __nv_bfloat16* q, int d, float scale_log2, const Seen& s, Key key, Value value,
                                          Widen widen) {
  const int lane = threadIdx.x & 31;
  RowSum r = {{0.f, 0.f, 0.f, 0.f}, -INFINITY, 0.f};
  for (int part = 0; part < 2; ++part) {
    const int begin = part == 0 ? 0 : s.lo, end = part == 0 ? s.sink_end : s.hi;
    for (int j0 = begin; j0 < end; j0 += 32) {
      const int j = j0 + lane;
      float t = -INFINITY;
      const auto* kp = j < end ? key(j) : nullptr;
      if (kp != nullptr) {
        float dot = 0.f;
        for (int c = 0; c < d; c += 8) {
          float2 f[4], g[4];
          widen(kp, c, f);
          widen8(*reinterpret_cast<const uint4*>(q + c), g);
#pragma unroll
          for (int i = 0; i < 4; ++i) dot = fmaf(g[i].x, f[i].x, fmaf(g[i].y, f[i].y, dot));
        }
        t = dot * scale_log2;
      }
      float top = t;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fmaxf(top, r.m);
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = exp2f(r.m - base), w = kp != nullptr ? exp2f(t - base) : 0.f;
      r.m = top;
      float sum = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      r.l = r.l * keep + sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) r.o[i] *= keep;
      const unsigned live = __ballot_sync(0xffffffffu, kp != nullptr);
      for (unsigned rest = live; rest != 0; rest &= rest - 1) {
        const int i = __ffs(rest) - 1;
        const float wi = __shfl_sync(0xffffffffu, w, i);
        if (4 * lane < d) {
          float2 f[4];
          widen(value(j0 + i), (4 * lane) & ~7, f);
          const float2 a = f[(lane & 1) * 2], b = f[(lane & 1) * 2 + 1];
          r.o[0] = fmaf(wi, a.x, r.o[0]);
          r.o[1] = fmaf(wi, a.y, r.o[1]);
          r.o[2] = fmaf(wi, b.x, r.o[2]);
          r.o[3] = fmaf(wi, b.y, r.o[3]);
        }
      }
    }
  }
  return r;
}

// Eight bf16 from the i-th.
struct WidenBf16 {
  __device__ __forceinline__ void operator()(const __nv_bfloat16* p, int i, float2 (&f)[4]) const {
    widen8(*reinterpret_cast<const uint4*>(p + i), f);
  }
};

// The sum's quotient to bf16, columns 4 lane .., and the log of the weights' sum.
__device__ __forceinline__ void put_row(const RowSum& r, int d, __nv_bfloat16* out, float* lse, float vscale) {
  const int lane = threadIdx.x & 31;
  const float inv = r.l == 0.f ? 0.f : vscale / r.l;
  if (4 * lane < d) {
    const float2 f[2] = {{r.l == 0.f ? 0.f : r.o[0] * inv, r.l == 0.f ? 0.f : r.o[1] * inv},
                         {r.l == 0.f ? 0.f : r.o[2] * inv, r.l == 0.f ? 0.f : r.o[3] * inv}};
    *reinterpret_cast<uint2*>(out + 4 * lane) = narrow4(f);
  }
  if (lse != nullptr && lane == 0) *lse = r.l == 0.f ? -INFINITY : (r.m + log2f(r.l)) * kLn2;
}

}  // namespace attn
}  // namespace gdn
