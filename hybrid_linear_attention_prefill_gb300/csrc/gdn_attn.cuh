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

}  // namespace attn
}  // namespace gdn
