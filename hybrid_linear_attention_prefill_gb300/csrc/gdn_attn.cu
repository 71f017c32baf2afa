// Attention of prompts (gdn_attn.cuh has the mathematics): a warp for each query and head.
#include "gdn_attn.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kRowWarps = 4;

}  // namespace

// grid: (blocks of four tokens, query heads)
__global__ void __launch_bounds__(32 * kRowWarps)
gdn_attn_rows_kernel(const attn::PromptArgs a, long long ntok) {
  __shared__ __align__(16) float qf[kRowWarps][attn::kMaxDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * kRowWarps + warp;
  if (t >= ntok) return;
  int b;
  if (a.cu == nullptr) {
    b = (int)(t / a.T);
  } else {  // the last sequence that starts at or before t
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.cu[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
  }
  const SeqChunk sq = seq_bounds(a.cu, b, a.T), sk = seq_bounds(a.cuk, b, a.Tk);
  if (t < sq.bos || t >= sq.bos + sq.len) return;
  const int h = blockIdx.y, hk = h / (a.Hq / a.Hkv);
  const __nv_bfloat16* q = a.q + t * a.qs + (long long)h * a.d;
  for (int c = lane; c < a.d; c += 32) qf[warp][c] = __bfloat162float(q[c]);
  __syncwarp();
  const int p = (int)(t - sq.bos) + sk.len - sq.len;
  const __nv_bfloat16 *k = a.k + sk.bos * a.ks + hk * a.d, *v = a.v + sk.bos * a.vs + hk * a.d;
  const attn::RowSum r = attn::row_sum(
      qf[warp], a.d, a.scale * attn::kLog2e, attn::seen_by(a.view, p), [&](int j) { return k + j * a.ks; },
      [&](int j) { return v + j * a.vs; }, attn::WidenBf16());
  attn::put_row(r, a.d, a.out + (t * a.Hq + h) * a.d, a.lse != nullptr ? a.lse + t * a.Hq + h : nullptr, 1.f);
}

cudaError_t launch_attn(const attn::PromptArgs& a, void* ws, cudaStream_t st) {
  (void)ws;
  const long long ntok = a.cu != nullptr ? (long long)a.T : (long long)a.B * a.T;
  gdn_attn_rows_kernel<<<dim3((unsigned)((ntok + kRowWarps - 1) / kRowWarps), (unsigned)a.Hq), 32 * kRowWarps, 0, st>>>(
      a, ntok);
  return cudaGetLastError();
}

}  // namespace gdn
