// Selective state space scan of a prompt (sm_103a), token by token:
//
//   S_t = exp(s_t A) S_{t-1} + s_t x_t B_t^T,   y_t = (S_t C_t + D x_t) silu(z_t)
//
// A warp holds four rows of one (sequence, value head)'s dv x dk state in registers, dk / 32
// consecutive elements a lane, and walks the sequence's tokens; the row sums S C go by warp
// shuffles.  The chain of tokens bounds it.
#include "gdn_common.cuh"
#include "gdn_ssm.cuh"

namespace gdn {

namespace {
constexpr int kScanWarps = 4;
constexpr int kScanRows = 4;
}  // namespace

// grid: (B * dv / 16, Hv)
template <int DK>
__global__ void __launch_bounds__(32 * kScanWarps)
gdn_ssm_scan_kernel(const SsmArgs a, const int32_t* __restrict__ cu, const float* init, float* fin, int* err, int B,
                    int T) {
  constexpr int E = DK / 32, R = kScanRows;
  const int slices = a.dv / (kScanWarps * R);
  const int b = blockIdx.x / slices, h = blockIdx.y;
  const int hk = h / (a.Hv / a.Hk);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = ((blockIdx.x - b * slices) * kScanWarps + warp) * R;
  const SeqChunk q = seq_bounds(cu, b, T);
  if (cu != nullptr && h == 0 && blockIdx.x == b * slices && threadIdx.x == 0) {
    const int lo = cu[b], hi = cu[b + 1];
    if (lo < 0 || hi < lo || hi > T || (b == 0 && lo != 0) || (b == B - 1 && hi != T)) atomicOr(err, 8);
  }
  const size_t at = (((size_t)b * a.Hv + h) * a.dv + row) * DK + lane * E;
  const float skip = a.D != nullptr ? a.D[h] : 0.f, decay_rate = a.A[h];
  // the state, and what its last sums rounded away (a slowly decaying state adds thousands of tokens)
  float s[R][E], lost[R][E];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < E; ++e) s[r][e] = lost[r][e] = 0.f;
    if (init != nullptr) ssm_load_row<E>(init + at + r * DK, s[r]);
  }
  for (long long t = q.bos; t < q.bos + q.len; ++t) {
    const float step = ssm_dt(a, t, h);
    const float decay_m1 = expm1f(step * decay_rate);
    float bv[E], cv[E], y[R];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      bv[e] = __bfloat162float(a.Bm[t * a.bs + hk * DK + lane * E + e]);
      cv[e] = __bfloat162float(a.Cm[t * a.cs + hk * DK + lane * E + e]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float u = step * __bfloat162float(a.x[t * a.xs + h * a.dv + row + r]);
      y[r] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float inc = fmaf(decay_m1, s[r][e], u * bv[e]) + lost[r][e];
        const float next = s[r][e] + inc;
        lost[r][e] = inc - (next - s[r][e]);
        s[r][e] = next;
        y[r] = fmaf(s[r][e], cv[e], y[r]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) y[r] += __shfl_xor_sync(0xffffffffu, y[r], o);
    if (lane < R) {
      float v = y[0];
#pragma unroll
      for (int r = 1; r < R; ++r) v = lane == r ? y[r] : v;
      v = fmaf(skip, __bfloat162float(a.x[t * a.xs + h * a.dv + row + lane]), v);
      if (a.z != nullptr) v *= ssm_silu(__bfloat162float(a.z[t * a.zs + h * a.dv + row + lane]));
      a.out[((size_t)t * a.Hv + h) * a.dv + row + lane] = __float2bfloat16_rn(v);
    }
  }
  if (fin != nullptr) {
#pragma unroll
    for (int r = 0; r < R; ++r) ssm_store_row<E>(fin + at + r * DK, s[r]);
  }
}

size_t ssm_scan_workspace(int B, int T, int Hk, int Hv, int dk, int dv, int packed) { return 256; }

cudaError_t launch_ssm_scan(const SsmArgs& a, const int32_t* cu, const float* init, float* fin, void* ws, int B, int T,
                            int dk, cudaStream_t st) {
  const dim3 grid((unsigned)(B * (a.dv / (kScanWarps * kScanRows))), a.Hv);
  int* err = static_cast<int*>(ws);
  switch (dk) {
    case 32: gdn_ssm_scan_kernel<32><<<grid, 32 * kScanWarps, 0, st>>>(a, cu, init, fin, err, B, T); break;
    case 64: gdn_ssm_scan_kernel<64><<<grid, 32 * kScanWarps, 0, st>>>(a, cu, init, fin, err, B, T); break;
    default: gdn_ssm_scan_kernel<128><<<grid, 32 * kScanWarps, 0, st>>>(a, cu, init, fin, err, B, T); break;
  }
  return cudaGetLastError();
}

}  // namespace gdn
