// Selective state space step, one token per sequence, the state updated in place (sm_103a):
//
//   s = softplus(dt + bias),  S <- exp(s A) S + s x B^T,  y = (S C + D x) silu(z)
//
// with S a dv x dk fp32 state per (sequence, value head).  The step reads and writes the state once
// (8 bytes an element) for five operations an element, so HBM bandwidth bounds it.  A warp holds
// whole state rows, dk / 32 consecutive elements a lane, a batch of rows in flight; the row sums
// S C go by warp shuffles.
#include "gdn_common.cuh"
#include "gdn_ssm.cuh"

namespace gdn {

namespace {
constexpr int kStepWarps = 8;
constexpr int kStepRows = 4;  // rows a warp has in flight together
}  // namespace

// One CTA per (sequence, value head).
template <int DK>
__global__ void __launch_bounds__(32 * kStepWarps)
gdn_ssm_step_kernel(const SsmArgs a, float* __restrict__ state) {
  constexpr int E = DK / 32, R = kStepRows;
  const int b = blockIdx.x / a.Hv, h = blockIdx.x - b * a.Hv;
  const int hk = h / (a.Hv / a.Hk);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float step = ssm_step_of(a, ssm_load_dt(a, b, h), ssm_bias(a, h));
  const SsmDecay decay = ssm_decay(step * a.A[h]);
  const float skip = a.D != nullptr ? a.D[h] : 0.f;
  float bv[E], cv[E];
  const __nv_bfloat16* br = a.Bm + b * a.bs + hk * DK + lane * E;
  const __nv_bfloat16* cr = a.Cm + b * a.cs + hk * DK + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    bv[e] = __bfloat162float(br[e]);
    cv[e] = __bfloat162float(cr[e]);
  }
  const int rows = a.dv / kStepWarps;  // 4, 8 or 16 a warp
  float* p0 = state + ((size_t)blockIdx.x * a.dv + warp * rows) * DK + lane * E;
  // this lane's x and gate value of the warp's rows
  const __nv_bfloat16* xr = a.x + b * a.xs + h * a.dv + warp * rows;
  const float xv = lane < rows ? __bfloat162float(xr[lane]) : 0.f;
  float zv = 0.f;
  if (a.z != nullptr && lane < rows) zv = __bfloat162float(a.z[b * a.zs + h * a.dv + warp * rows + lane]);
  float s[R][E], next[R][E];
#pragma unroll
  for (int r = 0; r < R; ++r) ssm_load_row<E>(p0 + r * DK, s[r]);
  for (int j = 0; j < rows; j += R) {
    if (j + R < rows) {  // the next rows' loads before this batch's arithmetic
#pragma unroll
      for (int r = 0; r < R; ++r) ssm_load_row<E>(p0 + (j + R + r) * DK, next[r]);
    }
    float y[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float u = step * __shfl_sync(0xffffffffu, xv, j + r);
      y[r] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s[r][e] = ssm_decayed(decay, s[r][e], u * bv[e]);
        y[r] = fmaf(s[r][e], cv[e], y[r]);
      }
      ssm_store_row<E>(p0 + (j + r) * DK, s[r]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) y[r] += __shfl_xor_sync(0xffffffffu, y[r], o);
    if (lane >= j && lane < j + R) {
      float v = y[0];
#pragma unroll
      for (int r = 1; r < R; ++r) v = lane == j + r ? y[r] : v;
      v = fmaf(skip, xv, v);
      if (a.z != nullptr) v *= silu2(make_float2(zv, zv)).x;
      a.out[(size_t)blockIdx.x * a.dv + warp * rows + lane] = __float2bfloat16_rn(v);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) s[r][e] = next[r][e];
  }
}

cudaError_t launch_ssm_step(const SsmArgs& a, float* state, int B, int dk, cudaStream_t st) {
  const unsigned grid = (unsigned)(B * a.Hv);
  switch (dk) {
    case 32: gdn_ssm_step_kernel<32><<<grid, 32 * kStepWarps, 0, st>>>(a, state); break;
    case 64: gdn_ssm_step_kernel<64><<<grid, 32 * kStepWarps, 0, st>>>(a, state); break;
    default: gdn_ssm_step_kernel<128><<<grid, 32 * kStepWarps, 0, st>>>(a, state); break;
  }
  return cudaGetLastError();
}

}  // namespace gdn
