// Selective state space step, one token per sequence, the state updated in place (sm_103a):
//
//   s = softplus(dt + bias),  S <- exp(s A) S + s x B^T,  y = (S C + D x) silu(z)
//
// with S a dv x dk fp32 state per (sequence, value head).  The step reads and writes the state once
// (8 bytes an element) for five operations an element, so HBM bandwidth bounds it.  A warp holds
// whole state rows, dk / 32 consecutive elements a lane, a batch of rows in flight; the row sums
// S C go by warp shuffles.  128 sequences of 32 heads, 128 x 128: 82.4 us, 6.57 TB/s.
#include "gdn_internal.h"
#include "gdn_ssm.cuh"

namespace gdn {

namespace {
constexpr int kStepWarps = 8;
constexpr int kStepRows = 4;  // rows a warp has in flight together
}  // namespace

// grid: ((sequence, value head), dv / (8 rows)); `rows` state rows a warp, 4, 8 or 16.
template <int DK>
__global__ void __launch_bounds__(32 * kStepWarps)
gdn_ssm_step_kernel(const SsmArgs a, float* __restrict__ state, int rows) {
  constexpr int E = DK / 32, R = kStepRows;
  const int b = blockIdx.x / a.Hv, h = blockIdx.x - b * a.Hv;
  const int hk = h / (a.Hv / a.Hk);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = (blockIdx.y * kStepWarps + warp) * rows;
  // every load before the first use of one
  float* p0 = state + ((size_t)blockIdx.x * a.dv + row0) * DK + lane * E;
  float s[R][E], next[R][E];
#pragma unroll
  for (int r = 0; r < R; ++r) ssm_load_row<E>(p0 + r * DK, s[r]);
  const uint32_t raw_dt = ssm_load_dt(a, b, h);
  const float bias = ssm_bias(a, h), rate = a.A[h];
  const float skip = a.D != nullptr ? a.D[h] : 0.f;
  __nv_bfloat16 br[E], cr[E], xr = __float2bfloat16_rn(0.f), zr = xr;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    br[e] = a.Bm[b * a.bs + hk * DK + lane * E + e];
    cr[e] = a.Cm[b * a.cs + hk * DK + lane * E + e];
  }
  if (lane < rows) {  // this lane's x and gate value of the warp's rows
    xr = a.x[b * a.xs + h * a.dv + row0 + lane];
    if (a.z != nullptr) zr = a.z[b * a.zs + h * a.dv + row0 + lane];
  }
  const float xv = __bfloat162float(xr), zv = __bfloat162float(zr);
  float bv[E], cv[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    bv[e] = __bfloat162float(br[e]);
    cv[e] = __bfloat162float(cr[e]);
  }
  const float step = ssm_step_of(a, raw_dt, bias);
  const SsmDecay decay = ssm_decay(step * rate);
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
      a.out[(size_t)blockIdx.x * a.dv + row0 + lane] = __float2bfloat16_rn(v);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) s[r][e] = next[r][e];
  }
}

cudaError_t launch_ssm_step(const SsmArgs& a, float* state, int B, int dk, cudaStream_t st) {
  // A warp streams up to 16 rows, the next four's loads in flight; with too few heads to fill the device four each,
  // so that more SMs share the state.
  const unsigned heads = (unsigned)(B * a.Hv);
  int rows = a.dv / kStepWarps;
  while (rows > kStepRows && heads * (a.dv / (kStepWarps * rows)) < 2u * (unsigned)device_sms()) rows >>= 1;
  const dim3 grid(heads, a.dv / (kStepWarps * rows));
  switch (dk) {
    case 32: gdn_ssm_step_kernel<32><<<grid, 32 * kStepWarps, 0, st>>>(a, state, rows); break;
    case 64: gdn_ssm_step_kernel<64><<<grid, 32 * kStepWarps, 0, st>>>(a, state, rows); break;
    default: gdn_ssm_step_kernel<128><<<grid, 32 * kStepWarps, 0, st>>>(a, state, rows); break;
  }
  return cudaGetLastError();
}

}  // namespace gdn
