// Root-mean-square norm with the residual's addition, to bf16 or to e4m3 with scales (sm_103a):
//
//   r = x + residual,   y = r / sqrt(mean(r^2) + eps) w,
//   e4m3: scale = max(max |y|, 2^-96) / 448 over a row or a group of columns, q = y / scale.
//
// Every element is read and written once for a handful of operations, so HBM bandwidth bounds it
// (one row: the latency of the loads and of the block's reductions).  A row stays in registers
// between its two reductions; a block for each few rows lets the SM's other blocks load meanwhile.
// 16,384 rows of 4,096 columns, bf16 in and out: 79.9 us, 6.72 TB/s; 4,096 rows to e4m3 in groups
// of 128: 22.4 us.  (Persistent blocks with the next rows on their way into shared memory: 89.4 us
// for the former.)
#include <cuda_fp8.h>

#include "gdn_internal.h"
#include "gdn_vec.cuh"

namespace gdn {

namespace {

constexpr int kNormMinThreads = 128;
constexpr int kRowShift = 12;  // groups are 2^gshift vectors of eight columns; this one holds the longest row

// The largest magnitude of three, or NaN.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

}  // namespace

// TPR threads a row (a power of two, 32..1024), VPT vectors of eight columns a thread; vector v of
// the row belongs to thread v % TPR, so a group of 32, 64 or 128 columns is 4, 8 or 16 consecutive
// lanes.  Blocks of max(TPR, 128) threads.
template <int VPT, bool E4M3>
__global__ void __launch_bounds__(1024)
gdn_add_norm_kernel(const __nv_bfloat16* __restrict__ x, long long xs, const __nv_bfloat16* residual,
                    const __nv_bfloat16* __restrict__ weight, __nv_bfloat16* residual_out, void* __restrict__ out,
                    float* __restrict__ scales, int rows, int D, int tpr, int gshift, int ngroups, float inv_d,
                    float eps) {
  __shared__ float part[32];
  __shared__ uint32_t part_max[32];
  const int nv = D / 8;
  const int rib = threadIdx.x / tpr, tid = threadIdx.x - rib * tpr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = tpr >> 5, w0 = rib * wpr;  // this row's warps in the block
  const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + rib;
  const bool live = row < rows;

  float2 r[VPT][4];
  float2 sq = make_float2(0.f, 0.f);
  uint4 xr[VPT], rr[VPT], wr[VPT];  // every load of the row before any use
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = tid + j * tpr;
    xr[j] = rr[j] = wr[j] = make_uint4(0, 0, 0, 0);
    if (live && v < nv) {
      xr[j] = *reinterpret_cast<const uint4*>(x + row * xs + 8 * v);
      if (residual != nullptr) rr[j] = *reinterpret_cast<const uint4*>(residual + row * D + 8 * v);
      wr[j] = *reinterpret_cast<const uint4*>(weight + 8 * v);
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = tid + j * tpr;
    widen8(xr[j], r[j]);
    if (residual != nullptr) {
      float2 f[4];
      widen8(rr[j], f);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[j][i] = fma2(r[j][i], make_float2(1.f, 1.f), f[i]);
    }
    if (residual_out != nullptr && live && v < nv)
      *reinterpret_cast<uint4*>(residual_out + row * D + 8 * v) = narrow8(r[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) sq = fma2(r[j][i], r[j][i], sq);
  }
  float ss = sq.x + sq.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (wpr > 1) {
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = lane < wpr ? part[w0 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  const float rstd = rsqrtf(fmaf(ss, inv_d, eps));

  // y in place; its largest magnitude as bits (a NaN's are above every number's, so it stays)
  uint32_t mx[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = tid + j * tpr;
    float big = 0.f;
    if (live && v < nv) {
      float2 w[4];
      widen8(wr[j], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[j][i] = mul2(mul2(r[j][i], make_float2(rstd, rstd)), w[i]);
        if (E4M3) big = max3_abs_nan(big, r[j][i].x, r[j][i].y);
      }
    }
    mx[j] = __float_as_uint(big);
  }
  if constexpr (!E4M3) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = tid + j * tpr;
      if (live && v < nv)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + row * D + 8 * v) = narrow8(r[j]);
    }
  } else {
    if (gshift == kRowShift) {  // one scale a row
#pragma unroll
      for (int j = 1; j < VPT; ++j) mx[0] = max(mx[0], mx[j]);
      mx[0] = __reduce_max_sync(0xffffffffu, mx[0]);
      if (wpr > 1) {
        if (lane == 0) part_max[warp] = mx[0];
        __syncthreads();
        mx[0] = __reduce_max_sync(0xffffffffu, lane < wpr ? part_max[w0 + lane] : 0u);
      }
#pragma unroll
      for (int j = 1; j < VPT; ++j) mx[j] = mx[0];
    } else {
      for (int o = 1; o < 1 << gshift; o <<= 1)
#pragma unroll
        for (int j = 0; j < VPT; ++j) mx[j] = max(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], o));
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = tid + j * tpr;
      if (!live || v >= nv) continue;
      // 2^-96 keeps scale and 1 / scale normal numbers; NaN bits compare above it
      const float scale = __uint_as_float(max(mx[j], __float_as_uint(0x1p-96f))) * (1.f / 448.f);
      const float inv = rcp_approx(scale);
      uint32_t q[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __nv_fp8x2_storage_t a =
            __nv_cvt_float2_to_fp8x2(mul2(r[j][2 * i], make_float2(inv, inv)), __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t b =
            __nv_cvt_float2_to_fp8x2(mul2(r[j][2 * i + 1], make_float2(inv, inv)), __NV_SATFINITE, __NV_E4M3);
        q[i] = (uint32_t)a | ((uint32_t)b << 16);
      }
      *reinterpret_cast<uint2*>(static_cast<unsigned char*>(out) + row * D + 8 * v) = make_uint2(q[0], q[1]);
      if ((v & ((1 << gshift) - 1)) == 0) scales[row * ngroups + (v >> gshift)] = scale;
    }
  }
}

template <int VPT>
static cudaError_t add_norm_v(const void* x, long long xs, const void* residual, const void* weight,
                              void* residual_out, void* out, float* scales, int rows, int D, int tpr, int group,
                              float eps, bool e4m3, cudaStream_t st) {
  using bf = __nv_bfloat16;
  const int threads = tpr < kNormMinThreads ? kNormMinThreads : tpr;
  const unsigned grid = (unsigned)(((long long)rows + threads / tpr - 1) / (threads / tpr));
  const int ngroups = group ? (D + group - 1) / group : 1;
  const int gshift = group == 32 ? 2 : group == 64 ? 3 : group == 128 ? 4 : kRowShift;
  const float inv_d = 1.f / (float)D;
  if (e4m3)
    gdn_add_norm_kernel<VPT, true><<<grid, threads, 0, st>>>(
        static_cast<const bf*>(x), xs, static_cast<const bf*>(residual), static_cast<const bf*>(weight),
        static_cast<bf*>(residual_out), out, scales, rows, D, tpr, gshift, ngroups, inv_d, eps);
  else
    gdn_add_norm_kernel<VPT, false><<<grid, threads, 0, st>>>(
        static_cast<const bf*>(x), xs, static_cast<const bf*>(residual), static_cast<const bf*>(weight),
        static_cast<bf*>(residual_out), out, scales, rows, D, tpr, gshift, ngroups, inv_d, eps);
  return cudaGetLastError();
}

cudaError_t launch_add_norm(const void* x, long long xs, const void* residual, const void* weight, void* residual_out,
                            void* out, float* scales, int rows, int D, int group, float eps, bool e4m3,
                            cudaStream_t st) {
  const int nv = D / 8;
  // Two vectors a thread; with few rows one, for the latency of a row (4,096 columns: 16,384 rows 79.7 us with two,
  // 80.9 with four; 4,096 rows 22.6 and 22.9, with one 26).
  const int want = rows < 2 * device_sms() ? 1 : 2;
  int tpr = 32;
  while (tpr < 1024 && want * tpr < nv) tpr <<= 1;
  const int vpt = (nv + tpr - 1) / tpr;
  auto run = [&](auto launch) {
    return launch(x, xs, residual, weight, residual_out, out, scales, rows, D, tpr, group, eps, e4m3, st);
  };
  if (vpt <= 1) return run(add_norm_v<1>);
  if (vpt <= 2) return run(add_norm_v<2>);
  if (vpt <= 4) return run(add_norm_v<4>);
  return cudaErrorInvalidValue;
}

}  // namespace gdn
