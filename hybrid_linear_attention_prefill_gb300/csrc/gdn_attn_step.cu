// Attention of one token of every sequence over a paged cache (gdn_attn.cuh has the mathematics): a warp
// for each sequence and query head.
#include <cuda_fp8.h>

#include "gdn_attn.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kRowWarps = 4;

struct WidenE4m3 {
  __device__ __forceinline__ void operator()(const __nv_fp8_e4m3* p, int i, float2 (&f)[4]) const {
    const uint2 raw = *reinterpret_cast<const uint2*>(p + i);
    const uint32_t w[2] = {raw.x, raw.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
      f[j] = __half22float2(__half2(h));
    }
  }
};

}  // namespace

// grid: (sequences, blocks of four query heads)
template <class T, class Widen>
__global__ void __launch_bounds__(32 * kRowWarps)
gdn_attn_step_rows_kernel(const attn::StepArgs a, int* __restrict__ err) {
  const int warp = threadIdx.x >> 5;
  const int b = blockIdx.x, h = blockIdx.y * kRowWarps + warp;
  if (h >= a.Hq) return;
  const int hk = h / (a.Hq / a.Hkv);
  const __nv_bfloat16* q = a.q + b * a.qs + (long long)h * a.d;
  const long long most = (long long)a.W * a.page;
  const int n = a.lens[b] < most ? a.lens[b] : (int)most;
  auto at = [&](const void* c, long long stride, int j) -> const T* {
    const int block = a.table[b * a.table_stride + j / a.page];
    if (block < 0 || block >= a.blocks) {
      atomicOr(err, 64);
      return nullptr;
    }
    return static_cast<const T*>(c) + block * stride + ((long long)hk * a.page + j % a.page) * a.d;
  };
  const float ks = a.kscale != nullptr ? a.kscale[hk] : 1.f, vs = a.vscale != nullptr ? a.vscale[hk] : 1.f;
  const attn::RowSum r = attn::row_sum(
      q, a.d, a.scale * ks * attn::kLog2e, attn::seen_by(a.view, n - 1), [&](int j) { return at(a.kc, a.kbs, j); },
      [&](int j) { return at(a.vc, a.vbs, j); }, Widen());
  const long long row = (long long)b * a.Hq + h;
  attn::put_row(r, a.d, a.out + row * a.d, a.lse != nullptr ? a.lse + row : nullptr, vs);
}

size_t attn_step_workspace(int B, int Hq, int Hkv, int d) { return 256; }

cudaError_t launch_attn_step(const attn::StepArgs& a, bool e4m3, void* ws, cudaStream_t st) {
  const dim3 grid((unsigned)a.B, (unsigned)((a.Hq + kRowWarps - 1) / kRowWarps));
  int* err = static_cast<int*>(ws);
  if (e4m3)
    gdn_attn_step_rows_kernel<__nv_fp8_e4m3, WidenE4m3><<<grid, 32 * kRowWarps, 0, st>>>(a, err);
  else
    gdn_attn_step_rows_kernel<__nv_bfloat16, attn::WidenBf16><<<grid, 32 * kRowWarps, 0, st>>>(a, err);
  return cudaGetLastError();
}

}  // namespace gdn
