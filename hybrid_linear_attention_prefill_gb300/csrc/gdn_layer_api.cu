// C ABI of the operators around the recurrence: causal convolution, selective state space scan (each
// for prompts and single tokens) and the norm with the residual's addition.  Argument checks here,
// kernels in gdn_conv.cu, gdn_ssm_scan.cu, gdn_ssm_step.cu and gdn_norm.cu.
#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_ssm.cuh"

namespace gdn {
cudaError_t launch_conv(const void*, long long, const void*, const void*, const int32_t*, const void*, void*, void*,
                        int, int, int, int, int, bool, cudaStream_t);
cudaError_t launch_conv_step(const void*, long long, const void*, const void*, void*, void*, int, int, int, bool,
                             cudaStream_t);
cudaError_t launch_add_norm(const void*, long long, const void*, const void*, void*, void*, float*, int, int, int,
                            float, bool, cudaStream_t);
cudaError_t launch_ssm_step(const SsmArgs&, float*, int, int, cudaStream_t);
size_t ssm_scan_workspace(int, int, int, int, int, int, int);
int ssm_scan_polls(int);
cudaError_t launch_ssm_scan(const SsmArgs&, const int32_t*, const float*, float*, void*, int, int, int, cudaStream_t);
}  // namespace gdn

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + nb && y < x + na;
}

// A bf16 operand of `tokens` rows of `width` elements: GDN_OK, or what is wrong with it.
int check_rows(const void* p, long long stride, long long tokens, long long width) {
  if (p == nullptr) return GDN_ERR_ARG;
  if (tokens > 1 && stride < width) return GDN_ERR_ARG;
  if (!aligned(p, 16) || (tokens > 1 && stride % 8 != 0)) return GDN_ERR_ALIGN;
  return GDN_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? GDN_OK : gdn::set_cuda_error(e, GDN_ERR_LAUNCH); }

bool conv_sizes_ok(int B, int T, int C, int K, unsigned flags) {
  return B >= 0 && T >= 0 && C > 0 && C % 8 == 0 && K >= 2 && K <= 4 && (flags & ~GDN_CONV_SILU) == 0;
}

bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

bool ssm_sizes_ok(int B, int T, int Hk, int Hv, int dk, int dv) {
  return B >= 0 && T >= 0 && Hk > 0 && Hv > 0 && Hv % Hk == 0 && Hv <= 65535 && dim_ok(dk) && dim_ok(dv);
}

int ssm_operands(const gdn::SsmArgs& a, long long tokens, int dk) {
  if (a.A == nullptr || a.dt == nullptr || a.out == nullptr) return GDN_ERR_ARG;
  int rc;
  if ((rc = check_rows(a.x, a.xs, tokens, (long long)a.Hv * a.dv)) != GDN_OK ||
      (rc = check_rows(a.Bm, a.bs, tokens, (long long)a.Hk * dk)) != GDN_OK ||
      (rc = check_rows(a.Cm, a.cs, tokens, (long long)a.Hk * dk)) != GDN_OK)
    return rc;
  if (a.z != nullptr && (rc = check_rows(a.z, a.zs, tokens, (long long)a.Hv * a.dv)) != GDN_OK) return rc;
  if (tokens > 1 && a.dts < a.Hv) return GDN_ERR_ARG;
  if (!aligned(a.out, 16) || !aligned(a.dt, a.dt_f32 ? 4 : 2) || !aligned(a.A, 4) || !aligned(a.D, 4) ||
      !aligned(a.dt_bias, 4))
    return GDN_ERR_ALIGN;
  return GDN_OK;
}

gdn::SsmArgs ssm_args(const void* x, long long xs, const void* dt, long long dts, const float* A, const void* Bm,
                      long long bs, const void* Cm, long long cs, const float* D, const void* z, long long zs,
                      const float* dt_bias, void* out, int Hk, int Hv, int dv, unsigned flags) {
  using bf = __nv_bfloat16;
  gdn::SsmArgs a;
  a.x = static_cast<const bf*>(x);
  a.dt = dt;
  a.A = A;
  a.Bm = static_cast<const bf*>(Bm);
  a.Cm = static_cast<const bf*>(Cm);
  a.D = D;
  a.z = static_cast<const bf*>(z);
  a.dt_bias = dt_bias;
  a.out = static_cast<bf*>(out);
  a.xs = xs;
  a.dts = dts;
  a.bs = bs;
  a.cs = cs;
  a.zs = zs;
  a.Hk = Hk;
  a.Hv = Hv;
  a.dv = dv;
  a.softplus = (flags & GDN_SSM_SOFTPLUS) != 0;
  a.dt_f32 = (flags & GDN_SSM_DT_F32) != 0;
  return a;
}

}  // namespace

extern "C" {

int gdn_conv(const gdn_conv_args* args) {
  gdn::clear_cuda_error();
  if (args == nullptr) return GDN_ERR_ARG;
  const auto& [x, x_stride, weight, bias, cu_seqlens, init_state, out, final_state, B, T, C, K, flags, stream] = *args;
  if (!conv_sizes_ok(B, T, C, K, flags)) return GDN_ERR_ARG;
  if (B == 0) return GDN_OK;
  const long long ntok = cu_seqlens != nullptr ? (long long)T : (long long)B * T;
  if (ntok > 0x7fffffffLL) return GDN_ERR_ARG;
  if (ntok == 0 && final_state == nullptr) return GDN_OK;
  if (ntok > 0) {
    if (weight == nullptr || out == nullptr) return GDN_ERR_ARG;
    const int rc = check_rows(x, x_stride, ntok, C);
    if (rc != GDN_OK) return rc;
  }
  for (const void* p : {weight, bias, (const void*)init_state, (const void*)out, (const void*)final_state})
    if (!aligned(p, 16)) return GDN_ERR_ALIGN;
  if (!aligned(cu_seqlens, 4)) return GDN_ERR_ALIGN;
  const size_t ns = (size_t)B * (K - 1) * C * 2;
  if (overlap(init_state, ns, final_state, ns)) return GDN_ERR_ARG;
  if (ntok > 0 && overlap(x, ((size_t)(ntok - 1) * x_stride + C) * 2, out, (size_t)ntok * C * 2)) return GDN_ERR_ARG;
  return done(gdn::launch_conv(x, x_stride, weight, bias, cu_seqlens, init_state, out, final_state, B, T, (int)ntok, C,
                               K, (flags & GDN_CONV_SILU) != 0, static_cast<cudaStream_t>(stream)));
}

int gdn_conv_step(const gdn_conv_step_args* args) {
  gdn::clear_cuda_error();
  if (args == nullptr) return GDN_ERR_ARG;
  const auto& [x, x_stride, weight, bias, state, out, B, C, K, flags, stream] = *args;
  if (!conv_sizes_ok(B, 1, C, K, flags)) return GDN_ERR_ARG;
  if (B == 0) return GDN_OK;
  if (weight == nullptr || state == nullptr || out == nullptr) return GDN_ERR_ARG;
  const int rc = check_rows(x, x_stride, B, C);
  if (rc != GDN_OK) return rc;
  for (const void* p : {weight, bias, (const void*)state, (const void*)out})
    if (!aligned(p, 16)) return GDN_ERR_ALIGN;
  return done(gdn::launch_conv_step(x, x_stride, weight, bias, state, out, B, C, K, (flags & GDN_CONV_SILU) != 0,
                                    static_cast<cudaStream_t>(stream)));
}

size_t gdn_ssm_workspace_bytes(int B, int T, int Hk, int Hv, int dk, int dv, int packed) {
  if (!ssm_sizes_ok(B, T, Hk, Hv, dk, dv)) return 0;
  return gdn::ssm_scan_workspace(B, T, Hk, Hv, dk, dv, packed);
}

int gdn_debug_ssm_wait_polls(int polls) { return gdn::ssm_scan_polls(polls); }

int gdn_ssm_scan(const gdn_ssm_scan_args* args) {
  gdn::clear_cuda_error();
  if (args == nullptr) return GDN_ERR_ARG;
  const auto& [x, x_stride, dt, dt_stride, A, Bm, b_stride, Cm, c_stride, D, z, z_stride, dt_bias, cu_seqlens,
               init_state, out, final_state, B, T, Hk, Hv, dk, dv, flags, workspace_given, workspace_bytes, stream] =
      *args;
  if (!ssm_sizes_ok(B, T, Hk, Hv, dk, dv) || (flags & ~(GDN_SSM_SOFTPLUS | GDN_SSM_DT_F32)) != 0) return GDN_ERR_ARG;
  if (B == 0) return GDN_OK;
  const long long ntok = cu_seqlens != nullptr ? (long long)T : (long long)B * T;
  if (ntok > 0x7fffffffLL || (long long)B * 8 > 0x7fffffffLL) return GDN_ERR_ARG;
  const gdn::SsmArgs a = ssm_args(x, x_stride, dt, dt_stride, A, Bm, b_stride, Cm, c_stride, D, z, z_stride, dt_bias,
                                  out, Hk, Hv, dv, flags);
  if (ntok > 0) {
    const int rc = ssm_operands(a, ntok, dk);
    if (rc != GDN_OK) return rc;
  }
  if (!aligned(cu_seqlens, 4) || !aligned(init_state, 16) || !aligned(final_state, 16)) return GDN_ERR_ALIGN;
  if (ntok == 0 && final_state == nullptr) return GDN_OK;
  if (ntok == 0 && A == nullptr) return GDN_ERR_ARG;
  const size_t need = gdn::ssm_scan_workspace(B, T, Hk, Hv, dk, dv, cu_seqlens != nullptr);
  void* workspace = workspace_given;
  if (workspace == nullptr) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return gdn::set_cuda_error(e, GDN_ERR_LAUNCH);
    const int rc = gdn::ensure_ssm_workspace(dev, need, static_cast<cudaStream_t>(stream), &workspace);
    if (rc != GDN_OK) return rc;
  } else {
    if (!aligned(workspace, 256)) return GDN_ERR_ALIGN;
    if (workspace_bytes < need) return GDN_ERR_SCRATCH;
  }
  return done(gdn::launch_ssm_scan(a, cu_seqlens, init_state, final_state, workspace, B, T, dk,
                                   static_cast<cudaStream_t>(stream)));
}

int gdn_ssm_step(const gdn_ssm_step_args* args) {
  gdn::clear_cuda_error();
  if (args == nullptr) return GDN_ERR_ARG;
  const auto& [x, x_stride, dt, dt_stride, A, Bm, b_stride, Cm, c_stride, D, z, z_stride, dt_bias, state, out, B, Hk,
               Hv, dk, dv, flags, stream] = *args;
  if (!ssm_sizes_ok(B, 1, Hk, Hv, dk, dv) || (flags & ~(GDN_SSM_SOFTPLUS | GDN_SSM_DT_F32)) != 0) return GDN_ERR_ARG;
  if (B == 0) return GDN_OK;
  if ((long long)B * Hv > 0x7fffffffLL || state == nullptr) return GDN_ERR_ARG;
  const gdn::SsmArgs a = ssm_args(x, x_stride, dt, dt_stride, A, Bm, b_stride, Cm, c_stride, D, z, z_stride, dt_bias,
                                  out, Hk, Hv, dv, flags);
  const int rc = ssm_operands(a, B, dk);
  if (rc != GDN_OK) return rc;
  if (!aligned(state, 16)) return GDN_ERR_ALIGN;
  return done(gdn::launch_ssm_step(a, state, B, dk, static_cast<cudaStream_t>(stream)));
}

int gdn_add_norm(const gdn_add_norm_args* args) {
  gdn::clear_cuda_error();
  if (args == nullptr) return GDN_ERR_ARG;
  const auto& [x, x_stride, residual, weight, residual_out, out, scales, rows, D, group, eps, flags, stream] = *args;
  const bool e4m3 = (flags & GDN_NORM_E4M3) != 0;
  if (rows < 0 || D <= 0 || D % 8 != 0 || D > 32768 || (flags & ~GDN_NORM_E4M3) != 0) return GDN_ERR_ARG;
  if (group != 0 && (!e4m3 || (group != 32 && group != 64 && group != 128))) return GDN_ERR_ARG;
  if (rows == 0) return GDN_OK;
  if (weight == nullptr || out == nullptr || (e4m3 && scales == nullptr)) return GDN_ERR_ARG;
  const int rc = check_rows(x, x_stride, rows, D);
  if (rc != GDN_OK) return rc;
  for (const void* p : {residual, weight, (const void*)residual_out})
    if (!aligned(p, 16)) return GDN_ERR_ALIGN;
  if (!aligned(out, e4m3 ? 8 : 16) || !aligned(scales, 4)) return GDN_ERR_ALIGN;
  return done(gdn::launch_add_norm(x, x_stride, residual, weight, residual_out, out, scales, rows, D, group, eps, e4m3,
                                   static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
