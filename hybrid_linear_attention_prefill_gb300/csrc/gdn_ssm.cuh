// What the selective state space scan and its single-token step share.
#pragma once

#include "gdn_vec.cuh"

namespace gdn {

// A call's tensors (token strides in elements).
struct SsmArgs {
  const __nv_bfloat16* x;   // [Ttot, Hv, dv]
  const void* dt;           // [Ttot, Hv], bf16 or fp32
  const float* A;           // [Hv]
  const __nv_bfloat16* Bm;  // [Ttot, Hk, dk]
  const __nv_bfloat16* Cm;  // [Ttot, Hk, dk]
  const float* D;           // [Hv] or null
  const __nv_bfloat16* z;   // [Ttot, Hv, dv] or null
  const float* dt_bias;     // [Hv] or null
  __nv_bfloat16* out;       // [Ttot, Hv, dv], contiguous
  long long xs, dts, bs, cs, zs;
  int Hk, Hv, dv;
  int softplus, dt_f32;
};

// The step of (token, head), softplus(dt + bias) or dt + bias, in two parts, so that the load can go ahead.
__device__ __forceinline__ uint32_t ssm_load_dt(const SsmArgs& a, long long t, int h) {  // as it is in memory
  const long long at = t * a.dts + h;
  return a.dt_f32 ? static_cast<const uint32_t*>(a.dt)[at] : (uint32_t) static_cast<const uint16_t*>(a.dt)[at];
}
__device__ __forceinline__ float ssm_step_of(const SsmArgs& a, uint32_t dt, float bias) {
  const float d = __uint_as_float(a.dt_f32 ? dt : dt << 16) + bias;
  return a.softplus && d <= 20.f ? log1pf(expf(d)) : d;  // beyond 20 they agree to fp32
}
__device__ __forceinline__ float ssm_bias(const SsmArgs& a, int h) { return a.dt_bias != nullptr ? a.dt_bias[h] : 0.f; }

// A decay by e^l, l <= 0, as keep S + (more S + what is added).  Above a half that is S + (e^l - 1) S:
// e^l itself, rounded near 1, is off the same way for every token or chunk of a slowly decaying state,
// which then adds up (2^-25 of it each time over thousands), while a sum's rounding errors have either
// sign.  Below a half the difference would cancel, and e^l S is taken as it is.
struct SsmDecay {
  float keep, more;
};
__device__ __forceinline__ SsmDecay ssm_decay(float l) {
  const bool near_one = l > -0.6931f;
  return {near_one ? 1.f : 0.f, near_one ? expm1f(l) : expf(l)};
}
__device__ __forceinline__ float ssm_decayed(const SsmDecay& d, float s, float add) {
  return fmaf(d.keep, s, fmaf(d.more, s, add));
}

// E (1, 2 or 4) consecutive fp32 of a state row.
template <int E>
__device__ __forceinline__ void ssm_load_row(const float* p, float (&s)[E]) {
  if constexpr (E == 4) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    s[0] = t.x; s[1] = t.y; s[2] = t.z; s[3] = t.w;
  } else if constexpr (E == 2) {
    const float2 t = *reinterpret_cast<const float2*>(p);
    s[0] = t.x; s[1] = t.y;
  } else {
    s[0] = *p;
  }
}
template <int E>
__device__ __forceinline__ void ssm_store_row(float* p, const float (&s)[E]) {
  if constexpr (E == 4) *reinterpret_cast<float4*>(p) = make_float4(s[0], s[1], s[2], s[3]);
  else if constexpr (E == 2) *reinterpret_cast<float2*>(p) = make_float2(s[0], s[1]);
  else *p = s[0];
}

}  // namespace gdn
