// Arithmetic on a few values at a time that the elementwise kernels share.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

// 1 / x and 2^x to a few units in the last place.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// The larger of x and lo, or NaN for a NaN.
__device__ __forceinline__ float max_nan(float x, float lo) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(lo));
  return y;
}

// Eight bf16, minus infinity as the lowest finite value.
__device__ __forceinline__ uint4 above_minus_inf(uint4 v) {
#define GDN_MAX2(x) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(0xff7fff7fu))
  GDN_MAX2(v.x);
  GDN_MAX2(v.y);
  GDN_MAX2(v.z);
  GDN_MAX2(v.w);
#undef GDN_MAX2
  return v;
}

// silu of two values above minus infinity, v / (1 + e^-v): an infinite divisor gives 0.  (One reciprocal for both,
// 1 / a = b / (a b), has to keep a NaN and large divisors out of the other's result, which costs as much as it saves:
// the scan of 32 ragged prompts takes 658 us with it, 652 so.)
__device__ __forceinline__ float2 silu2_above(float2 v) {
  const float2 t = mul2(v, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  const float2 d = fma2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), make_float2(1.f, 1.f), make_float2(1.f, 1.f));
  return mul2(v, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
}
// silu of any two values; of minus infinity 0.
__device__ __forceinline__ float2 silu2(float2 v) {
  constexpr float kLow = -0x1.fffffep127f;
  return silu2_above(make_float2(max_nan(v.x, kLow), max_nan(v.y, kLow)));
}

// Four or eight bf16 as pairs of fp32, and back.
__device__ __forceinline__ float2 widen2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void widen8(const uint4& r, float2 (&f)[4]) {
  f[0] = widen2(r.x);
  f[1] = widen2(r.y);
  f[2] = widen2(r.z);
  f[3] = widen2(r.w);
}
__device__ __forceinline__ uint4 narrow8(const float2 (&f)[4]) {
  return make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y),
                    pack_bf16(f[3].x, f[3].y));
}

__device__ __forceinline__ void widen4(const uint2& r, float2 (&f)[2]) {
  f[0] = widen2(r.x);
  f[1] = widen2(r.y);
}
__device__ __forceinline__ uint2 narrow4(const float2 (&f)[2]) {
  return make_uint2(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y));
}

}  // namespace gdn
