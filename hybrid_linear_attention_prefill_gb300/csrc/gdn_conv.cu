// Short causal convolution of every channel over its sequence's tokens, for prompts and for single
// tokens (sm_103a):
//
//   y[t, c] = act( bias[c] + sum_{k < K} w[c, k] x[t - K + 1 + k, c] ),   act = silu or none,
//
// inputs before a sequence from its state [K - 1, C] (oldest first) or zeros.  Each element is read
// and written once (4 bytes) for 2 K + ~6 operations, so HBM bandwidth bounds it.  A thread owns
// eight consecutive channels (one 16-byte access a token) and walks a run of tokens with the last
// K - 1 inputs in registers, so that only a run's first K - 1 inputs are read twice.
#include "gdn_common.cuh"

namespace gdn {

namespace {

constexpr int kConvThreads = 128;
constexpr int kConvRun = 16;  // tokens a thread walks


__device__ __forceinline__ void widen8(const uint4& r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.f + __expf(-x)); }

// A thread's eight channels' weights w[k][i] and biases.
template <int K>
struct Taps {
  float w[K][8], b[8];
  __device__ __forceinline__ void load(const __nv_bfloat16* weight, const __nv_bfloat16* bias, int c) {
    uint4 raw[K];
#pragma unroll
    for (int j = 0; j < K; ++j) raw[j] = *reinterpret_cast<const uint4*>(weight + (size_t)c * K + 8 * j);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float f[8];
      widen8(raw[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[(8 * j + i) % K][(8 * j + i) / K] = f[i];  // [channel][tap] order
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0.f;
    if (bias != nullptr) widen8(*reinterpret_cast<const uint4*>(bias + c), b);
  }
  // The output of the token with input `cur` after `past` (oldest first).
  template <bool SILU>
  __device__ __forceinline__ uint4 apply(const uint4 (&past)[K - 1], const uint4& cur) const {
    float acc[8], f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = b[i];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      widen8(k < K - 1 ? past[k < K - 1 ? k : 0] : cur, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[k][i], f[i], acc[i]);
    }
    if (SILU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = silu(acc[i]);
    }
    return narrow8(acc);
  }
};

// The last sequence that starts at or before token t (out-of-order boundaries give some sequence).
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ cu, int B, int t) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace

// grid: (ceil(Ttot / run) + B when the final states are wanted, channel blocks).  The first blocks
// compute outputs; block ceil(Ttot / run) + b copies sequence b's final state.
template <int K, bool SILU>
__global__ void __launch_bounds__(kConvThreads)
gdn_conv_kernel(const __nv_bfloat16* __restrict__ x, long long xs, const __nv_bfloat16* __restrict__ weight,
                const __nv_bfloat16* __restrict__ bias, const int32_t* __restrict__ cu,
                const __nv_bfloat16* __restrict__ init, __nv_bfloat16* __restrict__ out,
                __nv_bfloat16* __restrict__ fin, int B, int T, int Ttot, int C, int runs) {
  const int c = (blockIdx.y * kConvThreads + threadIdx.x) * 8;
  if (c >= C) return;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if ((int)blockIdx.x >= runs) {  // a final state
    const int b = blockIdx.x - runs;
    const SeqChunk s = seq_bounds(cu, b, T);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int p = s.len - (K - 1) + j;  // position of the input in the sequence; negative: in its state
      uint4 v = zero;
      if (p >= 0) v = *reinterpret_cast<const uint4*>(x + (s.bos + p) * xs + c);
      else if (init != nullptr) v = *reinterpret_cast<const uint4*>(init + ((size_t)b * (K - 1) + K - 1 + p) * C + c);
      *reinterpret_cast<uint4*>(fin + ((size_t)b * (K - 1) + j) * C + c) = v;
    }
    return;
  }
  const int t0 = blockIdx.x * kConvRun, t1 = min(t0 + kConvRun, Ttot);
  Taps<K> taps;
  taps.load(weight, bias, c);
  int b, start, end;  // the sequence of token t and its bounds
  if (cu == nullptr) {
    b = t0 / T;
    start = b * T;
    end = start + T;
  } else {
    b = find_seq(cu, B, t0);
    start = max(0, min(cu[b], t0));
    end = b + 1 < B ? cu[b + 1] : Ttot;
  }
  uint4 past[K - 1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int t = t0 - (K - 1) + j;
    past[j] = zero;
    if (t >= start) past[j] = *reinterpret_cast<const uint4*>(x + (long long)t * xs + c);
    else if (init != nullptr)
      past[j] = *reinterpret_cast<const uint4*>(init + ((size_t)b * (K - 1) + K - 1 + (t - start)) * C + c);
  }
  auto step = [&](int t, const uint4& cur) {
    if (t >= end) {  // the next sequence that has tokens begins here
      if (cu == nullptr) {
        ++b;
        end += T;
      } else {
        b = find_seq(cu, B, t);
        end = b + 1 < B ? cu[b + 1] : Ttot;
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
        past[j] = init != nullptr ? *reinterpret_cast<const uint4*>(init + ((size_t)b * (K - 1) + j) * C + c) : zero;
    }
    *reinterpret_cast<uint4*>(out + (size_t)t * C + c) = taps.template apply<SILU>(past, cur);
#pragma unroll
    for (int j = 0; j + 1 < K - 1; ++j) past[j] = past[j + 1];
    past[K - 2] = cur;
  };
  int t = t0;
  for (; t + 4 <= t1; t += 4) {  // four tokens' loads in flight
    uint4 cur[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) cur[u] = *reinterpret_cast<const uint4*>(x + (long long)(t + u) * xs + c);
#pragma unroll
    for (int u = 0; u < 4; ++u) step(t + u, cur[u]);
  }
  for (; t < t1; ++t) step(t, *reinterpret_cast<const uint4*>(x + (long long)t * xs + c));
}

// One thread per (sequence, eight channels).
template <int K, bool SILU>
__global__ void __launch_bounds__(kConvThreads)
gdn_conv_step_kernel(const __nv_bfloat16* __restrict__ x, long long xs, const __nv_bfloat16* __restrict__ weight,
                     const __nv_bfloat16* __restrict__ bias, __nv_bfloat16* __restrict__ state,
                     __nv_bfloat16* __restrict__ out, int C) {
  const int c = (blockIdx.y * kConvThreads + threadIdx.x) * 8, b = blockIdx.x;
  if (c >= C) return;
  __nv_bfloat16* sp = state + (size_t)b * (K - 1) * C + c;
  uint4 past[K - 1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) past[j] = *reinterpret_cast<const uint4*>(sp + (size_t)j * C);
  const uint4 cur = *reinterpret_cast<const uint4*>(x + b * xs + c);
  Taps<K> taps;
  taps.load(weight, bias, c);
  *reinterpret_cast<uint4*>(out + (size_t)b * C + c) = taps.template apply<SILU>(past, cur);
#pragma unroll
  for (int j = 0; j + 1 < K - 1; ++j) *reinterpret_cast<uint4*>(sp + (size_t)j * C) = past[j + 1];
  *reinterpret_cast<uint4*>(sp + (size_t)(K - 2) * C) = cur;
}

template <int K, bool SILU>
cudaError_t conv_k(const void* x, long long xs, const void* weight, const void* bias, const int32_t* cu,
                   const void* init, void* out, void* fin, int B, int T, int Ttot, int C, cudaStream_t st) {
  using bf = __nv_bfloat16;
  const int runs = (Ttot + kConvRun - 1) / kConvRun;
  const unsigned gx = (unsigned)runs + (fin != nullptr ? (unsigned)B : 0u);
  gdn_conv_kernel<K, SILU><<<dim3(gx, (C / 8 + kConvThreads - 1) / kConvThreads), kConvThreads, 0, st>>>(
      static_cast<const bf*>(x), xs, static_cast<const bf*>(weight), static_cast<const bf*>(bias), cu,
      static_cast<const bf*>(init), static_cast<bf*>(out), static_cast<bf*>(fin), B, T, Ttot, C, runs);
  return cudaGetLastError();
}

template <int K, bool SILU>
cudaError_t conv_step_k(const void* x, long long xs, const void* weight, const void* bias, void* state, void* out,
                        int B, int C, cudaStream_t st) {
  using bf = __nv_bfloat16;
  gdn_conv_step_kernel<K, SILU><<<dim3(B, (C / 8 + kConvThreads - 1) / kConvThreads), kConvThreads, 0, st>>>(
      static_cast<const bf*>(x), xs, static_cast<const bf*>(weight), static_cast<const bf*>(bias),
      static_cast<bf*>(state), static_cast<bf*>(out), C);
  return cudaGetLastError();
}

cudaError_t launch_conv(const void* x, long long xs, const void* weight, const void* bias, const int32_t* cu,
                        const void* init, void* out, void* fin, int B, int T, int Ttot, int C, int K, bool silu,
                        cudaStream_t st) {
#define GDN_CONV_CASE(KK)                                                                                   \
  case KK:                                                                                                  \
    return silu ? conv_k<KK, true>(x, xs, weight, bias, cu, init, out, fin, B, T, Ttot, C, st)              \
                : conv_k<KK, false>(x, xs, weight, bias, cu, init, out, fin, B, T, Ttot, C, st);
  switch (K) {
    GDN_CONV_CASE(2)
    GDN_CONV_CASE(3)
    GDN_CONV_CASE(4)
    default: return cudaErrorInvalidValue;
  }
#undef GDN_CONV_CASE
}

cudaError_t launch_conv_step(const void* x, long long xs, const void* weight, const void* bias, void* state, void* out,
                             int B, int C, int K, bool silu, cudaStream_t st) {
#define GDN_CONV_CASE(KK)                                                                \
  case KK:                                                                               \
    return silu ? conv_step_k<KK, true>(x, xs, weight, bias, state, out, B, C, st)       \
                : conv_step_k<KK, false>(x, xs, weight, bias, state, out, B, C, st);
  switch (K) {
    GDN_CONV_CASE(2)
    GDN_CONV_CASE(3)
    GDN_CONV_CASE(4)
    default: return cudaErrorInvalidValue;
  }
#undef GDN_CONV_CASE
}

}  // namespace gdn
