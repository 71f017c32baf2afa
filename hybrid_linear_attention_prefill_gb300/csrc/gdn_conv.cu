// Short causal convolution of every channel over its sequence's tokens, for prompts and for single
// tokens (sm_103a):
//
//   y[t, c] = act( bias[c] + sum_{k < K} w[c, k] x[t - K + 1 + k, c] ),   act = silu or none,
//
// inputs before a sequence from its state [K - 1, C] (oldest first) or zeros.  Each element is read
// and written once (4 bytes) for 2 K + ~6 operations, so HBM bandwidth bounds it.  A thread owns
// four consecutive channels (an 8-byte access a token: with eight, its weights and window leave
// room for too few loads in flight) and walks a run of tokens with the last K - 1 inputs in
// registers, so that only a run's first K - 1 inputs are read twice.  72,102 tokens of 8,192
// channels: 367 us, 6.44 TB/s; 4,096 tokens: 27.2 us.
#include "gdn_internal.h"
#include "gdn_vec.cuh"

namespace gdn {

namespace {

constexpr int kConvThreads = 128;
// Blocks an SM: 72 registers a thread.  More blocks spill, fewer have too few loads in flight (72,102 tokens of
// 8,192 channels: 372 us with 7, 385 with 6, 448 with 8).
constexpr int kConvBlocks = 7;
constexpr int kConvBatch = 8;  // tokens whose loads a thread has in flight

// A thread's four channels' weights and biases, in pairs.
template <int K>
struct Taps {
  float2 w[K][2], b[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* weight, const __nv_bfloat16* bias, int c) {
    uint2 raw[K];
#pragma unroll
    for (int j = 0; j < K; ++j) raw[j] = *reinterpret_cast<const uint2*>(weight + (size_t)c * K + 4 * j);
    float f[4 * K];  // [channel][tap]
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float2 t[2];
      widen4(raw[j], t);
#pragma unroll
      for (int i = 0; i < 2; ++i) f[4 * j + 2 * i] = t[i].x, f[4 * j + 2 * i + 1] = t[i].y;
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) w[k][i] = make_float2(f[2 * i * K + k], f[(2 * i + 1) * K + k]);
#pragma unroll
    for (int i = 0; i < 2; ++i) b[i] = make_float2(0.f, 0.f);
    if (bias != nullptr) widen4(*reinterpret_cast<const uint2*>(bias + c), b);
  }
  // The output of the token with input `cur` after `past` (oldest first).
  template <bool SILU>
  __device__ __forceinline__ uint2 apply(const float2 (&past)[K - 1][2], const float2 (&cur)[2]) const {
    float2 acc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      acc[i] = fma2(w[0][i], past[0][i], b[i]);
#pragma unroll
      for (int k = 1; k < K - 1; ++k) acc[i] = fma2(w[k][i], past[k][i], acc[i]);
      acc[i] = fma2(w[K - 1][i], cur[i], acc[i]);
      if (SILU) acc[i] = silu2(acc[i]);
    }
    return narrow4(acc);
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

// grid: (runs + B when the final states are wanted, channel blocks).  The first blocks compute outputs, `run`
// tokens each; block runs + b copies sequence b's final state.
template <int K, bool SILU>
__global__ void __launch_bounds__(kConvThreads, kConvBlocks)
gdn_conv_kernel(const __nv_bfloat16* __restrict__ x, long long xs, const __nv_bfloat16* __restrict__ weight,
                const __nv_bfloat16* __restrict__ bias, const int32_t* __restrict__ cu,
                const __nv_bfloat16* __restrict__ init, __nv_bfloat16* __restrict__ out,
                __nv_bfloat16* __restrict__ fin, int B, int T, int Ttot, int C, int runs, int run) {
  const int c = (blockIdx.y * kConvThreads + threadIdx.x) * 4;
  if (c >= C) return;
  const uint2 zero = make_uint2(0, 0);
  if ((int)blockIdx.x >= runs) {  // a final state
    const int b = blockIdx.x - runs;
    const SeqChunk s = seq_bounds(cu, b, T);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int p = s.len - (K - 1) + j;  // position of the input in the sequence; negative: in its state
      uint2 v = zero;
      if (p >= 0) v = *reinterpret_cast<const uint2*>(x + (s.bos + p) * xs + c);
      else if (init != nullptr) v = *reinterpret_cast<const uint2*>(init + ((size_t)b * (K - 1) + K - 1 + p) * C + c);
      *reinterpret_cast<uint2*>(fin + ((size_t)b * (K - 1) + j) * C + c) = v;
    }
    return;
  }
  const int t0 = blockIdx.x * run, t1 = t0 + min(run, Ttot - t0);
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
  float2 past[K - 1][2];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int t = t0 - (K - 1) + j;
    uint2 v = zero;
    if (t >= start) v = *reinterpret_cast<const uint2*>(x + (long long)t * xs + c);
    else if (init != nullptr)
      v = *reinterpret_cast<const uint2*>(init + ((size_t)b * (K - 1) + K - 1 + (t - start)) * C + c);
    widen4(v, past[j]);
  }
  const __nv_bfloat16* xp = x + (long long)t0 * xs + c;
  __nv_bfloat16* op = out + (size_t)t0 * C + c;
  uint2 next[kConvBatch];
#pragma unroll
  for (int u = 0; u < kConvBatch; ++u) next[u] = u < t1 - t0 ? *reinterpret_cast<const uint2*>(xp + u * xs) : zero;
  auto token = [&](const uint2& in) {
    float2 f[2];
    widen4(in, f);
    *reinterpret_cast<uint2*>(op) = taps.template apply<SILU>(past, f);
    op += C;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j + 1 < K - 1; ++j) past[j][i] = past[j + 1][i];
      past[K - 2][i] = f[i];
    }
  };
  for (int t = t0;; t += kConvBatch) {
    xp += kConvBatch * xs;
    if (min(end, t1) - t >= kConvBatch) {  // all of the batch in the run and in the sequence
#pragma unroll
      for (int u = 0; u < kConvBatch; ++u) {
        token(next[u]);
        if (kConvBatch + u < t1 - t) next[u] = *reinterpret_cast<const uint2*>(xp + u * xs);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kConvBatch; ++u) {
        if (u >= t1 - t) break;
        if (t + u >= end) {  // the next sequence that has tokens begins here
          if (cu == nullptr) {
            ++b;
            end = b + 1 < B ? end + T : Ttot;
          } else {
            b = find_seq(cu, B, t + u);
            end = b + 1 < B ? cu[b + 1] : Ttot;
          }
#pragma unroll
          for (int j = 0; j < K - 1; ++j)
            widen4(init != nullptr ? *reinterpret_cast<const uint2*>(init + ((size_t)b * (K - 1) + j) * C + c) : zero,
                   past[j]);
        }
        token(next[u]);
        if (kConvBatch + u < t1 - t) next[u] = *reinterpret_cast<const uint2*>(xp + u * xs);
      }
    }
    if (t1 - t <= kConvBatch) break;
  }
}

// One thread per (sequence, four channels).
template <int K, bool SILU>
__global__ void __launch_bounds__(kConvThreads)
gdn_conv_step_kernel(const __nv_bfloat16* __restrict__ x, long long xs, const __nv_bfloat16* __restrict__ weight,
                     const __nv_bfloat16* __restrict__ bias, __nv_bfloat16* __restrict__ state,
                     __nv_bfloat16* __restrict__ out, int C) {
  const int c = (blockIdx.y * kConvThreads + threadIdx.x) * 4, b = blockIdx.x;
  if (c >= C) return;
  __nv_bfloat16* sp = state + (size_t)b * (K - 1) * C + c;
  uint2 past[K - 1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) past[j] = *reinterpret_cast<const uint2*>(sp + (size_t)j * C);
  const uint2 cur = *reinterpret_cast<const uint2*>(x + b * xs + c);
  Taps<K> taps;
  taps.load(weight, bias, c);
  float2 pf[K - 1][2], cf[2];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) widen4(past[j], pf[j]);
  widen4(cur, cf);
  *reinterpret_cast<uint2*>(out + (size_t)b * C + c) = taps.template apply<SILU>(pf, cf);
#pragma unroll
  for (int j = 0; j + 1 < K - 1; ++j) *reinterpret_cast<uint2*>(sp + (size_t)j * C) = past[j + 1];
  *reinterpret_cast<uint2*>(sp + (size_t)(K - 2) * C) = cur;
}

template <int K, bool SILU>
cudaError_t conv_k(const void* x, long long xs, const void* weight, const void* bias, const int32_t* cu,
                   const void* init, void* out, void* fin, int B, int T, int Ttot, int C, cudaStream_t st) {
  using bf = __nv_bfloat16;
  // Runs of 128 tokens read a fortieth of the inputs twice; shorter ones where they would not give every SM its blocks
  // half over again (72,102 tokens of 8,192 channels: 367 us with 128, 373 with 64, 379 with 32, 412 with 16; 4,096
  // tokens take 32: 27.5 us, with 16 29.1).
  const int cb = (C / 4 + kConvThreads - 1) / kConvThreads;
  int run = 128;
  while (run > kConvBatch && 2LL * (Ttot / run) * cb < 3LL * kConvBlocks * device_sms()) run >>= 1;
  const int runs = (int)(((long long)Ttot + run - 1) / run);
  const unsigned gx = (unsigned)runs + (fin != nullptr ? (unsigned)B : 0u);
  gdn_conv_kernel<K, SILU><<<dim3(gx, cb), kConvThreads, 0, st>>>(
      static_cast<const bf*>(x), xs, static_cast<const bf*>(weight), static_cast<const bf*>(bias), cu,
      static_cast<const bf*>(init), static_cast<bf*>(out), static_cast<bf*>(fin), B, T, Ttot, C, runs, run);
  return cudaGetLastError();
}

template <int K, bool SILU>
cudaError_t conv_step_k(const void* x, long long xs, const void* weight, const void* bias, void* state, void* out,
                        int B, int C, cudaStream_t st) {
  using bf = __nv_bfloat16;
  gdn_conv_step_kernel<K, SILU><<<dim3(B, (C / 4 + kConvThreads - 1) / kConvThreads), kConvThreads, 0, st>>>(
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
