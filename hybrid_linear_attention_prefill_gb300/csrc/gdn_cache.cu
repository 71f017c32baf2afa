// A paged key-value cache: the plan of a step (new blocks, each new token's slot) and the writing of the
// new tokens' keys and values (sm_103a).
//
// Plan.  Request b holds n_b tokens and gets a_b more: it needs ceil((n_b + a_b) / page) - ceil(n_b / page)
// blocks, taken from the top of the stack of free ones in the requests' order, so a request's first is a
// prefix sum of needs away from the top.  One cluster does it in one launch: every CTA sums over all
// requests for itself (a few thousand integers), the cluster's barrier puts every read before the first
// write (lengths and the stack's height may be updated in place), and the CTAs share the tokens.
// Latency bounds it: three dependent loads and the sums beside a launch.  One token of 128 requests takes 6.1 us on a
// GB300 where an empty launch takes about 4, 72,102 tokens of 32 prompts 10.3 us.  (By a clock around single calls, 2 to 3
// more: 12.9; 15.0 with a cluster of eight, 19.1 with eight and a token a thread, each of which it looked up.)
//
// Append.  A copy of whole 16-byte pieces (to e4m3: eight values a thread, divided by their head's scale
// and rounded once), bound by bandwidth: 72,102 tokens of 8 heads in 89.9 us, 6.6 TB/s in and out.  128 tokens take 4.1 us
// with a token a thread (by a clock around single calls 6.9, and 8.9 with the four that the long call has on their way).
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "gdn_cache.h"
#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_vec.cuh"

namespace cg = cooperative_groups;

namespace gdn {

namespace {

constexpr int kPlanThreads = 1024, kPlanFew = 256;  // of a CTA; where that many do for requests and tokens
constexpr int kPlanRun = 4;           // tokens of packed requests that a thread takes together
// CTAs of the cluster for many tokens (72,102: 20.1 us with 4, 15.0 with 8, 12.9 with 16).  The portable eight where the
// requests' integers leave an SM one CTA: a processing cluster need not have sixteen SMs.
constexpr int kPlanCtas = 16, kPlanCtasWide = 8, kPlanShared = 100 * 1024;
constexpr int kPlanAlone = 4096;      // tokens that one CTA takes by itself
constexpr int kAppendThreads = 256;
constexpr int kAppendAhead = 4;       // tokens a thread has on their way, where that leaves two CTAs an SM

// Sum over the threads before this one, and over all (in every thread).
__device__ __forceinline__ long long block_scan(long long v, long long* part, long long& all) {
  const int warps = blockDim.x / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  __syncthreads();  // part may still be read for the round before
  if (lane == 31) part[warp] = sum;
  __syncthreads();
  long long w = lane < warps ? part[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return sum - v + (warp > 0 ? before : 0);
}

// x / y of x below 2^31, with 2^32 / y rounded down: one too few at most before the correction.
__device__ __forceinline__ int over(int x, int y, uint32_t inverse) {
  const int q = (int)__umulhi((uint32_t)x, inverse);
  return q + (x - q * y >= y);
}
__device__ __forceinline__ void prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p)); }

}  // namespace

__global__ void __launch_bounds__(kPlanThreads) gdn_cache_plan_kernel(const CachePlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  int32_t* start = plan_smem;   // [B] first new token of a request
  int32_t* held = start + a.B;  // [B] tokens before
  int32_t* base = held + a.B;   // [B] blocks taken by the requests before; -1: nothing for this one
  __shared__ long long part[32];
  __shared__ int lacking;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int threads = blockDim.x;
  const uint32_t inverse = 0xffffffffu / (uint32_t)a.page;
  if (tid == 0) lacking = 0;
  int count = *a.free_count;
  count = count < 0 ? 0 : count > a.capacity ? a.capacity : count;
  const int ahead = rank * threads + tid;
  if ((ahead & 31) == 0 && ahead < count) prefetch(a.free_blocks + count - 1 - ahead);

  long long carry = 0, taken = 0;
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int b = b0 + tid;
    long long need = 0;
    int n = -1;
    bool able = false;
    if (b < a.B) {
      n = a.lens[b];
      int lo = b, hi = b + 1;
      if (a.cu != nullptr) {
        const SeqChunk s = seq_bounds(a.cu, b, a.T);
        lo = (int)s.bos;
        hi = lo + s.len;
      }
      start[b] = lo;
      held[b] = n;
      // (blocks that a count of tokens begins, without leaving 32 bits: those of the last token and before)
      const bool fits = n >= 0 && (long long)n + hi - lo <= 0x7fffffffLL;
      const int have = n > 0 ? over(n - 1, a.page, inverse) + 1 : 0;
      const int want = fits && n + hi - lo > 0 ? over(n + hi - lo - 1, a.page, inverse) + 1 : 0;
      able = fits && want <= a.W;
      need = able ? want - have : 0;
      // what comes next is fetched beside the sums, and the stack's top
      if (n > 0 && have <= a.W && n - (have - 1) * a.page < a.page) prefetch(a.table + b * a.table_stride + have - 1);
    }
    long long all;
    const long long before = carry + block_scan(need, part, all);
    carry += all;
    if (b < a.B) {
      const bool granted = able && (need == 0 || before + need <= count);
      base[b] = !granted ? -1 : need == 0 ? 0 : (int)before;
      if (granted && need > 0 && before + need > taken) taken = before + need;
      if (!granted && n >= 0) atomicAdd(&lacking, 1);
    }
  }
  // the most that any granted request reaches
  for (int o = 16; o > 0; o >>= 1) {
    const long long y = __shfl_xor_sync(0xffffffffu, taken, o);
    taken = y > taken ? y : taken;
  }
  __syncthreads();
  if ((tid & 31) == 0) part[tid >> 5] = taken;
  // every CTA has read the lengths and the stack's height (and part is written)
  if (ctas > 1) cluster.sync();
  else __syncthreads();

  if (rank == 0) {
    for (int b = tid; b < a.B; b += threads) {
      const int len = a.cu != nullptr ? seq_bounds(a.cu, b, a.T).len : 1;
      a.new_lens[b] = base[b] >= 0 ? held[b] + len : held[b];
    }
    if (tid == 0) {
      long long most = 0;
      for (int w = 0; w < threads / 32; ++w) most = part[w] > most ? part[w] : most;
      *a.new_count = count - (int)most;
      if (a.refused != nullptr) *a.refused = lacking;
    }
  }
  // table entries: a warp a request of packed ones, a thread one that gets a token
  const bool packed = a.cu != nullptr;
  const int per = packed ? 32 : 1, lane = packed ? tid & 31 : 0;
  for (int b = (rank * threads + tid) / per; b < a.B; b += ctas * threads / per) {
    if (base[b] < 0) continue;
    const int n = held[b], end = n + (packed ? seq_bounds(a.cu, b, a.T).len : 1);
    const int have = n > 0 ? over(n - 1, a.page, inverse) + 1 : 0;
    const int need = end > 0 ? over(end - 1, a.page, inverse) + 1 - have : 0;
    for (int i = lane; i < need; i += 32) a.table[b * a.table_stride + have + i] = a.free_blocks[count - 1 - base[b] - i];
  }
  // slots: a thread has a run of packed tokens, and looks a request or a block up where one begins
  const int run = packed ? kPlanRun : 1;
  const bool wide = (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0;
  for (long long t0 = ((long long)rank * threads + tid) * run; t0 < a.T; t0 += (long long)ctas * threads * run) {
    int b = (int)t0;
    if (packed) {  // the last request that starts at or before t0
      int lo = 0, hi = a.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= t0) lo = mid; else hi = mid;
      }
      b = lo;
    }
    int4 out = make_int4(-1, -1, -1, -1);
    int at = -1, first = 0, len = 0, n = 0, taken_before = -1, have = 0, col = -1, block = -1;
#pragma unroll
    for (int i = 0; i < kPlanRun; ++i) {
      const long long t = t0 + i;
      if (i >= run || t >= a.T || a.B == 0) break;
      while (b + 1 < a.B && start[b + 1] <= t) ++b;
      if (b != at) {
        at = b;
        first = start[b];
        len = packed ? seq_bounds(a.cu, b, a.T).len : 1;
        n = held[b];
        taken_before = base[b];
        have = n > 0 ? over(n - 1, a.page, inverse) + 1 : 0;
        col = -1;
      }
      if (t < first || t >= first + (long long)len || taken_before < 0) continue;
      const int p = n + (int)(t - first), c = over(p, a.page, inverse);
      if (c != col) {
        col = c;
        block = c < have ? a.table[b * a.table_stride + c] : a.free_blocks[count - 1 - taken_before - (c - have)];
      }
      const long long slot = (long long)block * a.page + (p - c * a.page);
      if (block >= 0 && slot <= 0x7fffffffLL) (&out.x)[i] = (int)slot;
    }
    if (run == kPlanRun && wide && t0 + kPlanRun <= a.T) {
      *reinterpret_cast<int4*>(a.slots + t0) = out;
    } else {
#pragma unroll
      for (int i = 0; i < kPlanRun; ++i)
        if (i < run && t0 + i < a.T) a.slots[t0 + i] = (&out.x)[i];
    }
  }
}

cudaError_t launch_cache_plan(const CachePlanArgs& a, cudaStream_t st) {
  const int smem = 3 * a.B * 4;
  cudaError_t e = set_smem_limit_once<gdn_cache_plan_kernel>(3 * kPlanMaxRequests * 4);
  if (e != cudaSuccess) return e;
  const unsigned ctas = a.T <= kPlanAlone ? 1 : smem <= kPlanShared ? kPlanCtas : kPlanCtasWide;
  if (ctas == 1) {
    const int threads = a.B <= kPlanFew && a.T <= (a.cu != nullptr ? kPlanRun : 1) * kPlanFew ? kPlanFew : kPlanThreads;
    gdn_cache_plan_kernel<<<1, threads, (size_t)smem, st>>>(a);
    return cudaGetLastError();
  }
  e = cudaFuncSetAttribute(gdn_cache_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gdn_cache_plan_kernel, a);
}

// A thread has one piece of eight values of a token's heads, k and v, and walks tokens.
// grid: (runs of tokens, pieces past one block's)
template <bool E4M3, int kAhead>
__global__ void __launch_bounds__(kAppendThreads) gdn_cache_append_kernel(const CacheAppendArgs a, int width, int rows) {
  const int per = a.d / 8, r = threadIdx.x / width;
  const int piece = blockIdx.y * width + (threadIdx.x - r * width);
  if (r >= rows || piece >= a.Hkv * per) return;
  const int h = piece / per, c = (piece - h * per) * 8;
  const float ks = E4M3 ? a.kscale[h] : 1.f, vs = E4M3 ? a.vscale[h] : 1.f;
  const long long most = (long long)a.blocks * a.page;
  const long long t0 = (long long)blockIdx.x * (rows * kAhead) + r;
  uint4 kx[kAhead], vx[kAhead];
  int slot[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const long long t = t0 + (long long)u * rows;
    slot[u] = -1;
    if (t < a.T) {
      slot[u] = a.slots[t];
      kx[u] = *reinterpret_cast<const uint4*>(a.k + t * a.ks + 8 * (long long)piece);
      vx[u] = *reinterpret_cast<const uint4*>(a.v + t * a.vs + 8 * (long long)piece);
    }
  }
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    if (slot[u] < 0 || slot[u] >= most) continue;
    const int block = slot[u] / a.page, off = slot[u] - block * a.page;
    const long long in = ((long long)h * a.page + off) * a.d + c;
    const long long ko = (long long)block * a.kbs + in, vo = (long long)block * a.vbs + in;
    if constexpr (E4M3) {
      auto put = [&](const uint4& x, float scale, unsigned char* to) {
        float2 f[4];
        widen8(x, f);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[i].x / scale, f[i].y / scale), __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<uint2*>(to) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
      };
      put(kx[u], ks, static_cast<unsigned char*>(a.kc) + ko);
      put(vx[u], vs, static_cast<unsigned char*>(a.vc) + vo);
    } else {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.kc) + ko) = kx[u];
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.vc) + vo) = vx[u];
    }
  }
}

cudaError_t launch_cache_append(const CacheAppendArgs& a, bool e4m3, cudaStream_t st) {
  const int pieces = a.Hkv * (a.d / 8);
  const int width = pieces < kAppendThreads ? pieces : kAppendThreads, rows = kAppendThreads / width;
  const int sms = device_sms();
  auto launch = [&](auto ahead) {
    constexpr int kAhead = decltype(ahead)::value;
    const int run = rows * kAhead;
    const dim3 grid((unsigned)((a.T + (long long)run - 1) / run), (unsigned)((pieces + width - 1) / width));
    if (e4m3)
      gdn_cache_append_kernel<true, kAhead><<<grid, kAppendThreads, 0, st>>>(a, width, rows);
    else
      gdn_cache_append_kernel<false, kAhead><<<grid, kAppendThreads, 0, st>>>(a, width, rows);
  };
  if ((long long)a.T * pieces >= 2LL * sms * kAppendAhead * kAppendThreads) launch(std::integral_constant<int, kAppendAhead>());
  else launch(std::integral_constant<int, 1>());
  return cudaGetLastError();
}

}  // namespace gdn
