// A paged key-value cache: the plan of a step (new blocks, each new token's slot) and the writing of the
// new tokens' keys and values (sm_103a).
//
// Plan.  Request b holds n_b tokens and gets a_b more: it needs ceil((n_b + a_b) / page) - ceil(n_b / page)
// blocks, taken from the top of the stack of free ones in the requests' order, so a request's first is a
// prefix sum of needs away from the top.  One cluster does it in one launch: every CTA sums over all
// requests for itself (a few thousand integers), the cluster's barrier puts every read before the first
// write (lengths and the stack's height may be updated in place), and the CTAs share the tokens.
// Latency bounds it: three dependent loads and the sums beside a launch.
//
// Append.  A copy of whole 16-byte pieces (to e4m3: eight values a thread, divided by their head's scale
// and rounded once), bound by bandwidth.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include "gdn_cache.h"
#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_vec.cuh"

namespace cg = cooperative_groups;

namespace gdn {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;          // of the cluster for many tokens
constexpr int kPlanAlone = 4096;      // tokens that one CTA takes by itself
constexpr int kAppendThreads = 256;
constexpr int kAppendAhead = 4;       // tokens a thread has on their way

// Sum over the threads before this one, and over all (in every thread).
__device__ __forceinline__ long long block_scan(long long v, long long* part, long long& all) {
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
  long long w = part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return sum - v + (warp > 0 ? before : 0);
}

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
  if (tid == 0) lacking = 0;
  int count = *a.free_count;
  count = count < 0 ? 0 : count > a.capacity ? a.capacity : count;

  long long carry = 0, taken = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
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
      const long long have = ((long long)n + a.page - 1) / a.page, want = ((long long)n + hi - lo + a.page - 1) / a.page;
      able = n >= 0 && want <= a.W && (long long)n + hi - lo <= 0x7fffffffLL;
      need = able ? want - have : 0;
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
  cluster.sync();  // every CTA has read the lengths and the stack's height (and part is written)

  if (rank == 0) {
    for (int b = tid; b < a.B; b += kPlanThreads) {
      const int len = a.cu != nullptr ? seq_bounds(a.cu, b, a.T).len : 1;
      a.new_lens[b] = base[b] >= 0 ? held[b] + len : held[b];
    }
    if (tid == 0) {
      long long most = 0;
      for (int w = 0; w < kPlanThreads / 32; ++w) most = part[w] > most ? part[w] : most;
      *a.new_count = count - (int)most;
      if (a.refused != nullptr) *a.refused = lacking;
    }
  }
  // table entries: a warp a request
  for (int b = rank * (kPlanThreads / 32) + (tid >> 5); b < a.B; b += ctas * (kPlanThreads / 32)) {
    if (base[b] < 0) continue;
    const int len = a.cu != nullptr ? seq_bounds(a.cu, b, a.T).len : 1;
    const int have = (int)(((long long)held[b] + a.page - 1) / a.page);
    const int need = (int)(((long long)held[b] + len + a.page - 1) / a.page) - have;
    for (int i = tid & 31; i < need; i += 32)
      a.table[b * a.table_stride + have + i] = a.free_blocks[count - 1 - base[b] - i];
  }
  for (long long t = (long long)rank * kPlanThreads + tid; t < a.T; t += (long long)ctas * kPlanThreads) {
    int b = (int)t;
    if (a.cu != nullptr) {  // the last request that starts at or before t
      int lo = 0, hi = a.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= t) lo = mid; else hi = mid;
      }
      b = lo;
    }
    long long slot = -1;
    const int len = a.cu != nullptr && a.B > 0 ? seq_bounds(a.cu, b, a.T).len : 1;
    if (a.B > 0 && t >= start[b] && t < start[b] + (long long)len && base[b] >= 0) {
      const long long p = held[b] + (t - start[b]);
      const int col = (int)(p / a.page), have = (int)(((long long)held[b] + a.page - 1) / a.page);
      const int block = col < have ? a.table[b * a.table_stride + col] : a.free_blocks[count - 1 - base[b] - (col - have)];
      if (block >= 0) slot = (long long)block * a.page + (p - (long long)col * a.page);
      if (slot > 0x7fffffffLL) slot = -1;
    }
    a.slots[t] = (int32_t)slot;
  }
}

cudaError_t launch_cache_plan(const CachePlanArgs& a, cudaStream_t st) {
  const int smem = 3 * a.B * 4;
  cudaError_t e = set_smem_limit_once<gdn_cache_plan_kernel>(3 * kPlanMaxRequests * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const unsigned ctas = a.T <= kPlanAlone ? 1 : kPlanCtas;
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
template <bool E4M3>
__global__ void __launch_bounds__(kAppendThreads) gdn_cache_append_kernel(const CacheAppendArgs a, int width, int rows) {
  const int per = a.d / 8, r = threadIdx.x / width;
  const int piece = blockIdx.y * width + (threadIdx.x - r * width);
  if (r >= rows || piece >= a.Hkv * per) return;
  const int h = piece / per, c = (piece - h * per) * 8;
  const float ks = E4M3 ? a.kscale[h] : 1.f, vs = E4M3 ? a.vscale[h] : 1.f;
  const long long most = (long long)a.blocks * a.page;
  const long long t0 = (long long)blockIdx.x * (rows * kAppendAhead) + r;
  uint4 kx[kAppendAhead], vx[kAppendAhead];
  int slot[kAppendAhead];
#pragma unroll
  for (int u = 0; u < kAppendAhead; ++u) {
    const long long t = t0 + (long long)u * rows;
    slot[u] = -1;
    if (t < a.T) {
      slot[u] = a.slots[t];
      kx[u] = *reinterpret_cast<const uint4*>(a.k + t * a.ks + 8 * (long long)piece);
      vx[u] = *reinterpret_cast<const uint4*>(a.v + t * a.vs + 8 * (long long)piece);
    }
  }
#pragma unroll
  for (int u = 0; u < kAppendAhead; ++u) {
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
  const int run = rows * kAppendAhead;
  const dim3 grid((unsigned)((a.T + (long long)run - 1) / run), (unsigned)((pieces + width - 1) / width));
  if (e4m3)
    gdn_cache_append_kernel<true><<<grid, kAppendThreads, 0, st>>>(a, width, rows);
  else
    gdn_cache_append_kernel<false><<<grid, kAppendThreads, 0, st>>>(a, width, rows);
  return cudaGetLastError();
}

}  // namespace gdn
