// Arguments of the paged cache's kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

constexpr int kPlanMaxRequests = 16384;  // three integers of each in shared memory

struct CachePlanArgs {
  const int32_t* lens;
  int32_t* table;
  long long table_stride;
  const int32_t *free_blocks, *free_count, *cu;
  int32_t *slots, *new_lens, *new_count, *refused;
  int B, T, W, capacity, page;
};
cudaError_t launch_cache_plan(const CachePlanArgs& a, cudaStream_t st);

struct CacheAppendArgs {
  const __nv_bfloat16 *k, *v;
  long long ks, vs;  // distances between tokens in elements
  void *kc, *vc;
  long long kbs, vbs;  // distances between blocks in elements
  const float *kscale, *vscale;
  const int32_t* slots;
  int T, Hkv, d, page, blocks;
};
cudaError_t launch_cache_append(const CacheAppendArgs& a, bool e4m3, cudaStream_t st);

}  // namespace gdn
