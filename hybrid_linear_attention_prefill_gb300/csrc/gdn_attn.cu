// Attention of prompts: the kernel for the width of a head (gdn_attn_tile.cuh).
#include "gdn_attn.cuh"

namespace gdn {

template <int kQuarters>
cudaError_t launch_attn_tiles(const attn::PromptArgs& a, int* status, cudaStream_t st);

cudaError_t launch_attn(const attn::PromptArgs& a, int* status, cudaStream_t st) {
  switch ((a.d + 31) / 32) {
    case 1: return launch_attn_tiles<1>(a, status, st);
    case 2: return launch_attn_tiles<2>(a, status, st);
    case 3: return launch_attn_tiles<3>(a, status, st);
    default: return launch_attn_tiles<4>(a, status, st);
  }
}

}  // namespace gdn
