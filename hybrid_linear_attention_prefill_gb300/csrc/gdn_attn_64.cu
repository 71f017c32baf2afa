// Attention of prompts with heads of 40 to 64 columns (gdn_attn_tile.cuh).
#include "gdn_attn_tile.cuh"

namespace gdn {
template cudaError_t launch_attn_tiles<2>(const attn::PromptArgs&, int*, cudaStream_t);
}  // namespace gdn
