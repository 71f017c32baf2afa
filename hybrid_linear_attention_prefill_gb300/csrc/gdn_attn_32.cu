// Attention of prompts with heads of 8 to 32 columns (gdn_attn_tile.cuh).
#include "gdn_attn_tile.cuh"

namespace gdn {
template cudaError_t launch_attn_tiles<1>(const attn::PromptArgs&, int*, cudaStream_t);
}  // namespace gdn
