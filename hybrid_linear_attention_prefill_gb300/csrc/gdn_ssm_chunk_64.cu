// The chunked selective scan's kernels for a state of 64 columns.
#include "gdn_ssm_chunk_kernels.cuh"

namespace gdn {
namespace ssm {
template cudaError_t launch_dk<64>(const Maps&, const SsmArgs&, const Segs&, float*, float*, const float*, float*,
                                    float*, int*, int, int, cudaStream_t);
}  // namespace ssm
}  // namespace gdn
