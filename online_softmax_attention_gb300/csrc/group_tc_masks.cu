// Grouped attention with packed query rows (group_tc.cuh) over a sliding window, with a mask.
#include "group_tc.cuh"

namespace attn {

cudaError_t launch_group_masks(const GroupParams &p, cudaStream_t s) { return launch_group_of<true, true>(p, s); }

}  // namespace attn
