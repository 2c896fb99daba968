// Grouped attention with packed query rows (group_tc.cuh) over a sliding window with sinks.
#include "group_tc.cuh"

namespace attn {

cudaError_t launch_group_window(const GroupParams &p, cudaStream_t s) {
    return p.mask ? launch_group_masks(p, s) : launch_group_of<true, false>(p, s);
}

}  // namespace attn
