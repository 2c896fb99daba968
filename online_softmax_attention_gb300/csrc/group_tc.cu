// Grouped attention with packed query rows (group_tc.cuh), without a window.
#include "group_tc.cuh"

namespace attn {

bool group_supported(int dtype, int D, int group) {
    return (dtype == ATTN_F16 || dtype == ATTN_BF16) && (D == 64 || D == 128) && group >= 1 && group <= BM &&
           tc_device_ok();
}

cudaError_t launch_group(const GroupParams &p, cudaStream_t s) { return launch_group_of<false, false>(p, s); }

}  // namespace attn
