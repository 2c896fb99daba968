// Backward on the tensor cores (bwd_tc.cuh) over a sliding window with sinks.
#include "bwd_tc.cuh"

namespace attn {

cudaError_t launch_bwd_window(const BwdParams &p, int num_ctas, cudaStream_t s, bool dkdv) {
    return launch_bwd<true>(p, num_ctas, s, dkdv);
}

}  // namespace attn
