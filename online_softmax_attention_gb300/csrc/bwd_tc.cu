// Backward on the tensor cores (bwd_tc.cuh), without a window.
#include "bwd_tc.cuh"

namespace attn {

bool tc_bwd_supported(const BwdParams &p) {
    if (p.dtype != ATTN_F16 && p.dtype != ATTN_BF16) return false;
    if (p.D != 64 && p.D != 128) return false;
    if (p.n_q <= 0 || p.n_k <= 0) return false;
    return tc_device_ok();
}

int tc_bwd_kv_block(const BwdParams &) { return BT; }
int tc_bwd_q_block(const BwdParams &) { return BT; }

cudaError_t launch_bwd_dkdv_tc(const BwdParams &p, int num_ctas, cudaStream_t s) {
    return p.window ? launch_bwd_window(p, num_ctas, s, true) : launch_bwd<false>(p, num_ctas, s, true);
}

cudaError_t launch_bwd_dq_tc(const BwdParams &p, int num_ctas, cudaStream_t s) {
    return p.window ? launch_bwd_window(p, num_ctas, s, false) : launch_bwd<false>(p, num_ctas, s, false);
}

}  // namespace attn
