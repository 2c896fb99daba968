// The kernels of tree.cuh for masks over a sliding window.
#include "tree.cuh"

namespace attn {

cudaError_t launch_tree_masks(const TreeParams &p, cudaStream_t s) { return launch_tree<true, true>(p, s); }

}  // namespace attn
