// The tree attention's kernels over a bf16 cache (tree_kernel.cuh).
#include "tree_kernel.cuh"

namespace fp8kv {
namespace tree {

cudaError_t launch_bf16(int head_dim, const Args& a, const Plan& p, cudaStream_t s) { return launch<2, false>(head_dim, a, p, s); }

}  // namespace tree
}  // namespace fp8kv
