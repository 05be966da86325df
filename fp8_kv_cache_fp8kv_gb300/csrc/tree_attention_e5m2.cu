// The tree attention's kernels over an E5M2 cache (tree_kernel.cuh).
#include "tree_kernel.cuh"

namespace fp8kv {
namespace tree {

cudaError_t launch_e5m2(int head_dim, const Args& a, const Plan& p, cudaStream_t s) { return launch<1, true>(head_dim, a, p, s); }

}  // namespace tree
}  // namespace fp8kv
