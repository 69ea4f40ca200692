// kvq_tree_tiered.cu -- instantiates the tree attention kernels of one cache format.
#include "kvq_tree_split.cuh"

namespace kvq {
TreeKernel tree_kernel_tiered(int D, int R) {
  return D == 64 ? tree::tree_kernel_info<KVQ_FMT_TIERED, 64>(R) : tree::tree_kernel_info<KVQ_FMT_TIERED, 128>(R);
}
}  // namespace kvq
