// kvq_tree_a3.cu -- instantiates the tree attention kernels of one cache format.
#include "kvq_tree_split.cuh"

namespace kvq {
TreeKernel tree_kernel_a3(int D, int R) {
  return D == 64 ? tree::tree_kernel_info<KVQ_FMT_ASYM3_OUTLIER, 64>(R) : tree::tree_kernel_info<KVQ_FMT_ASYM3_OUTLIER, 128>(R);
}
}  // namespace kvq
