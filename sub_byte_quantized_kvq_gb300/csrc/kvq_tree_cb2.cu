// kvq_tree_cb2.cu -- instantiates the tree attention kernels of one cache format.
#include "kvq_tree_split.cuh"

namespace kvq {
TreeKernel tree_kernel_cb2(int D, int R) {
  return D == 64 ? tree::tree_kernel_info<KVQ_FMT_CB2_OUTLIER, 64>(R) : tree::tree_kernel_info<KVQ_FMT_CB2_OUTLIER, 128>(R);
}
}  // namespace kvq
