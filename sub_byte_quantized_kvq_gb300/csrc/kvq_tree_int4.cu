// kvq_tree_int4.cu -- instantiates the tree attention kernels of one cache format.
#include "kvq_tree_split.cuh"

namespace kvq {
TreeKernel tree_kernel_int4(int D, int R) {
  return D == 64 ? tree::tree_kernel_info<KVQ_FMT_INT4_G32, 64>(R) : tree::tree_kernel_info<KVQ_FMT_INT4_G32, 128>(R);
}
}  // namespace kvq
