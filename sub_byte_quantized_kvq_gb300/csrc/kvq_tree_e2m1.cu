// kvq_tree_e2m1.cu -- instantiates the tree attention kernels of one cache format.
#include "kvq_tree_split.cuh"

namespace kvq {
TreeKernel tree_kernel_e2m1(int D, int R) {
  return D == 64 ? tree::tree_kernel_info<KVQ_FMT_FP4_E2M1_S16, 64>(R) : tree::tree_kernel_info<KVQ_FMT_FP4_E2M1_S16, 128>(R);
}
}  // namespace kvq
