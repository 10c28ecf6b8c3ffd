// Tensor-core tree attention instances: fp16 queries and caches.
#include "tree_tc_launch.cuh"

namespace pkv {

PKV_DEFINE_TREE_TC(f16, __half, __half)

}  // namespace pkv
