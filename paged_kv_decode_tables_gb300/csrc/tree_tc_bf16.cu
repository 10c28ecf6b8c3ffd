// Tensor-core tree attention instances: bf16 queries and caches.
#include "tree_tc_launch.cuh"

namespace pkv {

PKV_DEFINE_TREE_TC(bf16, __nv_bfloat16, __nv_bfloat16)

}  // namespace pkv
