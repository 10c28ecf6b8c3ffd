// Tensor-core tree attention instances: bf16 queries over E5M2 caches.
#include "tree_tc_launch.cuh"

namespace pkv {

PKV_DEFINE_TREE_TC(bf16_e5m2, __nv_bfloat16, fp8_e5m2_t)

}  // namespace pkv
