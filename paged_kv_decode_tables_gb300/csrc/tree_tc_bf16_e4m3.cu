// Tensor-core tree attention instances: bf16 queries over E4M3 caches.
#include "tree_tc_launch.cuh"

namespace pkv {

PKV_DEFINE_TREE_TC(bf16_e4m3, __nv_bfloat16, fp8_e4m3_t)

}  // namespace pkv
