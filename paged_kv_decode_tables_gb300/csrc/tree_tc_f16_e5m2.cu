// Tensor-core tree attention instances: fp16 queries over E5M2 caches.
#include "tree_tc_launch.cuh"

namespace pkv {

PKV_DEFINE_TREE_TC(f16_e5m2, __half, fp8_e5m2_t)

}  // namespace pkv
