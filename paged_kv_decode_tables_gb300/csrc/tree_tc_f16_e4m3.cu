// Tensor-core tree attention instances: fp16 queries over E4M3 caches.
#include "tree_tc_launch.cuh"

namespace pkv {

PKV_DEFINE_TREE_TC(f16_e4m3, __half, fp8_e4m3_t)

}  // namespace pkv
