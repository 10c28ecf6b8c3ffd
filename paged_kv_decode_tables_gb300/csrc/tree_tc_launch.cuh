// Host-side launcher of the tensor-core tree attention instances.
#pragma once

#include <atomic>

#include "attention_launch.cuh"
#include "pkv_launch.cuh"
#include "tree_tc.cuh"

namespace pkv {
namespace detail {

template <typename T, typename KV, int D, int BS, bool BIASED>
pkv_status_t launch_tree_tc_kernel(const TreeParams &p, int ctas, cudaStream_t stream) {
  using Cfg = TreeTcCfg<T, KV, D, BS>;
  static std::atomic<unsigned long long> done{0};
  auto kernel = tree_tc_kernel<T, KV, D, BS, BIASED>;
  if constexpr (Cfg::NWG == 2) {
    // The kernel deals its launch registers out anew; compiled to fewer than it
    // deals out (they come in eights) its warps would wait for the rest forever.
    static const bool enough = [&] {
      cudaFuncAttributes a = {};
      return cudaFuncGetAttributes(&a, kernel) == cudaSuccess &&
             (a.numRegs + 7) / 8 * 8 * 4 >= 2 * Cfg::kSoftRegs + Cfg::kPrepRegs + Cfg::kIssueRegs;
    }();
    if (!enough) return PKV_ERR_UNSUPPORTED;
  }
  if (!ensure_smem_attr(kernel, Cfg::kSmem, done)) return PKV_ERR_CUDA;
  return launch_programmatic(kernel, dim3(ctas), dim3(Cfg::kThreads), Cfg::kSmem, stream, p) ==
                 cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

template <typename T, typename KV, int D, int BS>
pkv_status_t launch_tree_tc_as(const TreeParams &p, int ctas, cudaStream_t stream) {
  if (p.cap > 0.f || p.alibi != nullptr || !(p.scale > 0.f))
    return launch_tree_tc_kernel<T, KV, D, BS, true>(p, ctas, stream);
  return launch_tree_tc_kernel<T, KV, D, BS, false>(p, ctas, stream);
}

template <typename T, typename KV, int D>
pkv_status_t launch_tree_tc_d(const TreeParams &p, int ctas, cudaStream_t s) {
  switch (p.block_size) {
    case 8: return launch_tree_tc_as<T, KV, D, 8>(p, ctas, s);
    case 16: return launch_tree_tc_as<T, KV, D, 16>(p, ctas, s);
    case 32: return launch_tree_tc_as<T, KV, D, 32>(p, ctas, s);
    default: return PKV_ERR_UNSUPPORTED;
  }
}

}  // namespace detail

#define PKV_DEFINE_TREE_TC(name, T, KV)                                                      \
  pkv_status_t launch_tree_tc_##name(const TreeParams &p, int D, int ctas, cudaStream_t s) { \
    switch (D) {                                                                             \
      case 64: return detail::launch_tree_tc_d<T, KV, 64>(p, ctas, s);                       \
      case 128: return detail::launch_tree_tc_d<T, KV, 128>(p, ctas, s);                     \
      case 256: return detail::launch_tree_tc_d<T, KV, 256>(p, ctas, s);                     \
      default: return PKV_ERR_UNSUPPORTED;                                                   \
    }                                                                                        \
  }

}  // namespace pkv
