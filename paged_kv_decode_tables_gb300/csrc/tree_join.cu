// Joins the units that the tree attention's split cut between CTAs: a
// log-sum-exp combination of their partial sums, out = sum_c 2^(m_c - M) acc_c
// / sum_c 2^(m_c - M) l_c with M = max m_c.  A row that sees no token has every
// l_c = 0 and gets zeros.
//
// CTA (c, y): the unit that describes itself at cut c (see tree_write_cut),
// its rows 8 y .. 8 y + 7, a row per warp; most cuts are none and their CTAs
// return after one load.  A warp takes its row's partials in order: the sum
// does not depend on timing.
#include "pkv_launch.cuh"
#include "tree.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;

// s + c += x (c: what the sum's roundings have lost so far; 0 once s is not finite).
__device__ __forceinline__ void add_carry(float &s, float &c, float x) {
  const float y = __fadd_rn(x, c), t = __fadd_rn(s, y);
  c = fabsf(t) < INFINITY ? __fsub_rn(y, __fsub_rn(t, s)) : 0.f;
  s = t;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) tree_join_kernel(const TreeParams p, int RT) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  allow_dependent_launch();
  const int c0 = blockIdx.x + 1;  // CTA 0's run starts no unit's middle
  const TreeCut cut = p.cuts[c0];
  const int r = blockIdx.y * kWarps + warp;
  if (!cut.valid || r >= cut.rows) return;
  // contributors: CTA c0 - 1 and every later one whose run starts before the unit's end
  int n = 1;
  {
    int c = c0;
    while (c + 31 < cut.parts && tree_start(cut.total, c + 31, cut.parts) < cut.end) c += 32, n += 32;
    const bool in = c + lane < cut.parts && tree_start(cut.total, c + lane, cut.parts) < cut.end;
    n += __popc(__ballot_sync(0xffffffffu, in));
  }
  // partial i: CTA c0 - 1 + i, its first stretch's slot but for a CTA whose
  // run began before the unit
  const int64_t tail = tree_start(cut.total, c0 - 1, cut.parts) < cut.begin ? 1 : 0;
  auto row_of = [&](int i) { return (2 * int64_t(c0 - 1 + i) + (i == 0 ? tail : 0)) * RT + r; };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(p.ml + row_of(i)).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  // Sums with their rounding errors carried along (Kahan): next to a part that
  // holds almost all the weight, hundreds of small ones would each vanish in
  // the rounding of a running sum.
  float acc[V], acc_c[V], l = 0.f, l_c = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = acc_c[e] = 0.f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const int64_t row = row_of(i);
    const float2 ml = __ldcg(p.ml + row);
    // a part whose row saw nothing has l = 0; one whose every score is NaN has l = NaN
    const float w = ml.x == -INFINITY ? 1.f : ex2(ml.x - M);
    add_carry(l, l_c, w * ml.y);
    const float *a = p.acc + row * D;
    if (ml.x != -INFINITY) {
#pragma unroll
      for (int e = 0; e < V; ++e) add_carry(acc[e], acc_c[e], w * __ldcg(a + e * 32 + lane));
    }
  }
  const float inv = l > 0.f || l != l ? __fdiv_rn(p.out_scale, l) : 0.f;
  const int R = cut.row0 + r;
  const int tok = cut.q0 + R / p.group, h = cut.kvh * p.group + R % p.group;
  T *o = static_cast<T *>(p.out) + int64_t(tok) * p.o_s0 + int64_t(h) * p.o_s1;
#pragma unroll
  for (int e = 0; e < V; ++e) o[int64_t(e * 32 + lane) * p.o_s2] = from_f32<T>(acc[e] * inv);
}

template <typename T>
pkv_status_t launch(const TreeParams &p, int D, int rows, int ctas, cudaStream_t s) {
  const dim3 grid(ctas - 1, (rows + kWarps - 1) / kWarps), block(kWarps * 32);
  cudaError_t e;
  switch (D) {
    case 64: e = launch_programmatic(tree_join_kernel<T, 64>, grid, block, 0, s, p, rows); break;
    case 128: e = launch_programmatic(tree_join_kernel<T, 128>, grid, block, 0, s, p, rows); break;
    case 256: e = launch_programmatic(tree_join_kernel<T, 256>, grid, block, 0, s, p, rows); break;
    default: return PKV_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

pkv_status_t launch_tree_join(const TreeParams &p, pkv_dtype_t dtype, int head_size, int rows,
                              int ctas, cudaStream_t stream) {
  if (ctas < 2) return PKV_OK;
  switch (dtype) {
    case PKV_F32: return launch<float>(p, head_size, rows, ctas, stream);
    case PKV_F16: return launch<__half>(p, head_size, rows, ctas, stream);
    case PKV_BF16: return launch<__nv_bfloat16>(p, head_size, rows, ctas, stream);
    default: return PKV_ERR_UNSUPPORTED;
  }
}

}  // namespace pkv
