// Joins the units that the tree attention's split cut between CTAs: a
// log-sum-exp combination of their partial sums, out = sum_c 2^(m_c - M) acc_c
// / sum_c 2^(m_c - M) l_c with M = max m_c.  A row that sees no token has every
// l_c = 0 and gets zeros.
//
// CTA (c, y): the unit that describes itself at cut c (see tree_write_cut), its
// dims 8 y .. 8 y + 7; most cuts are none and their CTAs return after one load.
// A thread takes four dims of a row, rows along the lanes as the partial
// results are laid out, and adds its partials in order: the sum does not
// depend on timing.
#include "pkv_launch.cuh"
#include "tree.cuh"

namespace pkv {

namespace {

constexpr int kQuads = 2;  // groups of four dims of a CTA

// s + c += x (c: what the sum's roundings have lost so far; 0 once s is not
// finite).  Next to a part that holds almost all the weight, hundreds of small
// ones would each vanish in the rounding of a plain running sum.
__device__ __forceinline__ void add_carry(float &s, float &c, float x) {
  const float y = __fadd_rn(x, c), t = __fadd_rn(s, y);
  c = fabsf(t) < INFINITY ? __fsub_rn(y, __fsub_rn(t, s)) : 0.f;
  s = t;
}

template <typename T, int D, int RT>
__global__ void __launch_bounds__(RT * kQuads) tree_join_kernel(const TreeParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int c0 = blockIdx.x + 1;  // CTA 0's run starts inside no unit
  const TreeCut &at = p.cuts[c0];
  const int r = threadIdx.x % RT, quad = blockIdx.y * kQuads + threadIdx.x / RT;
  if (!at.valid || r >= at.rows) return;
  const TreeCut cut = at;
  auto start_of = [&](int64_t c) { return cut.each * c + (c < cut.extra ? c : cut.extra); };
  // Partial i: of CTA c0 - 1 + i, its run's first stretch, but for a CTA whose
  // run began before the unit.
  const int64_t part0 = 2 * int64_t(c0 - 1) + (start_of(c0 - 1) < cut.begin ? 1 : 0);
  const int more = int(min(int64_t(cut.parts - c0), tree_div(cut.end - start_of(c0) - 1, cut.each) + 1));
  auto part_of = [&](int i) { return i == 0 ? part0 : 2 * int64_t(c0 - 1 + i); };
  auto counts = [&](int i) { return start_of(c0 - 1 + i) < cut.end; };
  int n = 1 + more;  // at least as many as there are: runs hold `each` tiles or one more
  while (n > 1 && !counts(n - 1)) --n;
  float M = -INFINITY;
#pragma unroll 8
  for (int i = 0; i < n; ++i) M = fmaxf(M, __ldcg(p.ml + part_of(i) * RT + r).x);
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, carry[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f, l_carry = 0.f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float2 ml = __ldcg(p.ml + part_of(i) * RT + r);
    const float4 a = __ldcg(p.acc + (part_of(i) * (D / 4) + quad) * RT + r);
    // a part whose row saw nothing has l = 0; one whose every score is NaN has l = NaN
    const float w = ml.x == -INFINITY ? 1.f : ex2(ml.x - M);
    add_carry(l, l_carry, w * ml.y);
    if (ml.x != -INFINITY) {
      add_carry(acc[0], carry[0], w * a.x);
      add_carry(acc[1], carry[1], w * a.y);
      add_carry(acc[2], carry[2], w * a.z);
      add_carry(acc[3], carry[3], w * a.w);
    }
  }
  const float inv = l == 0.f ? 0.f : __fdiv_rn(p.out_scale, l);
  const int R = cut.row0 + r;
  T *o = static_cast<T *>(p.out) + int64_t(cut.q0 + R / p.group) * p.o_s0 +
         int64_t(cut.kvh * p.group + R % p.group) * p.o_s1;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[int64_t(quad * 4 + e) * p.o_s2] = from_f32<T>(acc[e] * inv);
}

template <typename T, int RT>
pkv_status_t launch(const TreeParams &p, int D, int ctas, cudaStream_t s) {
  const dim3 grid(ctas - 1, D / (4 * kQuads)), block(RT * kQuads);
  cudaError_t e;
  switch (D) {
    case 64: e = launch_programmatic(tree_join_kernel<T, 64, RT>, grid, block, 0, s, p); break;
    case 128: e = launch_programmatic(tree_join_kernel<T, 128, RT>, grid, block, 0, s, p); break;
    case 256: e = launch_programmatic(tree_join_kernel<T, 256, RT>, grid, block, 0, s, p); break;
    default: return PKV_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

pkv_status_t launch_tree_join(const TreeParams &p, pkv_dtype_t dtype, int head_size, int ctas,
                              cudaStream_t stream) {
  if (ctas < 2) return PKV_OK;
  switch (dtype) {
    case PKV_F32: return launch<float, kTreeSimtRows>(p, head_size, ctas, stream);
    case PKV_F16: return launch<__half, kTreeTcRows>(p, head_size, ctas, stream);
    case PKV_BF16: return launch<__nv_bfloat16, kTreeTcRows>(p, head_size, ctas, stream);
    default: return PKV_ERR_UNSUPPORTED;
  }
}

}  // namespace pkv
