// Tree attention in fp32, on the CUDA cores (the split, the masks and the join
// are described in tree.cuh).
//
// One CTA of 128 threads takes 32 query rows against tiles of 64 tokens: the
// tile's keys go to shared memory token by token, thread (rg, tg) computes
// the scores of rows 4 rg .. 4 rg + 3 with tokens tg, tg + 16, ..., the
// online softmax runs over the 16 lanes that share rows, and after the tile's
// values have replaced its keys the thread adds its rows' products for dims
// 4 tg .. 4 tg + 3 (+ 64 j).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "attention_launch.cuh"
#include "pkv_launch.cuh"
#include "tree.cuh"

namespace pkv {

namespace {

constexpr int kRT = kTreeSimtRows, kTT = kTreeSimtTokens, kUC = kTreeSimtUnitCost, kThreads = 128;

template <int D>
struct SimtCfg {
  static constexpr int kPitch = D + 4;  // floats; spreads the rows of a column over the banks
  static constexpr int kSmem = (kRT * kPitch + kTT * kPitch + kRT * (kTT + 4)) * 4;
};

template <int D, int BS>
__global__ void __launch_bounds__(kThreads, kTreeSimtCtasPerSm) tree_simt_kernel(const TreeParams p) {
  using Cfg = SimtCfg<D>;
  constexpr int X = 4;  // elements of 16 bytes: a key chunk's dims, a value load's tokens
  constexpr int kPitch = Cfg::kPitch, kPP = kTT + 4;
  extern __shared__ __align__(16) float tree_simt_smem[];
  float *qs = tree_simt_smem;
  float *kv = qs + kRT * kPitch;
  float *ps = kv + kTT * kPitch;
  __shared__ TreeScratch<kThreads> scratch;
  __shared__ int ids[kTT / 8];
  const int tid = threadIdx.x, rg = tid >> 4, tg = tid & 15;
  grid_dependency_wait();
  allow_dependent_launch();
  const TreeRun run = tree_find_run<kTT, kRT, kUC, kThreads>(p, scratch);
  if (run.begin >= run.end) {
    if (tid == 0) tree_write_cut<kUC>(p, run, nullptr);
    return;
  }
  const TreeLogit logit(p);
  const bool plain = p.cap == 0.f && p.alibi == nullptr;
  TreeWalk<kTT, kRT, kUC> walk;
  walk.start(p, run);
  TreeStretch st;
  bool first = true;
  while (walk.next(p, st)) {
    if (first && tid == 0) tree_write_cut<kUC>(p, run, &st);
    // queries of the row tile (rows past the end: zeros)
    __syncthreads();
    for (int i = tid; i < kRT * D; i += kThreads) {
      const int r = i / D, d = i % D, R = st.row0 + r;
      float x = 0.f;
      if (r < st.rows)
        x = static_cast<const float *>(p.q)[int64_t(st.q.q0 + R / p.group) * p.q_s0 +
                                            int64_t(st.kvh * p.group + R % p.group) * p.q_s1 +
                                            int64_t(d) * p.q_s2];
      qs[r * kPitch + d] = x;
    }
    int node[4];
    int qpos[4];
    float slope[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int R = st.row0 + min(rg * 4 + i, st.rows - 1);
      node[i] = R / p.group;
      slope[i] = p.alibi ? p.alibi[st.kvh * p.group + R % p.group] * kLog2e : 0.f;
      qpos[i] = p.positions ? p.positions[st.q.q0 + node[i]] : st.q.ctx + node[i];
    }
    float m[4], l[4], acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) acc[i][e] = 0.f;
    }
    const int64_t row = tree_table_row(p, st.seq);
    const float *kb = static_cast<const float *>(p.k) + int64_t(st.kvh) * p.k_s1;
    const float *vb = static_cast<const float *>(p.v) + int64_t(st.kvh) * p.v_s1;
    for (int tile = st.tile0; tile < st.tile1; ++tile) {
      const int t0 = tile * kTT, n = min(kTT, st.q.L - t0);  // n <= 0: no tokens at all
      __syncthreads();
      if (tid < kTT / BS && tid * BS < n) ids[tid] = tree_block_id(p, row, t0 / BS + tid);
      __syncthreads();
      for (int i = tid; i < kTT * (D / X); i += kThreads) {
        const int t = i % kTT, c = i / kTT;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < n)
          f = __ldg(reinterpret_cast<const float4 *>(kb + int64_t(ids[t / BS]) * p.k_s0 +
                                                     (c * BS + t % BS) * X));
        *reinterpret_cast<float4 *>(kv + t * kPitch + c * X) = f;
      }
      __syncthreads();
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = *reinterpret_cast<const float4 *>(qs + (rg * 4 + i) * kPitch + d);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          b[j] = *reinterpret_cast<const float4 *>(kv + (tg + 16 * j) * kPitch + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = fmaf(a[i].x, b[j].x,
                           fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
      }
      const bool tail = t0 + kTT > st.q.ctx;  // tokens that not every row sees
      float shrinks[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = m[i], x4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = t0 + tg + 16 * j;
          float x = p.cap > 0.f ? logit.capped_exact(s[i][j]) : logit.plain(s[i][j]);
          bool seen = true;
          int kpos = t;
          if (tail && t >= st.q.ctx) {
            const int jn = t - st.q.ctx;
            seen = t < st.q.L;
            if (seen) {
              if (p.positions) kpos = p.positions[st.q.q0 + jn];
              seen = p.mask ? jn < p.mask_cols &&
                                  p.mask[int64_t(st.q.q0 + node[i]) * p.m_s0 + jn * p.m_s1] != 0
                            : jn <= node[i];
            }
          }
          x = fmaf(slope[i], float(kpos - qpos[i]), x);
          x4[j] = seen ? x : -INFINITY;
          top = fmaxf(top, x4[j]);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float ref = top == -INFINITY ? 0.f : top;
        const float shrink = ex2(m[i] - ref);
        m[i] = top;
        shrinks[i] = shrink;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // without cap and bias the scaled score goes into the difference unrounded
          const float e = ex2(plain && x4[j] != -INFINITY
                                  ? fmaf(s[i][j], logit.scale_log2, -ref)
                                  : x4[j] - ref);
          sum += e;
          ps[(rg * 4 + i) * kPP + tg + 16 * j] = e;
        }
        l[i] = fmaf(l[i], shrink, sum);
      }
      __syncthreads();
      for (int i = tid; i < (kTT / X) * D; i += kThreads) {
        const int d = i % D, t = i / D * X;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < n)
          f = __ldg(reinterpret_cast<const float4 *>(vb + int64_t(ids[t / BS]) * p.v_s0 + d * BS + t % BS));
        kv[t * kPitch + d] = f.x;  // (t < n: the 4 tokens are of one page; zeros past the end)
        kv[(t + 1) * kPitch + d] = t + 1 < n ? f.y : 0.f;
        kv[(t + 2) * kPitch + d] = t + 2 < n ? f.z : 0.f;
        kv[(t + 3) * kPitch + d] = t + 3 < n ? f.w : 0.f;
      }
      __syncthreads();
      // The tile's products are summed by themselves and then added: next to a
      // token that holds almost all the weight, thousands of small ones would each
      // vanish in the rounding of a running sum.
      float add[4][D / 16];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < D / 16; ++e) add[i][e] = 0.f;
      auto product = [&](auto masked) {
#pragma unroll 2
        for (int t = 0; t < kTT; ++t) {
          float pr[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) pr[i] = ps[(rg * 4 + i) * kPP + t];
#pragma unroll
          for (int e = 0; e < D / 64; ++e) {
            const float4 v = *reinterpret_cast<const float4 *>(kv + t * kPitch + e * 64 + tg * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // a value that a row does not see may be anything, NaN too
              if (masked.value && pr[i] == 0.f) continue;
              add[i][4 * e] = fmaf(pr[i], v.x, add[i][4 * e]);
              add[i][4 * e + 1] = fmaf(pr[i], v.y, add[i][4 * e + 1]);
              add[i][4 * e + 2] = fmaf(pr[i], v.z, add[i][4 * e + 2]);
              add[i][4 * e + 3] = fmaf(pr[i], v.w, add[i][4 * e + 3]);
            }
          }
        }
      };
      if (tail)
        product(std::true_type{});
      else
        product(std::false_type{});
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[i][e] = fmaf(acc[i][e], shrinks[i], add[i][e]);
    }
    // the 16 lanes of a row hold a share of its sum each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
    }
    const bool whole = st.tile0 == 0 && st.tile1 == st.tiles;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = rg * 4 + i;
      if (r >= st.rows) continue;
      if (whole) {
        const int R = st.row0 + r;
        float *o = static_cast<float *>(p.out) + int64_t(st.q.q0 + R / p.group) * p.o_s0 +
               int64_t(st.kvh * p.group + R % p.group) * p.o_s1;
        const float inv = l[i] == 0.f ? 0.f : __fdiv_rn(p.out_scale, l[i]);
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
          o[int64_t((e >> 2) * 64 + tg * 4 + (e & 3)) * p.o_s2] = acc[i][e] * inv;
      } else {
        const int64_t part = (2 * int64_t(blockIdx.x) + (first ? 0 : 1)) * kRT + r;
        if (tg == 0) p.ml[part] = make_float2(m[i], l[i]);
#pragma unroll
        for (int e = 0; e < D / 64; ++e)
          p.acc[((part - r) / kRT * (D / 4) + e * 16 + tg) * kRT + r] =
              make_float4(acc[i][4 * e], acc[i][4 * e + 1], acc[i][4 * e + 2], acc[i][4 * e + 3]);
      }
    }
    first = false;
  }
  if (first && tid == 0) tree_write_cut<kUC>(p, run, nullptr);
}

template <int D, int BS>
pkv_status_t launch(const TreeParams &p, int ctas, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  auto kernel = tree_simt_kernel<D, BS>;
  constexpr int smem = SimtCfg<D>::kSmem;
  if (!detail::ensure_smem_attr(kernel, smem, done)) return PKV_ERR_CUDA;
  return launch_programmatic(kernel, dim3(ctas), dim3(kThreads), smem, stream, p) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

template <int D>
pkv_status_t by_block(const TreeParams &p, int ctas, cudaStream_t s) {
  switch (p.block_size) {
    case 8: return launch<D, 8>(p, ctas, s);
    case 16: return launch<D, 16>(p, ctas, s);
    case 32: return launch<D, 32>(p, ctas, s);
    default: return PKV_ERR_UNSUPPORTED;
  }
}

}  // namespace

pkv_status_t launch_tree_simt(const TreeParams &p, int D, int ctas, cudaStream_t stream) {
  switch (D) {
    case 64: return by_block<64>(p, ctas, stream);
    case 128: return by_block<128>(p, ctas, stream);
    default: return PKV_ERR_UNSUPPORTED;
  }
}

}  // namespace pkv
