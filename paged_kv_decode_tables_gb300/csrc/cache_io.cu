// Writing tokens into the paged caches (with quantisation to 8-bit codes) and
// reading sequences back out of them.
//
// Both are copies with a change of layout, bounded by memory: a key chunk is
// 16 bytes of one token in the cache, and a value page holds each head dim's
// tokens next to one another, so values are transposed in 8 x 8 blocks (8
// tokens x 8 dims) in registers, between 16-byte accesses on the token side
// and 8-token runs on the cache side.
//
// Quantisation: code = the nearest code of the format to x / scale (an IEEE
// fp32 division; ties to even, beyond the largest finite value: that value,
// NaN stays NaN).  Reading back: code value * scale in fp32, rounded once to
// the output's type.
#include <type_traits>

#include "cache_io.cuh"
#include "pkv_launch.cuh"
#include "pkv_ptx.cuh"

namespace pkv {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// N elements from p, in accesses of up to 16 bytes (`aligned`: p is on such a
// boundary) or one by one.
template <typename E, int N, bool ALIGNED>
__device__ __forceinline__ void load_elems(const E *p, E (&v)[N]) {
  constexpr int kBytes = N * int(sizeof(E));
  if constexpr (ALIGNED && kBytes % 16 == 0) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i)
      reinterpret_cast<uint4 *>(v)[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
  } else if constexpr (ALIGNED && kBytes % 8 == 0) {
#pragma unroll
    for (int i = 0; i < kBytes / 8; ++i)
      reinterpret_cast<uint2 *>(v)[i] = __ldg(reinterpret_cast<const uint2 *>(p) + i);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i];
  }
}

template <typename E, int N, bool ALIGNED>
__device__ __forceinline__ void store_elems(E *p, const E (&v)[N]) {
  constexpr int kBytes = N * int(sizeof(E));
  if constexpr (ALIGNED && kBytes % 16 == 0) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i)
      reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(v)[i];
  } else if constexpr (ALIGNED && kBytes % 8 == 0) {
#pragma unroll
    for (int i = 0; i < kBytes / 8; ++i)
      reinterpret_cast<uint2 *>(p)[i] = reinterpret_cast<const uint2 *>(v)[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = v[i];
  }
}

// x / scale in fp32, correctly rounded.  DIV: by a division; else, for scales in
// [2^-60, 2^60], by Markstein's correction of the product with the rounded
// reciprocal (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): with inv = RN(1 / scale), q = RN(x inv) and the
// exact remainder c = x - q scale, RN(q + c inv) = RN(x / scale).  Three
// instructions instead of about ten; the divisions bound the copy.  A quotient
// beyond 10^30 saturates in the code either way, and one below 10^-30 is far
// below half of the smallest code (and keeps the sign of a zero).
template <bool DIV>
struct Quotient {
  float scale, inv;
  __device__ __forceinline__ explicit Quotient(float s) : scale(s), inv(1.f / s) {}
  __device__ __forceinline__ float operator()(float x) const {
    if constexpr (DIV) return __fdiv_rn(x, scale);
    const float q = x * inv;
    const float r = fmaf(fmaf(-q, scale, x), inv, q);
    return fabsf(q) > 1e-30f && fabsf(q) < 1e30f ? r : q;
  }
};

// Two elements as codes of the cache, the first in the low byte.
template <typename T, typename KV, bool DIV>
__device__ __forceinline__ uint32_t to_codes2(T a, T b, const Quotient<DIV> &by) {
  const float x = by(to_f32<T>(a)), y = by(to_f32<T>(b));
  uint16_t r;
  if constexpr (std::is_same<KV, fp8_e4m3_t>::value)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  else
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}

template <typename T, typename KV>
__device__ __forceinline__ T from_cache(KV c, float scale) {
  if constexpr (is_fp8<KV>::value) {
    uint32_t lo, hi;
    fp8x4_to_f16x2<KV>(c.bits, lo, hi);
    return from_f32<T>(unpack2<__half>(lo).x * scale);
  } else {
    return c;
  }
}

// ------------------------------------------------------------------- write --

constexpr int kWSide = 128;            // threads on the keys, and as many on the values
constexpr int kWThreads = 2 * kWSide;

// CTA (x, h): TOK tokens of kv head h, half of its warps on the keys and half on
// the values.  The tile's tokens are cut into groups of up to 8 consecutive
// slots that do not cross a multiple of 8: a group of 8 is a block of 8 tokens
// x 8 dims that is written 8 tokens at a time (a prompt), shorter ones go token
// by token (decode steps: every token has a page of its own).
template <typename T, typename KV, bool VEC, int TOK, bool DIV>
__global__ void __launch_bounds__(kWThreads) cache_write_kernel(const CacheWriteParams p) {
  constexpr int X = 16 / int(sizeof(KV));
  __shared__ int64_t slots[TOK];                  // -1: not written
  __shared__ int64_t page_k[TOK], page_v[TOK];    // element offset of the token's page
  __shared__ int slot_of[TOK];                    // slot in the page, -1: not written
  __shared__ int group_first[TOK], group_size[TOK];
  __shared__ int heads_of_warp[2];
  const int tid = threadIdx.x, D = p.head_size, BS = p.block_size, h = blockIdx.y;
  const int64_t i0 = int64_t(blockIdx.x) * TOK;
  grid_dependency_wait();
  allow_dependent_launch();
  int64_t slot = -1;
  if (tid < TOK) {
    if (i0 + tid < p.num_tokens) slot = p.slots[(i0 + tid) * p.slot_stride];
    if (slot >= p.num_slots) {
      flag_error(p.err, PKV_ERRF_BLOCK_ID);
      slot = -1;
    }
    if (slot < 0) slot = -1;
    const int64_t blk = slot < 0 ? 0 : slot / BS;
    page_k[tid] = blk * p.kc_s0 + int64_t(h) * p.kc_s1;
    page_v[tid] = blk * p.vc_s0 + int64_t(h) * p.vc_s1;
    slot_of[tid] = slot < 0 ? -1 : int(slot - blk * BS);
    slots[tid] = slot;
  }
  __syncthreads();
  bool head = false;
  unsigned heads = 0;
  if (tid < (TOK + 31) / 32 * 32) {
    head = slot >= 0 && (tid == 0 || slots[tid - 1] != slot - 1 || slot % 8 == 0);
    heads = __ballot_sync(kFull, head);
    if ((tid & 31) == 0) heads_of_warp[tid >> 5] = __popc(heads);
  }
  __syncthreads();
  if (head) {
    const int g = (tid >= 32 ? heads_of_warp[0] : 0) + __popc(heads & ((1u << (tid & 31)) - 1u));
    int n = 1;
    while (tid + n < TOK && slots[tid + n] == slot + n && (slot + n) % 8 != 0) ++n;
    group_first[g] = tid;
    group_size[g] = n;
  }
  const int ng = heads_of_warp[0] + (TOK > 32 ? heads_of_warp[1] : 0);
  __syncthreads();
  if (tid < kWSide) {
    // values: (group, 8 dims) blocks
    const T *value = static_cast<const T *>(p.value) + int64_t(h) * p.v_s1;
    KV *vc = static_cast<KV *>(p.value_cache);
    const int shift = 31 - __clz(D / 8);
    const Quotient<DIV> by(p.v_scale);
    for (int i = tid; i < ng << shift; i += kWSide) {
      const int g = i >> shift, d = (i - (g << shift)) * 8;
      const int t0 = group_first[g], n = group_size[g];
      KV *dst = vc + page_v[t0] + int64_t(d) * BS + slot_of[t0];
      alignas(16) T x[8][8];  // [token][dim]
      if constexpr (!is_fp8<KV>::value) {
        if (n == 8) {
          alignas(16) KV b[8][8];  // [dim][token]
#pragma unroll
          for (int t = 0; t < 8; ++t)
            load_elems<T, 8, VEC>(value + (i0 + t0 + t) * p.v_s0 + d, x[t]);
#pragma unroll
          for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e][t] = x[t][e];
#pragma unroll
          for (int e = 0; e < 8; ++e) store_elems<KV, 8, true>(dst + e * BS, b[e]);
          continue;
        }
      }
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t < n) load_elems<T, 8, VEC>(value + (i0 + t0 + t) * p.v_s0 + d, x[t]);
      if constexpr (is_fp8<KV>::value) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) w[t] = to_codes2<T, KV, DIV>(x[2 * t][e], x[2 * t + 1][e], by);
          if (n == 8) {
            *reinterpret_cast<uint2 *>(dst + e * BS) =
                make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
          } else {
#pragma unroll
            for (int t = 0; t < 7; ++t)
              if (t < n) dst[e * BS + t].bits = uint8_t(w[t >> 1] >> (t & 1) * 8);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int t = 0; t < 7; ++t)
            if (t < n) dst[e * BS + t] = x[t][e];
      }
    }
  } else {
    // keys: chunks of a token across lanes, so rows are read whole; four loads in flight
    const T *key = static_cast<const T *>(p.key) + int64_t(h) * p.k_s1;
    KV *kc = static_cast<KV *>(p.key_cache);
    const int shift = 31 - __clz(D / X);
    const Quotient<DIV> by(p.k_scale);
    constexpr int U = 4;
    for (int i = tid - kWSide; i < TOK << shift; i += U * kWSide) {
      alignas(16) T x[U][X];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = i + u * kWSide, t = j >> shift, c = j - (t << shift);
        if (t < TOK && slot_of[t] >= 0)
          load_elems<T, X, VEC>(key + (i0 + t) * p.k_s0 + c * X, x[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = i + u * kWSide, t = j >> shift, c = j - (t << shift);
        if (t >= TOK || slot_of[t] < 0) continue;
        KV *dst = kc + page_k[t] + (int64_t(c) * BS + slot_of[t]) * X;
        if constexpr (is_fp8<KV>::value) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = to_codes2<T, KV, DIV>(x[u][2 * e], x[u][2 * e + 1], by);
          *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16,
                                                       w[4] | w[5] << 16, w[6] | w[7] << 16);
        } else {
          store_elems<KV, X, true>(dst, x[u]);
        }
      }
    }
  }
}

// -------------------------------------------------------------------- read --

constexpr int kRThreads = 256;

// A warp per (page of a sequence, kv head).  The pages of all sequences are
// numbered without a scan of their counts: sequence s takes the numbers from
// cu[s] / BS + 2 s on, which leaves it at least as many as the pages that its
// tokens touch (a few numbers stay unused); the warp finds s by a search with
// 32 probes a step.
template <typename T, typename KV, bool VEC>
__global__ void __launch_bounds__(kRThreads) cache_read_kernel(const CacheReadParams p) {
  constexpr int X = 16 / int(sizeof(KV));
  const int lane = threadIdx.x & 31, D = p.head_size, BS = p.block_size;
  const int64_t w = int64_t(blockIdx.x) * (kRThreads / 32) + (threadIdx.x >> 5);
  const int64_t u = w / p.num_kv_heads;
  const int h = int(w - u * p.num_kv_heads);
  grid_dependency_wait();
  allow_dependent_launch();
  // the last s with cu[s] / BS + 2 s <= u
  int lo = 0, hi = p.num_seqs;  // s is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int s = lo + lane * step;
    const bool le = s < hi && (s == lo || max(p.cu[s], 0) / BS + 2 * int64_t(s) <= u);
    const unsigned b = __ballot_sync(kFull, le);
    const int last = 31 - __clz(int(b));  // lane 0 is always set
    lo += last * step;
    hi = min(hi, lo + step);
  }
  const int s = lo;
  const int c0 = p.cu[s], c1 = p.cu[s + 1];
  const int first = p.starts ? p.starts[s] : 0;
  int64_t row = int64_t(s) * p.bt_s0, cap = p.max_blocks_per_seq;
  if (p.indptr) {
    const int a = p.indptr[s];
    row = int64_t(max(a, 0)) * p.bt_s1;
    cap = a < 0 ? 0 : int64_t(p.indptr[s + 1]) - a;
  }
  if (c0 < 0 || c1 < c0 || c1 > p.num_tokens || cap < 0) {
    if (lane == 0) flag_error(p.err, PKV_ERRF_INDPTR);
    return;
  }
  if (first < 0 || int64_t(first) + (c1 - c0) > cap * BS) {
    if (lane == 0 && c1 > c0) flag_error(p.err, PKV_ERRF_SEQ_LEN);
    if (first < 0) return;
  }
  const int64_t page = first / BS + (u - (c0 / BS + 2 * int64_t(s)));
  // tokens [t0, t1) of the sequence stand in this page
  const int64_t t0 = max(page * BS, int64_t(first));
  const int64_t t1 = min((page + 1) * BS, int64_t(first) + (c1 - c0));
  if (t0 >= t1 || page >= cap) return;
  int blk = p.bt[row + page * p.bt_s1];
  if (blk < 0 || blk >= p.num_blocks) {
    if (lane == 0) flag_error(p.err, PKV_ERRF_BLOCK_ID);
    blk = 0;
  }
  const int a = int(t0 - page * BS), b = int(t1 - page * BS);  // slots [a, b)
  const int64_t out0 = c0 + (page * BS - first);               // output row of slot 0
  const KV *kc = static_cast<const KV *>(p.key_cache) + int64_t(blk) * p.kc_s0 + int64_t(h) * p.kc_s1;
  const KV *vc = static_cast<const KV *>(p.value_cache) + int64_t(blk) * p.vc_s0 + int64_t(h) * p.vc_s1;
  T *key = static_cast<T *>(p.key) + out0 * p.k_s0 + int64_t(h) * p.k_s1;
  T *value = static_cast<T *>(p.value) + out0 * p.v_s0 + int64_t(h) * p.v_s1;
  const int chunks = D / X;
  for (int i = lane; i < chunks * BS; i += 32) {
    const int t = i / chunks, c = i - t * chunks;
    if (t < a || t >= b) continue;
    alignas(16) KV q[X];
    alignas(16) T x[X];
    load_elems<KV, X, true>(kc + (c * BS + t) * X, q);
#pragma unroll
    for (int e = 0; e < X; ++e) x[e] = from_cache<T, KV>(q[e], p.k_scale);
    store_elems<T, X, VEC>(key + int64_t(t) * p.k_s0 + c * X, x);
  }
  // blocks of 8 tokens x 8 dims, the page's token groups next to one another
  const int groups = BS / 8;
  for (int i = lane; i < groups * (D / 8); i += 32) {
    const int g = i % groups, d = i / groups * 8;
    alignas(16) KV q[8][8];  // [dim][token]
#pragma unroll
    for (int e = 0; e < 8; ++e) load_elems<KV, 8, true>(vc + (d + e) * BS + g * 8, q[e]);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (g * 8 + t < a || g * 8 + t >= b) continue;
      alignas(16) T x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = from_cache<T, KV>(q[e][t], p.v_scale);
      store_elems<T, 8, VEC>(value + int64_t(g * 8 + t) * p.v_s0 + d, x);
    }
  }
}

// ------------------------------------------------------------------ launch --

// Tokens of a CTA: 64 (a prompt's tiles), or 16 where that leaves fewer than 512
// CTAs (decode steps: 512 tokens x 8 kv heads in E4M3 would be 64 CTAs whose
// threads write 64 bytes one by one eight times over).
template <typename T, typename KV, bool VEC, bool DIV>
cudaError_t write_vec(const CacheWriteParams &p, cudaStream_t s) {
  const int64_t tiles = (int64_t(p.num_tokens) + 63) / 64;
  if (tiles * p.num_kv_heads >= 512)
    return launch_programmatic(cache_write_kernel<T, KV, VEC, 64, DIV>, dim3(tiles, p.num_kv_heads),
                               dim3(kWThreads), 0, s, p);
  return launch_programmatic(cache_write_kernel<T, KV, VEC, 16, DIV>,
                             dim3((int64_t(p.num_tokens) + 15) / 16, p.num_kv_heads), dim3(kWThreads),
                             0, s, p);
}

template <typename T, typename KV>
cudaError_t write_as(const CacheWriteParams &p, bool vec, cudaStream_t s) {
  if constexpr (is_fp8<KV>::value) {
    auto plain = [](float x) { return x >= 0x1p-60f && x <= 0x1p60f; };
    if (!plain(p.k_scale) || !plain(p.v_scale))
      return vec ? write_vec<T, KV, true, true>(p, s) : write_vec<T, KV, false, true>(p, s);
  }
  return vec ? write_vec<T, KV, true, false>(p, s) : write_vec<T, KV, false, false>(p, s);
}

template <typename T, typename KV>
cudaError_t read_as(const CacheReadParams &p, bool vec, cudaStream_t s) {
  const int64_t pages = p.num_tokens / p.block_size + 2 * int64_t(p.num_seqs);
  const int64_t warps = pages * p.num_kv_heads;
  const dim3 grid((warps + kRThreads / 32 - 1) / (kRThreads / 32));
  if (vec) return launch_programmatic(cache_read_kernel<T, KV, true>, grid, dim3(kRThreads), 0, s, p);
  return launch_programmatic(cache_read_kernel<T, KV, false>, grid, dim3(kRThreads), 0, s, p);
}

// F(T, KV) for the element types of (dtype, kv); F returns a cudaError_t.
template <typename F>
pkv_status_t dispatch(pkv_dtype_t dtype, int32_t kv, F &&f) {
  cudaError_t e;
  const int k = kv == PKV_KV_AUTO ? 0 : (kv == PKV_KV_FP8_E4M3 ? 1 : 2);
  if (dtype == PKV_F32 && k == 0)
    e = f(float(), float());
  else if (dtype == PKV_F16)
    e = k == 0 ? f(__half(), __half()) : (k == 1 ? f(__half(), fp8_e4m3_t()) : f(__half(), fp8_e5m2_t()));
  else if (dtype == PKV_BF16)
    e = k == 0 ? f(__nv_bfloat16(), __nv_bfloat16())
               : (k == 1 ? f(__nv_bfloat16(), fp8_e4m3_t()) : f(__nv_bfloat16(), fp8_e5m2_t()));
  else
    return PKV_ERR_UNSUPPORTED;
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

pkv_status_t launch_cache_write(const CacheWriteParams &p, pkv_dtype_t dtype, int32_t kv, bool vec,
                                cudaStream_t stream) {
  return dispatch(dtype, kv, [&](auto t, auto c) {
    return write_as<decltype(t), decltype(c)>(p, vec, stream);
  });
}

pkv_status_t launch_cache_read(const CacheReadParams &p, pkv_dtype_t dtype, int32_t kv, bool vec,
                               cudaStream_t stream) {
  return dispatch(dtype, kv, [&](auto t, auto c) {
    return read_as<decltype(t), decltype(c)>(p, vec, stream);
  });
}

}  // namespace pkv
