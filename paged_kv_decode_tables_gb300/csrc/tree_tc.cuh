// Tree attention on the 5th-generation tensor cores: fp16 / bf16 queries over
// 16-bit or 8-bit caches (the split, the masks and the join: tree.cuh).
//
// One CTA per SM runs its stretches of (sequence, kv head, 128 query rows) x
// tiles of 64 tokens.  Per tile
//   S = Q K^T     M = 128 rows, N = tokens, K = head dims: Q from tensor memory
//   O += P V      M = 128 rows, N = head dims, K = tokens: P from tensor memory
// with S, P and O in tensor memory.  The pages are used as they lie in the
// cache, fetched by whole-page bulk copies:
// - a key page [D / 8][BS][8] holds 8 tokens x 16 bytes in 128 contiguous
//   bytes, the core matrix of an operand without swizzling: the 8-token
//   groups number h of all pages of the tile (a page apart) make one MMA, so S
//   comes out with its tokens permuted at 16 tokens a page (column 32 h + 8 page
//   + i is token 16 page + 8 h + i), which a softmax does not mind;
// - a value page [D][BS] has rows of 16, 32 or 64 bytes of one dim's tokens:
//   an operand with K = tokens adjacent, for 32 (64) bytes under the 32 (64)
//   byte swizzle, which exchanges 16-byte pieces within rows; the prep warps
//   do that in place (half of the rows at 16 tokens a page).
// 8-bit codes are widened by the prep warps to f16 (exact for both formats)
// in the 16-bit page layout; queries then enter as f16, bf16 ones scaled by a
// power of two per row.  P enters as a hi + lo pair of 16-bit values (about
// 2^-17 relative error with bf16, less with f16; a single bf16 would cost as
// much as rounding the output once more), two MMAs a product, in the columns of
// the S tile that it came from.
//
// Roles: warps 0-3 (and 4-7 up to head size 128) softmax, one row per thread;
// then 4 prep warps, a copy warp each for keys and values, a warp for each
// product's MMAs.  The two softmax groups take alternate tiles, each with its own running max, sum and output accumulator:
// they never wait for one another within a unit and are combined at its end.
// The running max is lazy: it moves only when a score passes it by 2^8 (log2
// units), and only then is the accumulator in tensor memory rescaled.
//
// What bounds it: at up to 128 rows a kv head and 16-bit caches the page reads
// from HBM, 0.68-0.74 us per tile and SM at head size 128 (32 KiB; the copy
// bandwidth's own is 0.73), of which the MMAs take 770 cycles and each of two
// softmax groups 1500 every other tile.  8-bit caches: the widening, 1.2 us a
// tile.  Start, end and join of a call take 25-35 us.
//
// Every wait is bounded, as in attention_fp8_tc.cuh: one that runs out raises a
// CTA-wide abort flag, every role winds down, waiting (bounded) for its own
// copies and MMAs, tensor memory is freed and the error flag is set.
#pragma once

#include <type_traits>

#include "attention_fp8_tc.cuh"
#include "tc_ptx.cuh"
#include "tree.cuh"

namespace pkv {

// L2 policy without preference, for pages that other CTAs read as well.
__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// Registers per thread of a group of four warps, up or down.
template <int N>
__device__ __forceinline__ void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
        "l"(*reinterpret_cast<uint64_t *>(&c)));
  return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
  return *reinterpret_cast<float2 *>(&r);
}

template <typename T, typename KV, int D, int BS>
struct TreeTcCfg {
  static constexpr bool kFp8 = is_fp8<KV>::value;
  using Op = typename std::conditional<kFp8, __half, T>::type;  // operand type of the MMAs
  static constexpr int CS = int(sizeof(KV));
  static constexpr int TT = 64;
  static constexpr int NWG = D == 256 ? 1 : 2;  // softmax groups, output accumulators
  static constexpr int kPages = TT / BS;
  // Score MMAs of a tile: 8-token group h of all pages (pages of 8 and 16
  // tokens), or all groups of a page (32 tokens), N = 64, 32, 32.
  static constexpr int kScoreMmas = BS == 8 ? 1 : 2;
  static constexpr int kNK = TT / kScoreMmas;
  static constexpr int kPageRaw = D * BS * CS;  // a key or value page in the cache
  static constexpr int kPage = D * BS * 2;      // and as operand
  static constexpr int kTile = TT * D * 2;
  static constexpr int kRawTile = TT * D * CS;
  // Operand slots OS and (8-bit caches) raw slots RS, each a key or value
  // tile, keys and values in turn: as many as fit.
  static constexpr int OS = kFp8 ? (D == 64 ? 8 : (D == 128 ? 6 : 4)) : (D == 64 ? 16 : (D == 128 ? 12 : 6));
  static constexpr int RS = kFp8 ? (D == 64 ? 16 : (D == 128 ? 14 : 4)) : OS;
  // OS is even: a slot holds keys only or values only.  A value slot is refilled
  // after the product, and with it the softmax, of the tile OS / 2 before: as
  // many mask buffers are enough.
  static constexpr int MB = OS / 2;
  static_assert(OS % 2 == 0 && RS % 2 == 0, "key and value slots apart");
  static_assert(OS <= 16 && RS <= 16 && MB <= 8, "barrier arrays");
  static constexpr int kSideWarps = kFp8 ? 2 : 4;  // prep warps on the values (and on 8-bit keys)
  static constexpr int kWords = TT / 32;        // mask words of a tile
  static constexpr int kSoftWarps = 4 * NWG;
    static constexpr int kThreads = (kSoftWarps + 8) * 32;
  // Registers per thread of the softmax, prep and issuing warps where there are
  // 512 threads: 2 x 168 + 104 + 72 = 4 x 128, what the launch gives them.  A
  // softmax row holds a tile's 64 scores at a time.
  static constexpr int kSoftRegs = 168, kPrepRegs = 104, kIssueRegs = 72;
  static_assert(NWG == 1 || (2 * kSoftRegs + kPrepRegs + kIssueRegs) * 128 == kThreads * 128, "registers");
  static constexpr int kUnits = 4;              // unit descriptors in flight
  // Query scales (8-bit caches): written up to two units ahead of the score MMAs,
  // read up to NSB units behind them.
  static constexpr int kQScales = 8;

  // Tensor memory: output accumulators, queries, score buffers.
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kQCol = NWG * D;
  static constexpr int kSCol = kQCol + D / 2;
  static constexpr int NSB = D == 64 ? 4 : (D == 128 ? 3 : 2);
  static_assert(kSCol + NSB * TT <= int(kTmemCols), "TMEM columns");
  static_assert(OS >= 2 * (NSB - 1), "a key tile must find a slot while NSB - 1 values wait");

  static constexpr int kOpOff = 0;
  static constexpr int kRawOff = OS * kTile;
  static constexpr int kMaskOff = kRawOff + (kFp8 ? RS * kRawTile : 0);
  static constexpr int kBadOff = kMaskOff + MB * kTreeTcRows * kWords * 4;
  static constexpr int kStatOff = kBadOff + MB * 16;                    // [2][2][128] (m, l)
  static constexpr int kQScaleOff = kStatOff + 4 * kTreeTcRows * 8;     // [kQScales][128]
  static constexpr int kUnitOff = kQScaleOff + (kFp8 ? kQScales * kTreeTcRows * 4 : 0);  // [kUnits]
  static constexpr int kBarOff = kUnitOff + kUnits * 64;
  static constexpr int kScratchOff = kBarOff + 100 * 8;
  static constexpr int kSmem = kScratchOff + int(sizeof(TreeScratch<kThreads>));
  static_assert(kSmem <= 232448, "shared memory");
  // Column (within a score buffer) of the tile's token t, and the token of a column.
  static __host__ __device__ constexpr int column(int t) {
    return BS == 16 ? ((t >> 3) & 1) * 32 + (t >> 4) * 8 + (t & 7) : t;
  }
  static __host__ __device__ constexpr int token(int c) {
    return BS == 16 ? ((c >> 3) & 3) * 16 + (c >> 5) * 8 + (c & 7) : c;
  }
};

// Unit descriptor of the ring (64 bytes at most).
struct TreeTcUnit {
  int32_t end, q0, T, L, ctx, kvh, row0, rows, tile0, tile1, tiles, first, seq, shared;
};
static_assert(sizeof(TreeTcUnit) <= 64, "unit descriptor");

namespace tc {

// Shared-memory descriptor of a K-major operand under the 32-byte (mode 6) or
// 64-byte (mode 4) swizzle: `sbo` bytes between groups of 8 rows.
__device__ __forceinline__ uint64_t smem_desc_swizzled(uint32_t saddr, uint32_t sbo, uint32_t mode) {
  return smem_desc(saddr, 16, sbo) | (uint64_t(mode) << 61);
}

// kind::f16, fp32 accumulator, both operands K-major; bf16 or f16.
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, int n, int m) {
  return idesc_f8f6f4(bf16 ? 1u : 0u, bf16 ? 1u : 0u, false, n, m);
}

// True in one lane of a whole warp.  MMAs and commits are issued under this and
// not under a test of the lane number: the compiler then knows that one
// thread runs, and its operands go to uniform registers directly (24 MMAs in
// 770 cycles; under `lane == 0` the same ones took 1320).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r));
  return r != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]^T (A: row = lane, two 16-bit elements of K per
// column), issued by one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

__device__ __forceinline__ void ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void st_x16u(uint32_t taddr, const uint32_t (&r)[16]) {
  float f[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(r[e]);
  st_x16(taddr, f);
}
__device__ __forceinline__ void ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

}  // namespace tc

// Bounded wait that gives up with the CTA's other roles (see tc_wait), in few
// instructions: it stands in two dozen places of a kernel whose loops just
// about fit the instruction cache.
__device__ __forceinline__ bool tree_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns,
                                          volatile int *abort) {
  uint64_t t0 = 0;
  while (!mbar_try_wait(bar, parity)) {
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > limit_ns) *abort = 1;
    if (*abort) return false;
  }
  return true;
}

// BIASED: scores are capped or biased (or their scale is not positive).  A kernel
// of its own: the loops of all roles just about fit the instruction cache, and
// code that a call does not need costs it speed.
template <typename T, typename KV, int D, int BS, bool BIASED>
__global__ void __launch_bounds__(TreeTcCfg<T, KV, D, BS>::kThreads, 1)
    tree_tc_kernel(const TreeParams p) {
  using Cfg = TreeTcCfg<T, KV, D, BS>;
  using Op = typename Cfg::Op;
  constexpr int TT = Cfg::TT, NWG = Cfg::NWG, OS = Cfg::OS, RS = Cfg::RS, MB = Cfg::MB,
                NSB = Cfg::NSB;
  constexpr int kPages = Cfg::kPages, kPage = Cfg::kPage, kPageRaw = Cfg::kPageRaw;
  constexpr int kTile = Cfg::kTile, kWords = Cfg::kWords, CS = Cfg::CS, RT = kTreeTcRows;
  constexpr bool kFp8 = Cfg::kFp8, kBf16 = std::is_same<Op, __nv_bfloat16>::value;
  constexpr int kPrep0 = Cfg::kSoftWarps, kKeyCopyWarp = kPrep0 + 4, kValueCopyWarp = kPrep0 + 5,
                kScoreWarp = kPrep0 + 6, kValueWarp = kPrep0 + 7;
  constexpr unsigned FULL = 0xffffffffu;
  // f16 probabilities are kept 2^7 larger (at most 2^15 with the lazy max), so
  // that small ones stay clear of f16's subnormals.
  constexpr float kLift = kBf16 ? 0.f : 7.f;
  constexpr float kLag = 8.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  extern __shared__ __align__(1024) uint8_t tree_tc_smem[];
  uint8_t *smem = tree_tc_smem;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kBarOff);
  uint64_t *raw_full = bars + 0;     // [RS <= 16] pages landed (tx bytes)
  uint64_t *raw_free = bars + 16;    // [RS] 8-bit caches: widened (2 prep warps)
  uint64_t *op_free = bars + 32;     // [OS <= 16] MMAs on the slot done (commit)
  // Operands ready, by tile modulo 8 and not by slot (16-bit keys need no prep,
  // and with an odd number of slots a slot holds keys and values in turn).
  uint64_t *k_ready = bars + 48;     // [8] 8-bit caches: keys widened (2 prep warps)
  uint64_t *v_ready = bars + 56;     // [8] values in operand layout (2 or 4 prep warps)
  uint64_t *s_full = bars + 64;      // [NSB <= 4] scores in TMEM (commit)
  uint64_t *p_full = bars + 68;      // [NSB] probabilities written (4 warps)
  uint64_t *pv_done = bars + 72;     // [NSB] value product done (commit)
  uint64_t *unit_full = bars + 76;   // [kUnits] descriptor written
  uint64_t *unit_free = bars + 80;   // [kUnits] descriptor read (all other warps)
  uint64_t *q_ready = bars + 84;     // queries in TMEM (4 prep warps)
  uint64_t *q_free = bars + 85;      // last score MMA of the unit done (commit)
  uint64_t *o_free = bars + 86;      // accumulators read (softmax warps)
  uint64_t *stat_full = bars + 87;   // group sums exchanged (softmax warps)
  uint64_t *prep_bar = bars + 88;    // the value prep warps among themselves
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 90);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 91);
  uint32_t *masks = reinterpret_cast<uint32_t *>(smem + Cfg::kMaskOff);  // [MB][128][kWords]
  uint32_t *bad = reinterpret_cast<uint32_t *>(smem + Cfg::kBadOff);     // [MB][4]
  float2 *stats = reinterpret_cast<float2 *>(smem + Cfg::kStatOff);      // [2][2][128]
  float *qscale = reinterpret_cast<float *>(smem + Cfg::kQScaleOff);     // [kQScales][128]
  auto &scratch = *reinterpret_cast<TreeScratch<Cfg::kThreads> *>(smem + Cfg::kScratchOff);
  auto unit_at = [&](int u) {
    return reinterpret_cast<TreeTcUnit *>(smem + Cfg::kUnitOff + (u % Cfg::kUnits) * 64);
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < RS; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_free[i], Cfg::kSideWarps);
    }
    for (int i = 0; i < OS; ++i) mbar_init(&op_free[i], 1);
    for (int i = 0; i < 8; ++i) {
      mbar_init(&k_ready[i], Cfg::kSideWarps);
      mbar_init(&v_ready[i], Cfg::kSideWarps);
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_ready, 4);
    mbar_init(q_free, 1);
    mbar_init(prep_bar, Cfg::kSideWarps);
    mbar_init(o_free, Cfg::kSoftWarps);
    mbar_init(stat_full, Cfg::kSoftWarps);
    for (int i = 0; i < Cfg::kUnits; ++i) {
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_free[i], Cfg::kSoftWarps + 7);
    }
    *abort_flag = 0;
    for (int i = 0; i < MB * 4; ++i) bad[i] = 0;
    fence_barrier_init();
  }
  if (warp == kScoreWarp) tc::tmem_alloc(tmem_slot, Cfg::kTmemCols);
  grid_dependency_wait();
  allow_dependent_launch();
  const TreeRun run = tree_find_run<TT, RT, kTreeTcUnitCost, Cfg::kThreads>(p, scratch);
  if (run.begin >= run.end && threadIdx.x == 0) tree_write_cut<kTreeTcUnitCost>(p, run, nullptr);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint64_t wait_ns = p.wait_limit_ns;
  const uint64_t drain_ns = min(wait_ns, uint64_t(100000000ull));
  bool failed = false;

  auto wait_one = [&](uint64_t *bar, uint32_t parity) { return tree_wait(bar, parity, wait_ns, abort_flag); };
  auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
    return bool(__all_sync(FULL, tree_wait(bar, parity, wait_ns, abort_flag)));
  };
  // A consumer warp's copy of unit u's descriptor.
  auto take_unit = [&](int u, TreeTcUnit &d) {
    const int r = u % Cfg::kUnits;
    if (!wait_warp(&unit_full[r], uint32_t(u / Cfg::kUnits) & 1u)) return false;
    d = *unit_at(u);
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&unit_free[r]);
    return true;
  };

  if (run.begin >= run.end) {
    // nothing to do: straight to the teardown
  } else if (warp < kPrep0) {
    if constexpr (NWG == 2) reg_alloc<Cfg::kSoftRegs>();
    // ----------------------------------------------------------- softmax --
    const int wg = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const TreeLogit logit(p);
    uint32_t g = 0;
    for (int u = 0; !failed; ++u) {
      TreeTcUnit d;
      if (!take_unit(u, d)) {
        failed = true;
        break;
      }
      if (d.end) break;
      const bool live = (warp & 3) * 32 < d.rows;  // a row of this warp is a query row
      const int R = d.row0 + min(r, d.rows - 1);
      const int node = R / p.group, head = d.kvh * p.group + R % p.group;
      const int node_at = node - d.row0 / p.group;
      float rowscale = 1.f, slope = 0.f;
      int qpos = 0;
      if (BIASED && p.alibi) {
        slope = p.alibi[head] * kLog2e;
        qpos = p.positions ? p.positions[d.q0 + node] : d.ctx + node;
      }
      float m = -INFINITY, l = 0.f;  // m: the reference that the accumulator is scaled to
      bool have = false;             // this group's accumulator holds something
      uint32_t mine = 0;             // its last tile
      for (int tile = d.tile0; tile < d.tile1; ++tile, ++g) {
        if (NWG == 2 && int(g & 1) != wg) continue;
        const uint32_t b = g % NSB, mb = g % MB;
        const uint32_t s = tmem + lanes + uint32_t(Cfg::kSCol + b * TT);
        if (!wait_warp(&s_full[b], (g / NSB) & 1u)) {
          failed = true;
          break;
        }
        tc::fence_after_sync();
        const int t0 = tile * TT;
        const bool tail = t0 + TT > d.ctx;
        uint32_t hurt[kWords], hurt_seen[kWords];  // tokens of the tile whose values are not finite
#pragma unroll
        for (int w = 0; w < kWords; ++w) hurt[w] = hurt_seen[w] = 0;
        bool any_hurt = false;
        if (tail) {
          // the prep warps' mask words and marks come with the value tile
          if (!wait_warp(&v_ready[g & 7], (g >> 3) & 1u)) {
            failed = true;
            break;
          }
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            hurt[w] = bad[mb * 4 + w];
            any_hurt |= hurt[w] != 0;
          }
        }
        if (live) {
          if (kFp8) rowscale = qscale[(u % Cfg::kQScales) * RT + min(r, d.rows - 1)];
          float mul = logit.scale_log2 * rowscale, top = -INFINITY;
          if (tail) {
            // Masked: the scores are replaced by their final values in log2 units
            // first.  (A small loop: it runs once or twice a unit, mostly from a
            // cold instruction cache.)
#pragma unroll 1
            for (int k = 0; k < TT / 8; ++k) {
              uint32_t z[8];
              tc::ld_x8(s + uint32_t(8 * k), z);
              tc::wait_ld();
              const int t8 = Cfg::token(8 * k);  // 8 tokens from here on
              const uint32_t bits = masks[(mb * RT + node_at) * kWords + (t8 >> 5)] >> (t8 & 31);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float y = __uint_as_float(z[e]) * rowscale;
                float x = BIASED && p.cap > 0.f ? logit.capped(y) : logit.plain(y);
                if (BIASED && p.alibi) {
                  const int t = t0 + t8 + e;
                  int kpos = t;
                  if (p.positions && t >= d.ctx && t < d.L) kpos = p.positions[d.q0 + t - d.ctx];
                  x = fmaf(slope, float(kpos - qpos), x);
                }
                z[e] = __float_as_uint((bits >> e) & 1u ? x : -INFINITY);
              }
              tc::st_x8(s + uint32_t(8 * k), z);
            }
            tc::wait_st();
            mul = 1.f;
          } else if constexpr (BIASED) {
            // Every row sees the tile, but its scores are capped or biased: the
            // same, half a tile at a time.  (Through tensor memory as well: beside
            // the 64 registers of the common path below there is no room for it.)
            const float b0 = slope * float(t0 - qpos);
#pragma unroll 1
            for (int h = 0; h < TT; h += 32) {
              uint32_t z[32];
              tc::ld_x32(s + uint32_t(h), z);
              tc::wait_ld();
              if (p.cap > 0.f) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  z[e] = __float_as_uint(logit.capped(__uint_as_float(z[e]) * rowscale));
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) z[e] = __float_as_uint(__uint_as_float(z[e]) * mul);
              }
              if (p.alibi) {
                // the bias of column h + e's token is slope * (t0 - qpos + token)
                const float bh = fmaf(slope, float(Cfg::token(h)), b0);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  z[e] = __float_as_uint(__uint_as_float(z[e]) + fmaf(slope, float(Cfg::token(e)), bh));
              }
              tc::st_x16u(s + uint32_t(h), reinterpret_cast<const uint32_t(&)[16]>(z[0]));
              tc::st_x16u(s + uint32_t(h + 16), reinterpret_cast<const uint32_t(&)[16]>(z[16]));
            }
            tc::wait_st();
            mul = 1.f;
          }
          // the row's scores of the tile, all at once
          uint32_t v[TT];
          {
            uint32_t v0[32], v1[32];
            tc::ld_x32(s, v0);
            tc::ld_x32(s + 32u, v1);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = v0[e], v[32 + e] = v1[e];
          }
          {
            float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < TT; ++e) t4[e & 3] = fmaxf(t4[e & 3], __uint_as_float(v[e]));
            top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * mul;
          }
          // the reference moves when a score passes it by 2^kLag
          const bool grow = top > m + kLag;  // (m = -inf: any score)
          if (__any_sync(FULL, grow)) {
            const float to = grow ? top : m;
            const float alpha = to == m ? 1.f : ex2(m - to);
            if (have) {
              // (the group's last tile)
              if (!wait_warp(&pv_done[mine % NSB], (mine / NSB) & 1u)) {
                failed = true;
                break;
              }
              tc::fence_after_sync();
              const uint32_t o = tmem + lanes + uint32_t(wg * D);
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t v[32];
                tc::ld_x32(o + uint32_t(c), v);
                tc::wait_ld();
                float f[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(v[e]) * alpha;
                tc::st_x16(o + uint32_t(c), f);
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(v[16 + e]) * alpha;
                tc::st_x16(o + uint32_t(c + 16), f);
              }
              tc::wait_st();
            }
            l *= alpha;
            m = to;
          }
          // probabilities, in token order: hi parts over the first half of the
          // scores' columns, lo parts over the second
          const float ref = m == -INFINITY ? 0.f : m - kLift;
          const float2 mul2 = make_float2(mul, mul), ref2 = make_float2(-ref, -ref);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t hi[TT / 4], lo[TT / 4];
#pragma unroll
            for (int w = 0; w < TT / 4; ++w) {
              const int c = Cfg::column(h * (TT / 2) + 2 * w);
              const float2 x = fma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), mul2, ref2);
              const float2 e = make_float2(ex2(x.x), ex2(x.y));
              sum[w & 1] = add2(sum[w & 1], e);
              hi[w] = pack2<Op>(e.x, e.y);
              const float2 f = unpack2<Op>(hi[w]);
              const float2 d2 = add2(e, make_float2(-f.x, -f.y));
              lo[w] = pack2<Op>(d2.x, d2.y);
            }
            tc::st_x16u(s + uint32_t(h * TT / 4), hi);
            tc::st_x16u(s + uint32_t(TT / 2 + h * TT / 4), lo);
          }
          tc::wait_st();
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
        if (any_hurt) {  // those that this row sees (the mask buffer is not ours after p_full)
#pragma unroll
          for (int w = 0; w < kWords; ++w)
            hurt_seen[w] = hurt[w] & masks[(mb * RT + node_at) * kWords + w];
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[b]);
        have = true;
        mine = g;
        if (any_hurt) {
          // Rows that see a token with values that are not finite add those after
          // the tile's product, which saw zeros there.  (Times any probability
          // above 0 they stay what they are.)
          if (!wait_warp(&pv_done[b], (g / NSB) & 1u)) {
            failed = true;
            break;
          }
          tc::fence_after_sync();
          if (live) {
            const int64_t row = tree_table_row(p, d.seq);
            const uint32_t o = tmem + lanes + uint32_t(wg * D);
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
#pragma unroll 1
              for (uint32_t left = hurt[w]; left != 0; left &= left - 1) {
                const int bit = __ffs(int(left)) - 1;
                const bool sees = (hurt_seen[w] >> bit) & 1u;
                const int tok = t0 + 32 * w + bit;
                const int64_t blk = tree_block_id(p, row, tok / BS);
                const KV *v = static_cast<const KV *>(p.v) + blk * p.v_s0 + int64_t(d.kvh) * p.v_s1 +
                              tok % BS;
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  float f[16];
                  tc::ld_x16(o + uint32_t(c), f);
                  tc::wait_ld();
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    float x;
                    if constexpr (kFp8) {
                      uint32_t w0, w1;
                      fp8x4_to_f16x2<KV>(v[(c + e) * BS].bits, w0, w1);
                      x = unpack2<__half>(w0).x;
                    } else {
                      x = to_f32<KV>(v[(c + e) * BS]);
                    }
                    if (sees && !(fabsf(x) < INFINITY)) f[e] += x;
                  }
                  tc::st_x16(o + uint32_t(c), f);
                  tc::wait_st();
                }
              }
            }
          }
          tc::fence_before_sync();
        }
      }
      if (failed) break;
      // ----- the unit's end: both groups' sums, then half of the columns each
      if (have && !wait_warp(&pv_done[mine % NSB], (mine / NSB) & 1u)) {
        failed = true;
        break;
      }
      const float mine_m = m == -INFINITY ? m : m - kLift;
      float w0 = 1.f, w1 = 0.f, M = mine_m, ls = l;
      if constexpr (NWG == 2) {
        // (two sets by unit parity: a group may be a unit ahead of the other)
        float2 *st2 = stats + (u & 1) * 2 * RT;
        st2[wg * RT + r] = make_float2(mine_m, l);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(stat_full);
        if (!wait_warp(stat_full, uint32_t(u) & 1u)) {
          failed = true;
          break;
        }
        const float2 a = st2[r], c = st2[RT + r];
        M = fmaxf(a.x, c.x);
        // (a group that saw nothing: m = -inf, l = 0, its accumulator unused)
        w0 = a.x == -INFINITY ? 0.f : ex2(a.x - M);
        w1 = c.x == -INFINITY ? 0.f : ex2(c.x - M);
        ls = (a.x == -INFINITY ? a.y : w0 * a.y) + (c.x == -INFINITY ? c.y : w1 * c.y);
      } else {
        if (mine_m == -INFINITY) w0 = 0.f;
      }
      tc::fence_after_sync();
      const bool whole = d.tile0 == 0 && d.tile1 == d.tiles;
      const float inv = ls == 0.f ? 0.f : __fdiv_rn(p.out_scale, ls);
      constexpr int kCols = D / NWG;
      T *orow = static_cast<T *>(p.out) + int64_t(d.q0 + node) * p.o_s0 + int64_t(head) * p.o_s1;
      const bool vec = p.o_s2 == 1 && (reinterpret_cast<uintptr_t>(orow) & 15u) == 0;
      const int64_t part = (2 * int64_t(blockIdx.x) + (d.first ? 0 : 1)) * RT + r;
      if (live) {
        if (!whole && wg == 0 && r < d.rows) p.ml[part] = make_float2(M, ls);
#pragma unroll 1
        for (int c = wg * kCols; c < (wg + 1) * kCols; c += 16) {
          float f[16], e1[16];
          tc::ld_x16(tmem + lanes + uint32_t(c), f);
          if constexpr (NWG == 2) tc::ld_x16(tmem + lanes + uint32_t(D + c), e1);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            // (an unused accumulator holds anything: leave it out, not times 0)
            float x = w0 == 0.f ? 0.f : f[e] * w0;
            if constexpr (NWG == 2) x = w1 == 0.f ? x : fmaf(e1[e], w1, x);
            f[e] = x;
          }
          if (r < d.rows) {
            if (whole) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = pack2<T>(f[2 * e] * inv, f[2 * e + 1] * inv);
              if (vec) {
                *reinterpret_cast<uint4 *>(orow + c) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(orow + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  orow[int64_t(c + e) * p.o_s2] = from_f32<T>(f[e] * inv);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                p.acc[((part - r) / RT * (D / 4) + (c + e) / 4) * RT + r] =
                    make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(o_free);
    }
  } else if (warp < kPrep0 + 4) {
    if constexpr (NWG == 2) reg_dealloc<Cfg::kPrepRegs>();
    // -------------------------------------------------------------- prep --
    const int pt = threadIdx.x - kPrep0 * 32, pw = warp - kPrep0;
    // 8-bit caches: two warps widen the keys, two the values (all four on one after
    // the other: 111 us instead of 99 on two sequences of 32k tokens).
    const int side = kFp8 ? pw >> 1 : 1;
    constexpr int kSide = Cfg::kSideWarps, kSideThreads = 32 * kSide;
    const int st = pt % kSideThreads, sw0 = pw % kSide;
    uint32_t g = 0;  // tiles
    uint32_t syncs = 0;
    for (int u = 0; !failed; ++u) {
      TreeTcUnit d;
      if (!take_unit(u, d)) {
        failed = true;
        break;
      }
      if (d.end) break;
      // Queries: row pt of the row tile to lane pt of tensor memory, fetched
      // while the last unit's score MMAs may still read theirs.
      const bool any_row = pw * 32 < d.rows;
      const int R = d.row0 + min(pt, d.rows - 1);
      const T *q = static_cast<const T *>(p.q) + int64_t(d.q0 + R / p.group) * p.q_s0 +
                   int64_t(d.kvh * p.group + R % p.group) * p.q_s1;
      const bool vec = p.q_s2 == 1 && (reinterpret_cast<uintptr_t>(q) & 15u) == 0;
      constexpr int kPart = D < 128 ? D : 128;  // dims held in registers
      uint32_t qw[kPart / 2];
      auto fetch = [&](int d0) {
        if (vec) {
#pragma unroll
          for (int c = 0; c < kPart / 8; ++c) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(q + d0) + c);
            qw[4 * c] = x.x, qw[4 * c + 1] = x.y, qw[4 * c + 2] = x.z, qw[4 * c + 3] = x.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < kPart / 2; ++e)
            qw[e] = pack2<T>(to_f32<T>(q[int64_t(d0 + 2 * e) * p.q_s2]),
                             to_f32<T>(q[int64_t(d0 + 2 * e + 1) * p.q_s2]));
        }
      };
      float up = 1.f;
      if (any_row) {
        if constexpr (!std::is_same<Op, T>::value) {
          // bf16 into f16: max |q| of the row brought into [2^14, 2^15), exactly
          float amax = 0.f;
#pragma unroll 1
          for (int d0 = D - kPart; d0 >= 0; d0 -= kPart) {
            fetch(d0);
#pragma unroll
            for (int e = 0; e < kPart / 2; ++e) {
              const float2 f = unpack2<T>(qw[e]);
              amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
          int k = 0;
          if (amax > 0.f && amax < INFINITY) k = clamp_int(141 - int(__float_as_uint(amax) >> 23), -100, 100);
          up = __uint_as_float(uint32_t(127 + k) << 23);
          qscale[(u % Cfg::kQScales) * RT + pt] = __uint_as_float(uint32_t(127 - k) << 23);
        } else {
          if (kFp8) qscale[(u % Cfg::kQScales) * RT + pt] = 1.f;
          fetch(0);
        }
      }
      if (u >= 1 && !wait_warp(q_free, uint32_t(u - 1) & 1u)) {
        failed = true;
        break;
      }
      if (any_row) {
        tc::fence_after_sync();
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += kPart) {
          if (d0 > 0) fetch(d0);
#pragma unroll
          for (int c = 0; c < kPart / 2; c += 16) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              w[e] = qw[c + e];
              if constexpr (!std::is_same<Op, T>::value) {
                const float2 f = unpack2<T>(w[e]);
                w[e] = pack2<__half>(f.x * up, f.y * up);
              }
            }
            tc::st_x16u(tmem + (uint32_t(32 * pw) << 16) + uint32_t(Cfg::kQCol + d0 / 2 + c), w);
          }
        }
        tc::wait_st();
        tc::fence_before_sync();
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(q_ready);
      const int node0 = d.row0 / p.group;
      const int nodes = (d.row0 + d.rows - 1) / p.group - node0 + 1;
      for (int tile = d.tile0; tile < d.tile1 && !failed; ++tile, ++g) {
        const int t0 = tile * TT;
        const int nt = min(TT, d.L - t0);  // tokens of the tile (<= 0: none)
        const bool tail = t0 + TT > d.ctx;
        const uint32_t mb = g % MB;
        {
          const int kv = side;
          const uint32_t n = 2 * g + kv, rs = n % RS, os = n % OS;
          if (!wait_warp(&raw_full[rs], (n / RS) & 1u) ||
              (kFp8 && n >= uint32_t(OS) && !wait_warp(&op_free[os], (n / OS - 1) & 1u))) {
            failed = true;
            break;
          }
          uint8_t *op = smem + os * kTile;
          if constexpr (kFp8) {
            const uint8_t *raw = smem + Cfg::kRawOff + rs * Cfg::kRawTile;
#pragma unroll 4
            for (int i = st; i < TT * D / 16; i += kSideThreads) {
              const uint4 w = *reinterpret_cast<const uint4 *>(raw + i * 16);
              uint32_t h[8];
              fp8x4_to_f16x2<KV>(w.x, h[0], h[1]);
              fp8x4_to_f16x2<KV>(w.y, h[2], h[3]);
              fp8x4_to_f16x2<KV>(w.z, h[4], h[5]);
              fp8x4_to_f16x2<KV>(w.w, h[6], h[7]);
              const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), b = make_uint4(h[4], h[5], h[6], h[7]);
              const int pg = i / (D * BS / 16), r = i % (D * BS / 16);
              uint8_t *page = op + pg * kPage;
              if (kv == 0) {  // chunk of 16 dims of a token -> two of 8
                const int c = r / BS, t = r % BS;
                *reinterpret_cast<uint4 *>(page + (2 * c * BS + t) * 16) = a;
                *reinterpret_cast<uint4 *>(page + ((2 * c + 1) * BS + t) * 16) = b;
              } else if (BS == 8) {  // two dims of 8 tokens
                *reinterpret_cast<uint4 *>(page + r * 32) = a;
                *reinterpret_cast<uint4 *>(page + r * 32 + 16) = b;
              } else if (BS == 16) {  // a dim's 16 tokens, 32-byte swizzle
                const int x = (r >> 2) & 1;
                *reinterpret_cast<uint4 *>(page + r * 32 + x * 16) = a;
                *reinterpret_cast<uint4 *>(page + r * 32 + (x ^ 1) * 16) = b;
              } else {  // half of a dim's 32 tokens, 64-byte swizzle
                const int dim = r >> 1, c = (r & 1) * 2, x = (dim >> 1) & 3;
                *reinterpret_cast<uint4 *>(page + dim * 64 + (c ^ x) * 16) = a;
                *reinterpret_cast<uint4 *>(page + dim * 64 + ((c + 1) ^ x) * 16) = b;
              }
            }
          } else if constexpr (BS == 16) {
            // rows 4-7 of every 8: exchange the two 16-byte halves
#pragma unroll 4
            for (int i = pt; i < kPages * D / 2; i += 128) {
              uint4 *r = reinterpret_cast<uint4 *>(op + (((i >> 2) << 3) + 4 + (i & 3)) * 32);
              const uint4 a = r[0], b = r[1];
              r[0] = b;
              r[1] = a;
            }
          } else if constexpr (BS == 32) {
            // piece c of row r to place c ^ ((r >> 1) & 3)
#pragma unroll 2
            for (int i = pt; i < kPages * D; i += 128) {
              uint4 *r = reinterpret_cast<uint4 *>(op + i * 64);
              const int x = (i >> 1) & 3;
              const uint4 a = r[0], b = r[1], c = r[2], e = r[3];
              r[x] = a;
              r[1 ^ x] = b;
              r[2 ^ x] = c;
              r[3 ^ x] = e;
            }
          }
          if (kv == 1 && tail) {
            // The warps' accesses to the same rows are apart from here on.
            if (st < 4) bad[mb * 4 + st] = 0;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(prep_bar);
            if (!wait_warp(prep_bar, syncs++ & 1u)) {
              failed = true;
              break;
            }
            // What each row sees of the tile, a bit per token.
            for (int i = sw0; i < nodes; i += kSide) {
              const int node = node0 + i;
#pragma unroll
              for (int w = 0; w < kWords; ++w) {
                const int t = t0 + 32 * w + lane;
                bool seen = t < d.ctx;
                if (!seen && t < d.L) {
                  const int j = t - d.ctx;
                  seen = p.mask ? j < p.mask_cols &&
                                      p.mask[int64_t(d.q0 + node) * p.m_s0 + int64_t(j) * p.m_s1] != 0
                                : j <= node;
                }
                const uint32_t bits = __ballot_sync(FULL, seen);
                if (lane == 0) masks[(mb * RT + i) * kWords + w] = bits;
              }
            }
            // Values past the end become zeros.  So do drafted tokens' values
            // that are not finite (rows that do not see the token must not: 0 *
            // NaN); such tokens are marked, and the rows that see one add its
            // values themselves.
            const int t8 = max(0, d.ctx - t0) / 8;  // 16-byte pieces: 8 tokens of a dim
            for (int i = st; i < (TT / 8 - t8) * D; i += kSideThreads) {
              const int t = (t8 + i / D) * 8, dim = i % D;
              const int sw = BS == 16 ? (dim >> 2) & 1 : (BS == 32 ? (dim >> 1) & 3 : 0);
              uint4 *e = reinterpret_cast<uint4 *>(op + t / BS * kPage + dim * BS * 2 +
                                                   ((t % BS / 8) ^ sw) * 16);
              if (t >= nt) {
                *e = make_uint4(0u, 0u, 0u, 0u);
                continue;
              }
              const uint4 x = *e;
              uint32_t w[4] = {x.x, x.y, x.z, x.w}, marks = 0;
              bool change = false;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                constexpr uint32_t kExp = kBf16 ? 0x7f80u : 0x7c00u;
                const int sh = (k & 1) * 16;
                const bool past = t + k >= nt;
                const bool odd = ((w[k >> 1] >> sh) & kExp) == kExp;
                if (past || odd) {
                  w[k >> 1] &= ~(0xffffu << sh);
                  change = true;
                  if (!past) marks |= 1u << k;
                }
              }
              if (change) *e = make_uint4(w[0], w[1], w[2], w[3]);
              if (marks) atomicOr(&bad[mb * 4 + t / 32], marks << (t & 31));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(kv == 0 ? &k_ready[g & 7] : &v_ready[g & 7]);
            if (kFp8) tc::mbar_arrive(&raw_free[rs]);
          }
        }
      }
    }
  } else {
    if constexpr (NWG == 2) reg_dealloc<Cfg::kIssueRegs>();
    if (warp == kKeyCopyWarp || warp == kValueCopyWarp) {
    // ------------------------------------------------------------ copies --
    // The key copy warp also steps through the run and hands out the units.
    // (One warp for both copies took about 950 cycles for each of them, more than
    // a tile's share of the HBM rate.)
    // pages that another row tile reads too stay in L2
    const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_normal();
    const uint32_t kv = warp == kKeyCopyWarp ? 0 : 1;
    const uint8_t *cache = static_cast<const uint8_t *>(kv == 0 ? p.k : p.v);
    const int64_t block_bytes = (kv == 0 ? p.k_s0 : p.v_s0) * CS;
    const int64_t head_bytes = (kv == 0 ? p.k_s1 : p.v_s1) * CS;
    TreeWalk<TT, RT, kTreeTcUnitCost> walk;
    if (kv == 0) walk.start(p, run);
    uint32_t t = 0;  // tiles issued
    int ids0 = 0, ids0_seq = -1;
    for (int u = 0; !failed; ++u) {
      TreeTcUnit d;
      if (kv == 0) {
        TreeStretch st;
        d.end = !walk.next(p, st);
        if (!d.end) {
          d.q0 = st.q.q0, d.T = st.q.T, d.L = st.q.L, d.ctx = st.q.ctx;
          d.kvh = st.kvh, d.row0 = st.row0, d.rows = st.rows;
          d.tile0 = st.tile0, d.tile1 = st.tile1, d.tiles = st.tiles;
          d.first = u == 0, d.seq = st.seq, d.shared = st.q.row_tiles > 1;
        }
        if (u == 0 && lane == 0) tree_write_cut<kTreeTcUnitCost>(p, run, d.end ? nullptr : &st);
        if (u >= Cfg::kUnits &&
            !wait_warp(&unit_free[u % Cfg::kUnits], uint32_t(u / Cfg::kUnits - 1) & 1u)) {
          failed = true;
          break;
        }
        if (lane == 0) {
          *unit_at(u) = d;
          tc::mbar_arrive(&unit_full[u % Cfg::kUnits]);
        }
        __syncwarp();
      } else if (!take_unit(u, d)) {
        failed = true;
        break;
      }
      if (d.end) break;
      const int64_t row = tree_table_row(p, d.seq);
      const int npages = (d.L + BS - 1) / BS;
      const uint8_t *base = cache + int64_t(d.kvh) * head_bytes;
      const uint64_t policy = d.shared ? again : once;
      const int page0 = d.tile0 * kPages;
      auto load_ids = [&](int page) {  // this lane's of 32 pages from `page` on
        return page + lane < npages ? tree_block_id(p, row, page + lane) : 0;
      };
      int ids;
      if (page0 == 0 && ids0_seq == d.seq) {
        ids = ids0;  // another kv head or row tile of the same sequence
      } else {
        ids = load_ids(page0);
        if (page0 == 0) {
          ids0 = ids;
          ids0_seq = d.seq;
        }
      }
      int next_ids = load_ids(page0 + 32);
      for (int tile = d.tile0; tile < d.tile1; ++tile, ++t) {
        const int pg = tile * kPages, rel = pg - page0;
        if (rel > 0 && (rel & 31) == 0) {
          ids = next_ids;
          next_ids = load_ids(pg + 32);
        }
        const int id = __shfl_sync(FULL, ids, ((rel & 31) + lane) & 31);
        const int np = max(0, min(kPages, npages - pg));
        const uint32_t n = 2 * t + kv, s = n % RS;
        if (n >= uint32_t(RS) &&
            !wait_warp(kFp8 ? &raw_free[s] : &op_free[s], (n / RS - 1) & 1u)) {
          failed = true;
          break;
        }
        if (lane == 0)
          mbar_arrive_expect_tx(&raw_full[s],
                                uint32_t(np * kPageRaw) + (kv == 0 ? p.extra_expect_tx : 0u));
        __syncwarp();
        if (lane < np)
          bulk_copy_g2s(smem + (kFp8 ? Cfg::kRawOff : 0) + s * Cfg::kRawTile + lane * kPageRaw,
                        base + int64_t(id) * block_bytes, uint32_t(kPageRaw), &raw_full[s], policy);
      }
    }
    // No copy may be in flight when the CTA exits.
    for (uint32_t i = t > uint32_t(RS / 2) ? t - RS / 2 : 0; i < t; ++i) {
      const uint32_t n = 2 * i + kv;
      mbar_wait_bounded(&raw_full[n % RS], (n / RS) & 1u, drain_ns);
    }
    __syncwarp();
    } else if (warp == kScoreWarp) {
    // -------------------------------------------------------- score MMAs --
    // (One elected thread waits and issues, here and in the next role: with
    // both products in one thread its waits and issues, about 1600 cycles a tile,
    // were what the kernel took; the MMAs themselves take half of that.)
    constexpr uint32_t idesc = tc::idesc_f16(kBf16, Cfg::kNK, RT);
    bool ok = true;
    if (tc::elect_one()) {
      uint32_t g = 0;  // tiles
      uint64_t *last = nullptr;
      uint32_t last_parity = 0;
      for (int u = 0; ok; ++u) {
        const int r = u % Cfg::kUnits;
        ok = wait_one(&unit_full[r], uint32_t(u / Cfg::kUnits) & 1u);
        if (!ok) break;
        const int end = unit_at(u)->end, nt = unit_at(u)->tile1 - unit_at(u)->tile0;
        tc::mbar_arrive(&unit_free[r]);
        if (end) break;
        ok = wait_one(q_ready, uint32_t(u) & 1u);
        for (int i = 0; ok && i < nt; ++i, ++g) {
          const uint32_t b = g % NSB, n = 2 * g, os = n % OS;
          ok = kFp8 ? wait_one(&k_ready[g & 7], (g >> 3) & 1u) : wait_one(&raw_full[os], (n / OS) & 1u);
          // the score buffer holds the probabilities of tile g - NSB until its product is done
          if (ok && g >= uint32_t(NSB)) ok = wait_one(&pv_done[b], (g / NSB - 1) & 1u);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t k0 = smem_addr(smem) + os * kTile;
#pragma unroll
          for (int h = 0; h < Cfg::kScoreMmas; ++h) {
            const uint32_t s = tmem + uint32_t(Cfg::kSCol + h * Cfg::kNK) + b * TT;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t at = k0 + uint32_t(ks * 2 * BS * 16);
              tc::mma_f16_ts(s, tmem + uint32_t(Cfg::kQCol + ks * 8),
                             BS == 32 ? tc::smem_desc(at + h * kPage, BS * 16, 128)
                                      : tc::smem_desc(at + h * 128, BS * 16, kPage),
                             idesc, ks > 0);
            }
          }
          if (i == nt - 1) tc::commit(q_free);
          tc::commit(&op_free[os]);
          tc::commit(&s_full[b]);
          last = &s_full[b];
          last_parity = (g / NSB) & 1u;
        }
      }
      // Every MMA issued must have finished before TMEM is freed.
      if (last != nullptr && !mbar_wait_bounded(last, last_parity, drain_ns)) ok = false;
    }
    failed = __any_sync(FULL, !ok) != 0;
    __syncwarp();
    } else if (warp == kValueWarp) {
    // -------------------------------------------------------- value MMAs --
    constexpr uint32_t idesc = tc::idesc_f16(kBf16, D, RT);
    bool ok = true;
    if (tc::elect_one()) {
      uint32_t t = 0;  // tiles
      uint64_t *last = nullptr;
      uint32_t last_parity = 0;
      for (int u = 0; ok; ++u) {
        const int r = u % Cfg::kUnits;
        ok = wait_one(&unit_full[r], uint32_t(u / Cfg::kUnits) & 1u);
        if (!ok) break;
        const int end = unit_at(u)->end, nt = unit_at(u)->tile1 - unit_at(u)->tile0;
        tc::mbar_arrive(&unit_free[r]);
        if (end) break;
        if (u > 0) ok = wait_one(o_free, uint32_t(u - 1) & 1u);
        for (int i = 0; ok && i < nt; ++i, ++t) {
          const uint32_t b = t % NSB, n = 2 * t + 1, os = n % OS;
          const uint32_t acc = NWG == 2 ? t & 1 : 0;
          const bool fresh = i < NWG;  // the first product into its accumulator
          ok = wait_one(&v_ready[t & 7], (t >> 3) & 1u) && wait_one(&p_full[b], (t / NSB) & 1u);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t v0 = smem_addr(smem) + os * kTile;
          const uint32_t o = tmem + acc * D, s = tmem + uint32_t(Cfg::kSCol) + b * TT;
#pragma unroll
          for (int ks = 0; ks < TT / 16; ++ks) {
            uint64_t vd;
            if constexpr (BS == 8)
              vd = tc::smem_desc(v0 + 2 * ks * kPage, kPage, 128);
            else if constexpr (BS == 16)
              vd = tc::smem_desc_swizzled(v0 + ks * kPage, 256, 6);
            else
              vd = tc::smem_desc_swizzled(v0 + (ks >> 1) * kPage + (ks & 1) * 32, 512, 4);
            tc::mma_f16_ts(o, s + uint32_t(ks * 8), vd, idesc, !(fresh && ks == 0));
            tc::mma_f16_ts(o, s + uint32_t(TT / 2 + ks * 8), vd, idesc, true);
          }
          tc::commit(&pv_done[b]);
          tc::commit(&op_free[os]);
          last = &pv_done[b];
          last_parity = (t / NSB) & 1u;
        }
      }
      if (last != nullptr && !mbar_wait_bounded(last, last_parity, drain_ns)) ok = false;
    }
    failed = __any_sync(FULL, !ok) != 0;
    __syncwarp();
    }
  }

  // ------------------------------------------------------------ teardown --
  if (failed && lane == 0) flag_error(p.err, PKV_ERRF_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kScoreWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

}  // namespace pkv
