// Tree attention on the 5th-generation tensor cores: fp16 / bf16 queries over
// 16-bit or 8-bit caches (the split, the masks and the join: tree.cuh).
//
// One CTA per SM runs its stretches of (sequence, kv head, 128 query rows) x
// tiles of TT tokens (128; 64 at head size 256).  Per tile
//   S = Q K^T     M = 128 rows, N = tokens, K = head dims: both from shared memory
//   O += P V      M = 128 rows, N = head dims, K = tokens: P from tensor memory
// with S, P and O in tensor memory.  The pages are used as they lie in the
// cache, fetched by whole-page bulk copies:
// - a key page [D / 8][BS][8] holds 8 tokens x 16 bytes in 128 contiguous
//   bytes, the core matrix of an operand without swizzling: the 8-token
//   groups number h of all pages of the tile (a page apart) make one MMA, so S
//   comes out with its tokens permuted (column h * TT / (BS / 8) + 8 * page + i
//   is token BS * page + 8 h + i), which a softmax does not mind;
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
// then 4 prep warps, the copy warp, the MMA warp.  The two softmax groups take
// alternate tiles, each with its own running max, sum and output accumulator:
// they never wait for one another within a unit and are combined at its end.
// The running max is lazy: it moves only when a score passes it by 2^8 (log2
// units), and only then is the accumulator in tensor memory rescaled.
//
// What bounds it: at up to 128 rows a kv head the page reads from HBM (a tile
// is 64 KiB at head size 128, about 2800 cycles of an SM's share of the HBM
// rate; its MMAs take about 1100, its softmax about 1000 issue slots of each
// scheduler).
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

template <typename T, typename KV, int D, int BS>
struct TreeTcCfg {
  static constexpr bool kFp8 = is_fp8<KV>::value;
  using Op = typename std::conditional<kFp8, __half, T>::type;  // operand type of the MMAs
  static constexpr int CS = int(sizeof(KV));
  static constexpr int TT = D == 256 ? 64 : 128;
  static constexpr int NWG = D == 256 ? 1 : 2;  // softmax groups, output accumulators
  static constexpr int kPages = TT / BS;
  static constexpr int kSub = BS / 8;           // 8-token groups of a page
  static constexpr int kNK = TT / kSub;         // N of a score MMA
  static constexpr int kPageRaw = D * BS * CS;  // a key or value page in the cache
  static constexpr int kPage = D * BS * 2;      // and as operand
  static constexpr int kTile = TT * D * 2;
  static constexpr int kRawTile = kFp8 ? TT * D : kTile;
  static constexpr int kQBytes = kTreeTcRows * D * 2;
  static constexpr int NQ = D == 64 ? 2 : 1;    // query buffers
  // Operand slots OS and (8-bit caches) raw slots RS, each a key or value
  // tile, keys and values in turn: as many as fit beside the queries.
  static constexpr int OS = kFp8 ? (D == 64 ? 4 : 3) : (D == 64 ? 8 : (D == 128 ? 5 : 4));
  static constexpr int RS = kFp8 ? (D == 64 ? 8 : (D == 128 ? 5 : 3)) : OS;
  // Mask buffers: a value slot is refilled only after the product of the tile
  // (OS + 1) / 2 before, and with it that tile's softmax, is done.
  static constexpr int MB = (OS + 1) / 2;
  static_assert(MB <= 4, "k_ready and v_ready are reused every 4 tiles");
  static constexpr int kWords = TT / 32;        // mask words of a tile
  static constexpr int kSoftWarps = 4 * NWG;
  static constexpr int kThreads = (kSoftWarps + 6) * 32;
  static constexpr int kUnits = 4;              // unit descriptors in flight

  static constexpr int kOpOff = 0;
  static constexpr int kRawOff = OS * kTile;
  static constexpr int kQOff = kRawOff + (kFp8 ? RS * kRawTile : 0);
  static constexpr int kMaskOff = kQOff + NQ * kQBytes;
  static constexpr int kBadOff = kMaskOff + MB * kTreeTcRows * kWords * 4;
  static constexpr int kStatOff = kBadOff + MB * 16;                    // [2][2][128] (m, l)
  static constexpr int kQScaleOff = kStatOff + 4 * kTreeTcRows * 8;     // [kUnits][128]
  static constexpr int kUnitOff = kQScaleOff + (kFp8 ? kUnits * kTreeTcRows * 4 : 0);  // [kUnits]
  static constexpr int kBarOff = kUnitOff + kUnits * 64;
  static constexpr int kScratchOff = kBarOff + 64 * 8;
  static constexpr int kSmem = kScratchOff + (kThreads / 32 + 3) * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kOCol = 2 * TT;          // accumulator g at kOCol + g * D
  static_assert(kOCol + NWG * D <= int(kTmemCols), "TMEM columns");

  // Columns (within a score buffer) of the 8-token group q of the 32-token
  // chunk j, whose tokens are 32 j + 8 q ..; the probabilities of tokens 32 j +
  // 16 a .. + 15 go to the 8 columns of group a (hi) and of group 2 + a (lo).
  static __host__ __device__ constexpr int col(int j, int q) {
    return BS == 8 ? 32 * j + 8 * q
                   : (BS == 16 ? (q & 1) * (TT / 2) + (2 * j + (q >> 1)) * 8 : q * (TT / 4) + j * 8);
  }
};

// Unit descriptor of the ring (64 bytes at most).
struct TreeTcUnit {
  int32_t end, q0, T, L, ctx, kvh, row0, rows, tile0, tile1, tiles, first, seq;
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

__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

// A from tensor memory: row = lane, two 16-bit elements of K per column.
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

template <typename T, typename KV, int D, int BS>
__global__ void __launch_bounds__(TreeTcCfg<T, KV, D, BS>::kThreads, 1)
    tree_tc_kernel(const TreeParams p) {
  using Cfg = TreeTcCfg<T, KV, D, BS>;
  using Op = typename Cfg::Op;
  constexpr int TT = Cfg::TT, NWG = Cfg::NWG, OS = Cfg::OS, RS = Cfg::RS, NQ = Cfg::NQ, MB = Cfg::MB;
  constexpr int kPages = Cfg::kPages, kPage = Cfg::kPage, kPageRaw = Cfg::kPageRaw;
  constexpr int kTile = Cfg::kTile, kWords = Cfg::kWords, CS = Cfg::CS, RT = kTreeTcRows;
  constexpr bool kFp8 = Cfg::kFp8, kBf16 = std::is_same<Op, __nv_bfloat16>::value;
  constexpr int kPrep0 = Cfg::kSoftWarps, kCopyWarp = kPrep0 + 4, kMmaWarp = kPrep0 + 5;
  constexpr unsigned FULL = 0xffffffffu;
  // f16 probabilities are kept 2^7 larger (at most 2^15 with the lazy max), so
  // that small ones stay clear of f16's subnormals.
  constexpr float kLift = kBf16 ? 0.f : 7.f;
  constexpr float kLag = 8.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  extern __shared__ __align__(1024) uint8_t tree_tc_smem[];
  uint8_t *smem = tree_tc_smem;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kBarOff);
  uint64_t *raw_full = bars + 0;     // [RS <= 8] pages landed (tx bytes)
  uint64_t *raw_free = bars + 8;     // [RS] 8-bit caches: widened (4 prep warps)
  // Operands ready, by tile modulo 4 and not by slot (16-bit keys need no prep,
  // and with an odd number of slots a slot holds keys and values in turn).
  uint64_t *k_ready = bars + 16;     // [4] 8-bit caches: keys widened (4 prep warps)
  uint64_t *v_ready = bars + 20;     // [4] values in operand layout (4 prep warps)
  uint64_t *op_free = bars + 24;     // [OS] MMAs on the slot done (commit)
  uint64_t *s_full = bars + 32;      // [2] scores in TMEM (commit)
  uint64_t *p_full = bars + 34;      // [2] probabilities written (4 warps)
  uint64_t *pv_done = bars + 36;     // [2] value product done (commit)
  uint64_t *q_ready = bars + 38;     // [NQ] queries written (4 prep warps)
  uint64_t *q_free = bars + 40;      // [NQ] last score MMA of the unit done (commit)
  uint64_t *o_free = bars + 42;      // accumulators read (softmax warps)
  uint64_t *stat_full = bars + 43;   // group sums exchanged (softmax warps)
  uint64_t *unit_full = bars + 44;   // [kUnits] descriptor written
  uint64_t *unit_free = bars + 48;   // [kUnits] descriptor read (all other warps)
  uint64_t *prep_bar = bars + 54;    // the prep warps among themselves
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 52);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 53);
  uint32_t *masks = reinterpret_cast<uint32_t *>(smem + Cfg::kMaskOff);  // [MB][128][kWords]
  uint32_t *bad = reinterpret_cast<uint32_t *>(smem + Cfg::kBadOff);     // [MB][4]
  float2 *stats = reinterpret_cast<float2 *>(smem + Cfg::kStatOff);      // [2][2][128]
  float *qscale = reinterpret_cast<float *>(smem + Cfg::kQScaleOff);     // [kUnits][128]
  int64_t *scratch = reinterpret_cast<int64_t *>(smem + Cfg::kScratchOff);
  auto unit_at = [&](int u) {
    return reinterpret_cast<TreeTcUnit *>(smem + Cfg::kUnitOff + (u % Cfg::kUnits) * 64);
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < RS; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_free[i], 4);
    }
    for (int i = 0; i < OS; ++i) mbar_init(&op_free[i], 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&k_ready[i], 4);
      mbar_init(&v_ready[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&q_ready[i], 4);
      mbar_init(&q_free[i], 1);
    }
    mbar_init(prep_bar, 4);
    mbar_init(o_free, Cfg::kSoftWarps);
    mbar_init(stat_full, Cfg::kSoftWarps);
    for (int i = 0; i < Cfg::kUnits; ++i) {
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_free[i], Cfg::kSoftWarps + 5);
    }
    *abort_flag = 0;
    for (int i = 0; i < MB * 4; ++i) bad[i] = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tc::tmem_alloc(tmem_slot, Cfg::kTmemCols);
  grid_dependency_wait();
  allow_dependent_launch();
  const TreeRun run = tree_find_run<TT, RT, Cfg::kThreads>(p, scratch);
  if (run.begin >= run.end && threadIdx.x == 0) tree_write_cut(p, run, nullptr);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint64_t wait_ns = p.wait_limit_ns;
  const uint64_t drain_ns = min(wait_ns, uint64_t(100000000ull));
  bool failed = false;

  auto wait_one = [&](uint64_t *bar, uint32_t parity) { return tc_wait(bar, parity, wait_ns, abort_flag); };
  auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
    return bool(__all_sync(FULL, tc_wait(bar, parity, wait_ns, abort_flag)));
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
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------ copies --
    // pages that another row tile reads too stay in L2
    const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_normal();
    TreeWalk<TT, RT> walk;
    walk.start(p, run);
    TreeStretch st;
    int64_t n = 0;  // items (key and value tiles in turn) issued
    int u = 0, ids0 = 0, ids0_seq = -1;
    bool first = true;
    while (!failed) {
      const bool more = walk.next(p, st);
      if (u >= Cfg::kUnits &&
          !wait_warp(&unit_free[u % Cfg::kUnits], uint32_t(u / Cfg::kUnits - 1) & 1u)) {
        failed = true;
        break;
      }
      if (lane == 0) {
        TreeTcUnit *d = unit_at(u);
        d->end = !more;
        if (more) {
          d->q0 = st.q.q0;
          d->T = st.q.T;
          d->L = st.q.L;
          d->ctx = st.q.ctx;
          d->kvh = st.kvh;
          d->row0 = st.row0;
          d->rows = st.rows;
          d->tile0 = st.tile0;
          d->tile1 = st.tile1;
          d->tiles = st.tiles;
          d->first = first;
          d->seq = st.seq;
          if (first) tree_write_cut(p, run, &st);
        }
        tc::mbar_arrive(&unit_full[u % Cfg::kUnits]);
      }
      __syncwarp();
      ++u;
      first = false;
      if (!more) break;
      const int64_t row = tree_table_row(p, st.seq);
      const int npages = (st.q.L + BS - 1) / BS;
      const uint8_t *kb = static_cast<const uint8_t *>(p.k) + int64_t(st.kvh) * p.k_s1 * CS;
      const uint8_t *vb = static_cast<const uint8_t *>(p.v) + int64_t(st.kvh) * p.v_s1 * CS;
      const int page0 = st.tile0 * kPages;
      auto load_ids = [&](int page) {  // this lane's of 32 pages from `page` on
        return page + lane < npages ? tree_block_id(p, row, page + lane) : 0;
      };
      int ids;
      if (page0 == 0 && ids0_seq == st.seq) {
        ids = ids0;  // another kv head or row tile of the same sequence
      } else {
        ids = load_ids(page0);
        if (page0 == 0) {
          ids0 = ids;
          ids0_seq = st.seq;
        }
      }
      int next_ids = load_ids(page0 + 32);
      for (int tile = st.tile0; tile < st.tile1 && !failed; ++tile) {
        const int pg = tile * kPages, rel = pg - page0;
        if (rel > 0 && (rel & 31) == 0) {
          ids = next_ids;
          next_ids = load_ids(pg + 32);
        }
        const int id = __shfl_sync(FULL, ids, ((rel & 31) + lane) & 31);
        const int np = max(0, min(kPages, npages - pg));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const int s = int(n % RS);
          if (n >= RS &&
              !wait_warp(kFp8 ? &raw_free[s] : &op_free[s], uint32_t(n / RS - 1) & 1u)) {
            failed = true;
            break;
          }
          if (lane == 0)
            mbar_arrive_expect_tx(&raw_full[s], uint32_t(np * kPageRaw) +
                                                    (kv == 0 ? p.extra_expect_tx : 0u));
          __syncwarp();
          if (lane < np) {
            uint8_t *dst = smem + (kFp8 ? Cfg::kRawOff + s * Cfg::kRawTile : s * kTile) + lane * kPageRaw;
            const uint8_t *src = kv == 0 ? kb + int64_t(id) * p.k_s0 * CS : vb + int64_t(id) * p.v_s0 * CS;
            bulk_copy_g2s(dst, src, uint32_t(kPageRaw), &raw_full[s], st.q.row_tiles > 1 ? again : once);
          }
        }
      }
    }
    // No copy may be in flight when the CTA exits.
    for (int64_t i = n > RS ? n - RS : 0; i < n; ++i)
      mbar_wait_bounded(&raw_full[i % RS], uint32_t(i / RS) & 1u, drain_ns);
    __syncwarp();
  } else if (warp >= kPrep0 && warp < kPrep0 + 4) {
    // -------------------------------------------------------------- prep --
    const int pt = threadIdx.x - kPrep0 * 32, pw = warp - kPrep0;
    int64_t g = 0;  // tiles
    uint32_t syncs = 0;
    for (int u = 0; !failed; ++u) {
      TreeTcUnit d;
      if (!take_unit(u, d)) {
        failed = true;
        break;
      }
      if (d.end) break;
      // queries: row pt of the row tile, K-major core matrices (chunk of 8 dims
      // 2048 bytes, row 16 bytes)
      const int qb = u % NQ;
      if (u >= NQ && !wait_warp(&q_free[qb], uint32_t(u / NQ - 1) & 1u)) {
        failed = true;
        break;
      }
      if (pt < d.rows) {
        const int R = d.row0 + pt;
        const T *q = static_cast<const T *>(p.q) + int64_t(d.q0 + R / p.group) * p.q_s0 +
                     int64_t(d.kvh * p.group + R % p.group) * p.q_s1;
        uint8_t *dst = smem + Cfg::kQOff + qb * Cfg::kQBytes + pt * 16;
        const bool vec = p.q_s2 == 1 && (reinterpret_cast<uintptr_t>(q) & 15u) == 0;
        auto chunk = [&](int c, uint32_t (&w)[4]) {  // dims 8 c .. 8 c + 7, packed as T
          if (vec) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(q) + c);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack2<T>(to_f32<T>(q[int64_t(c * 8 + 2 * e) * p.q_s2]),
                              to_f32<T>(q[int64_t(c * 8 + 2 * e + 1) * p.q_s2]));
          }
        };
        if constexpr (std::is_same<Op, T>::value) {
          if (kFp8) qscale[(u % Cfg::kUnits) * RT + pt] = 1.f;
#pragma unroll 8
          for (int c = 0; c < D / 8; ++c) {
            uint32_t w[4];
            chunk(c, w);
            *reinterpret_cast<uint4 *>(dst + c * 2048) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          // bf16 into f16: max |q| of the row brought into [2^14, 2^15), exactly
          float amax = 0.f;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            uint32_t w[4];
            chunk(c, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack2<T>(w[e]);
              amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
          int k = 0;
          if (amax > 0.f && amax < INFINITY) k = clamp_int(141 - int(__float_as_uint(amax) >> 23), -100, 100);
          const float up = __uint_as_float(uint32_t(127 + k) << 23);
          qscale[(u % Cfg::kUnits) * RT + pt] = __uint_as_float(uint32_t(127 - k) << 23);
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            uint32_t w[4];
            chunk(c, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack2<T>(w[e]);
              w[e] = pack2<__half>(f.x * up, f.y * up);
            }
            *reinterpret_cast<uint4 *>(dst + c * 2048) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&q_ready[qb]);
      const int node0 = d.row0 / p.group;
      const int nodes = (d.row0 + d.rows - 1) / p.group - node0 + 1;
      for (int tile = d.tile0; tile < d.tile1 && !failed; ++tile, ++g) {
        const int t0 = tile * TT;
        const int nt = min(TT, d.L - t0);  // tokens of the tile (<= 0: none)
        const bool tail = t0 + TT > d.ctx;
        const int mb = int(g % MB);
#pragma unroll 1
        for (int kv = kFp8 ? 0 : 1; kv < 2; ++kv) {
          const int64_t n = 2 * g + kv;
          const int rs = int(n % RS), os = int(n % OS);
          if (!wait_warp(&raw_full[rs], uint32_t(n / RS) & 1u) ||
              (kFp8 && n >= OS && !wait_warp(&op_free[os], uint32_t(n / OS - 1) & 1u))) {
            failed = true;
            break;
          }
          uint8_t *op = smem + os * kTile;
          if constexpr (kFp8) {
            const uint8_t *raw = smem + Cfg::kRawOff + rs * Cfg::kRawTile;
#pragma unroll 4
            for (int i = pt; i < TT * D / 16; i += 128) {
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
            if (pt < 4) bad[mb * 4 + pt] = 0;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(prep_bar);
            if (!wait_warp(prep_bar, syncs++ & 1u)) {
              failed = true;
              break;
            }
            // What each row sees of the tile, a bit per token.
            for (int i = pw; i < nodes; i += 4) {
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
            for (int i = pt; i < (TT / 8 - t8) * D; i += 128) {
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
            tc::mbar_arrive(kv == 0 ? &k_ready[g & 3] : &v_ready[g & 3]);
            if (kFp8) tc::mbar_arrive(&raw_free[rs]);
          }
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issue --
    // The unit loop is the whole warp's, the MMAs are lane 0's.
    constexpr uint32_t idesc_k = tc::idesc_f16(kBf16, Cfg::kNK, RT);
    constexpr uint32_t idesc_v = tc::idesc_f16(kBf16, D, RT);
    uint64_t *last = nullptr;
    uint32_t last_parity = 0;
    int64_t g = 0, pend = -1;  // pend: the tile whose value product is due
    bool pend_fresh = false;   // the first product into its accumulator
    int pend_unit = 0;
    auto value_product = [&]() -> bool {
      const int b = int(pend & 1), acc = NWG == 2 ? b : 0;
      const int64_t n = 2 * pend + 1;
      const int os = int(n % OS);
      if (!wait_one(&p_full[b], uint32_t(pend >> 1) & 1u) ||
          !wait_one(&v_ready[pend & 3], uint32_t(pend >> 2) & 1u) ||
          (pend_fresh && pend_unit > 0 && !wait_one(o_free, uint32_t(pend_unit - 1) & 1u)))
        return false;
      if (!kFp8 && !wait_one(&raw_full[os], uint32_t(n / OS) & 1u)) return false;
      tc::fence_after_sync();
      const uint32_t v0 = smem_addr(smem + os * kTile);
      const uint32_t o = tmem + uint32_t(Cfg::kOCol + acc * D), s = tmem + uint32_t(b * TT);
#pragma unroll
      for (int ks = 0; ks < TT / 16; ++ks) {
        uint64_t vd;
        if constexpr (BS == 8)
          vd = tc::smem_desc(v0 + 2 * ks * kPage, kPage, 128);
        else if constexpr (BS == 16)
          vd = tc::smem_desc_swizzled(v0 + ks * kPage, 256, 6);
        else
          vd = tc::smem_desc_swizzled(v0 + (ks >> 1) * kPage + (ks & 1) * 32, 512, 4);
        tc::mma_f16_ts(o, s + uint32_t(Cfg::col(ks >> 1, ks & 1)), vd, idesc_v, !(pend_fresh && ks == 0));
        tc::mma_f16_ts(o, s + uint32_t(Cfg::col(ks >> 1, 2 + (ks & 1))), vd, idesc_v, true);
      }
      tc::commit(&op_free[os]);
      tc::commit(&pv_done[b]);
      last = &pv_done[b];
      last_parity = uint32_t(pend >> 1) & 1u;
      return true;
    };
    for (int u = 0; !failed; ++u) {
      TreeTcUnit d;
      if (!take_unit(u, d)) {
        failed = true;
        break;
      }
      if (d.end) break;
      if (lane == 0) {
        const int qb = u % NQ;
        bool ok = wait_one(&q_ready[qb], uint32_t(u / NQ) & 1u);
        const uint32_t q0 = smem_addr(smem + Cfg::kQOff + qb * Cfg::kQBytes);
        for (int tile = d.tile0; ok && tile < d.tile1; ++tile, ++g) {
          const int b = int(g & 1);
          const int64_t n = 2 * g;
          const int os = int(n % OS);
          ok = kFp8 ? wait_one(&k_ready[g & 3], uint32_t(g >> 2) & 1u)
                    : wait_one(&raw_full[os], uint32_t(n / OS) & 1u);
          // the score buffer holds the probabilities of tile g - 2 until its product is done
          if (ok && g >= 2) ok = wait_one(&pv_done[b], uint32_t((g >> 1) - 1) & 1u);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t k0 = smem_addr(smem + os * kTile);
#pragma unroll 1
          for (int h = 0; h < Cfg::kSub; ++h) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              tc::mma_f16_ss(tmem + uint32_t(b * TT + h * Cfg::kNK),
                             tc::smem_desc(q0 + ks * 4096, 2048, 128),
                             tc::smem_desc(k0 + h * 128 + ks * 2 * BS * 16, BS * 16, kPage), idesc_k,
                             ks > 0);
          }
          if (tile == d.tile1 - 1) tc::commit(&q_free[qb]);
          tc::commit(&op_free[os]);
          tc::commit(&s_full[b]);
          last = &s_full[b];
          last_parity = uint32_t(g >> 1) & 1u;
          if (pend >= 0 && !value_product()) {
            ok = false;
            break;
          }
          pend = g;
          pend_unit = u;
          pend_fresh = NWG == 2 ? tile < d.tile0 + 2 : tile == d.tile0;
        }
        // The unit's last product does not wait for the next unit's scores.
        if (ok && pend >= 0 && !value_product()) ok = false;
        pend = -1;
        failed = !ok;
      }
      failed = __shfl_sync(FULL, int(failed), 0) != 0;
    }
    if (lane == 0 && last != nullptr && !mbar_wait_bounded(last, last_parity, drain_ns)) failed = true;
    __syncwarp();
  } else {
    // ----------------------------------------------------------- softmax --
    const int wg = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const TreeLogit logit(p);
    int64_t g = 0;
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
      if (p.alibi) {
        slope = p.alibi[head] * kLog2e;
        qpos = p.positions ? p.positions[d.q0 + node] : d.ctx + node;
      }
      const bool simple = p.cap == 0.f && !p.alibi && p.scale > 0.f;
      float m = -INFINITY, l = 0.f;  // m: the reference that the accumulator is scaled to
      bool have = false;             // this group's accumulator holds something
      int64_t mine = -1;             // its last tile
      for (int tile = d.tile0; tile < d.tile1; ++tile, ++g) {
        if (NWG == 2 && int(g & 1) != wg) continue;
        const int b = int(g & 1), mb = int(g % MB);
        const uint32_t s = tmem + lanes + uint32_t(b * TT);
        if (!wait_warp(&s_full[b], uint32_t(g >> 1) & 1u)) {
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
          if (!wait_warp(&v_ready[g & 3], uint32_t(g >> 2) & 1u)) {
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
          if (kFp8) rowscale = qscale[(u % Cfg::kUnits) * RT + min(r, d.rows - 1)];
          // pass 1: the tile's maximum, in log2 units; unless the scores are only
          // scaled, they are replaced by their final values
          float mul = logit.scale_log2 * rowscale, top = -INFINITY;
          if (simple && !tail) {
            float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < TT / 32; ++j) {
              uint32_t v[32];
              tc::ld_x32(s + uint32_t(32 * j), v);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) t4[e & 3] = fmaxf(t4[e & 3], __uint_as_float(v[e]));
            }
            top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * mul;
          } else {
#pragma unroll 1
            for (int j = 0; j < TT / 32; ++j) {
              const uint32_t bits = tail ? masks[(mb * RT + node_at) * kWords + j] : FULL;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t v[8];
                tc::ld_x8(s + uint32_t(Cfg::col(j, q)), v);
                tc::wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float z = __uint_as_float(v[e]) * rowscale;
                  float x = p.cap > 0.f ? logit.capped(z) : logit.plain(z);
                  if (p.alibi) {
                    const int t = t0 + 32 * j + 8 * q + e;
                    int kpos = t;
                    if (p.positions && t >= d.ctx && t < d.L) kpos = p.positions[d.q0 + t - d.ctx];
                    x = fmaf(slope, float(kpos - qpos), x);
                  }
                  x = (bits >> (8 * q + e)) & 1u ? x : -INFINITY;
                  v[e] = __float_as_uint(x);
                  top = fmaxf(top, x);
                }
                tc::st_x8(s + uint32_t(Cfg::col(j, q)), v);
              }
            }
            tc::wait_st();
            mul = 1.f;
          }
          // the reference moves when a score passes it by 2^kLag
          const bool grow = top > m + kLag;  // (m = -inf: any score)
          if (__any_sync(FULL, grow)) {
            const float to = grow ? top : m;
            const float alpha = to == m ? 1.f : ex2(m - to);
            if (have) {
              if (NWG == 1 && !wait_warp(&pv_done[(g - 1) & 1], uint32_t((g - 1) >> 1) & 1u)) {
                failed = true;
                break;
              }
              tc::fence_after_sync();
              const uint32_t o = tmem + lanes + uint32_t(Cfg::kOCol + wg * D);
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
          // pass 2: probabilities, a hi and a lo part, over the scores' columns
          const float ref = m == -INFINITY ? 0.f : m - kLift;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < TT / 32; ++j) {
            uint32_t v[4][8];
#pragma unroll
            for (int q = 0; q < 4; ++q) tc::ld_x8(s + uint32_t(Cfg::col(j, q)), v[q]);
            tc::wait_ld();
            uint32_t hi[2][8], lo[2][8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float a = ex2(fmaf(__uint_as_float(v[q][e]), mul, -ref));
                const float c = ex2(fmaf(__uint_as_float(v[q][e + 1]), mul, -ref));
                sum[e >> 1] += a;
                sum[e >> 1] += c;
                const uint32_t h = pack2<Op>(a, c);
                const float2 f = unpack2<Op>(h);
                hi[q >> 1][(q & 1) * 4 + e / 2] = h;
                lo[q >> 1][(q & 1) * 4 + e / 2] = pack2<Op>(a - f.x, c - f.y);
              }
            }
            tc::st_x8(s + uint32_t(Cfg::col(j, 0)), hi[0]);
            tc::st_x8(s + uint32_t(Cfg::col(j, 1)), hi[1]);
            tc::st_x8(s + uint32_t(Cfg::col(j, 2)), lo[0]);
            tc::st_x8(s + uint32_t(Cfg::col(j, 3)), lo[1]);
          }
          tc::wait_st();
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
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
          if (!wait_warp(&pv_done[b], uint32_t(g >> 1) & 1u)) {
            failed = true;
            break;
          }
          tc::fence_after_sync();
          if (live) {
            const int64_t row = tree_table_row(p, d.seq);
            const uint32_t o = tmem + lanes + uint32_t(Cfg::kOCol + wg * D);
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
      if (mine >= 0 && !wait_warp(&pv_done[mine & 1], uint32_t(mine >> 1) & 1u)) {
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
          tc::ld_x16(tmem + lanes + uint32_t(Cfg::kOCol + c), f);
          if constexpr (NWG == 2) tc::ld_x16(tmem + lanes + uint32_t(Cfg::kOCol + D + c), e1);
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
                *reinterpret_cast<float4 *>(p.acc + part * D + c + e) =
                    make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(o_free);
    }
  }

  // ------------------------------------------------------------ teardown --
  if (failed && lane == 0) flag_error(p.err, PKV_ERRF_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

}  // namespace pkv
