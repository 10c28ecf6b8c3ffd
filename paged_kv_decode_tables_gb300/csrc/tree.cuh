// Attention of drafted token trees over a paged cache: what its kernels share.
//
// Rows.  Sequence s has T_s drafted tokens (cu_query_lens), the last T_s of
// its seq_lens[s] cached tokens.  A kv head serves T_s * group query rows; row
// R is drafted token R / group under query head R % group of the kv head's
// group.  Rows are taken RT at a time (a row tile).
//
// Units and split.  A unit is (sequence, kv head, row tile); its work is its
// sequence's tiles of TT tokens (at least one).  All units' tiles, laid end to
// end, are cut into equal runs, one per CTA, whatever the lengths are: a batch
// of uneven sequences and a single long one both fill the GPU, and the
// partial results are bounded by two per CTA (a run's first and last unit) --
// the workspace depends on the GPU and the head size only.  In the line a unit
// has UC places in front of its tiles, for what it costs beside them; a run that
// starts or ends in those starts or ends at the unit's first tile.  A unit inside one
// run is written to `out` by its CTA; the others are joined by
// tree_join_kernel from their partial sums (acc = sum 2^(x - m) v, l = sum
// 2^(x - m), m; x in log2 units).
#pragma once

#include <cuda_runtime.h>

#include "../../include/paged_kv.h"
#include "pkv_ptx.cuh"

namespace pkv {

// A unit cut between CTAs, as the CTA whose run starts first inside it
// describes it for the join.
struct TreeCut {
  int32_t valid;
  int32_t q0, rows, kvh, row0;  // first query row of the sequence, rows of the tile from row0 on
  int32_t parts;                // CTAs of the split
  int64_t begin, end;           // the unit's places in the line
  int64_t each, extra;          // places of a run; the first `extra` runs have one more
};

struct TreeParams {
  const void *q;
  int64_t q_s0, q_s1, q_s2;
  const void *k;
  int64_t k_s0, k_s1;
  const void *v;
  int64_t v_s0, v_s1;
  const int32_t *bt;
  int64_t bt_s0, bt_s1;
  const int32_t *indptr;
  const int32_t *seq_lens;
  const int32_t *cu_q;       // [num_seqs + 1]
  const uint8_t *mask;       // [num_tokens, mask_cols], or null (a chain)
  int64_t m_s0, m_s1;
  const int32_t *positions;  // [num_tokens], or null (place in the sequence)
  const float *alibi;        // [num_heads], or null
  int32_t *err;
  void *out;
  int64_t o_s0, o_s1, o_s2;
  TreeCut *cuts;  // workspace: [CTAs]
  // Partial results, two per CTA: (m, l) of each row, and the sums, four dims of
  // a row together and rows adjacent (threads are rows).
  float2 *ml;   // workspace: [2 * CTAs][RT]
  float4 *acc;  // workspace: [2 * CTAs][D / 4][RT]
  int32_t num_seqs, num_tokens, num_heads, num_kv_heads, group, num_blocks, max_blocks_per_seq;
  int32_t block_size, mask_cols;
  float scale;      // of the score: args->scale (x k_scale for fp8 caches)
  float cap;        // logits_soft_cap, or 0
  float out_scale;  // v_scale for fp8 caches, else 1
  uint64_t wait_limit_ns;
  uint32_t extra_expect_tx;
};

// What the kernels need of one sequence.  Bad device data (negative or
// descending cu_query_lens, rows past num_tokens, lengths past the table or
// shorter than the drafted tokens) is clamped, and flagged where `flag`.
struct TreeSeq {
  int32_t q0, T, L, ctx;  // first query row, drafted tokens, tokens, tokens before the drafted
  int32_t tiles, row_tiles;
};

template <int TT, int RT>
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int s, bool flag) {
  TreeSeq r;
  int L = p.seq_lens[s];
  const int q0 = p.cu_q[s], q1 = p.cu_q[s + 1];
  int64_t cap_pages = p.max_blocks_per_seq;
  if (p.indptr != nullptr) {
    const int a = p.indptr[s], b = p.indptr[s + 1];
    cap_pages = int64_t(b) - a;
    if (a < 0 || cap_pages < 0) {
      if (flag) flag_error(p.err, PKV_ERRF_INDPTR);
      cap_pages = 0;
    }
  }
  // (token numbers plus a tile stay within 31 bits)
  const int64_t most = min(cap_pages * p.block_size, int64_t(0x7fffff00));
  if (L < 0 || int64_t(L) > most) {
    if (flag) flag_error(p.err, PKV_ERRF_SEQ_LEN);
    L = L < 0 ? 0 : int(most);
  }
  int T = 0;
  if (q0 < 0 || q1 < q0 || q1 > p.num_tokens) {
    if (flag) flag_error(p.err, PKV_ERRF_INDPTR);
  } else {
    T = q1 - q0;
  }
  if (T > L) {
    // rows without a cached token of their own: only the first L are drafted
    // tokens of the cache, all rows are computed over those
    if (flag) flag_error(p.err, PKV_ERRF_SEQ_LEN);
  }
  r.q0 = q0;
  r.T = T;
  r.L = L;
  r.ctx = L > T ? L - T : 0;
  r.tiles = L > 0 ? int((unsigned(L) + (TT - 1)) / TT) : 1;
  r.row_tiles = int((int64_t(T) * p.group + (RT - 1)) / RT);
  return r;
}

// What a sequence's units weigh: their tiles, and `extra` for what a unit costs
// beside them (queries, masks, epilogue).
__device__ __forceinline__ int64_t tree_weight(const TreeParams &p, const TreeSeq &q, int extra) {
  return int64_t(q.row_tiles) * p.num_kv_heads * (q.tiles + extra);
}

// Block-table row of sequence s (its page j: bt[row + j * bt_s1]).
__device__ __forceinline__ int64_t tree_table_row(const TreeParams &p, int s) {
  if (p.indptr == nullptr) return int64_t(s) * p.bt_s0;
  const int a = p.indptr[s];
  return int64_t(a < 0 ? 0 : a) * p.bt_s1;
}

// Block id of a sequence's page (an id out of range is flagged and read as
// block 0).
__device__ __forceinline__ int tree_block_id(const TreeParams &p, int64_t row, int64_t page) {
  int id = __ldg(p.bt + row + page * p.bt_s1);
  if (id < 0 || id >= p.num_blocks) {
    flag_error(p.err, PKV_ERRF_BLOCK_ID);
    id = 0;
  }
  return id;
}

// a / b for a >= 0, b > 0: 32-bit wherever they fit (a 64-bit division is a few
// hundred cycles on the way to a CTA's first load).
__device__ __forceinline__ int64_t tree_div(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return int64_t(uint32_t(a) / uint32_t(b));
  return a / b;
}

// A CTA's place in the work: its run [begin, end) of tiles, and the sequence
// that `begin` falls into (`base`: that sequence's first tile).
struct TreeRun {
  int64_t begin, end, base, each, extra;
  int32_t seq, parts;
  TreeSeq q;
  // Where the run of CTA c starts.
  __device__ __forceinline__ int64_t start_of(int64_t c) const {
    return each * c + (c < extra ? c : extra);
  }
};

// Shared memory of tree_find_run.
template <int NT>
struct TreeScratch {
  int64_t sums[NT / 32];
  int64_t base;
  int32_t seq;
  TreeSeq q;
};

// Sums the batch's tiles over the CTA's NT threads and finds the run of CTA
// blockIdx.x.  Every thread returns the same run; begin == end: nothing to do.
template <int TT, int RT, int UC, int NT>
__device__ __forceinline__ TreeRun tree_find_run(const TreeParams &p, TreeScratch<NT> &sh) {
  constexpr int NW = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // a thread's sequences: one, or a piece of a longer batch
  const int per = p.num_seqs <= NT ? 1 : (p.num_seqs + NT - 1) / NT;
  const int s0 = int(min(int64_t(tid) * per, int64_t(p.num_seqs)));
  const int s1 = min(s0 + per, p.num_seqs);
  int64_t mine = 0;
  TreeSeq q = {};
  for (int s = s0; s < s1; ++s) {
    q = tree_seq<TT, RT>(p, s, blockIdx.x == 0);
    mine += tree_weight(p, q, UC);
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) sh.sums[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int64_t t = sh.sums[w];
    if (w < warp) before += t;
    total += t;
  }
  TreeRun r;
  r.parts = int(min(int64_t(gridDim.x), total));
  r.begin = r.end = r.base = r.each = r.extra = 0;
  r.seq = 0;
  if (int(blockIdx.x) >= r.parts) return r;  // the same for every thread
  r.each = tree_div(total, r.parts);
  r.extra = total - r.each * r.parts;
  r.begin = r.start_of(blockIdx.x);
  r.end = r.start_of(int64_t(blockIdx.x) + 1);
  const int64_t first = before + incl - mine;
  if (r.begin >= first && r.begin < first + mine) {
    int64_t at = first;
    int s = s0;
    if (per > 1) {
      for (; s < s1; ++s) {
        q = tree_seq<TT, RT>(p, s, false);
        const int64_t w = tree_weight(p, q, UC);
        if (r.begin < at + w) break;
        at += w;
      }
    }
    sh.seq = s;
    sh.base = at;
    sh.q = q;
  }
  __syncthreads();
  r.seq = sh.seq;
  r.base = sh.base;
  r.q = sh.q;
  return r;
}

// One stretch of tiles of one unit within a CTA's run.
struct TreeStretch {
  int32_t seq, kvh, row0, rows;  // rows: valid rows from row0 on, at most RT
  int32_t tile0, tile1, tiles;
  int64_t begin;  // the unit's first place in the line
  TreeSeq q;
};

// Steps through a run stretch by stretch (one thread, or threads in step).
template <int TT, int RT, int UC>
struct TreeWalk {
  TreeRun run;
  int64_t pos, base;
  int32_t seq;
  TreeSeq q;
  bool fresh;

  __device__ __forceinline__ void start(const TreeParams &p, const TreeRun &r) {
    run = r;
    pos = r.begin;
    base = r.base;
    seq = r.seq;
    q = r.q;
  }
  __device__ __forceinline__ bool next(const TreeParams &p, TreeStretch &s) {
    if (pos >= run.end) return false;
    int64_t w;
    while (pos >= base + (w = tree_weight(p, q, UC))) {
      base += w;
      ++seq;
      q = tree_seq<TT, RT>(p, seq, false);
    }
    const int64_t off = pos - base;
    const int per = q.tiles + UC;
    const int64_t u = tree_div(off, per);
    const int v0 = int(off - u * per), v1 = int(min(int64_t(per), v0 + (run.end - pos)));
    s.begin = pos - v0;
    pos += v1 - v0;
    if (v1 <= UC) return false;  // the run ends before the unit's tiles do begin
    s.seq = seq;
    s.q = q;
    s.kvh = q.row_tiles == 1 ? int(u) : int(tree_div(u, q.row_tiles));
    s.row0 = int(u - int64_t(s.kvh) * q.row_tiles) * RT;
    s.rows = int(min(int64_t(RT), int64_t(q.T) * p.group - s.row0));
    s.tile0 = max(0, v0 - UC);
    s.tile1 = v1 - UC;
    s.tiles = q.tiles;
    return true;
  }
};

// Describes the unit that CTA blockIdx.x's run starts inside of, for the
// join; one thread.  `s` is the run's first stretch (null: an empty run).
template <int UC>
__device__ __forceinline__ void tree_write_cut(const TreeParams &p, const TreeRun &r,
                                               const TreeStretch *s) {
  TreeCut c = {};
  if (s != nullptr && s->tile0 > 0) {
    c.begin = s->begin;
    c.end = c.begin + s->tiles + UC;
    // the first run that starts between the unit's tiles describes it
    c.valid = r.start_of(int64_t(blockIdx.x) - 1) <= c.begin + UC;
    c.q0 = s->q.q0;
    c.rows = s->rows;
    c.kvh = s->kvh;
    c.row0 = s->row0;
    c.parts = r.parts;
    c.each = r.each;
    c.extra = r.extra;
  }
  p.cuts[blockIdx.x] = c;
}

// log2(e) * logit of a score `d` (the dot product): scaled, capped, biased.
// capped: cap * tanh(z / cap) as cap - 2 cap / (1 + e^(2 z / cap)), which is
// exact to about 3e-7 * cap (ex2 and the reciprocal are good to 2^-22);
// capped_exact: with tanhf, for fp32 outputs.
struct TreeLogit {
  float scale_log2, cap_log2, cap_arg;
  __device__ __forceinline__ explicit TreeLogit(const TreeParams &p) {
    constexpr float kLog2E = 1.44269504088896340736f;
    scale_log2 = p.scale * kLog2E;
    cap_log2 = p.cap * kLog2E;
    cap_arg = p.cap > 0.f ? p.scale / p.cap : 0.f;
  }
  __device__ __forceinline__ float plain(float d) const { return d * scale_log2; }
  __device__ __forceinline__ float capped_exact(float d) const {
    return cap_log2 * tanhf(d * cap_arg);
  }
  __device__ __forceinline__ float capped(float d) const {
    const float e = ex2(d * (cap_arg * 2.88539008177792681472f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return fmaf(-2.f * cap_log2, r, cap_log2);
  }
};

// The fp32 kernel's row tile, token tile and CTAs per SM, and the tensor-core
// kernel's rows (one CTA per SM).
constexpr int kTreeSimtRows = 32, kTreeSimtTokens = 64, kTreeSimtCtasPerSm = 2;
constexpr int kTreeTcRows = 128;
// What a unit costs beside its tiles, in tiles.  (Measured on 128 ragged trees of up
// to 16 tokens / 32 of 40-64: 6 tiles 180 / 130 us, 10 tiles 188 / 122, 16 tiles 202 /
// 126, none 230 / 185.)
constexpr int kTreeSimtUnitCost = 1, kTreeTcUnitCost = 8;

pkv_status_t launch_tree_simt(const TreeParams &p, int head_size, int ctas, cudaStream_t stream);
// Queries and caches of 16 bits, and 16-bit queries over 8-bit caches.
pkv_status_t launch_tree_tc_f16(const TreeParams &p, int head_size, int ctas, cudaStream_t s);
pkv_status_t launch_tree_tc_bf16(const TreeParams &p, int head_size, int ctas, cudaStream_t s);
pkv_status_t launch_tree_tc_f16_e4m3(const TreeParams &p, int head_size, int ctas, cudaStream_t s);
pkv_status_t launch_tree_tc_f16_e5m2(const TreeParams &p, int head_size, int ctas, cudaStream_t s);
pkv_status_t launch_tree_tc_bf16_e4m3(const TreeParams &p, int head_size, int ctas, cudaStream_t s);
pkv_status_t launch_tree_tc_bf16_e5m2(const TreeParams &p, int head_size, int ctas, cudaStream_t s);
// `ctas`: the attention kernel's grid.
pkv_status_t launch_tree_join(const TreeParams &p, pkv_dtype_t dtype, int head_size, int ctas,
                              cudaStream_t stream);

}  // namespace pkv
