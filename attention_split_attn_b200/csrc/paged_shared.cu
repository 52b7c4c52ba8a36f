// paged_shared.cu -- attention of groups of rows whose block tables begin with
// the same cells (attn_decode_shared): the shared cells of a group are read
// once for all its rows, on the sm_100a tensor cores (tcgen05 + TMEM), the
// cells of single rows by paged_stream.cu, and one combine folds both.
//
//   out = sum_c e^(x_c - M) v_c / (sum_c e^(x_c - M) + e^(sigma - M))
// splits over any partition of the cells: each part leaves (m, l, O) with its
// own maximum m, and parts fold as in the split-K combine.
//
// What bounds it.  A group of n rows with G query heads per KV head turns the
// reading of a KV head's cells into a product of n G rows with them: 4 n G D
// flops per cell against 4 D bytes, so the tensor cores bind from a few
// hundred rows x heads on, HBM below; with the softmax's exponential per
// (row, head, cell) on the special-function unit close behind the tensor cores
// at head dim 128 (2048 cycles of each per pair of 128 x 128 tiles) and ahead
// of them at 64.
//
// Kernels:
//  * shared_plan_kernel (one CTA) checks the groups, cuts their rows into
//    blocks (up to two tiles of 128 / G rows x G heads), and writes each block's cell
//    range and tile count, the prefix of the blocks' work, every row's block and
//    its own first cell, and the own parts' tile prefix for paged_stream.cu.
//  * shared_kernel: one persistent CTA per SM.  The flattened (block, KV head,
//    128-cell tile) space is cut into equal runs, one per CTA, whatever the
//    mix of groups; a run's piece of a unit (block, KV head) goes through
//      warp 0       TMA producer: the block's Q, then K and V tiles through
//                   rings.  A tile is fetched in boxes of C cells, C the largest
//                   power of two up to 128 that divides the page size, one
//                   lane per box; boxes that no row of the block sees are
//                   fetched from page n_pages, where the TMA reads zeros.
//      warp 1       tcgen05.mma issuer: S = Q K^T, then O += P V with P in
//                   tensor memory over the columns of S.
//      warps 4-7    softmax of slot 0; warps 8-11 of slot 1.  Thread t of a slot
//                   owns lane t: row t / G of the tile, query head t % G.
//    A block of more than one tile of rows runs one tile per slot, and both use
//    every K/V tile; a block of one tile runs its even cell tiles on slot 0
//    and the odd ones on slot 1 (each K/V tile used once), so that one slot's
//    products run under the other's softmax in both cases.  At head dim 256
//    tensor memory holds one slot.
//  * the combine (paged_combine.cu) folds, per (row, query head), the pieces'
//    records, the own part's records and the sink.  A row whose cells were all
//    seen by one piece is finished by that piece and skipped there.
//
// Cells that a row must not see never reach it: their weight is an exact 0,
// V rows outside the block's range are zeroed in shared memory, and a tile that
// hides some of the cells in the block's range from some row is searched for
// infinities and NaN; if it holds any, P V of that tile runs on the CUDA cores
// over each row's visible cells only (0 * NaN would be NaN).
// Cell tiles go from the last to the first: with ALiBi the nearest cells carry
// the largest logits, so the running maximum settles at once.
// Measured: 2048 rows of one sequence at depth 12000 (64 / 8 heads, D 128, bf16,
// 874 GF) 0.90 to 0.98 ms in this kernel under ncu, 0.98 to 1.03 ms a call with
// plan and combine (850 to 890 TFLOP/s); a pair of tiles takes 4060 cycles, a
// slot's softmax (2050) and its P V and next S (2000) one after the other, the
// two slots in turn, against 2048 cycles of tensor work.
// All waits are bounded; a timeout records ATTN_ERR_DEVICE_TIMEOUT, raises a
// CTA-wide flag that ends every role, drains the copies, makes every row of the
// CTA's run NaN and frees TMEM.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "decode_tile.cuh"
#include "internal.h"
#include "paged.cuh"
#include "tcgen05.cuh"

namespace attn {

namespace {

constexpr int kShRows = 128;    // lanes of a slot (MMA M)
constexpr int kShCells = 128;   // cells per tile (MMA N of S, K of P V)

template <int D>
struct ShLayout {
  static constexpr int NSLOT = D <= 128 ? 2 : 1;
  static constexpr int BOX = kShRows * 128;               // 128 rows x 128 B (64 values)
  static constexpr int TILE = kShRows * D * 2;            // a Q, K or V tile: D / 64 boxes
  static constexpr int NK = D == 64 ? 3 : D == 128 ? 2 : 1;
  static constexpr int NV = D == 64 ? 4 : D == 128 ? 3 : 1;
  static constexpr int OFF_Q = 0;                         // [NSLOT][TILE]
  static constexpr int OFF_K = OFF_Q + NSLOT * TILE;
  static constexpr int OFF_V = OFF_K + NK * TILE;
  static constexpr int OFF_BAR = OFF_V + NV * TILE;
  // q_full, q_empty, k_full[NK], k_empty[NK], v_full[NV], v_empty[NV],
  // s_full[2], p_full[2], pv_done[2], merge_full, merge_empty, mma_done, never
  static constexpr int N_BAR = 2 + 2 * NK + 2 * NV + 6 + 4;
  static constexpr int OFF_MISC = OFF_BAR + N_BAR * 8;    // TMEM address, abort flag, first block, bad[2]
  static constexpr int OFF_ML = OFF_MISC + 32;            // [128][2] floats: slot 1's (m, l) at a merge
  static constexpr int BYTES = OFF_ML + kShRows * 8;
  static constexpr int SMEM = BYTES + 1024;               // slack for 1024-byte alignment
  static constexpr int THREADS = 384;                     // 12 warps: 3 warpgroups
  // register split: 128 x 72 + 256 x 216 = 384 x 168, what the launch holds
  static constexpr int LOW_REGS = 72, HIGH_REGS = 216;
  static_assert(128 * LOW_REGS + 256 * HIGH_REGS <= THREADS * 168, "register split");
  static constexpr uint32_t TMEM_COLS = 512;              // S_s at 128 s, O_s at 256 + D s
  static_assert(NSLOT * 128 <= 256 && 256 + NSLOT * D <= (int)TMEM_COLS, "TMEM columns");
  static_assert(SMEM <= 232448, "shared memory");
};

struct ShBars {
  uint64_t *q_full, *q_empty, *k_full, *k_empty, *v_full, *v_empty, *s_full, *p_full, *pv_done, *merge_full,
      *merge_empty, *mma_done, *never;
};

template <int D>
__device__ __forceinline__ ShBars sh_bars(unsigned char* sm) {
  using L = ShLayout<D>;
  uint64_t* b = reinterpret_cast<uint64_t*>(sm + L::OFF_BAR);
  ShBars r;
  r.q_full = b;
  r.q_empty = b + 1;
  r.k_full = b + 2;
  r.k_empty = r.k_full + L::NK;
  r.v_full = r.k_empty + L::NK;
  r.v_empty = r.v_full + L::NV;
  r.s_full = r.v_empty + L::NV;
  r.p_full = r.s_full + 2;
  r.pv_done = r.p_full + 2;
  r.merge_full = r.pv_done + 2;
  r.merge_empty = r.merge_full + 1;
  r.mma_done = r.merge_empty + 1;
  r.never = r.mma_done + 1;
  return r;
}

__device__ __forceinline__ bool sh_wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort_flag,
                                        uint64_t limit_ns = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t spin = 1;; ++spin) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((spin & 63u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > limit_ns) {
        record_status(status, ATTN_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool sh_wait_warp(uint64_t* bar, uint32_t parity, int* status, volatile int* abort_flag,
                                             uint64_t limit_ns = kWaitLimitNs) {
  const bool ok = sh_wait(bar, parity, status, abort_flag, limit_ns);
  return __all_sync(0xffffffffu, ok);
}

// A place in an N-stage ring and its barriers' phase (the MMA issuer's: no
// division between a barrier and the MMAs behind it).
template <int N>
struct RingPos {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == N) {
      stage = 0;
      phase ^= 1u;
    }
  }
};
// The i-th use of an N-stage ring.
template <int N>
__device__ __forceinline__ int ring_stage(int64_t i) { return (int)(i % N); }
template <int N>
__device__ __forceinline__ uint32_t ring_phase(int64_t i) { return (uint32_t)((i / N) & 1); }

// ---------------------------------------------------------------------------
// planner
// ---------------------------------------------------------------------------

// One CTA: everything between its loads and its stores happens in shared
// memory, so its time is a few dependent loads and barriers.
constexpr int kPlanThreads = 1024;   // at most; 256 for few rows and groups (cheaper barriers)
constexpr int kPlanBlocks = 1024;   // blocks kept in shared memory; a plan that may hold more works in the workspace

// Exclusive scan of x over the CTA on top of *carry (the same in every
// thread), which grows by the total.
__device__ __forceinline__ int64_t cta_excl_scan(int64_t x, int64_t* carry, long long* wsum) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int64_t v = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += y;
  }
  __syncthreads();   // the previous scan's sums are read
  if (lane == 31) wsum[wid] = v;
  __syncthreads();
  int64_t s = lane < (int)(blockDim.x >> 5) ? wsum[lane] : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += y;
  }
  const int64_t before = __shfl_sync(0xffffffffu, s, wid > 0 ? wid - 1 : 0);
  const int64_t excl = *carry + (wid > 0 ? before : 0) + v - x;
  *carry += __shfl_sync(0xffffffffu, s, 31);
  return excl;
}

struct PlanShared {
  SharedBlock blocks[kPlanBlocks];
  int64_t off[kPlanBlocks + 1];
  int first_run[kPlanBlocks + 1];   // when units <= W
  long long wsum[32];
};

// Dynamic shared memory: PlanShared, or only its wsum when the blocks and
// their offsets live in the workspace.
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedPlan sp) {
  extern __shared__ long long plan_smem[];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const PagedPlan& p = sp.p;
  const int tid = threadIdx.x, nthr = blockDim.x, R = p.d.R, Hkv = p.d.Hkv;
  const bool in_smem = sp.max_blk <= kPlanBlocks;
  PlanShared* ps = reinterpret_cast<PlanShared*>(plan_smem);
  SharedBlock* blocks = in_smem ? ps->blocks : sp.blocks;
  int64_t* off = in_smem ? ps->off : sp.blk_off;
  long long* wsum = in_smem ? ps->wsum : plan_smem;

  // the first rows' ranges and the groups are loaded together: one latency
  PagedRow first_row{};
  if (tid < R) first_row = paged_row(p, tid);   // (own_lo of this plan is NULL: the whole range)

  // 1. are the groups well formed?  One that ends behind the rows is if its
  // rows see nothing: a sequence whose rows did not fit (attn_page_tables'
  // seq_row runs on, its rows have row_end 0).
  bool any_bad = false, bad = false, past = false;
  for (int i = tid; i <= sp.n_groups; i += nthr) {
    const int b = __ldg(sp.group_begin + i);
    bad |= b < 0 || (i == 0 && b > R) || (i > 0 && b < __ldg(sp.group_begin + i - 1));
    past |= b > R;
  }
  if (__syncthreads_or(bad || past) && !(any_bad = __syncthreads_or(bad))) {
    __shared__ int tail;   // the first row of the one group that ends behind the rows
    for (int i = tid; i < sp.n_groups; i += nthr) {
      const int b = __ldg(sp.group_begin + i);
      if (b <= R && __ldg(sp.group_begin + i + 1) > R) tail = b;
    }
    __syncthreads();
    bool seen = false;
    for (int64_t r = (int64_t)tail + tid; r < R; r += nthr) seen |= paged_row(p, (int)r).tiles() > 0;
    any_bad = __syncthreads_or(seen);
  }
  if (any_bad && tid == 0) record_status(p.d.status, ATTN_ERR_INVALID_ARG);
  const int n_groups = any_bad ? 0 : sp.n_groups;

  // 2. blocks of at most block_rows rows (a group of one row shares nothing)
  const int cap = p.width * p.P;
  int64_t nb = 0;
  for (int base = 0; base < n_groups; base += nthr) {
    const int i = base + tid;
    int r0 = 0, n = 0, len = 0, table = 0;
    if (i < n_groups) {
      r0 = __ldg(sp.group_begin + i);
      n = min(__ldg(sp.group_begin + i + 1), R) - r0;   // (below 0 for a group behind the rows)
      len = min(__ldg(sp.group_len + i), cap);
      if (n > 0) table = p.row_table ? __ldg(p.row_table + r0) : r0;
      if (n < 2 || len <= 0 || table < 0 || table >= p.n_tables) n = 0;
    }
    const int mine = (n + sp.block_rows - 1) / sp.block_rows;
    const int64_t at = cta_excl_scan(mine, &nb, wsum);
    for (int k = 0; k < mine; ++k) {
      SharedBlock b;
      b.row0 = r0 + k * sp.block_rows;
      b.n_rows = min(sp.block_rows, n - k * sp.block_rows);
      b.table = table;
      b.len = len;
      b.lo = 0x7fffffff;
      b.hi = 0;
      b.w = (sp.n_slot == 2 && b.n_rows > sp.rpt) ? 2 : 1;
      b.kt0 = b.nt = 0;
      b.clo[0] = b.clo[1] = 0;
      b.chi[0] = b.chi[1] = 0x7fffffff;
      blocks[at + k] = b;
    }
  }
  const int n_blk = (int)nb;
  __syncthreads();

  // 3. rows: their block, its cell range, and the own parts' tile prefix
  int64_t carry = 0;
  for (int base = 0; base < R; base += nthr) {
    const int r = base + tid;
    int64_t tiles = 0;
    if (r < R) {
      PagedRow row = base == 0 ? first_row : paged_row(p, r);
      int k = -1, own = 0;
      {   // the last block with row0 <= r
        int lo = 0, hi = n_blk;
        while (hi - lo > 0) {
          const int mid = (lo + hi) >> 1;
          if (blocks[mid].row0 <= r) lo = mid + 1;
          else hi = mid;
        }
        if (lo > 0 && r < blocks[lo - 1].row0 + blocks[lo - 1].n_rows) k = lo - 1;
      }
      if (k >= 0) {
        SharedBlock* b = blocks + k;
        own = b->len;
        const int e = min(row.end, own);
        if (e > row.begin) {
          const int s = b->w == 2 && r - b->row0 >= sp.rpt ? 1 : 0;
          atomicMin(&b->lo, row.begin);
          atomicMax(&b->hi, e);
          atomicMax(&b->clo[s], row.begin);
          atomicMin(&b->chi[s], e);
        }
      }
      sp.row_blk[r] = k;
      sp.own_lo[r] = own;
      row.begin = max(row.begin, own);
      row.end = max(row.end, row.begin);
      row.tile0 = row.begin / 16;
      tiles = row.tiles();
    }
    const int64_t at = cta_excl_scan(tiles, &carry, wsum);
    if (r < R) p.d.row_tiles[r] = at;
  }
  if (tid == 0) p.d.row_tiles[R] = carry;
  __syncthreads();

  // 4. the blocks' tiles, and the prefix of their work in tiles of one slot
  int64_t work = 0;
  for (int base = 0; base < n_blk; base += nthr) {
    const int k = base + tid;
    int64_t x = 0;
    if (k < n_blk) {
      SharedBlock b = blocks[k];
      if (!in_smem) {   // updated by atomics: read past the L1 cache
        b.lo = __ldcg(&blocks[k].lo);
        b.hi = __ldcg(&blocks[k].hi);
        for (int s = 0; s < 2; ++s) {
          b.clo[s] = __ldcg(&blocks[k].clo[s]);
          b.chi[s] = __ldcg(&blocks[k].chi[s]);
        }
      }
      b.lo = min(b.lo, b.hi);
      b.kt0 = b.lo / kShCells;
      b.nt = b.hi > b.lo ? (b.hi + kShCells - 1) / kShCells - b.kt0 : 0;
      if (b.w == 1) {   // one tile of rows: both slots work on it
        b.clo[1] = b.clo[0];
        b.chi[1] = b.chi[0];
      }
      blocks[k] = b;
      if (in_smem) sp.blocks[k] = b;
      x = (int64_t)b.nt * b.w;
    }
    const int64_t at = cta_excl_scan(x, &work, wsum);
    if (k < n_blk) off[k] = at;
  }
  if (tid == 0) off[n_blk] = work;
  __syncthreads();

  // 5. runs.  Units (block, KV head) that outnumber the runs: equal runs of
  // the flattened work, wherever their ends fall.  Fewer units: every unit
  // gets runs of its own, in proportion to its work, so that a run sets up and
  // writes out one piece only (a piece costs about as much as two tiles) --
  // while runs are short: rounding to whole runs leaves them uneven, by 20% and
  // more for a few units of different lengths.
  const int W = sp.W;
  const int64_t T = work * Hkv;
  const bool parts = in_smem && (int64_t)n_blk * Hkv <= W && T > 0 && T <= 16 * W;
  const SharedRun none{n_blk, 0, 0, 0, {}};
  if (!parts) {
    for (int w = tid; w <= W; w += nthr) {
      SharedRun s = none;
      const int64_t t = div64(T * w, W);
      if (t < T) {
        int lo = 0, hi = n_blk;   // the last block whose work starts at or before t
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (Hkv * off[mid] <= t) lo = mid;
          else hi = mid;
        }
        const int bw = blocks[lo].w, nt = blocks[lo].nt;
        const int64_t in = t - Hkv * off[lo], unit = (int64_t)nt * bw;   // (the last such block has work)
        s.k = lo;
        s.g = (int)div64(in, unit);
        s.i = (int)((in - s.g * unit + bw - 1) / bw);
        if (s.i == nt) {   // the unit's end: the start of the next unit with a tile
          s.i = 0;
          if (++s.g == Hkv) {
            s.g = 0;
            do ++s.k;
            while (s.k < n_blk && blocks[s.k].nt == 0);
          }
        }
        if (s.k < n_blk) s.b = blocks[s.k];
      }
      sp.runs[w] = s;
    }
    for (int64_t base = 0; base < (int64_t)n_blk * Hkv; base += nthr) {
      const int64_t u = base + tid;
      int2 v = make_int2(0, -1);
      if (u < (int64_t)n_blk * Hkv) {
        const int k = (int)div64(u, Hkv), g = (int)(u - (int64_t)k * Hkv);
        const SharedBlock& b = blocks[k];
        if (b.nt > 0) {
          const int64_t at = Hkv * off[k] + (int64_t)g * b.nt * b.w, last = at + (int64_t)(b.nt - 1) * b.w;
          v = make_int2(run_of(at, T, W), run_of(last, T, W));
        }
      }
      if (u < (int64_t)n_blk * Hkv) sp.unit_runs[u] = v;
    }
  } else {
    // units <= W: their first runs, kept in shared memory (the scan's order)
    const int units = n_blk * Hkv;
    int64_t used = 0;
    int* first_run = ps->first_run;
    for (int base = 0; base < units; base += nthr) {
      const int u = base + tid;
      int n = 0;
      if (u < units) {
        const SharedBlock& b = blocks[u / Hkv];
        // floor(share of the runs beyond one each) + 1, at most one per tile
        if (b.nt > 0) n = min(b.nt, 1 + (int)div64((int64_t)b.nt * b.w * (W - units), T));
      }
      const int64_t at = cta_excl_scan(n, &used, wsum);
      if (u < units) {
        first_run[u] = (int)at;
        sp.unit_runs[u] = make_int2((int)at, (int)at + n - 1);
      }
    }
    if (tid == 0) first_run[units] = (int)used;
    __syncthreads();
    for (int w = tid; w <= W; w += nthr) {
      SharedRun s = none;
      if (w < used) {
        int lo = 0, hi = units;   // the last unit whose first run is at or before w
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (first_run[mid] <= w) lo = mid;
          else hi = mid;
        }
        s.k = lo / Hkv;
        s.g = lo - s.k * Hkv;
        s.b = blocks[s.k];
        s.i = (int)div64((int64_t)s.b.nt * (w - first_run[lo]), first_run[lo + 1] - first_run[lo]);
      }
      sp.runs[w] = s;
    }
  }
}

// ---------------------------------------------------------------------------
// runs and pieces
// ---------------------------------------------------------------------------

// A run's piece of a unit: tiles [i0, i1) of a block, KV head g (tile i is
// cell tile kt0 + nt - 1 - i).
struct Piece {
  SharedBlock b;
  int g;
  int i0, i1;
  __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == b.nt; }
  __device__ __forceinline__ int kt(int i) const { return b.kt0 + b.nt - 1 - i; }
};

struct PieceCursor {
  const SharedBlock* blocks;
  SharedBlock b;            // block k, once loaded
  int k, g, i, loaded;
  int ke, ge, ie;           // where the run ends
  int Hkv;
  // The next piece with a tile (every role steps alike).
  __device__ __forceinline__ bool next(Piece* pc) {
    while (k < ke || (k == ke && (g < ge || (g == ge && i < ie)))) {
      if (loaded != k) {
        b = blocks[k];
        loaded = k;
      }
      pc->b = b;
      pc->g = g;
      pc->i0 = i;
      pc->i1 = (k == ke && g == ge) ? ie : b.nt;
      i = 0;
      if (++g == Hkv) {
        g = 0;
        ++k;
      }
      if (pc->i0 < pc->i1) return true;
    }
    return false;
  }
};

__device__ __forceinline__ PieceCursor run_cursor(const SharedPlan& sp, int run) {
  PieceCursor c;
  const SharedRun* s = sp.runs + run;
  c.blocks = sp.blocks;
  c.k = c.loaded = s->k;
  c.g = s->g;
  c.i = s->i;
  c.b = s->b;
  c.ke = s[1].k;
  c.ge = s[1].g;
  c.ie = s[1].i;
  c.Hkv = sp.p.d.Hkv;
  return c;
}

// ---------------------------------------------------------------------------
// softmax of a tile
// ---------------------------------------------------------------------------

template <typename KT>
__device__ __forceinline__ uint32_t sh_pack(float lo, float hi) {
  uint32_t r;
  if constexpr (Storage<KT>::kDtype == ATTN_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename KT>
__device__ __forceinline__ float sh_widen(uint32_t bits) {
  if constexpr (Storage<KT>::kDtype == ATTN_BF16) return __uint_as_float(bits << 16);
  else return __half2float(__ushort_as_half((unsigned short)bits));
}

// Whether a 16-byte piece of V holds an infinity or NaN.
template <typename KT>
__device__ __forceinline__ bool sh_non_finite(const uint4& w) {
  constexpr uint32_t E = Storage<KT>::kDtype == ATTN_BF16 ? 0x7f807f80u : 0x7c007c00u;
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) bad |= (~ws[k] & E & 0xffffu) == 0 || (~ws[k] & E & 0xffff0000u) == 0;
  return bad;
}

// NaN-propagating maximum of 128 values.
__device__ __forceinline__ float sh_max128(const float* x) {
  float mx[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) mx[k] = fmax_nan(x[2 * k], x[2 * k + 1]);
#pragma unroll
  for (int i = 8; i < kShCells; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) mx[k] = fmax3_nan(mx[k], x[i + 2 * k], x[i + 2 * k + 1]);
  return fmax_nan(fmax_nan(mx[0], mx[1]), fmax_nan(mx[2], mx[3]));
}

// c tanh(u / c) of any u, y = u / c.  sh_cap_far: c (1 - 2 / (e^(2|y|) + 1)),
// whose difference costs an error near 2e-7 c, whatever u.  sh_cap: the same
// for |y| > 1/4, where that is 8e-7 of u at most, and below it the odd Taylor
// series in y, u (1 + y^2 (-1/3 + ... + 62/2835 y^6)), off by 8.9e-3 y^10 <
// 9e-9 of u before roundings.  NaN stays NaN.
__device__ __forceinline__ float sh_cap_far(float u, float c, float k) {   // k = 2 log2(e) / c
  const float e = ex2(fabsf(u) * k);
  return copysignf(c * (1.f - __fdividef(2.f, e + 1.f)), u);
}
__device__ __forceinline__ float sh_cap(float u, float c, float inv_c, float k) {
  const float y = u * inv_c, w = y * y;
  const float h = w * fmaf(w, fmaf(w, fmaf(w, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f);
  return fabsf(y) <= 0.25f ? fmaf(u, h, u) : sh_cap_far(u, c, k);
}

// Logits of one lane's row of a tile in the log2 domain, with softcap and
// ALiBi: x_i = log2e cap(scale s_i) + ls (c_i - (row_end - 1)), where c_i <=
// row_end - 1 for every cell that counts.  The softcap is the odd Taylor
// series of c tanh(u / c) through u^9 in the raw product s (coefficients with
// scale and log2(e) folded in) where every |u| of the warp is at most 0.4 c --
// truncation below 3.7e-7 c.  Elsewhere, and where a coefficient would not be
// a normal float (softcaps beyond about 2300 at head dim 128): sh_cap_far for c
// <= 256, where its error is 6e-5 at most, an eighth of an f16 weight's rounding
// step, and sh_cap beyond.  (Five groups at D 64 with c = 1, where every tile
// goes there: 241 us, with sh_cap for all c 285 us.)
__device__ __forceinline__ void sh_transform(const SharedPlan& sp, float* x, float ls, float off) {
  if (sp.p.d.lg.softcap > 0.f) {
    float sm = 0.f;
#pragma unroll
    for (int i = 0; i < kShCells; i += 2) sm = fmax3(sm, fabsf(x[i]), fabsf(x[i + 1]));
    const bool poly = sp.s_lim > 0.f && __all_sync(0xffffffffu, sm <= sp.s_lim);
    if (poly) {
      const float2 C9 = f2(sp.c9), C7 = f2(sp.c7), C5 = f2(sp.c5), C3 = f2(sp.c3), C1 = f2(sp.scale2);
#pragma unroll
      for (int i = 0; i < kShCells; i += 2) {
        const float2 s = f2(x[i], x[i + 1]);
        const float2 w = mul2(s, s);
        const float2 h = fma2(w, fma2(w, fma2(w, fma2(w, C9, C7), C5), C3), C1);
        const float2 y = mul2(s, h);
        x[i] = y.x;
        x[i + 1] = y.y;
      }
    } else {
      const float c = sp.p.d.lg.softcap, scale = sp.p.d.lg.scale;
      const float inv_c = fminf(1.f / c, 3.0e38f), k = fminf(2.f * kLog2e / c, 3.0e38f);
      if (c <= 256.f) {
#pragma unroll
        for (int i = 0; i < kShCells; ++i) x[i] = sh_cap_far(x[i] * scale, c, k) * kLog2e;
      } else {
#pragma unroll
        for (int i = 0; i < kShCells; ++i) x[i] = sh_cap(x[i] * scale, c, inv_c, k) * kLog2e;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kShCells; ++i) x[i] *= sp.scale2;
  }
  if (sp.p.d.lg.slopes) {
#pragma unroll
    for (int i = 0; i < kShCells; ++i) x[i] += fmaf(ls, (float)i, off);
  }
}

// P V of one lane's row on the CUDA cores, over its visible cells [a, b) of
// the tile: O = O * factor + sum_c P[c] V[c] in tensor memory, P read back from
// the first 64 columns of the slot's S region.
template <typename KT, int D>
__device__ __noinline__ void sh_pv_cuda_cores(uint32_t tP, int a, int b, const unsigned char* Vs, uint32_t tO,
                                              bool first, float factor) {
  using L = ShLayout<D>;
#pragma unroll 1
  for (int ch = 0; ch < D / 32; ++ch) {
    float o[32];
    uint32_t ou[32];
    tmem_ld32(tO + ch * 32, ou);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = first ? 0.f : __uint_as_float(ou[e]) * factor;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      uint32_t pw[32];
      __syncwarp();   // the lanes' cell loops end at different places
      tmem_ld32(tP + half * 32, pw);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 64; ++k) {
        const int c = half * 64 + k;
        if (c < a || c >= b) continue;
        const float pc = sh_widen<KT>((k & 1) ? pw[k >> 1] >> 16 : pw[k >> 1] & 0xffffu);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int d = ch * 32 + q * 8;
          float v[8];
          unpack_vec<KT>(*reinterpret_cast<const uint4*>(Vs + (d >> 6) * L::BOX + c * 128 +
                                                         ((((d & 63) >> 3) ^ (c & 7)) << 4)), v);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[q * 8 + e] = fmaf(pc, v[e], o[q * 8 + e]);
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 32; ++e) ou[e] = __float_as_uint(o[e]);
    tmem_st32(tO + ch * 32, ou);
    tmem_wait_st();
  }
}

// 8 floats to a 32-byte aligned address: a whole sector per lane.
__device__ __forceinline__ void st_global_v8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
}

// 32 consecutive output values starting at element i0.
__device__ __forceinline__ void sh_store32(const OutSpec& o, int64_t i0, const float* v, bool vec) {
  if (vec && o.type == ATTN_F32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(o.out) + i0);
#pragma unroll
    for (int k = 0; k < 8; ++k) dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  } else if (vec) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.out) + i0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = o.type == ATTN_BF16 ? sh_pack<__nv_bfloat16>(v[8 * k + 2 * e], v[8 * k + 2 * e + 1])
                                   : sh_pack<__half>(v[8 * k + 2 * e], v[8 * k + 2 * e + 1]);
      dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) store_from_float(o.out, i0 + e, o.type, v[e]);
  }
}

// The softmax warpgroup of a slot.  PLAIN: no softcap, no ALiBi, scale > 0.
template <typename KT, int D, bool PLAIN>
__device__ __forceinline__ void sh_softmax(const SharedPlan& sp, PieceCursor cur, unsigned char* sm, const ShBars& B,
                                           volatile int* abort_flag, volatile int* bad_flag, uint32_t tmem, int slot,
                                           int quarter, int lane, int run) {
  using L = ShLayout<D>;
  int* status = sp.p.d.status;
  const int t = quarter * 32 + lane, G = sp.p.d.G, Hq = sp.p.d.Hq;
  const int row_l = t / G, head_l = t - row_l * G;
  const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
  const uint32_t tS = lane_base + (uint32_t)slot * 128u, tO = lane_base + 256u + (uint32_t)slot * D;
  float2* ml_sh = reinterpret_cast<float2*>(sm + L::OFF_ML);
  uint32_t n_s = 0, n_done = 0, n_merge = 0;   // phases used of s_full, pv_done and the merge barriers
  int64_t vbase = 0;                            // V tiles of the pieces before this one
  Piece pc;
  while (cur.next(&pc)) {
    const bool pair = pc.b.w == 2 || L::NSLOT == 1;
    const int n = pc.i1 - pc.i0, step = pair ? 1 : 2;
    // this lane's row and its visible cells [a, e) of the shared part; lanes
    // without a row see everything (they compute on zeros or another block's
    // rows and store nothing)
    const int j = (pair ? slot * sp.rpt : 0) + row_l;
    const bool rvalid = row_l < sp.rpt && j < pc.b.n_rows;
    const int r = pc.b.row0 + j, h = pc.g * G + head_l;
    int a = 0, e = 0x7fffffff, raw_end = 1;
    bool own = false;
    if (rvalid) {
      const PagedRow row = paged_row(sp.p, r);
      a = row.begin;
      e = max(min(row.end, pc.b.len), a);
      raw_end = row.raw_end;
      own = sp.p.d.row_tiles[r + 1] > sp.p.d.row_tiles[r];
    }
    const bool idle = !__any_sync(0xffffffffu, rvalid);   // a warp of no rows only keeps step
    const float ls = (!PLAIN && sp.p.d.lg.slopes && rvalid) ? __ldg(sp.p.d.lg.slopes + h) * kLog2e : 0.f;

    float m = neg_inf(), l = 0.f;   // running maximum (log2 domain) and sum
    bool ok = true, has = false;
    for (int i = pair ? 0 : slot; i < n; i += step) {
      const int c0 = pc.kt(pc.i0 + i) * kShCells;
      const bool first = !has;
      has = true;
      if (!sh_wait_warp(&B.s_full[slot], n_s & 1u, status, abort_flag)) { ok = false; break; }
      ++n_s;
      tc_fence_after();
      if (idle) {
        tc_fence_before();
        mbar_arrive(&B.p_full[slot]);
        continue;
      }
      const int va = max(a - c0, 0), vb = min(e - c0, kShCells);   // visible cells of this tile: [va, vb)
      float x[kShCells];
      {
        uint32_t* raw = reinterpret_cast<uint32_t*>(x);
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, raw + q * 32);
        tmem_wait_ld();
      }
      if (!PLAIN) sh_transform(sp, x, ls, ls * (float)(c0 - (raw_end - 1)));
      if (!__all_sync(0xffffffffu, va == 0 && vb == kShCells)) {
#pragma unroll
        for (int q = 0; q < kShCells; ++q) x[q] = (q >= va && q < vb) ? x[q] : neg_inf();
      }
      const float mt = sh_max128(x) * (PLAIN ? sp.scale2 : 1.f);
      // lazy rescaling: the maximum moves only when it grows by more than 8
      // (a factor of 2^8), so weights stay below 256 and O is rescaled rarely
      const bool need = !(mt <= m + 8.f);   // NaN compares false: a NaN maximum always rescales
      float factor = 1.f;
      if (need) {
        const float mn = fmax_nan(m, mt);
        factor = m == neg_inf() ? 0.f : ex2(m - mn);
        l *= factor;
        m = mn;
      }
      const float2 E = f2(m == neg_inf() ? 0.f : -m), SC = f2(sp.scale2);
      uint32_t pk[kShCells / 2];
      float2 acc[4] = {f2(0.f), f2(0.f), f2(0.f), f2(0.f)};
#pragma unroll
      for (int q = 0; q < kShCells; q += 2) {
        const float2 y = PLAIN ? fma2(f2(x[q], x[q + 1]), SC, E) : add2(f2(x[q], x[q + 1]), E);
        const float p0 = ex2(y.x), p1 = ex2(y.y);
        acc[(q >> 1) & 3] = add2(acc[(q >> 1) & 3], f2(p0, p1));
        pk[q / 2] = sh_pack<KT>(p0, p1);
      }
      const float2 s2 = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
      l += s2.x + s2.y;

      // A tile that hides cells from some row of the slot (every warp of the
      // slot decides alike): zero the V rows outside the block's range, and
      // look for values that a weight of 0 must not meet.
      bool bad = false;
      const int64_t vt = vbase + i;
      unsigned char* Vs = sm + L::OFF_V + ring_stage<L::NV>(vt) * L::TILE;
      if (pc.b.clo[slot] > c0 || pc.b.chi[slot] < c0 + kShCells) {
        if (!sh_wait_warp(&B.v_full[ring_stage<L::NV>(vt)], ring_phase<L::NV>(vt), status, abort_flag)) {
          ok = false;
          break;
        }
        const int z0 = pc.b.lo - c0, z1 = pc.b.hi - c0;   // cells that some row of the block sees
        for (int u = lane; u < kShCells * (D / 8); u += 32) {
          const int c = u & (kShCells - 1), ch = u / kShCells;
          uint4* at = reinterpret_cast<uint4*>(Vs + (ch >> 3) * L::BOX + c * 128 + ((ch & 7) << 4));
          if (c < z0 || c >= z1) *at = make_uint4(0u, 0u, 0u, 0u);
          else bad |= sh_non_finite<KT>(*at);
        }
        fence_async_smem();   // the zeros, before the tensor core reads V
        bad = __any_sync(0xffffffffu, bad);
      }
      // P V of the previous tile of this slot is complete: the tensor core
      // issued it before this tile's S, and S's completion covers every MMA
      // issued before it.
      if (!first && !bad && __any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          tmem_ld32(tO + ch * 32, o);
          tmem_wait_ld();
          const float2 F = f2(factor);
#pragma unroll
          for (int q = 0; q < 32; q += 2) {
            const float2 v = mul2(f2(__uint_as_float(o[q]), __uint_as_float(o[q + 1])), F);
            o[q] = __float_as_uint(v.x);
            o[q + 1] = __float_as_uint(v.y);
          }
          tmem_st32(tO + ch * 32, o);
          tmem_wait_st();
        }
      }
      // P into the first 64 columns of this slot's S region (S is read)
      __syncwarp();
      tmem_st32(tS, pk);
      tmem_st32(tS + 32, pk + 32);
      tmem_wait_st();
      if (bad) sh_pv_cuda_cores<KT, D>(tS, va, vb, Vs, tO, first, factor);
      if (t == 0) bad_flag[slot] = bad ? 1 : 0;   // warp 0 of a slot holds rows whenever any warp does
      tc_fence_before();
      mbar_arrive(&B.p_full[slot]);
    }
    vbase += n;
    if (!ok) return;
    if (has) {
      if (!sh_wait_warp(&B.pv_done[slot], n_done & 1u, status, abort_flag)) return;
      ++n_done;
      tc_fence_after();
    }
    // a block of one tile of rows: slot 1's tiles join slot 0's state
    const bool merge = !pair && n > 1;
    float f0 = 1.f, f1 = 0.f;
    if (merge && slot == 1) {
      ml_sh[t] = make_float2(m, l);
      tc_fence_before();
      mbar_arrive(B.merge_full);
      if (!sh_wait_warp(B.merge_empty, n_merge & 1u, status, abort_flag)) return;
      ++n_merge;
      tc_fence_after();
      continue;
    }
    if (!has) continue;
    if (merge) {
      if (!sh_wait_warp(B.merge_full, n_merge & 1u, status, abort_flag)) return;
      ++n_merge;
      tc_fence_after();
      const float2 ml1 = ml_sh[t];
      const float M = fmax_nan(m, ml1.x);
      f0 = m == neg_inf() ? 0.f : ex2(m - M);
      f1 = ml1.x == neg_inf() ? 0.f : ex2(ml1.x - M);
      l = l * f0 + ml1.y * f1;
      m = M;
    }
    const bool fin = pc.whole() && !own;
    float f = 1.f;
    bool is_nan = false, is_zero = m == neg_inf();   // no cell seen: O may hold anything
    if (fin && !idle) {
      const float sigma = (sp.p.d.lg.sinks && rvalid) ? __ldg(sp.p.d.lg.sinks + h) * kLog2e : neg_inf();
      const float Mf = fmax_nan(m, sigma);
      is_nan = isnan(Mf) || Mf == -neg_inf();
      if (!is_nan && Mf != neg_inf()) {
        const float fo = ex2(m - Mf);
        f = fo / (l * fo + ex2(sigma - Mf));
      }
    }
    const int64_t rec = pc.i0 == 0 ? (int64_t)r * Hq + h
                                   : (int64_t)sp.p.d.R * Hq + (int64_t)run * 256 + (pair ? slot * 128 : 0) + t;
    if (!fin && rvalid) {
      sp.rec_ml[2 * rec] = m * 0.6931471805599453f;   // natural logarithms, as the combine folds
      sp.rec_ml[2 * rec + 1] = l;
    }
    const int64_t ob = (int64_t)r * sp.p.d.out.sr + (int64_t)h * sp.p.d.out.sh;
    if (!idle) {
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o0[32];
        float v[32];
        __syncwarp();   // lanes without a row skip the stores
        tmem_ld32(tO + ch * 32, o0);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 32; ++q) v[q] = __uint_as_float(o0[q]) * f0;
        if (merge) {   // (only slot 0 gets here; a slot that saw nothing has a weight of 0 and any O)
          tmem_ld32(tO + (uint32_t)D + ch * 32, o0);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 32; ++q)
            v[q] = (f0 == 0.f ? 0.f : v[q]) + (f1 == 0.f ? 0.f : __uint_as_float(o0[q]) * f1);
        }
#pragma unroll
        for (int q = 0; q < 32; ++q) v[q] = is_nan ? qnan() : is_zero ? 0.f : v[q] * f;
        if (!rvalid) continue;
        if (fin) {
          sh_store32(sp.p.d.out, ob + ch * 32, v, sp.out_vec != 0);
        } else {
          float* dst = sp.rec_o + rec * D + ch * 32;
#pragma unroll
          for (int q = 0; q < 32; q += 8) st_global_v8(dst + q, v + q);
        }
      }
    }
    tc_fence_before();
    if (merge) mbar_arrive(B.merge_empty);
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------

// S (TMEM, 128 x 128 f32) = Q . K^T: both K-major tiles of D / 64 boxes.
template <int D>
__device__ __forceinline__ void sh_issue_s(uint32_t d_tmem, uint64_t q_desc, uint64_t k_desc, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t off = (uint64_t)(((kk >> 2) * ShLayout<D>::BOX + (kk & 3) * 32) >> 4);
    umma_ss(d_tmem, q_desc + off, k_desc + off, idesc, kk > 0 ? 1u : 0u);
  }
}
// O (TMEM, 128 x D f32) (+)= P . V, P in tensor memory (16 cells = 8 columns
// per MMA), V MN-major: 8-cell groups 1024 bytes apart, boxes BOX apart.
template <int D>
__device__ __forceinline__ void sh_issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t v_desc, uint32_t idesc,
                                            bool accumulate) {
#pragma unroll
  for (int kk = 0; kk < kShCells / 16; ++kk)
    umma_ts(d_tmem, p_tmem + (uint32_t)kk * 8u, v_desc + (uint64_t)((kk * 2048) >> 4), idesc,
            (accumulate || kk > 0) ? 1u : 0u);
}

// After a wait that ran out: every (row, query head) of the run's pieces gets a
// NaN record (the combine makes it NaN), or a NaN output where its piece would
// have finished it.  By the 256 threads of the softmax warps.
template <int D>
__device__ __noinline__ void sh_poison(const SharedPlan& sp, int run) {
  const int G = sp.p.d.G, Hq = sp.p.d.Hq;
  PieceCursor cur = run_cursor(sp, run);
  Piece pc;
  while (cur.next(&pc)) {
    for (int u = (int)threadIdx.x - 128; u < pc.b.n_rows * G; u += 256) {
      const int j = u / G, head_l = u - j * G, r = pc.b.row0 + j, h = pc.g * G + head_l;
      const int slot = j >= sp.rpt ? 1 : 0;   // (only a block of two tiles of rows has a second one)
      const bool own = sp.p.d.row_tiles[r + 1] > sp.p.d.row_tiles[r];
      if (pc.whole() && !own) {
        const int64_t ob = (int64_t)r * sp.p.d.out.sr + (int64_t)h * sp.p.d.out.sh;
        for (int d = 0; d < D; ++d) store_from_float(sp.p.d.out.out, ob + d, sp.p.d.out.type, qnan());
      } else {
        const int64_t rec = pc.i0 == 0 ? (int64_t)r * Hq + h
                                       : (int64_t)sp.p.d.R * Hq + (int64_t)run * 256 + slot * 128 +
                                             (j - slot * sp.rpt) * G + head_l;
        sp.rec_ml[2 * rec] = qnan();
        sp.rec_ml[2 * rec + 1] = qnan();
      }
    }
  }
}

template <typename KT, int D, bool PLAIN>
__global__ void __launch_bounds__(ShLayout<D>::THREADS, 1)
shared_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ SharedPlan sp) {
  using L = ShLayout<D>;
  constexpr int NK = L::NK, NV = L::NV;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = align1024(smem_raw);
  const ShBars B = sh_bars<D>(sm);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::OFF_MISC + 4);
  volatile int* bad_flag = reinterpret_cast<volatile int*>(sm + L::OFF_MISC + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, run = blockIdx.x;
  int* status = sp.p.d.status;
  const int G = sp.p.d.G;

  if (threadIdx.x == 0) {
    mbar_init(B.q_full, 1);
    mbar_init(B.q_empty, 1);
    for (int s = 0; s < NK; ++s) { mbar_init(&B.k_full[s], 1); mbar_init(&B.k_empty[s], 1); }
    for (int s = 0; s < NV; ++s) { mbar_init(&B.v_full[s], 1); mbar_init(&B.v_empty[s], 1); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&B.s_full[s], 1);
      mbar_init(&B.p_full[s], kShRows);
      mbar_init(&B.pv_done[s], 1);
      bad_flag[s] = 0;
    }
    mbar_init(B.merge_full, kShRows);
    mbar_init(B.merge_empty, kShRows);
    mbar_init(B.mma_done, 1);
    mbar_init(B.never, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, L::TMEM_COLS);
  {
    // lanes that hold no row: zero those rows of the Q tiles once (the loads
    // write the others), so that their S stays finite
    const int used = sp.rpt * G, spare = kShRows - used;
    for (int i = threadIdx.x; i < L::NSLOT * spare * (D / 8); i += L::THREADS) {
      const int row = used + i % spare, c = i / spare, ch = c % (D / 8), s = c / (D / 8);
      *reinterpret_cast<uint4*>(sm + L::OFF_Q + s * L::TILE + (ch >> 3) * L::BOX + row * 128 + (ch & 7) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_smem();   // visible to the tensor core
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait_prior_grid();   // the plan

  PieceCursor cur = run_cursor(sp, run);

  if (warp >= 4) {
    // ---- softmax warpgroups ----
    setmaxnreg_inc<L::HIGH_REGS>();
    const int slot = (warp >> 2) - 1;
    // (the test of the bounded waits: nothing arrives at this barrier)
    const bool go = sp.stall_ns == 0 || sh_wait_warp(B.never, 0, status, abort_flag, sp.stall_ns);
    if (go && slot < L::NSLOT)
      sh_softmax<KT, D, PLAIN>(sp, cur, sm, B, abort_flag, bad_flag, tmem, slot, warp & 3, lane, run);
  } else {
    setmaxnreg_dec<L::LOW_REGS>();
    if (warp == 0) {
      // ---- TMA producer (lane q fetches box q of a tile) ----
      const uint64_t pol = policy_evict_last();
      const int C = sp.box_cells, boxes = kShCells / C;
      const uint32_t q_bytes = (uint32_t)(sp.rpt * G) * (uint32_t)(D * 2);
      int64_t nK = 0, nV = 0, nQ = 0;
      Piece pc;
      bool ok = true;
      while (ok && cur.next(&pc)) {
        const int slots = pc.b.w == 2 ? 2 : 1;
        if (nQ > 0 && !sh_wait_warp(B.q_empty, (uint32_t)((nQ - 1) & 1), status, abort_flag)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(B.q_full, (uint32_t)slots * q_bytes);
          for (int s = 0; s < slots; ++s)
#pragma unroll
            for (int bx = 0; bx < D / 64; ++bx)
              tma_load_3d(sm + L::OFF_Q + s * L::TILE + bx * L::BOX, &tmQ, B.q_full, bx * 64, pc.g * G,
                          pc.b.row0 + s * sp.rpt, pol);
        }
        ++nQ;
        PagedRow row;
        row.table = pc.b.table;
        for (int i = pc.i0; i < pc.i1; ++i) {
          // the tile's pages (boxes outside the block's range read zeros)
          const int c = pc.kt(i) * kShCells + lane * C;
          int page = sp.p.n_pages, off = 0;
          if (lane < boxes && c < pc.b.hi && c + C > pc.b.lo) {
            page = paged_page(sp.p, row, c);
            off = c % sp.p.P;
          }
          const int sk = ring_stage<NK>(nK);
          if (nK >= NK && !sh_wait_warp(&B.k_empty[sk], ring_phase<NK>(nK - NK), status, abort_flag)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&B.k_full[sk], (uint32_t)L::TILE);
          __syncwarp();
          if (lane < boxes)
#pragma unroll
            for (int bx = 0; bx < D / 64; ++bx)
              tma_load_4d(sm + L::OFF_K + sk * L::TILE + bx * L::BOX + lane * C * 128, &tmK, &B.k_full[sk], bx * 64,
                          pc.g, off, page, pol);
          ++nK;
          const int sv = ring_stage<NV>(nV);
          if (nV >= NV && !sh_wait_warp(&B.v_empty[sv], ring_phase<NV>(nV - NV), status, abort_flag)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&B.v_full[sv], (uint32_t)L::TILE);
          __syncwarp();
          if (lane < boxes)
#pragma unroll
            for (int bx = 0; bx < D / 64; ++bx)
              tma_load_4d(sm + L::OFF_V + sv * L::TILE + bx * L::BOX + lane * C * 128, &tmV, &B.v_full[sv], bx * 64,
                          pc.g, off, page, pol);
          ++nV;
        }
      }
      // leave no copy in flight (completed loads return at once)
      for (int64_t k = nK > NK ? nK - NK : 0; k < nK; ++k)
        mbar_wait_bounded(&B.k_full[ring_stage<NK>(k)], ring_phase<NK>(k), nullptr);
      for (int64_t k = nV > NV ? nV - NV : 0; k < nV; ++k)
        mbar_wait_bounded(&B.v_full[ring_stage<NV>(k)], ring_phase<NV>(k), nullptr);
      if (nQ > 0) mbar_wait_bounded(B.q_full, (uint32_t)((nQ - 1) & 1), nullptr);
    } else if (warp == 1) {
      // ---- MMA issuer ----
      if (lane == 0) {
        constexpr int bf = Storage<KT>::kDtype == ATTN_BF16 ? 1 : 0;
        constexpr uint32_t idS = umma_idesc_f16(kShRows, kShCells, bf, 0, 0);
        constexpr uint32_t idO = umma_idesc_f16(kShRows, D, bf, 0, 1);
        const uint64_t q_desc = umma_desc_sw128(smem_u32(sm + L::OFF_Q), 16, 1024);
        const uint64_t k_desc = umma_desc_sw128(smem_u32(sm + L::OFF_K), 16, 1024);
        const uint64_t v_desc = umma_desc_sw128(smem_u32(sm + L::OFF_V), L::BOX, 1024);
        constexpr uint64_t kTileDesc = (uint64_t)(L::TILE >> 4);
        RingPos<NK> ck;
        RingPos<NV> cv;
        int64_t nQ = 0;
        uint32_t n_p0 = 0, n_p1 = 0;
        bool ok = true;
        Piece pc;
        // S of the next K tile for slots [s0, s1) (Q tile = slot, or 0 for a
        // block of one tile of rows), then that K stage is free
        auto wait_k = [&]() {
          if (!sh_wait(&B.k_full[ck.stage], ck.phase, status, abort_flag)) return false;
          tc_fence_after();
          return true;
        };
        auto issue_s = [&](int s, int q) {
          sh_issue_s<D>(tmem + (uint32_t)s * 128u, q_desc + (uint64_t)q * kTileDesc,
                        k_desc + (uint64_t)ck.stage * kTileDesc, idS);
          umma_commit(&B.s_full[s]);
        };
        auto k_done = [&]() {
          umma_commit(&B.k_empty[ck.stage]);
          ck.next();
        };
        auto wait_p = [&](int s) {
          const bool w = sh_wait(&B.p_full[s], (s ? n_p1 : n_p0) & 1u, status, abort_flag);
          if (s) ++n_p1;
          else ++n_p0;
          tc_fence_after();
          return w;
        };
        auto issue_pv = [&](int s, bool acc) {
          if (bad_flag[s] == 0)
            sh_issue_pv<D>(tmem + 256u + (uint32_t)s * D, tmem + (uint32_t)s * 128u,
                           v_desc + (uint64_t)cv.stage * kTileDesc, idO, acc);
        };
        auto wait_v = [&]() {
          const bool w = sh_wait(&B.v_full[cv.stage], cv.phase, status, abort_flag);
          tc_fence_after();
          return w;
        };
        while (ok && cur.next(&pc)) {
          const int n = pc.i1 - pc.i0;
          if (!sh_wait(B.q_full, (uint32_t)(nQ & 1), status, abort_flag)) break;
          ++nQ;
          tc_fence_after();
          if (pc.b.w == 2 || L::NSLOT == 1) {
            const int slots = pc.b.w == 2 ? 2 : 1;
            if (!wait_k()) break;
            for (int s = 0; s < slots; ++s) issue_s(s, s);
            k_done();
            for (int i = 0; ok && i < n; ++i) {
              const bool more = i + 1 < n;
              if (!more) umma_commit(B.q_empty);   // every S of the piece is issued
              if (more && !wait_k()) { ok = false; break; }
              for (int s = 0; s < slots; ++s) {
                if ((s == 0 && !wait_v()) || !wait_p(s)) { ok = false; break; }
                issue_pv(s, i > 0);
                if (!more) {
                  umma_commit(&B.pv_done[s]);
                } else {
                  issue_s(s, s);
                  if (s == slots - 1) k_done();
                }
              }
              if (!ok) break;
              umma_commit(&B.v_empty[cv.stage]);
              cv.next();
            }
          } else {
            for (int i = 0; ok && i < min(n, 2); ++i) {
              if (!wait_k()) { ok = false; break; }
              issue_s(i, 0);
              k_done();
            }
            if (ok && n <= 2) umma_commit(B.q_empty);
            for (int i = 0; ok && i < n; ++i) {
              const int s = i & 1;
              if (!wait_v() || !wait_p(s)) { ok = false; break; }
              issue_pv(s, i >= 2);
              umma_commit(&B.v_empty[cv.stage]);
              cv.next();
              if (i + 2 < n) {
                if (!wait_k()) { ok = false; break; }
                issue_s(s, 0);
                k_done();
                if (i + 3 == n) umma_commit(B.q_empty);
              } else {
                umma_commit(&B.pv_done[s]);
              }
            }
          }
        }
        umma_commit(B.mma_done);   // arrives once every MMA issued above has retired
      }
    }   // warps 2 and 3 have no role
  }

  tc_fence_before();
  __syncthreads();
  if (warp >= 4 && *abort_flag) sh_poison<D>(sp, run);
  if (warp == 1) {
    tc_fence_after();
    mbar_wait_bounded(B.mma_done, 0, status);
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

template <typename KT, int D, bool PLAIN>
cudaError_t launch_sh_t(const SharedPlan& sp, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                        cudaStream_t stream) {
  auto kern = shared_kernel<KT, D, PLAIN>;
  using L = ShLayout<D>;
  static std::atomic<unsigned long long> smem_set{0ull};
  cudaError_t e = set_smem_limit_once(smem_set, kern, L::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<unsigned long long> plan_set{0ull};
  if ((e = set_smem_limit_once(plan_set, shared_plan_kernel, (int)sizeof(PlanShared))) != cudaSuccess) return e;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(sp.p.d.R <= 256 && sp.n_groups < 256 ? 256 : kPlanThreads);
  cfg.dynamicSmemBytes = sp.max_blk <= kPlanBlocks ? sizeof(PlanShared) : 32 * sizeof(long long);
  if ((e = cudaLaunchKernelEx(&cfg, shared_plan_kernel, sp)) != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)sp.W);
  cfg.blockDim = dim3(L::THREADS);
  cfg.dynamicSmemBytes = L::SMEM;
  return cudaLaunchKernelEx(&cfg, kern, tmQ, tmK, tmV, sp);
}

template <typename KT, int D>
cudaError_t launch_sh_d(const SharedPlan& sp, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                        cudaStream_t stream) {
  return sp.plain ? launch_sh_t<KT, D, true>(sp, tmQ, tmK, tmV, stream)
                  : launch_sh_t<KT, D, false>(sp, tmQ, tmK, tmV, stream);
}

}  // namespace

cudaError_t launch_shared(const SharedPlan& sp, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                          cudaStream_t stream) {
  const bool bf = sp.p.d.kv_type == ATTN_BF16;
  switch (sp.p.d.D) {
    case 64: return bf ? launch_sh_d<__nv_bfloat16, 64>(sp, tmQ, tmK, tmV, stream)
                       : launch_sh_d<__half, 64>(sp, tmQ, tmK, tmV, stream);
    case 128: return bf ? launch_sh_d<__nv_bfloat16, 128>(sp, tmQ, tmK, tmV, stream)
                        : launch_sh_d<__half, 128>(sp, tmQ, tmK, tmV, stream);
    default: return bf ? launch_sh_d<__nv_bfloat16, 256>(sp, tmQ, tmK, tmV, stream)
                       : launch_sh_d<__half, 256>(sp, tmQ, tmK, tmV, stream);
  }
}

}  // namespace attn
