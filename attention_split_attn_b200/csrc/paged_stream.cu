// paged_stream.cu -- balanced persistent split-K decode over a paged cache
// (attn_decode_paged, and the rows' own cells of attn_decode_shared): the
// scheme of decode_stream.cu with its tiles cut at multiples of 16 cells, so
// that a tile lies in one page (page sizes are multiples of 16), and found
// through the row's block table.
//
// The flattened (row, KV head, 16-cell tile) space, the equal runs of the W
// resident warps, the record slots and the combine are those of
// decode_stream.cu.  What a page adds per tile is its id: the warp's lanes
// read the ids of the next 32 tiles of a row at once, so a run pays the table's
// load latency once per 32 tiles and not per tile; the tile's TMA box is
// {128 bytes, 1 head, 16 cells, 1 page} of a 4-D map over [page][cell][head][D].
// An id outside the pool is replaced by n_pages, where the TMA reads zeros.
// 16 rows of 1024 to 8192 cells (302 MB, 8 KV heads, D 128, bf16): 47.5 us, 6.4
// TB/s; one row of 130857 cells (536 MB): 80 to 86 us.
#include <algorithm>

#include "common.cuh"
#include "decode_tile.cuh"
#include "decode_tile8.cuh"
#include "internal.h"
#include "mma.cuh"
#include "paged.cuh"
#include "quant.cuh"

namespace attn {

namespace {

constexpr int kInlineRows = 64;   // up to this many rows every warp computes the tile prefix itself

template <typename KT, int D, int NH>
struct PsTraits {
  using State = WarpTileState<KT, D, NH>;
  static constexpr int ES = 2;
};
template <int D, int NH>
struct PsTraits<e4m3_code, D, NH> {
  using State = WarpTileState8<e4m3_code, D, NH>;
  static constexpr int ES = 1;
};
template <int D, int NH>
struct PsTraits<i8_code, D, NH> {
  using State = WarpTileState8<i8_code, D, NH>;
  static constexpr int ES = 1;
};

template <int D, int ES>
struct PsRing {
  static constexpr int NS = 2;                       // ring stages per warp
  static constexpr int TILE = kWarpTile * D * ES;    // K (or V) of one tile
  static constexpr int STAGE = 2 * TILE;
  static constexpr int BAR_OFF = NS * STAGE;         // a barrier per stage, and one that nothing arrives at
  static constexpr int SLOT_OFF = BAR_OFF + (NS + 1) * 8;   // first pool slot of the last 2 NS tiles issued
  static constexpr int RT_OFF = SLOT_OFF + 2 * NS * 4;   // inline row tile prefix [kInlineRows + 1]
  static constexpr int TOTAL = RT_OFF + (kInlineRows + 1) * 8 + 1024;   // + alignment slack for the swizzle
};

// row_tiles[r] = sum over r' < r of its tile count; row_tiles[R] = total.
__global__ void __launch_bounds__(1024) paged_plan_kernel(const PagedPlan p) {
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  __shared__ long long wsum[32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  long long carry = 0;
  for (int base = 0; base < p.d.R; base += 1024) {
    const int r = base + tid;
    const long long n = r < p.d.R ? paged_row(p, r).tiles() : 0;
    long long x = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) wsum[wid] = x;
    __syncthreads();
    if (wid == 0) {
      long long v = wsum[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += y;
      }
      wsum[lane] = v;
    }
    __syncthreads();
    const long long excl = x - n + (wid > 0 ? wsum[wid - 1] : 0);
    if (r < p.d.R) p.d.row_tiles[r] = carry + excl;
    carry += wsum[31];
    __syncthreads();
  }
  if (tid == 0) p.d.row_tiles[p.d.R] = carry;
}

// Position in the flattened tile space: row r, KV head g, tile j of nt.
struct PsCursor {
  int r, g;
  int64_t j, nt;
  PagedRow row;
};

__device__ __forceinline__ void ps_load_row(const PagedPlan& p, const int64_t* row_tiles, PsCursor& c) {
  c.nt = row_tiles[c.r + 1] - row_tiles[c.r];
  c.row = paged_row(p, c.r);
}

__device__ __forceinline__ void ps_next(const PagedPlan& p, const int64_t* row_tiles, PsCursor& c) {
  if (++c.j < c.nt) return;
  c.j = 0;
  if (++c.g < p.d.Hkv) return;
  c.g = 0;
  do {
    ++c.r;
    ps_load_row(p, row_tiles, c);
  } while (c.nt == 0 && c.r + 1 < p.d.R);
}

template <typename KT, int D, int NH>
__global__ void __launch_bounds__(32)
paged_stream_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const PagedPlan p) {
  using Tr = PsTraits<KT, D, NH>;
  using Ring = PsRing<D, Tr::ES>;
  constexpr int NS = Ring::NS;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Ring::BAR_OFF);
  volatile int32_t* slots = reinterpret_cast<volatile int32_t*>(smem + Ring::SLOT_OFF);
  const int lane = threadIdx.x;
  if (lane == 0) {
    for (int i = 0; i <= NS; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int64_t* row_tiles = p.d.row_tiles;
  if (p.d.plan_inline) {
    int64_t* rt = reinterpret_cast<int64_t*>(smem + Ring::RT_OFF);
    int64_t carry = 0;
    for (int base = 0; base < p.d.R; base += 32) {
      const int r = base + lane;
      const int64_t n = r < p.d.R ? paged_row(p, r).tiles() : 0;
      int64_t x = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      if (r < p.d.R) rt[r] = carry + x - n;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) rt[p.d.R] = carry;
    __syncwarp();
    row_tiles = rt;
    if (blockIdx.x == 0)   // the combine reads the prefix from the workspace
      for (int r = lane; r <= p.d.R; r += 32) p.d.row_tiles[r] = row_tiles[r];
  }

  const int64_t W = p.d.W, Hkv = p.d.Hkv;
  const int64_t T = Hkv * row_tiles[p.d.R];
  const int64_t w = blockIdx.x;
  const int64_t t0 = div64(T * w, W), t1 = div64(T * (w + 1), W);
  if (t0 >= t1) return;

  // the row holding tile t0: the last r with Hkv * row_tiles[r] <= t0
  // (32-ary search: each round the lanes probe 32 evenly spaced rows)
  int lo = 0, hi = p.d.R;   // answer in [lo, hi)
  while (hi - lo > 1) {
    const int64_t span = hi - lo;
    const int64_t step = (span + 31) / 32;
    const int64_t probe = lo + lane * step;
    const bool ok = probe < hi && Hkv * row_tiles[probe] <= t0;
    const unsigned m = __ballot_sync(0xffffffffu, ok);
    const int k = 31 - __clz(m);       // lane 0 always qualifies (row_tiles[lo] <= t0)
    lo = (int)(lo + k * step);
    hi = (int)((int64_t)hi < lo + step ? (int64_t)hi : lo + step);
  }
  PsCursor c;
  c.r = lo;
  ps_load_row(p, row_tiles, c);
  {
    const int64_t off = t0 - Hkv * row_tiles[c.r];
    c.g = (int)div64(off, c.nt);
    c.j = off - c.g * c.nt;
  }
  PsCursor ic = c;   // issue cursor, NS tiles ahead (the same in every lane)
  const int64_t n = t1 - t0;
  const uint64_t pol = policy_evict_first();
  int64_t issued = 0;
  // ids of the pages of tiles id_j .. id_j + 31 of row id_r, one per lane
  int32_t ids = -1;
  int id_r = -1;
  int64_t id_j = 0;
  auto issue = [&](int64_t i) {   // tile i of the run, at the issue cursor
    if (ic.r != id_r || ic.j < id_j || ic.j >= id_j + 32) {
      id_r = ic.r;
      id_j = ic.j;
      ids = ic.j + lane < ic.nt ? paged_page(p, ic.row, (int32_t)((ic.row.tile0 + ic.j + lane) * kWarpTile)) : 0;
    }
    const int32_t page = __shfl_sync(0xffffffffu, ids, (int)(ic.j - id_j));
    if (lane == 0) {
      const int32_t c0 = (int32_t)((ic.row.tile0 + ic.j) * kWarpTile), off = c0 % p.P;
      const int stg = (int)(i % NS);
      unsigned char* stage = smem + stg * Ring::STAGE;
      slots[i % (2 * NS)] = page < p.n_pages ? page * p.P + off : -1;
      constexpr int NB = D * Tr::ES / 128, EPB = 128 / Tr::ES;
      mbar_arrive_expect_tx(&full[stg], Ring::STAGE);
#pragma unroll
      for (int sub = 0; sub < NB; ++sub) {
        tma_load_4d(stage + sub * (kWarpTile * 128), &tmK, &full[stg], sub * EPB, ic.g, off, page, pol);
        tma_load_4d(stage + Ring::TILE + sub * (kWarpTile * 128), &tmV, &full[stg], sub * EPB, ic.g, off, page, pol);
      }
    }
    __syncwarp();
  };
  // The issue cursor only advances right before issuing a tile that exists,
  // so it never moves past the last tile of the run.
  for (; issued < (n < NS ? n : (int64_t)NS); ++issued) {
    if (issued > 0) ps_next(p, row_tiles, ic);
    issue(issued);
  }

  auto make_ctx = [&](const PsCursor& cc) {
    RowCtx rc;
    rc.begin = rc.s_begin = cc.row.begin;
    rc.end = rc.s_end = cc.row.end;
    rc.pos_base = 0;
    rc.row_seq = 0;
    rc.row_pos = (int64_t)cc.row.raw_end - 1;
    return rc;
  };
  auto tile_cell = [&](const PsCursor& cc) { return (int)((cc.row.tile0 + cc.j) * kWarpTile); };
  RowCtx rc = make_ctx(c);
  typename Tr::State st;
  st.reset();
  st.init_offsets(lane);
  st.load_q(p.d, c.r, c.g * p.d.G, lane);

  bool aborted = p.stall_ns > 0;   // (the test of the bounded waits)
  if (aborted) stall_bounded(&full[NS], p.stall_ns, p.d.status);
  __syncwarp();
  int64_t k = 0;
  if constexpr (Tr::ES == 1) st.prefetch_slot(p.d, c.g, slots[0], lane);
  for (; k < n && !aborted; ++k) {
    const int stg = (int)(k % NS);
    if constexpr (Tr::ES == 1) {
      st.take_prefetched();
      if (k + 1 < n) {   // the next tile's per-cell scales, a tile ahead
        const int g = c.j + 1 < c.nt ? c.g : (c.g + 1 < Hkv ? c.g + 1 : 0);
        st.prefetch_slot(p.d, g, slots[(k + 1) % (2 * NS)], lane);
      }
    }
    // (the lanes go on or give up together)
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[stg], (uint32_t)((k / NS) & 1), p.d.status))) {
      aborted = true;
      break;
    }
    unsigned char* stage = smem + stg * Ring::STAGE;
    st.load_tile(stage);
    auto refill = [&]() {
      __syncwarp();
      if (issued < n) {
        // the lanes' shared-memory reads of this stage precede its async refill
        if (lane == 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        ps_next(p, row_tiles, ic);
        issue(issued);
        ++issued;
      }
    };
    if (decltype(st)::kEarlyRelease) refill();
    st.template compute<true>(p.d, rc, c.r, tile_cell(c), false, lane, stage);
    if (!decltype(st)::kEarlyRelease) refill();
    const bool last = (k + 1 == n);
    if (c.j + 1 == c.nt || last) {
      // the pair ends here (or this warp's run does): emit its record
      st.finish_sums();
      const int64_t pair = (int64_t)c.r * Hkv + c.g;
      const int64_t pair_start = Hkv * row_tiles[c.r] + (int64_t)c.g * c.nt;
      const int64_t slot = pair_start >= t0 ? W + pair : w;
      st.write_partial(p.d.part.o, p.d.part.ml, slot, p.d.G, lane, false);
      if (!last) {
        ps_next(p, row_tiles, c);
        rc = make_ctx(c);
        st.reset();
        st.load_q(p.d, c.r, c.g * p.d.G, lane);
      }
    } else {
      ++c.j;
    }
  }
  if (aborted) {
    // poison the record in progress and those of the run's later pairs (the
    // workspace may hold an earlier call's), and leave no copy in flight
    for (;;) {
      const int64_t pair = (int64_t)c.r * Hkv + c.g;
      const int64_t pair_start = Hkv * row_tiles[c.r] + (int64_t)c.g * c.nt;
      st.write_partial(p.d.part.o, p.d.part.ml, pair_start >= t0 ? W + pair : w, p.d.G, lane, true);
      if (pair_start + c.nt >= t1) break;
      c.j = c.nt - 1;
      ps_next(p, row_tiles, c);
    }
    if (lane == 0)
      for (int64_t kk = k; kk < issued; ++kk) mbar_wait_bounded(&full[kk % NS], (uint32_t)((kk / NS) & 1), nullptr);
    __syncwarp();
  }
}

template <typename KT, int D, int NH>
cudaError_t launch_ps_t(const PagedPlan& p, const CUtensorMap& tmK, const CUtensorMap& tmV, cudaStream_t stream) {
  auto kern = paged_stream_kernel<KT, D, NH>;
  using Ring = PsRing<D, PsTraits<KT, D, NH>::ES>;
  static std::atomic<unsigned long long> smem_set{0ull};
  cudaError_t e = set_smem_limit_once(smem_set, kern, Ring::TOTAL);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!p.d.plan_inline && !p.own_lo) {
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    if ((e = cudaLaunchKernelEx(&cfg, paged_plan_kernel, p)) != cudaSuccess) return e;
  }
  cfg.gridDim = dim3((unsigned)p.d.W);
  cfg.blockDim = dim3(32);
  cfg.dynamicSmemBytes = Ring::TOTAL;
  return cudaLaunchKernelEx(&cfg, kern, tmK, tmV, p);
}

template <typename KT>
cudaError_t launch_ps_k(const PagedPlan& p, const CUtensorMap& tmK, const CUtensorMap& tmV, cudaStream_t stream) {
  const bool h16 = p.d.G > 8;
  switch (p.d.D) {
    case 64: return h16 ? launch_ps_t<KT, 64, 16>(p, tmK, tmV, stream) : launch_ps_t<KT, 64, 8>(p, tmK, tmV, stream);
    case 128: return h16 ? launch_ps_t<KT, 128, 16>(p, tmK, tmV, stream) : launch_ps_t<KT, 128, 8>(p, tmK, tmV, stream);
    default: return h16 ? launch_ps_t<KT, 256, 16>(p, tmK, tmV, stream) : launch_ps_t<KT, 256, 8>(p, tmK, tmV, stream);
  }
}

template <typename KT, int D, int NH>
int ps_blocks_per_sm() {
  int n = 0;
  using Ring = PsRing<D, PsTraits<KT, D, NH>::ES>;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, paged_stream_kernel<KT, D, NH>, 32, Ring::TOTAL) !=
          cudaSuccess ||
      n <= 0) {
    cudaGetLastError();
    // no device: the shared-memory bound of a 228 KB SM with 1 KB reserved per CTA
    n = (228 * 1024) / (Ring::TOTAL + 1024);
  }
  return n;
}

template <typename KT>
int ps_blocks_k(int D, bool h16) {
  switch (D) {
    case 64: return h16 ? ps_blocks_per_sm<KT, 64, 16>() : ps_blocks_per_sm<KT, 64, 8>();
    case 128: return h16 ? ps_blocks_per_sm<KT, 128, 16>() : ps_blocks_per_sm<KT, 128, 8>();
    default: return h16 ? ps_blocks_per_sm<KT, 256, 16>() : ps_blocks_per_sm<KT, 256, 8>();
  }
}

}  // namespace

int paged_stream_warps(int kv_type, int D, int G, int sms) {
  int per_sm;
  if (kv_type == ATTN_FP8_E4M3)
    per_sm = D == 128 ? ps_blocks_per_sm<e4m3_code, 128, 8>() : ps_blocks_per_sm<e4m3_code, 256, 8>();
  else if (kv_type == ATTN_I8)
    per_sm = D == 128 ? ps_blocks_per_sm<i8_code, 128, 8>() : ps_blocks_per_sm<i8_code, 256, 8>();
  else
    per_sm = kv_type == ATTN_F16 ? ps_blocks_k<__half>(D, G > 8) : ps_blocks_k<__nv_bfloat16>(D, G > 8);
  return std::max(1, per_sm) * std::max(1, sms);
}

cudaError_t launch_paged_stream(const PagedPlan& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                cudaStream_t stream) {
  if (p.d.kv_type == ATTN_FP8_E4M3)
    return p.d.D == 128 ? launch_ps_t<e4m3_code, 128, 8>(p, tmK, tmV, stream)
                        : launch_ps_t<e4m3_code, 256, 8>(p, tmK, tmV, stream);
  if (p.d.kv_type == ATTN_I8)
    return p.d.D == 128 ? launch_ps_t<i8_code, 128, 8>(p, tmK, tmV, stream)
                        : launch_ps_t<i8_code, 256, 8>(p, tmK, tmV, stream);
  if (p.d.kv_type == ATTN_F16) return launch_ps_k<__half>(p, tmK, tmV, stream);
  return launch_ps_k<__nv_bfloat16>(p, tmK, tmV, stream);
}

}  // namespace attn
