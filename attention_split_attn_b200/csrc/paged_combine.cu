// paged_combine.cu -- folds the split records of every (row, query head) of a
// paged decode: of decode_shared the shared part's home record and the records
// of the runs after it, then of the row's own cells the home record and the
// slots of the warps after it, then the sink (combine.cu's rules: NaN in any
// maximum or in the sink gives NaN, a row that saw nothing is +0).
//
// Bound by the latency of a few dependent loads (the row's place, its records'
// places, the records) and, for one long row, by the number of its records:
// 1776 warps leave 222 of them per (row, KV head) at 8 KV heads, which one warp
// took 35 us to fold.  So
//  * `wpi` warps of a CTA share an item (row, query head) while the items alone
//    would leave the SMs short of warps: warp w takes the records w, w + wpi,
//    ... of each round, and the wpi partial results fold in warp order through
//    shared memory (the same order on every run);
//  * with many items a warp takes `ipw` of them: its lanes look up an item each
//    -- after a prompt nearly all are finished already -- and the warp folds
//    the rest one by one;
//  * eight records (four at head dim 256) are in flight per warp.
#include <algorithm>

#include "common.cuh"
#include "decode_tile.cuh"
#include "internal.h"
#include "paged.cuh"

namespace attn {

namespace {

constexpr int kCombWarps = 8;

template <int D>
struct Fold {
  static constexpr int EPL = D / 32;
  float M, L, O[EPL];
  __device__ __forceinline__ void reset() {
    M = neg_inf();
    L = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) O[i] = 0.f;
  }
  __device__ __forceinline__ void add(float m, float l, const float2* v) {
    const float mn = fmax_nan(M, m), mu = (mn == neg_inf()) ? 0.f : mn;
    const float c = ex2((M - mu) * kLog2e), f = ex2((m - mu) * kLog2e);
    L = fmaf(L, c, l * f);
#pragma unroll
    for (int i = 0; i < EPL / 2; ++i) {
      O[2 * i] = fmaf(O[2 * i], c, v[i].x * f);
      O[2 * i + 1] = fmaf(O[2 * i + 1], c, v[i].y * f);
    }
    M = mn;
  }
};

template <int D, bool SHARED>
__global__ void __launch_bounds__(32 * kCombWarps) paged_combine_kernel(const SharedPlan sp, const PagedPlan own,
                                                                        int wpi, int ipw) {
  using F = Fold<D>;
  constexpr int EPL = F::EPL, NF = D == 256 ? 4 : 8;   // NF: records in flight
  __shared__ float2 part[kCombWarps][D / 2];
  __shared__ float2 part_ml[kCombWarps];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % wpi;   // this warp's share of its item
  const int round = wpi > 1 ? NF : 32;   // records a warp looks up at a time
  const DecodePlan& d = own.d;
  const int items = d.R * d.Hq;   // (checked: below 2^31)
  const int64_t item0 = ((int64_t)blockIdx.x * (kCombWarps / wpi) + warp / wpi) * ipw;

  // this lane's item: its shared records (run s0 at home, then runs to s1,
  // lane slot `sl`) and its own ones (warps o0 .. o1)
  const int item_l = (int)min(item0 + lane, (int64_t)items - 1);
  const int r_l = item_l / d.Hq, h_l = item_l - r_l * d.Hq, g_l = h_l / d.G;
  const int64_t T = (int64_t)d.Hkv * d.row_tiles[d.R], W = d.W;
  const int64_t t_l = d.row_tiles[r_l], nt_l = d.row_tiles[r_l + 1] - t_l;
  int s0 = 0, s1 = -1, sl = 0, o0 = 0, o1 = -1;
  if (SHARED) {
    const int k = sp.row_blk[r_l];
    if (k >= 0) {
      const int2 u = sp.unit_runs[(int64_t)k * d.Hkv + g_l];
      const int j = r_l - sp.blocks[k].row0, slot = (sp.blocks[k].w == 2 && j >= sp.rpt) ? 1 : 0;
      s0 = u.x;
      s1 = u.y;
      sl = slot * 128 + (j - slot * sp.rpt) * d.G + h_l - g_l * d.G;
    }
  }
  if (nt_l > 0) {
    const int64_t at = (int64_t)d.Hkv * t_l + g_l * nt_l;
    o0 = run_of(at, T, W);
    o1 = run_of(at + nt_l - 1, T, W);
  }
  const float sigma_l = d.lg.sinks ? __ldg(d.lg.sinks + h_l) : neg_inf();
  // (one shared piece and no own cells: finished by that piece)
  const bool todo = lane < ipw && item0 + lane < items && !(SHARED && s0 == s1 && nt_l == 0);
  unsigned left = __ballot_sync(0xffffffffu, todo);
  while (left || wpi > 1) {   // (wpi > 1: one item, and every warp reaches the barrier)
    const bool live = left != 0;
    const int q = live ? __ffs(left) - 1 : 0;
    left &= left - 1;
    const int64_t item = item0 + q;
    const int r = __shfl_sync(0xffffffffu, r_l, q), h = __shfl_sync(0xffffffffu, h_l, q);
    const int g = __shfl_sync(0xffffffffu, g_l, q), hh = h - g * d.G;
    const int a0 = __shfl_sync(0xffffffffu, s0, q), a1 = __shfl_sync(0xffffffffu, s1, q);
    const int b0 = __shfl_sync(0xffffffffu, o0, q), b1 = __shfl_sync(0xffffffffu, o1, q);
    const int asl = __shfl_sync(0xffffffffu, sl, q);
    F f;
    f.reset();
#pragma unroll 1
    for (int p = SHARED ? 0 : 1; live && p < 2; ++p) {
      const float* po = p ? d.part.o : sp.rec_o;
      const float* pml = p ? d.part.ml : sp.rec_ml;
      const int w0 = p ? b0 : a0, w1 = p ? b1 : a1;
      for (int base = w0 + round * sub; base <= w1; base += round * wpi) {
        const int w = base + lane;
        bool has = lane < round && w <= w1;
        int64_t rec = 0;
        if (p == 0) {
          rec = w == w0 ? item : (int64_t)items + (int64_t)w * 256 + asl;
          if (has && w > w0 && w < w1) {   // a run without a tile leaves no record (the ends have one)
            const SharedRun *x = sp.runs + w, *y = x + 1;
            has = x->k != y->k || x->g != y->g || x->i != y->i;
          }
        } else {
          rec = (w == w0 ? W + (int64_t)r * d.Hkv + g : w) * d.G + hh;
          if (has && w > w0 && w < w1 && T < W) has = div64(T * w, W) < div64(T * (w + 1), W);
        }
        unsigned m = __ballot_sync(0xffffffffu, has);
        while (m) {
          float2 ml[NF], v[NF][EPL / 2];
#pragma unroll
          for (int u = 0; u < NF; ++u) {
            const bool there = m != 0;
            const int64_t rr = __shfl_sync(0xffffffffu, rec, there ? __ffs(m) - 1 : 0);
            m &= m - 1;   // (0 stays 0)
            ml[u] = there ? *reinterpret_cast<const float2*>(pml + rr * 2) : make_float2(neg_inf(), 0.f);
#pragma unroll
            for (int i = 0; i < EPL / 2; ++i)
              v[u][i] = there ? *reinterpret_cast<const float2*>(po + rr * D + lane * EPL + 2 * i) : make_float2(0.f, 0.f);
          }
#pragma unroll
          for (int u = 0; u < NF; ++u) f.add(ml[u].x, ml[u].y, v[u]);
        }
      }
    }
    if (wpi > 1) {
#pragma unroll
      for (int i = 0; i < EPL / 2; ++i) part[warp][lane * (EPL / 2) + i] = make_float2(f.O[2 * i], f.O[2 * i + 1]);
      if (lane == 0) part_ml[warp] = make_float2(f.M, f.L);
      __syncthreads();
      if (!live || sub != 0) return;
      for (int u = 1; u < wpi; ++u) {
        float2 v[EPL / 2];
#pragma unroll
        for (int i = 0; i < EPL / 2; ++i) v[i] = part[warp + u][lane * (EPL / 2) + i];
        f.add(part_ml[warp + u].x, part_ml[warp + u].y, v);
      }
    }
    const float sigma = __shfl_sync(0xffffffffu, sigma_l, q);
    const int64_t ob = (int64_t)r * d.out.sr + (int64_t)h * d.out.sh + lane * EPL;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      store_from_float(d.out.out, ob + i, d.out.type, fold_with_sink(f.M, f.L, f.O[i], sigma));
    if (wpi > 1) return;
  }
}

template <bool SHARED>
cudaError_t launch_t(const SharedPlan& sp, const PagedPlan& own, int sms, cudaStream_t stream) {
  // Warps per item 8, 4, 2 while items x warps stay within the 24 resident warps per SM,
  // then items per warp 1 .. 32 to stay there (131072 items of a prompt: 58 us
  // at 32 items a warp, 77 at 8, where the lookups of four times the warps cost more;
  // 52 us since the sinks are read with the lookups).
  const int64_t items = (int64_t)own.d.R * own.d.Hq, room = 24LL * sms;
  int wpi = kCombWarps;
  while (wpi > 1 && items * wpi > room) wpi >>= 1;
  const int ipw = wpi > 1 ? 1 : (int)std::min<int64_t>(32, std::max<int64_t>(1, items / room));
  const int64_t per_cta = (int64_t)(kCombWarps / wpi) * ipw;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((items + per_cta - 1) / per_cta));
  cfg.blockDim = dim3(32 * kCombWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (own.d.D) {
    case 64: return cudaLaunchKernelEx(&cfg, paged_combine_kernel<64, SHARED>, sp, own, wpi, ipw);
    case 128: return cudaLaunchKernelEx(&cfg, paged_combine_kernel<128, SHARED>, sp, own, wpi, ipw);
    default: return cudaLaunchKernelEx(&cfg, paged_combine_kernel<256, SHARED>, sp, own, wpi, ipw);
  }
}

}  // namespace

cudaError_t launch_paged_combine(const SharedPlan* sp, const PagedPlan& own, int sms, cudaStream_t stream) {
  return sp ? launch_t<true>(*sp, own, sms, stream) : launch_t<false>(SharedPlan{}, own, sms, stream);
}

}  // namespace attn
