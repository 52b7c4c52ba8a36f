// paged.cuh -- rows and pages of a paged cache, shared by its kernels.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace attn {

// The cells a row may see, and the 16-cell tiles (cut at multiples of 16
// cells) that hold them.
struct PagedRow {
  int32_t begin, end;   // clipped to [0, table_width * page_size); end >= begin
  int32_t raw_end;      // row_end as given (ALiBi distances)
  int32_t table;        // the row's block table
  int32_t tile0;        // begin / 16
  __device__ __forceinline__ int64_t tiles() const { return end > begin ? (end + 15) / 16 - tile0 : 0; }
};

__device__ __forceinline__ PagedRow paged_row(const PagedPlan& p, int r) {
  PagedRow v;
  int32_t b = p.d.f.row_begin ? __ldg(p.d.f.row_begin + r) : 0;
  v.raw_end = __ldg(p.d.f.row_end + r);
  if (p.own_lo) b = max(b, __ldg(p.own_lo + r));
  v.begin = max(b, 0);
  v.end = max(min(v.raw_end, p.width * p.P), v.begin);
  v.table = p.row_table ? __ldg(p.row_table + r) : r;
  if (v.table < 0 || v.table >= p.n_tables) {   // padding rows (an empty range) may name no table
    if (v.end > v.begin) record_status(p.d.status, ATTN_ERR_INVALID_ARG);
    v.table = 0;
    v.end = v.begin;
  }
  v.tile0 = v.begin / 16;
  return v;
}

// The page of the row's cell c; n_pages (where the TMA reads zeros) for an id
// outside the pool.
__device__ __forceinline__ int32_t paged_page(const PagedPlan& p, const PagedRow& row, int32_t c) {
  const int32_t id = __ldg(p.table + (int64_t)row.table * p.table_sr + c / p.P);
  if (id >= 0 && id < p.n_pages) return id;
  record_status(p.d.status, ATTN_ERR_INVALID_ARG);
  return p.n_pages;
}

// a / b of nonnegative numbers, b > 0: in 32 bits where both fit (a 64-bit
// division is about 150 dependent instructions, 0.4 us on an idle SM).
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  if (((uint64_t)(a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// The run that holds tile t of T tiles cut into W runs [T w / W, T (w + 1) / W).
__device__ __forceinline__ int run_of(int64_t t, int64_t T, int64_t W) {
  return (int)div64((t + 1) * W + T - 1, T) - 1;
}

// The test of the bounded waits: `bar`, which nothing arrives at, for limit_ns;
// records the timeout as mbar_wait_bounded does.
__device__ __forceinline__ void stall_bounded(uint64_t* bar, uint64_t limit_ns, int* status) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, 0) && global_timer_ns() - t0 <= limit_ns) {
  }
  record_status(status, ATTN_ERR_DEVICE_TIMEOUT);
}

// 4-D tiled TMA load into shared memory, completing on `bar` (tx bytes).
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, int c3, uint64_t cache_hint) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;"
      ::"r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)),
        "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(cache_hint)
      : "memory");
}

}  // namespace attn
