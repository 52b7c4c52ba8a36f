// page_tables.cu -- block tables, slot map and row ranges of a serving step,
// built on the GPU from the sequences' lengths.
//
// For sequence i (len_i cells held, new_i rows in this step, P cells a page):
//   held_i = ceil(len_i / P),  need_i = ceil((len_i + new_i) / P) - held_i,
// first row = exclusive scan of max(new_i, 0), first ring entry = exclusive
// scan of need_i (new_i >= 0), first returned entry = exclusive scan of
// held_i - keep_i (new_i < 0).  Row t of sequence i sits at position
// p = len_i + t - first row, on page index p / P: an old table entry below
// held_i, else ring[head + first entry + p / P - held_i].
//
// One launch: the scans are small (a few thousand sequences) and the row
// writes are not, so every CTA repeats the scans over all sequences in shared
// memory and then writes its own rows, finding a row's sequence by binary
// search in the scanned row counts.  No CTA waits for another: the ring
// entries that are read ([head, head + count)) and written (from head + count
// on), and the table entries that are read (below held) and written (from
// held on), are disjoint, and the counters have separate in and out arrays.
// The work is bound by launch latency and two dependent loads (length, then
// table or ring entry): about 12 bytes written per row.  3.8 us a call for 16
// sequences (the launch and the host call), 8.4 us for 509 sequences and about
// 50000 rows.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace attn {

namespace {

constexpr int kPtThreads = 512;
constexpr int kPtMaxSeqs = 16384;

// Totals of the rounds so far: rows, pages asked for, pages returned.
struct Sums {
  int64_t rows, need, rel;
};

__device__ __forceinline__ int64_t warp_incl(int64_t x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  return x;
}

__device__ __forceinline__ int32_t sat32(int64_t x) { return (int32_t)(x > 0x7fffffffLL ? 0x7fffffffLL : x); }

__global__ void __launch_bounds__(kPtThreads) page_tables_kernel(const PageTablesPlan p) {
  // [n] each: the end of the sequence's rows, its first ring entry (-1: it does
  // not grow), and the first returned page of those that end
  extern __shared__ int32_t sh[];
  __shared__ int64_t wsum[3][kPtThreads / 32];
  __shared__ int32_t used_sh;
  const attn_page_args& a = p.a;
  const int n = a.n_seqs, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  int32_t* row_last = sh;
  int32_t* ring_first = sh + n;
  int32_t* rel_first = sh + 2 * n;
  // No early trigger for the next kernel: it may look at row_end before its own
  // wait (attn_decode's prefix of few rows does).
  pdl_wait_prior_grid();
  int32_t head = __ldg(a.free_state), count = __ldg(a.free_state + 1);
  if (head < 0 || head >= a.n_pages || count < 0 || count > a.n_pages) {
    if (a.n_pages > 0) record_status(p.status, ATTN_ERR_INVALID_ARG);
    head = count = 0;
  }
  const int64_t cap = (int64_t)a.table_width * a.page_size;   // cells of a table row
  if (tid == 0) used_sh = 0;
  Sums carry{0, 0, 0};
  for (int base = 0; base < n; base += kPtThreads) {
    const int i = base + tid;
    int32_t len = 0, nw = 0, keep = 0;
    bool bad = false;
    if (i < n) {
      len = __ldg(a.seq_len + i);
      nw = __ldg(a.new_len + i);
      keep = (a.n_keep && nw < 0) ? max(__ldg(a.n_keep + i), 0) : 0;
      bad = len < 0 || len > cap;
      if (bad) record_status(p.status, ATTN_ERR_INVALID_ARG);
    }
    const int64_t grow = nw > 0 ? nw : 0;
    const int32_t held = bad ? 0 : (int32_t)(((int64_t)len + a.page_size - 1) / a.page_size);
    const bool fits = !bad && len + grow <= cap;
    const int64_t need = fits ? (len + grow + a.page_size - 1) / a.page_size - held : 0;
    const int64_t rel = (nw < 0 && held > keep) ? held - keep : 0;
    int64_t x[3] = {warp_incl(grow, lane), warp_incl(need, lane), warp_incl(rel, lane)};
    __syncthreads();   // the previous round's wsum is read
    if (lane == 31)
      for (int k = 0; k < 3; ++k) wsum[k][wid] = x[k];
    __syncthreads();
    int64_t tot[3] = {0, 0, 0};
    for (int w = 0; w < kPtThreads / 32; ++w)
      for (int k = 0; k < 3; ++k) {
        if (w < wid) x[k] += wsum[k][w];
        tot[k] += wsum[k][w];
      }
    if (i < n) {
      const int64_t r_end = carry.rows + x[0], q_end = carry.need + x[1];
      const bool ok = nw >= 0 && fits && (need == 0 || q_end <= count) && r_end <= a.n_rows;
      row_last[i] = sat32(r_end);
      ring_first[i] = ok ? (int32_t)(q_end - need) : -1;
      rel_first[i] = sat32(carry.rel + x[2] - rel);
      if (ok && need > 0) atomicMax(&used_sh, (int32_t)q_end);
      if (blockIdx.x == 0) {
        if (a.seq_row) {
          a.seq_row[i + 1] = sat32(r_end);
          if (i == 0) a.seq_row[0] = 0;
        }
        a.seq_len_out[i] = nw < 0 ? 0 : ok ? len + (int32_t)grow : len;
      }
    }
    carry.rows += tot[0];
    carry.need += tot[1];
    carry.rel += tot[2];
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    if (n == 0 && a.seq_row) a.seq_row[0] = 0;
    const int64_t room = (int64_t)a.n_pages - count;   // returned pages never overwrite free ones
    if (carry.rel > room) record_status(p.status, ATTN_ERR_INVALID_ARG);
    a.free_state_out[0] = a.n_pages > 0 ? (int32_t)(((int64_t)head + used_sh) % a.n_pages) : 0;
    a.free_state_out[1] = (int32_t)(count - used_sh + (carry.rel < room ? carry.rel : room));
  }

  // rows
  for (int64_t t = (int64_t)blockIdx.x * kPtThreads + tid; t < a.n_rows; t += (int64_t)gridDim.x * kPtThreads) {
    int lo = 0, hi = n;   // the first sequence whose rows end after t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (row_last[mid] > t) hi = mid;
      else lo = mid + 1;
    }
    int32_t slot = -1, seq = -1, end = 0;
    if (lo < n) {
      seq = lo;
      const int32_t rf = ring_first[lo];
      if (rf >= 0) {
        const int32_t len = __ldg(a.seq_len + lo);
        const int32_t held = (len + a.page_size - 1) / a.page_size;
        const int32_t pos = len + (int32_t)(t - (lo > 0 ? row_last[lo - 1] : 0));
        const int32_t pi = pos / a.page_size, off = pos - pi * a.page_size;
        int32_t* entry = a.page_table + (int64_t)lo * a.table_stride + pi;
        int32_t page;
        if (pi < held) {
          page = *entry;
        } else {
          page = a.free_ring[((int64_t)head + rf + (pi - held)) % a.n_pages];
          if (off == 0) *entry = page;
        }
        end = pos + 1;
        if (page >= 0 && page < a.n_pages) slot = page * a.page_size + off;
        else record_status(p.status, ATTN_ERR_INVALID_ARG);
      }
    }
    a.slot[t] = slot;
    if (a.row_seq) a.row_seq[t] = seq;
    if (a.row_end) a.row_end[t] = end;
  }

  // returned pages: a warp per ended sequence
  if (carry.rel == 0) return;
  const int warps = gridDim.x * (kPtThreads / 32);
  for (int i = blockIdx.x * (kPtThreads / 32) + wid; i < n; i += warps) {
    if (__ldg(a.new_len + i) >= 0) continue;
    const int32_t len = __ldg(a.seq_len + i);
    if (len <= 0 || len > cap) continue;
    const int32_t held = (int32_t)(((int64_t)len + a.page_size - 1) / a.page_size);
    const int32_t keep = a.n_keep ? max(__ldg(a.n_keep + i), 0) : 0;
    for (int32_t j = keep + lane; j < held; j += 32) {
      const int64_t k = (int64_t)count + rel_first[i] + (j - keep);   // free pages ahead of this one
      if (k >= a.n_pages) break;
      const int32_t page = a.page_table[(int64_t)i * a.table_stride + j];
      if (page < 0 || page >= a.n_pages) record_status(p.status, ATTN_ERR_INVALID_ARG);
      a.free_ring[((int64_t)head + k) % a.n_pages] = page;
    }
  }
}

}  // namespace

int max_page_seqs() { return kPtMaxSeqs; }

cudaError_t launch_page_tables(const PageTablesPlan& p, int sms, cudaStream_t stream) {
  static std::atomic<unsigned long long> smem_set{0ull};
  cudaError_t e = set_smem_limit_once(smem_set, page_tables_kernel, kPtMaxSeqs * 3 * (int)sizeof(int32_t));
  if (e != cudaSuccess) return e;
  // a CTA per 1024 rows (two per thread) or per 64 sequences (their returned
  // pages), at most one per SM
  const int64_t want = std::max<int64_t>((p.a.n_rows + 2 * kPtThreads - 1) / (2 * kPtThreads), (p.a.n_seqs + 63) / 64);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(want, sms)));
  cfg.blockDim = dim3(kPtThreads);
  cfg.dynamicSmemBytes = (size_t)p.a.n_seqs * 3 * sizeof(int32_t);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_tables_kernel, p);
}

}  // namespace attn
