// paged_api.cu -- the C ABI of the paged-cache operations (include/attn.h):
// argument checks, workspace layout, tile maps and launches.  As in api.cu, a
// call that the kernels do not cover is refused before anything is launched.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "attn.h"
#include "internal.h"

namespace attn {
namespace {

int32_t refuse(int32_t status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return status;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool is16(int32_t t) { return t == ATTN_F16 || t == ATTN_BF16; }
bool is8(int32_t t) { return t == ATTN_FP8_E4M3 || t == ATTN_I8; }
int esize(int32_t t) { return t == ATTN_F32 ? 4 : is16(t) ? 2 : 1; }
size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// cells of a pool or of a table row: slots and positions are int32, tiles are
// rounded up to 256 cells
constexpr int64_t kMaxCells = 0x7fffffffLL - 256;

int32_t check_pool(const char* op, int32_t n_pages, int32_t page_size) {
  if (n_pages < 0 || page_size < 1) return refuse(ATTN_ERR_INVALID_ARG, "%s: n_pages < 0 or page_size < 1", op);
  if ((int64_t)n_pages * page_size > kMaxCells)
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: %d pages of %d cells pass the 2^31 slots", op, n_pages, page_size);
  return ATTN_OK;
}

// Strides of a paged cache: nonnegative, multiples of 16 bytes, and no two
// cells in one place (zero strides; overlaps beyond that are the caller's).
int32_t check_cache(const char* op, const void* k, const void* v, int32_t type, int32_t n_pages, int32_t page_size,
                    int32_t heads, int64_t sp, int64_t sc, int64_t sh) {
  if (sp < 0 || sc < 0 || sh < 0) return refuse(ATTN_ERR_INVALID_ARG, "%s: negative kv stride", op);
  if (n_pages == 0) return ATTN_OK;
  if (!k || !v) return refuse(ATTN_ERR_INVALID_ARG, "%s: k or v is NULL", op);
  const int es = esize(type);
  if (!aligned16(k) || !aligned16(v) || (n_pages > 1 && (sp * es) % 16) || (page_size > 1 && (sc * es) % 16) ||
      (heads > 1 && (sh * es) % 16))
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: k, v and their strides must be multiples of 16 bytes", op);
  if ((n_pages > 1 && sp == 0) || (page_size > 1 && sc == 0) || (heads > 1 && sh == 0))
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: zero kv stride (broadcast caches are not supported)", op);
  return ATTN_OK;
}

int32_t check_scales(const char* op, int32_t type, int32_t n_pages, int32_t page_size, int32_t heads, const void* ks,
                     const void* vs, int64_t ss) {
  if (!is8(type)) {
    if (ks || vs) return refuse(ATTN_ERR_INVALID_ARG, "%s: k_scale/v_scale are only for e4m3/int8 caches", op);
    return ATTN_OK;
  }
  if (n_pages > 0 && (!ks || !vs))
    return refuse(ATTN_ERR_INVALID_ARG, "%s: an e4m3/int8 cache needs k_scale and v_scale", op);
  if ((int64_t)n_pages * page_size > 1 && ss < heads)
    return refuse(ATTN_ERR_INVALID_ARG, "%s: scale_stride_cell is smaller than n_head_kv", op);
  return ATTN_OK;
}

// Whether two arrays of int32 share an entry.
struct I32Array {
  const int32_t* p;
  int64_t n;
};
bool overlap(const I32Array& x, const I32Array& y) {
  return x.p && y.p && x.n > 0 && y.n > 0 && x.p < y.p + y.n && y.p < x.p + x.n;
}

int32_t check_pages(const attn_page_args* a) {
  const char* op = "page_tables";
  if (!a) return refuse(ATTN_ERR_INVALID_ARG, "args is NULL");
  for (int i = 0; i < 4; ++i)
    if (a->reserved[i] != 0) return refuse(ATTN_ERR_INVALID_ARG, "reserved fields must be zero");
  if (a->n_seqs < 0 || a->n_rows < 0 || a->table_width < 0)
    return refuse(ATTN_ERR_INVALID_ARG, "%s: negative size", op);
  if (a->n_seqs > max_page_seqs())
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: %d sequences > %d", op, a->n_seqs, max_page_seqs());
  int32_t st = check_pool(op, a->n_pages, a->page_size);
  if (st != ATTN_OK) return st;
  if ((int64_t)(a->table_width + 1LL) * a->page_size > kMaxCells)
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: a table row of %d pages passes 2^31 cells", op, a->table_width);
  if (!a->free_state || !a->free_state_out) return refuse(ATTN_ERR_INVALID_ARG, "%s: free_state is NULL", op);
  if (a->n_rows > 0 && !a->slot) return refuse(ATTN_ERR_INVALID_ARG, "%s: slot is NULL", op);
  if (a->n_pages > 0 && !a->free_ring) return refuse(ATTN_ERR_INVALID_ARG, "%s: free_ring is NULL", op);
  if (a->free_state == a->free_state_out)
    return refuse(ATTN_ERR_INVALID_ARG, "%s: free_state_out must not be the input array", op);
  if (a->n_seqs > 0) {
    if (!a->seq_len || !a->new_len || !a->seq_len_out)
      return refuse(ATTN_ERR_INVALID_ARG, "%s: seq_len, new_len or seq_len_out is NULL", op);
    if (a->table_width > 0 && !a->page_table) return refuse(ATTN_ERR_INVALID_ARG, "%s: page_table is NULL", op);
    if (a->n_seqs > 1 && a->table_stride < a->table_width)
      return refuse(ATTN_ERR_INVALID_ARG, "%s: table_stride is smaller than table_width", op);
    if (a->seq_len == a->seq_len_out)
      return refuse(ATTN_ERR_INVALID_ARG, "%s: seq_len_out must not be the input array", op);
  }
  // every CTA reads the inputs while others write: an array that is written is no other one's
  const int64_t n = a->n_seqs, rows = a->n_rows;
  const I32Array all[] = {
      {a->slot, rows}, {a->row_seq, rows}, {a->row_end, rows}, {a->seq_row, n + 1}, {a->seq_len_out, n},
      {a->free_state_out, 2}, {a->page_table, n > 0 ? (n - 1) * a->table_stride + a->table_width : 0},
      {a->free_ring, a->n_pages}, {a->seq_len, n}, {a->new_len, n}, {a->n_keep, n}, {a->free_state, 2}};
  constexpr int kWritten = 8, kAll = sizeof(all) / sizeof(all[0]);
  for (int i = 0; i < kWritten; ++i)
    for (int j = i + 1; j < kAll; ++j)
      if (overlap(all[i], all[j]))
        return refuse(ATTN_ERR_INVALID_ARG, "%s: an array that is written overlaps another one", op);
  return ATTN_OK;
}

int32_t check_append(const attn_append_args* a) {
  const char* op = "append_paged";
  if (!a) return refuse(ATTN_ERR_INVALID_ARG, "args is NULL");
  for (int i = 0; i < 4; ++i)
    if (a->reserved[i] != 0) return refuse(ATTN_ERR_INVALID_ARG, "reserved fields must be zero");
  if (a->n_rows < 0 || a->n_head_kv <= 0) return refuse(ATTN_ERR_INVALID_ARG, "%s: n_rows < 0 or n_head_kv <= 0", op);
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256)
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128, 256}", op, a->head_dim);
  if (a->new_type != ATTN_F32 && !is16(a->new_type))
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: new rows must be F32, F16 or BF16", op);
  if (!is16(a->kv_type) && !is8(a->kv_type))
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: the cache must be F16, BF16, e4m3 or int8", op);
  int32_t st = check_pool(op, a->n_pages, a->page_size);
  if (st != ATTN_OK) return st;
  if ((st = check_scales(op, a->kv_type, a->n_pages, a->page_size, a->n_head_kv, a->k_scale, a->v_scale,
                         a->scale_stride_cell)) != ATTN_OK)
    return st;
  if ((st = check_cache(op, a->k, a->v, a->kv_type, a->n_pages, a->page_size, a->n_head_kv, a->kv_stride_page,
                        a->kv_stride_cell, a->kv_stride_head)) != ATTN_OK)
    return st;
  if (a->new_stride_row < 0 || a->new_stride_head < 0) return refuse(ATTN_ERR_INVALID_ARG, "%s: negative stride", op);
  if (a->n_rows == 0) return ATTN_OK;
  if (!a->k_new || !a->v_new || !a->slot) return refuse(ATTN_ERR_INVALID_ARG, "%s: k_new, v_new or slot is NULL", op);
  const int es = esize(a->new_type);
  if (!aligned16(a->k_new) || !aligned16(a->v_new) || (a->n_rows > 1 && (a->new_stride_row * es) % 16) ||
      (a->n_head_kv > 1 && (a->new_stride_head * es) % 16))
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: new rows and their strides must be multiples of 16 bytes", op);
  if (a->n_rows > (1 << 30) || (int64_t)a->n_rows * a->n_head_kv > (1LL << 33))   // (the kernels' row numbers are int32)
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: too many rows", op);
  return ATTN_OK;
}

// Sharing takes four launches and a plan, 10 to 20 us more than row by row,
// and saves at most the reading of all rows' tables.  Below 64 MB of them (at
// 5.4 TB/s 12 us) row by row is the faster form whatever the groups: 8 rows
// of 1100 cells, 8 KV heads, D 128 (38 MB) take 13 us against 32 us.  The rule
// sees what the tables can hold, not the lengths, which are on the device.
constexpr int64_t kShareBytes = 64LL << 20;
bool runs_shared(const attn_paged_args* a, int32_t op) {
  if (op != ATTN_OP_DECODE_SHARED || !is16(a->kv_type) || a->n_groups == 0 || a->n_pages == 0) return false;
  const double bytes = (double)a->n_rows * a->n_head_kv * a->table_width * a->page_size * 4.0 * a->head_dim;
  return bytes > (double)kShareBytes;
}

int32_t check_paged(const attn_paged_args* a, int32_t op_id) {
  const bool shared = op_id == ATTN_OP_DECODE_SHARED;
  if (op_id != ATTN_OP_DECODE_PAGED && !shared) return refuse(ATTN_ERR_INVALID_ARG, "unknown op %d", op_id);
  const char* op = shared ? "decode_shared" : "decode_paged";
  if (!a) return refuse(ATTN_ERR_INVALID_ARG, "args is NULL");
  for (int i = 1; i < 4; ++i)
    if (a->reserved[i] != 0) return refuse(ATTN_ERR_INVALID_ARG, "reserved fields must be zero");
  if (a->reserved[0] < 0 || a->reserved[0] > 1000000)
    return refuse(ATTN_ERR_INVALID_ARG, "%s: reserved[0] (the bounded-wait test) must be 0..1000000 us", op);
  if (a->n_rows < 0 || a->n_tables < 0 || a->table_width < 0 || a->n_groups < 0)
    return refuse(ATTN_ERR_INVALID_ARG, "%s: negative size", op);
  if (a->n_head_q <= 0 || a->n_head_kv <= 0 || a->n_head_q % a->n_head_kv != 0)
    return refuse(ATTN_ERR_INVALID_ARG, "%s: n_head_q (%d) is not a positive multiple of n_head_kv (%d)", op,
                  a->n_head_q, a->n_head_kv);
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256)
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128, 256}", op, a->head_dim);
  const int G = a->n_head_q / a->n_head_kv;
  if (is16(a->kv_type)) {
    if (a->q_type != a->kv_type) return refuse(ATTN_ERR_UNSUPPORTED, "%s: Q must be in the cache dtype", op);
    if (G > 16) return refuse(ATTN_ERR_UNSUPPORTED, "%s: %d q heads per KV head > 16", op, G);
  } else if (is8(a->kv_type)) {
    if (!is16(a->q_type)) return refuse(ATTN_ERR_UNSUPPORTED, "%s: Q must be F16 or BF16 over an e4m3/int8 cache", op);
    if (G > 8) return refuse(ATTN_ERR_UNSUPPORTED, "%s: %d q heads per KV head > 8 over an e4m3/int8 cache", op, G);
    if (a->head_dim == 64) return refuse(ATTN_ERR_UNSUPPORTED, "%s: head_dim 64 over an e4m3/int8 cache", op);
  } else {
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: the cache must be F16, BF16, e4m3 or int8", op);
  }
  if (a->out_type != ATTN_F32 && !is16(a->out_type))
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: out must be F32, F16 or BF16", op);
  int32_t st = check_pool(op, a->n_pages, a->page_size);
  if (st != ATTN_OK) return st;
  if (a->page_size % 16) return refuse(ATTN_ERR_UNSUPPORTED, "%s: page_size must be a multiple of 16", op);
  if ((int64_t)a->table_width * a->page_size > kMaxCells)
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: a table row of %d pages passes 2^31 cells", op, a->table_width);
  if ((st = check_scales(op, a->kv_type, a->n_pages, a->page_size, a->n_head_kv, a->k_scale, a->v_scale,
                         a->scale_stride_cell)) != ATTN_OK)
    return st;
  if ((st = check_cache(op, a->k, a->v, a->kv_type, a->n_pages, a->page_size, a->n_head_kv, a->kv_stride_page,
                        a->kv_stride_cell, a->kv_stride_head)) != ATTN_OK)
    return st;
  if (a->scale != a->scale) return refuse(ATTN_ERR_INVALID_ARG, "%s: scale is NaN", op);
  if (a->q_stride_row < 0 || a->q_stride_head < 0 || a->o_stride_row < 0 || a->o_stride_head < 0)
    return refuse(ATTN_ERR_INVALID_ARG, "%s: negative stride", op);
  if (!shared && (a->n_groups || a->group_begin || a->group_len))
    return refuse(ATTN_ERR_INVALID_ARG, "%s: groups are decode_shared's", op);
  if (a->n_rows == 0) return ATTN_OK;
  if (!a->q || !a->out || !a->row_end) return refuse(ATTN_ERR_INVALID_ARG, "%s: q, out or row_end is NULL", op);
  if (a->n_tables > 0 && a->table_width > 0 && !a->page_table)
    return refuse(ATTN_ERR_INVALID_ARG, "%s: page_table is NULL", op);
  if (a->n_tables > 1 && a->table_stride < a->table_width)
    return refuse(ATTN_ERR_INVALID_ARG, "%s: table_stride is smaller than table_width", op);
  if (!a->row_table && a->n_tables < a->n_rows)
    return refuse(ATTN_ERR_INVALID_ARG, "%s: %d tables for %d rows and no row_table", op, a->n_tables, a->n_rows);
  if (shared && a->n_groups > 0 && (!a->group_begin || !a->group_len))
    return refuse(ATTN_ERR_INVALID_ARG, "%s: group_begin or group_len is NULL", op);
  if (!aligned16(a->q) || (a->n_rows > 1 && a->q_stride_row % 8) || (a->n_head_q > 1 && a->q_stride_head % 8))
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: Q must be 16-byte aligned with strides that are multiples of 8", op);
  if (shared && ((a->n_rows > 1 && a->q_stride_row == 0) || (a->n_head_q > 1 && a->q_stride_head == 0)))
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: zero q stride", op);
  if ((int64_t)a->n_rows * a->n_head_q > 0x7fffffffLL)
    return refuse(ATTN_ERR_UNSUPPORTED, "%s: too many rows", op);
  return ATTN_OK;
}

// Workspace: the row tile prefix, then the split records ([slots][G][D] and
// [slots][G][2] floats; a slot per warp and per (row, KV head)).
struct PagedWs {
  size_t tiles_off, o_off, ml_off, total;
};
PagedWs paged_ws(const attn_paged_args* a, int W) {
  PagedWs w{};
  const size_t G = (size_t)(a->n_head_q / a->n_head_kv);
  w.o_off = align256(((size_t)a->n_rows + 1) * sizeof(int64_t));
  const size_t records = ((size_t)W + (size_t)a->n_rows * a->n_head_kv) * G;
  w.ml_off = w.o_off + align256(records * a->head_dim * sizeof(float));
  w.total = w.ml_off + align256(records * 2 * sizeof(float));
  return w;
}

// What decode_shared adds: the plan (blocks of rows, their work prefix, each
// row's block and own first cell) and the shared pieces' records: a home record
// per (row, q head) and 256 lanes per run.
struct SharedWs {
  size_t blocks_off, off_off, runs_off, unit_off, blk_off, own_off, o_off, ml_off, total;
};
int shared_slots(int D) { return D <= 128 ? 2 : 1; }
int64_t shared_block_rows(const attn_paged_args* a) {
  return (int64_t)shared_slots(a->head_dim) * (128 / (a->n_head_q / a->n_head_kv));
}
size_t shared_max_blocks(const attn_paged_args* a) {
  return (size_t)std::min(a->n_groups, a->n_rows) + (size_t)a->n_rows / (size_t)shared_block_rows(a) + 1;
}
SharedWs shared_ws(const attn_paged_args* a, size_t base, int sms) {
  SharedWs w{};
  const size_t R = (size_t)a->n_rows;
  const size_t nb = shared_max_blocks(a);
  w.blocks_off = align256(base);
  w.off_off = w.blocks_off + align256(nb * sizeof(SharedBlock));
  w.runs_off = w.off_off + align256((nb + 1) * sizeof(int64_t));
  w.unit_off = w.runs_off + align256(((size_t)sms + 1) * sizeof(SharedRun));
  w.blk_off = w.unit_off + align256(nb * a->n_head_kv * sizeof(int2));
  w.own_off = w.blk_off + align256(R * sizeof(int32_t));
  w.o_off = w.own_off + align256(R * sizeof(int32_t));
  const size_t records = R * a->n_head_q + (size_t)sms * 256;
  w.ml_off = w.o_off + align256(records * a->head_dim * sizeof(float));
  w.total = w.ml_off + align256(records * 2 * sizeof(float));
  return w;
}

// The pool as a 4-D map [page][cell][head][D] with boxes of 128 bytes of one
// head of box_cells cells of a page.
int32_t pool_map(CUtensorMap* map, const void* base, const attn_paged_args* a, int box_cells) {
  const int es = esize(a->kv_type), D = a->head_dim;
  const int64_t dims[4] = {D, a->n_head_kv, a->page_size, a->n_pages};
  // a stride of an extent-1 dimension is never used; give the encoder a legal one
  const int64_t strides[3] = {(a->n_head_kv > 1 ? a->kv_stride_head : D) * es, a->kv_stride_cell * es,
                              (a->n_pages > 1 ? a->kv_stride_page : (int64_t)D) * es};
  const int32_t box[4] = {128 / es, 1, box_cells, 1};
  return encode_map(map, base, a->kv_type, 4, dims, strides, box);
}

void fill_plan(PagedPlan* p, const attn_paged_args* a, const PagedWs& wl, char* ws, int W, int* status) {
  memset(p, 0, sizeof(*p));
  DecodePlan& d = p->d;
  d.R = a->n_rows; d.Hq = a->n_head_q; d.Hkv = a->n_head_kv; d.G = a->n_head_q / a->n_head_kv; d.D = a->head_dim;
  d.N = a->n_pages * a->page_size;
  d.q = QSpec{a->q, a->q_type, a->q_stride_row, a->q_stride_head};
  d.out = OutSpec{a->out, a->out_type, a->o_stride_row, a->o_stride_head};
  d.f.row_begin = a->row_begin;
  d.f.row_end = a->row_end;
  d.lg = Logits{a->scale, a->softcap, a->alibi_slopes, a->sinks};
  d.kv_type = a->kv_type;
  d.k_scale = a->k_scale; d.v_scale = a->v_scale; d.scale_sc = a->scale_stride_cell;
  d.status = status;
  d.W = W;
  d.row_tiles = reinterpret_cast<int64_t*>(ws + wl.tiles_off);
  d.part.o = reinterpret_cast<float*>(ws + wl.o_off);
  d.part.ml = reinterpret_cast<float*>(ws + wl.ml_off);
  d.plan_inline = a->n_rows <= 64 ? 1 : 0;   // kInlineRows of the stream kernel
  p->P = a->page_size; p->n_pages = a->n_pages;
  p->table = a->page_table; p->table_sr = a->table_stride;
  p->n_tables = a->n_tables; p->width = a->table_width;
  p->row_table = a->row_table;
  p->stall_ns = (uint64_t)a->reserved[0] * 1000ull;
}

// The plan of the shared part (the softcap's series as in api.cu: the odd
// Taylor terms of c tanh(scale s / c) in the raw product s, times log2(e)).
void fill_shared(SharedPlan* sp, const PagedPlan& p, const attn_paged_args* a, const SharedWs& w, char* ws, int sms) {
  memset(sp, 0, sizeof(*sp));
  sp->p = p;
  sp->p.own_lo = nullptr;
  sp->p.stall_ns = 0;
  sp->n_groups = a->n_groups;
  sp->group_begin = a->group_begin; sp->group_len = a->group_len;
  sp->n_slot = shared_slots(a->head_dim);
  sp->rpt = 128 / p.d.G;
  sp->block_rows = (int32_t)shared_block_rows(a);
  sp->blocks = reinterpret_cast<SharedBlock*>(ws + w.blocks_off);
  sp->blk_off = reinterpret_cast<int64_t*>(ws + w.off_off);
  sp->max_blk = (int32_t)shared_max_blocks(a);
  sp->runs = reinterpret_cast<SharedRun*>(ws + w.runs_off);
  sp->unit_runs = reinterpret_cast<int2*>(ws + w.unit_off);
  sp->row_blk = reinterpret_cast<int32_t*>(ws + w.blk_off);
  sp->own_lo = reinterpret_cast<int32_t*>(ws + w.own_off);
  sp->rec_o = reinterpret_cast<float*>(ws + w.o_off);
  sp->rec_ml = reinterpret_cast<float*>(ws + w.ml_off);
  sp->W = sms;
  sp->box_cells = 16;
  while (sp->box_cells < 128 && a->page_size % (2 * sp->box_cells) == 0) sp->box_cells *= 2;
  const double L2E = 1.4426950408889634, sc = a->scale, c = a->softcap;
  sp->scale2 = (float)(sc * L2E);
  sp->plain = !(a->softcap > 0.f) && !a->alibi_slopes && sp->scale2 > 1e-30f && sp->scale2 < 1e30f;
  if (a->softcap > 0.f) {
    const double s2 = sc * sc / (c * c);
    const double c3 = -1.0 / 3.0 * sc * s2 * L2E, c5 = 2.0 / 15.0 * sc * s2 * s2 * L2E;
    const double c7 = -17.0 / 315.0 * sc * s2 * s2 * s2 * L2E, c9 = 62.0 / 2835.0 * sc * s2 * s2 * s2 * s2 * L2E;
    const double lim = 0.4 * c / std::fabs(sc);
    auto normal = [](double v) { return std::fabs(v) >= 1.1754943508222875e-38 && std::fabs(v) <= 3.0e38; };
    if (normal(sc) && normal(c3) && normal(c5) && normal(c7) && normal(c9) && normal(lim) && normal(lim * lim)) {
      sp->c3 = (float)c3; sp->c5 = (float)c5; sp->c7 = (float)c7; sp->c9 = (float)c9;
      sp->s_lim = (float)lim;
    }
  }
  sp->stall_ns = (uint64_t)a->reserved[0] * 1000ull;
  const int64_t ovec = 16 / esize(a->out_type);
  sp->out_vec = aligned16(a->out) && (a->n_rows <= 1 || a->o_stride_row % ovec == 0) &&
                (a->n_head_q <= 1 || a->o_stride_head % ovec == 0);
}

// Q as [rows][heads][D] with boxes of 128 / G rows of the G heads of a KV head.
int32_t q_map(CUtensorMap* map, const attn_paged_args* a, int G) {
  const int D = a->head_dim;
  const int64_t dims[3] = {D, a->n_head_q, a->n_rows};
  const int64_t strides[2] = {(a->n_head_q > 1 ? a->q_stride_head : D) * 2, (a->n_rows > 1 ? a->q_stride_row : D) * 2};
  const int32_t box[3] = {64, G, 128 / G};
  return encode_map(map, a->q, a->q_type, 3, dims, strides, box);
}

int32_t run_paged(const attn_paged_args* a, int32_t op, void* ws, size_t ws_bytes, void* stream) {
  int32_t st = check_paged(a, op);
  if (st != ATTN_OK) return st;
  if (a->n_rows == 0) return ATTN_OK;
  int sms = 0, *status = nullptr;
  if ((st = device_facts(&sms, &status)) != ATTN_OK) return st;
  const int W = paged_stream_warps(a->kv_type, a->head_dim, a->n_head_q / a->n_head_kv, sms);
  const PagedWs wl = paged_ws(a, W);
  const bool shared = runs_shared(a, op);
  const SharedWs sw = shared ? shared_ws(a, wl.total, sms) : SharedWs{};
  const size_t need = shared ? sw.total : wl.total;
  if (ws == nullptr || ws_bytes < need)
    return refuse(ATTN_ERR_WORKSPACE, "paged decode needs %zu workspace bytes, got %zu", need, ws_bytes);
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return refuse(ATTN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  CUtensorMap tmK, tmV;
  memset(&tmK, 0, sizeof(tmK));
  memset(&tmV, 0, sizeof(tmV));
  PagedPlan p;
  fill_plan(&p, a, wl, static_cast<char*>(ws), W, status);
  if (a->n_pages > 0) {
    if ((st = pool_map(&tmK, a->k, a, 16)) != ATTN_OK) return st;
    if ((st = pool_map(&tmV, a->v, a, 16)) != ATTN_OK) return st;
  } else {
    p.width = 0;   // no pages: every range is empty
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (shared) {
    SharedPlan sp;
    fill_shared(&sp, p, a, sw, static_cast<char*>(ws), sms);
    CUtensorMap tmQ, sK, sV;
    if ((st = q_map(&tmQ, a, p.d.G)) != ATTN_OK) return st;
    if ((st = pool_map(&sK, a->k, a, sp.box_cells)) != ATTN_OK) return st;
    if ((st = pool_map(&sV, a->v, a, sp.box_cells)) != ATTN_OK) return st;
    if ((e = launch_shared(sp, tmQ, sK, sV, s)) != cudaSuccess)
      return refuse(ATTN_ERR_CUDA, "shared decode launch: %s", cudaGetErrorString(e));
    p.stall_ns = 0;             // (sp's own is the test's)
    p.own_lo = sp.own_lo;       // the stream kernel takes the rows' own cells, planned above
    p.d.plan_inline = 0;
    if ((e = launch_paged_stream(p, tmK, tmV, s)) != cudaSuccess)
      return refuse(ATTN_ERR_CUDA, "paged decode launch: %s", cudaGetErrorString(e));
    if ((e = launch_paged_combine(&sp, p, sms, s)) != cudaSuccess)
      return refuse(ATTN_ERR_CUDA, "combine launch: %s", cudaGetErrorString(e));
    return ATTN_OK;
  }
  e = launch_paged_stream(p, tmK, tmV, s);
  if (e != cudaSuccess) return refuse(ATTN_ERR_CUDA, "paged decode launch: %s", cudaGetErrorString(e));
  e = launch_paged_combine(nullptr, p, sms, s);
  if (e != cudaSuccess) return refuse(ATTN_ERR_CUDA, "combine launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int32_t attn_page_tables(const attn_page_args* a, void* stream) {
  int32_t st = check_pages(a);
  if (st != ATTN_OK) return st;
  int sms = 0, *status = nullptr;
  if ((st = device_facts(&sms, &status)) != ATTN_OK) return st;
  const PageTablesPlan p{*a, status};
  const cudaError_t e = launch_page_tables(p, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return refuse(ATTN_ERR_CUDA, "page_tables launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

int32_t attn_append_paged(const attn_append_args* a, void* stream) {
  int32_t st = check_append(a);
  if (st != ATTN_OK) return st;
  if (a->n_rows == 0 || a->n_pages == 0) return ATTN_OK;
  int sms = 0, *status = nullptr;
  if ((st = device_facts(&sms, &status)) != ATTN_OK) return st;
  const cudaError_t e = launch_append_paged(*a, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return refuse(ATTN_ERR_CUDA, "append_paged launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

int32_t attn_paged_supports(const attn_paged_args* a, int32_t op) { return check_paged(a, op); }

size_t attn_paged_workspace_size(const attn_paged_args* a, int32_t op) {
  if (check_paged(a, op) != ATTN_OK || a->n_rows == 0) return 0;
  int sms = 148, *status = nullptr;
  device_facts(&sms, &status);
  const size_t n = paged_ws(a, paged_stream_warps(a->kv_type, a->head_dim, a->n_head_q / a->n_head_kv, sms)).total;
  return runs_shared(a, op) ? shared_ws(a, n, sms).total : n;
}

int32_t attn_decode_paged(const attn_paged_args* a, void* ws, size_t ws_bytes, void* stream) {
  return run_paged(a, ATTN_OP_DECODE_PAGED, ws, ws_bytes, stream);
}

int32_t attn_decode_shared(const attn_paged_args* a, void* ws, size_t ws_bytes, void* stream) {
  return run_paged(a, ATTN_OP_DECODE_SHARED, ws, ws_bytes, stream);
}

}  // extern "C"
