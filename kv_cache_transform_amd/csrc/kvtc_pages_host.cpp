// Host side of the paged-cache calls: argument checks, sizes and launches.
// Nothing here allocates or throws apart from the error message.
#include <cmath>
#include <cstdio>

#include "kvtc_pages.h"

using namespace kvtc;

namespace {

// Tokens of a table row, and entries of all rows: small enough that the
// kernels' positions a few tiles past an end stay in 32 bits.
constexpr int64_t kMostEntries = (int64_t)1 << 30;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
size_t elem_bytes(int dtype) { return dtype == KVTC_F32 ? 4 : 2; }
bool is_dtype(int d) { return d == KVTC_F32 || d == KVTC_BF16; }

// Launches go to the stream's device, which need not be the calling thread's
// current one; that one is current again afterwards.
struct OnDeviceOf {
  int before = -1;
  explicit OnDeviceOf(hipStream_t s) {
    hipDevice_t of = 0;
    int now = 0;
    if (!s || hipGetDevice(&now) != hipSuccess || hipStreamGetDevice(s, &of) != hipSuccess || of == now) return;
    if (hipSetDevice(of) == hipSuccess) before = now;
  }
  ~OnDeviceOf() {
    if (before >= 0) (void)hipSetDevice(before);
  }
};

template <class L>
kvtc_status enqueue(hipStream_t s, const char* what, L launch) {
  OnDeviceOf guard(s);
  const int e = launch();
  if (e == 0) return KVTC_OK;
  char msg[160];
  std::snprintf(msg, sizeof(msg), "%s: %s", what, hipGetErrorString((hipError_t)e));
  return report(KVTC_E_HIP, msg);
}

size_t row_elems(const kvtc_pages& p) { return (size_t)p.kv_heads * p.head_dim; }

// v: whether the call uses the V pages; data: whether it uses page memory at all
kvtc_status check_pages(const kvtc_pages* p, bool v, bool data) {
  if (!p) return report(KVTC_E_INVALID, "null pages");
  if (!is_dtype(p->dtype)) return report(KVTC_E_INVALID, "pages: bad dtype");
  if (p->n_blocks <= 0 || p->block_size <= 0) return report(KVTC_E_INVALID, "pages: bad n_blocks or block_size");
  if (p->kv_heads <= 0 || p->head_dim <= 0) return report(KVTC_E_INVALID, "pages: bad kv_heads or head_dim");
  if (p->head_dim % 8 || p->head_dim > KVTC_MAX_HEAD_DIM)
    return report(KVTC_E_UNSUPPORTED, "pages: head_dim must be a multiple of 8 up to KVTC_MAX_HEAD_DIM");
  if (p->kv_heads > 65535) return report(KVTC_E_UNSUPPORTED, "pages: more than 65535 heads");
  if ((int64_t)p->n_blocks * p->block_size > (int64_t)INT32_MAX)
    return report(KVTC_E_UNSUPPORTED, "pages: 2^31 rows or more");
  if (!data) return KVTC_OK;
  if (!p->k || !aligned16(p->k) || (v && (!p->v || !aligned16(p->v))))
    return report(KVTC_E_INVALID, "pages: k and v must be non-null and 16-byte aligned");
  const size_t need = (size_t)p->n_blocks * p->block_size * row_elems(*p) * elem_bytes(p->dtype);
  if (p->k_capacity < need || (v && p->v_capacity < need))
    return report(KVTC_E_CAPACITY, "pages: capacity below n_blocks * block_size rows");
  return KVTC_OK;
}

kvtc_status check_count(int32_t n) {
  if (n <= 0) return report(KVTC_E_INVALID, "bad number of requests");
  if (n > KVTC_MAX_JOBS) return report(KVTC_E_CAPACITY, "more than KVTC_MAX_JOBS requests");
  return KVTC_OK;
}

kvtc_status check_requests(const kvtc_requests* r, const kvtc_pages& p, bool data) {
  if (!r) return report(KVTC_E_INVALID, "null requests");
  const kvtc_status st = check_count(r->n_requests);
  if (st != KVTC_OK) return st;
  if (r->table_width <= 0 || r->table_stride < r->table_width)
    return report(KVTC_E_INVALID, "requests: bad table_width or table_stride");
  if ((int64_t)r->table_width * p.block_size >= kMostEntries || (int64_t)r->table_width * r->n_requests >= kMostEntries)
    return report(KVTC_E_UNSUPPORTED, "requests: a table row of 2^30 tokens, or 2^30 table entries, or more");
  if (!data) return KVTC_OK;
  if (!r->block_table || !r->lens || !aligned4(r->block_table) || !aligned4(r->lens) || !aligned4(r->status))
    return report(KVTC_E_INVALID, "requests: block_table and lens must be non-null, all 4-byte aligned");
  return KVTC_OK;
}

kvtc_status check_queries(const kvtc_queries* q, const kvtc_pages& p, const kvtc_requests& r, bool out, bool data,
                          kvtc_queries* dense) {
  if (!q) return report(KVTC_E_INVALID, "null queries");
  if (q->q_heads <= 0 || q->q_heads % p.kv_heads || q->q_heads > 65535)
    return report(KVTC_E_INVALID, "queries: q_heads must be a positive multiple of kv_heads below 2^16");
  *dense = *q;
  const int64_t row = (int64_t)q->q_heads * p.head_dim;
  if (!dense->q_stride) dense->q_stride = row;
  if (!dense->out_stride) dense->out_stride = row;
  if (dense->q_stride < row || dense->q_stride % 8 || (out && (dense->out_stride < row || dense->out_stride % 8)))
    return report(KVTC_E_INVALID, "queries: strides must cover a row and be multiples of 8");
  if (attend_most_chunks(p, r, *q) >= (int64_t)INT32_MAX)
    return report(KVTC_E_UNSUPPORTED, "requests * heads * tokens of the tables past the kernels' 2^31 chunks");
  if (!data) return KVTC_OK;
  if (!q->q || !aligned16(q->q) || (out && (!q->out || !aligned16(q->out) || !aligned4(q->lse))))
    return report(KVTC_E_INVALID, "queries: q and out must be non-null and 16-byte aligned");
  if (out && !std::isfinite(q->scale)) return report(KVTC_E_INVALID, "queries: scale must be finite");
  return KVTC_OK;
}

kvtc_status check_selection(const kvtc_selection* s, bool keep, bool data) {
  if (s->budget <= 0) return report(KVTC_E_INVALID, "selection: budget must be positive");
  if (keep && (s->first < 0 || s->last < 0 || (int64_t)s->first + s->last > s->budget))
    return report(KVTC_E_INVALID, "selection: first and last must be >= 0 and fit in the budget");
  if (data && (!s->blocks || !aligned4(s->blocks)))
    return report(KVTC_E_INVALID, "selection: blocks must be non-null and 4-byte aligned");
  return KVTC_OK;
}

kvtc_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || !aligned16(ws)) return report(KVTC_E_INVALID, "workspace must be non-null and aligned");
  if (have < need) return report(KVTC_E_CAPACITY, "workspace below kvtc_page_workspace_bytes");
  return KVTC_OK;
}

size_t workspace_bytes(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q, const kvtc_selection* s) {
  const size_t a = attend_ws_bytes(p, r, q), b = s ? select_ws_bytes(p, r) : 0;
  return a > b ? a : b;
}

}  // namespace

extern "C" {

kvtc_status kvtc_page_tables(const kvtc_page_plan* a, hipStream_t stream) {
  if (!a) return report(KVTC_E_INVALID, "null plan");
  const kvtc_status st = check_count(a->n_requests);
  if (st != KVTC_OK) return st;
  if (a->block_size <= 0 || a->n_blocks <= 0 || a->n_free < 0 || a->n_slots < 0)
    return report(KVTC_E_INVALID, "plan: bad block_size, n_blocks, n_free or n_slots");
  if (a->table_width <= 0 || a->table_stride < a->table_width)
    return report(KVTC_E_INVALID, "plan: bad table_width or table_stride");
  if (!a->new_lens || !a->block_table || (a->n_free && !a->free_blocks) || (a->n_slots && !a->slots))
    return report(KVTC_E_INVALID, "plan: null new_lens, block_table, free_blocks or slots");
  for (const void* p : {(const void*)a->old_lens, (const void*)a->new_lens, (const void*)a->free_blocks,
                        (const void*)a->free_from, (const void*)a->block_table, (const void*)a->slots,
                        (const void*)a->starts, (const void*)a->taken, (const void*)a->status})
    if (!aligned4(p)) return report(KVTC_E_INVALID, "plan: pointers must be 4-byte aligned");
  if (a->free_from && (a->free_from == a->taken || a->free_from == a->starts))
    return report(KVTC_E_INVALID, "plan: an output overlaps free_from");
  if ((int64_t)a->n_blocks * a->block_size > (int64_t)INT32_MAX)
    return report(KVTC_E_UNSUPPORTED, "plan: 2^31 rows or more");
  if ((int64_t)a->table_width * a->block_size >= kMostEntries || (int64_t)a->table_width * a->n_requests >= kMostEntries)
    return report(KVTC_E_UNSUPPORTED, "plan: a table row of 2^30 tokens, or 2^30 table entries, or more");
  return enqueue(stream, "page tables launch", [&] { return launch_page_tables(*a, stream); });
}

kvtc_status kvtc_page_write(const kvtc_pages* p, const kvtc_page_rows* r, hipStream_t stream) {
  const kvtc_status st = check_pages(p, true, true);
  if (st != KVTC_OK) return st;
  if (!r || r->n_rows < 0 || !is_dtype(r->dtype)) return report(KVTC_E_INVALID, "rows: null, bad n_rows or dtype");
  if (r->n_rows == 0) return KVTC_OK;
  const size_t e = elem_bytes(r->dtype);
  if (!r->k || !r->v || !r->slots || (uintptr_t)r->k % e || (uintptr_t)r->v % e || !aligned4(r->slots) ||
      !aligned4(r->status))
    return report(KVTC_E_INVALID, "rows: k, v and slots must be non-null and aligned to their elements");
  if (r->k_stride < 0 || r->v_stride < 0) return report(KVTC_E_INVALID, "rows: negative stride");
  return enqueue(stream, "page write launch", [&] { return launch_page_write(*p, *r, stream); });
}

kvtc_status kvtc_page_bounds(const kvtc_pages* p, const kvtc_requests* r, const int32_t* from_lens, void* bounds,
                             size_t bounds_capacity, hipStream_t stream) {
  kvtc_status st = check_pages(p, false, true);
  if (st == KVTC_OK) st = check_requests(r, *p, true);
  if (st != KVTC_OK) return st;
  if (!bounds || !aligned16(bounds) || !aligned4(from_lens))
    return report(KVTC_E_INVALID, "bounds must be non-null and 16-byte aligned");
  if (bounds_capacity < (size_t)p->n_blocks * 2 * row_elems(*p) * elem_bytes(p->dtype))
    return report(KVTC_E_CAPACITY, "bounds_capacity below n_blocks * 2 rows");
  return enqueue(stream, "page bounds launch", [&] { return launch_page_bounds(*p, *r, from_lens, bounds, stream); });
}

size_t kvtc_page_workspace_bytes(const kvtc_pages* p, const kvtc_requests* r, const kvtc_queries* q,
                                 const kvtc_selection* s) {
  kvtc_queries dense;
  if (check_pages(p, false, false) != KVTC_OK || check_requests(r, *p, false) != KVTC_OK ||
      check_queries(q, *p, *r, false, false, &dense) != KVTC_OK || (s && check_selection(s, false, false) != KVTC_OK))
    return 0;
  return workspace_bytes(*p, *r, dense, s);
}

kvtc_status kvtc_page_select(const kvtc_pages* p, const kvtc_requests* r, const kvtc_queries* q, const void* bounds,
                             size_t bounds_capacity, const kvtc_selection* s, void* d_ws, size_t ws_bytes,
                             hipStream_t stream) {
  kvtc_queries dense;
  kvtc_status st = check_pages(p, false, false);
  if (st == KVTC_OK) st = check_requests(r, *p, true);
  if (st == KVTC_OK) st = check_queries(q, *p, *r, false, true, &dense);
  if (st != KVTC_OK) return st;
  if (!s) return report(KVTC_E_INVALID, "null selection");
  st = check_selection(s, true, true);
  if (st != KVTC_OK) return st;
  if (!bounds || !aligned16(bounds)) return report(KVTC_E_INVALID, "bounds must be non-null and 16-byte aligned");
  if (bounds_capacity < (size_t)p->n_blocks * 2 * row_elems(*p) * elem_bytes(p->dtype))
    return report(KVTC_E_CAPACITY, "bounds_capacity below n_blocks * 2 rows");
  st = check_workspace(d_ws, ws_bytes, workspace_bytes(*p, *r, dense, s));
  if (st != KVTC_OK) return st;
  return enqueue(stream, "page select launch",
                 [&] { return launch_page_select(*p, *r, dense, bounds, *s, d_ws, stream); });
}

kvtc_status kvtc_page_attend(const kvtc_pages* p, const kvtc_requests* r, const kvtc_queries* q,
                             const kvtc_selection* s, void* d_ws, size_t ws_bytes, hipStream_t stream) {
  kvtc_queries dense;
  kvtc_status st = check_pages(p, true, true);
  if (st == KVTC_OK) st = check_requests(r, *p, true);
  if (st == KVTC_OK) st = check_queries(q, *p, *r, true, true, &dense);
  if (st == KVTC_OK && s) st = check_selection(s, false, true);
  if (st == KVTC_OK) st = check_workspace(d_ws, ws_bytes, workspace_bytes(*p, *r, dense, nullptr));
  if (st != KVTC_OK) return st;
  const kvtc_selection none = {nullptr, 0, 0, 0};
  return enqueue(stream, "page attend launch",
                 [&] { return launch_page_attend(*p, *r, dense, s ? *s : none, d_ws, stream); });
}

}  // extern "C"
