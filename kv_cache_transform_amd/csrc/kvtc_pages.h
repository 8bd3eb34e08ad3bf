// Shared by the paged-cache calls' host checks (kvtc_pages_host.cpp) and
// their kernels (kvtc_pages.hip): kernel arguments, workspace layout and
// launchers.
#pragma once

#include "kvtc_internal.h"

namespace kvtc {

constexpr int kPageThreads = 256;

// Scores of kvtc_page_select: one ordered 32-bit key per (request, KV head,
// table entry).
__host__ __device__ inline size_t select_ws_bytes(const kvtc_pages& p, const kvtc_requests& r) {
  return align_up((size_t)r.n_requests * p.kv_heads * r.table_width * 4, kAlign);
}

// Every launcher returns a hipError_t value cast to int.
int launch_page_tables(const kvtc_page_plan& a, hipStream_t s);
int launch_page_write(const kvtc_pages& p, const kvtc_page_rows& r, hipStream_t s);
int launch_page_bounds(const kvtc_pages& p, const kvtc_requests& r, const int32_t* from, void* bounds, hipStream_t s);
int launch_page_select(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q, const void* bounds,
                       const kvtc_selection& sel, void* ws, hipStream_t s);
int launch_page_attend(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q, const kvtc_selection& sel,
                       void* ws, hipStream_t s);

}  // namespace kvtc
