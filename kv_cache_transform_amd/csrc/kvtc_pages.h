// Shared by the paged-cache calls' host checks (kvtc_pages_host.cpp) and
// their kernels (kvtc_pages.hip): kernel arguments, workspace layout and
// launchers.
#pragma once

#include "kvtc_internal.h"

namespace kvtc {

// Set kvtc_last_error's message of this thread and return st (kvtc_host.cpp).
kvtc_status report(kvtc_status st, const char* msg);

constexpr int kPageThreads = 256;

// Scores of kvtc_page_select: one ordered 32-bit key per (request, KV head,
// table entry).
__host__ __device__ inline size_t select_ws_bytes(const kvtc_pages& p, const kvtc_requests& r) {
  return align_up((size_t)r.n_requests * p.kv_heads * r.table_width * 4, kAlign);
}

// kvtc_page_attend: the number of workgroups, their waves, positions per chunk
// of work (a tile of 32, in fp32 16, per wave), the chunks that a short row
// counts as more than it has, and head_dim as the kernels round it up. Sizes
// alone decide, so that a workspace can be sized without a device. One
// workgroup of four waves per CU keeps enough loads in flight and leaves the
// fewest pieces to join: 51 us for 16 x 8K tokens against 58 with two and 63
// with three, the same with one of eight waves.
constexpr int kAttendWorkers = 256, kAttendWaves = 4;
constexpr uint32_t kAttendRow = 2;
__host__ __device__ constexpr int attend_dp(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
__host__ __device__ constexpr int attend_chunk(int dtype) { return kAttendWaves * (dtype == KVTC_F32 ? 16 : 32); }
inline int64_t attend_most_chunks(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q) {
  const int64_t ch = attend_chunk(p.dtype), rows = (int64_t)p.kv_heads * ((q.q_heads / p.kv_heads + 15) / 16);
  return r.n_requests * rows * (((int64_t)r.table_width * p.block_size + ch - 1) / ch + kAttendRow);
}
inline uint32_t attend_workers(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q) {
  const int64_t n = attend_most_chunks(p, r, q);
  return (uint32_t)(n < kAttendWorkers ? n : kAttendWorkers);
}
// Workspace: an entry per workgroup, then two pieces of rows per workgroup: gt
// (up to 16) query heads' dp sums each, their gt maxima (base 2) and their gt
// sums of weights, in whole 16 bytes.
__host__ __device__ constexpr size_t part_floats(int gt, int dp) { return ((size_t)gt * (dp + 2) + 3) / 4 * 4; }
inline size_t attend_meta_bytes() { return align_up((size_t)kAttendWorkers * 16, kAlign); }
inline size_t attend_ws_bytes(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q) {
  const int group = q.q_heads / p.kv_heads, gt = group < 16 ? group : 16;
  return attend_meta_bytes() +
         align_up(attend_workers(p, r, q) * 2 * part_floats(gt, attend_dp(p.head_dim)) * 4, kAlign);
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
