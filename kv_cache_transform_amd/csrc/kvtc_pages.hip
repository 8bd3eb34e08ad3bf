// Kernels of the paged-cache calls: block tables and slot maps, the write of
// new rows, key bounds per page, and the selection of pages by a score on
// those bounds. (Attention over the pages: kvtc_attend.hip.)
#include "kvtc_pages_device.h"

namespace kvtc {
namespace {

// ------------------------------------------------- block tables, slot maps ---

// Each workgroup scans the requests' growth (tokens) and need (pages) into
// LDS, which is cheaper than a launch before it, and then fills its share of
// the table entries and slots, each found by a binary search in the scans.
__global__ void __launch_bounds__(kPageThreads) tables_kernel(kvtc_page_plan a) {
  extern __shared__ uint32_t lds[];
  __shared__ uint64_t part[kPageThreads / 64];
  uint32_t* start = lds;                       // first token of each request
  uint32_t* page = lds + a.n_requests;         // first page of each request, behind free_from
  const int bs = a.block_size;
  const int64_t from = a.free_from ? max(a.free_from[0], 0) : 0;
  const uint64_t kCap = 0xFFFFFFFFull;         // past every n_slots and n_free
  uint64_t tokens = 0, needed = 0, taken = 0;
  for (int base = 0; base < a.n_requests; base += kPageThreads) {
    const int i = base + (int)threadIdx.x;
    int old = 0, now = 0;
    bool ok = false;
    if (i < a.n_requests) {
      old = a.old_lens ? a.old_lens[i] : 0;
      now = a.new_lens[i];
      ok = old >= 0 && now >= old && now <= a.table_width * bs;
    }
    const uint64_t grow = ok ? now - old : 0;
    const uint64_t need = ok ? pages_of(now, bs) - pages_of(old, bs) : 0;
    uint64_t sum_t, sum_p, sum_g;
    const uint64_t t0 = tokens + scan_threads(grow, part, &sum_t);
    const uint64_t p0 = needed + scan_threads(need, part, &sum_p);
    const bool fits = t0 + grow <= (uint64_t)a.n_slots && (need == 0 || from + p0 + need <= (uint64_t)a.n_free);
    scan_threads(ok && fits ? need : (uint64_t)0, part, &sum_g);
    if (i < a.n_requests) {
      start[i] = (uint32_t)min(t0, kCap);
      page[i] = (uint32_t)min(p0, kCap);
      if (blockIdx.x == 0) {
        if (a.starts) a.starts[i] = (int32_t)min(t0, (uint64_t)INT32_MAX);
        if (!ok) set_status(a.status, i, KVTC_E_INVALID);
        else if (!fits) set_status(a.status, i, KVTC_E_CAPACITY);
      }
    }
    tokens += sum_t;
    needed += sum_p;
    taken += sum_g;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (a.starts) a.starts[a.n_requests] = (int32_t)min(tokens, (uint64_t)INT32_MAX);
    if (a.taken) *a.taken = (int32_t)taken;
  }
  __syncthreads();
  const uint32_t stride = gridDim.x * kPageThreads, me = blockIdx.x * kPageThreads + threadIdx.x;
  // pages given out: requests are served in order, so they are the first `taken` needed ones
  for (uint64_t e = me; e < taken; e += stride) {
    const int i = owner_of(page, a.n_requests, (uint32_t)e);
    const int at = pages_of(a.old_lens ? a.old_lens[i] : 0, bs) + (int)((uint32_t)e - page[i]);
    a.block_table[(size_t)i * a.table_stride + at] = a.free_blocks[from + e];
  }
  for (uint64_t t = me; t < (uint64_t)a.n_slots; t += stride) {
    int slot = -1;
    if (t < tokens) {
      const int i = owner_of(start, a.n_requests, (uint32_t)t);
      const int old = a.old_lens ? a.old_lens[i] : 0, now = a.new_lens[i];
      const int p = old + (int)((uint32_t)t - start[i]), at = p / bs, had = pages_of(old, bs);
      const uint32_t need = pages_of(now, bs) - had;
      const bool fits = (uint64_t)start[i] + (now - old) <= (uint64_t)a.n_slots &&
                        (need == 0 || from + (uint64_t)page[i] + need <= (uint64_t)a.n_free);
      if (fits) {
        const int id = at < had ? a.block_table[(size_t)i * a.table_stride + at]
                                : a.free_blocks[from + page[i] + (at - had)];
        if (id >= 0 && id < a.n_blocks) slot = id * bs + p % bs;
        else set_status(a.status, i, KVTC_E_INVALID);
      }
    }
    a.slots[t] = slot;
  }
}

// ------------------------------------------------------------ write of rows ---

template <class S, class D>
__global__ void __launch_bounds__(kPageThreads) write_kernel(kvtc_pages p, kvtc_page_rows r) {
  const int F = p.kv_heads * p.head_dim;
  const int64_t rows = (int64_t)p.n_blocks * p.block_size;
  for (int64_t i = blockIdx.x; i < r.n_rows; i += gridDim.x) {
    const int64_t slot = r.slots[i];
    if (slot >= rows && threadIdx.x == 0) set_status(r.status, 0, KVTC_E_INVALID);
    if (slot < 0 || slot >= rows) continue;
    const S* ks = (const S*)r.k + i * r.k_stride;
    const S* vs = (const S*)r.v + i * r.v_stride;
    D* kd = (D*)p.k + slot * F;
    D* vd = (D*)p.v + slot * F;
    for (int f = threadIdx.x; f < F; f += kPageThreads) {
      Elem<D>::put(kd + f, Elem<S>::get(ks + f));
      Elem<D>::put(vd + f, Elem<S>::get(vs + f));
    }
  }
}

// -------------------------------------------------------------- key bounds ---

template <class T>
__global__ void __launch_bounds__(kPageThreads) bounds_kernel(kvtc_pages p, kvtc_requests r, const int32_t* from, T* bounds) {
  const int i = blockIdx.y, bs = p.block_size, F = p.kv_heads * p.head_dim;
  const int len = checked_len(r, bs, i);
  if (len < 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(r.status, i, KVTC_E_INVALID);
    return;
  }
  const int a = from ? max(from[i], 0) / bs : 0;
  for (int64_t j = a + (int64_t)blockIdx.x; j * bs < len; j += gridDim.x) {
    const int id = r.block_table[(int64_t)i * r.table_stride + j];
    if (id < 0 || id >= p.n_blocks) {
      if (threadIdx.x == 0) set_status(r.status, i, KVTC_E_INVALID);
      continue;
    }
    const int rows = min((int64_t)bs, len - j * bs);
    for (int f = threadIdx.x; f < F; f += kPageThreads) {
      const T* k = (const T*)p.k + (int64_t)id * bs * F + f;
      float lo = Elem<T>::get(k), hi = lo;
      bool nan = lo != lo;
      for (int t = 1; t < rows; ++t) {
        const float x = Elem<T>::get(k + (int64_t)t * F);
        nan |= x != x;
        lo = fminf(lo, x);
        hi = fmaxf(hi, x);
      }
      if (nan) lo = hi = __uint_as_float(0x7FC00000u);
      Elem<T>::put(bounds + ((int64_t)id * 2) * F + f, lo);
      Elem<T>::put(bounds + ((int64_t)id * 2 + 1) * F + f, hi);
    }
  }
}

// ------------------------------------------------------- selection of pages ---

// An unsigned integer that orders like the score: NaN above every number,
// pages that are kept always above that; 0 is left for "never".
constexpr uint32_t kKeyKeep = 0xFFFFFFFFu, kKeyNan = 0xFFFFFFFEu;
__device__ __forceinline__ uint32_t score_key(double s) {
  const float f = (float)s + 0.0f;             // -0 counts as 0
  const uint32_t u = __float_as_uint(f);
  return f != f ? kKeyNan : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One workgroup per (KV head, request): a wave scores a page at a time, then
// the threshold is found bit by bit and the pages above it listed in order.
template <class T>
__global__ void __launch_bounds__(kPageThreads) select_kernel(kvtc_pages p, kvtc_requests r, kvtc_queries q, const T* bounds, kvtc_selection sel, uint32_t* keys) {
  __shared__ uint64_t part[kPageThreads / 64];
  __shared__ double up[KVTC_MAX_HEAD_DIM], down[KVTC_MAX_HEAD_DIM];
  const int h = blockIdx.x, i = blockIdx.y, bs = p.block_size, D = p.head_dim, F = p.kv_heads * D;
  const int G = q.q_heads / p.kv_heads, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int len = checked_len(r, bs, i);
  if (len < 0) {
    if (threadIdx.x == 0) set_status(r.status, i, KVTC_E_INVALID);
    len = 0;
  }
  const int n = pages_of(len, bs);
  for (int d = threadIdx.x; d < D; d += kPageThreads) {
    double u = 0, w = 0;
    for (int g = 0; g < G; ++g) {
      const float x = Elem<T>::get((const T*)q.q + i * q.q_stride + (int64_t)(h * G + g) * D + d);
      // (a NaN enters both sums)
      u += x < 0 ? 0.0 : (double)x;
      w += x > 0 ? 0.0 : (double)x;
    }
    up[d] = u;
    down[d] = w;
  }
  __syncthreads();
  uint32_t* key = keys + ((int64_t)i * p.kv_heads + h) * r.table_width;
  for (int j = wave; j < n; j += kPageThreads / 64) {
    const int id = r.block_table[(int64_t)i * r.table_stride + j];
    const bool ok = id >= 0 && id < p.n_blocks;
    double s = 0;
    if (ok)
      for (int d = lane; d < D; d += 64) {
        const T* b = bounds + (int64_t)id * 2 * F + h * D + d;
        s += up[d] * (double)Elem<T>::get(b + F) + down[d] * (double)Elem<T>::get(b);
      }
    for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m, 64);
    if (lane == 0) {
      key[j] = !ok ? 0u : j < sel.first || j >= n - sel.last ? kKeyKeep : score_key(s);
      if (!ok) set_status(r.status, i, KVTC_E_INVALID);
    }
  }
  __syncthreads();
  // the largest threshold that at least `budget` keys reach (0 with fewer)
  uint32_t least = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t t = least | (1u << bit);
    uint64_t mine = 0, all;
    for (int j = threadIdx.x; j < n; j += kPageThreads) mine += key[j] >= t;
    scan_threads(mine, part, &all);
    if (all >= (uint64_t)sel.budget) least = t;
  }
  uint64_t above = 0;
  {
    uint64_t mine = 0;
    for (int j = threadIdx.x; j < n; j += kPageThreads) mine += key[j] > least;
    scan_threads(mine, part, &above);
  }
  // those above it, and of those at it the first ones
  const uint64_t ties = least ? sel.budget - above : 0;
  int32_t* out = sel.blocks + ((int64_t)i * p.kv_heads + h) * sel.budget;
  uint64_t done = 0, tied = 0;
  for (int base = 0; base < n; base += kPageThreads) {
    const int j = base + (int)threadIdx.x;
    const uint32_t k = j < n ? key[j] : 0u;
    const bool tie = k && k == least;
    uint64_t sum;
    const uint64_t before = tied + scan_threads((uint64_t)tie, part, &sum);
    tied += sum;
    const bool take = k && (k > least || (tie && before < ties));
    const uint64_t at = done + scan_threads((uint64_t)take, part, &sum);
    done += sum;
    if (take) out[at] = j;
  }
  for (int j = (int)done + (int)threadIdx.x; j < sel.budget; j += kPageThreads) out[j] = -1;
}

int grid_for(int64_t n, int most) { return (int)std::min<int64_t>(std::max<int64_t>(n, 1), most); }

}  // namespace

int launch_page_tables(const kvtc_page_plan& a, hipStream_t s) {
  const size_t lds = (size_t)a.n_requests * 8;
  const int grid = grid_for(((int64_t)a.n_slots + 4 * kPageThreads - 1) / (4 * kPageThreads), 1024);
  hipLaunchKernelGGL(tables_kernel, dim3(grid), dim3(kPageThreads), lds, s, a);
  return (int)hipGetLastError();
}

int launch_page_write(const kvtc_pages& p, const kvtc_page_rows& r, hipStream_t s) {
  const int grid = grid_for(r.n_rows, 4096);
  if (p.dtype == KVTC_F32 && r.dtype == KVTC_F32)
    hipLaunchKernelGGL((write_kernel<float, float>), dim3(grid), dim3(kPageThreads), 0, s, p, r);
  else if (p.dtype == KVTC_F32)
    hipLaunchKernelGGL((write_kernel<uint16_t, float>), dim3(grid), dim3(kPageThreads), 0, s, p, r);
  else if (r.dtype == KVTC_F32)
    hipLaunchKernelGGL((write_kernel<float, uint16_t>), dim3(grid), dim3(kPageThreads), 0, s, p, r);
  else
    hipLaunchKernelGGL((write_kernel<uint16_t, uint16_t>), dim3(grid), dim3(kPageThreads), 0, s, p, r);
  return (int)hipGetLastError();
}

int launch_page_bounds(const kvtc_pages& p, const kvtc_requests& r, const int32_t* from, void* bounds, hipStream_t s) {
  const dim3 grid(grid_for(r.table_width, std::max(1, 8192 / r.n_requests)), r.n_requests);
  if (p.dtype == KVTC_F32)
    hipLaunchKernelGGL(bounds_kernel<float>, grid, dim3(kPageThreads), 0, s, p, r, from, (float*)bounds);
  else
    hipLaunchKernelGGL(bounds_kernel<uint16_t>, grid, dim3(kPageThreads), 0, s, p, r, from, (uint16_t*)bounds);
  return (int)hipGetLastError();
}

int launch_page_select(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q, const void* bounds,
                       const kvtc_selection& sel, void* ws, hipStream_t s) {
  const dim3 grid(p.kv_heads, r.n_requests);
  if (p.dtype == KVTC_F32)
    hipLaunchKernelGGL(select_kernel<float>, grid, dim3(kPageThreads), 0, s, p, r, q, (const float*)bounds, sel, (uint32_t*)ws);
  else
    hipLaunchKernelGGL(select_kernel<uint16_t>, grid, dim3(kPageThreads), 0, s, p, r, q, (const uint16_t*)bounds, sel, (uint32_t*)ws);
  return (int)hipGetLastError();
}

}  // namespace kvtc
