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

// Scores of the pages [blockIdx.x * span, + span) of request blockIdx.z for KV
// head blockIdx.y. LP lanes (a power of two) share a page, 16 bytes of each
// bound to a lane, so a load instruction covers whole 16 * LP byte rows; each
// lane keeps its dims' two query sums in fp64. Reading the bounds is what
// it costs: about 60 vector instructions for 2 KB a wave are a third of the
// time that HBM takes for them.
template <class T>
__global__ void __launch_bounds__(kPageThreads) score_kernel(kvtc_pages p, kvtc_requests r, kvtc_queries q, const T* bounds,
                                                             kvtc_selection sel, uint32_t* keys, int span, int LP) {
  constexpr int EL = 16 / sizeof(T);
  typedef T row16 __attribute__((ext_vector_type(EL)));
  const int h = blockIdx.y, i = blockIdx.z, bs = p.block_size, D = p.head_dim, F = p.kv_heads * D;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, d0 = (lane & (LP - 1)) * EL;
  const int len = checked_len(r, bs, i), n = pages_of(len, bs), j0 = (int)blockIdx.x * span;
  if (len < 0 && j0 == 0 && h == 0 && threadIdx.x == 0) set_status(r.status, i, KVTC_E_INVALID);
  if (j0 >= n) return;
  const int j1 = min(n, j0 + span);
  const bool there = d0 < D, all = n <= sel.budget;     // all: every page is selected, whatever its score
  double up[EL], down[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) up[e] = down[e] = 0.0;
  const int G = q.q_heads / p.kv_heads;
  const T* qh = (const T*)q.q + i * q.q_stride + (int64_t)h * G * D + (there ? d0 : 0);
  for (int g = 0; g < G && !all; ++g) {
    const row16 x = *(const row16*)(qh + (int64_t)g * D);
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      const T xe = x[e];
      const float v = Elem<T>::get(&xe);
      up[e] += v < 0 ? 0.0 : (double)v;         // (a NaN enters both sums)
      down[e] += v > 0 ? 0.0 : (double)v;
    }
  }
  uint32_t* key = keys + ((int64_t)i * p.kv_heads + h) * r.table_width;
  const int32_t* table = r.block_table + (int64_t)i * r.table_stride;
  const int step = kPageThreads / LP;
  for (int base = j0; base < j1; base += step) {
    const int j = base + (int)threadIdx.x / LP;
    const int id = j < j1 ? table[j] : -1;
    const bool ok = id >= 0 && id < p.n_blocks;
    const bool keep = all || j < sel.first || j >= n - sel.last;
    double s0 = 0.0, s1 = 0.0;
    if (ok && !keep && there) {
      const T* b = bounds + (int64_t)id * 2 * F + h * D + d0;
      const row16 lo = *(const row16*)b, hi = *(const row16*)(b + F);
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        const T le = lo[e], he = hi[e];
        s0 = fma(down[e], (double)Elem<T>::get(&le), s0);
        s1 = fma(up[e], (double)Elem<T>::get(&he), s1);
      }
    }
    s0 += s1;
    for (int m = LP >> 1; m; m >>= 1) s0 += __shfl_xor(s0, m, 64);
    if (j < j1 && (lane & (LP - 1)) == 0) {
      key[j] = !ok ? 0u : keep ? kKeyKeep : score_key(s0);
      if (!ok) set_status(r.status, i, KVTC_E_INVALID);
    }
  }
}

// The pages of the highest keys, in ascending order: one workgroup per (KV
// head, request). The threshold is found by counting digits of kDigit bits,
// the first over the range that the keys really span, so that they spread
// over the counters (their leading bits, sign and exponent, hardly differ);
// each further digit only among the keys that share those before it. A
// thread has kOwn consecutive keys, in registers for the first kOwn *
// kPickThreads pages; past them they are read again for every digit.
constexpr int kPickThreads = 1024, kOwn = 8, kDigit = 11;

template <class V>
__device__ __forceinline__ V scan_picks(V v, V* part, V* sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  V x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const V y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) part[wave] = x;
  __syncthreads();
  V before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPickThreads / 64; ++w) {
    const V y = part[w];
    if (w < wave) before += y;
    all += y;
  }
  *sum = all;
  return before + x - v;
}

__global__ void __launch_bounds__(kPickThreads) pick_kernel(kvtc_pages p, kvtc_requests r, kvtc_selection sel, const uint32_t* keys) {
  __shared__ uint32_t count[1 << kDigit], part[kPickThreads / 64], found[2], range[2];
  const int h = blockIdx.x, i = blockIdx.y, bs = p.block_size, tid = threadIdx.x;
  const int n = pages_of(checked_len(r, bs, i), bs), span = kOwn * kPickThreads;
  const uint32_t* key = keys + ((int64_t)i * p.kv_heads + h) * r.table_width;
  int32_t* out = sel.blocks + ((int64_t)i * p.kv_heads + h) * sel.budget;
  uint32_t own[kOwn];
  auto read = [&](int base) {      // this thread's keys of pages [base, base + span)
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const int j = base + tid * kOwn + x;
      own[x] = j < n ? key[j] : 0u;
    }
  };
  auto each = [&](auto f) {        // f(key) for every key of this thread
    for (int base = 0; base < n; base += span) {
      if (base || n > span) read(base);
#pragma unroll
      for (int x = 0; x < kOwn; ++x) f(own[x]);
    }
  };
  read(0);
  // Only keys between those that are never taken and those that always are
  // can be the threshold; is there a choice at all?
  if (tid < 2) range[tid] = tid ? 0u : 0xFFFFFFFFu;
  uint32_t lo = 0xFFFFFFFFu, hi = 0u, valid = 0, kept = 0;
  each([&](uint32_t k) {
    valid += k != 0;
    kept += k == kKeyKeep;
    if (k && k != kKeyKeep) {
      lo = min(lo, k);
      hi = max(hi, k);
    }
  });
  uint32_t n_valid, n_kept;
  scan_picks(valid, part, &n_valid);
  scan_picks(kept, part, &n_kept);
  uint32_t least = 1, ties = 0;       // taken: keys above least, and the first `ties` at it
  if (n_valid > (uint32_t)sel.budget) {
    atomicMin(&range[0], lo);
    atomicMax(&range[1], hi);
    uint32_t want = sel.budget - n_kept;       // of the keys in [lo, hi], the host has seen to want >= 0
    __syncthreads();
    lo = range[0];
    hi = range[1];
    if (want == 0) {
      least = kKeyNan;
      ties = 0;
    } else {
      // the keys in question are lo + [0, 2^bits)
      int bits = 32 - __clz((int)max(hi - lo, 1u));
      for (;;) {
        const int low = max(bits - kDigit, 0);
        for (int x = tid; x < 1 << kDigit; x += kPickThreads) count[x] = 0;
        __syncthreads();
        const uint32_t top = hi - lo;
        each([&](uint32_t k) {
          if (k >= lo && k - lo <= top && k != kKeyKeep) atomicAdd(&count[(k - lo) >> low], 1u);
        });
        __syncthreads();
        // from the highest digit down: thread t holds digits 2 (last - t) + 1 and 2 (last - t)
        const int x = 2 * (kPickThreads - 1 - tid);
        const uint32_t b = count[x + 1], a = count[x];
        uint32_t sum;
        const uint32_t above = scan_picks(a + b, part, &sum);
        if (above < want && want <= above + a + b) {
          const bool second = want > above + b;
          found[0] = x + (second ? 0 : 1);
          found[1] = want - above - (second ? b : 0);
        }
        __syncthreads();
        lo += found[0] << low;
        want = found[1];
        if (low == 0) break;
        hi = min(hi, lo + ((1u << low) - 1));
        bits = low;
        __syncthreads();
      }
      least = lo;
      ties = want;
    }
  }
  // 16 bits each: taken for sure, and ties, of this thread's keys of one span
  uint32_t done = 0, tied = 0;
  for (int base = 0; base < n; base += span) {
    if (base || n > span) read(base);
    uint32_t mine = 0;
    const bool every = n_valid <= (uint32_t)sel.budget;
#pragma unroll
    for (int x = 0; x < kOwn; ++x) mine += every ? (own[x] != 0) : (own[x] > least ? 1u : 0u) + (own[x] == least ? 1u << 16 : 0u);
    uint32_t sum;
    const uint32_t before = scan_picks(mine, part, &sum);
    uint32_t at_tie = tied + (before >> 16), at = done + (before & 0xFFFFu) + min(at_tie, ties);
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const bool tie = !every && own[x] == least;
      const bool take = every ? own[x] != 0 : own[x] > least || (tie && at_tie < ties);
      if (tie) ++at_tie;
      if (take) out[at++] = base + tid * kOwn + x;
    }
    done += sum & 0xFFFFu;
    tied += sum >> 16;
  }
  for (uint32_t j = done + min(tied, ties) + tid; j < (uint32_t)sel.budget; j += kPickThreads) out[j] = -1;
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

template <class T>
void launch_scores(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q, const void* bounds,
                   const kvtc_selection& sel, uint32_t* keys, hipStream_t s) {
  int lp = 1;
  while (lp * 16 < p.head_dim * (int)sizeof(T)) lp *= 2;
  // Pages per workgroup: enough workgroups to fill the GPU a few times over
  // where there are as many pages, in whole steps of kPageThreads / lp.
  const int64_t most = (int64_t)r.n_requests * p.kv_heads * r.table_width, step = kPageThreads / lp;
  const int64_t span = std::min<int64_t>(16, std::max<int64_t>(1, most / (4096 * step))) * step;
  const dim3 grid((unsigned)((r.table_width + span - 1) / span), p.kv_heads, r.n_requests);
  hipLaunchKernelGGL(score_kernel<T>, grid, dim3(kPageThreads), 0, s, p, r, q, (const T*)bounds, sel, keys, (int)span, lp);
}

int launch_page_select(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q, const void* bounds,
                       const kvtc_selection& sel, void* ws, hipStream_t s) {
  if (p.dtype == KVTC_F32) launch_scores<float>(p, r, q, bounds, sel, (uint32_t*)ws, s);
  else launch_scores<uint16_t>(p, r, q, bounds, sel, (uint32_t*)ws, s);
  hipLaunchKernelGGL(pick_kernel, dim3(p.kv_heads, r.n_requests), dim3(kPickThreads), 0, s, p, r, sel, (const uint32_t*)ws);
  return (int)hipGetLastError();
}

}  // namespace kvtc
