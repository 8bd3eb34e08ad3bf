// Kernels of the paged-cache calls: block tables and slot maps, the write of
// new rows, key bounds per page, and the selection of pages by a score on
// those bounds. (Attention over the pages: kvtc_attend.hip.)
#include "kvtc_pages_device.h"

namespace kvtc {
namespace {

// ------------------------------------------------- block tables, slot maps ---

// Every workgroup scans the requests' growth in tokens and pages itself (a few
// loads and one scan; a launch before this one would cost more) and keeps
// them in LDS; then it fills its share of the table entries and, kSlotRun at a
// time, of the slots, each found by one binary search in the scans.
constexpr int kSlotRun = 4;
__host__ __device__ constexpr size_t tables_lds_bytes(int n) { return (size_t)n * 16; }

__global__ void __launch_bounds__(kPageThreads) tables_kernel(kvtc_page_plan a, BlockDiv div) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  __shared__ uint32_t part[2 * kPageThreads / 64], taken;
  const int n = a.n_requests, bs = a.block_size, tid = threadIdx.x;
  uint32_t* start = lds;                       // first token of each request
  uint32_t* page = lds + n;                    // first page of each request, behind free_from
  int32_t* olds = (int32_t*)lds + 2 * n;       // tokens before; of a request that is refused -1
  uint32_t* had = lds + 3 * n;                 // pages before
  const uint32_t from = a.free_from ? (uint32_t)max(a.free_from[0], 0) : 0u;
  if (tid == 0) taken = 0;
  const int each = (n + kPageThreads - 1) / kPageThreads, i0 = tid * each, i1 = min(i0 + each, n);
  uint32_t scan[2] = {0, 0}, total[2];         // tokens, pages
  for (int i = i0; i < i1; ++i) {
    const int old = a.old_lens ? a.old_lens[i] : 0, now = a.new_lens[i];
    const bool ok = old >= 0 && now >= old && now <= a.table_width * bs;
    const int before = ok ? pages_of(old, div) : 0;
    const uint32_t grow = ok ? now - old : 0, need = ok ? pages_of(now, div) - before : 0;
    olds[i] = ok ? old : -1;
    had[i] = before;
    start[i] = grow;
    page[i] = need;
    scan[0] = add_sat(scan[0], grow);
    scan[1] = add_sat(scan[1], need);
  }
  scan_threads<kPageThreads / 64>(scan, part, total);
  uint32_t t = scan[0], b = scan[1], most = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t grow = start[i], need = page[i];
    const bool ok = olds[i] >= 0;
    const bool fits = add_sat(t, grow) <= (uint32_t)a.n_slots &&
                      (need == 0 || add_sat(from, add_sat(b, need)) <= (uint32_t)a.n_free);
    if (ok && fits && need) most = b + need;   // those served are the first that need pages
    start[i] = t;
    page[i] = b;
    if (!ok || !fits) {
      olds[i] = -1;
      if (blockIdx.x == 0) set_status(a.status, i, ok ? KVTC_E_CAPACITY : KVTC_E_INVALID);
    }
    if (a.starts && blockIdx.x == 0) a.starts[i] = (int32_t)min(t, (uint32_t)INT32_MAX);
    t = add_sat(t, grow);
    b = add_sat(b, need);
  }
  most = last_lane(wave_scan(most, 0u, [](uint32_t x, uint32_t y) { return max(x, y); }));
  if ((tid & 63) == 0 && most) atomicMax(&taken, most);
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    if (a.starts) a.starts[n] = (int32_t)min(total[0], (uint32_t)INT32_MAX);
    if (a.taken) *a.taken = (int32_t)taken;
  }
  const uint32_t stride = gridDim.x * kPageThreads, me = blockIdx.x * kPageThreads + tid;
  for (uint32_t e = me; e < taken; e += stride) {
    const int i = owner_of(page, n, e);
    a.block_table[(size_t)i * a.table_stride + had[i] + (e - page[i])] = a.free_blocks[from + e];
  }
  const bool whole = ((uintptr_t)a.slots & 15) == 0;
  for (uint64_t s0 = (uint64_t)me * kSlotRun; s0 < (uint64_t)a.n_slots; s0 += (uint64_t)stride * kSlotRun) {
    int slot[kSlotRun];
    // the request, its token and the page of the slot before
    int i = s0 < total[0] ? owner_of(start, n, (uint32_t)s0) : 0;
    int at = -1, id = -1;
#pragma unroll
    for (int x = 0; x < kSlotRun; ++x) {
      const uint64_t s = s0 + x;
      slot[x] = -1;
      if (s >= total[0]) continue;
      while (i + 1 < n && start[i + 1] <= s) {
        ++i;
        at = -1;
      }
      if (olds[i] < 0) continue;
      const int p = olds[i] + (int)((uint32_t)s - start[i]), j = (int)div_block(p, div);
      if (j != at) {
        at = j;
        id = (uint32_t)j < had[i] ? a.block_table[(size_t)i * a.table_stride + j] : a.free_blocks[from + page[i] + (j - had[i])];
        if (id < 0 || id >= a.n_blocks) {
          id = -1;
          set_status(a.status, i, KVTC_E_INVALID);
        }
      }
      if (id >= 0) slot[x] = id * bs + (p - j * bs);
    }
    if (whole && s0 + kSlotRun <= (uint64_t)a.n_slots) {
      *(int4*)(a.slots + s0) = int4{slot[0], slot[1], slot[2], slot[3]};
    } else {
#pragma unroll
      for (int x = 0; x < kSlotRun; ++x)
        if (s0 + x < (uint64_t)a.n_slots) a.slots[s0 + x] = slot[x];
    }
  }
}

// ------------------------------------------------------------ write of rows ---

// 8 elements in fp32 or as stored, and back.
typedef uint32_t u32x8 __attribute__((ext_vector_type(8), aligned(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
template <class S> struct Row8;
template <> struct Row8<float> { typedef u32x8 type; };
template <> struct Row8<uint16_t> { typedef u32x4 type; };

template <class S, class D>
__device__ __forceinline__ typename Row8<D>::type convert8(typename Row8<S>::type x) {
  if constexpr (sizeof(S) == sizeof(D)) {
    return x;
  } else if constexpr (sizeof(S) == 4) {
    const f32x8 f = __builtin_bit_cast(f32x8, x);
    bf16x8 b;
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = (__bf16)f[e];
    return __builtin_bit_cast(u32x4, b);
  } else {
    u32x8 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r[2 * e] = x[e] << 16;
      r[2 * e + 1] = x[e] & 0xFFFF0000u;
    }
    return r;
  }
}

// A wave takes a row of K and V, 8 elements a lane at a time. A copy: bounded
// by HBM (or, for a step's few rows, by one load after another: the rows are
// read before their slot is known). WHOLE: rows can be read in 16-byte pieces.
template <class S, class D, bool WHOLE>
__global__ void __launch_bounds__(kPageThreads) write_kernel(kvtc_pages p, kvtc_page_rows r) {
  typedef typename Row8<S>::type src8;
  typedef typename Row8<D>::type dst8;
  const int F = p.kv_heads * p.head_dim, lane = threadIdx.x & 63;
  const int64_t rows = (int64_t)p.n_blocks * p.block_size;
  const int64_t first = blockIdx.x * (kPageThreads / 64) + (threadIdx.x >> 6), step = (int64_t)gridDim.x * (kPageThreads / 64);
  for (int64_t i = first; i < r.n_rows; i += step) {
    const int64_t slot = r.slots[i];
    const S* ks = (const S*)r.k + i * r.k_stride;
    const S* vs = (const S*)r.v + i * r.v_stride;
    const bool there = slot >= 0 && slot < rows;
    if (slot >= rows && lane == 0) set_status(r.status, 0, KVTC_E_INVALID);
    D* kd = (D*)p.k + (there ? slot : 0) * F;
    D* vd = (D*)p.v + (there ? slot : 0) * F;
    if constexpr (WHOLE) {
      for (int f = 8 * lane; f < F; f += 1024) {
        const bool two = f + 512 < F;
        src8 a[2], b[2];
        a[0] = *(const src8*)(ks + f);
        b[0] = *(const src8*)(vs + f);
        if (two) {
          a[1] = *(const src8*)(ks + f + 512);
          b[1] = *(const src8*)(vs + f + 512);
        }
        if (!there) continue;
        *(dst8*)(kd + f) = convert8<S, D>(a[0]);
        *(dst8*)(vd + f) = convert8<S, D>(b[0]);
        if (two) {
          *(dst8*)(kd + f + 512) = convert8<S, D>(a[1]);
          *(dst8*)(vd + f + 512) = convert8<S, D>(b[1]);
        }
      }
    } else if (there) {
      for (int f = lane; f < F; f += 64) {
        Elem<D>::put(kd + f, Elem<S>::get(ks + f));
        Elem<D>::put(vd + f, Elem<S>::get(vs + f));
      }
    }
  }
}

// -------------------------------------------------------------- key bounds ---

// A wave takes one page's rows over 1 KB of their columns, 16 bytes a lane,
// with the three-operand minimum and maximum that pass a NaN on (an ordinary
// one would drop it). One pass over the keys: HBM bounds a whole cache, the
// scan and two loads in a row a step's last pages. The page list follows from
// the lengths: every workgroup scans them, as in tables_kernel.
constexpr int kBoundRows = 8;      // rows in flight per lane

template <class T>
__device__ __forceinline__ void widen(u32x4 x, float* f) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(x[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(x[e] << 16);
      f[2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
    }
  }
}
template <class T>
__device__ __forceinline__ u32x4 narrow(const float* f) {      // values that T holds
  u32x4 x;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    x[e] = sizeof(T) == 4 ? __float_as_uint(f[e]) : (__float_as_uint(f[2 * e]) >> 16) | (__float_as_uint(f[2 * e + 1]) & 0xFFFF0000u);
  return x;
}

template <class T>
__global__ void __launch_bounds__(kPageThreads) bounds_kernel(kvtc_pages p, kvtc_requests r, BlockDiv div, const int32_t* from, T* bounds) {
  constexpr int EL = 16 / sizeof(T);
  extern __shared__ uint32_t first[];          // pages of the requests before each one
  __shared__ uint32_t part[kPageThreads / 64];
  const int n = r.n_requests, bs = p.block_size, F = p.kv_heads * p.head_dim, tid = threadIdx.x, lane = tid & 63;
  auto since = [&](int i) { return from ? (int)div_block(max(from[i], 0), div) : 0; };
  const int each = (n + kPageThreads - 1) / kPageThreads, i0 = tid * each, i1 = min(i0 + each, n);
  uint32_t scan[1] = {0}, sum[1];
  for (int i = i0; i < i1; ++i) {
    const int len = checked_len(r, bs, i);
    if (len < 0 && blockIdx.x == 0) set_status(r.status, i, KVTC_E_INVALID);
    const uint32_t pages = max(pages_of(len, div) - since(i), 0);
    first[i] = pages;
    scan[0] += pages;
  }
  scan_threads<kPageThreads / 64>(scan, part, sum);
  uint32_t before = scan[0];
  const uint32_t total = sum[0];
  for (int i = i0; i < i1; ++i) {
    const uint32_t pages = first[i];
    first[i] = before;
    before += pages;
  }
  __syncthreads();
  const int slabs = (F + 64 * EL - 1) / (64 * EL);
  const uint64_t units = (uint64_t)total * slabs, step = (uint64_t)gridDim.x * (kPageThreads / 64);
  for (uint64_t u = (uint64_t)blockIdx.x * (kPageThreads / 64) + (tid >> 6); u < units; u += step) {
    const uint32_t e = (uint32_t)(u / slabs);
    const int f = ((int)(u % slabs) * 64 + lane) * EL;
    const int i = owner_of(first, n, e), j = since(i) + (int)(e - first[i]);
    const int id = r.block_table[(int64_t)i * r.table_stride + j];
    if (id < 0 || id >= p.n_blocks) {
      if (lane == 0) set_status(r.status, i, KVTC_E_INVALID);
      continue;
    }
    if (f >= F) continue;
    const int rows = min(bs, r.lens[i] - j * bs);
    const T* k = (const T*)p.k + (int64_t)id * bs * F + f;
    float lo[EL], hi[EL];
    widen<T>(*(const u32x4*)k, lo);
#pragma unroll
    for (int x = 0; x < EL; ++x) hi[x] = lo[x];
    for (int t = 0; t < rows; t += kBoundRows) {
      u32x4 x[kBoundRows];
#pragma unroll
      for (int c = 0; c < kBoundRows; ++c) x[c] = *(const u32x4*)(k + (int64_t)min(t + c, rows - 1) * F);   // the last row again past the end
#pragma unroll
      for (int c = 0; c < kBoundRows; ++c) {
        float v[EL];
        widen<T>(x[c], v);
#pragma unroll
        for (int y = 0; y < EL; ++y) {
          lo[y] = __builtin_elementwise_minimum(lo[y], v[y]);
          hi[y] = __builtin_elementwise_maximum(hi[y], v[y]);
        }
      }
    }
    T* b = bounds + (int64_t)id * 2 * F + f;
    *(u32x4*)b = narrow<T>(lo);
    *(u32x4*)(b + F) = narrow<T>(hi);
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

// x + its value in the lane that CTRL names.
template <int CTRL>
__device__ __forceinline__ double add_moved(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint64_t v = (uint64_t)lane_move<CTRL>(0u, (uint32_t)(u >> 32)) << 32 | lane_move<CTRL>(0u, (uint32_t)u);
  return x + __builtin_bit_cast(double, v);
}
// The sum over every aligned group of LP lanes (a power of two), in each lane:
// neighbours, pairs, then the mirrored half rows and rows, whose lanes hold
// equal sums by then, then across rows.
__device__ __forceinline__ double sum_lanes(double x, int LP) {
  if (LP > 1) x = add_moved<0xB1>(x);        // quad_perm 1 0 3 2
  if (LP > 2) x = add_moved<0x4E>(x);        // quad_perm 2 3 0 1
  if (LP > 4) x = add_moved<0x141>(x);       // row_half_mirror
  if (LP > 8) x = add_moved<0x140>(x);       // row_mirror
  if (LP > 16) x += __shfl_xor(x, 16, 64);
  if (LP > 32) x += __shfl_xor(x, 32, 64);
  return x;
}

// Scores of `span` pages of request blockIdx.z for KV head blockIdx.x. Heads
// come first in the order of workgroups, and each request starts at another
// of its spans, because workgroups go to the 8 dies in turn: with spans first,
// every short request's only workgroups landed on one die (18 us against 15
// for 16 ragged requests of up to 64K tokens). LP lanes (a power of two) share
// a page, 16 bytes of each bound to a lane, so a load instruction covers whole
// 16 * LP byte rows; the query sums, a dim a thread, come from LDS. Reading
// the bounds is what it costs (134 MB of 32 x 1024 pages of 8 heads in 37 us);
// the sums in fp64, which make the choice independent of their order, are a
// fifth of it (30 us without).
constexpr int kScoreAhead = 4;     // pages per lane whose bounds, and queries, are loaded at a time

template <class T>
__global__ void __launch_bounds__(kPageThreads) score_kernel(kvtc_pages p, kvtc_requests r, kvtc_queries q, const T* bounds,
                                                             BlockDiv div, kvtc_selection sel, uint32_t* keys, int span, int LP) {
  constexpr int EL = 16 / sizeof(T);
  typedef T row16 __attribute__((ext_vector_type(EL)));
  const int h = blockIdx.x, i = blockIdx.z, bs = p.block_size, D = p.head_dim, F = p.kv_heads * D;
  const int lane = threadIdx.x & 63, d0 = (lane & (LP - 1)) * EL;
  __shared__ __attribute__((aligned(16))) double sums[2][KVTC_MAX_HEAD_DIM];
  const int j0 = (int)((blockIdx.y + i) % gridDim.y) * span, step = kPageThreads / LP, jl = j0 + (int)threadIdx.x / LP;
  const int32_t* table = r.block_table + (int64_t)i * r.table_stride;
  int id[kScoreAhead];
  auto look_up = [&](int base) {       // (before the length is known: within the table's row all the same)
#pragma unroll
    for (int x = 0; x < kScoreAhead; ++x) id[x] = table[min(base + x * step + jl - j0, r.table_width - 1)];
  };
  look_up(j0);
  // a thread sums one dim over the queries; the lanes that need it read it from LDS
  const int G = q.q_heads / p.kv_heads, dq = (int)threadIdx.x;
  const T* qh = (const T*)q.q + i * q.q_stride + (int64_t)h * G * D + min(dq, D - 1);
  T qs[kScoreAhead];
  auto load_queries = [&](int g) {
#pragma unroll
    for (int x = 0; x < kScoreAhead; ++x) qs[x] = qh[(int64_t)min(g + x, G - 1) * D];
  };
  load_queries(0);
  const int len = checked_len(r, bs, i), n = pages_of(len, div);
  if (len < 0 && j0 == 0 && h == 0 && threadIdx.x == 0) set_status(r.status, i, KVTC_E_INVALID);
  if (j0 >= n) return;
  const int j1 = min(n, j0 + span);
  const bool there = d0 < D, all = n <= sel.budget;     // all: every page is selected, whatever its score
  double u = 0.0, w = 0.0;
  for (int g = 0; g < G && !all; g += kScoreAhead) {
    if (g) load_queries(g);
#pragma unroll
    for (int x = 0; x < kScoreAhead; ++x) {
      const float v = g + x < G ? Elem<T>::get(&qs[x]) : 0.0f;
      u += (double)(v < 0 ? 0.0f : v);         // (a NaN enters both sums)
      w += (double)(v > 0 ? 0.0f : v);
    }
  }
  if (dq < LP * EL) {       // dims past D: 0
    sums[0][dq] = dq < D ? u : 0.0;
    sums[1][dq] = dq < D ? w : 0.0;
  }
  __syncthreads();
  double up[EL], down[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) {
    up[e] = sums[0][d0 + e];
    down[e] = sums[1][d0 + e];
  }
  uint32_t* key = keys + ((int64_t)i * p.kv_heads + h) * r.table_width;
  for (int base = j0; base < j1; base += kScoreAhead * step) {
    if (base > j0) look_up(base);
    row16 lo[kScoreAhead], hi[kScoreAhead];
    bool ok[kScoreAhead], keep[kScoreAhead];
#pragma unroll
    for (int x = 0; x < kScoreAhead; ++x) {
      const int j = base + x * step + jl - j0;
      ok[x] = j < j1 && id[x] >= 0 && id[x] < p.n_blocks;
      keep[x] = all || j < sel.first || j >= n - sel.last;
      if (ok[x] && !keep[x] && there) {
        const T* b = bounds + (int64_t)id[x] * 2 * F + h * D + d0;
        lo[x] = *(const row16*)b;
        hi[x] = *(const row16*)(b + F);
      }
    }
#pragma unroll
    for (int x = 0; x < kScoreAhead; ++x) {
      const int j = base + x * step + jl - j0;
      double s0 = 0.0, s1 = 0.0;
      if (ok[x] && !keep[x] && there)
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          const T le = lo[x][e], he = hi[x][e];
          s0 = fma(down[e], (double)Elem<T>::get(&le), s0);
          s1 = fma(up[e], (double)Elem<T>::get(&he), s1);
        }
      s0 = sum_lanes(s0 + s1, LP);
      if (j < j1 && (lane & (LP - 1)) == 0) {
        key[j] = !ok[x] ? 0u : keep[x] ? kKeyKeep : score_key(s0);
        if (!ok[x]) set_status(r.status, i, KVTC_E_INVALID);
      }
    }
  }
}

// The pages of the highest keys, in ascending order: one workgroup per (KV
// head, request). The threshold is found by counting digits of DIGIT bits,
// the first over the range that the keys really span, so that they spread
// over the counters (their leading bits, sign and exponent, hardly differ);
// each further digit only among the keys that share those before it. A
// thread has kOwn consecutive keys, in registers for the first kOwn *
// NT pages; past them they are read again for every digit.
// NT threads, as many as give each two counters of a digit: 256 where they
// hold all of a table row's keys, for their barriers are the faster ones.
constexpr int kOwn = 8;

template <int NT>
__global__ void __launch_bounds__(NT) pick_kernel(kvtc_pages p, kvtc_requests r, BlockDiv div, kvtc_selection sel, const uint32_t* keys) {
  constexpr int W = NT / 64, span = kOwn * NT, DIGIT = NT == 1024 ? 11 : 9;
  static_assert(2 * NT == 1 << DIGIT, "two counters a thread");
  __shared__ uint32_t count[1 << DIGIT], part[2 * W], ends[2 * W], found[3];
  const int h = blockIdx.x, i = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = pages_of(checked_len(r, p.block_size, i), div);
  const uint32_t* key = keys + ((int64_t)i * p.kv_heads + h) * r.table_width;
  int32_t* out = sel.blocks + ((int64_t)i * p.kv_heads + h) * sel.budget;
  const uint32_t budget = sel.budget;
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
      if (n > span) read(base);
#pragma unroll
      for (int x = 0; x < kOwn; ++x) f(own[x]);
    }
  };
  read(0);
#pragma unroll
  for (int x = tid; x < 1 << DIGIT; x += NT) count[x] = 0;
  // Only keys between those that are never taken and those that always are
  // can be the threshold; is there a choice at all?
  uint32_t lo = 0xFFFFFFFFu, hi = 0u, some[2] = {0, 0}, sums[2];      // valid, kept
  each([&](uint32_t k) {
    some[0] += k != 0;
    some[1] += k == kKeyKeep;
    if (k && k != kKeyKeep) {
      lo = min(lo, k);
      hi = max(hi, k);
    }
  });
  lo = last_lane(wave_scan(lo, 0xFFFFFFFFu, [](uint32_t x, uint32_t y) { return min(x, y); }));
  hi = last_lane(wave_scan(hi, 0u, [](uint32_t x, uint32_t y) { return max(x, y); }));
  if (lane == 0) {
    ends[wave] = lo;
    ends[W + wave] = hi;
  }
  scan_threads<W>(some, part, sums);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    lo = min(lo, ends[w]);
    hi = max(hi, ends[W + w]);
  }
  const bool every = sums[0] <= budget;
  uint32_t least = kKeyNan, ties = 0, want = budget - sums[1];   // taken: keys above least, and the first `ties` at it
  if (!every && want > 0) {
    // want of the keys lo + [0, 2^bits), in which more than that lie
    int bits = 32 - __clz((int)max(hi - lo, 1u));
    for (;;) {
      const int low = max(bits - DIGIT, 0);
      const uint32_t top = hi - lo;
      each([&](uint32_t k) {
        if (k >= lo && k - lo <= top && k != kKeyKeep) atomicAdd(&count[(k - lo) >> low], 1u);
      });
      __syncthreads();
      // from the highest digit down: thread t has digits x + 1 and x
      const int x = 2 * (NT - 1 - tid);
      const uint32_t b = count[x + 1], a = count[x];
      uint32_t above[1] = {a + b}, sum[1];
      scan_threads<W>(above, part, sum);
      count[x + 1] = count[x] = 0;
      if (above[0] < want && want <= above[0] + a + b) {
        const bool second = want > above[0] + b;
        found[0] = x + (second ? 0 : 1);
        found[1] = want - above[0] - (second ? b : 0);
        found[2] = second ? a : b;
      }
      __syncthreads();
      lo += found[0] << low;
      want = found[1];
      if (low == 0) {
        least = lo;
        ties = want;
        break;
      }
      if (want == found[2]) {      // all of this digit's keys
        least = lo - 1;
        break;
      }
      hi = min(hi, lo + ((1u << low) - 1));
      bits = low;
    }
  }
  // 16 bits each: taken for sure, and ties, of this thread's keys of one span
  uint32_t done = 0, tied = 0;
  for (int base = 0; base < n; base += span) {
    if (n > span) read(base);
    uint32_t mine[1] = {0}, sum[1];
#pragma unroll
    for (int x = 0; x < kOwn; ++x) mine[0] += every ? (own[x] != 0) : (own[x] > least ? 1u : 0u) + (own[x] == least ? 1u << 16 : 0u);
    scan_threads<W>(mine, part, sum);
    uint32_t at_tie = tied + (mine[0] >> 16), at = done + (mine[0] & 0xFFFFu) + min(at_tie, ties);
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const bool tie = !every && own[x] == least;
      const bool take = every ? own[x] != 0 : own[x] > least || (tie && at_tie < ties);
      if (tie) ++at_tie;
      if (take) out[at++] = base + tid * kOwn + x;
    }
    done += sum[0] & 0xFFFFu;
    tied += sum[0] >> 16;
  }
  for (uint32_t j = done + min(tied, ties) + tid; j < budget; j += NT) out[j] = -1;
}

int grid_for(int64_t n, int most) { return (int)std::min<int64_t>(std::max<int64_t>(n, 1), most); }

}  // namespace

int launch_page_tables(const kvtc_page_plan& a, hipStream_t s) {
  const int64_t runs = ((int64_t)a.n_slots + kSlotRun - 1) / kSlotRun;
  const int grid = grid_for((runs + kPageThreads - 1) / kPageThreads, 1024);
  const size_t lds = tables_lds_bytes(a.n_requests);
  allow_lds(tables_kernel, lds + 256);     // with what the kernel declares itself
  hipLaunchKernelGGL(tables_kernel, dim3(grid), dim3(kPageThreads), lds, s, a, block_div(a.block_size));
  return (int)hipGetLastError();
}

template <class S, class D>
int launch_write(const kvtc_pages& p, const kvtc_page_rows& r, hipStream_t s) {
  const int grid = grid_for(((int64_t)r.n_rows + kPageThreads / 64 - 1) / (kPageThreads / 64), 1 << 14);
  const bool whole = (((uintptr_t)r.k | (uintptr_t)r.v) & 15) == 0 && (r.k_stride | r.v_stride) % (int64_t)(16 / sizeof(S)) == 0;
  if (whole) hipLaunchKernelGGL((write_kernel<S, D, true>), dim3(grid), dim3(kPageThreads), 0, s, p, r);
  else hipLaunchKernelGGL((write_kernel<S, D, false>), dim3(grid), dim3(kPageThreads), 0, s, p, r);
  return (int)hipGetLastError();
}

int launch_page_write(const kvtc_pages& p, const kvtc_page_rows& r, hipStream_t s) {
  if (p.dtype == KVTC_F32) return r.dtype == KVTC_F32 ? launch_write<float, float>(p, r, s) : launch_write<uint16_t, float>(p, r, s);
  return r.dtype == KVTC_F32 ? launch_write<float, uint16_t>(p, r, s) : launch_write<uint16_t, uint16_t>(p, r, s);
}

int launch_page_bounds(const kvtc_pages& p, const kvtc_requests& r, const int32_t* from, void* bounds, hipStream_t s) {
  const int64_t slabs = ((int64_t)p.kv_heads * p.head_dim * (p.dtype == KVTC_F32 ? 4 : 2) + 1023) / 1024;
  const int grid = grid_for((int64_t)r.n_requests * r.table_width * slabs / (kPageThreads / 64) + 1, 2048);
  const size_t lds = (size_t)r.n_requests * 4;
  if (p.dtype == KVTC_F32)
    hipLaunchKernelGGL(bounds_kernel<float>, dim3(grid), dim3(kPageThreads), lds, s, p, r, block_div(p.block_size), from, (float*)bounds);
  else
    hipLaunchKernelGGL(bounds_kernel<uint16_t>, dim3(grid), dim3(kPageThreads), lds, s, p, r, block_div(p.block_size), from, (uint16_t*)bounds);
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
  const int64_t steps = std::min<int64_t>(16, std::max<int64_t>(1, most / (4096 * step)));
  const int64_t span = std::max(steps, ((int64_t)r.table_width / step + 65534) / 65535) * step;     // at most 65535 spans
  const dim3 grid(p.kv_heads, (unsigned)((r.table_width + span - 1) / span), r.n_requests);
  hipLaunchKernelGGL(score_kernel<T>, grid, dim3(kPageThreads), 0, s, p, r, q, (const T*)bounds,
                     block_div(p.block_size), sel, keys, (int)span, lp);
}

int launch_page_select(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q, const void* bounds,
                       const kvtc_selection& sel, void* ws, hipStream_t s) {
  if (p.dtype == KVTC_F32) launch_scores<float>(p, r, q, bounds, sel, (uint32_t*)ws, s);
  else launch_scores<uint16_t>(p, r, q, bounds, sel, (uint32_t*)ws, s);
  const dim3 grid(p.kv_heads, r.n_requests);
  if (r.table_width <= 256 * kOwn)
    hipLaunchKernelGGL(pick_kernel<256>, grid, dim3(256), 0, s, p, r, block_div(p.block_size), sel, (const uint32_t*)ws);
  else
    hipLaunchKernelGGL(pick_kernel<1024>, grid, dim3(1024), 0, s, p, r, block_div(p.block_size), sel, (const uint32_t*)ws);
  return (int)hipGetLastError();
}

}  // namespace kvtc
