// Attention of one new token over the pages (kvtc_page_attend).
//
// For each (request, KV head), G query heads share the keys and values:
// s = scale K q, p = exp(s - max), out = p V / sum p. Every key and value is
// read once, for 2 G / element bytes operations a byte, so HBM bounds it:
// 6.6 TB/s over eight requests of 64K tokens (8 heads of 128, bf16, 325 us),
// where a copy of the reads alone reaches 6.3 to 6.9 by its order of rows.
// Short work is bound by its chain: lengths, pages, rows, join (14 us for one
// request of 8K tokens, 6 of which HBM needs).
//
// attend_kernel: one workgroup per CU takes an equal share of the work, counted
// in chunks of positions of one row (request, KV head, 16 query heads); the
// shares follow from the lengths on the device, so ragged batches stay balanced
// and a captured graph follows new lengths. Inside a chunk each wave has a tile
// of positions of its own and keeps its own running maximum and sums; the
// waves join in LDS at the end of a row's piece. A row that lies in one share
// is finished there, pieces of the others go to the workspace and join_kernel
// adds them in a fixed order (4 us, most of it the second launch).
#include "kvtc_pages_device.h"

namespace kvtc {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct AttendArgs {
  kvtc_pages p;
  kvtc_requests r;
  kvtc_queries q;
  kvtc_selection sel;
  BlockDiv div;
  int32_t group;        // query heads per KV head
  int32_t tiles;        // tiles of 16 query heads per KV head
  int32_t gt;           // query heads of a full tile
  float* part;          // pieces of rows, two per workgroup
  uint4* meta;          // per workgroup: the row that its range starts inside (see join_kernel)
};

// One wave's tile: positions [P, P + TK) of a row, in TK / TG = 4 groups of TG.
// Lane l = 16 g + r.
//
// bf16, TK = 32, v_mfma_f32_16x16x32_bf16 (16 rows x 32 deep, lane l gives
// row r, depth 8 g .. + 8): the first product is S^T = K q^T in two blocks of
// 16 keys; block t's row r is position 4 t + r % 4 of group r / 4, so that the
// result, rows 4 g + i of query r, is positions 4 t + i of group g: exactly the
// depths that the lane gives as the second product's operand. That is
// out^T = V^T p^T: the lane loads the rows of group g, 16 bytes (dims 8 r ..
// + 8) of each, whole 256-byte rows per instruction, and transposes 8 x 8 in
// registers; product j yields dims 8 r' + j of query r in its rows r'.
//
// f32, TK = 16, v_mfma_f32_16x16x4_f32 (lane l gives row r, depth g): key row r
// is position r % 4 of group r / 4, the depths in the order that 16-byte reads
// bring; the result's rows 4 g + i are the positions whose values the lane has.
//
// Values are read past the caches (each is used once) straight into registers.
// The keys' operand wants 64 bytes of each of 16 rows, half a cache line, which
// such reads fetch twice (8 x 64K tokens: 386 us against 359 with cached key
// reads), so keys go to LDS first, whole rows an instruction and without a
// register, and come back as operands: CPR pieces of 16 bytes a row, exchanged
// within each row (place) so that eight lanes' reads meet all banks.
template <class T, int DP>
struct Keys {
  static constexpr int KR = sizeof(T) == 2 ? 2 : 1, TG = 4 * KR, EL = 16 / sizeof(T), CPR = DP / EL;
  static constexpr int kNt = 2;                    // the non-temporal bit of a load
  static constexpr int RPI = 64 / CPR, NX = 16 * KR / RPI, BYTES = 16 * KR * CPR * 16;
  // The tile's position (in order) that lane l fetches with instruction x.
  __device__ __forceinline__ static constexpr int at(int x, int l) { return x * RPI + l / CPR; }
  __device__ __forceinline__ static int place(int pos, int c) {
    return c ^ (KR == 2 ? (pos & 3) | ((pos >> 3) & 1) << 2 : pos & 7);
  }
  __device__ __forceinline__ static int elem(int x, int l, int D) {      // of the row, that lane l fetches
    const int d = place(at(x, l), l % CPR) * EL;
    return d < D ? d : 0;
  }
  __device__ __forceinline__ static void copy(uint8_t* to, const T* rows, int row, int offset) {
    const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc((void*)rows, 0, TG * row, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, offset, 0, 0, kNt);
  }
  // Rows `row` bytes apart, and an instruction's rows lie in one group y: its
  // first `split(y)` rows from first(y) on, the others from second(y) on, each
  // the same for all lanes. Lanes on the other side of a split sit out.
  template <bool TWO, class First, class Second, class Split>
  __device__ __forceinline__ static void load_groups(uint8_t* buf, First first, Second second, Split split, int row, int D, int l) {
    static_assert(RPI <= TG, "one group an instruction");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      const int y = x * RPI / TG, pos = at(x, l) % TG, in = elem(x, l, D) * (int)sizeof(T);
      uint8_t* to = buf + 1024 * x;
      if (!TWO || split(y) >= TG) {
        copy(to, first(y), row, pos * row + in);
      } else if (pos < split(y)) {
        copy(to, first(y), row, pos * row + in);
      } else {
        copy(to, second(y), row, (pos - split(y)) * row + in);
      }
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  // Rows anywhere: row(x) is the lane's for instruction x.
  template <class Row>
  __device__ __forceinline__ static void load_rows(uint8_t* buf, Row row, int D, int l) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int x = 0; x < NX; ++x)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(row(x) + elem(x, l, D)),
                                       (__attribute__((address_space(3))) void*)(buf + 1024 * x), 16, 0, kNt);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  // The copies to LDS are counted like loads, but the compiler does not wait
  // for them before it reads LDS, nor for its reads before a copy overwrites
  // them: landed<N>() after N loads that follow the copies, and free().
  template <int N>
  __device__ __forceinline__ static void landed() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ __forceinline__ static void free() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  // operand piece s (dims 4 EL s + EL g .. + EL) of block t's row r; dims past
  // D meet zeros of q, but a NaN must not
  __device__ __forceinline__ static u32x4 piece(const uint8_t* buf, int t, int s, int D, int g, int r) {
    const int pos = TG * (r >> 2) + 4 * t + (r & 3);
    const u32x4 k = *(const u32x4*)(buf + (pos * CPR + place(pos, 4 * s + g)) * 16);
    return D == DP || (4 * s + g) * EL < D ? k : u32x4{0, 0, 0, 0};
  }
};

template <class T, int DP> struct Tile;

template <int DP>
struct Tile<uint16_t, DP> {
  typedef Keys<uint16_t, DP> KK;
  static constexpr int TK = 32, TG = 8, KS = DP / 32, VB = DP >= 128 ? DP / 128 : 1, VW = DP >= 128 ? 4 : 2, ND = 2 * VW;
  static constexpr int OUT = VB * ND;                 // accumulators of 4 (out^T)
  typedef uint32_t vvec __attribute__((ext_vector_type(VW)));
  vvec v[TG][VB];
  // row(e): the head's elements of position e of the lane's group; dims past D are never stored
  template <class Row>
  __device__ __forceinline__ void load_values(Row row, int D, int r) {
#pragma unroll
    for (int e = 0; e < TG; ++e)
#pragma unroll
      for (int b = 0; b < VB; ++b) {
        const int d = 128 * b + ND * r;
        v[e][b] = __builtin_nontemporal_load((const vvec*)(row(e) + (d < D ? d : 0)));
      }
  }
  // positions whose bit of live is clear are not attended to: their weight is 0, but 0 x NaN is not
  __device__ __forceinline__ void mask_rows(uint32_t live) {
#pragma unroll
    for (int e = 0; e < TG; ++e)
#pragma unroll
      for (int b = 0; b < VB; ++b)
        if (!(live >> e & 1)) v[e][b] = vvec(0);
  }
  struct Query {
    u32x4 f[KS];
    __device__ __forceinline__ void load(const uint16_t* q, int D, int g, bool there) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int d = 32 * s + 8 * g;
        f[s] = there && d < D ? *(const u32x4*)(q + d) : u32x4{0, 0, 0, 0};
      }
    }
  };
  __device__ __forceinline__ static void scores(const Query& q, const uint8_t* keys, float* s, int D, int g, int r) {
    u32x4 k[2][KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      k[0][i] = KK::piece(keys, 0, i, D, g, r);
      k[1][i] = KK::piece(keys, 1, i, D, g, r);
    }
    KK::free();
    f32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[0][i]), __builtin_bit_cast(bf16x8, q.f[i]), a, 0, 0, 0);
      b = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[1][i]), __builtin_bit_cast(bf16x8, q.f[i]), b, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = a[i];
      s[4 + i] = b[i];
    }
  }
  // The weights enter as two bf16 terms: 16 bits of them, where a single
  // term's 8 would add as much error again as the rounding of a bf16 out; the
  // matrix units have the time.
  __device__ __forceinline__ void add_values(const float* p, f32x4* o) const {
    u32x4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bf16x2 h = {(__bf16)p[2 * e], (__bf16)p[2 * e + 1]};
      const bf16x2 l = {(__bf16)(p[2 * e] - (float)h[0]), (__bf16)(p[2 * e + 1] - (float)h[1])};
      hi[e] = __builtin_bit_cast(uint32_t, h);
      lo[e] = __builtin_bit_cast(uint32_t, l);
    }
#pragma unroll
    for (int b = 0; b < VB; ++b)
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        u32x4 even, odd;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          even[e] = __builtin_amdgcn_perm(v[2 * e + 1][b][w], v[2 * e][b][w], 0x05040100);
          odd[e] = __builtin_amdgcn_perm(v[2 * e + 1][b][w], v[2 * e][b][w], 0x07060302);
        }
        f32x4& x = o[b * ND + 2 * w];
        f32x4& y = o[b * ND + 2 * w + 1];
        x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even), __builtin_bit_cast(bf16x8, hi), x, 0, 0, 0);
        y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, odd), __builtin_bit_cast(bf16x8, hi), y, 0, 0, 0);
        x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even), __builtin_bit_cast(bf16x8, lo), x, 0, 0, 0);
        y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, odd), __builtin_bit_cast(bf16x8, lo), y, 0, 0, 0);
      }
  }
};

template <int DP>
struct Tile<float, DP> {
  typedef Keys<float, DP> KK;
  static constexpr int TK = 16, TG = 4, KS = DP / 16, VB = DP / 64, ND = 4;
  static constexpr int OUT = VB * ND;
  f32x4 v[TG][VB];
  template <class Row>
  __device__ __forceinline__ void load_values(Row row, int D, int r) {
#pragma unroll
    for (int e = 0; e < TG; ++e)
#pragma unroll
      for (int b = 0; b < VB; ++b) {
        const int d = 64 * b + ND * r;
        v[e][b] = __builtin_nontemporal_load((const f32x4*)(row(e) + (d < D ? d : 0)));
      }
  }
  __device__ __forceinline__ void mask_rows(uint32_t live) {
#pragma unroll
    for (int e = 0; e < TG; ++e)
#pragma unroll
      for (int b = 0; b < VB; ++b)
        if (!(live >> e & 1)) v[e][b] = f32x4{0, 0, 0, 0};
  }
  struct Query {
    f32x4 f[KS];
    __device__ __forceinline__ void load(const float* q, int D, int g, bool there) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int d = 16 * s + 4 * g;
        f[s] = there && d < D ? *(const f32x4*)(q + d) : f32x4{0, 0, 0, 0};
      }
    }
  };
  __device__ __forceinline__ static void scores(const Query& q, const uint8_t* keys, float* s, int D, int g, int r) {
    f32x4 k[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) k[i] = __builtin_bit_cast(f32x4, KK::piece(keys, 0, i, D, g, r));
    KK::free();
    f32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};      // two chains: one would wait for each result
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int x = 0; x < 4; x += 2) {
        a = __builtin_amdgcn_mfma_f32_16x16x4f32(k[i][x], q.f[i][x], a, 0, 0, 0);
        b = __builtin_amdgcn_mfma_f32_16x16x4f32(k[i][x + 1], q.f[i][x + 1], b, 0, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = a[i] + b[i];
  }
  __device__ __forceinline__ void add_values(const float* p, f32x4* o) const {
#pragma unroll
    for (int e = 0; e < TG; ++e)
#pragma unroll
      for (int b = 0; b < VB; ++b)
#pragma unroll
        for (int j = 0; j < ND; ++j)
          o[b * ND + j] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[e][b][j], p[e], o[b * ND + j], 0, 0, 0);
  }
};

// max over the four lanes l, l ^ 16, l ^ 32, l ^ 48 (one query's positions); sum likewise
__device__ __forceinline__ float max_groups(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, 64));
  return fmaxf(x, __shfl_xor(x, 32, 64));
}
__device__ __forceinline__ float sum_groups(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

// DP: head_dim rounded up to 64, 128 or 256. PAGES: in how many pages the TG
// positions of a group can lie, so how many a lane looks up a tile: 1 where
// block_size is a multiple of TG, 2 where it is larger; 0 for smaller pages,
// where a lane looks up each of its rows (8 x 16K tokens, bf16: 89 us with
// pages of 16, 94 with pages of 20, 127 with those taken row by row).
//
// The next tile's keys are loaded as soon as this one's scores are computed,
// its values after the second product: 16 KB a wave in flight at head_dim 128
// (a second buffer of keys changed nothing: 339 us against 338 over 8 x 64K
// tokens). Lookups run ahead by a tile for each load in their chain, and are
// only looked at when they are needed: a wait for one would be a wait for all
// data loaded before it. (At PAGES = 0 there are too many to hold; they are
// waited for.)
template <class T, int DP, int PAGES>
__global__ void __launch_bounds__(64 * kAttendWaves) attend_kernel(AttendArgs a) {
  constexpr int NW = kAttendWaves, kThreads = 64 * NW;
  typedef Tile<T, DP> TT;
  typedef Keys<T, DP> KK;
  constexpr int TK = TT::TK, TG = TT::TG, CH = NW * TK, NS = TK / 4;
  constexpr int NL = PAGES ? PAGES : TG + KK::NX;       // lookups of a lane: its group's pages, or its value rows and its key rows
  constexpr uint32_t kFull = (1u << TG) - 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ uint32_t scan_part[NW];
  __shared__ float wm[NW][16], wl[NW][16];
  static_assert(KK::BYTES == 16 * DP * 4, "a wave's sums take the place of its keys");
  float* wo = (float*)lds;                                              // [NW][16][DP]
  uint32_t* pre = (uint32_t*)(lds + NW * KK::BYTES);                    // units of the requests before each one, per row
  int32_t* lens = (int32_t*)pre + a.r.n_requests;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
  const int n_req = a.r.n_requests, bs = a.p.block_size, D = a.p.head_dim, rows_each = a.p.kv_heads * a.tiles;
  const int64_t F = (int64_t)a.p.kv_heads * D;
  uint8_t* keys = lds + wave * KK::BYTES;

  // positions of a request: its tokens, or those of as many selected pages as it has pages
  auto positions = [&](int len) -> int { return a.sel.blocks ? min(a.sel.budget, pages_of(len, a.div)) * bs : len; };
  // A row counts as its chunks, and one that a range holds with others as
  // kAttendRow more: so much longer its start and end take (128 ragged
  // requests of up to 16K tokens: 269 us without, 159 with).
  uint32_t total, range;
  auto extra = [&](uint32_t n) -> uint32_t { return n < range ? kAttendRow : 0u; };
  {
    const int each = (n_req + kThreads - 1) / kThreads, i0 = threadIdx.x * each, i1 = min(i0 + each, n_req);
    uint32_t scan[1] = {0}, sum[1];
    for (int i = i0; i < i1; ++i) {
      int len = checked_len(a.r, bs, i);
      if (len < 0) {
        if (blockIdx.x == 0) set_status(a.r.status, i, KVTC_E_INVALID);
        len = 0;
      }
      lens[i] = len;
      pre[i] = (uint32_t)((positions(len) + CH - 1) / CH);
      scan[0] += pre[i];
    }
    scan_threads<NW>(scan, scan_part, sum);
    range = sum[0] * rows_each / gridDim.x;
    scan[0] = 0;
    for (int i = i0; i < i1; ++i) scan[0] += pre[i] ? pre[i] + extra(pre[i]) : 0u;
    scan_threads<NW>(scan, scan_part, sum);
    for (int i = i0; i < i1; ++i) {
      const uint32_t n = pre[i];
      pre[i] = scan[0];
      scan[0] += n ? n + extra(n) : 0u;
    }
    total = sum[0] * rows_each;
  }
  __syncthreads();
  // Range w of as many as there are units for starts at floor(w total / ranges):
  // equal rows then end where ranges do whenever they can, and no range is empty.
  const uint32_t ranges = max(min(gridDim.x, total), 1u), share = total / ranges, rest = total - share * ranges;
  auto start_of = [&](uint32_t w) -> uint32_t { return w * share + w * rest / ranges; };
  // Workgroups go to the 8 dies in turn. Rows' first ranges go to consecutive
  // workgroups, then their second ones, and so on, so that the heads of the
  // same positions, whose pieces lie side by side, are read by different dies
  // (8 x 64K tokens: 337 us in plain order, 325 so).
  const uint32_t n_rows = n_req * rows_each, turns = gridDim.x / n_rows;
  const uint32_t wid = blockIdx.x < n_rows * turns ? blockIdx.x % n_rows * turns + blockIdx.x / n_rows : blockIdx.x;
  const uint32_t u0 = start_of(min(wid, ranges)), u1 = start_of(min(wid + 1, ranges));
  // requests without a token have no chunk
  for (int i = blockIdx.x * NW + wave; i < n_req; i += gridDim.x * NW)
    if (lens[i] == 0) {
      for (int d = lane; d < a.q.q_heads * D; d += 64) Elem<T>::put((T*)a.q.out + i * a.q.out_stride + d, 0.0f);
      for (int h = lane; a.q.lse && h < a.q.q_heads; h += 64) a.q.lse[(int64_t)i * a.q.q_heads + h] = -INFINITY;
    }
  uint4 meta = {0, 0, 0, 0};

  for (uint32_t u = u0; u < u1;) {
    // the row: request i, KV head h, query tile qt; of its units, `more` and
    // its n chunks, [off, end), of its chunks [c0, c1)
    const int i = owner_of(pre, n_req, u / rows_each);
    const int len = lens[i], n_pos = positions(len), n_pages = pages_of(len, a.div);
    const uint32_t n = (uint32_t)((n_pos + CH - 1) / CH), at = u - pre[i] * rows_each;
    const uint32_t more = extra(n), row = at / (n + more), off = at - row * (n + more), end = min(n + more, off + (u1 - u));
    const uint32_t c0 = off > more ? off - more : 0u, c1 = end > more ? end - more : 0u;
    if (c0 == c1) {
      u += end - off;
      continue;
    }
    const int h = (int)row / a.tiles, qt = (int)row % a.tiles;
    const int nq = min(16, a.group - 16 * qt);
    const int32_t* list = a.sel.blocks ? a.sel.blocks + ((int64_t)i * a.p.kv_heads + h) * a.sel.budget : nullptr;
    const int32_t* table = a.r.block_table + (int64_t)i * a.r.table_stride;
    const int64_t q_at = ((int64_t)h * a.group + 16 * qt) * D;
    const T* kh = (const T*)a.p.k + h * D;
    const T* vh = (const T*)a.p.v + h * D;

    // A position's page, in steps between which a load is on its way: the entry
    // of the table (from the list, or the page's index), the entry's page, and
    // from that the position's row and the number of tokens from there on.
    auto first_of = [&](uint32_t ch) -> int { return (int)ch * CH + wave * TK + TG * g; };      // of the lane's group
    auto split_of = [&](uint32_t ch) -> int {      // how many of its positions lie in its first page
      const int pos = first_of(ch);
      return pos < n_pos ? min(bs - (pos - (int)div_block(pos, a.div) * bs), TG) : TG;
    };
    auto pos_of = [&](uint32_t ch, int x) -> int {
      if constexpr (PAGES > 0) return first_of(ch) + (x ? min(split_of(ch), TG - 1) : 0);
      else return x < TG ? first_of(ch) + x : (int)ch * CH + wave * TK + KK::at(x - TG, lane);
    };
    auto entry_of = [&](uint32_t ch, int x) -> int {
      const int slot = (int)div_block(min(pos_of(ch, x), n_pos - 1), a.div);
      return list ? list[slot] : slot;
    };
    auto page_of = [&](int entry) -> int { return table[entry >= 0 && entry < n_pages ? entry : 0]; };
    bool bad = false;
    auto row_of = [&](uint32_t ch, int x, int entry, int id, int* left) -> int {
      const int pos = pos_of(ch, x), off = pos - (int)div_block(min(pos, n_pos - 1), a.div) * bs;
      *left = 0;
      if (pos >= n_pos || entry < 0 || entry >= n_pages) return 0;
      if (id < 0 || id >= a.p.n_blocks) {
        bad = true;
        return 0;
      }
      *left = max(len - (entry * bs + off), 0);
      return id * bs + off;
    };
    TT t;
    int row_at[NL], split = TG;
    uint32_t live = 0;
    // rows of a tile's positions, and which positions of the lane's group are attended to
    auto resolve = [&](uint32_t ch, const int* entry, const int* id) -> uint32_t {
      uint32_t bits = 0;
      if constexpr (PAGES == 2) split = split_of(ch);
#pragma unroll
      for (int x = 0; x < NL; ++x) {
        int left;
        row_at[x] = row_of(ch, x, entry[x], id[x], &left);
        if constexpr (PAGES > 0) {
          const int from = x ? split : 0, there = min(left, x ? TG - split : split);
          bits |= ((1u << there) - 1) << from;
        } else if (x < TG) {
          bits |= left > 0 ? 1u << x : 0u;
        }
      }
      return bits;
    };
    auto load_keys = [&]() {
      if constexpr (PAGES > 0)
        KK::template load_groups<PAGES == 2>(
            keys, [&](int y) { return kh + (int64_t)__builtin_amdgcn_readlane(row_at[0], 16 * y) * F; },
            [&](int y) { return kh + (int64_t)__builtin_amdgcn_readlane(row_at[PAGES - 1], 16 * y) * F; },
            [&](int y) { return __builtin_amdgcn_readlane(split, 16 * y); }, (int)(F * sizeof(T)), D, lane);
      else
        KK::load_rows(keys, [&](int x) { return kh + (int64_t)row_at[TG + x] * F; }, D, lane);
    };
    auto load_values = [&]() {
      if constexpr (PAGES > 0) {
        const T* first = vh + (int64_t)row_at[0] * F;
        const T* second = vh + (int64_t)row_at[PAGES - 1] * F;
        t.load_values([&](int e) { return PAGES == 1 || e < split ? first + e * F : second + (e - split) * F; }, D, r);
      } else {
        t.load_values([&](int e) { return vh + (int64_t)row_at[e] * F; }, D, r);
      }
    };
    typename TT::Query q;
    const float c = a.q.scale * kLog2e;
    float m = -INFINITY, l = 0.0f;
    f32x4 o[TT::OUT];

    // of the next tile, and (PAGES > 0) of the one after
    int entry[NL], id[NL], entry2[NL];
    auto look_up = [&](uint32_t ch) {
#pragma unroll
      for (int x = 0; x < NL; ++x) entry[x] = entry_of(ch, x);
#pragma unroll
      for (int x = 0; x < NL; ++x) id[x] = page_of(entry[x]);
    };
    // Chunk ch, whose loads are on their way; `more` loads the next one's.
    auto tile = [&](uint32_t ch, auto more) {
      uint32_t live_next = 0;
      if constexpr (more) {
        if constexpr (PAGES == 0) look_up(ch + 1);
        live_next = resolve(ch + 1, entry, id);
#pragma unroll
        for (int x = 0; x < PAGES; ++x) {
          entry[x] = entry2[x];
          id[x] = page_of(entry2[x]);
        }
#pragma unroll
        for (int x = 0; x < PAGES; ++x) entry2[x] = entry_of(ch + 3, x);
      }
      float s[NS];
      KK::template landed<TG * TT::VB + (more && PAGES == 1 ? 1 : 0)>();     // loads that follow the keys: values, a page at least
      TT::scores(q, keys, s, D, g, r);
      if constexpr (more) load_keys();
#pragma unroll
      for (int e = 0; e < NS; ++e) s[e] *= c;
      if (__any(live != kFull)) {
#pragma unroll
        for (int e = 0; e < NS; ++e)
          if (!(live >> e & 1)) s[e] = -INFINITY;
        t.mask_rows(live);
      }
      // The maximum that the weights are taken relative to moves only when a
      // score passes it by 2^8, far from fp32's range, so that almost no tile
      // has to look across lanes or rescale the sums.
      float top = s[0];
#pragma unroll
      for (int e = 1; e < NS; ++e) top = fmaxf(top, s[e]);
      if (__any(top > m + 8.0f)) {
        const float to = fmaxf(m, max_groups(top)), f = __builtin_amdgcn_exp2f(m - (to == -INFINITY ? 0.0f : to));
        m = to;
        l *= f;
#pragma unroll
        for (int j = 0; j < TT::OUT; ++j) o[j] *= f;
      }
      const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int e = 0; e < NS; ++e) {
        s[e] = __builtin_amdgcn_exp2f(s[e] - base);
        l += s[e];
      }
      t.add_values(s, o);
      if constexpr (more) load_values();
      live = live_next;
    };
    look_up(c0);
    q.load((const T*)a.q.q + i * a.q.q_stride + q_at + (int64_t)r * D, D, g, r < nq);
#pragma unroll
    for (int j = 0; j < TT::OUT; ++j) o[j] = f32x4{0, 0, 0, 0};
    live = resolve(c0, entry, id);
#pragma unroll
    for (int x = 0; x < PAGES; ++x) {
      entry[x] = entry_of(c0 + 1, x);
      entry2[x] = entry_of(c0 + 2, x);
      id[x] = page_of(entry[x]);
    }
    load_keys();
    load_values();
    for (uint32_t ch = c0; ch + 1 < c1; ++ch) tile(ch, std::true_type{});
    tile(c1 - 1, std::false_type{});
    if (bad) set_status(a.r.status, i, KVTC_E_INVALID);

    // join the waves
    l = sum_groups(l);
    if (g == 0) {
      wm[wave][r] = m;
      wl[wave][r] = l;
    }
    __syncthreads();
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, wm[w][r]);
    const float f = __builtin_amdgcn_exp2f(m - (M == -INFINITY ? 0.0f : M));
    if (r < nq) {
#pragma unroll
      for (int b = 0; b < TT::VB; ++b)
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int j = 0; j < TT::ND; ++j)
            wo[((size_t)wave * 16 + r) * DP + b * 16 * TT::ND + (4 * g + x) * TT::ND + j] = o[b * TT::ND + j][x] * f;
    }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == n;
    float* part = a.part + (2 * (size_t)wid + (c0 ? 0 : 1)) * part_floats(a.gt, DP);
    for (int x = threadIdx.x; x < nq * (DP / 4); x += kThreads) {
      const int qr = x / (DP / 4), d = x % (DP / 4) * 4;
      f32x4 v = {0, 0, 0, 0};
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, wm[w][qr]);
      const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        v += *(const f32x4*)(wo + ((size_t)w * 16 + qr) * DP + d);
        sum += wl[w][qr] * __builtin_amdgcn_exp2f(wm[w][qr] - base);
      }
      if (whole) {
        const float z = sum == 0.0f ? 0.0f : 1.0f / sum;
        T* out = (T*)a.q.out + i * a.q.out_stride + q_at + (int64_t)qr * D + d;
        if (d < D)
#pragma unroll
          for (int e = 0; e < 4; ++e) Elem<T>::put(out + e, v[e] * z);
        if (d == 0 && a.q.lse)
          a.q.lse[(int64_t)i * a.q.q_heads + (int64_t)h * a.group + 16 * qt + qr] =
              sum == 0.0f ? -INFINITY : (base + __builtin_amdgcn_logf(sum)) * kLn2;
      } else {
        *(f32x4*)(part + (size_t)qr * DP + d) = v;
        if (d == 0) {
          part[(size_t)a.gt * DP + qr] = top;
          part[(size_t)a.gt * (DP + 1) + qr] = sum;
        }
      }
    }
    // The range starts inside this row's chunks, and their first one lies in the range before: this workgroup's
    // entry tells join_kernel the row and the last range it reaches.
    if (u == u0 && c0 > 0 && c0 <= u0 - start_of(wid - 1)) {
      const uint32_t tail = u0 - c0 + n - 1;     // the row's last unit
      uint32_t lo = wid, hi = ranges - 1;
      while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) >> 1;
        if (start_of(mid) <= tail) lo = mid;
        else hi = mid - 1;
      }
      meta = uint4{1u + (uint32_t)i, row, lo, 0};
    }
    __syncthreads();
    u += end - off;
  }
  if (threadIdx.x == 0) a.meta[wid] = meta;
}

// Adds the pieces of one row and query head: workgroup (w, query) does so if
// range w is the second that the row reaches. Pieces lie in slot 1 of range
// w - 1 and slot 0 of ranges w .. last.
template <class T, int DP>
__global__ void __launch_bounds__(kPageThreads) join_kernel(AttendArgs a) {
  constexpr int LANES = DP / 4, PER = kPageThreads / LANES, kAhead = 4;     // threads on one piece, pieces at a time
  __shared__ f32x4 sums[PER][LANES];
  __shared__ float tops[PER], weights[PER];
  const uint4 meta = a.meta[blockIdx.x];
  const int i = (int)meta.x - 1, h = (int)meta.y / a.tiles, qt = (int)meta.y % a.tiles, qr = blockIdx.y;
  if (i < 0 || qr >= min(16, a.group - 16 * qt)) return;
  const int w0 = (int)blockIdx.x - 1, n = (int)meta.z - w0 + 1, D = a.p.head_dim;
  const int d = threadIdx.x % LANES, y = threadIdx.x / LANES;
  // each thread: pieces y, y + PER, ..., kAhead of them loaded at a time, relative to a maximum of its own
  float top = -INFINITY, sum = 0.0f;
  f32x4 v = {0, 0, 0, 0};
  for (int x0 = y; x0 < n; x0 += kAhead * PER) {
    f32x4 pv[kAhead];
    float pm[kAhead], pl[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int x = x0 + k * PER, at = min(x, n - 1);
      const float* p = a.part + (2 * (size_t)(w0 + at) + (at ? 0 : 1)) * part_floats(a.gt, DP);
      pv[k] = *(const f32x4*)(p + (size_t)qr * DP + 4 * d);
      pm[k] = p[(size_t)a.gt * DP + qr];
      pl[k] = p[(size_t)a.gt * (DP + 1) + qr];
    }
    float to = top;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) to = fmaxf(to, pm[k]);
    const float base = to == -INFINITY ? 0.0f : to, f0 = __builtin_amdgcn_exp2f(top - base);
    top = to;
    sum *= f0;
    v *= f0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (x0 + k * PER >= n) continue;
      const float f = __builtin_amdgcn_exp2f(pm[k] - base);
      sum += f * pl[k];
      v += f * pv[k];
    }
  }
  sums[y][d] = v;
  if (d == 0) {
    tops[y] = top;
    weights[y] = sum;
  }
  __syncthreads();
  if (y) return;
  top = tops[0];
#pragma unroll
  for (int x = 1; x < PER; ++x) top = fmaxf(top, tops[x]);
  const float base = top == -INFINITY ? 0.0f : top;
  sum = 0.0f;
  v = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    const float f = __builtin_amdgcn_exp2f(tops[x] - base);
    v += f * sums[x][d];
    sum += f * weights[x];
  }
  const float z = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t hq = (int64_t)h * a.group + 16 * qt + qr;
  T* out = (T*)a.q.out + i * a.q.out_stride + hq * D + 4 * d;
  if (4 * d < D)
#pragma unroll
    for (int e = 0; e < 4; ++e) Elem<T>::put(out + e, v[e] * z);
  if (d == 0 && a.q.lse)
    a.q.lse[(int64_t)i * a.q.q_heads + hq] = sum == 0.0f ? -INFINITY : (base + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <class T, int DP, int PAGES>
void launch_pieces(const AttendArgs& a, uint32_t grid, hipStream_t s) {
  const size_t lds = (size_t)kAttendWaves * Keys<T, DP>::BYTES + (size_t)a.r.n_requests * 8;
  allow_lds(attend_kernel<T, DP, PAGES>, lds + 1024);      // with what the kernel declares itself
  hipLaunchKernelGGL((attend_kernel<T, DP, PAGES>), dim3(grid), dim3(64 * kAttendWaves), lds, s, a);
}

template <class T, int DP>
int launch(const AttendArgs& a, uint32_t grid, hipStream_t s) {
  constexpr int TG = Tile<T, DP>::TG;
  if (a.p.block_size % TG == 0) launch_pieces<T, DP, 1>(a, grid, s);
  else if (a.p.block_size > TG) launch_pieces<T, DP, 2>(a, grid, s);
  else launch_pieces<T, DP, 0>(a, grid, s);
  if (grid > 1)
    hipLaunchKernelGGL((join_kernel<T, DP>), dim3(grid, a.gt), dim3(kPageThreads), 0, s, a);
  return (int)hipGetLastError();
}

}  // namespace

int launch_page_attend(const kvtc_pages& p, const kvtc_requests& r, const kvtc_queries& q, const kvtc_selection& sel,
                       void* ws, hipStream_t s) {
  AttendArgs a;
  a.p = p;
  a.r = r;
  a.q = q;
  a.sel = sel;
  a.div = block_div(p.block_size);
  a.group = q.q_heads / p.kv_heads;
  a.tiles = (a.group + 15) / 16;
  a.gt = std::min(a.group, 16);
  a.meta = (uint4*)ws;
  a.part = (float*)((uint8_t*)ws + attend_meta_bytes());
  const uint32_t grid = attend_workers(p, r, q);
  const int D = p.head_dim;
  if (p.dtype == KVTC_F32)
    return D <= 64 ? launch<float, 64>(a, grid, s) : D <= 128 ? launch<float, 128>(a, grid, s) : launch<float, 256>(a, grid, s);
  return D <= 64 ? launch<uint16_t, 64>(a, grid, s) : D <= 128 ? launch<uint16_t, 128>(a, grid, s) : launch<uint16_t, 256>(a, grid, s);
}

}  // namespace kvtc
