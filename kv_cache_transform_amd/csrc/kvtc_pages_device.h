// Device helpers of the paged-cache kernels (kvtc_pages.hip, kvtc_attend.hip).
#pragma once

#include "kvtc_device.h"
#include "kvtc_pages.h"

namespace kvtc {

template <class T> struct Elem;
template <> struct Elem<float> {
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
};
template <> struct Elem<uint16_t> {
  static __device__ __forceinline__ float get(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
  // round to nearest even; a NaN stays one
  static __device__ __forceinline__ void put(uint16_t* p, float v) {
    *p = v != v ? (uint16_t)0x7FC0u : (uint16_t)bf16_bits_rne(v);
  }
};

// Tokens of request i that a call attends to, or -1 for a length that the
// table cannot hold.
__device__ __forceinline__ int checked_len(const kvtc_requests& r, int block_size, int i) {
  const int n = r.lens[i];
  return n < 0 || n > r.table_width * block_size ? -1 : n;
}
__device__ __forceinline__ void set_status(int32_t* status, int i, int st) {
  if (status) status[i] = st;
}

// Lane moves inside the vector unit (a shuffle goes through LDS and takes
// several times as long): `fill` where the pattern has no source lane.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t lane_move(uint32_t fill, uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)fill, (int)x, CTRL, ROWS, 0xF, false);
}
// f over all lanes up to each one (an inclusive scan); e is f's neutral
// element. Shifts by 1, 2, 4 and 8 inside the rows of 16 lanes, then the last
// lane of row 0 and 2 to rows 1 and 3, then that of row 1 to rows 2 and 3.
template <class Fn>
__device__ __forceinline__ uint32_t wave_scan(uint32_t x, uint32_t e, Fn f) {
  x = f(x, lane_move<0x111>(e, x));
  x = f(x, lane_move<0x112>(e, x));
  x = f(x, lane_move<0x114>(e, x));
  x = f(x, lane_move<0x118>(e, x));
  x = f(x, lane_move<0x142, 0xA>(e, x));
  x = f(x, lane_move<0x143, 0xC>(e, x));
  return x;
}
// Sums stop at 2^32 - 1, past every size that the kernels compare them with.
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }
__device__ __forceinline__ uint32_t last_lane(uint32_t x) { return (uint32_t)__builtin_amdgcn_readlane((int)x, 63); }

// Exclusive scans (saturating) of N values over the workgroup's WAVES waves,
// their totals in sum. part: N * WAVES words of LDS.
template <int WAVES, int N>
__device__ __forceinline__ void scan_threads(uint32_t (&v)[N], uint32_t* part, uint32_t (&sum)[N]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint32_t x = wave_scan(v[k], 0u, add_sat);
    if (lane == 63) part[k * WAVES + wave] = x;
    // the scan of the lanes before this one: x - v wherever nothing saturated
    v[k] = lane_move<0x138>(0u, x);      // a shift by one lane over the whole wave
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const uint32_t y = part[k * WAVES + w];
      if (w < wave) before = add_sat(before, y);
      all = add_sat(all, y);
    }
    sum[k] = all;
    v[k] = add_sat(before, v[k]);
  }
}

// The last index i in [0, n) with first[i] <= x (first[0] = 0, ascending).
__device__ __forceinline__ int owner_of(const uint32_t* first, int n, uint32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Division of n < 2^31 by the block size d: with s = ceil(log2 d) - 1 and
// m = floor(2^(32+s) / d) + 1, m d - 2^(32+s) is in (0, d], so
// floor(n m / 2^(32+s)) is the quotient for n < 2^(32+s) / d, which is at
// least 2^31. d = 1 has m = 0.
struct BlockDiv {
  uint32_t m, d;
  int s;
};
__device__ __forceinline__ uint32_t div_block(uint32_t n, const BlockDiv& b) {
  return b.m ? __umulhi(n, b.m) >> b.s : n;
}
__device__ __forceinline__ int pages_of(int tokens, const BlockDiv& b) {
  return tokens > 0 ? (int)div_block((uint32_t)tokens - 1, b) + 1 : 0;
}
inline BlockDiv block_div(int d) {
  BlockDiv b = {0, (uint32_t)d, 0};
  if (d > 1) {
    while ((2u << b.s) < (uint32_t)d) ++b.s;     // 2^s < d <= 2^(s+1)
    b.m = (uint32_t)(((uint64_t)1 << (32 + b.s)) / (uint32_t)d + 1);
  }
  return b;
}

}  // namespace kvtc
