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
__device__ __forceinline__ int pages_of(int tokens, int block_size) {
  return tokens > 0 ? (tokens - 1) / block_size + 1 : 0;
}
__device__ __forceinline__ void set_status(int32_t* status, int i, int st) {
  if (status) status[i] = st;
}

// Exclusive scan of v over the workgroup's kPageThreads threads; the total in
// *sum. part: kPageThreads / 64 words of LDS.
template <class V>
__device__ __forceinline__ V scan_threads(V v, V* part, V* sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  V x = v;
  for (int d = 1; d < 64; d <<= 1) {
    const V y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) part[wave] = x;
  __syncthreads();
  V before = 0, all = 0;
  for (int w = 0; w < kPageThreads / 64; ++w) {
    if (w < wave) before += part[w];
    all += part[w];
  }
  *sum = all;
  return before + x - v;
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
inline BlockDiv block_div(int d) {
  BlockDiv b = {0, (uint32_t)d, 0};
  if (d > 1) {
    while ((2u << b.s) < (uint32_t)d) ++b.s;     // 2^s < d <= 2^(s+1)
    b.m = (uint32_t)(((uint64_t)1 << (32 + b.s)) / (uint32_t)d + 1);
  }
  return b;
}

}  // namespace kvtc
