// attn_common.cuh -- what the kernels of the paged-cache attention share: where a token's row lies,
// the e4m3 rows with their power of two.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gdn_kernels.h"

namespace gdn {

// Sequence of packed row t: the n with cu[n] <= t < cu[n + 1] (token n is sequence n's when cu is
// NULL).  -1 for a row behind the last sequence, -2 where cu is not a valid prefix sum there.
__device__ __forceinline__ int attn_seq_of(const int32_t* cu, int N, int T, int t, int& first, int& len) {
  first = t;
  len = 1;
  if (!cu) return t;
  int lo = 0, hi = N;  // the last index with cu[index] <= t, if cu is sorted
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  const int a = __ldg(cu + lo);
  if (lo == N) return a >= 0 && a <= t ? -1 : -2;
  const int b = __ldg(cu + lo + 1);
  if (a < 0 || t < a || t >= b || b > T) return -2;
  first = a;
  len = b - a;
  return lo;
}

// 2^(b - 127) of an exponent byte
__device__ __forceinline__ float e8m0_value(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

// two e4m3 codes (low byte first) -> two floats, exactly
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(v, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace gdn
