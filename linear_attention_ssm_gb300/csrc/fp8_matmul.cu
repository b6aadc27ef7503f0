// fp8_matmul.cu -- activations times weights, both e4m3 codes with fp32 scales by blocks of 128.
//
//   out[t, n] = sum_b sx[t, b] sw[n / 128, b] sum_{k in block b} x[t, k] w[n, k]
#include <cuda_fp8.h>

#include "attn_common.cuh"
#include "gdn_kernels.h"

namespace gdn {
namespace {

constexpr int kTile = 16, kK = 128;

__global__ void matmul_kernel(const Fp8Matmul p) {
  __shared__ float xs[kTile][kK + 1], ws[kTile][kK + 1];
  const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
  const long t0 = (long)blockIdx.y * kTile, n0 = (long)blockIdx.x * kTile;
  const int kb = (p.k + kK - 1) / kK;
  float acc = 0.f;
  for (int b = 0; b < kb; ++b) {
    for (int i = threadIdx.x; i < kTile * kK; i += kTile * kTile) {
      const int r = i / kK, c = i % kK, k = b * kK + c;
      xs[r][c] = k < p.k && t0 + r < p.tokens ? __half2float(__nv_cvt_fp8_to_halfraw(p.x[(t0 + r) * p.x_stride + k], __NV_E4M3)) : 0.f;
      ws[r][c] = k < p.k && n0 + r < p.n ? __half2float(__nv_cvt_fp8_to_halfraw(p.w[(n0 + r) * p.w_stride + k], __NV_E4M3)) : 0.f;
    }
    __syncthreads();
    float d = 0.f;
    for (int c = 0; c < kK; ++c) d = fmaf(xs[ty][c], ws[tx][c], d);
    if (t0 + ty < p.tokens && n0 + tx < p.n)
      acc = fmaf(d, p.x_scale[(t0 + ty) * kb + b] * p.w_scale[(n0 + tx) / kK * kb + b], acc);
    __syncthreads();
  }
  if (t0 + ty < p.tokens && n0 + tx < p.n) {
    const long at = (t0 + ty) * p.out_stride + n0 + tx;
    if (p.out_f32) static_cast<float*>(p.out)[at] = acc;
    else static_cast<uint16_t*>(p.out)[at] = f2bf(acc);
  }
}

}  // namespace

cudaError_t launch_fp8_matmul(const LaunchEnv& env, const Fp8Matmul& p) {
  const dim3 grid((p.n + kTile - 1) / kTile, (p.tokens + kTile - 1) / kTile);
  matmul_kernel<<<grid, kTile * kTile, 0, env.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
