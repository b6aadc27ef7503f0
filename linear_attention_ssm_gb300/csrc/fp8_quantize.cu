// fp8_quantize.cu -- bf16 values to e4m3 codes with an fp32 scale for each block of 128 columns and 1 or 128 rows.
//
//   s = max(max |x| / 448, 2^-126) over the block,   c = e4m3(x / s), to nearest, at most 448 in magnitude
//
// Both divisions are IEEE ones, so codes and scales are the definition's to the bit.  A NaN makes its block's scale
// NaN; an infinity makes it infinite, and the infinity's own code NaN.
#include <cuda_fp8.h>

#include "gdn_kernels.h"

namespace gdn {
namespace {

constexpr int kCols = 128;  // of a block

struct QuantizeParams {
  const uint16_t* x;
  long x_stride;  // elements
  int rows, cols;
  uint8_t* codes;
  long codes_stride;
  float* scales;  // [rows or row blocks][ceil(cols / 128)]
};

// the larger one, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float scale_of(float top) { return max_nan(__fdiv_rn(top, 448.f), 1.17549435e-38f); }

__device__ __forceinline__ uint8_t code_of(float x, float s) {
  return __nv_cvt_float_to_fp8(__fdiv_rn(x, s), __NV_SATFINITE, __NV_E4M3);
}

// One CTA: kRows x 128 values.
template <int kRows>
__global__ void quantize_kernel(const QuantizeParams p) {
  __shared__ float tops[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int col0 = blockIdx.x * kCols;
  const long row0 = (long)blockIdx.y * kRows;
  float top = 0.f;
  for (int r = warp; r < kRows; r += warps) {
    const long row = row0 + r;
    if (row >= p.rows) break;
    for (int c = lane; c < kCols; c += 32)
      if (col0 + c < p.cols) top = max_nan(top, fabsf(bf2f(p.x[row * p.x_stride + col0 + c])));
  }
  for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
  if (warps > 1) {
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    for (int w = 0; w < warps; ++w) top = max_nan(top, tops[w]);
  }
  const float s = scale_of(top);
  for (int r = warp; r < kRows; r += warps) {
    const long row = row0 + r;
    if (row >= p.rows) break;
    for (int c = lane; c < kCols; c += 32)
      if (col0 + c < p.cols)
        p.codes[row * p.codes_stride + col0 + c] = code_of(bf2f(p.x[row * p.x_stride + col0 + c]), s);
  }
  if (tid == 0) p.scales[blockIdx.y * (long)gridDim.x + blockIdx.x] = s;
}

}  // namespace

cudaError_t launch_fp8_quantize(const LaunchEnv& env, const uint16_t* x, long x_stride, int rows, int cols, int block_rows,
                                uint8_t* codes, long codes_stride, float* scales) {
  QuantizeParams p = {x, x_stride, rows, cols, codes, codes_stride, scales};
  const unsigned nb = (cols + kCols - 1) / kCols;
  // rows beyond the grid's second dimension go by further launches
  const int step = block_rows * 65535;
  for (long r = 0; r < rows; r += step) {
    p.x = x + r * x_stride;
    p.codes = codes + r * codes_stride;
    p.scales = scales + r / block_rows * nb;
    p.rows = (int)(rows - r < step ? rows - r : step);
    const dim3 grid(nb, (p.rows + block_rows - 1) / block_rows);
    if (block_rows == 1) quantize_kernel<1><<<grid, 32, 0, env.stream>>>(p);
    else quantize_kernel<kCols><<<grid, 256, 0, env.stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace gdn
