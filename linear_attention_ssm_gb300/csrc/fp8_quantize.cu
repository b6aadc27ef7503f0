// fp8_quantize.cu -- bf16 values to e4m3 codes with an fp32 scale for each block of 128 columns and 1 or 128 rows.
//
//   s = max(max |x| / 448, 2^-126) over the block,   c = e4m3(x / s), to nearest, at most 448 in magnitude
//
// Both divisions are IEEE ones, so codes and scales are the definition's to the bit.  A NaN makes its block's scale
// NaN; an infinity makes it infinite, and the infinity's own code NaN.
#include <cuda_fp8.h>

#include "attn_common.cuh"
#include "gdn_kernels.h"

namespace gdn {
namespace {

constexpr int kCols = 128;      // of a block
constexpr int kThreads = 256;
constexpr int kRowLanes = 8;    // lanes that share a block's 128 columns of a row, 16 values each
constexpr int kPasses = 4;      // rows of a 128 x 128 block that a thread has a part of

struct QuantizeParams {
  const uint16_t* x;
  long x_stride;  // elements
  int rows, cols, blocks;  // blocks: of a row
  const uint16_t* x_end;   // behind the last value
  uint8_t* codes;
  long codes_stride;
  float* scales;  // [rows or row blocks][blocks]
};

// Sixteen bf16 values of a row as eight words, low half first: from column c on, zeroes behind the row's end.  A row may
// begin at any even address: it is read in pieces of 16 aligned bytes, which are shifted into place, and value by value where
// such a piece would reach behind the tensor.
__device__ __forceinline__ void load16(const QuantizeParams& p, const uint16_t* row, int c, uint32_t (&v)[8]) {
  const uint16_t* from = row + c;
  const int count = p.cols - c;  // values that are there
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(from) & 15);
  const uint4* piece = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(from) - off);
  const int pieces = off ? 3 : 2;
  if (count <= 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0;
    return;
  }
  if (off == 0 && count >= 16) {
    const uint4 a = ld_once(piece), b = ld_once(piece + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
  if (reinterpret_cast<const uint16_t*>(piece + pieces) <= p.x_end) {
    const uint4 a = ld_once(piece), b = ld_once(piece + 1), z = make_uint4(0, 0, 0, 0), d = off ? ld_once(piece + 2) : z;
    uint32_t w[13] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, d.x, d.y, d.z, d.w, 0};
    if (off & 8)
#pragma unroll
      for (int i = 0; i < 10; ++i) w[i] = w[i + 2];
    if (off & 4)
#pragma unroll
      for (int i = 0; i < 9; ++i) w[i] = w[i + 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = off & 2 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t lo = 0, hi = 0;
      if (2 * i < count) asm volatile("ld.global.u16 %0, [%1];" : "=r"(lo) : "l"(from + 2 * i));
      if (2 * i + 1 < count) asm volatile("ld.global.u16 %0, [%1];" : "=r"(hi) : "l"(from + 2 * i + 1));
      v[i] = lo | hi << 16;
    }
  }
  if (count < 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 2 * i >= count ? 0 : 2 * i + 1 >= count ? v[i] & 0xFFFFu : v[i];
}

// The larger magnitude's bits of each half: the order of magnitudes is that of the bits, NaN above infinity.
__device__ __forceinline__ uint32_t max_bits(const uint32_t (&v)[8], uint32_t top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __vmaxu2(top, v[i] & 0x7FFF7FFFu);
  return top;
}
__device__ __forceinline__ float scale_of(uint32_t top) {  // of the larger half
  const float m = __uint_as_float(max(top & 0xFFFFu, top >> 16) << 16), s = __fdiv_rn(m, 448.f);
  return m != m ? m : fmaxf(s, 1.17549435e-38f);
}

// x / s as IEEE division rounds it, for 2^-90 <= s <= 2^120 and quotients that matter to a code (2^-11 and more): with r the
// rounded 1 / s, q = x r is within two units of the quotient, and one more step with what is left of x gives the rounded
// quotient (after P. Markstein, Computation of elementary functions on the IBM RISC System/6000 processor, 1990, where r is
// close enough for what is left to be exact; here it is rounded for 35 pairs of significands).  x and the largest value are
// bf16, so that there are 128 x 128 pairs of significands, and a CPU test goes through them all.  What is left is taken as
// q s - x, so that a -0 stays one: x - q s is +0 there, and the sum with q = -0 +0.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = __fmul_rn(x, r);
  return __fmaf_rn(-__fmaf_rn(q, s, -x), r, q);
}

__device__ __forceinline__ uint32_t two_codes(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// The codes of sixteen values, written from column c on.
__device__ __forceinline__ void store16(const QuantizeParams& p, uint8_t* row, int c, const uint32_t (&v)[8], float s) {
  uint32_t code[4];
  if (s >= 0x1p-90f && s <= 0x1p120f) {
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = v[2 * i], b = v[2 * i + 1];
      code[i] = two_codes(quotient(__uint_as_float(a << 16), s, r), quotient(__uint_as_float(a & 0xFFFF0000u), s, r)) |
                two_codes(quotient(__uint_as_float(b << 16), s, r), quotient(__uint_as_float(b & 0xFFFF0000u), s, r)) << 16;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = v[2 * i], b = v[2 * i + 1];
      code[i] = two_codes(__fdiv_rn(__uint_as_float(a << 16), s), __fdiv_rn(__uint_as_float(a & 0xFFFF0000u), s)) |
                two_codes(__fdiv_rn(__uint_as_float(b << 16), s), __fdiv_rn(__uint_as_float(b & 0xFFFF0000u), s)) << 16;
    }
  }
  if (c <= p.cols - 16) {
    *reinterpret_cast<uint4*>(row + c) = make_uint4(code[0], code[1], code[2], code[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < p.cols) row[c + i] = (uint8_t)(code[i >> 2] >> 8 * (i & 3));
  }
}

// Rows of 128: eight lanes a block, 32 blocks a CTA in the order of memory.  One read, one write of every value: HBM bounds it.
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantizeParams p) {
  await_grid();
  const unsigned block = blockIdx.x * (kThreads / kRowLanes) + threadIdx.x / kRowLanes, all = (unsigned)p.rows * p.blocks;
  const int lane = threadIdx.x % kRowLanes;
  const bool in = block < all;
  const unsigned row = in ? block / p.blocks : 0, col = in ? block - row * p.blocks : 0;
  const int c = in ? col * kCols + lane * 16 : p.cols;
  uint32_t v[8];
  load16(p, p.x + row * p.x_stride, c, v);
  uint32_t top = max_bits(v, 0);
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(~0u, top, o));
  if (!in) return;
  const float s = scale_of(top);
  if (c < p.cols) store16(p, p.codes + row * p.codes_stride, c, v, s);
  if (lane == 0) p.scales[block] = s;
}

// One 128 x 128 block a CTA; its values stay in the registers between their maximum and their codes.
__global__ void __launch_bounds__(kThreads, 5) quantize_blocks_kernel(const QuantizeParams p) {
  __shared__ uint32_t tops[kThreads / 32];
  await_grid();
  const int lane = threadIdx.x % kRowLanes, c = blockIdx.x * kCols + lane * 16;
  const long row0 = (long)blockIdx.y * kCols + threadIdx.x / kRowLanes;
  uint32_t v[kPasses][8], top = 0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const long row = row0 + i * (kThreads / kRowLanes);
    load16(p, p.x + row * p.x_stride, row < p.rows ? c : p.cols, v[i]);
    top = max_bits(v[i], top);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(~0u, top, o));
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = __vmaxu2(top, tops[w]);
  const float s = scale_of(top);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const long row = row0 + i * (kThreads / kRowLanes);
    if (row < p.rows && c < p.cols) store16(p, p.codes + row * p.codes_stride, c, v[i], s);
  }
  if (threadIdx.x == 0) p.scales[blockIdx.y * (long)p.blocks + blockIdx.x] = s;
}

}  // namespace

cudaError_t launch_fp8_quantize(const LaunchEnv& env, const uint16_t* x, long x_stride, int rows, int cols, int block_rows,
                                uint8_t* codes, long codes_stride, float* scales) {
  QuantizeParams p = {x, x_stride, rows, cols, (int)((cols + kCols - 1L) / kCols), nullptr, codes, codes_stride, scales};
  p.x_end = x + (rows - 1L) * x_stride + cols;
  // what a launch holds: 2^31 blocks of a row, 65535 rows of blocks
  const long step = block_rows == 1 ? 0x7FFFFFFFL / p.blocks : kCols * 65535L;
  for (long r = 0; r < rows; r += step) {
    p.x = x + r * x_stride;
    p.codes = codes + r * codes_stride;
    p.scales = scales + r / block_rows * p.blocks;
    p.rows = (int)(rows - r < step ? rows - r : step);
    constexpr int kBlocks = kThreads / kRowLanes;
    const cudaError_t e =
        block_rows == 1
            ? launch_early(quantize_rows_kernel, dim3((unsigned)(((long)p.rows * p.blocks + kBlocks - 1) / kBlocks)), kThreads, 0,
                           env.stream, p)
            : launch_early(quantize_blocks_kernel, dim3(p.blocks, (unsigned)((p.rows + kCols - 1L) / kCols)), kThreads, 0,
                           env.stream, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gdn
