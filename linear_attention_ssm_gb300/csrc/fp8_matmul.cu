// fp8_matmul.cu -- activations times weights, both e4m3 codes with fp32 scales by blocks of 128.
//
//   out[t, n] = sum_b sx[t, b] sw[n / 128, b] sum_{k in block b} x[t, k] w[n, k]
//
// The inner sum is four tcgen05 instructions on one 128-byte-wide stage of each operand; its result lies in tensor memory
// and is taken into the running fp32 sums of the registers with the block's scales, while the next block's products run
// into the other half of the accumulators.
#include <stdlib.h>
#include <string.h>

#include "attn_common.cuh"
#include "gdn_kernels.h"

namespace gdn {
namespace {

constexpr int kBlockK = 128;  // codes of a stage's row, one scale block
constexpr uint32_t kWaitLimit = 1u << 20;  // polls of one mbarrier before giving up

// Instruction descriptor: D fp32, A and B e4m3, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] = A[smem] B[smem]^T over one stage: four steps of 32 codes, the first one on nothing.
__device__ __forceinline__ void mma_e4m3_k4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 a1, a2, a3, b1, b2, b3;\n"
      "setp.ne.b32 p, 0, 0;\n"
      "setp.ne.b32 q, 1, 0;\n"
      "add.s64 a1, %1, 2;\nadd.s64 a2, %1, 4;\nadd.s64 a3, %1, 6;\n"
      "add.s64 b1, %2, 2;\nadd.s64 b2, %2, 4;\nadd.s64 b3, %2, 6;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, q;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, q;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc)
      : "memory");
}

struct MatmulParams {
  CUtensorMap tmap_x;  // [tokens][k] codes, 128-byte swizzle
  CUtensorMap tmap_w;  // [n][k]
  const float* x_scale;
  const float* w_scale;
  int tokens, n, blocks;  // blocks: of k
  int split;              // CTAs that share a tile's k
  void* out;
  long out_stride;
  int out_f32;
  unsigned* err;
};

__device__ __forceinline__ void store_out(const MatmulParams& p, long t, long n, float v) {
  const long at = t * p.out_stride + n;
  if (p.out_f32) static_cast<float*>(p.out)[at] = v;
  else static_cast<uint16_t*>(p.out)[at] = f2bf(v);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// an address of this CTA's shared memory, in the CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// ---------------------------------------------------------------- few tokens: weights as the rows of a tile

template <int kTokens>
struct Narrow {
  static constexpr int kStageBytes = (128 + kTokens) * kBlockK;
  static constexpr int kStages = kTokens <= 16 ? 6 : kTokens <= 32 ? 5 : kTokens <= 64 ? 4 : 3;
  static constexpr int kColumns = 2 * kTokens < 32 ? 32 : 2 * kTokens;  // of tensor memory
  static constexpr int kParts = kTokens > 64 ? 2 : 1;  // of a row's sums, each in a thread of its own
  static constexpr int kCols = kTokens / kParts;
  static constexpr int kThreads = 64 + 128 * kParts;  // loads, products, sums
  static constexpr size_t kSmem = 1024 + kStages * kStageBytes + 4 * 2 * kTokens * 4 + 256;
  static_assert(kTokens * 128 * 4 <= kStages * kStageBytes, "the sums lie in the ring at the end");
};

// One CTA: 128 rows of w times kTokens tokens over its cluster rank's part of k; the parts are added up in the order of
// the ranks through the cluster's shared memory.
template <int kTokens>
__global__ void __launch_bounds__(Narrow<kTokens>::kThreads, 2) narrow_kernel(const __grid_constant__ MatmulParams p) {
  using C = Narrow<kTokens>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  float* scales = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);  // [warps][2][kCols]
  uint64_t* bars = reinterpret_cast<uint64_t*>(scales + 4 * 2 * kTokens);
  __shared__ uint32_t tmem_slot;
  const uint32_t full = smem_u32(bars), empty = full + 8 * C::kStages, done = empty + 8 * C::kStages, taken = done + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = p.split, rank = blockIdx.x % split;
  const long n0 = (long)(blockIdx.x / split) * 128, t0 = (long)blockIdx.y * kTokens;
  const int b0 = (int)((long)p.blocks * rank / split), b1 = (int)((long)p.blocks * (rank + 1) / split);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(done + 8 * i, 1);
      mbar_init(taken + 8 * i, 4 * C::kParts);
    }
    fence_mbar_init();
    prefetch_tensormap(&p.tmap_x);
    prefetch_tensormap(&p.tmap_w);
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_slot), C::kColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  await_grid();

  constexpr int kCols = C::kCols;
  const int col0 = C::kParts > 1 && warp >= 6 ? kCols : 0;
  float acc[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
  bool ok = true;
  // A bounded wait; after one that ran out this warp takes no more work, and the others' waits run out in turn.
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity, kWaitLimit)) {
      raise_error(p.err, kErrTimeout);
      ok = false;
    }
    return ok;
  };
  if (warp == 0) {
    if (lane == 0) {
      int b = b0;
      for (; b < b1; ++b) {
        const int i = (b - b0) % C::kStages, pass = (b - b0) / C::kStages;
        if (pass && !await(empty + 8 * i, (pass - 1) & 1)) break;
        const uint32_t at = smem_u32(smem + i * C::kStageBytes);
        mbar_arrive_expect_tx(full + 8 * i, C::kStageBytes);
        tma_load_2d(at, &p.tmap_w, b * kBlockK, (int)n0, full + 8 * i);
        tma_load_2d(at + 128 * kBlockK, &p.tmap_x, b * kBlockK, (int)t0, full + 8 * i);
      }
      // copies in flight land before the CTA ends, after a wait that ran out too
      for (int c = max(b0, b - C::kStages); c < b; ++c)
        mbar_wait(full + 8 * ((c - b0) % C::kStages), ((c - b0) / C::kStages) & 1, kWaitLimit);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      for (int b = b0; b < b1; ++b) {
        const int j = b - b0, i = j % C::kStages, half = j & 1;
        if (!await(full + 8 * i, (j / C::kStages) & 1)) break;
        if (j >= 2 && !await(taken + 8 * half, ((j >> 1) - 1) & 1)) break;
        tc_fence_after();
        const uint32_t at = smem_u32(smem + i * C::kStageBytes);
        mma_e4m3_k4(tmem + half * kTokens, sw128_desc(at), sw128_desc(at + 128 * kBlockK), idesc_e4m3_f32(128, kTokens));
        mma_commit(empty + 8 * i);
        mma_commit(done + 8 * half);
      }
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;
    float* mine = scales + (warp - 2) * 2 * kCols;
    constexpr int kOwn = (kCols + 31) / 32;  // tokens whose scales a lane fetches
    float next[kOwn], next_w = 0.f;
    auto fetch = [&](int b) {
      if (b >= b1) return;
      next_w = p.w_scale[(n0 >> 7) * p.blocks + b];
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int c = lane + 32 * i;
        const long t = t0 + col0 + c;
        next[i] = c < kCols && t < p.tokens ? p.x_scale[t * p.blocks + b] : 0.f;
      }
    };
    fetch(b0);
    for (int b = b0; b < b1 && ok; ++b) {
      const int j = b - b0, half = j & 1;
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        if (lane + 32 * i < kCols) mine[half * kCols + lane + 32 * i] = next[i] * next_w;
      fetch(b + 1);
      await(done + 8 * half, (j >> 1) & 1);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      __syncwarp();
      tc_fence_after();
      constexpr int kStep = kCols < 32 || C::kParts > 1 ? 16 : 32;  // the registers hold no more beside the sums
#pragma unroll
      for (int c = 0; c < kCols; c += kStep) {
        float d[kStep];
        tmem_ld_cols<kStep>(tmem + ((uint32_t)(quarter * 32) << 16) + half * kTokens + col0 + c, d);
        if (c + kStep == kCols) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(taken + 8 * half);
        }
#pragma unroll
        for (int i = 0; i < kStep; i += 4) {
          const float4 s = *reinterpret_cast<const float4*>(mine + half * kCols + c + i);
          acc[c + i] = fmaf(d[i], s.x, acc[c + i]);
          acc[c + i + 1] = fmaf(d[i + 1], s.y, acc[c + i + 1]);
          acc[c + i + 2] = fmaf(d[i + 2], s.z, acc[c + i + 2]);
          acc[c + i + 3] = fmaf(d[i + 3], s.w, acc[c + i + 3]);
        }
      }
    }
  }
  __syncwarp();
  const int row = (warp & 3) * 32 + lane;
  if (split == 1) {
    if (warp >= 2 && n0 + row < p.n) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (t0 + col0 + i < p.tokens) store_out(p, t0 + col0 + i, n0 + row, acc[i]);
    }
  } else {
    // every product of this CTA is done when its sums are: the ring is free
    float* sums = reinterpret_cast<float*>(smem);
    __syncthreads();
    if (warp >= 2) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) sums[(col0 + i) * 128 + row] = acc[i];
    }
    cluster_sync();
    if (warp >= 2 && n0 + row < p.n) {
      const int c1 = kTokens * (rank + 1) / split;
      for (int c = kTokens * rank / split + (col0 != 0); c < c1 && t0 + c < p.tokens; c += C::kParts) {
        const uint32_t at = smem_u32(sums + c * 128 + row);
        float y = 0.f;
        for (int r = 0; r < split; ++r) y += ld_cluster(in_cta(at, r));
        store_out(p, t0 + c, n0 + row, y);
      }
    }
    __syncwarp();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::kColumns);
}

template <int kTokens>
cudaError_t launch_narrow(const LaunchEnv& env, MatmulParams& p, const Fp8Matmul& m) {
  using C = Narrow<kTokens>;
  static int done[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(narrow_kernel<kTokens>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = 1;
  }
  e = encode_u8_2d_sw128(&p.tmap_x, m.x, m.k, m.tokens, m.x_stride, kBlockK, kTokens);
  if (e != cudaSuccess) return e;
  const long tiles = (m.n + 127) / 128, groups = (m.tokens + kTokens - 1) / kTokens;
  int split = 1;
  if (getenv("GDN_S")) split = atoi(getenv("GDN_S"));
  else while (split < 8 && 2 * split <= p.blocks && tiles * groups * split * 2 <= 304) split *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  p.split = split;
  cfg.gridDim = dim3((unsigned)(split * tiles), (unsigned)groups);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = env.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, narrow_kernel<kTokens>, p);
}

}  // namespace

cudaError_t launch_fp8_matmul(const LaunchEnv& env, const Fp8Matmul& m) {
  MatmulParams p;
  memset(&p, 0, sizeof p);
  p.x_scale = m.x_scale;
  p.w_scale = m.w_scale;
  p.tokens = m.tokens;
  p.n = m.n;
  p.blocks = (m.k + kBlockK - 1) / kBlockK;
  p.out = m.out;
  p.out_stride = m.out_stride;
  p.out_f32 = m.out_f32;
  p.err = env.err;
  cudaError_t e = encode_u8_2d_sw128(&p.tmap_w, m.w, m.k, m.n, m.w_stride, kBlockK, 128);
  if (e != cudaSuccess) return e;
  if (m.tokens <= 16) return launch_narrow<16>(env, p, m);
  if (m.tokens <= 32) return launch_narrow<32>(env, p, m);
  if (m.tokens <= 64) return launch_narrow<64>(env, p, m);
  return launch_narrow<128>(env, p, m);
}

}  // namespace gdn
