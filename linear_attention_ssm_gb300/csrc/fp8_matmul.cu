// fp8_matmul.cu -- activations times weights, both e4m3 codes with fp32 scales by blocks of 128.
//
//   out[t, n] = sum_b sx[t, b] sw[n / 128, b] sum_{k in block b} x[t, k] w[n, k]
//
// The inner sum is four tcgen05 instructions on one 128-byte-wide stage of each operand; its result lies in tensor memory
// and is taken into the running fp32 sums of the registers with the block's scales, while the next block's products run
// into the other half of the accumulators.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "attn_common.cuh"
#include "gdn_kernels.h"

namespace gdn {
namespace {

constexpr int kBlockK = 128;  // codes of a stage's row, one scale block
constexpr uint32_t kWaitLimit = 1u << 20;  // polls of one mbarrier before giving up

// A whole warp works on barriers, copies and products without a branch: every lane polls, and what one lane issues stands
// under a predicate of elect.sync in one piece of assembly.  Measured for a warp: a poll that finds its phase complete takes
// 58 cycles this way, 255 in a branch of one lane; four products and two arrivals 270, 340 in a branch of the elected lane
// and 560 in one of `lane == 0`, whose operands have to be gathered from that lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, bool cluster) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t done;
    if (cluster)
      asm volatile(
          "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
          : "=r"(done)
          : "r"(bar), "r"(parity)
          : "memory");
    else
      asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                   : "=r"(done)
                   : "r"(bar), "r"(parity)
                   : "memory");
    if (__all_sync(~0u, done)) return true;
  }
  return false;
}
// The two loads of a stage, `bytes` in all, counted by `bar`; the second one goes to the same place of kShare CTAs, named by
// the bits of `all`, and is counted in each.
template <int kShare>
__device__ __forceinline__ void warp_load_stage(uint32_t bar, uint32_t bytes, uint32_t dst0, const void* map0, int y0,
                                                uint32_t dst1, const void* map1, int y1, int x, uint16_t all) {
  if constexpr (kShare == 1)
    asm volatile(
        "{\n.reg .pred e;\n"
        "elect.sync _|e, 0xFFFFFFFF;\n"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%2], [%3, {%8, %4}], [%0];\n"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%5], [%6, {%8, %7}], [%0];\n"
        "}" ::"r"(bar),
        "r"(bytes), "r"(dst0), "l"(map0), "r"(y0), "r"(dst1), "l"(map1), "r"(y1), "r"(x)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred e;\n"
        "elect.sync _|e, 0xFFFFFFFF;\n"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%2], [%3, {%8, %4}], [%0];\n"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.multicast::cluster [%5], "
        "[%6, {%8, %7}], [%0], %9;\n"
        "}" ::"r"(bar),
        "r"(bytes), "r"(dst0), "l"(map0), "r"(y0), "r"(dst1), "l"(map1), "r"(y1), "r"(x), "h"(all)
        : "memory");
}
__device__ __forceinline__ void first_lane_arrive(uint32_t bar, int lane) {
  asm volatile("{\n.reg .pred p;\nsetp.eq.s32 p, %1, 0;\n@p mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(bar), "r"(lane)
               : "memory");
}

// Instruction descriptor: D fp32, A and B e4m3, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] = A[smem] B[smem]^T over one stage, by the whole warp: four steps of 32 codes, the first one on nothing.  When it
// is done `stage` gets an arrival, in each of the kShare CTAs named by the bits of `all`, and `result` one.
template <int kShare = 1>
__device__ __forceinline__ void warp_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t stage, uint32_t result, uint16_t all = 1) {
  if constexpr (kShare == 1)
    asm volatile(
      "{\n.reg .pred e, p, q;\n.reg .b64 a1, a2, a3, b1, b2, b3;\n"
      "elect.sync _|e, 0xFFFFFFFF;\n"
      "setp.ne.b32 p, 0, 0;\n"
      "setp.ne.b32 q, 1, 0;\n"
      "add.s64 a1, %1, 2;\nadd.s64 a2, %1, 4;\nadd.s64 a3, %1, 6;\n"
      "add.s64 b1, %2, 2;\nadd.s64 b2, %2, 4;\nadd.s64 b3, %2, 6;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, q;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, q;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(stage), "r"(result)
      : "memory");
  else
    asm volatile(
      "{\n.reg .pred e, p, q;\n.reg .b64 a1, a2, a3, b1, b2, b3;\n"
      "elect.sync _|e, 0xFFFFFFFF;\n"
      "setp.ne.b32 p, 0, 0;\n"
      "setp.ne.b32 q, 1, 0;\n"
      "add.s64 a1, %1, 2;\nadd.s64 a2, %1, 4;\nadd.s64 a3, %1, 6;\n"
      "add.s64 b1, %2, 2;\nadd.s64 b2, %2, 4;\nadd.s64 b3, %2, 6;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, q;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, q;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%4], %6;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(stage), "r"(result), "h"(all)
      : "memory");
}

struct MatmulParams {
  CUtensorMap tmap_x;  // [tokens][k] codes, 128-byte swizzle
  CUtensorMap tmap_w;  // [n][k]
  const uint8_t *x, *w;
  long x_stride, w_stride;
  const float* x_scale;
  const float* w_scale;
  int tokens, n, k, blocks;  // blocks: of k
  int split;              // CTAs that share a tile's k
  int tiles_m, tiles_n;
  int wide_out;           // rows of out are whole 32-byte sectors
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

// ---------------------------------------------------------------- up to 16 tokens: weights through the registers once

// D += A B, m16n8k16 with binary16 operands and fp32 sums.  Lane l has rows l / 4 and l / 4 + 8 of A at the k of its
// place l % 4, column l / 4 of B at the same k, and columns 2 (l % 4), + 1 of D's two rows.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float code_value(const uint8_t* p) {
  uint32_t b;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(b) : "l"(p));
  return __half2float(__ushort_as_half((unsigned short)e4m3x4_to_half4(b).x));
}

constexpr int kFewWarps = 8;

// One CTA: 16 rows of w and up to 8 kTiles tokens; its warps share the blocks of k.  A lane takes 16 codes of its two rows
// and of its token at a time and widens them to binary16, which holds them exactly; which of a quad's lanes has which k does
// not matter as long as both operands agree.  HBM bounds the kernel: 16 KB of weights in flight for each CTA, several CTAs an
// SM, no barrier before the sums meet.
template <int kTiles>
__global__ void __launch_bounds__(kFewWarps * 32, kTiles == 1 ? 3 : 2) few_kernel(const __grid_constant__ MatmulParams p) {
  __shared__ float parts[kFewWarps][kTiles][4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const long n0 = (long)blockIdx.x * 16;
  await_grid();
  float acc[kTiles][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  const uint8_t *wa = p.w + (n0 + r) * p.w_stride, *wb = wa + 8 * p.w_stride;
  const bool has_a = n0 + r < p.n, has_b = n0 + r + 8 < p.n;
  const float* sw = p.w_scale + (n0 >> 7) * p.blocks;

  constexpr int kAhead = 2;  // blocks loaded together
  const int whole = p.k & ~15;  // codes that come 16 at a time
  for (int b0 = warp * kAhead; b0 < p.blocks; b0 += kFewWarps * kAhead) {
    uint4 a[kAhead][4], x[kAhead][kTiles][2];
    float s[kAhead][kTiles][2];
    const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int b = b0 + u, k0 = b * kBlockK + c * 16, k1 = k0 + 64;
      const bool in = b < p.blocks;
      a[u][0] = in && has_a && k0 < whole ? ld_once(wa + k0) : none;
      a[u][1] = in && has_b && k0 < whole ? ld_once(wb + k0) : none;
      a[u][2] = in && has_a && k1 < whole ? ld_once(wa + k1) : none;
      a[u][3] = in && has_b && k1 < whole ? ld_once(wb + k1) : none;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const long t = i * 8 + r;
        const uint8_t* row = p.x + t * p.x_stride;
        const bool has = in && t < p.tokens;
        x[u][i][0] = has && k0 < whole ? ld_once(row + k0) : none;
        x[u][i][1] = has && k1 < whole ? ld_once(row + k1) : none;
        const long q = i * 8 + 2 * c;
        s[u][i][0] = in && q < p.tokens ? p.x_scale[q * p.blocks + b] * sw[b] : 0.f;
        s[u][i][1] = in && q + 1 < p.tokens ? p.x_scale[(q + 1) * p.blocks + b] * sw[b] : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float d[kTiles][4];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t va[4] = {a[u][2 * h].x, a[u][2 * h].y, a[u][2 * h].z, a[u][2 * h].w};
        const uint32_t vb[4] = {a[u][2 * h + 1].x, a[u][2 * h + 1].y, a[u][2 * h + 1].z, a[u][2 * h + 1].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint2 fa = e4m3x4_to_half4(va[q]), fb = e4m3x4_to_half4(vb[q]);
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            const uint32_t vx[4] = {x[u][i][h].x, x[u][i][h].y, x[u][i][h].z, x[u][i][h].w};
            const uint2 fx = e4m3x4_to_half4(vx[q]);
            mma_f16(d[i], fa.x, fb.x, fa.y, fb.y, fx.x, fx.y);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(d[i][j], s[u][i][j & 1], acc[i][j]);
    }
  }
  if (whole < p.k && warp == 0) {  // the last codes of a row, one by one
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long t = i * 8 + 2 * c + (j & 1);
        if (t >= p.tokens || !(j < 2 ? has_a : has_b)) continue;
        float d = 0.f;
        for (int k = whole; k < p.k; ++k) d = fmaf(code_value((j < 2 ? wa : wb) + k), code_value(p.x + t * p.x_stride + k), d);
        acc[i][j] = fmaf(d, p.x_scale[t * p.blocks + p.blocks - 1] * sw[p.blocks - 1], acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) parts[warp][i][j][lane] = acc[i][j];
  __syncthreads();
  // value v of the tile: row v % 16 of the weights, token v / 16
  for (int v = threadIdx.x; v < kTiles * 128; v += kFewWarps * 32) {
    const int row = v & 15, t = v >> 4;
    if (n0 + row >= p.n || t >= p.tokens) continue;
    const int j = (row >> 3) * 2 + (t & 1), l = (row & 7) * 4 + (t & 7) / 2;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) y += parts[w][t >> 3][j][l];
    store_out(p, t, n0 + row, y);
  }
}

// ---------------------------------------------------------------- few tokens: weights as the rows of a tile

template <int kTokens>
struct Narrow {
  static constexpr int kStageBytes = (128 + kTokens) * kBlockK;
  static constexpr int kStages = kTokens <= 16 ? 6 : kTokens <= 32 ? 5 : kTokens <= 64 ? 4 : 3;
  static constexpr int kBufs = kTokens <= 32 ? 8 : 256 / kTokens;  // results of blocks in tensor memory
  static constexpr int kColumns = kBufs * kTokens;
  static constexpr int kParts = kTokens > 64 ? 2 : 1;  // of a row's sums, each in a thread of its own
  static constexpr int kCols = kTokens / kParts;
  static constexpr int kThreads = 64 + 128 * kParts;  // loads, products, sums
  static constexpr int kAhead = 8;  // blocks whose scales are fetched together, one such group ahead
  static constexpr size_t kSmem = 1024 + kStages * kStageBytes + 2 * kAhead * kTokens * 4 + 256;
  static_assert(kTokens * 128 * 4 <= kStages * kStageBytes, "the sums lie in the ring at the end");
};

// One CTA: 128 rows of w times kTokens tokens over its cluster rank's part of k; the parts are added up in the order of
// the ranks through the cluster's shared memory.
template <int kTokens>
__global__ void __launch_bounds__(Narrow<kTokens>::kThreads, 2) narrow_kernel(const __grid_constant__ MatmulParams p) {
  using C = Narrow<kTokens>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  float* scales = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);  // [kParts][2][kAhead][kCols]
  uint64_t* bars = reinterpret_cast<uint64_t*>(scales + 2 * C::kAhead * kTokens);
  __shared__ uint32_t tmem_slot;
  const uint32_t full = smem_u32(bars), empty = full + 8 * C::kStages, done = empty + 8 * C::kStages, taken = done + 8 * C::kBufs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = p.split, rank = blockIdx.x % split;
  const long n0 = (long)(blockIdx.x / split) * 128, t0 = (long)blockIdx.y * kTokens;
  const int b0 = (int)((long)p.blocks * rank / split), b1 = (int)((long)p.blocks * (rank + 1) / split);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
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
  // A bounded wait; after one that ran out the warp takes no more work, and the others' waits run out in turn.
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (ok && !warp_wait(bar, parity, false)) {
      raise_error(p.err, kErrTimeout);
      ok = false;
    }
    return ok;
  };
  if (warp == 0) {
    int b = b0;
    for (; b < b1; ++b) {
      const int i = (b - b0) % C::kStages, pass = (b - b0) / C::kStages;
      if (pass && !await(empty + 8 * i, (pass - 1) & 1)) break;
      const uint32_t at = smem_u32(smem + i * C::kStageBytes);
      warp_load_stage<1>(full + 8 * i, C::kStageBytes, at, &p.tmap_w, (int)n0, at + 128 * kBlockK, &p.tmap_x, (int)t0,
                         b * kBlockK, 1);
    }
    // copies in flight land before the CTA ends, after a wait that ran out too
    for (int c = max(b0, b - C::kStages); c < b; ++c)
      mbar_wait(full + 8 * ((c - b0) % C::kStages), ((c - b0) / C::kStages) & 1, kWaitLimit);
  } else if (warp == 1) {
    for (int b = b0; b < b1; ++b) {
      const int j = b - b0, i = j % C::kStages, buf = j % C::kBufs;
      if (!await(full + 8 * i, (j / C::kStages) & 1)) break;
      if (j >= C::kBufs && !await(taken + 8 * buf, (j / C::kBufs - 1) & 1)) break;
      tc_fence_after();
      const uint32_t at = smem_u32(smem + i * C::kStageBytes);
      warp_mma_e4m3(tmem + buf * kTokens, sw128_desc(at), sw128_desc(at + 128 * kBlockK), idesc_e4m3_f32(128, kTokens),
                    empty + 8 * i, done + 8 * buf);
    }
  } else {
    const int quarter = warp & 3;
    constexpr int kAhead = C::kAhead, kOwn = (kCols * kAhead + 127) / 128;
    const int part = C::kParts > 1 && warp >= 6, thread = threadIdx.x - 64 - part * 128;
    float* mine = scales + part * 2 * kAhead * kCols;
    // the products of the two scales for blocks b .. b + 7: a thread has every 128th
    float next[kOwn];
    auto fetch = [&](int b) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int at = thread + 128 * i, ahead = at % kAhead, c = at / kAhead;
        const long t = t0 + col0 + c;
        next[i] = 0.f;
        if (c < kCols && t < p.tokens && b + ahead < b1)
          next[i] = p.x_scale[t * p.blocks + b + ahead] * p.w_scale[(n0 >> 7) * p.blocks + b + ahead];
      }
    };
    fetch(b0);
    for (int b = b0; b < b1; ++b) {  // to the end after a wait that ran out too: the others are at the barrier
      const int j = b - b0, buf = j % C::kBufs;
      const float* now = mine + (j / kAhead & 1) * kAhead * kCols + j % kAhead * kCols;
      if (j % kAhead == 0) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          const int at = thread + 128 * i, ahead = at % kAhead, c = at / kAhead;
          if (c < kCols) mine[(j / kAhead & 1) * kAhead * kCols + ahead * kCols + c] = next[i];
        }
        // the group before the last one was read before the last one's barrier
        asm volatile("bar.sync %0, 128;" ::"r"(1 + part) : "memory");
        fetch(b + kAhead);
      }
      if (!await(done + 8 * buf, (j / C::kBufs) & 1)) continue;
      tc_fence_after();
      constexpr int kStep = kCols < 32 || C::kParts > 1 ? 16 : 32;  // the registers hold no more beside the sums
#pragma unroll
      for (int c = 0; c < kCols; c += kStep) {
        float d[kStep];
        tmem_ld_cols<kStep>(tmem + ((uint32_t)(quarter * 32) << 16) + buf * kTokens + col0 + c, d);
        if (c + kStep == kCols) {
          tc_fence_before();
          first_lane_arrive(taken + 8 * buf, lane);
        }
#pragma unroll
        for (int i = 0; i < kStep; i += 4) {
          const float4 s = *reinterpret_cast<const float4*>(now + c + i);
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

// ---------------------------------------------------------------- many tokens: tokens as the rows of a tile

struct Wide {
  static constexpr int kTileM = 128, kTileN = 256;  // tokens, rows of w
  static constexpr int kStageBytes = (kTileM + kTileN) * kBlockK;
  static constexpr int kStages = 4;
  static constexpr int kWarps = 8;  // of sums: each has 32 tokens x 128 columns
  static constexpr int kThreads = 128 + 32 * kWarps;  // one warp loads, one issues products, two stand by
  static constexpr int kPitch = 17;  // of a warp's 32 x 16 values on their way out
  static constexpr int kAhead = 8;  // blocks whose scales are fetched together, one such group ahead
  static constexpr int kScales = 2 * kAhead * (32 * kWarps + 8);  // a token's for its two threads; the weights' for a warp
  static constexpr size_t kSmem = 1024 + kStages * kStageBytes + kWarps * 32 * kPitch * 4 + kScales * 4 + 256;
};

// four bytes to shared memory, without waiting for them
__device__ __forceinline__ void copy4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// tmem_ld32 in two steps: the values are there after the second one
__device__ __forceinline__ void tmem_ld32_begin(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_end(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                 "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Tile `id` of the grid of tiles: eight rows of tiles at a time, so that the tiles that are worked on together share both
// operands in L2.
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int& m, int& n) {
  const int group = 8 * tiles_n, g = id / group, in = id - g * group, rows = min(8, tiles_m - 8 * g);
  n = in / rows;
  m = 8 * g + in - n * rows;
}

// kShare CTAs of a cluster take tiles of the same rows of w, above one another: each loads its share of them for all.
template <int kShare>
__global__ void __launch_bounds__(Wide::kThreads, 1) wide_kernel(const __grid_constant__ MatmulParams p) {
  using C = Wide;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  float* stage_out = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);
  float* scales = stage_out + C::kWarps * 32 * C::kPitch;  // [2][kAhead][kWarps][32], then [2][kWarps][kAhead]
  uint64_t* bars = reinterpret_cast<uint64_t*>(scales + C::kScales);
  __shared__ uint32_t tmem_slot;
  const uint32_t full = smem_u32(bars), empty = full + 8 * C::kStages, done = empty + 8 * C::kStages, taken = done + 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % kShare, first = blockIdx.x / kShare, step = gridDim.x / kShare;
  constexpr uint16_t kAll = (1 << kShare) - 1;  // the cluster's CTAs
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 2 * kShare);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(done + 8 * i, 1);
      mbar_init(taken + 8 * i, C::kWarps / 2);
    }
    fence_mbar_init();
    prefetch_tensormap(&p.tmap_x);
    prefetch_tensormap(&p.tmap_w);
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  if constexpr (kShare > 1) cluster_sync();  // the others' barriers are there
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  await_grid();

  bool ok = true;
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (ok && !warp_wait(bar, parity, false)) {
      raise_error(p.err, kErrTimeout);
      ok = false;
    }
    return ok;
  };
  const int tiles = p.tiles_m * p.tiles_n;
  // 384 threads are launched with 168 registers each; 56 in the first four warps leave 224 for those of the sums
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == 0) {
    int i = 0, pass = 0;  // stage, passes over the ring
    for (int id = first; id < tiles && ok; id += step) {
      int m, n;
      tile_of(id, p.tiles_m, p.tiles_n, m, n);
      for (int b = 0; b < p.blocks; ++b) {
        if (pass && !await(empty + 8 * i, (pass - 1) & 1)) break;
        const uint32_t at = smem_u32(smem + i * C::kStageBytes);
        constexpr int kPart = C::kTileN / kShare;
        warp_load_stage<kShare>(full + 8 * i, C::kStageBytes, at, &p.tmap_x, (m * kShare + rank) * C::kTileM,
                                at + (C::kTileM + rank * kPart) * kBlockK, &p.tmap_w, n * C::kTileN + rank * kPart, b * kBlockK,
                                kAll);
        if (++i == C::kStages) i = 0, ++pass;
      }
    }
    // copies in flight land before the CTA ends, after a wait that ran out too
      for (int c = 0; c < C::kStages; ++c) {
        const int passes = pass + (c < i);  // loads into stage c
        if (passes) mbar_wait(full + 8 * c, (passes - 1) & 1, kWaitLimit);
      }
  } else if (warp < 3) {
    // each of these warps issues the products of one half of the columns
    const int side = warp - 1;
    int i = 0, pass = 0, j = 0;
    for (int id = first; id < tiles && ok; id += step)
      for (int b = 0; b < p.blocks; ++b, ++j) {
        const int buf = 2 * side + (j & 1);
        if (!await(full + 8 * i, pass & 1)) break;
        if (j >= 2 && !await(taken + 8 * buf, ((j >> 1) - 1) & 1)) break;
        tc_fence_after();
        const uint32_t at = smem_u32(smem + i * C::kStageBytes);
        warp_mma_e4m3<kShare>(tmem + buf * 128, sw128_desc(at), sw128_desc(at + (C::kTileM + side * 128) * kBlockK),
                      idesc_e4m3_f32(128, 128), empty + 8 * i, done + 8 * buf, kAll);
        if (++i == C::kStages) i = 0, ++pass;
      }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int quarter = warp & 3, side = (warp - 4) >> 2;  // of the columns
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + side * 256;
    float* mine = stage_out + (warp - 4) * 32 * C::kPitch;
    constexpr int kAhead = C::kAhead;
    float* own_x = scales + (warp - 4) * 32;  // its tokens' scales, a row for each block of two groups
    float* own_w = scales + 2 * kAhead * 32 * C::kWarps + (warp - 4) * kAhead;
    int j = 0, group = 0;
    for (int id = first; id < tiles && ok; id += step) {
      int m, n;
      tile_of(id, p.tiles_m, p.tiles_n, m, n);
      const long t0 = (long)(m * kShare + rank) * C::kTileM + quarter * 32, t = t0 + lane;
      const long n0 = (long)n * C::kTileN + side * 128;
      // tokens and columns behind the last ones take the last ones' scales: what they are multiplied with is not written
      const float* sw = p.w_scale + (min(n0, (long)p.n - 1) >> 7) * p.blocks;
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
      // a group of blocks' scales, eight blocks of four tokens at a time: a sector of each token's row
      auto fetch = [&](int b) {
        const int to = (group + (b > 0)) & 1, u = lane & 7;
        if (b + u < p.blocks) {
          const float* from = p.x_scale + b + u;
          float* x_to = own_x + (to * kAhead + u) * 32 * C::kWarps;
#pragma unroll
          for (int i = lane >> 3; i < 32; i += 4) copy4(x_to + i, from + min(t0 + i, (long)p.tokens - 1) * p.blocks);
          if (lane < kAhead) copy4(own_w + to * kAhead * C::kWarps + u, sw + b + u);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      fetch(0);
      float2 s = make_float2(0.f, 0.f);
      uint32_t d[2][32];
      // Block b's products are there: its scale, and the first 32 of its columns on their way.
      auto begin = [&](int b) {
        if (b % kAhead == 0) {
          if (b) ++group;
          fetch(b + kAhead);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          __syncwarp();
        }
        const int at = (group & 1) * kAhead + b % kAhead;
        const float v = own_x[at * 32 * C::kWarps + lane] * own_w[((group & 1) * C::kWarps) * kAhead + b % kAhead];
        s = make_float2(v, v);
        if (!await(done + 8 * (2 * side + (j & 1)), (j >> 1) & 1)) return;
        tc_fence_after();
        tmem_ld32_begin(lanes + (j & 1) * 128, d[0]);
      };
      begin(0);
#pragma unroll 1
      for (int b = 0; b < p.blocks && ok; ++b) {
        const float2 now = s;
        const uint32_t at = lanes + (j & 1) * 128;
        // 32 columns are on their way while the 32 before them are added: the next block's first ones beside its last
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld32_end(d[c & 1]);
          if (c < 3) {
            tmem_ld32_begin(at + (c + 1) * 32, d[~c & 1]);
          } else {
            tc_fence_before();
            first_lane_arrive(taken + 8 * (2 * side + (j & 1)), lane);
            ++j;
            if (b + 1 < p.blocks) begin(b + 1);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[c * 16 + i] = __ffma2_rn(make_float2(__uint_as_float(d[c & 1][2 * i]), __uint_as_float(d[c & 1][2 * i + 1])),
                                         now, acc[c * 16 + i]);
        }
      }
      ++group;
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
      if (!ok) break;
      if (p.wide_out) {  // whole sectors of a row from its thread
        if (t < p.tokens) {
          const long at = t * p.out_stride + n0;
          if (p.out_f32) {
            float* to = static_cast<float*>(p.out) + at;
#pragma unroll
            for (int i = 0; i < 128 / 8; ++i) {
              uint32_t v[8];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[2 * q] = __float_as_uint(acc[4 * i + q].x);
                v[2 * q + 1] = __float_as_uint(acc[4 * i + q].y);
              }
              if (n0 + 8 * i < p.n) st_global32(to + 8 * i, v);
            }
          } else {
            uint16_t* to = static_cast<uint16_t*>(p.out) + at;
#pragma unroll
            for (int i = 0; i < 128 / 16; ++i) {
              uint32_t v[8];
#pragma unroll
              for (int q = 0; q < 8; ++q) v[q] = pack_bf2(acc[8 * i + q].x, acc[8 * i + q].y);
              if (n0 + 16 * i < p.n) st_global32(to + 16 * i, v);
            }
          }
        }
      } else {  // rows of any alignment: 32 x 16 values at a time through shared memory, half a row a store
#pragma unroll
        for (int c = 0; c < 128 / 16; ++c) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            mine[lane * C::kPitch + 2 * i] = acc[c * 8 + i].x;
            mine[lane * C::kPitch + 2 * i + 1] = acc[c * 8 + i].y;
          }
          __syncwarp();
          const int col = lane & 15;
          if (n0 + c * 16 + col < p.n)
            for (int r = lane >> 4; r < 32 && t0 + r < p.tokens; r += 2)
              store_out(p, t0 + r, n0 + c * 16 + col, mine[r * C::kPitch + col]);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (kShare > 1) cluster_sync();  // what the others load and signal here has come
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int kShare>
cudaError_t launch_wide(const LaunchEnv& env, MatmulParams& p, const Fp8Matmul& m) {
  using C = Wide;
  static int clusters[64] = {0};  // that fit the device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kShare;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kShare);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = env.stream;
  cfg.attrs = attr;
  cfg.numAttrs = kShare > 1 ? 2 : 1;
  int fit = dev < 64 ? clusters[dev] : 0;
  if (!fit) {
    e = cudaFuncSetAttribute(wide_kernel<kShare>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    if (kShare == 1) e = device_sm_count(&fit);
    else {
      cudaLaunchConfig_t q = cfg;
      q.attrs = attr + 1;
      q.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&fit, wide_kernel<kShare>, &q);
    }
    if (e != cudaSuccess) return e;
    if (getenv("GDN_VERBOSE")) fprintf(stderr, "clusters of %d: %d\n", kShare, fit);
    if (dev < 64) clusters[dev] = fit;
  }
  e = encode_u8_2d_sw128(&p.tmap_x, m.x, m.k, m.tokens, m.x_stride, kBlockK, C::kTileM);
  if (e == cudaSuccess) e = encode_u8_2d_sw128(&p.tmap_w, m.w, m.k, m.n, m.w_stride, kBlockK, C::kTileN / kShare);
  if (e != cudaSuccess) return e;
  p.tiles_m = (int)((m.tokens + (long)C::kTileM * kShare - 1) / (C::kTileM * kShare));
  p.tiles_n = (int)((m.n + (long)C::kTileN - 1) / C::kTileN);
  const long bytes = m.out_f32 ? 4 : 2;
  p.wide_out = (reinterpret_cast<uintptr_t>(m.out) & 31u) == 0 && m.out_stride * bytes % 32 == 0 && m.n * bytes % 32 == 0;
  const long tiles = (long)p.tiles_m * p.tiles_n;
  cfg.gridDim = dim3((unsigned)(tiles < fit ? tiles : fit) * kShare);
  return cudaLaunchKernelEx(&cfg, wide_kernel<kShare>, p);
}

}  // namespace

cudaError_t launch_fp8_matmul(const LaunchEnv& env, const Fp8Matmul& m) {
  MatmulParams p;
  memset(&p, 0, sizeof p);
  p.x = m.x;
  p.w = m.w;
  p.x_stride = m.x_stride;
  p.w_stride = m.w_stride;
  p.k = m.k;
  p.x_scale = m.x_scale;
  p.w_scale = m.w_scale;
  p.tokens = m.tokens;
  p.n = m.n;
  p.blocks = (m.k + kBlockK - 1) / kBlockK;
  p.out = m.out;
  p.out_stride = m.out_stride;
  p.out_f32 = m.out_f32;
  p.err = env.err;
  if (getenv("GDN_WIDE") && atoi(getenv("GDN_WIDE")) && m.tokens > 128) { const int s = atoi(getenv("GDN_WIDE")); return s == 4 ? launch_wide<4>(env, p, m) : s == 2 ? launch_wide<2>(env, p, m) : launch_wide<1>(env, p, m); }
  const unsigned few = (unsigned)((m.n + 15L) / 16);
  if (m.tokens <= 8) return launch_early(few_kernel<1>, dim3(few), kFewWarps * 32, 0, env.stream, p);
  if (m.tokens <= 16 && !getenv("GDN_NOFEW2")) return launch_early(few_kernel<2>, dim3(few), kFewWarps * 32, 0, env.stream, p);
  cudaError_t e = encode_u8_2d_sw128(&p.tmap_w, m.w, m.k, m.n, m.w_stride, kBlockK, 128);
  if (e != cudaSuccess) return e;
  if (m.tokens <= 16) return launch_narrow<16>(env, p, m);
  if (m.tokens <= 32) return launch_narrow<32>(env, p, m);
  if (m.tokens <= 64) return launch_narrow<64>(env, p, m);
  return launch_narrow<128>(env, p, m);
}

}  // namespace gdn
