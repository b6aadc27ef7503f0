// fp8_matmul.cu -- activations times weights, both e4m3 codes with fp32 scales by blocks of 128.
//
//   out[t, n] = sum_b sx[t, b] sw[n / 128, b] sum_{k in block b} x[t, k] w[n, k]
//
// The inner sum is four tcgen05 instructions on one 128-byte-wide stage of each operand; its result lies in tensor memory
// and is taken into the running fp32 sums of the registers with the block's scales, while the next blocks' products run
// into other places there.  Up to 16 tokens are too few for that: weights pass through the registers once.
#include <string.h>

#include "attn_common.cuh"
#include "gdn_kernels.h"

namespace gdn {
namespace {

constexpr int kBlockK = 128;  // codes of a stage's row, one scale block
constexpr uint32_t kWaitLimit = 1u << 20;  // polls of one mbarrier before giving up
#ifdef GDN_TEST_HOOKS
constexpr uint32_t kTestWaitLimit = 1u << 12;
__device__ unsigned g_test_give_up;  // 1: the first warp of a tile's sums takes its first wait as run out
#endif

// A whole warp works on barriers, copies and products without a branch: every lane polls, and what one lane issues stands
// under a predicate of elect.sync in one piece of assembly.  Measured for a warp: a poll that finds its phase complete takes
// 58 cycles this way, 255 in a branch of one lane; four products and two arrivals 270, 340 in a branch of the elected lane
// and 560 in one of `lane == 0`, whose operands have to be gathered from that lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t limit) {
  for (uint32_t i = 0; i < limit; ++i) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    if (__all_sync(~0u, done)) return true;
  }
  return false;
}
// The two loads of a stage, `bytes` in all, counted by `bar`.
__device__ __forceinline__ void warp_load_stage(uint32_t bar, uint32_t bytes, uint32_t dst0, const void* map0, int y0,
                                                uint32_t dst1, const void* map1, int y1, int x) {
  asm volatile(
      "{\n.reg .pred e;\n"
      "elect.sync _|e, 0xFFFFFFFF;\n"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%2], [%3, {%8, %4}], [%0];\n"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%5], [%6, {%8, %7}], [%0];\n"
      "}" ::"r"(bar),
      "r"(bytes), "r"(dst0), "l"(map0), "r"(y0), "r"(dst1), "l"(map1), "r"(y1), "r"(x)
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
// is done `stage` gets an arrival, and `result` too where `last`.
__device__ __forceinline__ void warp_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t stage, uint32_t result, bool last) {
  asm volatile(
      "{\n.reg .pred e, f, p, q;\n.reg .b64 a1, a2, a3, b1, b2, b3;\n"
      "elect.sync _|e, 0xFFFFFFFF;\n"
      "setp.ne.and.b32 f, %6, 0, e;\n"
      "setp.ne.b32 p, 0, 0;\n"
      "setp.ne.b32 q, 1, 0;\n"
      "add.s64 a1, %1, 2;\nadd.s64 a2, %1, 4;\nadd.s64 a3, %1, 6;\n"
      "add.s64 b1, %2, 2;\nadd.s64 b2, %2, 4;\nadd.s64 b3, %2, 6;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, q;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, q;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n"
      "@f tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(stage), "r"(result), "r"((int)last)
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
  int rows_x, stages;  // tokens of a stage, stages of the ring
  int whole_out;           // rows of out are whole 32-byte sectors
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
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
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
// not matter as long as both operands agree.  What bounds the kernel is its way to memory: 32 KB of weights in flight for each
// CTA, two CTAs an SM, no barrier before the sums meet.  (Three of them have 80 registers a thread and spill: one token x
// 16384 x 2048 9.3 us, 8.8 with two; x 2048 x 6144 5.5 and 5.2; x 8192 x 8192 16.1 and 13.9.)  One token x 16384 x 2048 at 3.8 TB/s
// is the start of the kernel and more than three waves of CTAs that live for one trip to memory each.
template <int kTiles>
__global__ void __launch_bounds__(kFewWarps * 32, 2) few_kernel(const __grid_constant__ MatmulParams p) {
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

// ---------------------------------------------------------------- more tokens: tiles of 128 tokens x 64 or 256 rows of w

constexpr int kMaxSplit = 4;

template <int kN>
struct Tiles {
  static constexpr bool kLarge = kN == 256;
  static constexpr int kTileM = 128, kTileN = kN;  // tokens, rows of w
  static constexpr int kRing = 196608;  // bytes: at least four (eight) stages, more of fewer tokens
  static constexpr int kMaxStages = 16;
  static constexpr int kBufs = 512 / kN;  // results of blocks in tensor memory, at most as many as stages
  // Blocks whose results are taken together.  A word between the warps or a load from tensor memory is 100 to 200 cycles on
  // its way: small tiles' 64 columns are added in less.
  static constexpr int kGroup = kLarge ? 1 : 2;
  static constexpr int kFirst = kLarge ? 4 : 2;  // warps before those of the sums: one loads, one issues products
  static constexpr int kWarps = 8;               // of sums: each has 32 tokens x half the columns
  static constexpr int kCols = kTileN / 2;
  static constexpr int kThreads = 32 * (kFirst + kWarps);
  static constexpr int kPitch = 17;  // of a warp's 32 x 16 values on their way out
  static constexpr int kPartPitch = kTileN + 4;  // of a part's sums, in the ring
  static_assert(kTileM * kPartPitch * 4 <= kRing, "");
  static constexpr int kAhead = 8;  // blocks whose scales are fetched together, one such group ahead
  static constexpr int kScales = 2 * kAhead * 33 * kWarps;  // a token's for its two threads; the weights' for a warp
  // rows on their way out lie in the ring where a CTA has one tile only
  static constexpr size_t kSmem = 1024 + kRing + (kLarge ? kWarps * 32 * kPitch * 4 : 0) + kScales * 4 + 384;
};

// four bytes to shared memory, without waiting for them
__device__ __forceinline__ void copy4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// tmem_ld_cols in two steps: the values are there after the second one
__device__ __forceinline__ void tmem_ld_begin(uint32_t taddr, uint32_t (&r)[32]) {
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
__device__ __forceinline__ void tmem_ld_end(uint32_t (&r)[32]) {
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

// kSplit: the CTAs of a cluster share a tile, each a part of its blocks; the parts are added up through the cluster's shared
// memory, each CTA its share of the tokens, beginning with its own part (all at once from one CTA they would queue there).
// Otherwise a CTA takes tile after tile.
//
// What bounds the large tiles is the sums' loop, about 1000 cycles a block, beside which the tensor cores are busy for 518: the
// wait for a load from tensor memory waits for all of a warp's, so that one load of 32 columns is under way (100 to 200
// cycles) beside 16 packed multiply-adds (3.3 cycles a warp's instruction), and two warps a scheduler do not cover the rest.
// 2048 x 4096 x 6144 takes 50 us, 2.0 PFLOP/s, at 2.04 GHz (two waves of 48 blocks); 8192 x 16384 x 4096 (27 tiles of 32 blocks
// a CTA) 451 us at first, 2.4 PFLOP/s, and 486 once the power limit has brought the clock to 1.91 GHz.  Two CTAs that shared
// a tile's loads by multicast, or one product over two SMs, were no faster.  The small ones are bound by what a block waits
// for: 64 x 2048 x 6144 9.1 us, 777 x 5003 x 2041 (140 large tiles of 16 blocks) 15.0 us.
template <int kN, bool kSplit>
__global__ void __launch_bounds__(Tiles<kN>::kThreads, 1) tile_kernel(const __grid_constant__ MatmulParams p) {
  using C = Tiles<kN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  float* stage_out = reinterpret_cast<float*>(smem + C::kRing);
  // [2][kAhead][kWarps][32] of tokens, then [2][kWarps][kAhead] of weights
  float* scales = C::kLarge ? stage_out + C::kWarps * 32 * C::kPitch : stage_out;
  uint64_t* bars = reinterpret_cast<uint64_t*>(scales + C::kScales);
  __shared__ uint32_t tmem_slot;
  const uint32_t full = smem_u32(bars), empty = full + 8 * C::kMaxStages, done = empty + 8 * C::kMaxStages;
  // a stage: rows_x tokens, then the rows of w.  Products take 128 tokens all the same: what lies behind the last one
  // reaches rows of the result that are not written
  const int stages = p.stages, x_bytes = p.rows_x * kBlockK, stage_bytes = x_bytes + kN * kBlockK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = kSplit ? p.split : 1, rank = kSplit ? blockIdx.x % split : 0;
  const int first = kSplit ? blockIdx.x / split : blockIdx.x, step = kSplit ? gridDim.x / split : gridDim.x;
  const int begin = kSplit ? (int)((long)p.blocks * rank / split) : 0;  // this CTA's blocks
  const int end = kSplit ? (int)((long)p.blocks * (rank + 1) / split) : p.blocks;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(full + 8 * i, 1 + C::kWarps);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < C::kBufs / C::kGroup; ++i) mbar_init(done + 8 * i, 1);
    fence_mbar_init();
    prefetch_tensormap(&p.tmap_x);
    prefetch_tensormap(&p.tmap_w);
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_slot), C::kBufs * kN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  await_grid();

  bool ok = true;
#ifdef GDN_TEST_HOOKS
  const uint32_t limit = !g_test_give_up ? kWaitLimit : warp == C::kFirst ? 0 : kTestWaitLimit;
#else
  constexpr uint32_t limit = kWaitLimit;
#endif
  // A warp whose wait ran out goes on to the barriers behind the sums: the others of its CTA and cluster may have
  // passed the same wait.
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (ok && !warp_wait(bar, parity, limit)) {
      raise_error(p.err, kErrTimeout);
      ok = false;
    }
    return ok;
  };
  const int tiles = p.tiles_m * p.tiles_n;
  // large tiles: 384 threads are launched with 168 registers each; 56 in the first four warps leave 224 for the sums'
  if (warp < C::kFirst) {
    if constexpr (C::kLarge) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      int i = 0, pass = 0;  // stage, passes over the ring
      for (int id = first; id < tiles && ok; id += step) {
        int m, n;
        tile_of(id, p.tiles_m, p.tiles_n, m, n);
        for (int b = begin; b < end; ++b) {
          if (pass && !await(empty + 8 * i, (pass - 1) & 1)) break;
          const uint32_t at = smem_u32(smem) + i * stage_bytes;
          warp_load_stage(full + 8 * i, stage_bytes, at, &p.tmap_x, m * C::kTileM, at + x_bytes, &p.tmap_w, n * C::kTileN,
                          b * kBlockK);
          if (++i == stages) i = 0, ++pass;
        }
      }
      // copies in flight land before the CTA ends, after a wait that ran out too
      for (int c = 0; c < stages; ++c) {
        const int passes = pass + (c < i);  // loads into stage c
        if (passes) mbar_wait(full + 8 * c, (passes - 1) & 1, limit);
      }
    } else if (warp == 1) {
      // A full stage has its loads and the word of the sums that they have read what lay in its place of tensor memory: one wait
      // for each block.  The tensor cores hold about two instructions ahead, and a wait takes 150 cycles beside them: with
      // two the products of a block took 711 cycles instead of 552.
      int i = 0, pass = 0, j = 0;
      for (int id = first; id < tiles && ok; id += step)
        for (int b = begin; b < end; ++b, ++j) {
          if (!await(full + 8 * i, pass & 1)) break;
          tc_fence_after();
          const uint32_t at = smem_u32(smem) + i * stage_bytes;
          warp_mma_e4m3(tmem + j % C::kBufs * kN, sw128_desc(at), sw128_desc(at + x_bytes),
                        idesc_e4m3_f32(C::kTileM, kN), empty + 8 * i, done + 8 * (j % C::kBufs / C::kGroup),
                        C::kGroup == 1 || j % C::kGroup == C::kGroup - 1 || b + 1 == end);
          if (++i == stages) i = 0, ++pass;
        }
      // products in flight end before the CTA does, after a wait that ran out too
      if (i || pass) warp_wait(empty + 8 * (i ? i - 1 : stages - 1), (i ? pass : pass - 1) & 1, limit);
    }
  } else {
    if constexpr (C::kLarge) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int quarter = warp & 3, own = warp - C::kFirst, side = own >> 2;  // side: of the columns
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + side * C::kCols;
    for (int i = 0; i < C::kBufs; ++i) first_lane_arrive(full + 8 * i, lane);  // tensor memory is free at first
    int stage = C::kBufs % stages;  // of the block that goes to the place just read
    float* mine = (C::kLarge ? stage_out : reinterpret_cast<float*>(smem)) + own * 32 * C::kPitch;
    constexpr int kAhead = C::kAhead;
    float* own_x = scales + own * 32;  // its tokens' scales, a row for each block of two groups
    float* own_w = scales + 2 * kAhead * 32 * C::kWarps + own * kAhead;
    int j = 0, group = 0;
    for (int id = first; id < tiles && ok; id += step) {
      int m, n;
      tile_of(id, p.tiles_m, p.tiles_n, m, n);
      const long t0 = (long)m * C::kTileM + quarter * 32, t = t0 + lane;
      const long n0 = (long)n * C::kTileN + side * C::kCols;
      // tokens and columns behind the last ones take the last ones' scales: what they are multiplied with is not written
      const float* sw = p.w_scale + (min(n0, (long)p.n - 1) >> 7) * p.blocks;
      float2 acc[C::kCols / 2];
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      // a group of blocks' scales, neighbours of a token's row by neighbouring lanes
      auto fetch = [&](int b) {
        const int to = (group + (b > begin)) & 1, u = lane % kAhead;
        if (b + u < end) {
          const float* from = p.x_scale + b + u;
          float* x_to = own_x + (to * kAhead + u) * 32 * C::kWarps;
#pragma unroll
          for (int i = lane / kAhead; i < 32; i += 32 / kAhead) copy4(x_to + i, from + min(t0 + i, (long)p.tokens - 1) * p.blocks);
          if (lane < kAhead) copy4(own_w + to * kAhead * C::kWarps + u, sw + b + u);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      fetch(begin);
      // the scale of block b; at the first one of a group, the next group's are fetched
      auto scale = [&](int b) {
        const int u = (b - begin) % kAhead;
        if (u == 0) {
          if (b > begin) ++group;
          fetch(b + kAhead);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          __syncwarp();
        }
        return own_x[((group & 1) * kAhead + u) * 32 * C::kWarps + lane] * own_w[(group & 1) * C::kWarps * kAhead + u];
      };
      auto add = [&](const uint32_t(&d)[32], int c, float s) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          acc[c * 16 + i] = __ffma2_rn(make_float2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])),
                                       make_float2(s, s), acc[c * 16 + i]);
      };
      auto read = [&]() {  // a block's results are read: its place is free
        first_lane_arrive(full + 8 * stage, lane);
        if (++stage == stages) stage = 0;
        ++j;
      };
      uint32_t d[2][32];
      if constexpr (C::kLarge) {
        float s = 0.f;
        // Block b's products are there: its scale, and the first 32 of its columns on their way.
        auto start = [&](int b) {
          s = scale(b);
          if (!await(done + 8 * (j & 1), j >> 1 & 1)) return;
          tc_fence_after();
          tmem_ld_begin(lanes + (j & 1) * kN, d[0]);
        };
        if (begin < end) start(begin);
#pragma unroll 1
        for (int b = begin; b < end && ok; ++b) {
          const float now = s;
          const uint32_t at = lanes + (j & 1) * kN;
          // 32 columns are on their way while the 32 before them are added: the next block's first ones beside its last
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld_end(d[c & 1]);
            if (c < 3) {
              tmem_ld_begin(at + (c + 1) * 32, d[~c & 1]);
            } else {
              tc_fence_before();
              read();
              if (b + 1 < end) start(b + 1);
            }
            add(d[c & 1], c, now);
          }
        }
      } else {
#pragma unroll 1
        for (int b = begin; b < end; b += 2) {
          const bool two = b + 1 < end;
          const float s0 = scale(b), s1 = two ? scale(b + 1) : 0.f;
          if (!await(done + 8 * (j % C::kBufs / 2), j / C::kBufs & 1)) break;
          tc_fence_after();
          tmem_ld_begin(lanes + j % C::kBufs * kN, d[0]);
          if (two) tmem_ld_begin(lanes + (j + 1) % C::kBufs * kN, d[1]);
          tmem_ld_end(d[0]);
          tmem_ld_end(d[1]);
          tc_fence_before();
          read();
          if (two) read();
          add(d[0], 0, s0);
          if (two) add(d[1], 0, s1);
        }
      }
      ++group;
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
      if constexpr (kSplit) {  // every product of this CTA is done when its sums are: the ring is free
        float* part = reinterpret_cast<float*>(smem) + (quarter * 32 + lane) * C::kPartPitch + side * C::kCols;
        asm volatile("bar.sync 1, %0;" ::"n"(C::kWarps * 32) : "memory");
        if (t < p.tokens)
#pragma unroll
          for (int i = 0; i < C::kCols / 4; ++i)
            reinterpret_cast<float4*>(part)[i] = make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x, acc[2 * i + 1].y);
        break;
      }
      // a small tile's CTA has no other one: its ring takes rows of any alignment on their way out
      if constexpr (!C::kLarge)
        if (!p.whole_out) asm volatile("bar.sync 1, %0;" ::"n"(C::kWarps * 32) : "memory");
      if (!ok) break;
      if (p.whole_out) {  // whole sectors of a row from its thread
        if (t < p.tokens) {
          const long at = t * p.out_stride + n0;
          if (p.out_f32) {
            float* to = static_cast<float*>(p.out) + at;
#pragma unroll
            for (int i = 0; i < C::kCols / 8; ++i) {
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
            for (int i = 0; i < C::kCols / 16; ++i) {
              uint32_t v[8];
#pragma unroll
              for (int q = 0; q < 8; ++q) v[q] = pack_bf2(acc[8 * i + q].x, acc[8 * i + q].y);
              if (n0 + 16 * i < p.n) st_global32(to + 16 * i, v);
            }
          }
        }
      } else {
        // Rows of any alignment, 32 x 16 words at a time through shared memory: half a row of fp32 values or a row of 32 bf16
        // ones a store, sixteen stores of a lane at once: 777 x 5003 x 2041 15.5 us (bf16 15.1), 19.8 with one store after another.
        if (p.out_f32) {
          const int half = lane >> 4, col = lane & 15;
          const long rows = p.tokens - t0 - half;
          float* to = static_cast<float*>(p.out) + (t0 + half) * p.out_stride + n0 + col;
#pragma unroll
          for (int c = 0; c < C::kCols / 16; ++c) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              mine[lane * C::kPitch + 2 * i] = acc[c * 8 + i].x;
              mine[lane * C::kPitch + 2 * i + 1] = acc[c * 8 + i].y;
            }
            __syncwarp();
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = mine[(2 * i + half) * C::kPitch + col];
            if (n0 + c * 16 + col < p.n) {
              float* at = to + c * 16;
#pragma unroll
              for (int i = 0; i < 16; ++i, at += 2 * p.out_stride)
                if (2 * i < rows) *at = v[i];
            }
          }
        } else {
          uint32_t* words = reinterpret_cast<uint32_t*>(mine);
          const uint16_t* values = reinterpret_cast<const uint16_t*>(mine) + lane;
          const long rows = p.tokens - t0;
          uint16_t* to = static_cast<uint16_t*>(p.out) + t0 * p.out_stride + n0 + lane;
#pragma unroll
          for (int c = 0; c < C::kCols / 32; ++c) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) words[lane * C::kPitch + i] = pack_bf2(acc[c * 16 + i].x, acc[c * 16 + i].y);
            __syncwarp();
            uint16_t* at = to + c * 32;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint16_t v[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = values[(16 * h + i) * 2 * C::kPitch];
              if (n0 + c * 32 + lane < p.n)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (16 * h + i < rows) at[(16 * h + i) * p.out_stride] = v[i];
            }
          }
        }
      }
    }
  }
  __syncwarp();
  if constexpr (kSplit) {
    cluster_sync();
    if (warp >= C::kFirst) {  // kN / 8 lanes take a token, a lane eight columns
      int m, n;
      tile_of(first, p.tiles_m, p.tiles_n, m, n);
      constexpr int kLanes = kN / 8, kTokens = 32 / kLanes;
      const int rows = (int)min((long)C::kTileM, p.tokens - (long)m * C::kTileM), last = rows * (rank + 1) / split;
      const long n0 = (long)n * C::kTileN + lane % kLanes * 8;
#pragma unroll 2
      for (int r = rows * rank / split + (warp - C::kFirst) * kTokens + lane / kLanes; r < last; r += C::kWarps * kTokens) {
        const long t = (long)m * C::kTileM + r;
        const uint32_t at = smem_u32(reinterpret_cast<float*>(smem) + r * C::kPartPitch + lane % kLanes * 8);
        float4 part[kMaxSplit][2];
#pragma unroll
        for (int i = 0; i < kMaxSplit; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            part[i][h] = i < split ? ld_cluster(in_cta(at + 16 * h, (rank + i) & (split - 1))) : make_float4(0.f, 0.f, 0.f, 0.f);
        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kMaxSplit; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            y[4 * h] += part[i][h].x;
            y[4 * h + 1] += part[i][h].y;
            y[4 * h + 2] += part[i][h].z;
            y[4 * h + 3] += part[i][h].w;
          }
        if (p.whole_out) {
          if (n0 < p.n) {
            if (p.out_f32) {
              float4* to = reinterpret_cast<float4*>(static_cast<float*>(p.out) + t * p.out_stride + n0);
              to[0] = make_float4(y[0], y[1], y[2], y[3]);
              to[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + t * p.out_stride + n0) =
                  make_uint4(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]), pack_bf2(y[4], y[5]), pack_bf2(y[6], y[7]));
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n0 + i < p.n) store_out(p, t, n0 + i, y[i]);
        }
      }
    }
    __syncwarp();
    cluster_sync();  // the others have read this CTA's part
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::kBufs * kN);
}

template <int kN, bool kSplit>
cudaError_t launch_tiles(const LaunchEnv& env, const MatmulParams& p, long ctas) {
  using C = Tiles<kN>;
  static int done[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(tile_kernel<kN, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = 1;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = env.stream;
  cfg.attrs = attr;
  cfg.numAttrs = kSplit ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, tile_kernel<kN, kSplit>, p);
}

template <int kN>
cudaError_t encode_tiles(MatmulParams& p, const Fp8Matmul& m) {
  p.tiles_m = (int)((m.tokens + 127L) / 128);
  p.tiles_n = (int)((m.n + (long)kN - 1) / kN);
  // Rows of x that are not there are not asked for: filling them with zeroes takes the time of loads (17 tokens x
  // 16384 x 2048 in tiles of 64 rows: 17.8 us with them, 12.5 without).  What the stage holds in their place reaches rows of
  // the result that are not written.
  p.rows_x = m.tokens < 128 ? (m.tokens + 7) / 8 * 8 : 128;
  const int fit = Tiles<kN>::kRing / ((p.rows_x + kN) * kBlockK);
  p.stages = fit < Tiles<kN>::kMaxStages ? fit : Tiles<kN>::kMaxStages;
  const cudaError_t e = encode_u8_2d_sw128(&p.tmap_x, m.x, m.k, m.tokens, m.x_stride, kBlockK, p.rows_x);
  return e == cudaSuccess ? encode_u8_2d_sw128(&p.tmap_w, m.w, m.k, m.n, m.w_stride, kBlockK, kN) : e;
}

cudaError_t launch_many(const LaunchEnv& env, MatmulParams& p, const Fp8Matmul& m) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long bytes = m.out_f32 ? 4 : 2;
  p.whole_out = (reinterpret_cast<uintptr_t>(m.out) & 31u) == 0 && m.out_stride * bytes % 32 == 0 && m.n * bytes % 32 == 0;
  // Tiles of 64 rows of w, a CTA each, while every one has an SM; a block costs them 0.27 us, the large ones' 0.5 us for four
  // times the products.  256 tokens x 4096 x 4096 (128 small tiles): 11.5 us, large 18.9; x 10240 (320): 33 : 19.9; 64 x
  // 16384 x 2048 (256): 14.7 : 11.8.  Few tiles share their k: 64 x 2048 x 6144 (32 tiles) 23 us with one CTA a tile,
  // 13.7 with two, 9.8 with four (9.1 by now), 11 with eight; 128 x 4096 x 4096 (64 tiles) 16.8, 11.2, 13.4 (256 CTAs).
  const long small = ((m.tokens + 127L) / 128) * ((m.n + 63L) / 64);
  if (small <= sms) {
    e = encode_tiles<64>(p, m);
    if (e != cudaSuccess) return e;
    p.split = 1;
    while (p.split < kMaxSplit && 2 * p.split <= p.blocks && 2 * p.split * small <= sms) p.split *= 2;
    if (p.split > 1) return launch_tiles<64, true>(env, p, small * p.split);
    return launch_tiles<64, false>(env, p, small);
  }
  e = encode_tiles<256>(p, m);
  if (e != cudaSuccess) return e;
  const long tiles = (long)p.tiles_m * p.tiles_n;
  // Two CTAs share a large tile where that saves the time of 16 blocks; the join takes 4 to 5 us.  32 tokens x 10240 x 5120 (40
  // tiles of 40 blocks): 22.4 us with one CTA a tile, 16.8 with two; 300 x 4096 x 4096 (48 of 32) 18.9 : 16.8; 64 x 16384 x
  // 2048 (64 of 16) 11.9 : 13.3.
  p.split = 2 * tiles <= sms && p.blocks >= 32 ? 2 : 1;
  if (p.split > 1) return launch_tiles<256, true>(env, p, tiles * p.split);
  return launch_tiles<256, false>(env, p, tiles < sms ? tiles : sms);
}

}  // namespace

#ifdef GDN_TEST_HOOKS
cudaError_t test_set_give_up_matmul(unsigned on) { return cudaMemcpyToSymbol(g_test_give_up, &on, sizeof on); }
#endif

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
  p.blocks = (m.k - 1) / kBlockK + 1;
  p.out = m.out;
  p.out_stride = m.out_stride;
  p.out_f32 = m.out_f32;
  p.err = env.err;
  const unsigned few = (unsigned)((m.n + 15L) / 16);
  if (m.tokens <= 8) return launch_early(few_kernel<1>, dim3(few), kFewWarps * 32, 0, env.stream, p);
  if (m.tokens <= 16) return launch_early(few_kernel<2>, dim3(few), kFewWarps * 32, 0, env.stream, p);
  return launch_many(env, p, m);
}

}  // namespace gdn
