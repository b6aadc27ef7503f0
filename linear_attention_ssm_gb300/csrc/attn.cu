// attn.cu -- softmax attention of new tokens over a paged key/value cache, on the tcgen05 tensor cores.
//
// A tile is 128 rows of one key head of one sequence: the group's query heads of consecutive tokens,
// row = token * group + head.  Per block of 128 keys
//   S = Q K^T (fp32, tensor memory)  ->  p = 2^(S - m)  ->  P (16 bits, tensor memory, over S)  ->  O += P V
// with the running maximum m and sum l of every row in the registers of the thread that owns the row, O
// in tensor memory.  m is raised (and O, l scaled down) only when a block exceeds it by more than 2^8:
// the weights stay below 2^8 and the common block leaves O alone.
//
// A tile's two S slots let one step's softmax run beside the other's products.  Long chunks at D = 128 take two
// tiles a CTA (kTiles = 2: K and V are read once for 256 rows) with slots of 64 keys, half a block; otherwise a CTA
// has one tile and slots of a block (kTiles = 1; at D = 256 O alone fills half the tensor memory).
//
// Warps: four a tile for the softmax; two that issue products (a tile's each, or with one tile one for
// the scores and one for O), so that one's waiting does not idle the tensor cores; one that loads Q, K and
// V by TMA, K and V into a ring of 32 KB stages; one that goes over the value rows that some row of the tile
// does not see.  An e4m3 cache has four or eight warps that widen its codes into the stages instead of the
// last two, and one that reads pages and scales ahead.
//
// A value that a row does not see has the weight 0 there, and 0 * NaN is not 0.  Value rows behind the last key
// (a page's unused rows may hold anything) are zeroes in their stage, and so are infinities and NaN in rows that
// some of the tile's tokens come before; the rows that do see those get them back at the segment's end
// (add_odd_values), which costs time only where there are any.
//
// Work: the (tile, block) pairs of all sequences in one line, cut into one equal piece for each SM.  A
// tile that a cut falls into leaves its parts (O, m, l) in the workspace for a second kernel to join,
// so a few long sequences spread over the whole GPU as a large batch does.
//
// Measured on a GB300 (of 1956 TFLOP/s of bf16 products; calls in a CUDA graph): a prompt of 8192 tokens, 32 heads of
// 128, 435 us, 1.26 PFLOP/s, 65 % -- products, nine tenths of the time by their own clocks, those of 64 keys at half the
// rate; from e4m3 pages 634 us.  2048 tokens after 30001, 16 heads of 256, 707 us, 1.47 PFLOP/s, 75 % (758 us in a row of
// calls, which meet the power limit) -- keys and values from L2, 128 KB a block for each SM.  Chunks of eight prompts of 17
// to 1500 tokens, 16 heads of 256, 131 us from bf16 pages, 880 TFLOP/s, and 244 us from e4m3 ones, 472 TFLOP/s --
// widening the codes, once for each tile, beside the softmax, whose instructions leave the caches between them.  17
// tokens after 1000, 48 heads of 128, 15 us -- latency, of two launches.
#include <cstring>

#include "attn_common.cuh"
#include "chunk_common.cuh"

namespace gdn {
namespace {

constexpr uint32_t kStage = 32768, kRaw = 16384;

// ---------------------------------------------------------------- layout of a CTA

// e4m3: what the warps that widen the codes and those of the softmax need to know of a block of keys.
struct BlockMeta {
  uint32_t kf[kBlock];  // a key's power of two relative to the block's largest, times 2^kWiden, twice in binary16
  uint32_t vf[kBlock];  // the same of a value
  float ku, ev;         // the block's largest key scale times the softmax scale; log2 of its largest value scale
  int have, flags;      // visible keys; kFirst, kLast: of a segment, kEnd: no more blocks; from kSeen on: keys that every row sees
};
enum : int { kFirst = 1, kLast = 2, kEnd = 4, kSeen = 3 };
constexpr int kMeta = 8;         // blocks that the pages and scales are ahead
constexpr float kWeight = 7.f;   // log2 of the factor on binary16 weights
constexpr int kWiden = 7;        // and of that on widened codes: 448 * 2^7 is the most that binary16 takes
constexpr float kUnitMin = 0x1p-126f, kUnitMax = 0x1.fffffep127f;  // bounds of a score's unit

template <int D, int kTiles, bool kE4M3>
struct Cfg {
  static constexpr int kSoftWarps = 4 * kTiles;
  static constexpr int kConvGroups = kE4M3 ? 3 - kTiles : 0;  // of four warps that widen codes, taking stages in turn
  static constexpr int kConvWarps = 4 * kConvGroups;
  static constexpr int kThreads = 32 * (kSoftWarps + 4 + kConvWarps);
  static constexpr uint32_t kQ = kTiles * 128 * D * 2;
  // The rings' stages: the products' (32 KB); e4m3: fewer of those, and the codes' (16 KB).
  static constexpr int kRawStages = kE4M3 ? 3 : 0;
  static constexpr int kStages = (int)((224 * 1024 - kQ) / kStage) - (kE4M3 ? 2 : 0);
  static constexpr int kParts = D / 128;  // stages of a block's keys, and of its values
  static constexpr uint32_t kOffStage = kQ;
  static constexpr uint32_t kOffRaw = kOffStage + kStages * kStage;
  static constexpr uint32_t kOffMeta = kOffRaw + kRawStages * kRaw;
  static constexpr uint32_t kOffBar = kOffMeta + (kE4M3 ? kMeta * sizeof(BlockMeta) : 0);
  static constexpr uint32_t kSmem = kOffBar + 1024 + 1024;  // barriers; alignment of the base
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kStages <= 6 && kRawStages <= 3 && kThreads <= 32 * 60, "places of the barriers and of the scan");
  // of the four warps behind the softmax's: the products (two), Q, K and V by TMA, value rows that some row
  // does not see (e4m3: scales)
  static constexpr int kMma0 = kSoftWarps, kMma1 = kSoftWarps + 1, kLoad = kSoftWarps + 2, kTail = kSoftWarps + 3;
  // Scores that a softmax warp holds at a time; a step's are read twice, for the maximum and for the weights.  Few
  // registers, and short code for the instruction cache that warps of several kinds share: with 64, 8192 prompt
  // tokens take 435 us (434 with 32), from e4m3 pages 688 (634); eight prompts' chunks at D = 256 154 (130), e4m3 271 (242).
  static constexpr int kCols = 32;
  // Keys whose scores a slot holds: a block's, or with two tiles half of them.  A tile has two slots, so that
  // its next scores are there when the weights of these are done (8192 prompt tokens 467 us; with a slot of 128
  // keys for each tile 605, with both halves' scores from one product 579).  A product of 64 keys costs what one
  // of 128 does (558 and 524 clocks at D = 128, measured alone): products take nine tenths of the time by that.
  static constexpr int kKeys = kTiles == 2 ? 64 : 128, kHalves = 128 / kKeys;
  static constexpr uint32_t kColO = 256;  // tensor memory: the slots, 256 columns, then O
};

struct Bars {
  uint32_t full, empty, tail, s_full, p_full, o_full, q_full, q_empty, done, meta_full, meta_empty, q_ready, raw_full, raw_empty;  // shared addresses of the first of each kind
};

// A position in the ring of stages: which stage, and which pass over the ring.
template <int kStages>
struct Ring {
  int i = 0;
  uint32_t pass = 0;
  __device__ __forceinline__ void step() {
    if (++i == kStages) {
      i = 0;
      pass ^= 1u;
    }
  }
  __device__ __forceinline__ void skip(long n) {
    const long at = i + n;
    pass ^= (uint32_t)(at / kStages) & 1u;
    i = (int)(at % kStages);
  }
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// 16 columns of this warp's 32 lanes; tmem_st_wait: this thread's stores so far have been done
__device__ __forceinline__ void tmem_st16_begin(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 2^e, e <= 15, twice in binary16 (0 below its range)
__device__ __forceinline__ uint32_t half2_power(int e) {
  const uint32_t h = e >= -14 ? (uint32_t)(15 + e) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
  return h | h << 16;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr uint32_t kInfBf16 = 0x7F807F80u;  // two magnitudes from here on are not finite
__device__ __forceinline__ uint32_t top_bf16(const uint4& x) {  // the largest of the even, of the odd magnitudes
  return __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
}
// Eight bf16 values, or 16 e4m3 codes, with those that are not finite as zeroes (codes: whether there were any).
__device__ __forceinline__ uint4 zero_odd_bf16(const uint4& x) {
  return make_uint4(x.x & ~__vcmpgeu2(x.x & 0x7FFF7FFFu, kInfBf16), x.y & ~__vcmpgeu2(x.y & 0x7FFF7FFFu, kInfBf16),
                    x.z & ~__vcmpgeu2(x.z & 0x7FFF7FFFu, kInfBf16), x.w & ~__vcmpgeu2(x.w & 0x7FFF7FFFu, kInfBf16));
}
__device__ __forceinline__ bool zero_odd_e4m3(uint4& x) {
  const uint32_t odd[4] = {__vcmpeq4(x.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu), __vcmpeq4(x.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu),
                           __vcmpeq4(x.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu), __vcmpeq4(x.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu)};
  x = make_uint4(x.x & ~odd[0], x.y & ~odd[1], x.z & ~odd[2], x.w & ~odd[3]);
  return (odd[0] | odd[1] | odd[2] | odd[3]) != 0;
}

// O of this warp's 32 rows plus the infinities and NaN among the values of keys key0 .. key1 - 1 of sequence n, up
// to each row's last one (any positive weight leaves them what they are).
template <int D, bool kE4M3>
__device__ __forceinline__ void add_odd_values(const AttnParams& p, uint32_t t_o, int n, int hk, int key0, int key1, int last) {
  key1 = min(key1, __reduce_max_sync(0xFFFFFFFFu, last) + 1);
  const int shift = p.cache.page_shift;
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    float o[16];
    tmem_ld16(t_o + c, o);
#pragma unroll 1
    for (int key = key0; key < key1; ++key) {
      int id = p.cache.table[(long)n * p.cache.max_pages + (key >> shift)];
      if ((unsigned)id >= (unsigned)p.cache.num_pages) id = 0;
      const long row = (((long)id * p.Hkv + hk) << shift) + (key & ((1 << shift) - 1));
      if (key > last) continue;
      if constexpr (kE4M3) {
        const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.cache.v) + row * D + c);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if ((w[i >> 2] >> (8 * (i & 3)) & 0x7Fu) == 0x7Fu) o[i] = __uint_as_float(0x7FFFFFFFu);
      } else {
        const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.cache.v) + row * D + c);
        const uint4 x = at[0], y = at[1];
        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t v = i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16;
          if ((v & 0x7F800000u) == 0x7F800000u) o[i] += __uint_as_float(v);
        }
      }
    }
    tmem_st16(t_o + c, o);
  }
}

template <int D, int kTiles, bool kE4M3>
__global__ void __launch_bounds__(Cfg<D, kTiles, kE4M3>::kThreads, 1) attn_kernel(const __grid_constant__ AttnParams p) {
  using C = Cfg<D, kTiles, kE4M3>;
  constexpr int kStages = C::kStages, kParts = C::kParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int step = kTiles * p.sub;

  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 59);
  volatile uint32_t* odd_seen = tmem_slot + 1;  // set where a value was zeroed that some row sees, and not cleared
  WalkStart* start = reinterpret_cast<WalkStart*>(bars + 60);
  long* scan = reinterpret_cast<long*>(bars + 66);
  const uint32_t b0 = smem_u32(bars);
  const Bars bar = {b0, b0 + 8 * 6, b0 + 8 * 12, b0 + 8 * 18, b0 + 8 * 22, b0 + 8 * 26, b0 + 8 * 30, b0 + 8 * 32, b0 + 8 * 34, b0 + 8 * 35, b0 + 8 * 43, b0 + 8 * 51,
                    b0 + 8 * 53, b0 + 8 * 56};
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar.full + 8 * i, kE4M3 ? 4 : 1);
      mbar_init(bar.empty + 8 * i, kTiles);
      mbar_init(bar.tail + 8 * i, 1);
    }
    for (int i = 0; i < 2 * kTiles; ++i) {
      mbar_init(bar.s_full + 8 * i, 1);
      mbar_init(bar.p_full + 8 * i, 4);
      mbar_init(bar.o_full + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar.q_full + 8 * i, 1);
      mbar_init(bar.q_ready + 8 * i, 4);
      mbar_init(bar.q_empty + 8 * i, 1);
    }
    mbar_init(bar.done, 2);
    if constexpr (kE4M3) {
      for (int i = 0; i < C::kRawStages; ++i) {
        mbar_init(bar.raw_full + 8 * i, 1);
        mbar_init(bar.raw_empty + 8 * i, 4);
      }
      for (int i = 0; i < kMeta; ++i) {
        mbar_init(bar.meta_full + 8 * i, 1);
        mbar_init(bar.meta_empty + 8 * i, 4 * 2 * kParts + C::kSoftWarps);  // each stage's four warps, the softmax's
      }
    }
    fence_mbar_init();
    prefetch_tensormap(&p.tmap_k);
    prefetch_tensormap(&p.tmap_v);
    prefetch_tensormap(&p.tmap_q);
    start->left = 0;
    *odd_seen = 0;
  }
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), 512);
  await_grid();
  if (tid < 2) p.desc[2 * blockIdx.x + tid] = make_int4(0, 0, 0, 0);
  find_start<C::kThreads>(p, step, scan, start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk walk;
  walk.begin(p, step, *start);
  Segment seg;
  bool ok = true;
  // A bounded wait of the whole warp, or (the products) of one thread.  After one that ran out the warp
  // takes no more work; the others' waits run out in turn.
  auto await_one = [&](uint32_t b, uint32_t parity) {
    if (!mbar_wait(b, parity, kWaitLimit)) {
      raise_error(p.err, kErrTimeout);
      ok = false;
    }
    return ok;
  };
  auto await = [&](uint32_t b, uint32_t parity) {
    await_one(b, parity);
    ok = __all_sync(0xFFFFFFFFu, ok);
    return ok;
  };

  auto finish = [&]() {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
  };

  if (warp < C::kSoftWarps) {
    // ------------------------------------------------------------------ softmax: one thread for a row
    const int sub = kTiles == 2 ? warp >> 2 : 0, w4 = warp & 3, row = w4 * 32 + lane;
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    const uint32_t t_o = tmem + lanes + C::kColO + sub * D;
    const int g = row % p.G, tok_in = row / p.G;
    uint8_t* sq = sm + sub * 128 * D * 2;
    // steps of this tile so far (slot and parity go by it), its products with V, blocks of the CTA; segments with rows
    uint32_t n_blk = 0, n_pv = 0, all_blk = 0, n_seg = 0;
    // Step b's slot, its barriers' parity, and its product with V.  A slot has barriers of its own: the next
    // scores may be here before the product of the step before them has ended, and no wait is for a phase that
    // could lie two behind.
    auto slot_of = [&](uint32_t b) { return 2 * sub + (b & 1u); };
    auto await_pv = [&](uint32_t b) { return await(bar.o_full + 8 * slot_of(b), (b >> 1) & 1u); };
    while (ok && walk.next(p, step, seg)) {
      const int hk = seg.hk, ntok = min(p.sub, seg.ntok - sub * p.sub);  // tokens of this tile
      const int row0 = seg.row0 + sub * p.sub, rows = max(ntok, 0) * p.G;
      const bool mine = tok_in < ntok;
      uint16_t* out = p.out + ((long)(row0 + tok_in) * p.Hq + hk * p.G + g) * D;
      if (seg.keys <= 0) {
        if (mine)
          for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(out)[c] = make_uint4(0, 0, 0, 0);
        continue;
      }
      float row_unit = p.scale_log2;  // e4m3: the power of two the row was divided by, less the factor on the keys
      if (kE4M3 && rows > 0) {
        // Q becomes binary16 where it lies, each thread its own row, divided by the power of two of its largest
        // finite value (a thread's pieces of 16 bytes lie in other banks than its neighbours')
        if (!await(bar.q_full + 8 * sub, n_seg++ & 1u)) break;
        if (w4 * 32 < rows) {
          auto at = [&](int c) { return reinterpret_cast<uint4*>(sq + sw128_offset(row, c * 8, 16384)); };
          uint32_t two = 0;  // of the even and of the odd values
#pragma unroll 2
          for (int c = 0; c < D / 8; ++c) {
            const uint4 x = *at(c);
            two = __vmaxu2(two, top_bf16(x));
          }
          uint32_t top = max(two & 0xFFFFu, two >> 16);
          if (top >= 0x7F80u) {  // an infinity or NaN among them
            top = 0;
#pragma unroll 1
            for (int c = 0; c < D; ++c) {
              const uint32_t x = reinterpret_cast<const uint16_t*>(at(c >> 3))[c & 7] & 0x7FFFu;
              if (x < 0x7F80u) top = max(top, x);
            }
          }
          const int e = min(max((int)(top >> 7) - 127, -120), 126);
          const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 2
          for (int c = 0; c < D / 8; ++c) {
            const uint4 x = *at(c);
            uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              y[k] = pack_half2(__uint_as_float(y[k] << 16) * inv, __uint_as_float(y[k] & 0xFFFF0000u) * inv);
            *at(c) = make_uint4(y[0], y[1], y[2], y[3]);
          }
          row_unit = __uint_as_float((uint32_t)(127 + e) << 23) * (1.f / (1 << kWiden));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.q_ready + 8 * sub);
      }
      if (p.z.p && mine && seg.j0 == 0 && seg.j1 == seg.nb) {  // the gate on its way to L2
        const uint16_t* z = p.z.p + (long)(row0 + tok_in) * p.z.token + (long)(hk * p.G + g) * p.z.head;
        for (int c = 0; c < D; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(z + c));
      }
      float m = -INFINITY, l = 0.f, r = -INFINITY;
      const int last = seg.pos0 + sub * p.sub + tok_in;  // the row's position: its last visible key
      const bool busy = w4 * 32 < rows;                   // this warp has rows at all
      constexpr int kCols = C::kCols, kKeys = C::kKeys, kHalves = C::kHalves;
      const uint32_t seg_blk = all_blk;
      all_blk += seg.j1 - seg.j0;
      if (kE4M3 && rows <= 0) {  // this tile has no rows in the segment: its warps still let its blocks go
        for (uint32_t b = seg_blk; b != all_blk && ok; ++b) {
          if (!await(bar.meta_full + 8 * (b % kMeta), b / kMeta & 1u)) break;
          if (lane == 0) mbar_arrive(bar.meta_empty + 8 * (b % kMeta));
        }
      }
      if (rows > 0) {
        const int i0 = seg.j0 * kHalves, i1 = seg.j1 * kHalves;  // steps of kKeys keys
        for (int i = i0; i < i1; ++i, ++n_blk) {
          const uint32_t slot = slot_of(n_blk), blk = seg_blk + (uint32_t)(i - i0) / kHalves;
          if (!await(bar.s_full + 8 * slot, (n_blk >> 1) & 1u)) break;
          tc_fence_after();
          if (busy) {
            const uint32_t t_s = tmem + lanes + slot * kKeys;
            const int lim = last + 1 - i * kKeys;  // columns from here on are not visible
            const bool masked = __any_sync(0xFFFFFFFFu, lim < kKeys);
            float ev = 0.f, unit = row_unit;  // log2 of the block's value scale; log2 units of this row's scores
            const BlockMeta* meta = reinterpret_cast<const BlockMeta*>(sm + C::kOffMeta) + blk % kMeta;
            if constexpr (kE4M3) {
              if (!await(bar.meta_full + 8 * (blk % kMeta), blk / kMeta & 1u)) break;
              ev = meta->ev;
              // A finite unit above zero: -inf (a masked score) times zero is NaN, and so is zero times infinity.  The
              // unit of a row of zeros over keys of zeros is 2^-237; where the bound acts, scores are below 2^-108.
              unit = fminf(fmaxf(unit * meta->ku, kUnitMin), kUnitMax);
            }
            float s[kCols], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int c0 = 0; c0 < kKeys; c0 += kCols) {
              tmem_ld32(t_s + c0, s);
              if (masked) {
#pragma unroll
                for (int k = 0; k < kCols; ++k)
                  if (c0 + k >= lim) s[k] = -INFINITY;
              }
#pragma unroll
              for (int k = 0; k < kCols; ++k) mx[k & 3] = fmaxf(mx[k & 3], s[k]);
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * unit;
            if (top > m + kLazy) {
              l *= ex2_approx(m - top);
              m = top;
            }
            // O is held in units of 2^r: the row's maximum times the block's largest value scale
            const float e = m + ev;
            const bool raise = e > r;
            if (__any_sync(0xFFFFFFFFu, raise)) {
              const float a = raise ? ex2_approx(r - e) : 1.f;
              if (raise) r = e;
              if (i > i0) {  // O holds the steps before this one: wait for their product, then scale
                if (!await_pv(n_pv - 1)) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  float o[16];
                  tmem_ld16(t_o + c, o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] *= a;
                  tmem_st16(t_o + c, o);
                }
              }
            }
            // weights 2^(s - m + d), d = e - r <= 0 the distance of this block's unit from O's; cut off at -40,
            // lest a block of tiny values vanish from l (P is zero in binary16 long before)
            const float d = kE4M3 && m > -INFINITY ? fmaxf(e - r, -40.f) : 0.f;
            const float off = (kE4M3 ? kWeight : 0.f) + (m == -INFINITY ? 0.f : d - m);
            const float2 unit2 = make_float2(unit, unit), off2 = make_float2(off, off);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
            for (int c0 = 0; c0 < kKeys; c0 += kCols) {
              tmem_ld32(t_s + c0, s);  // again: the weights go over scores that have been read
              if (masked) {
#pragma unroll
                for (int k = 0; k < kCols; ++k)
                  if (c0 + k >= lim) s[k] = -INFINITY;
              }
              float w[16];
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int at = 2 * (i + k);
                  float2 x = __ffma2_rn(make_float2(s[at], s[at + 1]), unit2, off2);
                  x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                  sum[k] = __fadd2_rn(sum[k], x);
                  // The weights' one rounding: the matrix instructions take both operands in one type, that of the cache
                  // (bf16: 2^-8 of a weight at most, while the sum l keeps fp32), or binary16 beside e4m3 codes (2^-11 where it is normal).
                  w[i + k] = __uint_as_float(kE4M3 ? pack_half2(x.x, x.y) : pack_bf2(x.x, x.y));
                }
              }
              tmem_st16_begin(t_s + c0 / 2, w);
            }
            tmem_st_wait();
            const float all = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            l += kE4M3 ? all * ex2_approx(-d - kWeight) : all;
          }
          if constexpr (kE4M3) {
            __syncwarp();
            if (lane == 0 && (i + 1) % kHalves == 0) mbar_arrive(bar.meta_empty + 8 * (blk % kMeta));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar.p_full + 8 * slot);
          ++n_pv;
        }
        if (!ok) break;
        if (!await_pv(n_pv - 1)) break;
        tc_fence_after();
        if (busy && __any_sync(0xFFFFFFFFu, *odd_seen != 0)) {
          // bf16: the sequence and the tile's first position from values that the loop holds anyway; kept for this
          // through the loop they cost it registers (2048 tokens after 30001: 706 us, 714 with them kept).  e4m3 the
          // other way round: the kernel is short of instruction cache (8192 prompt tokens: 633 us, 677 with the lookup).
          int n = seg.n, key0 = seg.pos0 + 1;
          if constexpr (!kE4M3) {
            int first, len;
            // (lane 0 has a row; below 0: bad cu_seqlens, whose rows are unspecified)
            n = max(attn_seq_of(p.cu, p.N, p.T, row0 + __shfl_sync(0xFFFFFFFFu, tok_in, 0), first, len), 0);
            key0 = last - sub * p.sub - tok_in + 1;
          }
          add_odd_values<D, kE4M3>(p, t_o, n, hk, max(key0, seg.j0 * kBlock), seg.j1 * kBlock, mine ? last : -1);
        }
        const bool whole = seg.j0 == 0 && seg.j1 == seg.nb;
        // O in units of 2^m (half the exponent at a time where both ends of the range meet)
        const float unit_o = kE4M3 && m > -INFINITY ? ex2_approx(0.5f * (r - m - kWeight - kWiden)) : 1.f;
        if (busy) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const uint16_t* z = p.z.p + (long)(row0 + tok_in) * p.z.token + (long)(hk * p.G + g) * p.z.head;
          const int part = 2 * blockIdx.x + (seg.j0 == 0 ? 1 : 0);
          float4* dst = p.part + (long)part * (kPartBytes / sizeof(float4)) + sub * (D / 4) * 128 + row;
          if (!whole) p.ml[(long)part * 256 + sub * 128 + row] = make_float2(m, l);
          uint4 zz[4];  // the gate of the next 32 values
          const bool gated = whole && mine && p.z.p;
          auto gate = [&](int c) {
#pragma unroll
            for (int k = 0; k < 4; ++k) zz[k] = gated ? *reinterpret_cast<const uint4*>(z + c + 8 * k) : make_uint4(0, 0, 0, 0);
          };
          gate(0);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(t_o + c, o);
            // two at a time: by both halves of the unit, the second with 1 / l in a tile that is whole
            auto times = [&](float f) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 y = __fmul2_rn(make_float2(o[i], o[i + 1]), make_float2(f, f));
                o[i] = y.x;
                o[i + 1] = y.y;
              }
            };
            if constexpr (kE4M3) times(unit_o);
            if (!whole) {
              if constexpr (kE4M3) times(unit_o);
#pragma unroll
              for (int i = 0; i < 8; ++i) dst[(c / 4 + i) * 128] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            } else {
              times(kE4M3 ? unit_o * inv : inv);
              if (__any_sync(0xFFFFFFFFu, l == 0.f)) {  // no visible key: zero
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : o[i];
              }
              if (p.z.p) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t zr[4] = {zz[k].x, zz[k].y, zz[k].z, zz[k].w};
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    float2 e = __fmul2_rn(make_float2(__uint_as_float(zr[x] << 16), __uint_as_float(zr[x] & 0xFFFF0000u)),
                                          make_float2(-kLog2e, -kLog2e));
                    e = __fadd2_rn(make_float2(ex2_approx(e.x), ex2_approx(e.y)), make_float2(1.f, 1.f));
                    const float2 y = __fmul2_rn(make_float2(o[8 * k + 2 * x], o[8 * k + 2 * x + 1]), make_float2(rcp_approx(e.x), rcp_approx(e.y)));
                    o[8 * k + 2 * x] = y.x;
                    o[8 * k + 2 * x + 1] = y.y;
                  }
                }
                if (c + 32 < D) gate(c + 32);
              }
              if (mine) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  uint32_t w[8];
#pragma unroll
                  for (int x = 0; x < 8; ++x) w[x] = pack_bf2(o[16 * k + 2 * x], o[16 * k + 2 * x + 1]);
                  if (p.wide_out) {
                    st_global32(out + c + 16 * k, w);
                  } else {
                    *reinterpret_cast<uint4*>(out + c + 16 * k) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(out + c + 16 * k + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                  }
                }
              }
            }
          }
        }
        if (!whole && warp == 0 && lane == 0)
          p.desc[2 * blockIdx.x + (seg.j0 == 0 ? 1 : 0)] =
              make_int4(seg.row0, seg.ntok, hk, kPart | (seg.j1 == seg.nb ? kPartLast : 0));
        tc_fence_before();
      }
    }
    finish();
    return;
  }
  if (kE4M3 && warp >= C::kSoftWarps + 4) {
    // ------------------------------------------------------------------ e4m3: codes -> binary16 stages
    // Four warps a stage, in groups that take the stages in turn: a stage's codes are widened (exactly, two
    // an instruction), multiplied by 2^kWiden and their row's power of two relative to the block's largest, and
    // written in the layout that the TMA gives a bf16 cache.  Products are exact for rows at most 2^22 below the
    // block's largest; down to 2^31 below they lose at most 2^-39 of its largest value, and rows further below are
    // zeroes, less than 2^-30 of it.
    constexpr int kGroups = C::kConvGroups > 0 ? C::kConvGroups : 1, kUnits = 8;
    constexpr int kRawStages = C::kRawStages > 0 ? C::kRawStages : 1;
    const int cw = warp & 3, group = (warp - (C::kSoftWarps + 4)) >> 2;
    const BlockMeta* metas = reinterpret_cast<const BlockMeta*>(sm + C::kOffMeta);
    // A thread's 16 codes of a stage, unit u: 128 rows of 128 codes (narrow), or 64 of 256 (a block's
    // values at D = 256: wide), in 64-code columns [rows][64].  Lanes 0-3 take a row's 64 codes, lanes 4-7
    // those of the row below: eight lanes read 128 neighbouring bytes, and the swizzle spreads their
    // stores over all banks.
    const int piece = lane & 3, odd = lane >> 2 & 1;
    const int row_narrow = cw * 4 + (lane >> 4) * 2 + odd, blk_narrow = lane >> 3 & 1, row_wide = cw * 2 + odd, blk_wide = lane >> 3;
    const int c_narrow = (2 * piece) ^ (row_narrow & 7), c_wide = (2 * piece) ^ (row_wide & 7);
    const int to_narrow = blk_narrow * 16384 + row_narrow * 128 + c_narrow * 16, to_wide = blk_wide * 8192 + row_wide * 128 + c_wide * 16;
    const int other_narrow = ((c_narrow ^ 1) - c_narrow) * 16, other_wide = ((c_wide ^ 1) - c_wide) * 16;  // to the second half
    // The order of the operands, each in kParts stages: K0 V0 K1 V1 .. with two tiles, with one K0 K1 V0 K2 V1 ..:
    // after a block's keys come the values of the block before it, if the segment has one, and the block's own
    // values, if it is the segment's last.  Where an operand has a stage for each group, a group has the same part
    // of every one; else the groups take the operands in turn.
    constexpr int kTurn = kGroups > kParts ? kGroups / kParts : 1;  // operands from one of this group's stages to its next
    static_assert(!kE4M3 || kGroups % kParts == 0, "a part of an operand for each group, or whole operands");
    const int part = kParts > 1 ? group : 0;
    uint32_t blk = 0xFFFFFFFFu;     // the latest block whose keys have been reached
    int mode = 2, flags = 0;        // 0: keys of blk, 1: values of the block before, 2: values of blk
    auto next_operand = [&]() {
      if (kTiles == 1 && mode == 0 && !(flags & kFirst)) {
        mode = 1;
        return true;
      }
      if (mode != 2 && (kTiles == 2 || (flags & kLast))) {
        mode = 2;
        return true;
      }
      mode = 0;
      ++blk;
      if (!await(bar.meta_full + 8 * (blk % kMeta), blk / kMeta & 1u)) return false;
      flags = metas[blk % kMeta].flags;
      return !(flags & kEnd);
    };
    Ring<kStages> ring;
    Ring<kRawStages> raw;
    ring.skip(group);
    raw.skip(group);
    bool on = start->left > 0;
    for (int ahead = kParts > 1 ? 1 : group + 1; on; ahead = kTurn) {
      for (int i = 0; i < ahead && on; ++i) on = next_operand();
      if (!on || !await(bar.raw_full + 8 * raw.i, raw.pass) || !await(bar.empty + 8 * ring.i, ring.pass ^ 1u)) break;
      const bool value = mode != 0, wide = value && D == 256;
      const uint32_t place = (mode == 1 ? blk - 1 : blk) % kMeta;
      const BlockMeta& meta = metas[place];
      const uint32_t* scale = value ? meta.vf : meta.kf;
      const int row0 = wide ? row_wide : row_narrow, base = wide ? part * 64 : 0, stride = wide ? 8 : 16;
      // rows behind the last visible key become zeroes (their scores are masked, their weights 0, and what lies
      // in them may be NaN), and so do NaN among values that some row does not see
      const int last = min(meta.have - 1 - base, 127), seen = (meta.flags >> kSeen) - base;
      const uint8_t* from = sm + C::kOffRaw + raw.i * kRaw + (wide ? blk_wide * 4096 : blk_narrow * 8192) + piece * 16;
      uint8_t* to = sm + C::kOffStage + ring.i * kStage + (wide ? to_wide : to_narrow);
      const int other = wide ? other_wide : other_narrow;
      auto widen = [&](int u, const uint4& x, uint32_t f) {
        const uint2 a = e4m3x4_to_half4(x.x), b = e4m3x4_to_half4(x.y), c = e4m3x4_to_half4(x.z), e = e4m3x4_to_half4(x.w);
        uint8_t* at = to + u * stride * 128;
        *reinterpret_cast<uint4*>(at) = make_uint4(mul_half2(a.x, f), mul_half2(a.y, f), mul_half2(b.x, f), mul_half2(b.y, f));
        *reinterpret_cast<uint4*>(at + other) = make_uint4(mul_half2(c.x, f), mul_half2(c.y, f), mul_half2(e.x, f), mul_half2(e.y, f));
      };
      if (value ? seen >= (wide ? 64 : 128) : last >= 127) {  // (keys have base 0)
        // A short loop: the kernel's roles share the instruction caches (8192 prompt tokens 633 us, 660 with two units a
        // pass, 740 with four; D = 256, eight prompts' chunks: 243, 242, 253)
#pragma unroll 1
        for (int u = 0; u < kUnits; ++u)
          widen(u, *reinterpret_cast<const uint4*>(from + (row0 + u * stride) * 64), scale[base + row0 + u * stride]);
      } else {
#pragma unroll 1
        for (int u = 0; u < kUnits; ++u) {
          const int row = row0 + u * stride;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (row <= last) x = *reinterpret_cast<const uint4*>(from + row * 64);
          if (value && row >= seen && zero_odd_e4m3(x)) *odd_seen = 1;
          widen(u, x, scale[base + row]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar.full + 8 * ring.i);
        mbar_arrive(bar.raw_empty + 8 * raw.i);
        mbar_arrive(bar.meta_empty + 8 * place);
      }
      ring.skip(kGroups);
      raw.skip(kGroups);
    }
    finish();
    return;
  }
  if (warp == C::kMma0 || warp == C::kMma1) {
    // ------------------------------------------------------------------ the products
    if (lane == 0) {
      // e4m3: both operands are binary16 (the format fields of the descriptor are zero)
      constexpr uint32_t kF16 = kE4M3 ? ~((1u << 7) | (1u << 10)) : ~0u;
      constexpr uint32_t kIdQK = idesc_bf16_f32(128, C::kKeys) & kF16, kIdPV = idesc_bf16_f32_bmn(128, D) & kF16;
      constexpr uint32_t kVBlock = D == 256 ? 8192 : 16384;  // bytes between 64-value blocks of a value stage
      const int which = warp - C::kMma0;
      Ring<kStages> ring;
      uint32_t q_par = 0, n_blk = 0;
      // a stage's share of the scores, and of O: of a block, or of its `half`
      auto qk = [&](int sub, uint32_t slot, int part, int half, const Ring<kStages>& at) {
        const uint32_t q = sb + sub * 128 * D * 2, k = sb + C::kOffStage + at.i * kStage + half * 8192;
#pragma unroll
        for (int d = 0; d < 2; ++d)
          mma_bf16_k4<2, 2>(tmem + slot * C::kKeys, sw128_desc(q + (2 * part + d) * 16384), sw128_desc(k + d * 16384), kIdQK,
                            part + d > 0);
      };
      auto pv = [&](int sub, uint32_t slot, int part, int half, const Ring<kStages>& at, bool acc) {
        const uint32_t v = sb + C::kOffStage + at.i * kStage + half * 8192;
        constexpr int kSteps = C::kKeys / kParts / 64;  // 64 keys each
#pragma unroll
        for (int d = 0; d < kSteps; ++d)
          mma_bf16_k4_ta<128>(tmem + C::kColO + sub * D, tmem + slot * C::kKeys + (part * kSteps + d) * 32,
                              sw128_mn_desc(v + d * 8192, kVBlock), kIdPV, acc || d > 0);
      };
      while (ok && walk.next(p, step, seg)) {
        if (seg.keys <= 0) continue;
        if constexpr (kTiles == 2) {
          // this tile's K0 V0 K1 V1 ..; both tiles let go of every stage
          const int t = which;
          const bool mine = t == 0 || seg.ntok > p.sub;
          if (mine) {
            if (!await_one((kE4M3 ? bar.q_ready : bar.q_full) + 8 * t, q_par)) break;
            q_par ^= 1u;
          }
          const int last = seg.j1 - 1;
          for (int j = seg.j0 - 1; j <= last && ok; ++j) {
            // The values of block j and the keys of the one after it, by halves: a half's weights go into O,
            // and the scores two halves on take their slot.
            Ring<kStages> values = ring;
            if (j >= seg.j0) ring.step();
            const Ring<kStages> keys = ring;
            if (j < last) ring.step();
            for (int half = 0; half < 2; ++half) {
              const uint32_t slot = 2 * t + half;
              if (j >= seg.j0) {
                if (mine && !await_one(bar.p_full + 8 * slot, n_blk & 1u)) break;
                if (half == 0 && !await_one(bar.full + 8 * values.i, values.pass)) break;
                if (mine) {
                  tc_fence_after();
                  pv(t, slot, 0, half, values, j > seg.j0 || half > 0);
                  mma_commit(bar.o_full + 8 * slot);
                  if (half) mma_commit(bar.empty + 8 * values.i);
                } else if (half) {
                  mbar_arrive(bar.empty + 8 * values.i);
                }
              }
              if (j < last) {
                if (half == 0 && !await_one(bar.full + 8 * keys.i, keys.pass)) break;
                if (mine) {
                  tc_fence_after();
                  qk(t, slot, 0, half, keys);
                  mma_commit(bar.s_full + 8 * slot);
                  if (half) mma_commit(bar.empty + 8 * keys.i);
                  if (half && j + 1 == last) mma_commit(bar.q_empty + 8 * t);
                } else if (half) {
                  mbar_arrive(bar.empty + 8 * keys.i);
                }
              }
            }
            n_blk += j >= seg.j0;
          }
          if (!mine) n_blk -= seg.j1 - seg.j0;
        } else {
          // K0 K1 V0 K2 V1 ..: one warp the keys, one the values
          const int n = seg.j1 - seg.j0;
          if (which == 0) {
            if (!await_one(kE4M3 ? bar.q_ready : bar.q_full, q_par)) break;
            q_par ^= 1u;
            for (int i = 0; i < n && ok; ++i, ++n_blk) {
              const uint32_t slot = n_blk & 1u;
              // the slot's weights have been used: the product of the block two before has ended
              if (n_blk >= 2 && !await_one(bar.o_full + 8 * slot, ((n_blk - 2) >> 1) & 1u)) break;
              for (int part = 0; part < kParts; ++part) {
                if (!await_one(bar.full + 8 * ring.i, ring.pass)) break;
                tc_fence_after();
                qk(0, slot, part, 0, ring);
                mma_commit(bar.empty + 8 * ring.i);
                ring.step();
              }
              if (!ok) break;
              mma_commit(bar.s_full + 8 * slot);
              if (i + 1 == n) mma_commit(bar.q_empty);
              ring.skip(i == 0 ? (n == 1 ? kParts : 0) : i + 1 < n ? kParts : 2 * kParts);  // the values in between
            }
          } else {
            ring.skip(n == 1 ? kParts : 2 * kParts);
            for (int i = 0; i < n && ok; ++i, ++n_blk) {
              const uint32_t slot = n_blk & 1u;
              if (!await_one(bar.p_full + 8 * slot, (n_blk >> 1) & 1u)) break;
              for (int part = 0; part < kParts; ++part) {
                if (!await_one(bar.full + 8 * ring.i, ring.pass)) break;
                tc_fence_after();
                pv(0, slot, part, 0, ring, i > 0 || part > 0);
                mma_commit(bar.empty + 8 * ring.i);
                ring.step();
              }
              if (!ok) break;
              mma_commit(bar.o_full + 8 * slot);
              if (i + 2 < n) ring.skip(kParts);
            }
          }
        }
      }
      // every product has ended, and every arrival it owes, before the CTA does
      mma_commit(bar.done);
      mbar_wait(bar.done, 0, kWaitLimit);
    }
  } else if (kE4M3 && warp == C::kTail) {
    // ------------------------------------------------------------------ e4m3: scales of the blocks
    const int shift = p.cache.page_shift;
    BlockMeta* metas = reinterpret_cast<BlockMeta*>(sm + C::kOffMeta);
    uint32_t blk = 0;
    auto page_of = [&](int j) {  // of the lane-th page of block j
      const int key = j * kBlock + (lane << shift);
      return (lane << shift) < kBlock && key < seg.keys
                 ? (int)ld_ahead4(p.cache.table + (long)seg.n * p.cache.max_pages + (key >> shift))
                 : 0;
    };
    while (ok && walk.next(p, step, seg)) {
      if (seg.keys <= 0) continue;
      int next = page_of(seg.j0);
      for (int j = seg.j0; j < seg.j1; ++j, ++blk) {
        int id = next;
        if ((unsigned)id >= (unsigned)p.cache.num_pages) {
          raise_error(p.err, kErrDeviceArgument);
          id = 0;
        }
        if (j + 1 < seg.j1) next = page_of(j + 1);
        const int row = (id * p.Hkv + seg.hk) << shift, have = min(seg.keys - j * kBlock, kBlock);
        // the exponent bytes of four keys
        const int at = __shfl_sync(0xFFFFFFFFu, row, (lane * 4) >> shift) + ((lane * 4) & ((1 << shift) - 1));
        uint32_t k4 = 0, v4 = 0;
        if (lane * 4 < have) {
          k4 = ld_ahead4(p.cache.k_scale + at);
          v4 = ld_ahead4(p.cache.v_scale + at);
        }
        if (!await(bar.meta_empty + 8 * (blk % kMeta), (blk / kMeta & 1u) ^ 1u)) break;
        uint32_t kt = 0, vt = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          kt = max(kt, lane * 4 + i < have ? (k4 >> (8 * i)) & 255u : 0u);
          vt = max(vt, lane * 4 + i < have ? (v4 >> (8 * i)) & 255u : 0u);
        }
        kt = __reduce_max_sync(0xFFFFFFFFu, kt);
        vt = __reduce_max_sync(0xFFFFFFFFu, vt);
        uint32_t kf[4], vf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = lane * 4 + i < have;
          kf[i] = in ? half2_power((int)((k4 >> (8 * i)) & 255u) - (int)kt + kWiden) : 0u;
          vf[i] = in ? half2_power((int)((v4 >> (8 * i)) & 255u) - (int)vt + kWiden) : 0u;
        }
        BlockMeta& m = metas[blk % kMeta];
        reinterpret_cast<uint4*>(m.kf)[lane] = make_uint4(kf[0], kf[1], kf[2], kf[3]);
        reinterpret_cast<uint4*>(m.vf)[lane] = make_uint4(vf[0], vf[1], vf[2], vf[3]);
        if (lane == 0) {
          m.ku = e8m0_value(kt) * p.scale_log2;
          m.ev = (float)((int)vt - 127);
          m.have = have;
          m.flags = (j == seg.j0 ? kFirst : 0) | (j + 1 == seg.j1 ? kLast : 0) | min(max(seg.pos0 + 1 - j * kBlock, 0), kBlock) << kSeen;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.meta_full + 8 * (blk % kMeta));
      }
    }
    if (ok && await(bar.meta_empty + 8 * (blk % kMeta), (blk / kMeta & 1u) ^ 1u) && lane == 0) {
      metas[blk % kMeta].flags = kEnd;
      mbar_arrive(bar.meta_full + 8 * (blk % kMeta));
    }
  } else if (warp == C::kLoad) {
    // ------------------------------------------------------------------ Q, K and V by TMA
    // bf16: into the products' stages; e4m3: the codes into their own
    constexpr int kRing = kE4M3 ? C::kRawStages : kStages;
    constexpr uint32_t kBytes = kE4M3 ? kRaw : kStage, kPitch = kE4M3 ? 64 : 128;  // of a stage; of a row of a 64-value column
    const uint32_t stage0 = sb + (kE4M3 ? C::kOffRaw : C::kOffStage);
    const uint32_t bar_full = kE4M3 ? bar.raw_full : bar.full, bar_empty = kE4M3 ? bar.raw_empty : bar.empty;
    const int page = 1 << p.cache.page_shift, box = min(page, 64), box_shift = min(p.cache.page_shift, 6);
    Ring<kRing> ring;
    uint32_t tails = 0, tail_par = 0, used = 0;  // stages whose last copy went to the tail barrier, its parity; stages in use
    uint32_t q_pass = 0, q_used = 0;             // bit t: parity of the next Q of tile t; Q was loaded at all
    while (ok && walk.next(p, step, seg)) {
      if (seg.keys > 0) {
        const int hk = seg.hk, keys = seg.keys;
        const int32_t* table = p.cache.table + (long)seg.n * p.cache.max_pages;
        // One stage: `rows` keys from key0 on (those below `keys`, by whole boxes), nd columns of 64 values
        // from column d0 on.
        auto load = [&](const CUtensorMap* map, int key0, int rows, int d0, int nd, bool value) {
          const int boxes = rows >> box_shift, have = min(max((keys - key0 + box - 1) >> box_shift, 0), boxes);
          const int key = key0 + (lane << box_shift);
          int id = lane < have ? (int)ld_ahead4(table + (key >> p.cache.page_shift)) : 0;  // its latency passes in the wait
          if (!await(bar_empty + 8 * ring.i, ring.pass ^ 1u)) return;
          const bool tail = !kE4M3 && value && key0 + rows > seg.pos0 + 1;  // the warp that goes over it passes it on
          const uint32_t to = (tail ? bar.tail : bar_full) + 8 * ring.i, bit = 1u << ring.i;
          used |= bit;
          tails = tail ? tails | bit : tails & ~bit;
          if (tail) tail_par ^= bit;
          int y = 0;
          if (lane < have) {
            if ((unsigned)id >= (unsigned)p.cache.num_pages) {
              raise_error(p.err, kErrDeviceArgument);
              id = 0;
            }
            y = ((id * p.Hkv + hk) << p.cache.page_shift) + (key & (page - 1));
          }
          if (lane == 0) mbar_arrive_expect_tx(to, (uint32_t)(have * box * nd) * kPitch);
          __syncwarp();
          if (lane < have) {
            const uint32_t dst = stage0 + ring.i * kBytes + (uint32_t)(lane << box_shift) * kPitch;
            for (int d = 0; d < nd; ++d) tma_load_2d(dst + d * rows * kPitch, map, (d0 + d) * 64, y, to);
          }
          ring.step();
        };
        auto keys_of = [&](int j) {
          for (int part = 0; part < kParts && ok; ++part) load(&p.tmap_k, j * kBlock, 128, 2 * part, 2, false);
        };
        auto values_of = [&](int j) {
          for (int part = 0; part < kParts && ok; ++part)
            load(&p.tmap_v, j * kBlock + part * 64, 128 / kParts, 0, D / 64, true);
        };
        keys_of(seg.j0);
        // the tile's queries (of a packed batch: the rows behind a sequence's last are the next one's, and
        // stay in rows that nobody reads)
        for (int t = 0; t < kTiles && ok && (t == 0 || seg.ntok > p.sub); ++t) {
          if (!await(bar.q_empty + 8 * t, (q_pass >> t & 1u) ^ 1u)) break;
          q_pass ^= 1u << t;
          q_used |= 1u << t;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar.q_full + 8 * t, p.sub * p.G * D * 2);
            for (int d = 0; d < D / 64; ++d)
              tma_load_3d(sb + t * 128 * D * 2 + d * 16384, &p.tmap_q, d * 64, hk * p.G, seg.row0 + t * p.sub, bar.q_full + 8 * t);
          }
        }
        __syncwarp();
        for (int j = seg.j0; j < seg.j1 && ok; ++j) {
          if (kTiles == 1) {
            if (j + 1 < seg.j1) keys_of(j + 1);
            if (ok) values_of(j);
          } else {
            values_of(j);
            if (ok && j + 1 < seg.j1) keys_of(j + 1);
          }
        }
      }
    }
    // After a wait that ran out, the copies in flight land before the CTA ends: the last copy into stage
    // i went out on this pass over the ring for the stages before ring.i, on the last one for the rest.
    if (!ok) {
      for (int i = 0; i < kRing; ++i) {
        if (!(used >> i & 1u)) continue;
        if (tails >> i & 1u) mbar_wait(bar.tail + 8 * i, (tail_par >> i & 1u) ^ 1u, kWaitLimit);
        else mbar_wait(bar_full + 8 * i, i < ring.i ? ring.pass : ring.pass ^ 1u, kWaitLimit);
      }
      for (int t = 0; t < kTiles; ++t)
        if (q_used >> t & 1u) mbar_wait(bar.q_full + 8 * t, (q_pass >> t & 1u) ^ 1u, kWaitLimit);
    }
  } else if (warp == C::kTail) {
    // ------------------------------------------------------------------ value rows that some row does not see
    Ring<kStages> ring;
    uint32_t used[kStages] = {};  // parity of each stage's tail barrier
    while (ok && walk.next(p, step, seg)) {
      if (seg.keys <= 0) continue;
      constexpr int kRows = 128 / kParts;
      const int n = seg.j1 - seg.j0, seen = seg.pos0 + 1;  // keys that every row sees
      int at = 0;                                         // stages of the segment passed
      auto pass = [&](int to) {
        ring.skip(to - at);
        at = to;
      };
      for (int i = max((max(seen, 0) >> 7) - seg.j0, 0); i < n && ok; ++i) {
        pass((kTiles == 1 && i + 1 < n ? 2 * i + 2 : 2 * i + 1) * kParts);
        for (int part = 0; part < kParts; ++part, pass(at + 1)) {
          const int key0 = (seg.j0 + i) * kBlock + part * kRows;
          if (key0 + kRows <= seen) continue;
          const int have = min(max(seg.keys - key0, 0), kRows), from = min(max(seen - key0, 0), have);
          uint32_t par = 0;
#pragma unroll
          for (int k = 0; k < kStages; ++k)
            if (k == ring.i) {
              par = used[k];
              used[k] ^= 1u;
            }
          if (!await(bar.tail + 8 * ring.i, par)) break;
          uint8_t* st = sm + C::kOffStage + ring.i * kStage;
          constexpr int kCol = D == 256 ? 512 : 1024;  // 16-byte pieces of a 64-value column
          uint4* col = reinterpret_cast<uint4*>(st);
          for (int d = 0; d < D / 64; ++d)
            for (int k = have * 8 + lane; k < kRows * 8; k += 32) col[d * kCol + k] = make_uint4(0, 0, 0, 0);
          for (int k0 = from * 8 + lane; k0 < have * 8; k0 += 32) {
            uint4 x[D / 64];
            uint32_t top = 0;
#pragma unroll
            for (int d = 0; d < D / 64; ++d) x[d] = col[d * kCol + k0];
#pragma unroll
            for (int d = 0; d < D / 64; ++d) top = __vmaxu2(top, top_bf16(x[d]));
            if (__vcmpgeu2(top, kInfBf16) == 0) continue;
#pragma unroll
            for (int d = 0; d < D / 64; ++d) col[d * kCol + k0] = zero_odd_bf16(x[d]);
            *odd_seen = 1;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar.full + 8 * ring.i);
        }
      }
      pass(2 * n * kParts);
    }
  }
  finish();
}

// Joins the parts of cut tiles: out = sum_c O_c 2^(m_c - m) / sum_c l_c 2^(m_c - m), c over the tile's
// parts, always in the same order.  The CTAs of the tile's first part do it; blockIdx.y takes a share of
// rows and columns, and where a tile has many parts the warps of a CTA share those.  The parts are listed
// first and several are loaded at a time, so that their loads do not wait for one another.
//   kTiles 1, 2: parts [tile][D / 4][128 rows], a lane has 16 columns of a row, a sector of the output;
//   kTiles 0: parts [row][D], a lane has 4 columns
template <int D, int kTiles>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnParams p, int ctas) {
  constexpr int kVec = kTiles ? 4 : 1, kAhead = kTiles ? 2 : 8;  // 16-byte pieces of a lane; parts in flight
  __shared__ int s_slot[kMaxCtas + 1];
  __shared__ int s_n;
  __shared__ float4 s_o[8][kVec][32];
  __shared__ float2 s_ml[8][32];
  await_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 d = p.desc[2 * blockIdx.x + 1];
  const int c1 = blockIdx.x + 1 + lane, w1 = warp == 0 && c1 < ctas ? p.desc[2 * c1].w : 0;
  if (!(d.w & kPart)) return;
  if (warp == 0) {
    int n = 1;
    if (lane == 0) s_slot[0] = 2 * blockIdx.x + 1;
    for (int c = blockIdx.x + 1; c < ctas; c += 32) {  // CTAs without work lie between the parts of a short line
      const int w = c == blockIdx.x + 1 ? w1 : c + lane < ctas ? p.desc[2 * (c + lane)].w : 0;
      const unsigned last = __ballot_sync(0xFFFFFFFFu, w & kPartLast);
      unsigned have = __ballot_sync(0xFFFFFFFFu, w & kPart);
      if (last) have &= (last & -last) * 2u - 1u;  // up to the first that ends a tile
      if (have >> lane & 1u) s_slot[n + __popc(have & ((1u << lane) - 1u))] = 2 * (c + lane);
      n += __popc(have);
      if (last) break;
    }
    if (lane == 0) s_n = n;
  }
  __syncthreads();
  const int parts = s_n;
  // (one token at 4000 keys, 76 parts a tile: 15.1 us with, 16.4 without)
  const int ways = parts >= 16 ? 8 : parts >= 8 ? 4 : 1, way = warp % ways, each = 8 / ways;  // warps of an item; items at a time
  const int subs = kTiles == 2 && d.y > p.sub ? 2 : 1;
  const int items = kTiles ? subs * 4 * (D / 16) : (p.G * (D / 4) + 31) / 32;
  for (int i0 = blockIdx.y * each; i0 < items; i0 += gridDim.y * each) {
    const int i = i0 + warp / ways;
    int col, row, sub = 0, rows = p.G;  // col: in pieces
    if constexpr (kTiles > 0) {
      const int rw = i / (D / 16);
      col = i % (D / 16) * 4;
      sub = rw >> 2;
      row = (rw & 3) * 32 + lane;
      rows = min(p.sub, d.y - sub * p.sub) * p.G;
    } else {
      col = (i * 32 + lane) % (D / 4);
      row = (i * 32 + lane) / (D / 4);
    }
    const bool some = i < items && row < rows;
    const int t = row / p.G, h = d.z * p.G + row - t * p.G;
    const long r = d.x + sub * p.sub + t;
    uint2 zz[kVec];  // the gate, on its way with the parts
#pragma unroll
    for (int v = 0; v < kVec; v += kVec > 1 ? 2 : 1) {
      if (!some || way != 0 || !p.z.p) continue;
      const uint16_t* z = p.z.p + r * p.z.token + h * p.z.head + (col + v) * 4;
      if constexpr (kVec > 1) {
        const uint4 y = *reinterpret_cast<const uint4*>(z);
        zz[v] = make_uint2(y.x, y.y);
        zz[v + 1] = make_uint2(y.z, y.w);
      } else {
        zz[v] = *reinterpret_cast<const uint2*>(z);
      }
    }
    float m = -INFINITY, l = 0.f;
    float4 o[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float2& ml, const float4 (&x)[kVec]) {
      const float m2 = fmaxf(m, ml.x), off = m2 == -INFINITY ? 0.f : m2;
      const float a = ex2_approx(m - off), b = ex2_approx(ml.x - off);
      l = l * a + ml.y * b;
#pragma unroll
      for (int v = 0; v < kVec; ++v)
        o[v] = make_float4(o[v].x * a + x[v].x * b, o[v].y * a + x[v].y * b, o[v].z * a + x[v].z * b, o[v].w * a + x[v].w * b);
      m = m2;
    };
    for (int k0 = way; k0 < parts; k0 += kAhead * ways) {
      float2 ml[kAhead];
      float4 x[kAhead][kVec];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const bool in = some && k0 + u * ways < parts;
        const long slot = s_slot[in ? k0 + u * ways : 0];
        const float4* part = p.part + slot * (long)(kPartBytes / sizeof(float4));
        ml[u] = in ? ld_l2(p.ml + slot * 256 + sub * 128 + row) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int v = 0; v < kVec; ++v)
          x[u][v] = !in ? make_float4(0.f, 0.f, 0.f, 0.f)
                        : ld_l2(kTiles > 0 ? part + (sub * (D / 4) + col + v) * 128 + row : part + row * (D / 4) + col);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) add(ml[u], x[u]);
    }
    if (ways > 1) {
      s_ml[warp][lane] = make_float2(m, l);
#pragma unroll
      for (int v = 0; v < kVec; ++v) s_o[warp][v][lane] = o[v];
      __syncthreads();
      if (way == 0) {
        for (int w = 1; w < ways; ++w) {
          float4 x[kVec];
#pragma unroll
          for (int v = 0; v < kVec; ++v) x[v] = s_o[warp + w][v][lane];
          add(s_ml[warp + w][lane], x);
        }
      }
      __syncthreads();
    }
    if (some && way == 0) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint32_t out[2 * kVec];
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        float y[4] = {o[v].x * inv, o[v].y * inv, o[v].z * inv, o[v].w * inv};
        if (l == 0.f) y[0] = y[1] = y[2] = y[3] = 0.f;
        if (p.z.p) {
          y[0] *= sigmoid_fast(__uint_as_float(zz[v].x << 16));
          y[1] *= sigmoid_fast(__uint_as_float(zz[v].x & 0xFFFF0000u));
          y[2] *= sigmoid_fast(__uint_as_float(zz[v].y << 16));
          y[3] *= sigmoid_fast(__uint_as_float(zz[v].y & 0xFFFF0000u));
        }
        out[2 * v] = pack_bf2(y[0], y[1]);
        out[2 * v + 1] = pack_bf2(y[2], y[3]);
      }
      uint16_t* to = p.out + (r * p.Hq + h) * D + col * 4;
      if constexpr (kVec > 1) {
        if (p.wide_out) {
          st_global32(to, out);
        } else {
          reinterpret_cast<uint4*>(to)[0] = make_uint4(out[0], out[1], out[2], out[3]);
          reinterpret_cast<uint4*>(to)[1] = make_uint4(out[4], out[5], out[6], out[7]);
        }
      } else {
        *reinterpret_cast<uint2*>(to) = make_uint2(out[0], out[1]);
      }
    }
  }
}

// Rows of K or V as the TMA sees them: 64 values wide.
cudaError_t encode_pages(CUtensorMap* map, const void* base, const PagedCache& c, int Hkv, int D) {
  if (c.e4m3)
    return encode_u8_2d(map, base, D, ((uint64_t)c.num_pages * Hkv) << c.page_shift, D, 64,
                        c.page_shift > 6 ? 64 : 1u << c.page_shift);
  return encode_bf16_2d_sw128(map, base, D, ((uint64_t)c.num_pages * Hkv) << c.page_shift, (uint64_t)D * 2, 64,
                              c.page_shift > 6 ? 64 : 1u << c.page_shift);
}

template <int D, int kTiles>
cudaError_t launch_join(const LaunchEnv& env, const AttnParams& p, int ctas) {
  const int items = kTiles ? 4 * kTiles * (D / 16) : (p.G * (D / 4) + 31) / 32;
  return launch_early(attn_join_kernel<D, kTiles>, dim3(ctas, items < 16 ? items : 16), 256, 0, env.stream, p, ctas);
}

template <int D, int kTiles, bool kE4M3>
cudaError_t launch_tiles(const LaunchEnv& env, const AttnParams& p, int ctas) {
  using C = Cfg<D, kTiles, kE4M3>;
  static int done[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(attn_kernel<D, kTiles, kE4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = 1;
  }
  e = launch_early(attn_kernel<D, kTiles, kE4M3>, dim3(ctas), C::kThreads, C::kSmem, env.stream, p);
  if (e != cudaSuccess) return e;
  return launch_join<D, kTiles>(env, p, ctas);
}

}  // namespace

// Descriptors, maxima and sums, and 128 KB of O for each of two parts a CTA.
size_t attn_workspace_bytes(int D) {
  (void)D;
  return 2 * kMaxCtas * (sizeof(int4) + 256 * sizeof(float2) + kPartBytes);
}

cudaError_t launch_attn(const LaunchEnv& env, int Hq, int Hkv, int D, const uint16_t* q, const PagedCache& cache,
                        const int32_t* kv_lens, const int32_t* cu, int N, int T, float scale, const HeadRows& z,
                        uint16_t* out, void* workspace) {
  AttnParams p;
  memset(&p, 0, sizeof p);
  p.q = q;
  p.cache = cache;
  p.kv_lens = kv_lens;
  p.cu = cu;
  p.z = z;
  p.out = out;
  p.err = env.err;
  p.scale_log2 = scale * kLog2e;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.N = N;
  p.T = T;
  p.sub = 128 / p.G;
  // What beginning and ending a tile costs beside one block, with 1 to 5: D = 256, eight prompts' chunks, bf16 173,
  // 148, 139, 130, 131 us, e4m3 299, 256, 249, 243, 239 (sixteen prompts of 50 to 900 tokens 139 with 3, 138, 145); D
  // = 128, a prompt of 8192, 457, 435, 440, 447, 455 us (497 with none), e4m3 687, 634, 625, 632, 641.
  p.lead = D == 128 ? 2 : 4;
  // Fewer CTAs on a short line: a part costs its reader as much as a block.  17 tokens after 1000, 16 key heads of
  // 128: 17.1 us with no such limit, 15.5 with 2, 16.0 with 3, 16.7 with 4; 16 tokens after 4000, 2 of 256: 31.7 us,
  // 26.6, 26.1, 27.6.
  p.least = p.lead;
  p.wide_out = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.desc = reinterpret_cast<int4*>(ws);
  p.ml = reinterpret_cast<float2*>(ws + 2 * kMaxCtas * sizeof(int4));
  p.part = reinterpret_cast<float4*>(ws + 2 * kMaxCtas * (sizeof(int4) + 256 * sizeof(float2)));
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  // One token of each sequence and few query heads to a key head: too few rows to fill a 128-row tile, and HBM
  // bounds the call.  By groups of 8 heads, this kernel against the tiles' (64 sequences of 30 to 30000 keys at
  // D = 256, 256 of 500 to 8000 at D = 128): D = 256 bf16 97 : 105 us, one sequence of 4000 keys 15 : 20; e4m3
  // 60 : 154; D = 128 bf16 426 : 463, e4m3 264 : 871; with 16 heads D = 128 bf16 223 : 256, e4m3 168 : 468, but
  // D = 256 bf16 169 : 107, e4m3 170 : 157 (a form of this kernel for them, which is not kept).
  if (!cu && p.G <= (D == 128 ? 16 : 8)) {
    p.sub = 1;
    // A tile's beginning and end, in blocks of HBM's time for an SM ("short": 400 sequences of 30 to 3000 keys).  bf16
    // with 1, 2, 3: D = 256 97, 98, 97 us, short 98, 99, 104; D = 128 421, 423, 428, short 179, 191, 205.  e4m3 at
    // D = 256 with 3, 4, 5: 64, 60, 60, short 86, 82, 78 (2048 tiles of 30 blocks: 507, 518, 528); at D = 128 with
    // 2, 3, 4: 256, 262, 267, short 146, 137, 146, with 16 heads to a key head 180, 169, 171.
    p.lead = !cache.e4m3 ? 1 : D == 128 ? 3 : 4;
    p.least = 2;  // one sequence of 16000 keys 17.1 us with 1, 15.4 with 2, 16.8 with 3; of 4000 14.3, 14.7, 17.5
    e = launch_attn_decode(env, p, D, ctas);
    if (e != cudaSuccess) return e;
    return D == 128 ? launch_join<128, 0>(env, p, ctas) : launch_join<256, 0>(env, p, ctas);
  }
  e = encode_pages(&p.tmap_k, cache.k, cache, Hkv, D);
  if (e == cudaSuccess) e = encode_pages(&p.tmap_v, cache.v, cache, Hkv, D);
  if (e == cudaSuccess) e = encode_bf16_3d_sw128(&p.tmap_q, q, D, Hq, T, 64, p.G, p.sub);
  if (e != cudaSuccess) return e;
  // Two tiles a CTA where a sequence has more rows than one holds, on average.  64 sequences of 2000 keys, 2 key
  // heads, 96 rows for each: one tile 43 us, two 46 (e4m3 53 : 59); 160 rows: 63 : 52 (99 : 65); a prompt of 8192
  // tokens, 8 key heads, 699 : 437 (1202 : 634).
  const bool two = (long)T * p.G > 128L * N;
  if (cache.e4m3) {
    if (D == 256) return launch_tiles<256, 1, true>(env, p, ctas);
    return two ? launch_tiles<128, 2, true>(env, p, ctas) : launch_tiles<128, 1, true>(env, p, ctas);
  }
  if (D == 256) return launch_tiles<256, 1, false>(env, p, ctas);
  return two ? launch_tiles<128, 2, false>(env, p, ctas) : launch_tiles<128, 1, false>(env, p, ctas);
}

}  // namespace gdn
