// attn_decode.cu -- softmax attention of one new token of each sequence over its paged cache.
//
// A key head's at most 16 query rows do not fill a tcgen05 tile, and every cached byte is used once: HBM
// bounds the kernel, so it is built to keep copies in flight and to finish a key quickly.  One warp loads
// keys and one values by TMA into a ring of 32 KB stages (192 KB in flight on every SM); the others take a
// stage's keys 16 at a time through both products with mma.sync (m16n8k16), transposed so that keys and
// values fill the 16 rows and the query rows the 8 columns:
//   S^T [16 keys x q] = K Q^T,   p = 2^(S - m),   O^T [D x q] += V^T P^T
// Each warp has its own running m, l and O in registers, so that the warps meet only where a segment
// ends; there they are joined.  (Work is cut into one piece for each SM as in the tile kernel.)
//
// An e4m3 cache is widened between shared memory and the registers, two codes an instruction, to
// binary16, which holds every code exactly.  The queries become binary16 too, each row divided by the
// power of two of its largest value: what that loses is below 2^-25 of that value.  Scores get the keys'
// powers of two, weights the values' (relative to the group's largest; O is held in units of 2^r, raised
// with it).  Weights are at most 2^8: times 2^7 they still fit binary16, and only weights below 2^-21 of
// a row's largest leave its normal range.
//
// Measured on a GB300 (of 6792 GB/s copied): 64 sequences of 30 to 30000 keys, 2 key heads of 256, bf16 97 us, 6.2
// TB/s, 91 %, e4m3 60 us; 256 sequences of 500 to 8000 e4m3 keys, 8 of 128, 263 us, 5.5 TB/s, 81 %; one sequence of
// 4000 keys 15 us -- the latency of two launches, HBM's share is 1.2.
#include <cstring>

#include "attn_common.cuh"
#include "chunk_common.cuh"

namespace gdn {
namespace {

constexpr float kWeight = 7.f;   // log2 of the factor on binary16 weights

template <int D, bool kE4M3, int kQ8>  // kQ8: columns of 8 query rows
struct DCfg {
  static constexpr int kRow = D * (kE4M3 ? 1 : 2);    // bytes of a key
  static constexpr int kBoxes = kRow / 128;           // 128-byte columns of a stage, [keys][128 bytes] swizzled
  static constexpr int kKeys = 32768 / (2 * kRow);    // keys of a stage: 32 (bf16, D = 256) to 128 (e4m3, D = 128)
  static constexpr int kHalf = kKeys * kRow;          // a stage's keys, then its values
  // Warps that compute, a group of keys each; where a stage has fewer groups than warps, the stages go to
  // sets of warps in turn.  A group is one mma tile of 16 keys, or two of e4m3 (64 sequences at D = 256 62 us both
  // ways, 256 at D = 128 262 and 263, with 16 heads to a key head 181 and 193; bf16 there 233 with two, 224).
  static constexpr int kWarps = 8;
  static constexpr int kTwo = kE4M3 ? 2 : 1, kGroup = 16 * kTwo;
  static constexpr int kGroups = kKeys / kGroup, kSets = kWarps / kGroups;
  static constexpr int kThreads = 32 * (kWarps + 2);  // and one that loads the keys, one the values
  static constexpr int kTiles = D / 16;               // of O^T
  static constexpr int kMergeRow = 33;                // 16-byte pieces from one mma tile of O^T to the next, where it is merged
  static constexpr int kMergeO = kWarps / 2 * kQ8 * kTiles * kMergeRow * 16, kMergeMl = kWarps / 2 * 32 * kQ8 * 16;
  static constexpr int kQBytes = 2 * kQ8 * 8 * D * 2;  // two segments' queries
  static constexpr int kScale = kE4M3 ? 2 * kKeys : 0;
  static constexpr int kFixed = kMergeO + kMergeMl + kQBytes + 1024 + 1024;
  static constexpr int kFit = (232448 - kFixed) / (2 * kHalf + 64 + kScale);
  static constexpr int kSlots = kFit < 6 ? kFit : 6;
  static_assert(kSlots >= 3, "stages to hide HBM's latency");
  static constexpr int kOffMerge = kSlots * 2 * kHalf;
  static constexpr int kOffMl = kOffMerge + kMergeO;
  static constexpr int kOffQ = kOffMl + kMergeMl;
  static constexpr int kOffScale = kOffQ + kQBytes;
  static constexpr int kOffMeta = kOffScale + kSlots * kScale;
  static constexpr int kOffBar = kOffMeta + kSlots * 32;
  static constexpr int kOffScan = kOffBar + 256;
  static constexpr int kSmem = kOffScan + 512 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

// What a stage holds.
struct Stage {
  int n;          // keys, 0: none (a segment whose token sees no key)
  int flags;
  int row0, hk;   // packed row, key head
  int part;       // slot of the segment's part in the workspace
  int pad[3];
};
enum : int { kFirst = 1, kLastOfSegment = 2, kEnd = 4, kWhole = 8, kEndsTile = 16 };

template <bool kF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// this thread's arrival on the barrier once its cp.async copies so far have landed (the barrier's count
// includes it)
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int D, bool kE4M3, int kQ8>
__global__ void __launch_bounds__(DCfg<D, kE4M3, kQ8>::kThreads, 1) attn_decode_kernel(const __grid_constant__ AttnParams p) {
  using C = DCfg<D, kE4M3, kQ8>;
  constexpr int kWarps = C::kWarps, kSlots = C::kSlots, kTiles = C::kTiles, kTwo = C::kTwo, kGroup = C::kGroup;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  Stage* stages = reinterpret_cast<Stage*>(sm + C::kOffMeta);
  const uint32_t ring_s = smem_u32(sm);
  const uint32_t full = smem_u32(sm + C::kOffBar), empty = full + 8 * kSlots, q_empty = empty + 8 * kSlots,
                 meet = q_empty + 16;
  long* scan = reinterpret_cast<long*>(sm + C::kOffScan);
  WalkStart* start = reinterpret_cast<WalkStart*>(scan + 20);
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(full + 8 * i, kE4M3 ? 2 + 64 : 2);  // both loading warps; their lanes' copies of the scales
      mbar_init(empty + 8 * i, kWarps);
    }
    for (int i = 0; i < 2; ++i) mbar_init(q_empty + 8 * i, kWarps);
    mbar_init(meet, kWarps);
    fence_mbar_init();
    prefetch_tensormap(&p.tmap_k);
    prefetch_tensormap(&p.tmap_v);
    start->left = 0;
  }
  await_grid();
  if (tid < 2) p.desc[2 * blockIdx.x + tid] = make_int4(0, 0, 0, 0);
  find_start<C::kThreads>(p, 1, scan, start);
  __syncthreads();
  if (start->left == 0) return;

  if (warp >= kWarps) {
    // ------------------------------------------------------------------ loading: keys, or values
    const bool keys = warp == kWarps;
    Walk walk;
    walk.begin(p, 1, *start);
    const int shift = p.cache.page_shift, rows_shift = min(shift, C::kKeys == 32 ? 5 : 6), rows = 1 << rows_shift;
    const CUtensorMap* map = keys ? &p.tmap_k : &p.tmap_v;
    const uint8_t* scale = keys ? p.cache.k_scale : p.cache.v_scale;
    const int row = lane << rows_shift;  // of the stage: this lane's first
    Segment seg = {};
    bool ok = true;
    int slot = 0, pass = 0, used = 0, segs = 0;
    auto await = [&](uint32_t b, uint32_t parity) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(b, parity, kWaitLimit))) {
        raise_error(p.err, kErrTimeout);
        ok = false;
      }
      return ok;
    };
    // page of this lane's rows of the stage that begins at key0
    auto page_id = [&](int key0, int lim) {
      return row < C::kKeys && key0 + row < lim
                 ? p.cache.table[(long)seg.n * p.cache.max_pages + ((key0 + row) >> shift)]
                 : -1;
    };
    while (ok && walk.next(p, 1, seg)) {
      const int first = seg.j0 * kBlock, lim = min(seg.keys, seg.j1 * kBlock);
      const int mark = (seg.j0 == 0 && seg.j1 == seg.nb ? kWhole : 0) | (seg.j1 == seg.nb ? kEndsTile : 0);
      int id = page_id(first, lim);
      for (int key0 = first; key0 == first || key0 < lim; key0 += C::kKeys) {
        const int n = min(max(lim - key0, 0), C::kKeys);
        const bool mine = row < n;
        if (mine && (unsigned)id >= (unsigned)p.cache.num_pages) {
          raise_error(p.err, kErrDeviceArgument);
          id = 0;
        }
        const int y = mine ? ((id * p.Hkv + seg.hk) << shift) + ((key0 + row) & ((1 << shift) - 1)) : 0;
        if (key0 + C::kKeys < lim) id = page_id(key0 + C::kKeys, lim);  // its latency passes in the wait
        if (!await(empty + 8 * slot, pass ^ 1)) break;
        if (keys && key0 == first && !await(q_empty + 8 * (segs & 1), (segs >> 1 & 1) ^ 1)) break;
        const uint32_t bar = full + 8 * slot;
        if (lane == 0) {
          uint32_t bytes = ((n + rows - 1) >> rows_shift) * rows * C::kRow;
          if (keys) {
            *reinterpret_cast<int4*>(&stages[slot]) =
                make_int4(n, mark | (key0 == first ? kFirst : 0) | (key0 + C::kKeys >= lim ? kLastOfSegment : 0), seg.row0, seg.hk);
            stages[slot].part = 2 * blockIdx.x + (seg.j0 == 0 ? 1 : 0);
            if (key0 == first) bytes += p.G * D * 2;
          }
          mbar_arrive_expect_tx(bar, bytes);
          if (keys && key0 == first)
            bulk_load(ring_s + C::kOffQ + (segs & 1) * (C::kQBytes / 2), p.q + ((long)seg.row0 * p.Hq + seg.hk * p.G) * D,
                      p.G * D * 2, bar);
        }
        __syncwarp();
        if (mine) {
          const uint32_t dst = ring_s + slot * 2 * C::kHalf + (keys ? 0 : C::kHalf) + (uint32_t)row * 128;
#pragma unroll
          for (int b = 0; b < C::kBoxes; ++b) tma_load_2d(dst + b * C::kKeys * 128, map, b * (kE4M3 ? 128 : 64), y, bar);
        }
        if constexpr (kE4M3) {  // the rows' exponent bytes, 16 a lane
          const int r16 = lane * 16, y16 = __shfl_sync(0xFFFFFFFFu, y, r16 >> rows_shift & 31) + (r16 & (rows - 1));
          if (r16 < n) cp_async16(ring_s + C::kOffScale + slot * C::kScale + (keys ? 0 : C::kKeys) + r16, scale + y16);
          cp_async_arrive(bar);
        }
        used |= 1 << slot;
        if (++slot == kSlots) {
          slot = 0;
          pass ^= 1;
        }
      }
      ++segs;
    }
    if (ok && await(empty + 8 * slot, pass ^ 1)) {
      if (lane == 0) {
        if (keys) stages[slot].flags = kEnd;
        mbar_arrive(full + 8 * slot);
      }
      if constexpr (kE4M3) cp_async_arrive(full + 8 * slot);
    } else {  // copies in flight land before the CTA ends
      for (int i = 0; i < kSlots; ++i)
        if (used >> i & 1) mbar_wait(full + 8 * i, i < slot ? pass : pass ^ 1, kWaitLimit);
    }
    if constexpr (kE4M3) asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }

  // ------------------------------------------------------------------ computing
  // The computing warps' barrier: bounded like every wait here, so that a warp that gave up holds nobody.
  uint32_t sync_par = 0;
  bool ok = true;
  const auto warps_sync = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(meet);
    if (ok && !__all_sync(0xFFFFFFFFu, mbar_wait(meet, sync_par, kWaitLimit))) {
      raise_error(p.err, kErrTimeout);
      ok = false;
    }
    sync_par ^= 1u;
  };
  uint32_t q[kQ8][D / 8];        // Q^T fragments of the segment's key head
  float qs[kQ8][2];              // log2 units of a score, for this lane's two query rows
  float o[kQ8][kTiles][4];       // O^T: rows d, columns the two query rows
  float m[kQ8][2], l[kQ8][2], r[kQ8][2];
  int turn = 0, segs = 0;        // whose stage this is; segments begun
  for (int slot = 0, pass = 0; ok; pass ^= (slot == kSlots - 1), slot = slot == kSlots - 1 ? 0 : slot + 1) {
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(full + 8 * slot, pass, kWaitLimit))) {
      raise_error(p.err, kErrTimeout);
      break;
    }
    const int4 ga = *reinterpret_cast<const int4*>(&stages[slot]);
    const int all = ga.x, flags = ga.y, row0 = ga.z, hk = ga.w, part = stages[slot].part;
    if (flags & kEnd) break;
    if (flags & kFirst) {
#pragma unroll
      for (int a = 0; a < kQ8; ++a) {
        const int row = a * 8 + g;
        const uint8_t* src = sm + C::kOffQ + (segs & 1) * (C::kQBytes / 2) + row * D * 2;
        if constexpr (!kE4M3) {
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {  // 64-value column x / 2, its 16-byte piece 2 c + x % 2
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < p.G) v = *reinterpret_cast<const uint4*>(src + (x >> 1) * 128 + (2 * c + (x & 1)) * 16);
            q[a][4 * x] = v.x;
            q[a][4 * x + 1] = v.y;
            q[a][4 * x + 2] = v.z;
            q[a][4 * x + 3] = v.w;
          }
          qs[a][0] = qs[a][1] = p.scale_log2;
        } else {
          uint32_t top = 0;
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {  // 128-value column x / 2, its 16-value piece 2 c + x % 2
            uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (row < p.G) {
              const uint4* s = reinterpret_cast<const uint4*>(src + (x >> 1) * 256 + (2 * c + (x & 1)) * 32);
              v[0] = s[0];
              v[1] = s[1];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              q[a][8 * x + 4 * i] = v[i].x;
              q[a][8 * x + 4 * i + 1] = v[i].y;
              q[a][8 * x + 4 * i + 2] = v[i].z;
              q[a][8 * x + 4 * i + 3] = v[i].w;
            }
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint32_t lo = q[a][i] << 16 & 0x7FFFFFFFu, hi = q[a][i] & 0x7FFF0000u;
            top = max(top, max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u));
          }
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          // the row divided by 2^e, e the exponent of its largest value (kept where both powers are normal)
          const int e = min(max((int)(top >> 23) - 127, -120), 126);
          const float inv = __uint_as_float((uint32_t)(127 - e) << 23), two = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            q[a][i] = pack_half2(__uint_as_float(q[a][i] << 16) * inv, __uint_as_float(q[a][i] & 0xFFFF0000u) * inv);
          qs[a][0] = __shfl_sync(0xFFFFFFFFu, two, 8 * c) * p.scale_log2;  // rows 2 c, 2 c + 1 sit in lanes 4 (2 c), ..
          qs[a][1] = __shfl_sync(0xFFFFFFFFu, two, 8 * c + 4) * p.scale_log2;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          m[a][i] = r[a][i] = -INFINITY;
          l[a][i] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[a][t][i] = 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty + 8 * (segs & 1));
      ++segs;
    }
    // this warp's group of the stage, if it has one
    const int group = warp % C::kGroups, n = warp / C::kGroups == turn ? min(max(all - group * kGroup, 0), kGroup) : 0;
    if (++turn == C::kSets) turn = 0;
    if (n > 0) {
      const uint32_t ks = ring_s + slot * 2 * C::kHalf + group * kGroup * 128, vs = ks + C::kHalf;
      if (n < kGroup) {  // value rows behind the last key may hold anything, and 0 * NaN is not 0
        for (int i = lane; i < (kGroup - n) * 8 * C::kBoxes; i += 32) {
          const int b = i / ((kGroup - n) * 8), x = i % ((kGroup - n) * 8);
          *reinterpret_cast<uint4*>(sm + (vs - ring_s) + b * C::kKeys * 128 + n * 128 + x * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      // S^T
      float s[kQ8][kTwo][2][4];
#pragma unroll
      for (int a = 0; a < kQ8; ++a)
#pragma unroll
        for (int y = 0; y < kTwo; ++y)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[a][y][0][i] = s[a][y][1][i] = 0.f;
#pragma unroll
      for (int x = 0; x < 2 * C::kBoxes; ++x) {  // column x / 2, 16-byte piece 2 c + x % 2 of rows g and g + 8
#pragma unroll
        for (int y = 0; y < kTwo; ++y) {
          const uint32_t at = ks + (x >> 1) * C::kKeys * 128 + (16 * y + g) * 128 + (((2 * c + (x & 1)) ^ g) << 4);
          const uint4 u = lds128(at), w = lds128(at + 1024);
          if constexpr (!kE4M3) {
#pragma unroll
            for (int a = 0; a < kQ8; ++a) {
              mma16816<false>(s[a][y][0], u.x, w.x, u.y, w.y, q[a][4 * x], q[a][4 * x + 1]);
              mma16816<false>(s[a][y][1], u.z, w.z, u.w, w.w, q[a][4 * x + 2], q[a][4 * x + 3]);
            }
          } else {
            const uint32_t ur[4] = {u.x, u.y, u.z, u.w}, wr[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint2 lo = e4m3x4_to_half4(ur[t]), hi = e4m3x4_to_half4(wr[t]);
#pragma unroll
              for (int a = 0; a < kQ8; ++a)
                mma16816<true>(s[a][y][t & 1], lo.x, hi.x, lo.y, hi.y, q[a][8 * x + 2 * t], q[a][8 * x + 2 * t + 1]);
            }
          }
        }
      }
      // this lane's keys, 16 y + g and 16 y + g + 8: their scales
      float kf[kTwo][2], vf[kTwo][2], ev = 0.f;
      if constexpr (kE4M3) {
        const uint8_t* sc = sm + C::kOffScale + slot * C::kScale + group * kGroup;
        uint32_t vb[kTwo][2], top = 0;
#pragma unroll
        for (int y = 0; y < kTwo; ++y)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = 16 * y + g + 8 * i;
            kf[y][i] = e8m0_value(sc[key]);
            vb[y][i] = key < n ? sc[C::kKeys + key] : 0u;
            top = max(top, vb[y][i]);
          }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        ev = (float)((int)top - 127);
#pragma unroll
        for (int y = 0; y < kTwo; ++y)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int diff = (int)vb[y][i] - (int)top + (int)kWeight;  // the value's power over the group's, times 2^7
            vf[y][i] = diff >= -126 ? __uint_as_float((uint32_t)(127 + diff) << 23) : 0.f;
          }
      }
      uint32_t pb[kQ8][kTwo][2];
#pragma unroll
      for (int a = 0; a < kQ8; ++a) {
        float x[kTwo][2][2];  // [key g, g + 8][query row]
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int y = 0; y < kTwo; ++y)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float v = (s[a][y][0][2 * i + k] + s[a][y][1][2 * i + k]) * (kE4M3 ? kf[y][i] * qs[a][k] : qs[a][k]);
              x[y][i][k] = 16 * y + g + 8 * i < n ? v : -INFINITY;
              top[k] = fmaxf(top[k], x[y][i][k]);
            }
        // m, and the unit r of O, are raised for the whole warp where one of its keys asks for it
        bool more = top[0] > m[a][0] + kLazy || top[1] > m[a][1] + kLazy;
        if constexpr (kE4M3) more = more || m[a][0] + ev > r[a][0] || m[a][1] + ev > r[a][1];
        if (__any_sync(0xFFFFFFFFu, more)) {
          float f[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], w));
            if (top[k] > m[a][k]) {
              l[a][k] *= ex2_approx(m[a][k] - top[k]);
              m[a][k] = top[k];
            }
            const float e = m[a][k] + ev;
            f[k] = e > r[a][k] ? ex2_approx(r[a][k] - e) : 1.f;
            r[a][k] = fmaxf(r[a][k], e);
          }
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            o[a][t][0] *= f[0];
            o[a][t][1] *= f[1];
            o[a][t][2] *= f[0];
            o[a][t][3] *= f[1];
          }
        }
        // weights 2^(s - m + d), d <= 0 the distance of this group's unit from O's; cut off at -40, lest a
        // group of tiny values vanish from l (P is zero in binary16 long before)
        float off[2], back[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float mk = m[a][k], e = kE4M3 && mk > -INFINITY ? fmaxf(mk + ev - r[a][k], -40.f) : 0.f;
          off[k] = mk > -INFINITY ? e - mk : 0.f;
          back[k] = kE4M3 ? ex2_approx(-e) : 1.f;
        }
#pragma unroll
        for (int y = 0; y < kTwo; ++y) {
          float w[2][2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            w[0][k] = ex2_approx(x[y][0][k] + off[k]);
            w[1][k] = ex2_approx(x[y][1][k] + off[k]);
            l[a][k] = kE4M3 ? fmaf(w[0][k] + w[1][k], back[k], l[a][k]) : l[a][k] + (w[0][k] + w[1][k]);
            if constexpr (kE4M3) {
              w[0][k] *= vf[y][0];
              w[1][k] *= vf[y][1];
            }
          }
          // the weights' one rounding: the matrix instructions take both operands in one type, bf16 or binary16 (l keeps fp32)
          pb[a][y][0] = transpose8x8(kE4M3 ? pack_half2(w[0][0], w[0][1]) : pack_bf2(w[0][0], w[0][1]));
          pb[a][y][1] = transpose8x8(kE4M3 ? pack_half2(w[1][0], w[1][1]) : pack_bf2(w[1][0], w[1][1]));
        }
      }
      // O^T += V^T P^T
      if constexpr (!kE4M3) {
        const int key = (lane & 7) + ((lane >> 4) << 3), half = lane >> 3 & 1;  // matrices: keys 0-7 / 8-15, values 0-7 / 8-15
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          const int piece = 2 * t + half;
#pragma unroll
          for (int y = 0; y < kTwo; ++y) {
            uint32_t v[4];
            ldmatrix_x4_trans(vs + (piece >> 3) * C::kKeys * 128 + (16 * y + key) * 128 + (((piece & 7) ^ (key & 7)) << 4), v);
#pragma unroll
            for (int a = 0; a < kQ8; ++a) mma16816<false>(o[a][t], v[0], v[1], v[2], v[3], pb[a][y][0], pb[a][y][1]);
          }
        }
      } else {
        // 16 values (piece g of a column) of keys 2c, 2c + 1, 2c + 8, 2c + 9; tile t of the column takes
        // values 2t (row g) and 2t + 1 (row g + 8)
#pragma unroll
        for (int b = 0; b < C::kBoxes; ++b) {
#pragma unroll
          for (int y = 0; y < kTwo; ++y) {
            uint32_t v[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = 2 * c + (i & 1) + 8 * (i >> 1);
              const uint4 x = lds128(vs + b * C::kKeys * 128 + (16 * y + key) * 128 + ((g ^ (key & 7)) << 4));
              v[i][0] = x.x;
              v[i][1] = x.y;
              v[i][2] = x.z;
              v[i][3] = x.w;
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
              const uint32_t sel = t & 1 ? 0x7362u : 0x5140u;  // two values of two keys side by side
              const uint2 lo = e4m3x4_to_half4(__byte_perm(v[0][t >> 1], v[1][t >> 1], sel)),
                          hi = e4m3x4_to_half4(__byte_perm(v[2][t >> 1], v[3][t >> 1], sel));
#pragma unroll
              for (int a = 0; a < kQ8; ++a) mma16816<true>(o[a][b * 8 + t], lo.x, lo.y, hi.x, hi.y, pb[a][y][0], pb[a][y][1]);
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + 8 * slot);
    if (flags & kLastOfSegment) {
      // ---- the warps' shares, joined
      float4* mo = reinterpret_cast<float4*>(sm + C::kOffMerge);
      float4* mml = reinterpret_cast<float4*>(sm + C::kOffMl);
#pragma unroll
      for (int a = 0; a < kQ8; ++a)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l[a][k] += __shfl_xor_sync(0xFFFFFFFFu, l[a][k], w);
          if constexpr (kE4M3) {  // O in units of 2^m (half the exponent at a time)
            const float h = m[a][k] == -INFINITY ? 0.f : ex2_approx(0.5f * (r[a][k] - m[a][k] - kWeight));
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              o[a][t][k] = o[a][t][k] * h * h;
              o[a][t][2 + k] = o[a][t][2 + k] * h * h;
            }
          }
        }
      // Half of the warps hand theirs over, the others add their own.  (Lane 4 r + c's piece lies where neither
      // eight neighbouring lanes nor the eight r of one c share banks.)
      auto place = [](int r, int c) { return (r >> 1) * 8 + ((2 * c + (r & 1)) ^ (2 * (r >> 1))); };
      constexpr int kHalfWarps = kWarps / 2;
      constexpr int kRow = C::kMergeRow;
      float4* slot_o = mo + (warp % kHalfWarps) * kQ8 * kTiles * kRow + place(g, c);
      float4* slot_ml = mml + (warp % kHalfWarps) * kQ8 * 32 + lane;
      if (warp < kHalfWarps) warps_sync();
#pragma unroll
      for (int a = 0; a < kQ8; ++a) {
        if (warp < kHalfWarps) {
          const float4 y = slot_ml[a * 32];
          float f0[2], f1[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float mk = k ? y.y : y.x, lk = k ? y.w : y.z, m2 = fmaxf(m[a][k], mk), off = m2 == -INFINITY ? 0.f : m2;
            f0[k] = ex2_approx(m[a][k] - off);
            f1[k] = ex2_approx(mk - off);
            l[a][k] = l[a][k] * f0[k] + lk * f1[k];
            m[a][k] = m2;
          }
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            const float4 x = slot_o[(a * kTiles + t) * kRow];
            slot_o[(a * kTiles + t) * kRow] = make_float4(o[a][t][0] * f0[0] + x.x * f1[0], o[a][t][1] * f0[1] + x.y * f1[1],
                                                        o[a][t][2] * f0[0] + x.z * f1[0], o[a][t][3] * f0[1] + x.w * f1[1]);
          }
        } else {
#pragma unroll
          for (int t = 0; t < kTiles; ++t) slot_o[(a * kTiles + t) * kRow] = make_float4(o[a][t][0], o[a][t][1], o[a][t][2], o[a][t][3]);
        }
        slot_ml[a * 32] = make_float4(m[a][0], m[a][1], l[a][0], l[a][1]);
      }
      if (warp >= kHalfWarps) warps_sync();
      warps_sync();
      // ---- out: the sum of what is left, eight values a thread
      const bool whole = flags & kWhole;
      for (int i = tid; i < p.G * (D / 8); i += 32 * kWarps) {
        const int row = i / (D / 8), d = i % (D / 8) * 8, a = row >> 3, at = (row & 7) >> 1, k = row & 1;
        float mk[kHalfWarps], lk[kHalfWarps], mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kHalfWarps; ++w) {  // lanes of one c hold the same: lane c
          const float* y = reinterpret_cast<const float*>(mml + (w * kQ8 + a) * 32 + at);
          mk[w] = y[k];
          lk[w] = y[2 + k];
          mx = fmaxf(mx, mk[w]);
        }
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, lx = 0.f;
#pragma unroll
        for (int w = 0; w < kHalfWarps; ++w) {
          const float f = mx == -INFINITY ? 0.f : ex2_approx(mk[w] - mx);
          lx += lk[w] * f;
          const float* x = reinterpret_cast<const float*>(mo + (w * kQ8 + a) * kTiles * kRow) + k;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // where value d + e of this row sits: mma tile, lane row, half
            const int t = kE4M3 ? (d >> 7) * 8 + ((d + e) >> 1 & 7) : d >> 4, lr = kE4M3 ? d >> 4 & 7 : e,
                      hf = kE4M3 ? e & 1 : d >> 3 & 1;
            v[e] += x[(t * kRow + place(lr, at)) * 4 + 2 * hf] * f;
          }
        }
        const float inv = whole ? (lx == 0.f ? 0.f : 1.f / lx) : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = lx == 0.f ? 0.f : v[e] * inv;  // no visible key: zero, whatever O holds
        if (whole) {
          const long h = hk * p.G + row;
          if (p.z.p) {
            const uint4 zz = *reinterpret_cast<const uint4*>(p.z.p + row0 * p.z.token + h * p.z.head + d);
            const uint32_t zr[4] = {zz.x, zz.y, zz.z, zz.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[2 * e] *= sigmoid_fast(__uint_as_float(zr[e] << 16));
              v[2 * e + 1] *= sigmoid_fast(__uint_as_float(zr[e] & 0xFFFF0000u));
            }
          }
          *reinterpret_cast<uint4*>(p.out + ((long)row0 * p.Hq + h) * D + d) =
              make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
        } else {
          float4* to = p.part + (long)part * (kPartBytes / sizeof(float4)) + (row * D + d) / 4;
          to[0] = make_float4(v[0], v[1], v[2], v[3]);
          to[1] = make_float4(v[4], v[5], v[6], v[7]);
          if (d == 0) p.ml[(long)part * 256 + row] = make_float2(mx, lx);
        }
      }
      if (!whole && tid == 0) p.desc[part] = make_int4(row0, 1, hk, kPart | (flags & kEndsTile ? kPartLast : 0));
      warps_sync();
    }
  }
}

template <int D, bool kE4M3, int kQ8>
cudaError_t launch_one(const LaunchEnv& env, const AttnParams& p, int ctas) {
  using C = DCfg<D, kE4M3, kQ8>;
  static int done[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(attn_decode_kernel<D, kE4M3, kQ8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = 1;
  }
  return launch_early(attn_decode_kernel<D, kE4M3, kQ8>, dim3(ctas), C::kThreads, C::kSmem, env.stream, p);
}

template <int D, bool kE4M3>
cudaError_t launch_rows(const LaunchEnv& env, const AttnParams& p, int ctas) {
  if constexpr (D == 128) {
    if (p.G > 8) return launch_one<D, kE4M3, 2>(env, p, ctas);
  }
  return launch_one<D, kE4M3, 1>(env, p, ctas);
}

}  // namespace

cudaError_t launch_attn_decode(const LaunchEnv& env, AttnParams& p, int D, int ctas) {
  const uint64_t rows = ((uint64_t)p.cache.num_pages * p.Hkv) << p.cache.page_shift;
  // rows of one copy: a page's, at most 64 and a stage's keys (32 for bf16 at D = 256)
  const int page = 1 << p.cache.page_shift, most = !p.cache.e4m3 && D == 256 ? 32 : 64, box = page < most ? page : most;
  cudaError_t e;
  if (p.cache.e4m3) {
    e = encode_u8_2d_sw128(&p.tmap_k, p.cache.k, D, rows, D, 128, box);
    if (e == cudaSuccess) e = encode_u8_2d_sw128(&p.tmap_v, p.cache.v, D, rows, D, 128, box);
  } else {
    e = encode_bf16_2d_sw128(&p.tmap_k, p.cache.k, D, rows, (uint64_t)D * 2, 64, box);
    if (e == cudaSuccess) e = encode_bf16_2d_sw128(&p.tmap_v, p.cache.v, D, rows, (uint64_t)D * 2, 64, box);
  }
  if (e != cudaSuccess) return e;
  if (p.cache.e4m3) return D == 128 ? launch_rows<128, true>(env, p, ctas) : launch_rows<256, true>(env, p, ctas);
  return D == 128 ? launch_rows<128, false>(env, p, ctas) : launch_rows<256, false>(env, p, ctas);
}

}  // namespace gdn
