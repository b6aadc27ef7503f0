// attn_common.cuh -- what the kernels of the paged-cache attention share: where a token's row lies,
// e4m3 codes and their powers of two, the line of work and how it is cut, launches.
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
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int a = cu[lo];
  if (lo == N) return a >= 0 && a <= t ? -1 : -2;
  const int b = cu[lo + 1];
  if (a < 0 || t < a || t >= b || b > T) return -2;
  first = a;
  len = b - a;
  return lo;
}

// 2^(b - 127) of an exponent byte
__device__ __forceinline__ float e8m0_value(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

// Loads that stay where they are written: not sunk to their use (ld_ahead4), not ahead of await_grid (all).  None is
// of the non-coherent kind, see launch_early.
__device__ __forceinline__ uint32_t ld_ahead4(const void* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
// 16 bytes that are read once
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// past L1
__device__ __forceinline__ float4 ld_l2(const float4* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float2 ld_l2(const float2* p) {
  float2 v;
  asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}

// 32 bytes of one thread (aligned to them): a whole sector
__device__ __forceinline__ void st_global32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// four e4m3 codes -> two pairs of binary16 values, low codes first
__device__ __forceinline__ uint2 e4m3x4_to_half4(uint32_t v) {
  uint2 r;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\n"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\ncvt.rn.f16x2.e4m3x2 %1, hi;\n}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
constexpr int kBlock = 128;     // keys of a block, the unit of work
constexpr int kMaxKeys = 0x7FFFFF00;  // of a sequence: a block or two further is within 31 bits too

struct AttnParams {
  CUtensorMap tmap_k;  // pages as [pages * Hkv * page][D] bf16, box 64 x min(page, 64), 128-byte swizzle
  CUtensorMap tmap_v;
  CUtensorMap tmap_q;  // [T][Hq][D] bf16, box 64 x G x sub, 128-byte swizzle
  const uint16_t* q;
  PagedCache cache;
  const int32_t* kv_lens;
  const int32_t* cu;
  HeadRows z;
  uint16_t* out;
  unsigned* err;
  float scale_log2;
  int Hq, Hkv, G, N, T;
  int sub;       // tokens of one tile: 128 / G on the tcgen05 cores, 1 in the one-token kernel
  bool wide_out; // out is 32-byte aligned
  int lead;      // blocks that beginning and ending a tile cost, in the line of work
  int least;     // units of the line that a CTA takes, if it takes any
  int4* desc;    // [2 * grid] what each part of a cut tile holds: packed row, tokens, key head, flags
  float2* ml;    // [2 * grid][256] maximum (log2 units) and sum of a row
  float4* part;  // [2 * grid][128 KB] unnormalised O
};

// ---------------------------------------------------------------- the line of work

// sum_{i < n} floor((a i + b) / 128), all arguments >= 0, n < 2^23, a <= 256: lattice points under a line,
// with the roles of the axes exchanged as in Euclid's algorithm.
__device__ __forceinline__ long floor_sum128(long n, int a, long b) {
  long s = n * (n - 1) / 2 * (a >> 7) + n * (b >> 7);
  uint32_t k = (uint32_t)n, m = 128, x = a & 127, c = (uint32_t)b & 127;
  for (;;) {
    const uint32_t y = x * k + c;
    if (y < m) return s;
    const uint32_t rows = y / m;
    c = y - rows * m;
    k = rows;
    const uint32_t t = m;
    m = x;
    x = t;
    const uint32_t q = x / m;  // 1 at least, from here on
    s += (long)k * (k - 1) / 2 * q;
    x -= q * m;
    if (c >= m) {
      const uint32_t r = c / m;
      s += (long)k * r;
      c -= r * m;
    }
  }
}

// One sequence's new tokens and cache.
struct SeqInfo {
  int first, len, kv;
};

__device__ __forceinline__ SeqInfo seq_info(const AttnParams& p, int n, bool report) {
  SeqInfo s = {n, 1, 0};
  bool bad = false;
  if (p.cu) {
    const int a = p.cu[n], b = p.cu[n + 1];
    bad = a < 0 || b < a || b > p.T;
    if (n == 0 && a > 0 && report) raise_error(p.err, kErrDeviceArgument);  // the rows before are nobody's
    s.first = a;
    s.len = bad ? 0 : b - a;
  }
  s.kv = p.kv_lens[n];
  if (s.kv < 0 || s.kv > min((long)p.cache.max_pages << p.cache.page_shift, (long)kMaxKeys)) {
    bad = true;
    s.kv = 0;
  }
  if (bad && report) raise_error(p.err, kErrDeviceArgument);
  return s;
}

// Keys that the last token of tile i sees; blocks of that tile (one at least, so that rows without a
// key are visited too); its length in the line of work, and that of the tiles before it: `lead` units
// that stand for beginning and ending a tile, then one for each block.
struct Tiles {
  int p0, len, step, lead;  // position of the first new token, new tokens, tokens of a tile
  __device__ __forceinline__ int count() const { return (len + step - 1) / step; }
  __device__ __forceinline__ int keys(int i) const { return p0 + (int)min((long)(i + 1) * step, (long)len); }
  __device__ __forceinline__ int blocks(int i) const {
    const int k = keys(i);
    return k <= kBlock ? 1 : (int)(((long)k + kBlock - 1) / kBlock);
  }
  __device__ __forceinline__ int units(int i) const { return blocks(i) + lead; }
  __device__ __forceinline__ long before(int i) const {
    const int last = count() - 1, full = min(i, last);
    if (full <= 0) return i > last && last >= 0 ? units(last) : 0;
    const long ahead = (long)kBlock - p0;  // tiles with at most one block: (t + 1) step <= ahead
    const int t0 = ahead < step ? 0 : (int)min((long)full, ahead / step);
    long s = t0 + (long)full * lead;
    if (full > t0) s += floor_sum128(full - t0, step, (long)(t0 + 1) * step + p0 + kBlock - 1);
    return s + (i > last ? units(last) : 0);
  }
};

// A run of blocks [j0, j1) of one tile.
struct Segment {
  int n, hk;
  int row0, ntok, pos0;  // packed row and position of the tile's first token, tokens
  int keys;              // that the tile's last token sees (<= 0: no row sees any)
  int j0, j1, nb;        // nb: the tile's blocks
};

struct WalkStart {
  long left, rem;
  int n, hk, tile, j;
  SeqInfo s;  // of sequence n
};

// A CTA's piece of the line, segment by segment.  Every warp walks it by itself.
struct Walk {
  long left;  // units not yet taken
  int n, hk, tile, j;
  SeqInfo s;
  Tiles t;

  __device__ __forceinline__ void load(const AttnParams& p, int step) {
    s = seq_info(p, n, false);
    t = {s.kv - s.len, s.len, step, p.lead};
  }
  __device__ __forceinline__ void begin(const AttnParams& p, int step, const WalkStart& w) {
    left = w.left;
    if (left > 0) {
      n = w.n;
      hk = w.hk;
      tile = w.tile;
      j = w.j;
      s = w.s;
      t = {s.kv - s.len, s.len, step, p.lead};
    }
  }
  __device__ __forceinline__ bool next(const AttnParams& p, int step, Segment& g) {
    for (;;) {
      if (left <= 0) return false;
      g.n = n;
      g.hk = hk;
      g.nb = t.blocks(tile);
      g.row0 = s.first + tile * step;
      g.ntok = min(step, s.len - tile * step);
      g.pos0 = t.p0 + tile * step;
      g.keys = t.keys(tile);
      const int end = (int)min((long)g.nb + p.lead, j + left);
      g.j0 = max(j - p.lead, 0);
      g.j1 = end - p.lead;
      left -= end - j;
      j = end;
      if (left > 0) {  // the next tile, key head, sequence
        j = 0;
        if (++tile == t.count()) {
          tile = 0;
          if (++hk == p.Hkv) {
            hk = 0;
            do {
              if (++n >= p.N) {
                left = 0;
                break;
              }
              load(p, step);
            } while (s.len == 0);
          }
        }
      }
      if (g.j1 > g.j0) return true;  // else the piece ends before the tile's first block
    }
  }
};

__device__ __forceinline__ long divide(long a, long b) {  // both >= 0, b > 0
  return (a | b) >> 32 ? a / b : (long)((uint32_t)a / (uint32_t)b);
}

// This CTA's piece of the line: an equal share of its units, p.least at least, found by the whole CTA.  `scan`: one long
// for each warp; start->left is 0 before the call and stays 0 for a CTA without work.  The caller
// synchronises before it reads *start.
template <int kThreads>
__device__ __forceinline__ void find_start(const AttnParams& p, int step, long* scan, WalkStart* start) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // units of one key head of sequence n
  SeqInfo seen = {0, 0, 0};  // the last one
  auto units_of = [&](int n, bool report) {
    const SeqInfo s = seq_info(p, n, report);
    seen = s;
    const Tiles t = {s.kv - s.len, s.len, step, p.lead};
    return s.len > 0 ? t.before(t.count()) : 0L;
  };
  // prefix sums over the threads: this thread's, and everything
  auto sums = [&](long u, long& before, long& all) {
    long inc = u;
    for (int o = 1; o < 32; o <<= 1) {
      const long x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    before = inc - u;
    all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += scan[w];
      all += scan[w];
    }
  };
  long per = 0, mine = 0, before, total;
  for (int n = tid; n < p.N; n += kThreads) {
    per = units_of(n, blockIdx.x == 0);
    mine += per * p.Hkv;
  }
  sums(mine, before, total);
  long share = divide(total, gridDim.x), extra = total - share * gridDim.x;
  if (share < p.least) {  // a short line: the last CTAs have no work
    share = p.least;
    extra = 0;
  }
  const long u0 = min(total, share * blockIdx.x + divide(extra * blockIdx.x, gridDim.x));
  const long u1 = min(total, share * (blockIdx.x + 1) + divide(extra * (blockIdx.x + 1), gridDim.x));
  if (u1 == u0) return;
  long base = 0;  // units of the sequences of the passes before (one pass where every thread had one sequence)
  for (int n0 = 0;; n0 += kThreads) {
    const int n = n0 + tid;
    if (p.N > kThreads) {
      __syncthreads();
      long all;
      per = n < p.N ? units_of(n, false) : 0;
      mine = per * p.Hkv;
      sums(mine, before, all);
      before += base;
      base += all;
    }
    if (mine > 0 && u0 >= before && u0 < before + mine) {
      start->left = u1 - u0;
      start->n = n;
      start->s = seen;
      start->hk = (int)divide(u0 - before, per);
      start->rem = u0 - before - start->hk * per;
    }
    if (p.N <= kThreads || u0 < base) break;
  }
  __syncthreads();
  // the tile: every thread looks at one stretch of them
  const SeqInfo s = start->s;
  const Tiles t = {s.kv - s.len, s.len, step, p.lead};
  const int count = t.count(), stretch = (count + kThreads - 1) / kThreads;
  const long rem = start->rem;
  const int lo = min(tid * stretch, count), hi = min(lo + stretch, count);
  if (lo < hi) {
    long at = lo == 0 ? 0 : t.before(lo);
    for (int i = lo; i < hi && rem >= at; ++i) {
      const int nb = t.units(i);
      if (rem < at + nb) {
        start->tile = i;
        start->j = (int)(rem - at);
      }
      at += nb;
    }
  }
}

// Flags of a part in AttnParams::desc.
enum : int { kPart = 1, kPartLast = 2 };

__device__ __forceinline__ uint8_t* align1024(uint8_t* q) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(q) + 1023) & ~(uintptr_t)1023);
}

__device__ __forceinline__ void mbar_arrive(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(addr) : "memory");
}

constexpr float kLazy = 8.f;  // a row's maximum is raised when a score exceeds it by this power of two
constexpr int kMaxCtas = 160;  // SMs of the largest part of this architecture
constexpr size_t kPartBytes = 131072;

// A launch that need not wait for the end of the kernel before it in the stream: every thread of the kernel calls
// await_grid() before it reads or writes memory, which waits for that kernel's end and its writes.  Those writes
// happen during this kernel's lifetime, so it reads nothing that another kernel may have written (lengths, pages, cu_seqlens,
// scales, gates, norms) through the non-coherent path (ld.global.nc, __ldg), which is for memory that stays as it
// is for a kernel's whole life, and which a compiler may move past the wait; plain loads and volatile asm stay behind it.
// No kernel here signals its dependents before it ends.
template <typename... A>
cudaError_t launch_early(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void await_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

cudaError_t launch_attn_decode(const LaunchEnv& env, AttnParams& p, int D, int ctas);

}  // namespace gdn
