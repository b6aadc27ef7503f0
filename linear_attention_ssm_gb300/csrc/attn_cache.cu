// attn_cache.cu -- the paged key/value cache: queries and keys normalised and rotated, keys and values
// written to their pages (bf16, or e4m3 with one power of two for a row) in one pass; rows read back.
//
// Both kernels move each byte once and do a few operations on it, so HBM bounds them: one warp (half
// a warp at D = 128) holds one head row of a token, 16 bytes a lane, four rows in flight.
#include "attn_common.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens of one CTA
constexpr int kUnroll = 4;     // rows whose loads a lane has in flight

struct Place {
  int seq;   // < 0: no sequence
  int pos;   // position in the sequence
  long row;  // page * rows per page slab: index of the head-0 row of the position; -1: no place in the cache
};

struct PrepareParams {
  HeadRows q, k, v;
  const uint16_t* qw;
  const uint16_t* kw;
  PagedCache cache;
  Rope rope;
  const int32_t* kv_lens;
  const int32_t* cu;
  unsigned* err;
  uint16_t* q_out;
  float eps;
  int Hq, Hkv, N, T, tokens;  // tokens: of one CTA
};

// p * f turns, reduced to [-1/2, 1/2]: p is split into two factors that fp32 holds, each product with
// the high part of f is kept exactly (product and its rounding error), whole turns are dropped from
// each, and only the sums of the remainders round.
__device__ __forceinline__ float turns_of(int p, float hi, float lo) {
  const float p1 = (float)((p >> 12) * 4096), p0 = (float)(p & 4095);
  float a = p1 * hi, b = p0 * hi;
  float ae = fmaf(p1, hi, -a), be = fmaf(p0, hi, -b);
  a -= rintf(a);
  b -= rintf(b);
  ae -= rintf(ae);
  const float t = (a + b) + (fmaf(p1 + p0, lo, be) + ae);
  return t - rintf(t);
}

// Row of the cache of position pos: its page's head-0 row, or -1.
__device__ __forceinline__ long cache_row(const PagedCache& c, int Hkv, int seq, int pos, bool& bad) {
  const int page = __ldg(c.table + (long)seq * c.max_pages + (pos >> c.page_shift));
  if ((unsigned)page >= (unsigned)c.num_pages) {
    bad = true;
    return -1;
  }
  return (((long)page * Hkv) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// Eight values of a row of which D / 8 neighbouring lanes hold one each: stores their codes and, by the
// row's first lane, the exponent byte (where `store` is set: the shuffles want the whole warp).
template <int D>
__device__ __forceinline__ void store_e4m3(const float (&x)[8], uint8_t* codes, uint8_t* byte, int lane,
                                           bool store) {
  uint32_t top = 0;  // the row's largest finite magnitude, as bits
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    top = max(top, b < 0x7F800000u ? b : 0u);
  }
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  // 448 = 1.75 * 2^8: the exponent of the magnitude less 8, one more when its significand is above 1.75
  const int e = max((int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), -117);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 y = make_float2(x[4 * i + 2 * j] * inv, x[4 * i + 2 * j + 1] * inv);
      // the conversion saturates: what is not finite becomes NaN here
      if (!isfinite(y.x)) y.x = __uint_as_float(0x7FFFFFFFu);
      if (!isfinite(y.y)) y.y = __uint_as_float(0x7FFFFFFFu);
      r |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (16 * j);
    }
    w[i] = r;
  }
  if (!store) return;
  *reinterpret_cast<uint2*>(codes + lane * 8) = make_uint2(w[0], w[1]);
  if (lane == 0) *byte = (uint8_t)(e + 127);
}

template <int D, bool kE4M3>
__global__ void __launch_bounds__(kThreads) prepare_kernel(const __grid_constant__ PrepareParams p) {
  constexpr int kLanes = D / 8;              // lanes of a row
  constexpr int kSlots = kThreads / kLanes;  // rows at a time
  __shared__ Place s_place[kMaxTokens];
  __shared__ __align__(16) float2 s_cs[kMaxTokens][D / 2];
  const int tid = threadIdx.x, lane = tid % kLanes, slot = tid / kLanes;
  const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);

  if (tid < nt) {
    Place pl;
    int first, len;
    bool bad = false;
    pl.seq = attn_seq_of(p.cu, p.N, p.T, t0 + tid, first, len);
    pl.pos = 0;
    pl.row = -1;
    if (pl.seq >= 0) {
      const int kv = __ldg(p.kv_lens + pl.seq);
      if (kv < 0 || kv > (int)min((long)p.cache.max_pages << p.cache.page_shift, 0x7FFFFFFFL)) {
        bad = true;
        pl.seq = -2;
      } else {
        pl.pos = kv - len + (t0 + tid - first);
        if (pl.pos >= 0) pl.row = cache_row(p.cache, p.Hkv, pl.seq, pl.pos, bad);
      }
    } else if (pl.seq == -2) {
      bad = true;
    }
    if (bad) raise_error(p.err, kErrDeviceArgument);
    s_place[tid] = pl;
  }
  __syncthreads();
  if (const int np = p.rope.rot / 2) {
    const int groups = kThreads / np, j = tid % np;
    if (tid < groups * np) {
      const double f = __ldg(p.rope.freqs + j) * 0.15915494309189533577;  // turns of one position
      const float hi = (float)f, lo = (float)(f - (double)hi);
      for (int t = tid / np; t < nt; t += groups) {
        float s, c;
        sincospif(2.f * turns_of(s_place[t].pos, hi, lo), &s, &c);
        s_cs[t][j] = make_float2(c * p.rope.magnitude, s * p.rope.magnitude);
      }
    }
  }
  // this lane's eight weights of the query and the key norm
  uint4 qw = make_uint4(0, 0, 0, 0), kw = qw;
  if (p.qw) qw = __ldg(reinterpret_cast<const uint4*>(p.qw) + lane);
  if (p.kw) kw = __ldg(reinterpret_cast<const uint4*>(p.kw) + lane);
  __syncthreads();

  const int hq = p.q.p ? p.Hq : 0, per = hq + 2 * p.Hkv, rows = nt * per;
  for (int base = slot; base < rows + slot; base += kSlots * kUnroll) {  // the same trips for every thread
    uint4 raw[kUnroll];
    int tok[kUnroll], head[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int idx = base + u * kSlots;
      tok[u] = idx / per;
      head[u] = idx - tok[u] * per;
      if (idx >= rows || s_place[tok[u]].seq < 0) tok[u] = -1;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (tok[u] >= 0) {
        const int h = head[u];
        const HeadRows& src = h < hq ? p.q : h < hq + p.Hkv ? p.k : p.v;
        const int hh = h < hq ? h : h < hq + p.Hkv ? h - hq : h - hq - p.Hkv;
        raw[u] = __ldcs(reinterpret_cast<const uint4*>(src.p + (t0 + tok[u]) * src.token + hh * src.head) + lane);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (__all_sync(0xFFFFFFFFu, tok[u] < 0)) continue;
      const bool is_q = head[u] < hq, is_k = !is_q && head[u] < hq + p.Hkv;
      float x[8];
      const uint32_t r[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
      }
      if (__any_sync(0xFFFFFFFFu, is_q || is_k)) {
        const int t = max(tok[u], 0);
        float y[8];
        const uint16_t* w_on = is_q ? p.qw : p.kw;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float rms = w_on ? rsqrtf(ss * (1.f / D) + p.eps) : 1.f;
        const uint4 w4 = is_q ? qw : kw;
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = x[2 * i] * rms;
          y[2 * i + 1] = x[2 * i + 1] * rms;
          if (w_on) {
            y[2 * i] *= __uint_as_float(w[i] << 16);
            y[2 * i + 1] *= __uint_as_float(w[i] & 0xFFFF0000u);
          }
        }
        if (p.rope.rot) {
          const int d0 = lane * 8;
          if (p.rope.interleaved) {
            if (d0 < p.rope.rot) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 cs = s_cs[t][d0 / 2 + i];
                const float a = y[2 * i], b = y[2 * i + 1];
                y[2 * i] = fmaf(a, cs.x, -b * cs.y);
                y[2 * i + 1] = fmaf(b, cs.x, a * cs.y);
              }
            }
          } else {  // the other half of a pair sits rot / 16 lanes away
            const int half = p.rope.rot / 2, off = half / 8;
            const bool low = d0 < half, in = d0 < p.rope.rot;
            const int src = in ? (low ? lane + off : lane - off) : lane;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xFFFFFFFFu, y[i], src, kLanes);
            if (in) {
              const float2* cs = &s_cs[t][low ? d0 : d0 - half];
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = fmaf(y[i], cs[i].x, (low ? -o[i] : o[i]) * cs[i].y);
            }
          }
        }
        if (is_q || is_k) {  // the one rounding to bf16
          raw[u] = make_uint4(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]), pack_bf2(y[4], y[5]), pack_bf2(y[6], y[7]));
        }
      }
      const Place pl = s_place[max(tok[u], 0)];
      if (tok[u] >= 0 && is_q)
        *(reinterpret_cast<uint4*>(p.q_out + ((long)(t0 + tok[u]) * p.Hq + head[u]) * D) + lane) = raw[u];
      const bool to_cache = tok[u] >= 0 && !is_q && pl.row >= 0;
      const int h = is_k ? head[u] - hq : head[u] - hq - p.Hkv;
      const long row = pl.row + ((long)h << p.cache.page_shift);
      if constexpr (kE4M3) {
        if (__any_sync(0xFFFFFFFFu, to_cache)) {
          const uint32_t b[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(b[i] << 16);
            x[2 * i + 1] = __uint_as_float(b[i] & 0xFFFF0000u);
          }
          uint8_t* codes = static_cast<uint8_t*>(is_k ? p.cache.k : p.cache.v) + row * D;
          uint8_t* byte = (is_k ? p.cache.k_scale : p.cache.v_scale) + row;
          store_e4m3<D>(x, codes, byte, lane, to_cache);
        }
      } else {
        if (to_cache)
          *(reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_k ? p.cache.k : p.cache.v) + row * D) + lane) = raw[u];
      }
    }
  }
}

struct ReadParams {
  PagedCache cache;
  const int32_t* starts;
  const int32_t* cu;
  unsigned* err;
  uint16_t* k_out;
  uint16_t* v_out;
  int Hkv, N, T, tokens;
};

// 16 bytes of the cache a lane: 8 bf16 values copied, or 16 codes widened.
template <int D, bool kE4M3>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kVals = kE4M3 ? 16 : 8, kLanes = D / kVals, kSlots = kThreads / kLanes;
  __shared__ long s_row[kMaxTokens];
  const int tid = threadIdx.x, lane = tid % kLanes, slot = tid / kLanes;
  const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);
  if (tid < nt) {
    int first, len;
    bool bad = false;
    long row = -1;
    const int seq = attn_seq_of(p.cu, p.N, p.T, t0 + tid, first, len);
    if (seq >= 0) {
      const long pos = (p.starts ? (long)__ldg(p.starts + seq) : 0L) + (t0 + tid - first);
      if (pos < 0 || pos >= min((long)p.cache.max_pages << p.cache.page_shift, 0x7FFFFFFFL)) bad = true;
      else row = cache_row(p.cache, p.Hkv, seq, (int)pos, bad);
    } else if (seq == -2) {
      bad = true;
    }
    if (bad) raise_error(p.err, kErrDeviceArgument);
    s_row[tid] = row;
  }
  __syncthreads();
  const int per = 2 * p.Hkv, rows = nt * per;
  for (int base = slot; base < rows; base += kSlots * kUnroll) {
    uint4 raw[kUnroll];
    uint32_t byte[kUnroll];
    uint16_t* dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int idx = base + u * kSlots;
      dst[u] = nullptr;
      if (idx >= rows) continue;
      const int tok = idx / per, hh = idx - tok * per, h = hh < p.Hkv ? hh : hh - p.Hkv;
      if (s_row[tok] < 0) continue;
      const bool is_k = hh < p.Hkv;
      const long row = s_row[tok] + ((long)h << p.cache.page_shift);
      const void* src = is_k ? p.cache.k : p.cache.v;
      raw[u] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(src) + row * (D * (kE4M3 ? 1 : 2))) + lane);
      if constexpr (kE4M3) byte[u] = __ldg((is_k ? p.cache.k_scale : p.cache.v_scale) + row);
      dst[u] = (is_k ? p.k_out : p.v_out) + ((long)(t0 + tok) * p.Hkv + h) * D + lane * kVals;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!dst[u]) continue;
      if constexpr (kE4M3) {
        const float s = e8m0_value(byte[u]);
        const uint32_t r[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = e4m3x2_to_float2((uint16_t)(r[i] & 0xFFFFu)), b = e4m3x2_to_float2((uint16_t)(r[i] >> 16));
          o[2 * i] = pack_bf2(a.x * s, a.y * s);
          o[2 * i + 1] = pack_bf2(b.x * s, b.y * s);
        }
        reinterpret_cast<uint4*>(dst[u])[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4*>(dst[u])[1] = make_uint4(o[4], o[5], o[6], o[7]);
      } else {
        *reinterpret_cast<uint4*>(dst[u]) = raw[u];
      }
    }
  }
}

// Tokens of a CTA: one while that fills the GPU eight CTAs deep, then more, so that the rotation's
// angles and the weights are formed for several tokens at a time.
int tokens_per_cta(int T, int sms) {
  const int t = (T + sms * 8 - 1) / (sms * 8);
  return t < 1 ? 1 : t > kMaxTokens ? kMaxTokens : t;
}

}  // namespace

cudaError_t launch_attn_prepare(const LaunchEnv& env, int Hq, int Hkv, int D, const HeadRows& q, const HeadRows& k,
                                const HeadRows& v, const uint16_t* qw, const uint16_t* kw, float eps,
                                const Rope& rope, const PagedCache& cache, const int32_t* kv_lens,
                                const int32_t* cu, int N, int T, uint16_t* q_out) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int tokens = tokens_per_cta(T, sms);
  const PrepareParams p = {q, k, v, qw, kw, cache, rope, kv_lens, cu, env.err, q_out, eps, Hq, Hkv, N, T, tokens};
  const int grid = (T + tokens - 1) / tokens;
  auto kern = D == 128 ? (cache.e4m3 ? prepare_kernel<128, true> : prepare_kernel<128, false>)
                       : (cache.e4m3 ? prepare_kernel<256, true> : prepare_kernel<256, false>);
  kern<<<grid, kThreads, 0, env.stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_attn_cache_read(const LaunchEnv& env, int Hkv, int D, const PagedCache& cache,
                                   const int32_t* starts, const int32_t* cu, int N, int T, uint16_t* k_out,
                                   uint16_t* v_out) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int tokens = tokens_per_cta(T, sms);
  const ReadParams p = {cache, starts, cu, env.err, k_out, v_out, Hkv, N, T, tokens};
  const int grid = (T + tokens - 1) / tokens;
  auto kern = D == 128 ? (cache.e4m3 ? cache_read_kernel<128, true> : cache_read_kernel<128, false>)
                       : (cache.e4m3 ? cache_read_kernel<256, true> : cache_read_kernel<256, false>);
  kern<<<grid, kThreads, 0, env.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
