// attn_cache.cu -- the paged key/value cache: queries and keys normalised and rotated, keys and values
// written to their pages (bf16, or e4m3 with one power of two for a row) in one pass; rows read back.
//
// Both kernels move each byte once and do a few operations on it, so HBM bounds them, and instructions
// next: a warp takes one token's heads (a share of them where tokens are few), so that the place in the
// cache, the angles and the products of weights with their cosines and sines are formed once for all
// heads, and a head costs a 16-byte load a lane, one reduction and two packed fused multiply-adds for
// each pair of values.  Four heads' loads are in flight.
#include "attn_common.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;  // loads that a lane has in flight

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
  int Hq, Hkv, N, T, split;  // split: warps of one token
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

// Heads of one kind of a token, D / 8 lanes a head (two heads at a time at D = 128): loads, `work` on the
// head's eight values of this lane (four words of two), `store`.  All lanes run every step.
template <int D, typename Work, typename Store>
__device__ __forceinline__ void each_head(const HeadRows& rows, long t, int heads, int first, int step, Work work, Store store) {
  constexpr int kAt = 256 / D;  // heads of the warp at a time
  const int lane = threadIdx.x & 31, mine = lane / (D / 8);
  const uint16_t* src = rows.p + t * rows.token + (lane % (D / 8)) * 8;
  for (int h0 = first * kAt; h0 < heads; h0 += step * kAt * kUnroll) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * step * kAt + mine;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (h < heads) raw[u] = __ldcs(reinterpret_cast<const uint4*>(src + h * rows.head));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * step * kAt;
      if (h < heads) store(h + mine, work(raw[u]), h + mine < heads);
    }
  }
}

__device__ __forceinline__ float2 bf2_to_float2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

template <int D, bool kE4M3>
__global__ void __launch_bounds__(32 * kWarps) prepare_kernel(const __grid_constant__ PrepareParams p) {
  constexpr int kLanes = D / 8;  // lanes of a head
  __shared__ __align__(16) float2 s_cs[kWarps][D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes;
  const long item = (long)blockIdx.x * kWarps + warp;
  const int t = (int)(item / p.split), share = (int)(item - (long)t * p.split);
  if (t >= p.T) return;
  int first, len;
  const int seq = attn_seq_of(p.cu, p.N, p.T, t, first, len);
  if (seq < 0) {
    if (seq == -2) raise_error(p.err, kErrDeviceArgument);
    return;
  }
  const int kv = __ldg(p.kv_lens + seq);
  if (kv < 0 || kv > min((long)p.cache.max_pages << p.cache.page_shift, 0x7FFFFFFFL)) {
    raise_error(p.err, kErrDeviceArgument);
    return;
  }
  const int pos = kv - len + (t - first);
  long place = -1;  // head-0 row of the position in the pool
  bool bad = false;
  if (pos >= 0) place = cache_row(p.cache, p.Hkv, seq, pos, bad);
  if (bad) raise_error(p.err, kErrDeviceArgument);

  // the token's cosines and sines
  const int rot = p.rope.rot, half = rot / 2;
  for (int j = lane; j < half; j += 32) {
    const double f = __ldg(p.rope.freqs + j) * 0.15915494309189533577;  // turns of one position
    const float hi = (float)f;
    float s, c;
    sincospif(2.f * turns_of(pos, hi, (float)(f - (double)hi)), &s, &c);
    s_cs[warp][j] = make_float2(c * p.rope.magnitude, s * p.rope.magnitude);
  }
  __syncwarp();
  // This lane's eight values of a head become x * a + y * b, y the values they are paired with (for halves
  // another lane's, half / 8 lanes away, else neighbours), times the norm's factor.
  const int d0 = sub * 8, away = half / 8;
  const bool turned = d0 < rot, low = d0 < half;
  const int partner = (lane - sub) + (!turned || p.rope.interleaved ? sub : low ? sub + away : sub - away);
  auto run = [&](const HeadRows& rows, const uint16_t* w, int heads, auto store) {
    float2 a[4], b[4];
    {
      float wx[8], wy[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int dy = p.rope.interleaved ? (d0 + i) ^ 1 : (partner % kLanes) * 8 + i;
        wx[i] = w ? bf2f(__ldg(w + d0 + i)) : 1.f;
        wy[i] = w ? bf2f(__ldg(w + dy)) : 1.f;
      }
      float fa[8], fb[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 cs = turned ? s_cs[warp][p.rope.interleaved ? (d0 + i) >> 1 : (low ? d0 : d0 - half) + i] : make_float2(1.f, 0.f);
        const bool minus = p.rope.interleaved ? !(i & 1) : low;
        fa[i] = wx[i] * cs.x;
        fb[i] = wy[i] * (minus ? -cs.y : cs.y);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = make_float2(fa[2 * i], fa[2 * i + 1]);
        b[i] = make_float2(fb[2 * i], fb[2 * i + 1]);
      }
    }
    each_head<D>(rows, t, heads, share, p.split, [&](const uint4& raw) {
      const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
      float2 x[4], y[4], ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = bf2_to_float2(r[i]);
      if (rot && !p.rope.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = bf2_to_float2(__shfl_sync(0xFFFFFFFFu, r[i], partner));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = make_float2(x[i].y, x[i].x);
      }
      float rms = 1.f;
      if (w) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = __ffma2_rn(x[i], x[i], ss);
        float s = ss.x + ss.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        rms = rsqrtf(s * (1.f / D) + p.eps);
      }
      uint32_t out[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // without a rotation the paired value does not enter at all (it may be an infinity)
        const float2 z = turned ? __ffma2_rn(x[i], a[i], __fmul2_rn(y[i], b[i])) : __fmul2_rn(x[i], a[i]);
        out[i] = pack_bf2(z.x * rms, z.y * rms);  // the one rounding to bf16
      }
      return make_uint4(out[0], out[1], out[2], out[3]);
    }, store);
  };
  auto to_cache = [&](void* pages, uint8_t* bytes) {
    return [=, &p](int h, const uint4& v, bool in) {
      const long row = place + ((long)h << p.cache.page_shift);
      if constexpr (kE4M3) {
        const uint32_t r[4] = {v.x, v.y, v.z, v.w};
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf2_to_float2(r[i]);
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
        }
        store_e4m3<D>(x, static_cast<uint8_t*>(pages) + row * D, bytes + row, sub, in);
      } else if (in) {
        *(reinterpret_cast<uint4*>(static_cast<uint16_t*>(pages) + row * D) + sub) = v;
      }
    };
  };
  if (p.q.p)
    run(p.q, p.qw, p.Hq, [&](int h, const uint4& v, bool in) {
      if (in) *(reinterpret_cast<uint4*>(p.q_out + ((long)t * p.Hq + h) * D) + sub) = v;
    });
  if (place >= 0) {
    run(p.k, p.kw, p.Hkv, to_cache(p.cache.k, p.cache.k_scale));
    each_head<D>(p.v, t, p.Hkv, share, p.split, [](const uint4& raw) { return raw; }, to_cache(p.cache.v, p.cache.v_scale));
  }
}

struct ReadParams {
  PagedCache cache;
  const int32_t* starts;
  const int32_t* cu;
  unsigned* err;
  uint16_t* k_out;
  uint16_t* v_out;
  int Hkv, N, T, split;
};

// 16 bytes of the cache a lane: 8 bf16 values copied, or 16 codes widened.  A warp's lanes hold a head's
// keys and its values side by side (at D = 256 in bf16, one and then the other), or those of two heads.
template <int D, bool kE4M3>
__global__ void __launch_bounds__(32 * kWarps) cache_read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kVals = kE4M3 ? 16 : 8, kLanes = D / kVals, kAt = 32 / kLanes;  // rows at a time: 1, 2 or 4
  const int lane = threadIdx.x & 31, sub = lane % kLanes, mine = lane / kLanes;
  const long item = (long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(item / p.split), share = (int)(item - (long)t * p.split);
  if (t >= p.T) return;
  int first, len;
  bool bad = false;
  long place = -1;
  const int seq = attn_seq_of(p.cu, p.N, p.T, t, first, len);
  if (seq >= 0) {
    const long pos = (p.starts ? (long)__ldg(p.starts + seq) : 0L) + (t - first);
    if (pos < 0 || pos >= min((long)p.cache.max_pages << p.cache.page_shift, 0x7FFFFFFFL)) bad = true;
    else place = cache_row(p.cache, p.Hkv, seq, (int)pos, bad);
  } else if (seq == -2) {
    bad = true;
  }
  if (bad) raise_error(p.err, kErrDeviceArgument);
  if (place < 0) return;
  // row r of the token: head r / 2, its keys (even) or values (odd)
  const bool keys0 = ((share * kAt + mine) & 1) == 0;
  const int rows = 2 * p.Hkv, step = p.split * kAt;
  for (int r0 = share * kAt; r0 < rows; r0 += step * kUnroll) {
    uint4 raw[kUnroll];
    uint32_t byte[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * step + mine;
      const bool is_k = kAt > 1 ? keys0 : (r & 1) == 0;
      const long row = place + ((long)(r >> 1) << p.cache.page_shift);
      if (r < rows) {
        raw[u] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(is_k ? p.cache.k : p.cache.v) +
                                                       row * (D * (kE4M3 ? 1 : 2))) + sub);
        if constexpr (kE4M3) byte[u] = __ldg((is_k ? p.cache.k_scale : p.cache.v_scale) + row);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * step + mine;
      if (r >= rows) continue;
      const bool is_k = kAt > 1 ? keys0 : (r & 1) == 0;
      uint16_t* dst = (is_k ? p.k_out : p.v_out) + ((long)t * p.Hkv + (r >> 1)) * D + sub * kVals;
      if constexpr (kE4M3) {
        const float s = e8m0_value(byte[u]);
        const uint32_t c[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2 h = e4m3x4_to_half4(c[i]);
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
          o[2 * i] = pack_bf2(a.x * s, a.y * s);
          o[2 * i + 1] = pack_bf2(b.x * s, b.y * s);
        }
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
      } else {
        *reinterpret_cast<uint4*>(dst) = raw[u];
      }
    }
  }
}

// Warps of one token: as many as bring sixteen warps to every SM, as long as each has loads to keep in
// flight (`units`: steps of a warp that has the token alone).
int warps_of_token(int T, int sms, int units) {
  const int want = (16 * sms + T - 1) / T, most = units < 8 ? units : 8;
  return want < 1 ? 1 : want > most ? most : want;
}
}  // namespace

cudaError_t launch_attn_prepare(const LaunchEnv& env, int Hq, int Hkv, int D, const HeadRows& q, const HeadRows& k,
                                const HeadRows& v, const uint16_t* qw, const uint16_t* kw, float eps,
                                const Rope& rope, const PagedCache& cache, const int32_t* kv_lens,
                                const int32_t* cu, int N, int T, uint16_t* q_out) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int split = warps_of_token(T, sms, (Hq * D + 255) / 256);
  const PrepareParams p = {q, k, v, qw, kw, cache, rope, kv_lens, cu, env.err, q_out, eps, Hq, Hkv, N, T, split};
  const unsigned grid = (unsigned)(((long)T * split + kWarps - 1) / kWarps);
  auto kern = D == 128 ? (cache.e4m3 ? prepare_kernel<128, true> : prepare_kernel<128, false>)
                       : (cache.e4m3 ? prepare_kernel<256, true> : prepare_kernel<256, false>);
  kern<<<grid, 32 * kWarps, 0, env.stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_attn_cache_read(const LaunchEnv& env, int Hkv, int D, const PagedCache& cache,
                                   const int32_t* starts, const int32_t* cu, int N, int T, uint16_t* k_out,
                                   uint16_t* v_out) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int split = warps_of_token(T, sms, (2 * Hkv * D * (cache.e4m3 ? 1 : 2) + 511) / 512);
  const ReadParams p = {cache, starts, cu, env.err, k_out, v_out, Hkv, N, T, split};
  const unsigned grid = (unsigned)(((long)T * split + kWarps - 1) / kWarps);
  auto kern = D == 128 ? (cache.e4m3 ? cache_read_kernel<128, true> : cache_read_kernel<128, false>)
                       : (cache.e4m3 ? cache_read_kernel<256, true> : cache_read_kernel<256, false>);
  kern<<<grid, 32 * kWarps, 0, env.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
