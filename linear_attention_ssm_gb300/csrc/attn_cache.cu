// attn_cache.cu -- the paged key/value cache: queries and keys normalised and rotated, keys and values
// written to their pages (bf16, or e4m3 with one power of two for a row) in one pass; rows read back.
//
// Both kernels move each byte once and do a few operations on it, so HBM bounds them, and instructions
// next: a warp takes one token's heads (a share of them where tokens are few), so that the place in the
// cache, the angles and the products of weights with their cosines and sines are formed once for all
// heads, and a head costs a 16-byte load a lane, one reduction and two packed fused multiply-adds for
// each pair of values.  Four heads' loads are in flight.
//
// Measured on a GB300 (of 6792 GB/s copied): 8192 tokens of 32 + 8 + 8 heads of 128 to bf16 pages 38 us, 5.2 TB/s;
// 14538 of 16 + 2 + 2 heads of 256 to e4m3 pages 59 us, 4.8 TB/s; 64 such tokens 5.7 us; 32768 e4m3 rows of 2 heads
// of 256 read in 14.7 us, 6.9 TB/s (in a row of calls, which find part of their 101 MB in L2).
#include "attn_common.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;   // of a CTA: short ones, so that the last wave of CTAs is short too
constexpr int kUnroll = 4;  // loads that a lane has in flight (8192 tokens: 41 us with 4, 47 with 8, 55 with 2)

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
  const int page = c.table[(long)seq * c.max_pages + (pos >> c.page_shift)];
  if ((unsigned)page >= (unsigned)c.num_pages) {
    bad = true;
    return -1;
  }
  return (((long)page * Hkv) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// Eight bf16 values of a row of which D / 8 neighbouring lanes hold eight each: stores their codes and, by
// the row's first lane, the exponent byte (where `store` is set: the shuffles want the whole warp).
template <int D>
__device__ __forceinline__ void store_e4m3(const uint4& v, uint8_t* codes, uint8_t* byte, int lane, bool store) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
  auto row_max = [&](uint32_t top) {  // of two 16-bit magnitudes a lane
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    return max(top & 0xFFFFu, top >> 16);
  };
  uint32_t mag[4], top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mag[i] = r[i] & 0x7FFF7FFFu;
    top = __vmaxu2(top, mag[i]);
  }
  top = row_max(top);
  const bool odd = __any_sync(0xFFFFFFFFu, top >= 0x7F80u);  // some row has a value that is not finite
  if (odd) {  // the largest of the others
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((mag[i] & 0xFFFFu) < 0x7F80u) t = max(t, mag[i] & 0xFFFFu);
      if (mag[i] >> 16 < 0x7F80u) t = max(t, mag[i] >> 16);
    }
    top = row_max(t);
  }
  // 448 = 1.75 * 2^8: the exponent of the magnitude less 8, one more when its significand is above 1.75
  const int e = max((int)(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0), -117);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 y = __fmul2_rn(make_float2(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xFFFF0000u)), make_float2(inv, inv));
    if (odd) {  // the conversion saturates: what is not finite becomes NaN here
      if (!isfinite(y.x)) y.x = __uint_as_float(0x7FFFFFFFu);
      if (!isfinite(y.y)) y.y = __uint_as_float(0x7FFFFFFFu);
    }
    w[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (16 * (i & 1));
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
      if (h < heads) raw[u] = ld_once(src + h * rows.head);
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
__global__ void __launch_bounds__(32 * kWarps, 8) prepare_kernel(const __grid_constant__ PrepareParams p) {
  constexpr int kLanes = D / 8;  // lanes of a head
  await_grid();
  __shared__ __align__(16) float2 s_cs[kWarps][D / 2];
  __shared__ float2 s_turns[D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes;
  const long item = (long)blockIdx.x * kWarps + warp;
  const int t = (int)(item / p.split), share = (int)(item - (long)t * p.split);
  // turns of one position, in two parts: the only fp64 arithmetic, once for the CTA's tokens
  const int rot = p.rope.rot, half = rot / 2;
  for (int j = threadIdx.x; j < half; j += 32 * kWarps) {
    const double f = p.rope.freqs[j] * 0.15915494309189533577;
    const float hi = (float)f;
    s_turns[j] = make_float2(hi, (float)(f - (double)hi));
  }
  __syncthreads();
  if (t >= p.T) return;
  int first, len;
  const int seq = attn_seq_of(p.cu, p.N, p.T, t, first, len);
  if (seq < 0) {
    if (seq == -2) raise_error(p.err, kErrDeviceArgument);
    return;
  }
  const int kv = p.kv_lens[seq];
  if (kv < 0 || kv > min((long)p.cache.max_pages << p.cache.page_shift, (long)kMaxKeys)) {
    raise_error(p.err, kErrDeviceArgument);
    return;
  }
  const int pos = kv - len + (t - first);
  long place = -1;  // head-0 row of the position in the pool
  bool bad = false;
  if (pos >= 0) place = cache_row(p.cache, p.Hkv, seq, pos, bad);
  if (bad) {  // nothing of the token is written, its queries neither
    raise_error(p.err, kErrDeviceArgument);
    return;
  }

  // the token's cosines and sines
  for (int j = lane; j < half; j += 32) {
    float s, c;
    sincospif(2.f * turns_of(pos, s_turns[j].x, s_turns[j].y), &s, &c);
    s_cs[warp][j] = make_float2(c * p.rope.magnitude, s * p.rope.magnitude);
  }
  __syncwarp();
  // This lane's eight values of a head become x * a + y * b, y the values they are paired with (for halves
  // another lane's, half / 8 lanes away, else neighbours), times the norm's factor.
  const int d0 = sub * 8, away = half / 8;
  const bool turned = d0 < rot, low = d0 < half;
  const int partner = (lane - sub) + (!turned || p.rope.interleaved ? sub : low ? sub + away : sub - away);
  const uint32_t paired = turned ? 0xFFFFFFFFu : 0u;  // without a rotation b is 0, and y too: it might be an infinity
  auto run = [&](const HeadRows& rows, const uint16_t* w, int heads, auto store) {
    float2 a[4], b[4];
    {
      uint4 own = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), pair = own;  // bf16 ones
      if (w) {
        own = reinterpret_cast<const uint4*>(w)[sub];
        pair = p.rope.interleaved ? own : reinterpret_cast<const uint4*>(w)[partner % kLanes];
      }
      const uint32_t wo[4] = {own.x, own.y, own.z, own.w}, wp[4] = {pair.x, pair.y, pair.z, pair.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = bf2_to_float2(wo[i]), y = bf2_to_float2(wp[i]);
        float4 cs = make_float4(1.f, 0.f, 1.f, 0.f);  // cos, sin of the two values
        if (turned && p.rope.interleaved) {
          const float2 f = s_cs[warp][d0 / 2 + i];
          cs = make_float4(f.x, -f.y, f.x, f.y);
        } else if (turned) {
          cs = *reinterpret_cast<const float4*>(&s_cs[warp][(low ? d0 : d0 - half) + 2 * i]);
          if (low) cs.y = -cs.y, cs.w = -cs.w;
        }
        a[i] = make_float2(x.x * cs.x, x.y * cs.z);
        b[i] = p.rope.interleaved ? make_float2(x.y * cs.y, x.x * cs.w) : make_float2(y.x * cs.y, y.y * cs.w);
      }
    }
    each_head<D>(rows, t, heads, share, p.split, [&](const uint4& raw) {
      const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
      float2 x[4], y[4], ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = bf2_to_float2(r[i]);
      if (rot && !p.rope.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = bf2_to_float2(__shfl_sync(0xFFFFFFFFu, r[i], partner) & paired);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = turned ? make_float2(x[i].y, x[i].x) : make_float2(0.f, 0.f);
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
        const float2 z = __fmul2_rn(__ffma2_rn(x[i], a[i], __fmul2_rn(y[i], b[i])), make_float2(rms, rms));
        out[i] = pack_bf2(z.x, z.y);  // the one rounding to bf16
      }
      return make_uint4(out[0], out[1], out[2], out[3]);
    }, store);
  };
  auto to_cache = [&](void* pages, uint8_t* bytes) {
    return [=, &p](int h, const uint4& v, bool in) {
      const long row = place + ((long)h << p.cache.page_shift);
      if constexpr (kE4M3) {
        store_e4m3<D>(v, static_cast<uint8_t*>(pages) + row * D, bytes + row, sub, in);
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
  int Hkv, N, T, tokens;  // tokens: of a warp, at most 32
  bool wide;              // the outputs are 32-byte aligned
};

// 16 bytes of the cache a lane: 8 bf16 values copied, or 16 codes widened.  A warp's lanes hold a head's
// keys and its values side by side (at D = 256 in bf16, one and then the other), or those of two heads.
template <int D, bool kE4M3>
__global__ void __launch_bounds__(32 * kWarps) cache_read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kVals = kE4M3 ? 16 : 8, kLanes = D / kVals, kAt = 32 / kLanes;  // rows at a time: 1, 2 or 4
  const int lane = threadIdx.x & 31, sub = lane % kLanes, mine = lane / kLanes;
  await_grid();
  // p.tokens tokens of a warp: their places are looked up side by side, a lane each
  const long t0 = ((long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.tokens;
  const int nt = (int)min((long)p.tokens, p.T - t0);
  if (nt <= 0) return;
  long place = -1;
  if (lane < nt) {
    const int t = (int)t0 + lane;
    int first, len;
    bool bad = false;
    const int seq = attn_seq_of(p.cu, p.N, p.T, t, first, len);
    if (seq >= 0) {
      const long pos = (p.starts ? (long)p.starts[seq] : 0L) + (t - first);
      if (pos < 0 || pos >= min((long)p.cache.max_pages << p.cache.page_shift, (long)kMaxKeys)) bad = true;
      else place = cache_row(p.cache, p.Hkv, seq, (int)pos, bad);
    } else if (seq == -2) {
      bad = true;
    }
    if (bad) raise_error(p.err, kErrDeviceArgument);
  }
  // step s of the warp: rows (s % per) * kAt .. of token s / per; row r is head r / 2, its keys (even) or
  // values (odd)
  const int per = (2 * p.Hkv + kAt - 1) / kAt, steps = nt * per;
  for (int s0 = 0, next = 0, tok_next = 0; s0 < steps; s0 += kUnroll) {
    uint4 raw[kUnroll];
    uint32_t byte[kUnroll];
    uint16_t* dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int s = s0 + u, tok = tok_next, r = next * kAt + mine, h = r >> 1;
      if (++next == per) {
        next = 0;
        ++tok_next;
      }
      const long at = __shfl_sync(0xFFFFFFFFu, place, tok & 31);
      const bool is_k = (r & 1) == 0;
      const long row = at + ((long)h << p.cache.page_shift);
      dst[u] = nullptr;
      if (s < steps && h < p.Hkv && at >= 0) {
        raw[u] = ld_once(static_cast<const uint8_t*>(is_k ? p.cache.k : p.cache.v) + row * (D * (kE4M3 ? 1 : 2)) + sub * 16);
        if constexpr (kE4M3) byte[u] = (is_k ? p.cache.k_scale : p.cache.v_scale)[row];
        dst[u] = (is_k ? p.k_out : p.v_out) + ((t0 + tok) * p.Hkv + h) * D + sub * kVals;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!dst[u]) continue;
      if constexpr (kE4M3) {
        const float s = e8m0_value(byte[u]);
        const uint32_t c[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2 h = e4m3x4_to_half4(c[i]);
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
          const float2 x = __fmul2_rn(a, make_float2(s, s)), y = __fmul2_rn(b, make_float2(s, s));
          o[2 * i] = pack_bf2(x.x, x.y);
          o[2 * i + 1] = pack_bf2(y.x, y.y);
        }
        if (p.wide) {
          st_global32(dst[u], o);
        } else {
          reinterpret_cast<uint4*>(dst[u])[0] = make_uint4(o[0], o[1], o[2], o[3]);
          reinterpret_cast<uint4*>(dst[u])[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      } else {
        *reinterpret_cast<uint4*>(dst[u]) = raw[u];
      }
    }
  }
}

// Warps of one token: as many as bring sixteen warps to every SM, as long as each has loads to keep in
// flight (`units`: steps of a warp that has the token alone).  64 tokens of 16 + 2 + 2 heads of 256: 5.8 us
// with eight warps a token, 10.1 with one; 600 of 32 + 8 + 8 heads of 128: 7.2 (four; before a later
// step 8.0, 9.4 with eight, 9.8 with one); 8192 of them: 38 us with one (then 42, 75 with eight).
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
  return launch_early(kern, dim3(grid), 32 * kWarps, 0, env.stream, p);
}

cudaError_t launch_attn_cache_read(const LaunchEnv& env, int Hkv, int D, const PagedCache& cache,
                                   const int32_t* starts, const int32_t* cu, int N, int T, uint16_t* k_out,
                                   uint16_t* v_out) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  // Eight loads a lane, or fewer tokens where that leaves SMs without sixteen warps: 32768 e4m3 rows of 2 heads
  // of 256 14.5 us, 17.6 with one token a warp; 2000 of them 3.0, 3.8 with eight loads a lane all the same.
  // Stores of 32 bytes where the outputs' alignment allows: 14.5 us, 18.7 with 16.
  const int per = (2 * Hkv * D * (cache.e4m3 ? 1 : 2) + 511) / 512;
  int tokens = per >= 8 ? 1 : 8 / per;
  while (tokens > 1 && (long)T < 16L * sms * tokens) tokens /= 2;
  const bool wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31u) == 0;
  const ReadParams p = {cache, starts, cu, env.err, k_out, v_out, Hkv, N, T, tokens, wide};
  const unsigned grid = (unsigned)(((long)T + (long)tokens * kWarps - 1) / ((long)tokens * kWarps));
  auto kern = D == 128 ? (cache.e4m3 ? cache_read_kernel<128, true> : cache_read_kernel<128, false>)
                       : (cache.e4m3 ? cache_read_kernel<256, true> : cache_read_kernel<256, false>);
  return launch_early(kern, dim3(grid), 32 * kWarps, 0, env.stream, p);
}

}  // namespace gdn
