// attn.cu -- softmax attention of new tokens over a paged key/value cache.
#include "attn_common.cuh"

namespace gdn {
namespace {

struct AttnParams {
  const uint16_t* q;
  PagedCache cache;
  const int32_t* kv_lens;
  const int32_t* cu;
  HeadRows z;
  uint16_t* out;
  unsigned* err;
  float scale_log2;
  int Hq, Hkv, N, T;
};

// One warp for one query head of one token: D / 32 values a lane, the keys one after the other.
template <int D, bool kE4M3>
__global__ void __launch_bounds__(256) attn_simple_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kV = D / 32;
  const long w = (long)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (w >= (long)p.T * p.Hq) return;
  const int t = (int)(w / p.Hq), h = (int)(w % p.Hq), hk = h / (p.Hq / p.Hkv);
  int first, len;
  const int seq = attn_seq_of(p.cu, p.N, p.T, t, first, len);
  if (seq < 0) {
    if (seq == -2) raise_error(p.err, kErrDeviceArgument);
    return;
  }
  int kv = __ldg(p.kv_lens + seq);
  if (kv < 0 || kv > (long)p.cache.max_pages << p.cache.page_shift) {
    raise_error(p.err, kErrDeviceArgument);
    kv = 0;
  }
  const int pos = kv - len + (t - first), mask = (1 << p.cache.page_shift) - 1;
  float q[kV], o[kV] = {}, m = -INFINITY, l = 0.f;
  for (int i = 0; i < kV; ++i) q[i] = bf2f(p.q[((long)t * p.Hq + h) * D + lane * kV + i]) * p.scale_log2;
  for (int j = 0; j <= pos; ++j) {
    const int page = __ldg(p.cache.table + (long)seq * p.cache.max_pages + (j >> p.cache.page_shift));
    if ((unsigned)page >= (unsigned)p.cache.num_pages) {
      raise_error(p.err, kErrDeviceArgument);
      continue;
    }
    const long row = (((long)page * p.Hkv + hk) << p.cache.page_shift) + (j & mask);
    float k[kV], v[kV];
    for (int i = 0; i < kV; ++i) {
      const long at = row * D + lane * kV + i;
      if (kE4M3) {
        __nv_fp8_e4m3 a, b;
        a.__x = static_cast<const uint8_t*>(p.cache.k)[at];
        b.__x = static_cast<const uint8_t*>(p.cache.v)[at];
        k[i] = (float)a * e8m0_value(p.cache.k_scale[row]);
        v[i] = (float)b * e8m0_value(p.cache.v_scale[row]);
      } else {
        k[i] = bf2f(static_cast<const uint16_t*>(p.cache.k)[at]);
        v[i] = bf2f(static_cast<const uint16_t*>(p.cache.v)[at]);
      }
    }
    float s = 0.f;
    for (int i = 0; i < kV; ++i) s = fmaf(q[i], k[i], s);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    const float m2 = fmaxf(m, s), a = exp2f(m - m2), e = exp2f(s - m2);
    l = l * a + e;
    for (int i = 0; i < kV; ++i) o[i] = fmaf(e, v[i], o[i] * a);
    m = m2;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int i = 0; i < kV; ++i) {
    float y = o[i] * inv;
    if (p.z.p) y *= sigmoidf_(bf2f(p.z.p[t * p.z.token + h * p.z.head + lane * kV + i]));
    p.out[((long)t * p.Hq + h) * D + lane * kV + i] = f2bf(y);
  }
}

}  // namespace

size_t attn_workspace_bytes(int D) {
  (void)D;
  return 256;
}

cudaError_t launch_attn(const LaunchEnv& env, int Hq, int Hkv, int D, const uint16_t* q, const PagedCache& cache,
                        const int32_t* kv_lens, const int32_t* cu, int N, int T, float scale, const HeadRows& z,
                        uint16_t* out, void* workspace) {
  (void)workspace;
  const AttnParams p = {q, cache, kv_lens, cu, z, out, env.err, scale * kLog2e, Hq, Hkv, N, T};
  const long grid = ((long)T * Hq + 7) / 8;
  auto kern = D == 128 ? (cache.e4m3 ? attn_simple_kernel<128, true> : attn_simple_kernel<128, false>)
                       : (cache.e4m3 ? attn_simple_kernel<256, true> : attn_simple_kernel<256, false>);
  kern<<<(unsigned)grid, 256, 0, env.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
