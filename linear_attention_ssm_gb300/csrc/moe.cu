// moe.cu -- a mixture-of-experts layer for a few tokens.
//
//   l = x Wr^T,  score = softmax(l) or sigmoid(l),  chosen = the top_k of score + bias
//   h_e = silu(x G_e^T) * (x U_e^T),  out = sum_e weight_e h_e D_e^T + sigmoid(x . g) shared(x)
#include <cuda_fp8.h>
#include <math.h>

#include "gdn_kernels.h"

namespace gdn {
namespace {

constexpr int kBlock = 128;
constexpr int kWarps = 8;

struct Layout {  // of the workspace
  size_t logits, ids, weights, hidden, bytes;
};
Layout layout(const Moe& m, int T, int k) {
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  Layout l;
  l.logits = 0;
  l.ids = l.logits + up((size_t)T * (m.E + 1) * 4);
  l.weights = l.ids + up((size_t)T * k * 4);
  l.hidden = l.weights + up((size_t)T * k * 4);
  l.bytes = l.hidden + up((size_t)T * ((size_t)k * m.I + m.Is) * 4);
  return l;
}

__device__ __forceinline__ float weight_at(const void* w, bool e4m3, size_t at) {
  if (!e4m3) return bf2f(static_cast<const uint16_t*>(w)[at]);
  return __half2float(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(w)[at], __NV_E4M3));
}
__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

// An order of floats as unsigned numbers: NaN is 0, below all others.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0;
  const uint32_t b = __float_as_uint(f + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}

__global__ void route_kernel(const Moe m, const MoeCall c, float* logits, int32_t* ids, float* weights) {
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* l = logits + (size_t)t * (m.E + 1);
  const uint16_t* x = c.x + t * c.x_stride;
  for (int e = warp; e <= m.E; e += kWarps) {
    const uint16_t* w = e < m.E ? m.router + (size_t)e * m.H : m.shared_gate;
    if (e < m.E ? c.ids_in != nullptr : w == nullptr) continue;
    float s = 0.f;
    for (int i = lane; i < m.H; i += 32) s = fmaf(bf2f(x[i]), bf2f(w[i]), s);
    s = warp_sum(s);
    if (lane == 0) l[e] = s;
  }
  __syncthreads();
  if (threadIdx.x) return;
  for (int j = 0; j < c.top_k; ++j) {
    const size_t at = (size_t)t * c.top_k + j;
    if (c.ids_in) {
      const int id = c.ids_in[at];
      if (id >= m.E) raise_error(c.err, kErrDeviceArgument);
      ids[at] = id < m.E ? id : -1;
      weights[at] = c.weights_in[at];
      continue;
    }
    uint32_t best = 0;
    int at_best = -1;
    float top = -INFINITY, sum = 0.f;
    for (int e = 0; e < m.E; ++e) top = fmaxf(top, l[e]);
    for (int e = 0; e < m.E; ++e) sum += expf(l[e] - top);
    for (int e = 0; e < m.E; ++e) {
      bool taken = false;
      for (int i = 0; i < j; ++i) taken |= ids[(size_t)t * c.top_k + i] == e;
      if (taken) continue;
      float s = l[e];
      if (m.router_bias) s = (c.sigmoid ? 1.f / (1.f + expf(-s)) : expf(s - top) / sum) + m.router_bias[e];
      if (at_best < 0 || order_key(s) > best) best = order_key(s), at_best = e;
    }
    ids[at] = at_best;
    const float a = l[at_best];
    if (c.renormalise) weights[at] = c.sigmoid ? fminf(a, 0.f) - log1pf(expf(-fabsf(a))) : a;
    else weights[at] = c.scale * (c.sigmoid ? 1.f / (1.f + expf(-a)) : expf(a - top) / sum);
  }
  float* w = weights + (size_t)t * c.top_k;
  if (!c.ids_in && c.renormalise) {
    float top = -INFINITY, sum = 0.f;
    for (int j = 0; j < c.top_k; ++j) top = fmaxf(top, w[j]);
    for (int j = 0; j < c.top_k; ++j) sum += w[j] = expf(w[j] - top);
    for (int j = 0; j < c.top_k; ++j) w[j] = c.scale * (w[j] / sum);
  }
  for (int j = 0; j < c.top_k; ++j) {
    if (c.ids_out) c.ids_out[(size_t)t * c.top_k + j] = ids[(size_t)t * c.top_k + j];
    if (c.weights_out) c.weights_out[(size_t)t * c.top_k + j] = w[j];
  }
}

// A warp's dot product of row `row` of a [rows, cols] matrix with a vector of bf16 or fp32 values.
template <typename X>
__device__ __forceinline__ float dot(const void* w, const float* scale, size_t matrix, int rows, int cols, int row, const X* x,
                                     int lane) {
  const size_t base = (matrix * rows + row) * cols;
  const int rb = (rows + kBlock - 1) / kBlock, cb = (cols + kBlock - 1) / kBlock;
  float s = 0.f;
  for (int b = 0; b < cb; ++b) {
    float d = 0.f;
    for (int i = b * kBlock + lane; i < min(cols, (b + 1) * kBlock); i += 32) {
      const float v = sizeof(X) == 2 ? bf2f((uint16_t)x[i]) : (float)x[i];
      d = fmaf(weight_at(w, scale != nullptr, base + i), v, d);
    }
    s = fmaf(d, scale ? scale[(matrix * rb + row / kBlock) * cb + b] : 1.f, s);
  }
  return warp_sum(s);
}

__global__ void hidden_kernel(const Moe m, const MoeCall c, const int32_t* ids, float* hidden) {
  const int slot = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int routed = c.T * c.top_k;
  const bool shared = slot >= routed;
  const int t = shared ? slot - routed : slot / c.top_k, I = shared ? m.Is : m.I;
  const int i = blockIdx.x * kWarps + warp, e = shared ? 0 : ids[slot];
  if (i >= I || e < 0) return;
  const void* w = shared ? m.shared_gate_up : m.gate_up;
  const float* sc = shared ? m.shared_gate_up_scale : m.gate_up_scale;
  const uint16_t* x = c.x + t * c.x_stride;
  const float g = dot(w, sc, 2 * (size_t)e, I, m.H, i, x, lane), u = dot(w, sc, 2 * (size_t)e + 1, I, m.H, i, x, lane);
  float* h = shared ? hidden + (size_t)routed * m.I + (size_t)t * m.Is : hidden + (size_t)slot * m.I;
  if (lane == 0) h[i] = silu(g) * u;
}

__global__ void out_kernel(const Moe m, const MoeCall c, const float* logits, const int32_t* ids, const float* weights,
                           const float* hidden) {
  const int t = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kWarps + warp;
  if (row >= m.H) return;
  float y = 0.f;
  for (int j = 0; j < c.top_k; ++j) {
    const size_t slot = (size_t)t * c.top_k + j;
    const int e = ids[slot];
    if (e < 0) continue;
    y = fmaf(weights[slot], dot(m.down, m.down_scale, e, m.H, m.I, row, hidden + slot * m.I, lane), y);
  }
  if (m.Is) {
    const float* h = hidden + (size_t)c.T * c.top_k * m.I + (size_t)t * m.Is;
    const float g = m.shared_gate ? 1.f / (1.f + expf(-logits[(size_t)t * (m.E + 1) + m.E])) : 1.f;
    y = fmaf(g, dot(m.shared_down, m.shared_down_scale, 0, m.H, m.Is, row, h, lane), y);
  }
  if (lane == 0) c.out[(size_t)t * m.H + row] = f2bf(y);
}

}  // namespace

size_t moe_workspace_bytes(const Moe& m, int T, int top_k) { return layout(m, T, top_k).bytes; }

cudaError_t launch_moe(const LaunchEnv& env, const Moe& m, MoeCall c, void* workspace) {
  c.err = env.err;
  const Layout l = layout(m, c.T, c.top_k);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* logits = reinterpret_cast<float*>(ws + l.logits);
  int32_t* ids = reinterpret_cast<int32_t*>(ws + l.ids);
  float* weights = reinterpret_cast<float*>(ws + l.weights);
  float* hidden = reinterpret_cast<float*>(ws + l.hidden);
  route_kernel<<<c.T, kWarps * 32, 0, env.stream>>>(m, c, logits, ids, weights);
  const int widest = m.I > m.Is ? m.I : m.Is, slots = c.T * c.top_k + (m.Is ? c.T : 0);
  hidden_kernel<<<dim3((widest + kWarps - 1) / kWarps, slots), kWarps * 32, 0, env.stream>>>(m, c, ids, hidden);
  out_kernel<<<dim3((m.H + kWarps - 1) / kWarps, c.T), kWarps * 32, 0, env.stream>>>(m, c, logits, ids, weights, hidden);
  return cudaGetLastError();
}

}  // namespace gdn
