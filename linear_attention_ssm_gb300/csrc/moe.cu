// moe.cu -- a mixture-of-experts layer for a few tokens.
//
//   l = x Wr^T,  score = softmax(l) or sigmoid(l),  chosen = the top_k of score + bias
//   h_e = silu(x G_e^T) * (x U_e^T),  out = sum_e weight_e h_e D_e^T + sigmoid(x . g) shared(x)
//
// The first kernel forms the logits and lays the tokens out; with more than 16 tokens a second one chooses (16 warps of every
// CTA of the last one do it otherwise: 64 tokens of 288 experts took 28 us there, 12 us with a kernel of their own).  The last
// kernel streams the chosen experts' weights once.  HBM bounds it where they are many: 64 tokens of 288 experts of 4096 x 1536
// and a shared one, 3.1 GB of e4m3 weights, 538 us, 5.7 TB/s with everything.  Latency does where they are few: one token of
// 64 experts of 2048 x 1024, 50 MB, 30 us, of which the logits take 3, the choice 5, and then 16 and 8 steps of about half a
// microsecond each wait for one another.
//
// Work is taken in units from one list by an atomic counter: 16 rows of a gate matrix with the 16 rows of the up projection
// beside them, over all of H (h for those places and up to 8 of the expert's tokens), then 32 rows of a down projection over
// all of I (for up to 4 tokens, whose h are in two parts), then 32 columns of the output for 8 tokens, whose sum over the
// experts is formed in the order of the choice.  An expert of more tokens has units for each group of them, one after another
// in the list: the first finds the weights in HBM, the others in L2.  A team of two warps has a ring of stages in shared
// memory: one warp takes units and copies their weights by TMA and their tokens' values by plain asynchronous copies, the
// other multiplies.  The ring runs ahead over the ends of units and from one kind to the next, and the wait for all of h falls
// into that time.  (Eight warps that both loaded and multiplied took 1027 us for the first of the sizes above, two warps that
// shared the products and of which one loaded 943; ten teams with rings of three stages 551 where these took 556, and 32
// instead of 30 for one token.)  A unit is waited for only by units of the next kind, and by then every unit of its kind has
// been taken by a team that runs and waits for nothing: the kernel ends however few of its CTAs run at a time.
//
// Products are m16n8k16 of mma.sync: weights fill the 16 rows, an expert's tokens the 8 columns, so that a weight is an operand
// as it lies in memory.  Both operands of a lane may come from any places of k as long as they are the same ones; a lane reads
// 16-byte chunks of its rows, and the tokens lie in memory in that order.  e4m3 weights become binary16 beside the tokens
// (exact; a token is divided by a power of two that brings its largest value to 2^15 .. 65280, the largest bf16 below 2^16:
// values down to 2^-32 of it, 2^-17 at least, are exact, and smaller ones lose at most half of 2^-24, 2^-40 of it).
//
// h is held in fp32 and split by the warp that multiplies: beside e4m3 weights into two binary16 parts in two columns, relative
// to the largest h of its token and expert, which the units of the first kind gather and which is there when all of h is: off
// by at most 2^-23 of itself or 2^-39 of the largest; beside bf16 weights into three bf16 parts, all 24 bits, in two columns
// and, by a second product, the third part in the second one.  (With two bf16 parts beside either, 16 bits, 64 tokens of 288
// experts took 557 us, now 537, and 17 of 32 in bf16 102.6, now 104.8.)
#include <string.h>

#include "attn_common.cuh"
#include "gdn_kernels.h"

namespace gdn {
namespace {

constexpr int kTeams = 8, kWarps = 2 * kTeams, kThreads = kWarps * 32;  // a team: a warp that loads, one that multiplies
constexpr int kMaxTokens = 64, kMaxTopK = 16, kMaxExperts = 1024;
constexpr int kMaxSlots = kMaxTokens * (kMaxTopK + 1);  // (token, expert) pairs
constexpr int kStageBytes = 4096;  // of weights: 32 rows of 128 bytes
constexpr int kValueRows = 8;       // beside them: columns of a product
constexpr int kStages = 4;
constexpr int kQueue = 8;           // units on their way: more than stages, and the one in hand
constexpr uint32_t kWaitLimit = 1u << 20;  // polls of one mbarrier before giving up
constexpr uint32_t kSpinLimit = 1u << 22;  // polls of the counter of finished units
constexpr int kBlock = 128;

struct Layout {  // of the workspace
  size_t counters, logits, ids, weights, x, x_scale, tops, hidden, shared_hidden, y, bytes;
};
__host__ __device__ inline int pad256(int n) { return (n + 255) & ~255; }
Layout layout(const Moe& m, int T, int k) {
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  Layout l;
  l.counters = 0;
  l.logits = l.counters + up((2 + (m.H + 31) / 32) * 4);
  l.ids = l.logits + up((size_t)T * (m.E + 1) * 4);
  l.weights = l.ids + up((size_t)T * k * 4);
  l.x = l.weights + up((size_t)T * k * 4);
  l.x_scale = l.x + up((size_t)T * pad256(m.H) * 2);
  l.tops = l.x_scale + up((size_t)T * 4);
  l.hidden = l.tops + up((size_t)T * (k + 1) * 16);
  l.shared_hidden = l.hidden + up((size_t)T * k * pad256(m.I) * 4);
  l.y = l.shared_hidden + up((size_t)T * pad256(m.Is) * 4);
  l.bytes = l.y + up((size_t)T * (k + (m.Is ? 1 : 0)) * m.H * 4);
  return l;
}

struct MoeParams {
  CUtensorMap gate_up, down, shared_gate_up, shared_down;  // boxes of 128 bytes x 16 rows x 2 halves, or x 32 rows x 1
  Moe m;
  MoeCall c;
  unsigned* counters;  // next unit; first units done; for each 32 rows of the output, down units done
  bool chosen;         // a kernel of its own chooses
  int32_t* ids;        // [T][top_k] and their weights, where a kernel of its own chooses
  float* weights;
  float* logits;       // [T][E + 1], the shared gate's behind the experts'
  uint16_t* x;         // [T][pad256(H)] tokens in the products' order, bf16 or binary16
  float* x_scale;      // [T] what a binary16 token is multiplied with
  uint4* tops;         // [T * top_k], then [T] for the shared expert: x is the largest finite |h| of a slot, as bits
  float* hidden;       // [T * top_k][pad256(I)] in the products' order
  float* shared_hidden;
  float* y;            // [slots][H] weighted rows of the experts
};

// Where 8 values from k on (a multiple of 8) lie in the products' order.  A 128-byte piece of a row of weights has 8 chunks of
// 16 bytes, of which lane c of a quad reads 2 c and 2 c + 1; the tokens' values beside them come 16 bytes a lane and load.
template <bool kE4M3>
__host__ __device__ __forceinline__ int place(int k) {
  const int g = (k >> 3) & 15;
  return (k & ~127) + 8 * (kE4M3 ? (g & 3) * 4 + (g >> 2) : (((g >> 3) * 2 + (g & 1)) * 4 + ((g >> 1) & 3)));
}

// The same for a single k of h, four values of which are 16 bytes: a lane's 16 bytes of weights go with 16 or 8 values, and its
// four values of a product lie beside the other three lanes' of the quad.
template <bool kE4M3>
__host__ __device__ __forceinline__ int hidden_place(int k) {
  constexpr int kChunk = kE4M3 ? 16 : 8, kRow = 8 * kChunk;  // values beside a chunk; a row of weights
  const int in = k & (kRow - 1), chunk = in / kChunk;
  return k - in + (((chunk & 1) * (kChunk / 4) + (in % kChunk) / 4) * 4 + (chunk >> 1)) * 4 + (k & 3);
}

// Loads of what other kernels or CTAs wrote, or read often: where they are written, through L1.
__device__ __forceinline__ uint4 ld_here(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_f32(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float2 lds_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// An order of floats as unsigned numbers above 1: NaN is 1, below all others; 0 stands for none.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 1;
  const uint32_t b = __float_as_uint(f + 0.f);
  return (b >> 31 ? ~b : b | 0x80000000u) + 1;
}

// The next kernel of the stream may take its places on the SMs: it waits for this one's end all the same.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }

// ---------------------------------------------------------------- tokens and logits

constexpr int kPrepareWarps = 8, kPrepareThreads = kPrepareWarps * 32;

// A CTA for each token's layout, then one for the dot products of 4 rows of the router (the shared gate's behind the last)
// with 8 tokens, whose warps split H.
constexpr int kRows = 4;
template <bool kE4M3>
__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(const __grid_constant__ MoeParams p) {
  __shared__ float tops[kPrepareWarps], parts[kPrepareWarps][32];
  let_next_start();
  await_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = p.m.H;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < 2 + (H + 31) / 32; i += kPrepareThreads) p.counters[i] = 0;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.c.T * (p.c.top_k + 1); i += kPrepareThreads) p.tops[i] = make_uint4(0, 0, 0, 0);
  if (blockIdx.x < p.c.T) {
    const int t = blockIdx.x;
    const uint16_t* x = p.c.x + t * p.c.x_stride;
    uint16_t* to = p.x + (size_t)t * pad256(H);
    float scale = 1.f;
    if (kE4M3) {
      float top = 0.f;  // the largest finite magnitude
      for (int k = threadIdx.x * 8; k < H; k += kPrepareThreads * 8) {
        const uint4 v = ld_once(x + k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = fabsf(__uint_as_float(w[i] << 16)), b = fabsf(__uint_as_float(w[i] & 0xFFFF0000u));
          if (a < INFINITY) top = fmaxf(top, a);
          if (b < INFINITY) top = fmaxf(top, b);
        }
      }
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      if (lane == 0) tops[warp] = top;
      __syncthreads();
      for (int w = 0; w < kPrepareWarps; ++w) top = fmaxf(top, tops[w]);
      // the largest value's exponent, raised to where the power of two has a reciprocal
      const int e = max((int)(__float_as_uint(top) >> 23), 16);
      scale = __uint_as_float((uint32_t)(e - 15) << 23);
      const float inverse = __uint_as_float((uint32_t)(254 - (e - 15)) << 23);
      for (int k = threadIdx.x * 8; k < H; k += kPrepareThreads * 8) {
        const uint4 v = ld_once(x + k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          h[i] = pack_half2(__uint_as_float(w[i] << 16) * inverse, __uint_as_float(w[i] & 0xFFFF0000u) * inverse);
        *reinterpret_cast<uint4*>(to + place<kE4M3>(k)) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    } else {
      for (int k = threadIdx.x * 8; k < H; k += kPrepareThreads * 8) *reinterpret_cast<uint4*>(to + place<kE4M3>(k)) = ld_once(x + k);
    }
    if (threadIdx.x == 0) p.x_scale[t] = scale;
    // zeroes behind the ends of rows, as the copies of weights have them
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int wide = pad256(p.m.I), shared_wide = pad256(p.m.Is);
    for (int k = H + threadIdx.x * 8; k < pad256(H); k += kPrepareThreads * 8) *reinterpret_cast<uint4*>(to + place<kE4M3>(k)) = zero;
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < p.c.top_k; ++s)
      for (int k = p.m.I + threadIdx.x * 4; k < wide; k += kPrepareThreads * 4)
        *reinterpret_cast<float4*>(p.hidden + ((size_t)t * p.c.top_k + s) * wide + hidden_place<kE4M3>(k)) = none;
    for (int k = p.m.Is + threadIdx.x * 4; k < shared_wide; k += kPrepareThreads * 4)
      *reinterpret_cast<float4*>(p.shared_hidden + (size_t)t * shared_wide + hidden_place<kE4M3>(k)) = none;
    return;
  }
  // rows of the router, unless the routing is given, then the shared gate
  const int groups = (p.c.T + 7) / 8, item = blockIdx.x - p.c.T, t0 = item % groups * 8;
  const int e0 = (p.c.ids_in ? p.m.E : 0) + item / groups * kRows, rows = min(kRows, p.m.E + (p.m.shared_gate ? 1 : 0) - e0);
  const int count = min(8, p.c.T - t0);
  float sum[32] = {};  // of row j and token i at 8 j + i
  for (int k = threadIdx.x * 8; k < H; k += kPrepareThreads * 8) {
    uint4 a[kRows], b[8];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      a[j] = j < rows ? ld_once((e0 + j < p.m.E ? p.m.router + (size_t)(e0 + j) * H : p.m.shared_gate) + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = i < count ? ld_here(p.c.x + (t0 + i) * p.c.x_stride + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= count) break;
      const uint32_t bw[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const uint32_t aw[4] = {a[j].x, a[j].y, a[j].z, a[j].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sum[8 * j + i] = fmaf(__uint_as_float(aw[q] << 16), __uint_as_float(bw[q] << 16), sum[8 * j + i]);
          sum[8 * j + i] = fmaf(__uint_as_float(aw[q] & 0xFFFF0000u), __uint_as_float(bw[q] & 0xFFFF0000u), sum[8 * j + i]);
        }
      }
    }
  }
  // lane l gets sum l of the warp: halves of what is left are exchanged
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float mine = lane & o ? sum[i + o] : sum[i], other = lane & o ? sum[i] : sum[i + o];
      sum[i] = mine + __shfl_xor_sync(~0u, other, o);
    }
  parts[warp][lane] = sum[0];
  __syncthreads();
  if (warp == 0 && lane / 8 < rows && lane % 8 < count) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kPrepareWarps; ++w) s += parts[w][lane];
    p.logits[(size_t)(t0 + lane % 8) * (p.m.E + 1) + e0 + lane / 8] = s;
  }
}

// ---------------------------------------------------------------- the choice

// What every CTA works out for itself: the tokens' experts and the experts' tokens.
struct Choice {  // on the way to the lists
  unsigned long long mask[kMaxExperts];  // tokens of an expert
  float weight[kMaxTokens][kMaxTopK];
  unsigned long long sums[kWarps];
  uint16_t index[kMaxExperts];           // the active expert's number
  int16_t id[kMaxTokens][kMaxTopK];      // negative: none
};
struct Lists {
  float weight[kMaxSlots];
  float x_scale[kMaxTokens];
  int active;                       // experts that have tokens
  uint16_t expert[kMaxExperts];     // of an active expert
  uint16_t first[kMaxExperts + 2];  // its first slot
  // groups of an expert's tokens, the columns of a unit of either kind: those before it, and the expert of a group
  uint16_t groups[2][kMaxExperts + 1];
  uint16_t owner[2][kMaxExperts + kMaxTokens * kMaxTopK / 4];
  uint16_t slot_of[kMaxTokens][kMaxTopK + 1];  // kNone: none; the shared expert's last
  uint8_t token[kMaxSlots];
};
// tokens of a group: 8 columns hold so many tokens, or their h in two parts
__host__ __device__ constexpr int group_of(int kind) { return kind ? 4 : 8; }
constexpr uint16_t kNone = 0xFFFF;

// One warp: token t's top_k experts and their weights, of choice j in lane j.  A lane holds the keys of every 32nd expert.
template <int kOwn>
__device__ __forceinline__ void choose(const MoeParams& p, int t, int lane, int& id, float& w) {
  const MoeCall& c = p.c;
  const int E = p.m.E;
  const float* l = p.logits + (size_t)t * (E + 1);
  float a[kOwn], top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) a[i] = lane + 32 * i < E ? ld_f32(l + lane + 32 * i) : -INFINITY;
  float bias[kOwn];  // on its way beside the logits
  if (p.m.router_bias) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) bias[i] = lane + 32 * i < E ? ld_f32(p.m.router_bias + lane + 32 * i) : 0.f;
  }
  if (!c.sigmoid && (p.m.router_bias || !c.renormalise)) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) top = fmaxf(top, a[i]);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
#pragma unroll
    for (int i = 0; i < kOwn; ++i) sum += lane + 32 * i < E ? expf(a[i] - top) : 0.f;
    sum = warp_sum(sum);
  }
  auto score = [&](float v) { return c.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) / sum; };
  uint32_t key[kOwn];  // 0: taken, or none
  if (p.m.router_bias) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      key[i] = lane + 32 * i < E ? order_key(score(a[i]) + bias[i]) : 0;
  } else {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) key[i] = lane + 32 * i < E ? order_key(a[i]) : 0;
  }
  id = 0;
  for (int j = 0; j < c.top_k; ++j) {
    uint32_t best = 0;
    int at = kMaxExperts;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (key[i] > best) best = key[i], at = lane + 32 * i;
    const uint32_t k = __reduce_max_sync(~0u, best), with = __ballot_sync(~0u, best == k);
    int e = __shfl_sync(~0u, at, __ffs(with) - 1);
    if (with & (with - 1)) e = __reduce_min_sync(~0u, best == k ? at : kMaxExperts);  // a tie
    if (lane == j) id = e;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (e == lane + 32 * i) key[i] = 0;
  }
  const bool chosen = lane < c.top_k;
  float mine = 0.f;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const float v = __shfl_sync(~0u, a[i], id & 31);
    if (chosen && id >> 5 == i) mine = v;
  }
  if (c.renormalise) {
    // in logarithms, relative to the largest: no score underflows before its sum is formed
    const float v = !c.sigmoid ? mine : fminf(mine, 0.f) - log1pf(expf(-fabsf(mine)));
    float high = chosen ? v : -INFINITY;
    for (int o = 16; o; o >>= 1) high = fmaxf(high, __shfl_xor_sync(~0u, high, o));
    const float x = chosen ? expf(v - high) : 0.f;
    w = x / warp_sum(x);
  } else {
    w = score(mine);
  }
  w *= c.scale;
  if (chosen && (p.chosen || blockIdx.x == 0)) {
    if (c.ids_out) c.ids_out[t * c.top_k + lane] = id;
    if (c.weights_out) c.weights_out[t * c.top_k + lane] = w;
  }
}
// Keys a lane, by the number of experts: 8 tokens of 64 experts 24.5 us with 2 and 25.8 with 10, of 128 25.6 with 4 and 26.6 with
// 10; 16 of 288 30.1 with 10 and 37.7 with 32 (64, whose choice has a kernel: 42.7 and 44.9).  256 experts take no less with 8
// than with 10: 30.1 (64 tokens: 40.9 and 41.2).
__device__ __forceinline__ void choose_any(const MoeParams& p, int t, int lane, int& id, float& w) {
  if (p.m.E <= 64) choose<2>(p, t, lane, id, w);
  else if (p.m.E <= 128) choose<4>(p, t, lane, id, w);
  else if (p.m.E <= 320) choose<10>(p, t, lane, id, w);
  else choose<32>(p, t, lane, id, w);
}
// A warp for each token, where the next kernel's CTAs do not choose for themselves: they have a warp for each of 16 tokens.
constexpr int kChooseWarps = 4;
__global__ void __launch_bounds__(kChooseWarps * 32) choose_kernel(const __grid_constant__ MoeParams p) {
  let_next_start();
  await_grid();
  const int t = blockIdx.x * kChooseWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= p.c.T) return;
  int id;
  float w;
  choose_any(p, t, lane, id, w);
  if (lane < p.c.top_k) {
    p.ids[t * p.c.top_k + lane] = id;
    p.weights[t * p.c.top_k + lane] = w;
  }
}

constexpr int kPass = kThreads / kMaxTopK;  // tokens at a time, a thread for each of their choices

// The whole CTA: every token's choice.
__device__ __forceinline__ void make_choice(const MoeParams& p, Choice& choice, Lists& s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, T = p.c.T, k = p.c.top_k, E = p.m.E;
  const int j = tid % kMaxTopK, t0 = tid / kMaxTopK;
  for (int e = tid; e < E; e += kThreads) choice.mask[e] = 0;
  if (tid < T) s.x_scale[tid] = ld_f32(p.x_scale + tid);
  if (p.c.ids_in || p.chosen) {
    const int32_t* ids = p.c.ids_in ? p.c.ids_in : p.ids;
    const float* weights = p.c.ids_in ? p.c.weights_in : p.weights;
    for (int t = t0; t < T && j < k; t += kPass) {
      int id;
      asm volatile("ld.global.b32 %0, [%1];" : "=r"(id) : "l"(ids + t * k + j));
      if (id >= E) {
        if (blockIdx.x == 0) raise_error(p.c.err, kErrDeviceArgument);
        id = -1;
      }
      choice.id[t][j] = (int16_t)max(id, -1);
      choice.weight[t][j] = ld_f32(weights + t * k + j);
    }
  } else if (warp < T) {
    int id;
    float w;
    choose_any(p, warp, lane, id, w);
    if (lane < k) {
      choice.id[warp][lane] = (int16_t)id;
      choice.weight[warp][lane] = w;
    }
  }
  __syncthreads();
}
// The whole CTA: what the units of work need to know.
__device__ __forceinline__ void make_lists(const MoeParams& p, Choice& choice, Lists& s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, T = p.c.T, k = p.c.top_k, E = p.m.E;
  const int j = tid % kMaxTopK, t0 = tid / kMaxTopK;
  for (int t = t0; t < T && j < k; t += kPass)
    if (choice.id[t][j] >= 0) atomicOr(&choice.mask[choice.id[t][j]], 1ull << t);
  __syncthreads();
  // Experts that have tokens, in order: each thread has some neighbours.  Of those before it, 16 bits each: experts, slots,
  // groups of the two kinds.
  constexpr int kOwn = (kMaxExperts + kThreads - 1) / kThreads;
  typedef unsigned long long u64;
  auto adds = [](int n) {
    return n ? 1ull | (u64)n << 16 | (u64)((n + group_of(0) - 1) / group_of(0)) << 32 | (u64)((n + group_of(1) - 1) / group_of(1)) << 48 : 0ull;
  };
  u64 own = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int e = tid * kOwn + i;
    own += adds(e < E ? __popcll(choice.mask[e]) : 0);
  }
  u64 before = own;
  for (int o = 1; o < 32; o <<= 1) {
    const u64 x = __shfl_up_sync(~0u, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) choice.sums[warp] = before;
  __syncthreads();
  u64 all = 0;
  before -= own;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += choice.sums[w];
    all += choice.sums[w];
  }
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int e = tid * kOwn + i, n = e < E ? __popcll(choice.mask[e]) : 0;
    if (n) {
      const int a = before & 0xFFFF;
      s.expert[a] = (uint16_t)e;
      s.first[a] = (uint16_t)(before >> 16);
      choice.index[e] = (uint16_t)a;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        const int g = before >> (32 + 16 * kind) & 0xFFFF;
        s.groups[kind][a] = (uint16_t)g;
        for (int q = 0; q * group_of(kind) < n; ++q) s.owner[kind][g + q] = (uint16_t)a;
      }
      before += adds(n);
    }
  }
  const int active = all & 0xFFFF, slots = all >> 16 & 0xFFFF;
  if (tid == 0) {
    s.active = active;
    s.first[active] = (uint16_t)slots;  // the shared expert's slots are behind the others'
    s.first[active + 1] = (uint16_t)(slots + T);
    s.groups[0][active] = (uint16_t)(all >> 32);
    s.groups[1][active] = (uint16_t)(all >> 48);
  }
  __syncthreads();
  for (int t = t0; t < T && j < k; t += kPass) {
    const int e = choice.id[t][j];
    bool again = e < 0;
    float w = 0.f;
#pragma unroll 4
    for (int q = 0; q < k; ++q) {
      const bool same = choice.id[t][q] == e;
      const float v = choice.weight[t][q];
      if (same) w += v;
      again |= same && q < j;
    }
    int slot = kNone;
    if (!again) {
      slot = s.first[choice.index[e]] + __popcll(choice.mask[e] & ((1ull << t) - 1));
      s.token[slot] = (uint8_t)t;
      s.weight[slot] = w;
    }
    s.slot_of[t][j] = (uint16_t)slot;
  }
  if (tid < T) {
    s.slot_of[tid][kMaxTopK] = p.m.Is ? (uint16_t)(slots + tid) : kNone;
    if (p.m.Is) {
      s.token[slots + tid] = (uint8_t)tid;
      s.weight[slots + tid] =
          p.m.shared_gate ? 1.f / (1.f + expf(-ld_f32(p.logits + (size_t)tid * (p.m.E + 1) + p.m.E))) : 1.f;
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- the experts

// D += A B: m16n8k16 with binary16 or bf16 operands and fp32 sums.  Lane l has rows l / 4 and l / 4 + 8 of A at the k of its
// place l % 4, column l / 4 of B at the same k, and columns 2 (l % 4), + 1 of D's two rows.
template <bool kHalf>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint2& upper, const uint2& lower, uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(upper.x), "r"(lower.x), "r"(upper.y), "r"(lower.y), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(upper.x), "r"(lower.x), "r"(upper.y), "r"(lower.y), "r"(b0), "r"(b1));
}
// The operand that a column of h needs beside a product's weights, from four values: the first part of them in even columns,
// the second in odd ones.  Binary16, after the product with a power of two:
__device__ __forceinline__ uint2 half_parts(const float4& h, float by, uint32_t odd) {  // odd: all ones, or 0
  const uint32_t a = pack_half2(h.x * by, h.y * by) & odd, b = pack_half2(h.z * by, h.w * by) & odd;
  const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return make_uint2(pack_half2(fmaf(h.x, by, -u.x), fmaf(h.y, by, -u.y)), pack_half2(fmaf(h.z, by, -v.x), fmaf(h.w, by, -v.y)));
}
// bf16, each part eight bits of the significand, cut off so that the three are exact; `third` is of odd columns, too.
__device__ __forceinline__ uint2 bf16_parts(const float4& h, uint32_t odd, uint2& third) {
  const float f[4] = {h.x, h.y, h.z, h.w};
  uint32_t part[4], rest[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = f[i] - __uint_as_float(__float_as_uint(f[i]) & odd & 0xFFFF0000u);  // h, or its last 16 bits
    part[i] = __float_as_uint(a);
    rest[i] = __float_as_uint(a - __uint_as_float(part[i] & (0xFFFF0000u | ~odd)));  // 0, or its last eight
  }
  third = make_uint2(__byte_perm(rest[0], rest[1], 0x7632), __byte_perm(rest[2], rest[3], 0x7632));
  return make_uint2(__byte_perm(part[0], part[1], 0x7632), __byte_perm(part[2], part[3], 0x7632));
}

__device__ __forceinline__ bool warp_poll(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(done)
               : "r"(bar), "r"(parity)
               : "memory");
  return __all_sync(~0u, done);
}
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitLimit && !warp_poll(bar, parity); ++i) {
  }
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// by one lane of the warp
__device__ __forceinline__ void first_arrive(uint32_t bar) {
  asm volatile("{\n.reg .pred e;\nelect.sync _|e, 0xFFFFFFFF;\n@e mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(bar) : "memory");
}
// A stage's load of weights, by one lane of the warp.
__device__ __forceinline__ void warp_load(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\n"
      "elect.sync _|e, 0xFFFFFFFF;\n"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %6;\n"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%1], [%2, {%3, %4, %5}], [%0];\n"
      "}" ::"r"(bar),
      "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "n"(kStageBytes)
      : "memory");
}
__device__ __forceinline__ void copy_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// every lane's: its copies up to here have landed
__device__ __forceinline__ void copies_done_to(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// A unit of work.
struct Unit {
  int kind;          // 0: 16 rows of gate and up, 1: 32 rows of down, 2: 32 columns of the output for 8 tokens
  int a;             // the active expert, `active` for the shared one
  bool shared;
  int row, k;        // first row; length of a row
  int first, count;  // slots of a group of the expert's tokens; the first token
};

// Of a team: a warp that loads and one that multiplies.  A stage of their ring has 4 KB of weights and behind them the tokens'
// values for the same k (loads through the cache take several thousand cycles while the copies fill the memory's queues):
// a row for each token, or two for its h.
template <bool kE4M3>
struct Stage {
  static constexpr int kK = kE4M3 ? 128 : 64;  // values of a row
  static constexpr int kRowBytes = 2 * kK;     // of values
  static constexpr int kBytes = (kStageBytes + kValueRows * kRowBytes + 1023) / 1024 * 1024;
};
struct Team {
  uint64_t full[kStages], empty[kStages];
  alignas(16) uint4 tops[kStages][4];   // of a unit's first stage: its slots' largest h
  alignas(8) float scales[kStages][2];  // of a stage's rows: of gate and up, or of down
  int queue[kQueue];         // units on their way; negative: no more
  int finished;              // units of the first kind
  int failed;                // a wait ran out
};

template <bool kE4M3>
struct Warp {
  using S = Stage<kE4M3>;
  const MoeParams& p;
  const Lists& s;
  Team& team;
  const int lane;
  const uint32_t ring, full, empty;           // in shared memory
  int units_a, units_b, units;                // of the first kind, of the first two, of all
  int hidden_units, out_units, shared_units;  // units of a group of either kind; of the shared expert's first kind

  __device__ __forceinline__ Warp(const MoeParams& params, const Lists& lists, Team& t, uint32_t at)
      : p(params), s(lists), team(t), lane(threadIdx.x & 31), ring(at), full(smem_u32(t.full)), empty(smem_u32(t.empty)) {
    hidden_units = (p.m.I + 15) / 16;
    out_units = (p.m.H + 31) / 32;
    shared_units = (p.m.Is + 15) / 16;
    units_a = s.groups[0][s.active] * hidden_units + shared_groups(0) * shared_units;
    units_b = units_a + rows_of_y() * out_units;
    units = units_b + (p.c.T + 7) / 8 * out_units;
  }
  __device__ __forceinline__ int shared_groups(int kind) const {
    return p.m.Is ? (p.c.T + group_of(kind) - 1) / group_of(kind) : 0;
  }
  // the whole warp: the other one, or this, gave up
  __device__ __forceinline__ bool failed() const { return __any_sync(~0u, *(volatile int*)&team.failed); }
  __device__ __forceinline__ int rows_of_y() const { return s.groups[1][s.active] + shared_groups(1); }  // units of 32 columns
  // Units of the groups of an expert that have the same rows follow one another: the second one finds the weights in L2.
  // The shared expert's are first.
  __device__ __forceinline__ Unit unit_of(int u) const {
    Unit n;
    if (u >= units_b) {
      n.kind = 2;
      n.first = (unsigned)(u - units_b) / (unsigned)out_units;
      n.row = (u - units_b - n.first * out_units) * 32;
      n.first *= 8;
      return n;
    }
    n.kind = u >= units_a;
    int v = n.kind ? u - units_a : u, groups = shared_groups(n.kind);
    const int before = groups * (n.kind ? out_units : shared_units);
    n.shared = v < before;
    if (n.shared) {
      n.a = s.active;
    } else {
      const int each = n.kind ? out_units : hidden_units;
      v -= before;
      n.a = s.owner[n.kind][(unsigned)v / (unsigned)each];
      const int g = s.groups[n.kind][n.a];
      groups = s.groups[n.kind][n.a + 1] - g;
      v -= g * each;
    }
    const int row = groups == 1 ? v : (unsigned)v / (unsigned)groups;
    n.row = row * (n.kind ? 32 : 16);
    n.k = !n.kind ? p.m.H : n.shared ? p.m.Is : p.m.I;
    n.first = s.first[n.a] + (v - row * groups) * group_of(n.kind);
    n.count = min(group_of(n.kind), s.first[n.a + 1] - n.first);
    return n;
  }
};

// The warp that loads.
template <bool kE4M3>
struct Loader : Warp<kE4M3> {
  using W = Warp<kE4M3>;
  using S = Stage<kE4M3>;
  using W::lane;
  using W::p;
  using W::s;
  using W::team;
  static constexpr int kPieces = S::kRowBytes / 16;             // of 16 bytes of a row of values
  static constexpr int kStep = 32 / kPieces, kIts = kValueRows / kStep;  // rows at a time
  static_assert(kStep % 2 == 0, "");
  // of the unit that is loaded
  int rows, steps, kind;
  const uint16_t* base;
  const uint4* tops;    // of its slots
  uint32_t from[kIts];  // this lane's piece of its rows of values
  uint32_t to;          // where the first one goes in a stage
  // the next stage to load
  int slot = 0, pass = 0, loaded = 0;
  bool ok = true, hidden_ready = false;

  __device__ __forceinline__ Loader(const MoeParams& params, const Lists& lists, Team& t, uint32_t at)
      : W(params, lists, t, at) {
    // pieces 4 apart are swapped in odd rows: a quarter warp reads 4 pieces of two rows
    const int row = lane / kPieces, piece = lane % kPieces;
    to = kStageBytes + row * S::kRowBytes + ((piece ^ (row & 1) << 2) << 4);
  }
  __device__ __forceinline__ void aim(const Unit& n) {
    kind = n.kind;
    rows = n.count * (kind + 1);
    steps = (n.k + S::kK - 1) / S::kK;
    base = !kind ? p.x : reinterpret_cast<const uint16_t*>(n.shared ? p.shared_hidden : p.hidden);
    const int first = n.first - (n.shared ? s.first[n.a] : 0);
    tops = p.tops + (n.shared ? p.c.T * p.c.top_k : 0) + first;
#pragma unroll
    for (int i = 0; i < kIts; ++i) {
      const int row = min(lane / kPieces + i * kStep, rows - 1);
      from[i] = (kind ? (first + row / 2) * 2 : (int)s.token[n.first + row]) * pad256(n.k) + (kind ? (row & 1) * S::kK : 0) +
                lane % kPieces * 8;
    }
  }
  __device__ __forceinline__ void load_values(uint32_t at, int k, uint32_t bar) {
    const int mine = rows - lane / kPieces;
    if (kE4M3 && kind && k == 0 && lane < rows / 2)
      copy_16(smem_u32(team.tops) + 64 * ((bar - this->full) / 8) + 16 * lane, tops + lane);
    k <<= kind;  // h is twice as long
    if (mine > 0) copy_16(at + to, base + from[0] + k);
    if (rows > kStep) {
#pragma unroll
      for (int i = 1; i < kIts; ++i)
        if (mine > i * kStep) copy_16(at + to + i * kStep * S::kRowBytes, base + from[i] + k);
    }
    copies_done_to(bar);  // the scales too
  }
  __device__ __forceinline__ void fail() {
    if (ok && lane == 0) {
      raise_error(p.c.err, kErrTimeout);
      *(volatile int*)&team.failed = 1;
    }
    ok = false;
  }
  // Every unit of the first kind is in the hands of a team that waits for nothing: h will be there.  Then `late` stages from
  // `at` on, of units from `unit` on, get its values.
  __device__ __forceinline__ void await_hidden(int mine, int late, int at, int unit) {
    for (uint32_t i = 0;; ++i) {
      int done = 0;
      asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(done) : "r"(smem_u32(&team.finished)) : "memory");
      if (__all_sync(~0u, done >= mine)) break;
      if (i == kSpinLimit || this->failed()) return fail();
      __nanosleep(32);
    }
    if (lane == 0 && mine) {
      __threadfence();
      atomicAdd(p.counters + 1, (unsigned)mine);
    }
    if (late == 0) {
      hidden_ready = true;
      return;
    }
    for (uint32_t i = 0;; ++i) {
      const unsigned done = (unsigned)ld_acquire_gpu(reinterpret_cast<const int*>(p.counters + 1));
      if (__all_sync(~0u, done >= (unsigned)this->units_a)) break;
      if (i == kSpinLimit) return fail();
      __nanosleep(32);
    }
    int st = 0;
    for (int i = 0; i < late; ++i) {
      if (i == 0 || st == steps) {
        aim(this->unit_of(team.queue[unit++ % kQueue]));
        st = 0;
      }
      load_values(this->ring + at * S::kBytes, st++ * S::kK, this->full + 8 * at);
      if (++at == kStages) at = 0;
    }
    hidden_ready = true;
  }
  // waits until the next stage may be loaded
  __device__ __forceinline__ void await_place() {
    const uint32_t bar = this->empty + 8 * slot;
    for (uint32_t i = 0; !warp_poll(bar, pass ^ 1); ++i)
      if (i == kWaitLimit || this->failed()) return fail();
  }
  __device__ __forceinline__ void next_stage() {
    if (++slot == kStages) slot = 0, pass ^= 1;
    ++loaded;
  }
  // a stage without anything: the queue has news
  __device__ __forceinline__ void pass_on() {
    if (ok) await_place();
    if (!ok) return;
    __syncwarp();
    const uint32_t bar = this->full + 8 * slot;
    arrive(bar);
    if (lane == 0) arrive(bar);
    next_stage();
  }

  __device__ __forceinline__ void run(unsigned ticket) {
    int mine = 0, late = 0, late_at = 0, late_unit = 0, pushed = 0;
    int next = (int)__shfl_sync(~0u, ticket, 0);
    while (ok && (unsigned)next < (unsigned)this->units) {
      const Unit n = this->unit_of(next);
      if (lane == 0) {
        team.queue[pushed % kQueue] = next;
        ticket = atomicAdd(p.counters, 1u);  // the next unit's number, known later
      }
      if (n.kind == 2) {  // nothing to load
        if (!hidden_ready) await_hidden(mine, late, late_at, late_unit);
        pass_on();
        ++pushed;
        next = (int)__shfl_sync(~0u, ticket, 0);
        continue;
      }
      aim(n);
      const float* scale = nullptr;  // lane 0: of gate, or of down; lane 1: of up, or of down
      if (kE4M3) {
        const int kb = (n.k + kBlock - 1) / kBlock, e = n.shared ? 0 : s.expert[n.a];
        if (n.kind) {
          const int rb = (p.m.H + kBlock - 1) / kBlock;
          scale = (n.shared ? p.m.shared_down_scale : p.m.down_scale) + ((size_t)e * rb + n.row / kBlock) * kb;
        } else {
          const int rb = ((n.shared ? p.m.Is : p.m.I) + kBlock - 1) / kBlock;
          scale = (n.shared ? p.m.shared_gate_up_scale : p.m.gate_up_scale) +
                  (((size_t)e * 2 + (lane & 1)) * rb + n.row / kBlock) * kb;
        }
      }
      const void* map = n.kind ? (n.shared ? &p.shared_down : &p.down) : (n.shared ? &p.shared_gate_up : &p.gate_up);
      const int z = n.shared ? 0 : s.expert[n.a] * (n.kind ? 1 : 2);
      const uint32_t scales = smem_u32(team.scales) + 4 * (lane & 1);
      if (n.kind == 0) ++mine;
      __syncwarp();
#pragma unroll 1
      for (int st = 0; st < steps; ++st) {
        if (kind && !hidden_ready) {
          if (late == kStages) {
            await_hidden(mine, late, late_at, late_unit);
            aim(n);
          } else if (late++ == 0) {
            late_at = slot;
            late_unit = pushed;
          }
        }
        await_place();
        if (!ok) break;
        const uint32_t bar = this->full + 8 * slot, at = this->ring + slot * S::kBytes;
        warp_load(at, map, st * S::kK, n.row, z, bar);
        if (kE4M3 && lane < 2) copy_4(scales + 8 * slot, scale + st);
        if (!kind || hidden_ready) load_values(at, st * S::kK, bar);
        next_stage();
      }
      ++pushed;
      next = (int)__shfl_sync(~0u, ticket, 0);
    }
    if (ok && !hidden_ready) await_hidden(mine, late, late_at, late_unit);
    if (lane == 0) team.queue[pushed % kQueue] = -1;
    pass_on();
    if (ok) return;
    // a wait ran out: copies in flight land before the CTA ends
    for (int i = 0; i < late && !hidden_ready; ++i) copies_done_to(this->full + (late_at + i) % kStages * 8);
    for (int i = 0; i < loaded && i < kStages; ++i) {
      if (slot-- == 0) slot = kStages - 1, pass ^= 1;
      warp_wait(this->full + 8 * slot, pass);
    }
  }
};

// The warp that multiplies.
template <bool kE4M3>
struct Multiplier : Warp<kE4M3> {
  using W = Warp<kE4M3>;
  using S = Stage<kE4M3>;
  using W::lane;
  using W::p;
  using W::s;
  using W::team;
  int worked = 0, now = 0, pass = 0;  // units; the next stage
  int owed = 0, owed_row = 0;         // units of the second kind not yet told; lane i: the row of unit i
  bool ok = true;

  __device__ __forceinline__ Multiplier(const MoeParams& params, const Lists& lists, Team& t, uint32_t at)
      : W(params, lists, t, at) {}

  __device__ __forceinline__ void await_stage() {
    const uint32_t bar = this->full + 8 * now;
    for (uint32_t i = 0; !warp_poll(bar, pass); ++i)
      if (i == kWaitLimit || this->failed()) return fail();
  }
  __device__ __forceinline__ void fail() {
    if (lane == 0) {
      raise_error(p.c.err, kErrTimeout);
      *(volatile int*)&team.failed = 1;
    }
    ok = false;
  }

  // One unit.  With h in two bf16 parts 64 tokens of 288 experts took 556 us so; 575 with a pass of the loop for each chunk,
  // 595 for each half of one; an earlier release of the stage made no difference.
  template <int kKind>
  __device__ __forceinline__ void work(const Unit& n) {
    const int r = lane >> 2, c = lane & 3, steps = (n.k + S::kK - 1) / S::kK;
    constexpr int kSteps = kE4M3 ? 4 : 2;  // products of a chunk
    constexpr int kLoads = kKind == 0 ? kSteps / 2 : kSteps;  // of a lane from its column's values for a chunk, 64 bytes apart
    // rows r and r + 8 of a group of 16: in gate and up, or in down
    constexpr uint32_t apart = kKind == 0 ? 2048 : 1024, group = kKind == 0 ? 1024 : 2048;
    // columns behind the last row of values repeat it, and are not stored
    const int row = min(r, n.count * (kKind + 1) - 1);
    const uint32_t weights = r * 128 + ((2 * c ^ r) << 4);
    const uint32_t values = kStageBytes + c * 16 + (kKind == 0 ? row * S::kRowBytes + (row & 1) * 64 : (row & ~1) * S::kRowBytes);
    const uint32_t odd = r & 1 ? ~0u : 0u;  // the column of the second part
    float by = 1.f, back = 1.f;             // h is multiplied with, and the sums of token c
    const uint32_t scales = smem_u32(team.scales);
    float acc[2][4] = {};
#pragma unroll 1
    for (int st = 0; st < steps; ++st) {
      await_stage();
      if (!ok) break;
      const uint32_t at = this->ring + now * S::kBytes;
      if (kE4M3 && kKind == 1 && st == 0) {
        auto up = [&](int i) {  // the exponent of a power of two that takes the largest h to 2^14 .. 2^15
          const uint4 top = lds128(smem_u32(team.tops) + 64 * now + 16 * i);
          return max(top.x >> 23, 15u) - 14;
        };
        by = __uint_as_float((254 - up(row >> 1)) << 23);
        back = __uint_as_float(up(min(c, n.count - 1)) << 23);
      }
      float part[2][4] = {};
#pragma unroll
      for (uint32_t j = 0; j < 2; ++j) {  // chunks 2 c and 2 c + 1 of the rows, swizzled
        uint4 w[2][2], b[kLoads];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h) w[g][h] = lds128(at + g * group + h * apart + (weights ^ j << 4));
#pragma unroll
        for (int q = 0; q < kLoads; ++q)
          b[q] = lds128(kKind == 0 ? (at + values) ^ (j * kLoads + q) << 6
                                   : ((at + values) ^ q << 6 ^ j << 6) + j * S::kRowBytes);
#pragma unroll
        for (int q = 0; q < kSteps; ++q) {
          uint2 v, third;
          if constexpr (kKind == 0) {
            v = q & 1 ? make_uint2(b[q / 2].z, b[q / 2].w) : make_uint2(b[q / 2].x, b[q / 2].y);
          } else {
            const float4 h = make_float4(__uint_as_float(b[q].x), __uint_as_float(b[q].y), __uint_as_float(b[q].z),
                                         __uint_as_float(b[q].w));
            v = kE4M3 ? half_parts(h, by, odd) : bf16_parts(h, odd, third);
          }
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint2 a[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t u[4] = {w[g][h].x, w[g][h].y, w[g][h].z, w[g][h].w};
              if constexpr (kE4M3) a[h] = e4m3x4_to_half4(u[q]);
              else a[h] = make_uint2(u[2 * q], u[2 * q + 1]);
            }
            mma_16816<kE4M3>(part[g], a[0], a[1], v.x, v.y);
            if constexpr (!kE4M3 && kKind == 1) mma_16816<false>(part[g], a[0], a[1], third.x, third.y);
          }
        }
      }
      // a block of k is summed by itself, then scaled
      const float2 scale = kE4M3 ? lds_f32x2(scales + 8 * now) : make_float2(1.f, 1.f);
      __syncwarp();
      first_arrive(this->empty + 8 * now);
      if (++now == kStages) now = 0, pass ^= 1;
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[g][i] = fmaf(part[g][i], i < 2 ? scale.x : scale.y, acc[g][i]);
    }
    if (!ok) return;
    const int rows = kKind == 1 ? p.m.H : n.shared ? p.m.Is : p.m.I;
    uint32_t top[2] = {0, 0};  // of tokens 2 c and the next
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int row = n.row + g * (kKind == 0 ? 8 : 16);
      if (row < rows) finish<kKind>(n, row, acc[g], back, top);
    }
    if constexpr (kE4M3 && kKind == 0) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < 2; ++j) top[j] = max(top[j], __shfl_xor_sync(~0u, top[j], o));
      uint4* tops = p.tops + (n.shared ? p.c.T * p.c.top_k - s.first[n.a] : 0) + n.first + 2 * c;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (r == 0 && 2 * c + j < n.count) atomicMax(&tops[j].x, top[j]);
    }
    __syncwarp();
    if (kKind == 0) {  // the other warp makes it known
      if (lane == 0)
        asm volatile("red.release.cta.shared.add.u32 [%0], 1;" ::"r"(smem_u32(&team.finished)) : "memory");
    } else {
      if (lane == owed) owed_row = n.row;
      ++owed;
    }
  }
  // what comes of a group of 16 rows' sums
  template <int kKind>
  __device__ __forceinline__ void finish(const Unit& n, int row, const float (&acc)[4], float back, uint32_t (&top)[2]) {
    const int r = lane >> 2, c = lane & 3;
    if constexpr (kKind == 0) {  // silu(gate) * up for place row + r, tokens 2 c and the next
      float* hidden = n.shared ? p.shared_hidden : p.hidden;
      const int first = n.first - (n.shared ? s.first[n.a] : 0), wide = pad256(n.shared ? p.m.Is : p.m.I);
      const int at = hidden_place<kE4M3>(row + r);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int rank = 2 * c + j;
        if (rank >= n.count) continue;
        const float xs = kE4M3 ? s.x_scale[s.token[n.first + rank]] : 1.f, g = acc[j] * xs, u = acc[2 + j] * xs;
        const float h = g / (1.f + expf(-g)) * u;
        hidden[(size_t)(first + rank) * wide + at] = h;
        const uint32_t size = __float_as_uint(h) & 0x7FFFFFFFu;
        if (size < 0x7F800000u) top[j] = max(top[j], size);
      }
    } else if (c < n.count) {  // rows row + r and row + 8 + r: the products with the two parts of token c's h
      float* y = p.y + (size_t)(n.first + c) * p.m.H + row + r;
      const float w = s.weight[n.first + c];
      y[0] = (acc[0] + acc[1]) * back * w;
      y[8] = (acc[2] + acc[3]) * back * w;
    }
  }

  // A fence waits for the stores before it: what units wrote is made known several units at a time.
  static constexpr int kOwed = 4;
  __device__ __forceinline__ void tell_rows() {
    __syncwarp();
    if (lane < owed) {
      __threadfence();
      atomicAdd(p.counters + 2 + owed_row / 32, 1u);
    }
    owed = 0;
  }

  // 32 columns of the output for 8 tokens, from the experts' rows in the order of the choice
  __device__ __forceinline__ void join(const Unit& n) {
    const int* done = reinterpret_cast<const int*>(p.counters + 2 + n.row / 32);
    for (uint32_t i = 0; !__all_sync(~0u, ld_acquire_gpu(done) >= this->rows_of_y()); ++i) {
      if (i == kSpinLimit) return fail();
      __nanosleep(32);
    }
    const int col = n.row + (lane & 7) * 4;
    if (col >= p.m.H) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = n.first + i * 4 + (lane >> 3);
      if (t >= p.c.T) break;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 6
      for (int j = 0; j <= p.c.top_k; ++j) {
        const int slot = s.slot_of[t][j == p.c.top_k ? kMaxTopK : j];
        if (slot == kNone) continue;
        const float4 v = ld_l2(reinterpret_cast<const float4*>(p.y + (size_t)slot * p.m.H + col));
        y.x += v.x;
        y.y += v.y;
        y.z += v.z;
        y.w += v.w;
      }
      *reinterpret_cast<uint2*>(p.c.out + (size_t)t * p.m.H + col) = make_uint2(pack_bf2(y.x, y.y), pack_bf2(y.z, y.w));
    }
  }

  __device__ __forceinline__ void run() {
    for (;; ++worked) {
      await_stage();
      if (!ok) return;
      const int u = team.queue[worked % kQueue];
      if (u < 0) break;
      const Unit n = this->unit_of(u);
      if (n.kind == 2) {
        __syncwarp();
        first_arrive(this->empty + 8 * now);
        if (++now == kStages) now = 0, pass ^= 1;
        tell_rows();
        join(n);
      } else if (n.kind == 0) {
        work<0>(n);
      } else {
        work<1>(n);
      }
      if (!ok) return;
      if (owed == kOwed) tell_rows();
    }
    tell_rows();
  }
};

struct Shared {  // behind the teams' stages
  Lists lists;
  Team team[kTeams];
};
template <bool kE4M3>
constexpr size_t smem_of() {
  return 1024 + (size_t)kTeams * Stage<kE4M3>::kBytes * kStages + sizeof(Shared);
}
static_assert(smem_of<true>() <= 232448 && smem_of<false>() <= 232448, "");
static_assert(sizeof(Choice) <= kTeams * kStages * Stage<false>::kBytes && kStages + 2 <= kQueue, "");

// 512 threads have 128 registers each, and 16 (bf16) or 20 bytes of a thread's are spilled.
template <bool kE4M3>
__global__ void __launch_bounds__(kThreads, 1) experts_kernel(const __grid_constant__ MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  Shared& shared = *reinterpret_cast<Shared*>(smem + kTeams * Stage<kE4M3>::kBytes * kStages);
  Lists& s = shared.lists;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = warp % kTeams;
  if (threadIdx.x == 0) {
    prefetch_tensormap(&p.gate_up);
    prefetch_tensormap(&p.down);
  }
  await_grid();
  unsigned ticket = 0;
  // Where there are fewer units than teams they are spread over the SMs: a CTA's first team takes one first, the last four when
  // the lists are there.
  auto take = [&](int first, int last) {
    if (warp >= first && warp < last && lane == 0) ticket = atomicAdd(p.counters, 1u);
  };
  Choice& choice = *reinterpret_cast<Choice*>(smem);  // where the stages will be
  take(0, 1);
  make_choice(p, choice, s);
  take(1, 4);
  make_lists(p, choice, s);
  take(4, kTeams);
  if (s.active == 0 && p.m.Is == 0) {  // no token has an expert
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < p.c.T * p.m.H / 8; i += gridDim.x * kThreads)
      reinterpret_cast<uint4*>(p.c.out)[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  Team& team = shared.team[mine];
  if (warp < kTeams && lane < kStages) {
    mbar_init(smem_u32(team.full + lane), 33);  // the weights; every lane's copies
    mbar_init(smem_u32(team.empty + lane), 1);
    if (lane == 0) team.finished = team.failed = 0;
  }
  fence_mbar_init();
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // copies come where the choice was
  __syncthreads();
  const uint32_t ring = smem_u32(smem + mine * Stage<kE4M3>::kBytes * kStages);
  if (warp < kTeams) {
    Loader<kE4M3> loader(p, s, team, ring);
    loader.run(ticket);
  } else {
    Multiplier<kE4M3> worker(p, s, team, ring);
    worker.run();
  }
}

template <bool kE4M3>
cudaError_t encode(CUtensorMap* map, const void* base, int k, int rows, int matrices, bool halves) {
  if (!base || !rows || !k) return cudaSuccess;
  return kE4M3 ? encode_u8_3d_sw128(map, base, k, rows, matrices, 128, halves ? 16 : 32, halves ? 2 : 1)
               : encode_bf16_3d_sw128(map, base, k, rows, matrices, 64, halves ? 16 : 32, halves ? 2 : 1);
}

template <bool kE4M3>
cudaError_t launch(const LaunchEnv& env, MoeParams& p) {
  static int done[64] = {0};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(experts_kernel<kE4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of<kE4M3>());
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev] = 1;
  }
  const Moe& m = p.m;
  e = encode<kE4M3>(&p.gate_up, m.gate_up, m.H, m.I, 2 * m.E, true);
  if (e == cudaSuccess) e = encode<kE4M3>(&p.down, m.down, m.I, m.H, m.E, false);
  if (e == cudaSuccess) e = encode<kE4M3>(&p.shared_gate_up, m.Is ? m.shared_gate_up : nullptr, m.H, m.Is, 2, true);
  if (e == cudaSuccess) e = encode<kE4M3>(&p.shared_down, m.Is ? m.shared_down : nullptr, m.Is, m.H, 1, false);
  if (e != cudaSuccess) return e;
  const int rows = (p.c.ids_in ? 0 : m.E) + (m.shared_gate ? 1 : 0), dots = (rows + kRows - 1) / kRows * ((p.c.T + 7) / 8);
  e = launch_early(prepare_kernel<kE4M3>, dim3(p.c.T + dots), kPrepareThreads, 0, env.stream, p);
  p.chosen = !p.c.ids_in && p.c.T > kWarps;  // more tokens than a CTA has warps
  if (e == cudaSuccess && p.chosen)
    e = launch_early(choose_kernel, dim3((p.c.T + kChooseWarps - 1) / kChooseWarps), kChooseWarps * 32, 0, env.stream, p);
  if (e != cudaSuccess) return e;
  return launch_early(experts_kernel<kE4M3>, dim3(sms), kThreads, smem_of<kE4M3>(), env.stream, p);
}

}  // namespace

size_t moe_workspace_bytes(const Moe& m, int T, int top_k) { return layout(m, T, top_k).bytes; }

cudaError_t launch_moe(const LaunchEnv& env, const Moe& m, MoeCall c, void* workspace) {
  MoeParams p;
  memset(&p, 0, sizeof p);
  c.err = env.err;
  p.m = m;
  p.c = c;
  const Layout l = layout(m, c.T, c.top_k);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.counters = reinterpret_cast<unsigned*>(ws + l.counters);
  p.logits = reinterpret_cast<float*>(ws + l.logits);
  p.ids = reinterpret_cast<int32_t*>(ws + l.ids);
  p.weights = reinterpret_cast<float*>(ws + l.weights);
  p.x = reinterpret_cast<uint16_t*>(ws + l.x);
  p.x_scale = reinterpret_cast<float*>(ws + l.x_scale);
  p.tops = reinterpret_cast<uint4*>(ws + l.tops);
  p.hidden = reinterpret_cast<float*>(ws + l.hidden);
  p.shared_hidden = reinterpret_cast<float*>(ws + l.shared_hidden);
  p.y = reinterpret_cast<float*>(ws + l.y);
  return m.gate_up_scale ? launch<true>(env, p) : launch<false>(env, p);
}

}  // namespace gdn
