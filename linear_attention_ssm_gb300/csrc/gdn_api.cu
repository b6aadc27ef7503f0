// gdn_api.cu -- the C ABI of libgdn.so: host-side validation, then one launch per call.
//
// Every entry point checks its arguments on the host before it launches anything; a call that
// returns an error has launched nothing.  Device-side faults (bad cu_seqlens contents, a bounded
// wait that ran out) set bits in a per-device error word that gdn_check_device_errors() reads.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <string>

#include "../../include/gdn.h"
#ifdef GDN_TEST_HOOKS
#include "../../include/gdn_debug.h"
#endif
#include "gdn_common.cuh"
#include "gdn_kernels.h"

namespace {

__device__ unsigned g_gdn_error_word;

thread_local std::string g_last_error;
#ifdef GDN_TEST_HOOKS
std::atomic<int> g_chunk_mode{0};  // the test library's chunk-design selection (gdn_debug.h)
#else
constexpr int g_chunk_mode = 0;    // the product library always takes the default design
#endif

constexpr int kMaxDevices = 64;
// Device address of the error word, per device index, looked up on the first call that needs it.
// Two host threads making their first call at once both store the same address.
std::atomic<unsigned*> g_err_ptr[kMaxDevices] = {};

gdn_status fail(gdn_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gdn_status fail(gdn_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

gdn_status ok() {
  g_last_error.clear();
  return GDN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

gdn_status check_geometry(const gdn_geometry* geo) {
  if (!geo) return fail(GDN_ERR_INVALID_ARGUMENT, "geometry is NULL");
  if (geo->num_k_heads <= 0 || geo->num_v_heads <= 0 || geo->num_v_heads % geo->num_k_heads != 0)
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "num_v_heads (%d) must be a positive multiple of num_k_heads (%d)",
                geo->num_v_heads, geo->num_k_heads);
  if (geo->head_k_dim != gdn::kHeadDim || geo->head_v_dim != gdn::kHeadDim)
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "head dims must be %d (got Dk=%d, Dv=%d)", gdn::kHeadDim,
                geo->head_k_dim, geo->head_v_dim);
  if (geo->conv_width != gdn::kConvWidth)
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "conv width must be %d (got %d)", gdn::kConvWidth, geo->conv_width);
  if (geo->num_k_heads > 64 || geo->num_v_heads > 192)
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "at most 64 K heads and 192 V heads (got %d, %d)", geo->num_k_heads,
                geo->num_v_heads);
  return GDN_OK;
}

int conv_channels(const gdn_geometry* g) {
  return 2 * g->num_k_heads * g->head_k_dim + g->num_v_heads * g->head_v_dim;
}

#define GDN_REQUIRE(ptr, name)                                                            \
  do {                                                                                    \
    if (!(ptr)) return fail(GDN_ERR_INVALID_ARGUMENT, "%s is NULL", name);                \
    if (!aligned16(ptr)) return fail(GDN_ERR_MISALIGNED, "%s is not 16-byte aligned", name); \
  } while (0)
#define GDN_OPTIONAL(ptr, name)                                                           \
  do {                                                                                    \
    if ((ptr) && !aligned16(ptr)) return fail(GDN_ERR_MISALIGNED, "%s is not 16-byte aligned", name); \
  } while (0)

gdn_status make_env(void* stream, gdn::LaunchEnv* env) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(GDN_ERR_CUDA, "device index %d out of range", dev);
  unsigned* err = g_err_ptr[dev].load(std::memory_order_acquire);
  if (!err) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_gdn_error_word);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaGetSymbolAddress: %s", cudaGetErrorString(e));
    err = static_cast<unsigned*>(p);
    g_err_ptr[dev].store(err, std::memory_order_release);
  }
  env->err = err;
  env->num_sms = 0;
  env->stream = static_cast<cudaStream_t>(stream);
  return GDN_OK;
}

gdn_status launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

const char* gdn_status_string(gdn_status s) {
  switch (s) {
    case GDN_OK: return "GDN_OK";
    case GDN_ERR_INVALID_ARGUMENT: return "GDN_ERR_INVALID_ARGUMENT";
    case GDN_ERR_UNSUPPORTED_GEOMETRY: return "GDN_ERR_UNSUPPORTED_GEOMETRY";
    case GDN_ERR_MISALIGNED: return "GDN_ERR_MISALIGNED";
    case GDN_ERR_CUDA: return "GDN_ERR_CUDA";
    case GDN_ERR_TIMEOUT: return "GDN_ERR_TIMEOUT";
    case GDN_ERR_DEVICE_ARGUMENT: return "GDN_ERR_DEVICE_ARGUMENT";
    case GDN_ERR_WORKSPACE: return "GDN_ERR_WORKSPACE";
  }
  return "GDN_ERR_UNKNOWN";
}

const char* gdn_last_error_message(void) { return g_last_error.c_str(); }

const char* gdn_version(void) { return "gdn-gb300 0.1 (sm_103a)"; }

gdn_status gdn_conv1d_prefill(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w,
                              const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                              const gdn_bf16* conv_state_in, gdn_bf16* conv_state_out, gdn_bf16* y, void* stream) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (num_seqs < 0 || total_tokens < 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "negative size (num_seqs=%d, total_tokens=%d)", num_seqs, total_tokens);
  if (num_seqs == 0 && total_tokens > 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "total_tokens=%d with no sequence", total_tokens);
  if (num_seqs == 0) return ok();
  GDN_REQUIRE(conv_w, "conv_w");
  if (!cu_seqlens) return fail(GDN_ERR_INVALID_ARGUMENT, "cu_seqlens is NULL");
  if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) return fail(GDN_ERR_MISALIGNED, "cu_seqlens is not 4-byte aligned");
  GDN_OPTIONAL(conv_state_in, "conv_state_in");
  GDN_OPTIONAL(conv_state_out, "conv_state_out");
  const int C = conv_channels(geo);
  if (total_tokens > 0) {
    GDN_REQUIRE(x, "x");
    GDN_REQUIRE(y, "y");
    const size_t bytes = (size_t)total_tokens * C * 2;
    if (overlaps(x, bytes, y, bytes)) return fail(GDN_ERR_INVALID_ARGUMENT, "y overlaps x");
  } else if (!conv_state_out) {
    return ok();
  }
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_conv1d_prefill(env, x, conv_w, cu_seqlens, num_seqs, total_tokens, C, conv_state_in,
                                             conv_state_out, y),
                  "conv1d launch");
}

size_t gdn_chunk_prefill_workspace_size(const gdn_geometry* geo, int32_t num_seqs, int32_t total_tokens) {
  if (!geo || num_seqs <= 0 || total_tokens < 0 || geo->num_k_heads <= 0 || geo->num_v_heads <= 0) return 0;
  return gdn::split_workspace_bytes(num_seqs, total_tokens, geo->num_k_heads, geo->num_v_heads);
}

size_t gdn_chunk_prefill_min_workspace_size(const gdn_geometry* geo, int32_t num_seqs, int32_t total_tokens) {
  (void)geo;
  (void)total_tokens;
  return num_seqs > 0 ? gdn::chunk_prefill_workspace_bytes(num_seqs) : 0;
}

}  // extern "C"

namespace {
// The gate inputs of a call: g and beta, or the projections a, b with A_log and dt_bias.
gdn_status check_gates(const gdn::GateSrc& gs) {
  if (gs.a) {
    if (!gs.b || !gs.A_log || !gs.dt_bias) return fail(GDN_ERR_INVALID_ARGUMENT, "a, b, A_log or dt_bias is NULL");
    if ((reinterpret_cast<uintptr_t>(gs.a) | reinterpret_cast<uintptr_t>(gs.b)) & 1u)
      return fail(GDN_ERR_MISALIGNED, "a or b is not 2-byte aligned");
    if ((reinterpret_cast<uintptr_t>(gs.A_log) | reinterpret_cast<uintptr_t>(gs.dt_bias)) & 3u)
      return fail(GDN_ERR_MISALIGNED, "A_log or dt_bias is not 4-byte aligned");
    return GDN_OK;
  }
  if (!gs.g || !gs.beta) return fail(GDN_ERR_INVALID_ARGUMENT, "g or beta is NULL");
  if ((reinterpret_cast<uintptr_t>(gs.g) | reinterpret_cast<uintptr_t>(gs.beta)) & 3u)
    return fail(GDN_ERR_MISALIGNED, "g or beta is not 4-byte aligned");
  return GDN_OK;
}

// The conv stage that gdn_prefill runs ahead of the chunk prefill (its output is the chunk stage's qkv).
struct ConvStage {
  const gdn_bf16* x;
  const gdn_bf16* w;
  const gdn_bf16* state_in;
  gdn_bf16* state_out;
  int C;
};

gdn_status chunk_prefill(const gdn_geometry* geo, const gdn_bf16* qkv, const gdn::GateSrc& gates,
                         const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens, float q_scale,
                         float l2_eps, const float* state_in, float* state_out, const gdn_bf16* z,
                         const gdn_bf16* norm_w, float rms_eps, gdn_bf16* out, void* workspace,
                         size_t workspace_bytes, void* stream, const ConvStage* conv = nullptr) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (num_seqs < 0 || total_tokens < 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "negative size (num_seqs=%d, total_tokens=%d)", num_seqs, total_tokens);
  if (num_seqs == 0 && total_tokens > 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "total_tokens=%d with no sequence", total_tokens);
  if ((long)num_seqs * geo->num_v_heads > 0x7FFFFFFFL)
    return fail(GDN_ERR_INVALID_ARGUMENT, "num_seqs * num_v_heads exceeds the grid limit");
  if (num_seqs == 0) return ok();
  if (!cu_seqlens) return fail(GDN_ERR_INVALID_ARGUMENT, "cu_seqlens is NULL");
  if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) return fail(GDN_ERR_MISALIGNED, "cu_seqlens is not 4-byte aligned");
  if (total_tokens > 0) {
    GDN_REQUIRE(qkv, "qkv");
    GDN_REQUIRE(out, "out");
    if ((s = check_gates(gates)) != GDN_OK) return s;
  }
  GDN_OPTIONAL(state_in, "state_in");
  GDN_OPTIONAL(state_out, "state_out");
  if (z) {
    GDN_REQUIRE(z, "z");
    GDN_REQUIRE(norm_w, "norm_w");
  }
  if (!(l2_eps >= 0.f) || !(rms_eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  const size_t need = gdn_chunk_prefill_min_workspace_size(geo, num_seqs, total_tokens);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes required (got %zu)", need, workspace_bytes);
  if (workspace && (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(GDN_ERR_MISALIGNED, "workspace is not 256-byte aligned");
  if (state_in && state_out && state_in != state_out) {
    const size_t sb = (size_t)num_seqs * geo->num_v_heads * gdn::kHeadDim * gdn::kHeadDim * 4;
    if (overlaps(state_in, sb, state_out, sb))
      return fail(GDN_ERR_INVALID_ARGUMENT, "state_out partially overlaps state_in");
  }
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  if (conv && (total_tokens > 0 || conv->state_out)) {  // every argument checked: the conv stage first
    s = launched(gdn::launch_conv1d_prefill(env, conv->x, conv->w, cu_seqlens, num_seqs, total_tokens, conv->C,
                                            conv->state_in, conv->state_out, const_cast<gdn_bf16*>(qkv)),
                 "conv1d launch");
    if (s != GDN_OK) return s;
  }
  return launched(gdn::launch_chunk_prefill(env, g_chunk_mode, qkv, gates, cu_seqlens, num_seqs, total_tokens,
                                            geo->num_k_heads, geo->num_v_heads, q_scale, l2_eps, state_in,
                                            state_out, z, norm_w, rms_eps, out, workspace, workspace_bytes),
                  "chunk prefill launch");
}
}  // namespace

extern "C" {

gdn_status gdn_chunk_prefill(const gdn_geometry* geo, const gdn_bf16* qkv, const float* g, const float* beta,
                             const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens, float q_scale,
                             float l2_eps, const float* state_in, float* state_out, const gdn_bf16* z,
                             const gdn_bf16* norm_w, float rms_eps, gdn_bf16* out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const gdn::GateSrc gates = {g, beta, nullptr, nullptr, nullptr, nullptr};
  return chunk_prefill(geo, qkv, gates, cu_seqlens, num_seqs, total_tokens, q_scale, l2_eps, state_in, state_out, z,
                       norm_w, rms_eps, out, workspace, workspace_bytes, stream);
}

gdn_status gdn_prefill(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w, const int32_t* cu_seqlens,
                       int32_t num_seqs, int32_t total_tokens, const gdn_bf16* conv_state_in,
                       gdn_bf16* conv_state_out, gdn_bf16* qkv, const float* g, const float* beta, float q_scale,
                       float l2_eps, const float* state_in, float* state_out, const gdn_bf16* z,
                       const gdn_bf16* norm_w, float rms_eps, gdn_bf16* out, void* workspace, size_t workspace_bytes,
                       void* stream) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (num_seqs > 0) {  // the conv stage's own arguments (the chunk stage checks the rest)
    GDN_REQUIRE(conv_w, "conv_w");
    GDN_OPTIONAL(conv_state_in, "conv_state_in");
    GDN_OPTIONAL(conv_state_out, "conv_state_out");
    if (total_tokens > 0) {
      GDN_REQUIRE(x, "x");
      GDN_REQUIRE(qkv, "qkv");
      const size_t bytes = (size_t)total_tokens * conv_channels(geo) * 2;
      if (overlaps(x, bytes, qkv, bytes)) return fail(GDN_ERR_INVALID_ARGUMENT, "qkv overlaps x");
    }
  }
  const gdn::GateSrc gates = {g, beta, nullptr, nullptr, nullptr, nullptr};
  const ConvStage conv = {x, conv_w, conv_state_in, conv_state_out, conv_channels(geo)};
  return chunk_prefill(geo, qkv, gates, cu_seqlens, num_seqs, total_tokens, q_scale, l2_eps, state_in, state_out, z,
                       norm_w, rms_eps, out, workspace, workspace_bytes, stream, &conv);
}

gdn_status gdn_chunk_prefill_fused_gates(const gdn_geometry* geo, const gdn_bf16* qkv, const gdn_bf16* a,
                                         const gdn_bf16* b, const float* A_log, const float* dt_bias,
                                         const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                                         float q_scale, float l2_eps, const float* state_in, float* state_out,
                                         const gdn_bf16* z, const gdn_bf16* norm_w, float rms_eps, gdn_bf16* out,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!a) return fail(GDN_ERR_INVALID_ARGUMENT, "a is NULL");
  const gdn::GateSrc gates = {nullptr, nullptr, a, b, A_log, dt_bias};
  return chunk_prefill(geo, qkv, gates, cu_seqlens, num_seqs, total_tokens, q_scale, l2_eps, state_in, state_out, z,
                       norm_w, rms_eps, out, workspace, workspace_bytes, stream);
}

gdn_status gdn_gated_rmsnorm(const gdn_geometry* geo, const gdn_bf16* o, const gdn_bf16* z, const gdn_bf16* norm_w,
                             float eps, gdn_bf16* out, int32_t total_tokens, void* stream) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (total_tokens < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "negative total_tokens");
  if (total_tokens == 0) return ok();
  GDN_REQUIRE(o, "o");
  GDN_REQUIRE(z, "z");
  GDN_REQUIRE(norm_w, "norm_w");
  GDN_REQUIRE(out, "out");
  if (!(eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_gated_rmsnorm(env, o, z, norm_w, eps, out, (long)total_tokens * geo->num_v_heads),
                  "gated rmsnorm launch");
}

}  // extern "C"

namespace {
gdn_status decode_step(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w, gdn_bf16* conv_state,
                       const gdn::GateSrc& gates, void* state, bool fp16_state, const gdn_bf16* z,
                       const gdn_bf16* norm_w, float q_scale, float l2_eps, float rms_eps, gdn_bf16* out,
                       int32_t batch, void* stream) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (geo->num_v_heads / geo->num_k_heads > gdn::decode_max_ratio())
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "decode supports at most %d V heads per K head",
                gdn::decode_max_ratio());
  if (batch < 0 || batch > 65535) return fail(GDN_ERR_INVALID_ARGUMENT, "batch must be in [0, 65535] (got %d)", batch);
  if (batch == 0) return ok();
  GDN_REQUIRE(x, "x");
  GDN_REQUIRE(conv_w, "conv_w");
  GDN_REQUIRE(conv_state, "conv_state");
  GDN_REQUIRE(state, "state");
  GDN_REQUIRE(z, "z");
  GDN_REQUIRE(norm_w, "norm_w");
  GDN_REQUIRE(out, "out");
  if ((s = check_gates(gates)) != GDN_OK) return s;
  if (!(l2_eps >= 0.f) || !(rms_eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_decode_step(env, x, conv_w, conv_state, gates, state, fp16_state, z, norm_w,
                                          q_scale, l2_eps, rms_eps, out, batch, geo->num_k_heads,
                                          geo->num_v_heads),
                  "decode launch");
}
}  // namespace

extern "C" {

gdn_status gdn_decode_step(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w, gdn_bf16* conv_state,
                           const float* g, const float* beta, float* state, const gdn_bf16* z,
                           const gdn_bf16* norm_w, float q_scale, float l2_eps, float rms_eps, gdn_bf16* out,
                           int32_t batch, void* stream) {
  const gdn::GateSrc gates = {g, beta, nullptr, nullptr, nullptr, nullptr};
  return decode_step(geo, x, conv_w, conv_state, gates, state, false, z, norm_w, q_scale, l2_eps, rms_eps, out,
                     batch, stream);
}

gdn_status gdn_decode_step_fused_gates(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w,
                                       gdn_bf16* conv_state, const gdn_bf16* a, const gdn_bf16* b, const float* A_log,
                                       const float* dt_bias, float* state, const gdn_bf16* z, const gdn_bf16* norm_w,
                                       float q_scale, float l2_eps, float rms_eps, gdn_bf16* out, int32_t batch,
                                       void* stream) {
  if (batch > 0 && !a) return fail(GDN_ERR_INVALID_ARGUMENT, "a is NULL");
  const gdn::GateSrc gates = {nullptr, nullptr, a, b, A_log, dt_bias};
  return decode_step(geo, x, conv_w, conv_state, gates, state, false, z, norm_w, q_scale, l2_eps, rms_eps, out,
                     batch, stream);
}

gdn_status gdn_kda_decode_step(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w,
                               gdn_bf16* conv_state, const float* g, float g_min, const float* beta, float* state,
                               const gdn_bf16* z, const gdn_bf16* norm_w, float q_scale, float l2_eps,
                               float rms_eps, gdn_bf16* out, int32_t batch, void* stream) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (geo->num_v_heads / geo->num_k_heads > gdn::decode_max_ratio())
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "decode supports at most %d V heads per K head",
                gdn::decode_max_ratio());
  if (batch < 0 || batch > 65535) return fail(GDN_ERR_INVALID_ARGUMENT, "batch must be in [0, 65535] (got %d)", batch);
  if (batch == 0) return ok();
  GDN_REQUIRE(x, "x");
  GDN_REQUIRE(conv_w, "conv_w");
  GDN_REQUIRE(conv_state, "conv_state");
  GDN_REQUIRE(g, "g");
  GDN_REQUIRE(state, "state");
  GDN_REQUIRE(z, "z");
  GDN_REQUIRE(norm_w, "norm_w");
  GDN_REQUIRE(out, "out");
  if (!beta) return fail(GDN_ERR_INVALID_ARGUMENT, "beta is NULL");
  if (reinterpret_cast<uintptr_t>(beta) & 3u) return fail(GDN_ERR_MISALIGNED, "beta is not 4-byte aligned");
  if (g_min != g_min) return fail(GDN_ERR_INVALID_ARGUMENT, "g_min is NaN");
  if (!(l2_eps >= 0.f) || !(rms_eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_kda_decode_step(env, x, conv_w, conv_state, g, g_min, beta, state, z, norm_w, q_scale,
                                              l2_eps, rms_eps, out, batch, geo->num_k_heads, geo->num_v_heads),
                  "KDA decode launch");
}

gdn_status gdn_kda_recurrence(const gdn_geometry* geo, const gdn_bf16* qkv, const float* g, float g_min,
                              const float* beta, const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                              float q_scale, float l2_eps, const float* state_in, float* state_out, const gdn_bf16* z,
                              const gdn_bf16* norm_w, float rms_eps, gdn_bf16* out, void* stream) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (num_seqs < 0 || total_tokens < 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "negative size (num_seqs=%d, total_tokens=%d)", num_seqs, total_tokens);
  if (num_seqs == 0 && total_tokens > 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "total_tokens=%d with no sequence", total_tokens);
  if (num_seqs > 65535) return fail(GDN_ERR_INVALID_ARGUMENT, "num_seqs must be at most 65535 (got %d)", num_seqs);
  if (num_seqs == 0) return ok();
  if (!cu_seqlens) return fail(GDN_ERR_INVALID_ARGUMENT, "cu_seqlens is NULL");
  if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) return fail(GDN_ERR_MISALIGNED, "cu_seqlens is not 4-byte aligned");
  if (total_tokens > 0) {
    GDN_REQUIRE(qkv, "qkv");
    GDN_REQUIRE(g, "g");
    GDN_REQUIRE(out, "out");
    if (!beta) return fail(GDN_ERR_INVALID_ARGUMENT, "beta is NULL");
    if (reinterpret_cast<uintptr_t>(beta) & 3u) return fail(GDN_ERR_MISALIGNED, "beta is not 4-byte aligned");
  }
  GDN_OPTIONAL(state_in, "state_in");
  GDN_OPTIONAL(state_out, "state_out");
  if (z) {
    GDN_REQUIRE(z, "z");
    GDN_REQUIRE(norm_w, "norm_w");
  }
  if (g_min != g_min) return fail(GDN_ERR_INVALID_ARGUMENT, "g_min is NaN");
  if (!(l2_eps >= 0.f) || !(rms_eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  if (state_in && state_out && state_in != state_out) {
    const size_t sb = (size_t)num_seqs * geo->num_v_heads * gdn::kHeadDim * gdn::kHeadDim * 4;
    if (overlaps(state_in, sb, state_out, sb))
      return fail(GDN_ERR_INVALID_ARGUMENT, "state_out partially overlaps state_in");
  }
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_kda_prefill(env, qkv, g, g_min, beta, cu_seqlens, num_seqs, total_tokens,
                                          geo->num_k_heads, geo->num_v_heads, q_scale, l2_eps, state_in, state_out,
                                          z, norm_w, rms_eps, out),
                  "KDA recurrence launch");
}

size_t gdn_kda_chunk_prefill_workspace_size(const gdn_geometry* geo, int32_t num_seqs, int32_t total_tokens) {
  if (!geo || num_seqs <= 0 || total_tokens < 0 || geo->num_v_heads <= 0) return 0;
  return gdn::kda_chunk_workspace_bytes(num_seqs, total_tokens, geo->num_v_heads);
}

static gdn_status kda_chunk_prefill(const gdn_geometry* geo, const gdn_bf16* qkv, const float* g, float g_min,
                                 const float* beta, const int32_t* cu_seqlens, int32_t num_seqs,
                                 int32_t total_tokens, float q_scale, float l2_eps, const float* state_in,
                                 float* state_out, const gdn_bf16* z, const gdn_bf16* norm_w, float rms_eps,
                                 gdn_bf16* out, void* workspace, size_t workspace_bytes, void* stream,
                                 const ConvStage* conv = nullptr) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (num_seqs < 0 || total_tokens < 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "negative size (num_seqs=%d, total_tokens=%d)", num_seqs, total_tokens);
  if (num_seqs == 0 && total_tokens > 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "total_tokens=%d with no sequence", total_tokens);
  if ((long)num_seqs * geo->num_v_heads > 0x7FFFFFFFL)
    return fail(GDN_ERR_INVALID_ARGUMENT, "num_seqs * num_v_heads exceeds the grid limit");
  if (num_seqs == 0) return ok();
  if (!cu_seqlens) return fail(GDN_ERR_INVALID_ARGUMENT, "cu_seqlens is NULL");
  if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) return fail(GDN_ERR_MISALIGNED, "cu_seqlens is not 4-byte aligned");
  if (total_tokens > 0) {
    GDN_REQUIRE(qkv, "qkv");
    GDN_REQUIRE(g, "g");
    GDN_REQUIRE(out, "out");
    if (!beta) return fail(GDN_ERR_INVALID_ARGUMENT, "beta is NULL");
    if (reinterpret_cast<uintptr_t>(beta) & 3u) return fail(GDN_ERR_MISALIGNED, "beta is not 4-byte aligned");
  }
  GDN_OPTIONAL(state_in, "state_in");
  GDN_OPTIONAL(state_out, "state_out");
  if (z) {
    GDN_REQUIRE(z, "z");
    GDN_REQUIRE(norm_w, "norm_w");
  }
  if (g_min != g_min) return fail(GDN_ERR_INVALID_ARGUMENT, "g_min is NaN");
  if (!(l2_eps >= 0.f) || !(rms_eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  const size_t need = gdn_kda_chunk_prefill_workspace_size(geo, num_seqs, total_tokens);
  if (!workspace || workspace_bytes < need)
    return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes required (got %zu)", need, workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return fail(GDN_ERR_MISALIGNED, "workspace is not 256-byte aligned");
  if (state_in && state_out && state_in != state_out) {
    const size_t sb = (size_t)num_seqs * geo->num_v_heads * gdn::kHeadDim * gdn::kHeadDim * 4;
    if (overlaps(state_in, sb, state_out, sb))
      return fail(GDN_ERR_INVALID_ARGUMENT, "state_out partially overlaps state_in");
  }
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  if (conv && (total_tokens > 0 || conv->state_out)) {  // every argument checked: the conv stage first
    s = launched(gdn::launch_conv1d_prefill(env, conv->x, conv->w, cu_seqlens, num_seqs, total_tokens, conv->C,
                                            conv->state_in, conv->state_out, const_cast<gdn_bf16*>(qkv)),
                 "conv1d launch");
    if (s != GDN_OK) return s;
  }
  return launched(gdn::launch_kda_chunk_prefill(env, qkv, g, g_min, beta, cu_seqlens, num_seqs, total_tokens,
                                                geo->num_k_heads, geo->num_v_heads, q_scale, l2_eps, state_in,
                                                state_out, z, norm_w, rms_eps, out, workspace),
                  "KDA chunk prefill launch");
}

gdn_status gdn_kda_chunk_prefill(const gdn_geometry* geo, const gdn_bf16* qkv, const float* g, float g_min,
                                 const float* beta, const int32_t* cu_seqlens, int32_t num_seqs,
                                 int32_t total_tokens, float q_scale, float l2_eps, const float* state_in,
                                 float* state_out, const gdn_bf16* z, const gdn_bf16* norm_w, float rms_eps,
                                 gdn_bf16* out, void* workspace, size_t workspace_bytes, void* stream) {
  return kda_chunk_prefill(geo, qkv, g, g_min, beta, cu_seqlens, num_seqs, total_tokens, q_scale, l2_eps, state_in,
                           state_out, z, norm_w, rms_eps, out, workspace, workspace_bytes, stream);
}

gdn_status gdn_kda_prefill(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w,
                           const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                           const gdn_bf16* conv_state_in, gdn_bf16* conv_state_out, gdn_bf16* qkv, const float* g,
                           float g_min, const float* beta, float q_scale, float l2_eps, const float* state_in,
                           float* state_out, const gdn_bf16* z, const gdn_bf16* norm_w, float rms_eps,
                           gdn_bf16* out, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (num_seqs > 0) {  // the conv stage's own arguments (the chunk stage checks the rest)
    GDN_REQUIRE(conv_w, "conv_w");
    GDN_OPTIONAL(conv_state_in, "conv_state_in");
    GDN_OPTIONAL(conv_state_out, "conv_state_out");
    if (total_tokens > 0) {
      GDN_REQUIRE(x, "x");
      GDN_REQUIRE(qkv, "qkv");
      const size_t bytes = (size_t)total_tokens * conv_channels(geo) * 2;
      if (overlaps(x, bytes, qkv, bytes)) return fail(GDN_ERR_INVALID_ARGUMENT, "qkv overlaps x");
    }
  }
  const ConvStage conv = {x, conv_w, conv_state_in, conv_state_out, conv_channels(geo)};
  return kda_chunk_prefill(geo, qkv, g, g_min, beta, cu_seqlens, num_seqs, total_tokens, q_scale, l2_eps, state_in,
                           state_out, z, norm_w, rms_eps, out, workspace, workspace_bytes, stream, &conv);
}

gdn_status gdn_decode_step_fp16_state(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w,
                                      gdn_bf16* conv_state, const float* g, const float* beta, gdn_f16* state,
                                      const gdn_bf16* z, const gdn_bf16* norm_w, float q_scale, float l2_eps,
                                      float rms_eps, gdn_bf16* out, int32_t batch, void* stream) {
  const gdn::GateSrc gates = {g, beta, nullptr, nullptr, nullptr, nullptr};
  return decode_step(geo, x, conv_w, conv_state, gates, state, true, z, norm_w, q_scale, l2_eps, rms_eps, out,
                     batch, stream);
}

gdn_status gdn_gates(const gdn_geometry* geo, const gdn_bf16* a, const gdn_bf16* b, const float* A_log,
                     const float* dt_bias, float* g, float* beta, int32_t rows, void* stream) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (rows < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "negative rows");
  if (rows == 0) return ok();
  GDN_REQUIRE(a, "a");
  GDN_REQUIRE(b, "b");
  GDN_REQUIRE(g, "g");
  GDN_REQUIRE(beta, "beta");
  if (!A_log || !dt_bias) return fail(GDN_ERR_INVALID_ARGUMENT, "A_log or dt_bias is NULL");
  if ((reinterpret_cast<uintptr_t>(A_log) | reinterpret_cast<uintptr_t>(dt_bias)) & 3u)
    return fail(GDN_ERR_MISALIGNED, "A_log or dt_bias is not 4-byte aligned");
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_gates(env, a, b, A_log, dt_bias, g, beta, rows, geo->num_v_heads), "gates launch");
}

size_t gdn_verify_stash_size(const gdn_geometry* geo, int32_t batch, int32_t rows) {
  if (check_geometry(geo) != GDN_OK || batch < 0 || rows < 1 || rows > gdn::kMaxVerifyRows) return 0;
  const int C = 2 * geo->num_k_heads * gdn::kHeadDim + geo->num_v_heads * gdn::kHeadDim;
  return (size_t)batch * rows * gdn::verify_stash_layout(C, geo->num_k_heads, geo->num_v_heads).bytes;
}

}  // extern "C"

namespace {
gdn_status check_verify_shape(const gdn_geometry* geo, int32_t batch, int32_t rows) {
  gdn_status s = check_geometry(geo);
  if (s != GDN_OK) return s;
  if (batch < 0 || batch > 65535) return fail(GDN_ERR_INVALID_ARGUMENT, "batch must be in [0, 65535] (got %d)", batch);
  if (rows < 1 || rows > gdn::kMaxVerifyRows)
    return fail(GDN_ERR_INVALID_ARGUMENT, "rows must be in [1, %d] (got %d)", gdn::kMaxVerifyRows, rows);
  if (!gdn::verify_supported(rows, geo->num_k_heads, geo->num_v_heads))
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "%d rows with %d V heads per K head exceed the verify kernel's shared memory",
                rows, geo->num_v_heads / geo->num_k_heads);
  return GDN_OK;
}

gdn_status verify(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w, const gdn_bf16* conv_state,
                  const float* g, const float* beta, const void* state, bool fp16_state, const gdn_bf16* z,
                  const gdn_bf16* norm_w, float q_scale, float l2_eps, float rms_eps, gdn_bf16* out, int32_t batch,
                  int32_t rows, void* stash, size_t stash_bytes, void* stream) {
  gdn_status s = check_verify_shape(geo, batch, rows);
  if (s != GDN_OK) return s;
  if (batch == 0) return ok();
  GDN_REQUIRE(x, "x");
  GDN_REQUIRE(conv_w, "conv_w");
  GDN_REQUIRE(conv_state, "conv_state");
  GDN_REQUIRE(state, "state");
  GDN_REQUIRE(z, "z");
  GDN_REQUIRE(norm_w, "norm_w");
  GDN_REQUIRE(out, "out");
  GDN_REQUIRE(stash, "stash");
  if (!g || !beta) return fail(GDN_ERR_INVALID_ARGUMENT, "g or beta is NULL");
  if ((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(beta)) & 3u)
    return fail(GDN_ERR_MISALIGNED, "g or beta is not 4-byte aligned");
  if (!(l2_eps >= 0.f) || !(rms_eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  const size_t need = gdn_verify_stash_size(geo, batch, rows);
  if (stash_bytes < need) return fail(GDN_ERR_WORKSPACE, "stash of %zu bytes required (got %zu)", need, stash_bytes);
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_verify(env, x, conv_w, conv_state, g, beta, state, fp16_state, z, norm_w, q_scale,
                                     l2_eps, rms_eps, out, stash, batch, rows, geo->num_k_heads, geo->num_v_heads),
                  "verify launch");
}

gdn_status verify_commit(const gdn_geometry* geo, const int32_t* committed_rows, const void* stash,
                         size_t stash_bytes, gdn_bf16* conv_state, void* state, bool fp16_state, int32_t batch,
                         int32_t rows, void* stream) {
  gdn_status s = check_verify_shape(geo, batch, rows);
  if (s != GDN_OK) return s;
  if (batch == 0) return ok();
  if (!committed_rows) return fail(GDN_ERR_INVALID_ARGUMENT, "committed_rows is NULL");
  if (reinterpret_cast<uintptr_t>(committed_rows) & 3u)
    return fail(GDN_ERR_MISALIGNED, "committed_rows is not 4-byte aligned");
  GDN_REQUIRE(stash, "stash");
  GDN_REQUIRE(conv_state, "conv_state");
  GDN_REQUIRE(state, "state");
  const size_t need = gdn_verify_stash_size(geo, batch, rows);
  if (stash_bytes < need)
    return fail(GDN_ERR_WORKSPACE, "stash of %zu bytes required for batch %d x rows %d (got %zu)", need, batch, rows,
                stash_bytes);
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_verify_commit(env, committed_rows, stash, conv_state, state, fp16_state, batch, rows,
                                            geo->num_k_heads, geo->num_v_heads),
                  "verify commit launch");
}
}  // namespace

extern "C" {

gdn_status gdn_verify(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w, const gdn_bf16* conv_state,
                      const float* g, const float* beta, const float* state, const gdn_bf16* z,
                      const gdn_bf16* norm_w, float q_scale, float l2_eps, float rms_eps, gdn_bf16* out,
                      int32_t batch, int32_t rows, void* stash, size_t stash_bytes, void* stream) {
  return verify(geo, x, conv_w, conv_state, g, beta, state, false, z, norm_w, q_scale, l2_eps, rms_eps, out, batch,
                rows, stash, stash_bytes, stream);
}

gdn_status gdn_verify_fp16_state(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w,
                                 const gdn_bf16* conv_state, const float* g, const float* beta, const gdn_f16* state,
                                 const gdn_bf16* z, const gdn_bf16* norm_w, float q_scale, float l2_eps,
                                 float rms_eps, gdn_bf16* out, int32_t batch, int32_t rows, void* stash,
                                 size_t stash_bytes, void* stream) {
  return verify(geo, x, conv_w, conv_state, g, beta, state, true, z, norm_w, q_scale, l2_eps, rms_eps, out, batch,
                rows, stash, stash_bytes, stream);
}

gdn_status gdn_verify_commit(const gdn_geometry* geo, const int32_t* committed_rows, const void* stash,
                             size_t stash_bytes, gdn_bf16* conv_state, float* state, int32_t batch, int32_t rows,
                             void* stream) {
  return verify_commit(geo, committed_rows, stash, stash_bytes, conv_state, state, false, batch, rows, stream);
}

gdn_status gdn_verify_commit_fp16_state(const gdn_geometry* geo, const int32_t* committed_rows, const void* stash,
                                        size_t stash_bytes, gdn_bf16* conv_state, gdn_f16* state, int32_t batch,
                                        int32_t rows, void* stream) {
  return verify_commit(geo, committed_rows, stash, stash_bytes, conv_state, state, true, batch, rows, stream);
}

// ---- allocation-free chunk prefill: the schedule lives in a fixed device array of this file
}  // extern "C"

namespace {
static __device__ __align__(256) unsigned char g_noalloc_scratch[GDN_NOALLOC_SCRATCH_BYTES];
// The array's device address per device index (the first call on a device looks it up; racing
// first calls store the same address).  It is not refreshed after cudaDeviceReset.
std::atomic<void*> g_noalloc_ptr[kMaxDevices] = {};
}  // namespace

extern "C" {

gdn_status gdn_chunk_prefill_noalloc(const gdn_geometry* geo, const gdn_bf16* qkv, const float* g,
                                     const float* beta, const int32_t* cu_seqlens, int32_t num_seqs,
                                     int32_t total_tokens, float q_scale, float l2_eps, const float* state_in,
                                     float* state_out, const gdn_bf16* z, const gdn_bf16* norm_w, float rms_eps,
                                     gdn_bf16* out, void* stream) {
  if (num_seqs > GDN_NOALLOC_MAX_SEQS)
    return fail(GDN_ERR_INVALID_ARGUMENT, "num_seqs=%d exceeds the %d sequences of the fixed scratch", num_seqs,
                GDN_NOALLOC_MAX_SEQS);
  if (gdn_chunk_prefill_min_workspace_size(geo, num_seqs, total_tokens) > GDN_NOALLOC_SCRATCH_BYTES)
    return fail(GDN_ERR_INVALID_ARGUMENT, "the fixed scratch is too small for num_seqs=%d", num_seqs);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(GDN_ERR_CUDA, "device index %d out of range", dev);
  void* scratch = g_noalloc_ptr[dev].load(std::memory_order_acquire);
  if (!scratch) {
    // host code only sees a stand-in for the array: its device address comes from the runtime
    e = cudaGetSymbolAddress(&scratch, g_noalloc_scratch);
    if (e != cudaSuccess || !scratch)
      return fail(GDN_ERR_CUDA, "cudaGetSymbolAddress(scratch): %s", cudaGetErrorString(e));
    g_noalloc_ptr[dev].store(scratch, std::memory_order_release);
  }
  return gdn_chunk_prefill(geo, qkv, g, beta, cu_seqlens, num_seqs, total_tokens, q_scale, l2_eps, state_in,
                           state_out, z, norm_w, rms_eps, out, scratch, GDN_NOALLOC_SCRATCH_BYTES, stream);
}

}  // extern "C"

namespace {

gdn_status check_attn_geometry(const gdn_attn_geometry* geo) {
  if (!geo) return fail(GDN_ERR_INVALID_ARGUMENT, "geometry is NULL");
  if (geo->num_kv_heads <= 0 || geo->num_q_heads <= 0 || geo->num_q_heads % geo->num_kv_heads != 0)
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "num_q_heads (%d) must be a positive multiple of num_kv_heads (%d)",
                geo->num_q_heads, geo->num_kv_heads);
  if (geo->head_dim != 128 && geo->head_dim != 256)
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "head_dim must be 128 or 256 (got %d)", geo->head_dim);
  if (geo->num_q_heads > 256 || geo->num_q_heads / geo->num_kv_heads > 64)
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "at most 256 query heads and 64 to a key head (got %d, %d key heads)",
                geo->num_q_heads, geo->num_kv_heads);
  return GDN_OK;
}

gdn_status check_paged_cache(const gdn_kv_cache* c, const int32_t* block_table, int32_t max_pages,
                             gdn::PagedCache* out) {
  if (!c) return fail(GDN_ERR_INVALID_ARGUMENT, "cache is NULL");
  if (c->type != GDN_CACHE_BF16 && c->type != GDN_CACHE_E4M3)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown cache type %d", c->type);
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "page_size must be 16, 32, 64 or 128 (got %d)", c->page_size);
  if (c->num_pages < 1 || max_pages < 1)
    return fail(GDN_ERR_INVALID_ARGUMENT, "num_pages (%d) and max_pages (%d) must be positive", c->num_pages,
                max_pages);
  GDN_REQUIRE(c->k, "cache k");
  GDN_REQUIRE(c->v, "cache v");
  if (c->type == GDN_CACHE_E4M3 && (!c->k_scale || !c->v_scale))
    return fail(GDN_ERR_INVALID_ARGUMENT, "k_scale or v_scale is NULL");
  if (c->type == GDN_CACHE_E4M3 && !(aligned16(c->k_scale) && aligned16(c->v_scale)))
    return fail(GDN_ERR_MISALIGNED, "k_scale or v_scale is not 16-byte aligned");
  if (!block_table) return fail(GDN_ERR_INVALID_ARGUMENT, "block_table is NULL");
  if (reinterpret_cast<uintptr_t>(block_table) & 3u)
    return fail(GDN_ERR_MISALIGNED, "block_table is not 4-byte aligned");
  out->k = c->k;
  out->v = c->v;
  out->k_scale = c->k_scale;
  out->v_scale = c->v_scale;
  out->table = block_table;
  out->max_pages = max_pages;
  out->num_pages = c->num_pages;
  out->page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  out->e4m3 = c->type == GDN_CACHE_E4M3;
  return GDN_OK;
}

// num_seqs, total_tokens and the arrays that go by sequence; *nothing: the call has no rows.
gdn_status check_attn_batch(const int32_t* per_seq, const char* name, bool required, const int32_t* cu_seqlens,
                            int32_t num_seqs, int32_t total_tokens, bool* nothing) {
  if (num_seqs < 0 || total_tokens < 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "negative size (num_seqs=%d, total_tokens=%d)", num_seqs, total_tokens);
  if (num_seqs == 0 && total_tokens > 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "total_tokens=%d with no sequence", total_tokens);
  *nothing = total_tokens == 0;
  if (*nothing) return GDN_OK;
  if (!cu_seqlens && num_seqs != total_tokens)
    return fail(GDN_ERR_INVALID_ARGUMENT, "without cu_seqlens num_seqs (%d) must be total_tokens (%d)", num_seqs,
                total_tokens);
  if (required && !per_seq) return fail(GDN_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(per_seq)) & 3u)
    return fail(GDN_ERR_MISALIGNED, "cu_seqlens or %s is not 4-byte aligned", name);
  return GDN_OK;
}

gdn_status check_head_rows(const gdn_bf16* p, int64_t token, int64_t head, const char* name) {
  GDN_REQUIRE(p, name);
  if ((token | head) & 7)
    return fail(GDN_ERR_MISALIGNED, "the strides of %s (%lld, %lld) must be multiples of 8 elements", name,
                (long long)token, (long long)head);
  return GDN_OK;
}

// Whether any of the heads' rows lies in the memory range [out, out + bytes).
bool rows_overlap(const gdn_bf16* p, int64_t token, int64_t head, int64_t tokens, int64_t heads, int64_t dim,
                  const void* out, size_t bytes) {
  const int64_t t = (tokens - 1) * token, h = (heads - 1) * head;
  const int64_t lo = (t < 0 ? t : 0) + (h < 0 ? h : 0), hi = (t > 0 ? t : 0) + (h > 0 ? h : 0) + dim;
  return overlaps(p + lo, (size_t)(hi - lo) * 2, out, bytes);
}

// Whether the memory range [out, out + bytes) has any of the pool's pages or scales.
bool overlaps_pool(const gdn_attn_geometry* geo, const gdn_kv_cache* c, const void* out, size_t bytes) {
  const size_t rows = (size_t)c->num_pages * geo->num_kv_heads * c->page_size;
  const size_t pool = rows * geo->head_dim * (c->type == GDN_CACHE_E4M3 ? 1 : 2);
  if (overlaps(c->k, pool, out, bytes) || overlaps(c->v, pool, out, bytes)) return true;
  return c->type == GDN_CACHE_E4M3 && (overlaps(c->k_scale, rows, out, bytes) || overlaps(c->v_scale, rows, out, bytes));
}

gdn_status attention(const gdn_attn_geometry* geo, const gdn_bf16* q, const gdn_kv_cache* cache,
                     const int32_t* block_table, int32_t max_pages, const int32_t* kv_lens,
                     const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens, float softmax_scale,
                     const gdn_bf16* z, int64_t z_token_stride, int64_t z_head_stride, gdn_bf16* out,
                     void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status s = check_attn_geometry(geo);
  if (s != GDN_OK) return s;
  bool nothing;
  if ((s = check_attn_batch(kv_lens, "kv_lens", true, cu_seqlens, num_seqs, total_tokens, &nothing)) != GDN_OK)
    return s;
  if (nothing) return ok();
  gdn::PagedCache c;
  if ((s = check_paged_cache(cache, block_table, max_pages, &c)) != GDN_OK) return s;
  GDN_REQUIRE(q, "q");
  GDN_REQUIRE(out, "out");
  if (z && (s = check_head_rows(z, z_token_stride, z_head_stride, "z")) != GDN_OK) return s;
  if (!(softmax_scale > 0.f) || softmax_scale > 1e38f)  // times log2(e) it is finite too
    return fail(GDN_ERR_INVALID_ARGUMENT, "softmax_scale must be positive and at most 1e38");
  const size_t bytes = (size_t)total_tokens * geo->num_q_heads * geo->head_dim * 2;
  if (overlaps(q, bytes, out, bytes)) return fail(GDN_ERR_INVALID_ARGUMENT, "out overlaps q");
  if (z && rows_overlap(z, z_token_stride, z_head_stride, total_tokens, geo->num_q_heads, geo->head_dim, out, bytes))
    return fail(GDN_ERR_INVALID_ARGUMENT, "out overlaps z");
  if (overlaps_pool(geo, cache, out, bytes)) return fail(GDN_ERR_INVALID_ARGUMENT, "out overlaps the cache");
  if ((int64_t)c.num_pages * geo->num_kv_heads * cache->page_size > 0x7FFFFFFFL)
    return fail(GDN_ERR_INVALID_ARGUMENT, "the pool has more than 2^31 rows");
  const size_t need = gdn::attn_workspace_bytes(geo->head_dim);
  if (!workspace || workspace_bytes < need)
    return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes required (got %zu)", need, workspace ? workspace_bytes : 0);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(GDN_ERR_MISALIGNED, "workspace is not 256-byte aligned");
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_attn(env, geo->num_q_heads, geo->num_kv_heads, geo->head_dim, q, c, kv_lens, cu_seqlens,
                                   num_seqs, total_tokens, softmax_scale, {z, z_token_stride, z_head_stride}, out,
                                   workspace),
                  "attention launch");
}

}  // namespace

extern "C" {

gdn_status gdn_attn_rope_frequencies(int32_t rot_dim, const gdn_rope_scaling* sc, double* freqs, double* magnitude) {
  if (!sc || !freqs || !magnitude) return fail(GDN_ERR_INVALID_ARGUMENT, "scaling, freqs or magnitude is NULL");
  if (rot_dim <= 0 || rot_dim % 2) return fail(GDN_ERR_INVALID_ARGUMENT, "rot_dim (%d) must be positive and even", rot_dim);
  if (sc->kind < GDN_ROPE_PLAIN || sc->kind > GDN_ROPE_RAMP)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown scaling kind %d", sc->kind);
  if (!(sc->base > 0.) || !std::isfinite(sc->base)) return fail(GDN_ERR_INVALID_ARGUMENT, "base must be positive");
  const bool scaled = sc->kind != GDN_ROPE_PLAIN;
  if (scaled && (!(sc->factor > 0.) || !std::isfinite(sc->factor)))
    return fail(GDN_ERR_INVALID_ARGUMENT, "factor must be positive");
  if (sc->kind == GDN_ROPE_BASE && rot_dim < 4)
    return fail(GDN_ERR_INVALID_ARGUMENT, "GDN_ROPE_BASE needs rot_dim >= 4");
  if (sc->kind == GDN_ROPE_RAMP && (!(sc->low < sc->high) || !(sc->original_positions > 0.)))
    return fail(GDN_ERR_INVALID_ARGUMENT, "low < high and original_positions > 0 are required");
  *magnitude = 1.;
  double base = sc->base;
  if (sc->kind == GDN_ROPE_BASE) base *= std::pow(sc->factor, rot_dim / (rot_dim - 2.));
  for (int j = 0; j < rot_dim / 2; ++j) {
    double f = std::pow(base, -2. * j / rot_dim);
    if (sc->kind == GDN_ROPE_LINEAR) f /= sc->factor;
    if (sc->kind == GDN_ROPE_RAMP) {
      const double turns = sc->original_positions * f / 6.283185307179586477;
      const double kept = std::fmin(std::fmax((turns - sc->low) / (sc->high - sc->low), 0.), 1.);
      f = f * kept + f / sc->factor * (1. - kept);
    }
    freqs[j] = f;
  }
  if (sc->kind == GDN_ROPE_RAMP && sc->factor > 1.) *magnitude = 0.1 * std::log(sc->factor) + 1.;
  return ok();
}

gdn_status gdn_attn_prepare(const gdn_attn_geometry* geo, const gdn_bf16* q, int64_t q_token_stride,
                            int64_t q_head_stride, const gdn_bf16* k, int64_t k_token_stride, int64_t k_head_stride,
                            const gdn_bf16* v, int64_t v_token_stride, int64_t v_head_stride, const gdn_bf16* q_norm_w,
                            const gdn_bf16* k_norm_w, float rms_eps, const gdn_rope* rope, const gdn_kv_cache* cache,
                            const int32_t* block_table, int32_t max_pages, const int32_t* kv_lens,
                            const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens, gdn_bf16* q_out,
                            void* stream) {
  gdn_status s = check_attn_geometry(geo);
  if (s != GDN_OK) return s;
  bool nothing;
  if ((s = check_attn_batch(kv_lens, "kv_lens", true, cu_seqlens, num_seqs, total_tokens, &nothing)) != GDN_OK)
    return s;
  if (nothing) return ok();
  gdn::PagedCache c;
  if ((s = check_paged_cache(cache, block_table, max_pages, &c)) != GDN_OK) return s;
  const int D = geo->head_dim;
  const size_t out_bytes = (size_t)total_tokens * geo->num_q_heads * D * 2;
  if (q) {
    if ((s = check_head_rows(q, q_token_stride, q_head_stride, "q")) != GDN_OK) return s;
    GDN_REQUIRE(q_out, "q_out");
    // Each row is read whole before it is written, by the same lanes: q_out may be q itself, but rows
    // at other places would be overwritten before they are read.  (One token or head has no stride.)
    const bool same = q == q_out && (q_head_stride == D || geo->num_q_heads == 1) &&
                      (q_token_stride == (int64_t)D * geo->num_q_heads || total_tokens == 1);
    if (!same && rows_overlap(q, q_token_stride, q_head_stride, total_tokens, geo->num_q_heads, D, q_out, out_bytes))
      return fail(GDN_ERR_INVALID_ARGUMENT, "q_out overlaps q without being it");
  }
  if ((s = check_head_rows(k, k_token_stride, k_head_stride, "k")) != GDN_OK) return s;
  if ((s = check_head_rows(v, v_token_stride, v_head_stride, "v")) != GDN_OK) return s;
  if (q && (rows_overlap(k, k_token_stride, k_head_stride, total_tokens, geo->num_kv_heads, D, q_out, out_bytes) ||
            rows_overlap(v, v_token_stride, v_head_stride, total_tokens, geo->num_kv_heads, D, q_out, out_bytes)))
    return fail(GDN_ERR_INVALID_ARGUMENT, "q_out overlaps k or v");
  if (q && overlaps_pool(geo, cache, q_out, out_bytes)) return fail(GDN_ERR_INVALID_ARGUMENT, "q_out overlaps the cache");
  GDN_OPTIONAL(q_norm_w, "q_norm_w");
  GDN_OPTIONAL(k_norm_w, "k_norm_w");
  if (!(rms_eps >= 0.f)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  gdn::Rope r = {nullptr, 0, 0, 1.f};
  if (rope && rope->rot_dim != 0) {
    if (rope->rot_dim < 0 || rope->rot_dim % 16 || rope->rot_dim > D)
      return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "rot_dim must be a multiple of 16 and at most %d (got %d)", D,
                  rope->rot_dim);
    if (!rope->freqs) return fail(GDN_ERR_INVALID_ARGUMENT, "freqs is NULL");
    if (reinterpret_cast<uintptr_t>(rope->freqs) & 7u) return fail(GDN_ERR_MISALIGNED, "freqs is not 8-byte aligned");
    r = {rope->freqs, rope->rot_dim, rope->interleaved, rope->magnitude};
  }
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_attn_prepare(env, geo->num_q_heads, geo->num_kv_heads, D,
                                           {q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride},
                                           {v, v_token_stride, v_head_stride}, q_norm_w, k_norm_w, rms_eps, r, c,
                                           kv_lens, cu_seqlens, num_seqs, total_tokens, q_out),
                  "attention prepare launch");
}

gdn_status gdn_attn_cache_read(const gdn_attn_geometry* geo, const gdn_kv_cache* cache, const int32_t* block_table,
                               int32_t max_pages, const int32_t* starts, const int32_t* cu_seqlens, int32_t num_seqs,
                               int32_t total_tokens, gdn_bf16* k_out, gdn_bf16* v_out, void* stream) {
  gdn_status s = check_attn_geometry(geo);
  if (s != GDN_OK) return s;
  bool nothing;
  if ((s = check_attn_batch(starts, "starts", false, cu_seqlens, num_seqs, total_tokens, &nothing)) != GDN_OK)
    return s;
  if (nothing) return ok();
  gdn::PagedCache c;
  if ((s = check_paged_cache(cache, block_table, max_pages, &c)) != GDN_OK) return s;
  GDN_REQUIRE(k_out, "k_out");
  GDN_REQUIRE(v_out, "v_out");
  const size_t bytes = (size_t)total_tokens * geo->num_kv_heads * geo->head_dim * 2;
  if (overlaps(k_out, bytes, v_out, bytes)) return fail(GDN_ERR_INVALID_ARGUMENT, "v_out overlaps k_out");
  if (overlaps_pool(geo, cache, k_out, bytes) || overlaps_pool(geo, cache, v_out, bytes))
    return fail(GDN_ERR_INVALID_ARGUMENT, "k_out or v_out overlaps the cache");
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_attn_cache_read(env, geo->num_kv_heads, geo->head_dim, c, starts, cu_seqlens, num_seqs,
                                              total_tokens, k_out, v_out),
                  "cache read launch");
}

size_t gdn_attn_workspace_size(const gdn_attn_geometry* geo) {
  return check_attn_geometry(geo) == GDN_OK ? gdn::attn_workspace_bytes(geo->head_dim) : 0;
}

gdn_status gdn_attn_prefill(const gdn_attn_geometry* geo, const gdn_bf16* q, const gdn_kv_cache* cache,
                            const int32_t* block_table, int32_t max_pages, const int32_t* kv_lens,
                            const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens, float softmax_scale,
                            const gdn_bf16* z, int64_t z_token_stride, int64_t z_head_stride, gdn_bf16* out,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (total_tokens > 0 && num_seqs > 0 && !cu_seqlens) return fail(GDN_ERR_INVALID_ARGUMENT, "cu_seqlens is NULL");
  return attention(geo, q, cache, block_table, max_pages, kv_lens, cu_seqlens, num_seqs, total_tokens, softmax_scale, z,
                   z_token_stride, z_head_stride, out, workspace, workspace_bytes, stream);
}

gdn_status gdn_attn_decode_step(const gdn_attn_geometry* geo, const gdn_bf16* q, const gdn_kv_cache* cache,
                                const int32_t* block_table, int32_t max_pages, const int32_t* kv_lens, int32_t batch,
                                float softmax_scale, const gdn_bf16* z, int64_t z_token_stride, int64_t z_head_stride,
                                gdn_bf16* out, void* workspace, size_t workspace_bytes, void* stream) {
  return attention(geo, q, cache, block_table, max_pages, kv_lens, nullptr, batch, batch, softmax_scale, z,
                   z_token_stride, z_head_stride, out, workspace, workspace_bytes, stream);
}

}  // extern "C"

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;  // bytes: what a tensor map holds

size_t span(int64_t rows, int64_t stride, int64_t cols) { return (size_t)((rows - 1) * stride + cols); }

// rows of codes
gdn_status check_codes(const uint8_t* p, int64_t stride, int32_t cols, const char* name) {
  GDN_REQUIRE(p, name);
  if (stride < cols || stride >= kMaxStride)
    return fail(GDN_ERR_INVALID_ARGUMENT, "the row stride of %s (%lld) must be at least its %d columns and below 2^40",
                name, (long long)stride, cols);
  if (stride & 15)
    return fail(GDN_ERR_MISALIGNED, "the row stride of %s (%lld) must be a multiple of 16 bytes", name, (long long)stride);
  return GDN_OK;
}

gdn_status check_moe_geometry(const gdn_moe_geometry* geo) {
  if (!geo) return fail(GDN_ERR_INVALID_ARGUMENT, "geometry is NULL");
  const struct {
    int v;
    const char* name;
    int least;
  } widths[3] = {{geo->hidden, "hidden", 16}, {geo->inter, "inter", 16}, {geo->shared_inter, "shared_inter", 0}};
  for (const auto& w : widths)
    if (w.v < w.least || w.v > GDN_MOE_MAX_WIDTH || w.v % 16)
      return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "%s (%d) must be a multiple of 16 from %d to %d", w.name, w.v, w.least,
                  GDN_MOE_MAX_WIDTH);
  if (geo->num_experts < 1 || geo->num_experts > GDN_MOE_MAX_EXPERTS)
    return fail(GDN_ERR_UNSUPPORTED_GEOMETRY, "num_experts (%d) must be 1 to %d", geo->num_experts, GDN_MOE_MAX_EXPERTS);
  return GDN_OK;
}

gdn_status check_moe_size(int32_t tokens, int32_t top_k) {
  if (tokens < 0 || tokens > GDN_MOE_MAX_TOKENS)
    return fail(GDN_ERR_INVALID_ARGUMENT, "tokens (%d) must be 0 to %d", tokens, GDN_MOE_MAX_TOKENS);
  if (top_k < 1 || top_k > GDN_MOE_MAX_TOP_K)
    return fail(GDN_ERR_INVALID_ARGUMENT, "top_k (%d) must be 1 to %d", top_k, GDN_MOE_MAX_TOP_K);
  return GDN_OK;
}

gdn::Moe moe_of(const gdn_moe_geometry* g, const gdn_moe_weights* w) {
  return {g->hidden, g->inter, g->num_experts, g->shared_inter,
          w ? w->router : nullptr, w ? w->router_bias : nullptr, w ? w->gate_up : nullptr, w ? w->down : nullptr,
          w ? w->shared_gate_up : nullptr, w ? w->shared_down : nullptr, w ? w->gate_up_scale : nullptr,
          w ? w->down_scale : nullptr, w ? w->shared_gate_up_scale : nullptr, w ? w->shared_down_scale : nullptr,
          w ? w->shared_gate : nullptr};
}

// Both calls of the expert layer; `c` has the routing.
gdn_status moe_step(const gdn_moe_geometry* geo, const gdn_moe_weights* w, gdn::MoeCall c, const gdn_bf16* x,
                    int64_t x_row_stride, int32_t tokens, gdn_bf16* out, void* workspace, size_t workspace_bytes,
                    void* stream) {
  gdn_status s;
  if (tokens == 0) return ok();
  if (!w) return fail(GDN_ERR_INVALID_ARGUMENT, "weights is NULL");
  if (w->type != GDN_WEIGHT_BF16 && w->type != GDN_WEIGHT_E4M3)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown weight type %d", w->type);
  const bool e4m3 = w->type == GDN_WEIGHT_E4M3, shared = geo->shared_inter > 0;
  const size_t H = geo->hidden, I = geo->inter, E = geo->num_experts, Is = geo->shared_inter, T = tokens;
  const size_t K = c.top_k, size = e4m3 ? 1 : 2, hb = (H + 127) / 128, ib = (I + 127) / 128, sb = (Is + 127) / 128;
  GDN_REQUIRE(x, "x");
  GDN_REQUIRE(out, "out");
  if (x_row_stride & 7)
    return fail(GDN_ERR_MISALIGNED, "the row stride of x (%lld) must be a multiple of 8 elements", (long long)x_row_stride);
  if (tokens > 1 && (x_row_stride < geo->hidden || x_row_stride >= kMaxStride / 2))
    return fail(GDN_ERR_INVALID_ARGUMENT, "the row stride of x (%lld) must be at least hidden (%d) and below 2^39",
                (long long)x_row_stride, geo->hidden);
  const struct {
    const void* p;
    size_t bytes;
    const char* name;
    bool needed, allowed;
  } parts[] = {{w->router, E * H * 2, "router", !c.ids_in, !c.ids_in},
               {w->router_bias, E * 4, "router_bias", false, !c.ids_in},
               {w->gate_up, E * 2 * I * H * size, "gate_up", true, true},
               {w->down, E * I * H * size, "down", true, true},
               {w->gate_up_scale, E * 2 * ib * hb * 4, "gate_up_scale", e4m3, e4m3},
               {w->down_scale, E * ib * hb * 4, "down_scale", e4m3, e4m3},
               {w->shared_gate_up, 2 * Is * H * size, "shared_gate_up", shared, shared},
               {w->shared_down, Is * H * size, "shared_down", shared, shared},
               {w->shared_gate_up_scale, 2 * sb * hb * 4, "shared_gate_up_scale", shared && e4m3, shared && e4m3},
               {w->shared_down_scale, sb * hb * 4, "shared_down_scale", shared && e4m3, shared && e4m3},
               {w->shared_gate, H * 2, "shared_gate", false, shared},
               {x, span(T, T > 1 ? x_row_stride : geo->hidden, geo->hidden) * 2, "x", true, true},
               {c.ids_in, T * K * 4, "ids", false, true},
               {c.weights_in, T * K * 4, "weights", false, true}};
  const struct {
    const void* p;
    size_t bytes;
    const char* name;
  } outs[] = {{out, T * H * 2, "out"}, {c.ids_out, T * K * 4, "ids"}, {c.weights_out, T * K * 4, "weights"}};
  for (const auto& a : parts) {
    if (!a.allowed) continue;  // not read
    if (a.needed) GDN_REQUIRE(a.p, a.name);
    GDN_OPTIONAL(a.p, a.name);
    for (const auto& o : outs)
      if (a.p && o.p && overlaps(a.p, a.bytes, o.p, o.bytes))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s overlaps %s", o.name, a.name);
  }
  for (int i = 0; i < 3; ++i) {
    GDN_OPTIONAL(outs[i].p, outs[i].name);
    for (int j = 0; j < i; ++j)
      if (outs[i].p && outs[j].p && overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s overlaps %s", outs[i].name, outs[j].name);
  }
  gdn::Moe m = moe_of(geo, w);
  if (!e4m3) m.gate_up_scale = m.down_scale = m.shared_gate_up_scale = m.shared_down_scale = nullptr;
  if (!shared) m.shared_gate = nullptr;
  const size_t need = gdn::moe_workspace_bytes(m, tokens, c.top_k);
  if (!workspace || workspace_bytes < need)
    return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes required (got %zu)", need, workspace ? workspace_bytes : 0);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(GDN_ERR_MISALIGNED, "workspace is not 256-byte aligned");
  for (const auto& a : parts)
    if (a.allowed && a.p && overlaps(a.p, a.bytes, workspace, need))
      return fail(GDN_ERR_INVALID_ARGUMENT, "workspace overlaps %s", a.name);
  for (const auto& o : outs)
    if (o.p && overlaps(o.p, o.bytes, workspace, need))
      return fail(GDN_ERR_INVALID_ARGUMENT, "workspace overlaps %s", o.name);
  c.x = x;
  c.x_stride = tokens > 1 ? x_row_stride : geo->hidden;
  c.T = tokens;
  c.out = out;
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_moe(env, m, c, workspace), "expert layer launch");
}

}  // namespace

extern "C" {

gdn_status gdn_fp8_quantize(const gdn_bf16* x, int64_t x_row_stride, int32_t rows, int32_t cols, int32_t block_rows,
                            uint8_t* codes, int64_t codes_row_stride, float* scales, void* stream) {
  gdn_status s;
  if (rows < 0 || cols < 1)
    return fail(GDN_ERR_INVALID_ARGUMENT, "rows (%d) must not be negative, cols (%d) must be positive", rows, cols);
  if (block_rows != 1 && block_rows != GDN_FP8_BLOCK)
    return fail(GDN_ERR_INVALID_ARGUMENT, "block_rows (%d) must be 1 or %d", block_rows, GDN_FP8_BLOCK);
  if (rows == 0) return ok();
  GDN_REQUIRE(x, "x");
  if (x_row_stride < cols || x_row_stride >= kMaxStride)
    return fail(GDN_ERR_INVALID_ARGUMENT, "the row stride of x (%lld) must be at least its %d columns and below 2^40",
                (long long)x_row_stride, cols);
  if ((s = check_codes(codes, codes_row_stride, cols, "codes")) != GDN_OK) return s;
  GDN_REQUIRE(scales, "scales");
  const size_t nx = span(rows, x_row_stride, cols) * 2, nc = span(rows, codes_row_stride, cols);
  const size_t ns = (size_t)(((int64_t)rows + block_rows - 1) / block_rows) * (((int64_t)cols + 127) / 128) * 4;
  if (overlaps(x, nx, codes, nc) || overlaps(x, nx, scales, ns))
    return fail(GDN_ERR_INVALID_ARGUMENT, "codes or scales overlap x");
  if (overlaps(codes, nc, scales, ns)) return fail(GDN_ERR_INVALID_ARGUMENT, "scales overlap codes");
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_fp8_quantize(env, x, x_row_stride, rows, cols, block_rows, codes, codes_row_stride, scales),
                  "quantisation launch");
}

gdn_status gdn_fp8_matmul(const uint8_t* x, int64_t x_row_stride, const float* x_scale, const uint8_t* w,
                          int64_t w_row_stride, const float* w_scale, int32_t tokens, int32_t n, int32_t k,
                          int32_t out_type, void* out, int64_t out_row_stride, void* stream) {
  gdn_status s;
  if (tokens < 0 || n < 0 || k < 1)
    return fail(GDN_ERR_INVALID_ARGUMENT, "tokens (%d) and n (%d) must not be negative, k (%d) must be positive", tokens, n,
                k);
  if (out_type != GDN_OUT_BF16 && out_type != GDN_OUT_F32)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown output type %d", out_type);
  if (tokens == 0 || n == 0) return ok();
  if ((s = check_codes(x, x_row_stride, k, "x")) != GDN_OK) return s;
  if ((s = check_codes(w, w_row_stride, k, "w")) != GDN_OK) return s;
  GDN_REQUIRE(x_scale, "x_scale");
  GDN_REQUIRE(w_scale, "w_scale");
  GDN_REQUIRE(out, "out");
  if (out_row_stride < n || out_row_stride >= kMaxStride)
    return fail(GDN_ERR_INVALID_ARGUMENT, "the row stride of out (%lld) must be at least its %d columns and below 2^40",
                (long long)out_row_stride, n);
  const size_t kb = ((size_t)k + 127) / 128, nb = ((size_t)n + 127) / 128;
  const size_t no = span(tokens, out_row_stride, n) * (out_type == GDN_OUT_F32 ? 4 : 2);
  if (overlaps(x, span(tokens, x_row_stride, k), out, no) || overlaps(w, span(n, w_row_stride, k), out, no) ||
      overlaps(x_scale, tokens * kb * 4, out, no) || overlaps(w_scale, nb * kb * 4, out, no))
    return fail(GDN_ERR_INVALID_ARGUMENT, "out overlaps an input");
  gdn::LaunchEnv env;
  if ((s = make_env(stream, &env)) != GDN_OK) return s;
  return launched(gdn::launch_fp8_matmul(env, {x, x_row_stride, x_scale, w, w_row_stride, w_scale, tokens, n, k, out,
                                               out_row_stride, out_type == GDN_OUT_F32}),
                  "8-bit product launch");
}

size_t gdn_moe_workspace_size(const gdn_moe_geometry* geo, int32_t tokens, int32_t top_k) {
  if (check_moe_geometry(geo) != GDN_OK || check_moe_size(tokens, top_k) != GDN_OK || tokens == 0) return 0;
  return gdn::moe_workspace_bytes(moe_of(geo, nullptr), tokens, top_k);
}

gdn_status gdn_moe_step(const gdn_moe_geometry* geo, const gdn_moe_weights* w, const gdn_moe_routing* routing,
                        const gdn_bf16* x, int64_t x_row_stride, int32_t tokens, int32_t* ids, float* weights,
                        gdn_bf16* out, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status s = check_moe_geometry(geo);
  if (s != GDN_OK) return s;
  if (!routing) return fail(GDN_ERR_INVALID_ARGUMENT, "routing is NULL");
  if ((s = check_moe_size(tokens, routing->top_k)) != GDN_OK) return s;
  if (routing->top_k > geo->num_experts)
    return fail(GDN_ERR_INVALID_ARGUMENT, "top_k (%d) exceeds the %d experts", routing->top_k, geo->num_experts);
  if (routing->scoring != GDN_SCORE_SOFTMAX && routing->scoring != GDN_SCORE_SIGMOID)
    return fail(GDN_ERR_INVALID_ARGUMENT, "unknown scoring %d", routing->scoring);
  if (!std::isfinite(routing->scale)) return fail(GDN_ERR_INVALID_ARGUMENT, "scale must be finite");
  gdn::MoeCall c = {};
  c.top_k = routing->top_k;
  c.sigmoid = routing->scoring == GDN_SCORE_SIGMOID;
  c.renormalise = routing->renormalise != 0;
  c.scale = routing->scale;
  c.ids_out = ids;
  c.weights_out = weights;
  return moe_step(geo, w, c, x, x_row_stride, tokens, out, workspace, workspace_bytes, stream);
}

gdn_status gdn_moe_step_routed(const gdn_moe_geometry* geo, const gdn_moe_weights* w, const int32_t* ids,
                               const float* weights, int32_t top_k, const gdn_bf16* x, int64_t x_row_stride,
                               int32_t tokens, gdn_bf16* out, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status s = check_moe_geometry(geo);
  if (s != GDN_OK) return s;
  if ((s = check_moe_size(tokens, top_k)) != GDN_OK) return s;
  if (tokens == 0) return ok();
  GDN_REQUIRE(ids, "ids");
  GDN_REQUIRE(weights, "weights");
  gdn::MoeCall c = {};
  c.top_k = top_k;
  c.scale = 1.f;
  c.ids_in = ids;
  c.weights_in = weights;
  return moe_step(geo, w, c, x, x_row_stride, tokens, out, workspace, workspace_bytes, stream);
}

}  // extern "C"

extern "C" {

gdn_status gdn_check_device_errors(void* stream) {
  gdn::LaunchEnv env;
  gdn_status s = make_env(stream, &env);
  if (s != GDN_OK) return s;
  cudaError_t e = cudaStreamSynchronize(env.stream);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaStreamSynchronize: %s", cudaGetErrorString(e));
  unsigned word = 0;
  e = cudaMemcpy(&word, env.err, sizeof word, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "reading the device error word: %s", cudaGetErrorString(e));
  if (word) {
    const unsigned zero = 0;
    e = cudaMemcpy(env.err, &zero, sizeof zero, cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "clearing the device error word: %s", cudaGetErrorString(e));
  }
  if (word & gdn::kErrTimeout) return fail(GDN_ERR_TIMEOUT, "an in-kernel wait ran out (word 0x%x)", word);
  if (word & gdn::kErrDeviceArgument)
    return fail(GDN_ERR_DEVICE_ARGUMENT, "a kernel rejected cu_seqlens, page, length or expert contents (word 0x%x)", word);
  return ok();
}

#ifdef GDN_TEST_HOOKS
gdn_status gdn_debug_set_chunk_mode(int mode) {
  if (mode < 0 || mode > 2) return fail(GDN_ERR_INVALID_ARGUMENT, "mode must be 0, 1 or 2");
  g_chunk_mode.store(mode);
  return ok();
}

int gdn_debug_get_chunk_mode(void) { return g_chunk_mode.load(); }

gdn_status gdn_debug_set_dropped_copy(unsigned which) {
  if (which & ~3u) return fail(GDN_ERR_INVALID_ARGUMENT, "which must be a combination of bits 0 and 1");
  cudaError_t e = gdn::test_set_dropped_copy_decode(which & 1u);
  if (e == cudaSuccess) e = gdn::test_set_dropped_copy_chunk((which >> 1) & 1u);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "setting the dropped-copy hook: %s", cudaGetErrorString(e));
  return ok();
}

gdn_status gdn_debug_set_matmul_give_up(int on) {
  const cudaError_t e = gdn::test_set_give_up_matmul(on != 0);
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "setting the hook: %s", cudaGetErrorString(e));
  return ok();
}
#endif

}  // extern "C"
