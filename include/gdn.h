/*
 * gdn.h -- C ABI of the GB300 (sm_103a) Gated DeltaNet (GDN) sublayer library, libgdn.so.
 *
 * The sublayer, as the pages define it (pegainfer PR #1152 "Reference golden for the GDN
 * sublayer", Summary and Code review; GLM-5.3-Flash kernel TDD ledger, slices I2-I4):
 *
 *   prefill:  x --(causal depthwise conv1d, width 4, + SiLU)--> qkv (bf16)
 *             qkv --(head expansion by repeat_interleave, L2 norm of q and k,
 *                    chunk-wise gated delta rule with an fp32 [value, key] state)--> o
 *             o, z --(gated RMSNorm with a sigmoid output gate)--> out
 *   decode:   the same for one token per sequence, fused in one launch (Qwen3.8 kernel
 *             architecture and TDD ledger, "Current dense-27B kernel map": scalar GDN
 *             recurrence and fused output gate).
 *
 * The recurrence (per sequence and V head; S is Dv x Dk, rows index the value dimension):
 *   S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,    o_t = q_scale S_t q_t
 * with k_t, q_t the L2-normalised key/query of K head floor(h / (Hv/Hk)).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller, contiguous, row-major, and
 *     16-byte aligned (else GDN_ERR_MISALIGNED).  The library never allocates, frees or keeps
 *     a reference to caller memory after the call returns.
 *   - bf16 tensors are passed as gdn_bf16 (raw 16-bit patterns); fp32 as float.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every call is
 *     asynchronous on that stream; arguments are validated on the host before any launch, and
 *     a call that returns an error has launched nothing.
 *   - Geometry: C = 2*Hk*Dk + Hv*Dv conv channels packed [q heads | k heads | v heads].  This
 *     build supports Dk = Dv = 128, conv width 4, Hv a multiple of Hk, Hk <= 64, Hv <= 192;
 *     anything else is refused with GDN_ERR_UNSUPPORTED_GEOMETRY, never silently mis-tiled.
 *   - Device-side argument faults (for example a cu_seqlens array that is not monotonic or does
 *     not end at total_tokens) are never turned into out-of-range accesses: the kernels clamp,
 *     skip the bad sequence and raise a device error word, reported by gdn_check_device_errors.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define GDN_API __attribute__((visibility("default")))
#else
#define GDN_API
#endif

typedef uint16_t gdn_bf16; /* IEEE bfloat16 bit pattern */
typedef uint16_t gdn_f16;  /* IEEE binary16 (half precision) bit pattern */

typedef enum {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARGUMENT = 1,     /* null pointer, negative size, aliasing that is not allowed */
  GDN_ERR_UNSUPPORTED_GEOMETRY = 2, /* geometry outside what the kernels are built for         */
  GDN_ERR_MISALIGNED = 3,           /* a tensor pointer is not 16-byte aligned                  */
  GDN_ERR_CUDA = 4,                 /* a CUDA runtime call or kernel launch failed              */
  GDN_ERR_TIMEOUT = 5,              /* a bounded in-kernel wait ran out (device error word)     */
  GDN_ERR_DEVICE_ARGUMENT = 6,      /* a kernel found a bad device-side argument (cu_seqlens)   */
  GDN_ERR_WORKSPACE = 7             /* workspace missing or smaller than the queried size       */
} gdn_status;

/* Head geometry.  The pages' model: 16 K heads and 48 V heads of width 128, a four-tap conv
 * (pegainfer PR #1152, Summary). */
typedef struct {
  int32_t num_k_heads; /* Hk */
  int32_t num_v_heads; /* Hv, a multiple of Hk; V head h reads K head h / (Hv/Hk) */
  int32_t head_k_dim;  /* Dk (128) */
  int32_t head_v_dim;  /* Dv (128) */
  int32_t conv_width;  /* W  (4)   */
} gdn_geometry;

/* Tokens per chunk of the chunk-wise prefill.  A chunk never crosses a sequence boundary.
 * (pegainfer PR #1152, Validation: 16- and 64-token runs fit in one chunk, 80- and 128-token
 * runs take two.) */
#define GDN_CHUNK_SIZE 64

/* Human-readable name of a status code (static storage). */
GDN_API const char* gdn_status_string(gdn_status status);

/* Detail of the last error returned on the calling host thread ("" if none). */
GDN_API const char* gdn_last_error_message(void);

/* Library version string (static storage). */
GDN_API const char* gdn_version(void);

/*
 * Causal depthwise conv1d (width W, no bias) + SiLU over packed variable-length sequences.
 * pegainfer PR #1152, Summary (a four-tap depthwise conv; conv1d.weight is its only weight) and
 * "Commands + measured numbers" (the conv leg, compared bit-exact); GLM-5.3-Flash ledger,
 * slice I3 (a decode step equals the full width-4 causal convolution).
 *
 *   y[t, c] = bf16( silu( sum_{i<W} w[c, i] * xin(t - (W-1) + i, c) ) ),  silu(a) = a*sigmoid(a)
 *
 * where xin(p, c) is x[p, c] inside the token's own sequence, the conv state of that sequence
 * for the W-1 positions before its start, and 0 when conv_state_in is NULL.  Accumulation is
 * fp32; the result is rounded once to bf16 (round to nearest even).
 *
 *   x              [total_tokens, C] bf16
 *   conv_w         [C, W] bf16; w[c, W-1] multiplies the current token
 *   cu_seqlens     [num_seqs + 1] int32 (device): sequence n is tokens cu[n] .. cu[n+1]-1;
 *                  cu[0] = 0, non-decreasing, cu[num_seqs] = total_tokens
 *   conv_state_in  [num_seqs, C, W-1] bf16 raw inputs before each sequence (oldest first), or NULL
 *   conv_state_out [num_seqs, C, W-1] bf16 last W-1 raw inputs of each sequence, or NULL; may be
 *                  the same buffer as conv_state_in (updated in place)
 *   y              [total_tokens, C] bf16; must not overlap x
 * total_tokens == 0 or num_seqs == 0 is a no-op that returns GDN_OK.
 */
GDN_API gdn_status gdn_conv1d_prefill(const gdn_geometry* geo, const gdn_bf16* x,
                                      const gdn_bf16* conv_w, const int32_t* cu_seqlens,
                                      int32_t num_seqs, int32_t total_tokens,
                                      const gdn_bf16* conv_state_in, gdn_bf16* conv_state_out,
                                      gdn_bf16* y, void* stream);

/*
 * Bytes of device workspace for the fast path of gdn_chunk_prefill at these sizes (0 when
 * num_seqs == 0).  With at least this much, the call runs as two kernels: one that forms, for
 * every 64-token chunk at once, the quantities that do not depend on the recurrent state (the
 * intra-chunk decay factors, the solve (I + A)^-1 and the masked query-key product, about 25 KB
 * per chunk and V head), and one that carries the state through the chunks.  From 4,096 tokens
 * on it also holds 32 state slots of Hv x 128 x 128 fp32 for the parts of long sequences (see
 * gdn_chunk_prefill).  The workspace contents need no initialisation and are dead when the call's
 * kernels finish.
 */
GDN_API size_t gdn_chunk_prefill_workspace_size(const gdn_geometry* geo, int32_t num_seqs,
                                                int32_t total_tokens);

/*
 * Smallest workspace gdn_chunk_prefill accepts (the per-call sequence schedule: 256 bytes plus
 * 4 bytes per sequence, rounded up to 256).  With less than gdn_chunk_prefill_workspace_size()
 * but at least this, the call runs one fused kernel that forms the state-independent quantities
 * chunk by chunk on the state chain itself: same results within the stated tolerances, slower.
 */
GDN_API size_t gdn_chunk_prefill_min_workspace_size(const gdn_geometry* geo, int32_t num_seqs,
                                                    int32_t total_tokens);

/*
 * Chunk-wise gated delta rule over packed variable-length sequences (prefill), optionally
 * fused with the sigmoid-gated RMSNorm.  pegainfer PR #1152, Consumer (stage order
 * prepare -> cumsum -> A -> solve -> recompute -> state -> output) and Code review (f32
 * recurrent state carried across chunks); GLM-5.3-Flash ledger, slice I4 (the chunk path
 * matches the sequential state and output at 63/64/65 tokens).
 *
 *   qkv        [total_tokens, C] bf16 conv output (gdn_conv1d_prefill's y): q heads | k heads | v heads
 *   g, beta    [total_tokens, Hv] fp32 log decay (<= 0) and write strength
 *   cu_seqlens [num_seqs + 1] int32 (device), as for gdn_conv1d_prefill
 *   q_scale    output scale applied to S q (1/sqrt(Dk) for the pages' model)
 *   l2_eps     epsilon of the q/k L2 norm x / sqrt(sum x^2 + eps) (1e-6)
 *   state_in   [num_seqs, Hv, Dv, Dk] fp32 initial states ([value, key]), or NULL for zeros
 *   state_out  [num_seqs, Hv, Dv, Dk] fp32 final states; may be the same buffer as state_in
 *   z, norm_w  NULL: `out` receives o = q_scale S_t q_t (bf16).  Otherwise z [total_tokens, Hv, Dv]
 *              and norm_w [Dv] bf16, and `out` receives the gated RMSNorm of o:
 *              o * (mean_d o^2 + rms_eps)^(-1/2) * norm_w * sigmoid(z), computed from the fp32 o
 *   out        [total_tokens, Hv, Dv] bf16
 *   workspace  256-byte aligned device memory of at least gdn_chunk_prefill_min_workspace_size()
 *              bytes (NULL if 0); gdn_chunk_prefill_workspace_size() bytes select the fast path
 *
 * Streams: with the fast-path workspace, a state_out buffer, at least 4,096 tokens and no stream
 * capture in progress, the call splits each sequence's chunks into segments and runs the
 * state-independent stage of segment k + 1 on a library-owned side stream (one per device, created
 * on first use and shared by every caller on that device) beside the state stage of segment k,
 * ordered by events the library creates once per host thread and device.  Everything the call
 * writes is ordered before later work on `stream`.  Calls from different streams whose side-stream
 * work is queued together run it one after the other.  Under stream capture, everything runs on
 * `stream` as one segment.
 *
 * Long sequences: from 4,096 tokens on, a sequence whose segment holds more than twice the chunks
 * one CTA slot would get (the segment's work spread over two CTAs per SM) is cut into three or four
 * parts that run at once, decided on the device from cu_seqlens; parts after the first start
 * from a state combined from the earlier parts' transitions.  Their launch runs on a second
 * library-owned stream (per device, like the side stream) and is joined to `stream` before the
 * call's work ends; under stream capture it runs on `stream`.  A part waits (bounded) for the
 * transitions it needs; a wait that runs out sets GDN_ERR_TIMEOUT in the device error word.  With
 * one segment and state_out equal to state_in, nothing is split.
 */
GDN_API gdn_status gdn_chunk_prefill(const gdn_geometry* geo, const gdn_bf16* qkv, const float* g,
                                     const float* beta, const int32_t* cu_seqlens,
                                     int32_t num_seqs, int32_t total_tokens, float q_scale,
                                     float l2_eps, const float* state_in, float* state_out,
                                     const gdn_bf16* z, const gdn_bf16* norm_w, float rms_eps,
                                     gdn_bf16* out, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * The whole prefill sublayer in one call: gdn_conv1d_prefill (its output written to qkv), then
 * gdn_chunk_prefill on it -- the "prepare" stage of pegainfer PR #1152 Consumer, conv included,
 * followed by the chunk stages.  Same arguments, results and errors as the two calls in
 * sequence (qkv: [total_tokens, C] bf16, must not overlap x; conv_state_out may alias
 * conv_state_in; workspace as for gdn_chunk_prefill), with every argument of both stages checked
 * before either is launched: a call that returns an error has launched nothing.
 */
GDN_API gdn_status gdn_prefill(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w,
                               const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                               const gdn_bf16* conv_state_in, gdn_bf16* conv_state_out,
                               gdn_bf16* qkv, const float* g, const float* beta, float q_scale,
                               float l2_eps, const float* state_in, float* state_out,
                               const gdn_bf16* z, const gdn_bf16* norm_w, float rms_eps,
                               gdn_bf16* out, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * The gates of the recurrence from their projections, for every row (token, or sequence of a
 * decode step) and V head:
 *   g[r, h]    = -exp(A_log[h]) * softplus(a[r, h] + dt_bias[h]),   softplus(x) = log(1 + e^x)
 *   beta[r, h] = sigmoid(b[r, h])
 * The pages name these inputs (Qwen3.8 kernel architecture and TDD ledger, "GDN alpha/beta
 * transforms"; PR #1152 Summary: A_log, dt_bias, the a / b projections, and a fixture that holds
 * g / beta only after this derivation) but give no formula: this is the gate of the published
 * Gated DeltaNet / Mamba-2 layers.
 *   a, b        [rows, Hv] bf16 projection outputs
 *   A_log, dt_bias  [Hv] fp32 (4-byte aligned)
 *   g, beta     [rows, Hv] fp32 outputs, ready for gdn_chunk_prefill / gdn_decode_step
 */
GDN_API gdn_status gdn_gates(const gdn_geometry* geo, const gdn_bf16* a, const gdn_bf16* b,
                             const float* A_log, const float* dt_bias, float* g, float* beta,
                             int32_t rows, void* stream);

/*
 * gdn_chunk_prefill and gdn_decode_step with the gates derived inside the kernels that use them,
 * from the projections a, b and the per-head A_log, dt_bias (the gdn_gates formula, the same
 * arithmetic, so the results have the same bits as gdn_gates followed by the plain call): g and
 * beta are never written to memory and no gates launch precedes the call.  Qwen3.8 kernel
 * architecture and TDD ledger, kernel map (the GDN alpha / beta transforms feed the recurrence);
 * pegainfer PR #1152 Summary (A_log, dt_bias and the a / b projections are the layer's inputs).
 *   a, b            [rows, Hv] bf16 (rows = total_tokens for the prefill, batch for the decode;
 *                   2-byte aligned)
 *   A_log, dt_bias  [Hv] fp32 (4-byte aligned)
 * Every other argument, the results and the errors are those of gdn_chunk_prefill and
 * gdn_decode_step (fp32 state).
 */
GDN_API gdn_status gdn_chunk_prefill_fused_gates(const gdn_geometry* geo, const gdn_bf16* qkv,
                                                 const gdn_bf16* a, const gdn_bf16* b,
                                                 const float* A_log, const float* dt_bias,
                                                 const int32_t* cu_seqlens, int32_t num_seqs,
                                                 int32_t total_tokens, float q_scale, float l2_eps,
                                                 const float* state_in, float* state_out,
                                                 const gdn_bf16* z, const gdn_bf16* norm_w,
                                                 float rms_eps, gdn_bf16* out, void* workspace,
                                                 size_t workspace_bytes, void* stream);
GDN_API gdn_status gdn_decode_step_fused_gates(const gdn_geometry* geo, const gdn_bf16* x,
                                               const gdn_bf16* conv_w, gdn_bf16* conv_state,
                                               const gdn_bf16* a, const gdn_bf16* b,
                                               const float* A_log, const float* dt_bias,
                                               float* state, const gdn_bf16* z,
                                               const gdn_bf16* norm_w, float q_scale, float l2_eps,
                                               float rms_eps, gdn_bf16* out, int32_t batch,
                                               void* stream);

/*
 * Sigmoid-gated RMSNorm, one row per (token, V head).  pegainfer PR #1152, Summary
 * (output_gate_type "sigmoid"; the in-tree kernel that hard-codes silu is wrong) and Code
 * review (rms_norm_eps == 1e-6).
 *   out[r, d] = o[r, d] * (mean_d o[r, :]^2 + eps)^(-1/2) * norm_w[d] * sigmoid(z[r, d])
 *   o, z, out  [total_tokens, Hv, Dv] bf16 (out may alias o);  norm_w [Dv] bf16
 */
GDN_API gdn_status gdn_gated_rmsnorm(const gdn_geometry* geo, const gdn_bf16* o, const gdn_bf16* z,
                                     const gdn_bf16* norm_w, float eps, gdn_bf16* out,
                                     int32_t total_tokens, void* stream);

/*
 * One fused decode step for `batch` independent sequences (one token each): conv step on the
 * conv shift register + SiLU, L2 norm of q/k, the gated delta rule update of the fp32 state in
 * place, and the sigmoid-gated RMSNorm.  Qwen3.8 kernel architecture and TDD ledger, "Current
 * dense-27B kernel map" (scalar GDN recurrence and fused output gate); spark_model
 * layer_struct.rs, the strided decode kernel fields (one launch for all sequences, state read
 * once and written once).
 *
 *   x           [batch, C] bf16 raw conv input of this token
 *   conv_w      [C, W] bf16
 *   conv_state  [batch, C, W-1] bf16, in/out: the previous W-1 raw inputs, oldest first
 *   g, beta     [batch, Hv] fp32
 *   state       [batch, Hv, Dv, Dk] fp32, in/out
 *   z           [batch, Hv, Dv] bf16;  norm_w [Dv] bf16
 *   out         [batch, Hv, Dv] bf16 gated output
 */
GDN_API gdn_status gdn_decode_step(const gdn_geometry* geo, const gdn_bf16* x,
                                   const gdn_bf16* conv_w, gdn_bf16* conv_state, const float* g,
                                   const float* beta, float* state, const gdn_bf16* z,
                                   const gdn_bf16* norm_w, float q_scale, float l2_eps,
                                   float rms_eps, gdn_bf16* out, int32_t batch, void* stream);

/*
 * gdn_decode_step with the recurrent state stored as IEEE binary16 ("FP16 h-state"): Qwen3.8
 * kernel architecture and TDD ledger, the FP16 h-state twins of the decode kernels (the same
 * arithmetic as the fp32 kernel; the state is half precision in memory only and is rounded once
 * per token boundary).  Each state element is widened to fp32 on load, the step runs exactly as in
 * gdn_decode_step (the output comes from the new state before rounding), and the new state is
 * rounded to binary16 (to nearest, ties to even) when it is stored.  This halves the state bytes
 * the step reads and writes.
 *
 *   state       [batch, Hv, Dv, Dk] binary16, in/out (16-byte aligned)
 *   all other arguments, results and errors as gdn_decode_step.
 *
 * A state element whose magnitude rounds above 65504 becomes an infinity; nothing clamps it.
 */
GDN_API gdn_status gdn_decode_step_fp16_state(const gdn_geometry* geo, const gdn_bf16* x,
                                              const gdn_bf16* conv_w, gdn_bf16* conv_state,
                                              const float* g, const float* beta, gdn_f16* state,
                                              const gdn_bf16* z, const gdn_bf16* norm_w,
                                              float q_scale, float l2_eps, float rms_eps,
                                              gdn_bf16* out, int32_t batch, void* stream);

/*
 * Multi-token verify: `rows` (K, 1..17) consecutive tokens of each of `batch` sequences run
 * through the decode step in order -- conv step, L2 norms, gated delta rule, gated RMSNorm --
 * starting from conv_state and state, exactly as K calls of gdn_decode_step would, but WITHOUT
 * modifying either state.  Every row's gated output is written; what a later commit needs is
 * written to `stash`.  Qwen3.8 kernel architecture and TDD ledger, "Transaction and width
 * vocabulary" (verify_rows; a target transaction resolves exactly once: commit publishes only the
 * selected GDN state, abort leaves the prior state); spark_model layer_struct.rs, the WY verify
 * kernels (K = 2..17) and the write-on-accept twin with its post-verdict fold.
 *
 *   x           [batch, rows, C] bf16 raw conv inputs
 *   conv_w      [C, W] bf16;  conv_state [batch, C, W-1] bf16 (read only)
 *   g, beta     [batch, rows, Hv] fp32
 *   state       [batch, Hv, Dv, Dk] fp32 (read only)
 *   z           [batch, rows, Hv, Dv] bf16;  norm_w [Dv] bf16
 *   out         [batch, rows, Hv, Dv] bf16: row r is the output of the r+1-th token
 *   stash       gdn_verify_stash_size(geo, batch, rows) bytes, 16-byte aligned; one record per
 *               (sequence, row) at ((b * rows) + r) * (stash_size / (batch * rows)) bytes: the
 *               row's raw conv inputs (C bf16), normalised keys (Hk x Dk fp32), its delta
 *               e = beta (v - decayed state . k) for every V head and value row (Hv x Dv fp32)
 *               and g (Hv fp32).
 * GDN_ERR_UNSUPPORTED_GEOMETRY when `rows` rows of Hv/Hk V heads do not fit the kernel's shared
 * memory (never for Hv/Hk <= 3).
 */
GDN_API size_t gdn_verify_stash_size(const gdn_geometry* geo, int32_t batch, int32_t rows);
GDN_API gdn_status gdn_verify(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w,
                              const gdn_bf16* conv_state, const float* g, const float* beta,
                              const float* state, const gdn_bf16* z, const gdn_bf16* norm_w,
                              float q_scale, float l2_eps, float rms_eps, gdn_bf16* out,
                              int32_t batch, int32_t rows, void* stash, size_t stash_bytes,
                              void* stream);

/*
 * Resolves a verify: for each sequence b, committed_rows[b] = m (device int32, 0..rows) rows are
 * committed -- conv_state and state become what m decode steps of that sequence's first m rows
 * would have left (m = 0: an abort, both states untouched).  Reads only stash records of rows
 * < m.  The states must be the ones the verify read (unchanged since).  A value outside
 * [0, rows] leaves that sequence untouched and raises GDN_ERR_DEVICE_ARGUMENT in the device
 * error word.  stash_bytes is the size of the stash buffer; a stash smaller than
 * gdn_verify_stash_size(geo, batch, rows) is refused with GDN_ERR_WORKSPACE (nothing launched).
 */
GDN_API gdn_status gdn_verify_commit(const gdn_geometry* geo, const int32_t* committed_rows,
                                     const void* stash, size_t stash_bytes, gdn_bf16* conv_state,
                                     float* state, int32_t batch, int32_t rows, void* stream);

/*
 * gdn_verify and gdn_verify_commit with the recurrent state stored as IEEE binary16 (Qwen3.8
 * ledger, the FP16 h-state twins of the WY verify kernels).  The verify widens the state and
 * computes in fp32 exactly as gdn_verify; the commit widens it, applies the committed rows and
 * stores the result rounded once to binary16 (to nearest, ties to even).  No per-row state is
 * ever stored, so that is the only rounding: a commit of m rows equals m calls of
 * gdn_decode_step_fp16_state up to the roundings those calls make between the rows.  The stash
 * is the same as gdn_verify's; m = 0 leaves the state's bits untouched.
 *   state       [batch, Hv, Dv, Dk] binary16 (read only in the verify; in/out in the commit)
 */
GDN_API gdn_status gdn_verify_fp16_state(const gdn_geometry* geo, const gdn_bf16* x,
                                         const gdn_bf16* conv_w, const gdn_bf16* conv_state,
                                         const float* g, const float* beta, const gdn_f16* state,
                                         const gdn_bf16* z, const gdn_bf16* norm_w, float q_scale,
                                         float l2_eps, float rms_eps, gdn_bf16* out, int32_t batch,
                                         int32_t rows, void* stash, size_t stash_bytes,
                                         void* stream);
GDN_API gdn_status gdn_verify_commit_fp16_state(const gdn_geometry* geo,
                                                const int32_t* committed_rows, const void* stash,
                                                size_t stash_bytes, gdn_bf16* conv_state,
                                                gdn_f16* state, int32_t batch, int32_t rows,
                                                void* stream);

/*
 * One fused decode step of the KDA (Kimi delta attention) layer: as gdn_decode_step, with a decay
 * per key channel instead of per head.  GLM-5.3-Flash kernel TDD ledger, slices I2 (an fp32
 * state indexed [value, key], the decay clamped then exponentiated, its own q output scale),
 * I2a (q/k normalised x / sqrt(sum x^2 + eps)) and I3 (the width-4 conv step).  Per V head:
 *   S <- S diag(exp(max(g, g_min)));   e = beta (v - S k);   S <- S + e k^T;   o = q_scale S q
 * followed by the same sigmoid-gated RMSNorm as gdn_decode_step.
 *   g           [batch, Hv, Dk] fp32 per-channel log decay (16-byte aligned)
 *   g_min       the clamp: decays below exp(g_min) are raised to it (-INFINITY: no clamp)
 *   all other arguments, results and errors as gdn_decode_step (fp32 state).
 */
GDN_API gdn_status gdn_kda_decode_step(const gdn_geometry* geo, const gdn_bf16* x,
                                       const gdn_bf16* conv_w, gdn_bf16* conv_state,
                                       const float* g, float g_min, const float* beta, float* state,
                                       const gdn_bf16* z, const gdn_bf16* norm_w, float q_scale,
                                       float l2_eps, float rms_eps, gdn_bf16* out, int32_t batch,
                                       void* stream);

/*
 * The KDA recurrence over packed variable-length sequences (the prefill's recurrent leg),
 * optionally fused with the sigmoid-gated RMSNorm: the step of gdn_kda_decode_step applied to
 * every token in order, each (sequence, V head) state carried from token to token.
 * GLM-5.3-Flash kernel TDD ledger, slices I2 (an fp32 state indexed [value, key], a per-channel
 * decay clamped then exponentiated, its own q output scale), I2a (q/k normalised
 * x / sqrt(sum x^2 + eps)) and I4 (the prefill matches the sequential state and output at every
 * length).  This is the sequential form: one CTA per (V head, sequence) walks the tokens, so a
 * call's time grows with its longest sequence.
 *   qkv        [total_tokens, C] bf16 conv output (gdn_conv1d_prefill's y): q heads | k heads | v heads
 *   g          [total_tokens, Hv, Dk] fp32 per-channel log decay (16-byte aligned)
 *   g_min      the clamp: decays below exp(g_min) are raised to it (-INFINITY: no clamp; NaN is rejected)
 *   beta       [total_tokens, Hv] fp32 write strength (4-byte aligned)
 *   cu_seqlens [num_seqs + 1] int32 (device), as for gdn_conv1d_prefill; num_seqs <= 65535.
 *              Contents that are not nondecreasing within [0, total_tokens] set
 *              GDN_ERR_DEVICE_ARGUMENT in the device error word; those sequences are not computed.
 *   q_scale, l2_eps, state_in, state_out, z, norm_w, rms_eps, out: as gdn_chunk_prefill (fp32
 *              states [num_seqs, Hv, Dv, Dk]; state_out may be state_in; a sequence of length 0
 *              copies its state).  No workspace.
 */
GDN_API gdn_status gdn_kda_recurrence(const gdn_geometry* geo, const gdn_bf16* qkv, const float* g,
                                      float g_min, const float* beta, const int32_t* cu_seqlens,
                                      int32_t num_seqs, int32_t total_tokens, float q_scale,
                                      float l2_eps, const float* state_in, float* state_out,
                                      const gdn_bf16* z, const gdn_bf16* norm_w, float rms_eps,
                                      gdn_bf16* out, void* stream);

/*
 * Workspace bytes of gdn_kda_chunk_prefill: 256 bytes of counters, the longest-first sequence
 * order and per-sequence chunk offsets (4 bytes per sequence each, rounded up to 256), then one
 * 108,032-byte record per (64-token chunk, V head) for at most (total_tokens + 63 num_seqs) / 64
 * chunks.  0 when num_seqs <= 0.
 */
GDN_API size_t gdn_kda_chunk_prefill_workspace_size(const gdn_geometry* geo, int32_t num_seqs,
                                                    int32_t total_tokens);

/*
 * The KDA recurrence of gdn_kda_recurrence in its chunk-wise form: the same arguments, results
 * and errors, computed 64 tokens at a time on the tensor cores instead of token by token, plus a
 * workspace.  GLM-5.3-Flash kernel TDD ledger, slices I2, I2a and I4 (the chunk form matches the
 * sequential state and output at 63, 64 and 65 tokens).  Per chunk of L tokens from the state S0,
 * with gamma_t the running sum of the clamped log decays of each key channel:
 *   A_ts = beta_t sum_c k^_t k^_s e^(gamma_t - gamma_s) (s < t),  T = (I + A)^-1,
 *   E = (V - S0 (K^ o e^gamma)^T) diag(beta) T^T,
 *   O = q_scale (S0 (Q^ o e^gamma)^T + E P^T),  P_ts = sum_c q^_t k^_s e^(gamma_t - gamma_s) (s <= t),
 *   S = S0 diag(e^gamma_L) + E (K^ o e^(gamma_L - gamma))
 * A first kernel forms every (chunk, V head)'s state-independent part in parallel; a second walks
 * each (sequence, V head) through its chunks with the fp32 state in tensor memory.  Every product
 * on the state's path takes bf16 high / low pairs of both operands; o's own products plain bf16.
 * Tolerances: those of gdn_chunk_prefill.
 *   g          [total_tokens, Hv, Dk] fp32 per-channel log decay (16-byte aligned); after the clamp
 *              every value must be finite and at most 0 (a decay) -- a -INFINITY log decay (with
 *              g_min = -INFINITY) makes that chunk's results NaN: clamp it, or use
 *              gdn_kda_recurrence
 *   workspace  256-byte aligned device memory of gdn_kda_chunk_prefill_workspace_size() bytes
 *              (GDN_ERR_WORKSPACE if NULL or smaller), overwritten
 *   num_seqs   at most 2^31 / Hv; cu_seqlens outside [0, total_tokens] or decreasing set
 *              GDN_ERR_DEVICE_ARGUMENT in the device error word, those sequences are not computed
 *   everything else as gdn_kda_recurrence.  Everything runs on `stream`.
 */
GDN_API gdn_status gdn_kda_chunk_prefill(const gdn_geometry* geo, const gdn_bf16* qkv, const float* g,
                                         float g_min, const float* beta, const int32_t* cu_seqlens,
                                         int32_t num_seqs, int32_t total_tokens, float q_scale,
                                         float l2_eps, const float* state_in, float* state_out,
                                         const gdn_bf16* z, const gdn_bf16* norm_w, float rms_eps,
                                         gdn_bf16* out, void* workspace, size_t workspace_bytes,
                                         void* stream);

/*
 * The KDA prefill in one call: gdn_conv1d_prefill (its output written to qkv), then
 * gdn_kda_chunk_prefill on it.  Same arguments, results and errors as the two calls in sequence
 * (qkv: [total_tokens, C] bf16, must not overlap x; conv_state_out may alias conv_state_in;
 * workspace as for gdn_kda_chunk_prefill), with every argument of both stages checked before
 * either is launched: a call that returns an error has launched nothing.
 */
GDN_API gdn_status gdn_kda_prefill(const gdn_geometry* geo, const gdn_bf16* x, const gdn_bf16* conv_w,
                                   const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                                   const gdn_bf16* conv_state_in, gdn_bf16* conv_state_out,
                                   gdn_bf16* qkv, const float* g, float g_min, const float* beta,
                                   float q_scale, float l2_eps, const float* state_in,
                                   float* state_out, const gdn_bf16* z, const gdn_bf16* norm_w,
                                   float rms_eps, gdn_bf16* out, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Capacity of the fixed scratch used by gdn_chunk_prefill_noalloc. */
#define GDN_NOALLOC_MAX_SEQS 16384
#define GDN_NOALLOC_SCRATCH_BYTES (256 + 4 * GDN_NOALLOC_MAX_SEQS) /* 65,792 bytes */

/*
 * gdn_chunk_prefill for callers that cannot allocate device memory when they call it -- for
 * example a host that hands all device memory to its own pool up front, or a latency-critical
 * loop where cudaMalloc/cudaFree (which can synchronise the device) are not allowed.  Same
 * arguments, results and errors as gdn_chunk_prefill, without the workspace pair: the call
 * allocates nothing and calls no allocating routine.
 *
 * Its scratch is one fixed device array of GDN_NOALLOC_SCRATCH_BYTES inside the library, which
 * every GPU that loads the library keeps until the process exits; it holds the schedule of up to
 * GDN_NOALLOC_MAX_SEQS sequences, and a larger num_seqs is refused with GDN_ERR_INVALID_ARGUMENT
 * (nothing launched).  The first call on a device looks up that array's device address with the
 * device current (cudaGetSymbolAddress) and the kernels' launch attributes, which under lazy
 * module loading may load the library's module and reserve its static arrays on that device:
 * make this first call before any stream capture, and before a caller's pool takes the device
 * memory it will not give back.  The address is kept per device index for the life of the
 * process; after cudaDeviceReset it is stale, and the call must not be used again.  Host threads
 * making their first call at the same time store the same address (the cache is atomic).
 * All calls on a device share
 * the array and it keeps the last call's contents: each call rewrites the whole schedule and
 * zeroes its work counter before the main kernel reads them, but two calls whose kernels overlap
 * on the GPU (for example on two unordered streams) race on the array and give wrong results.
 * The scratch holds the minimum workspace only, so the call runs gdn_chunk_prefill's one-kernel
 * path.  There is no counterpart of this entry point on the pages.
 */
GDN_API gdn_status gdn_chunk_prefill_noalloc(const gdn_geometry* geo, const gdn_bf16* qkv, const float* g,
                                             const float* beta, const int32_t* cu_seqlens, int32_t num_seqs,
                                             int32_t total_tokens, float q_scale, float l2_eps,
                                             const float* state_in, float* state_out, const gdn_bf16* z,
                                             const gdn_bf16* norm_w, float rms_eps, gdn_bf16* out,
                                             void* stream);

/* ------------------------------------------------------------------------------------------------
 * Softmax attention over a paged key/value cache: the attention layers that stand between the GDN
 * layers of a hybrid model (Qwen3.8 kernel architecture and TDD ledger, "Current dense-27B kernel
 * map": d256 grouped-query attention, KV cache, 8-bit KV, batched KV writes).
 *
 *   q, k, v --gdn_attn_prepare--> q' and the sequence's pages    (norm, rotation, quantisation)
 *   q', pages --gdn_attn_prefill / gdn_attn_decode_step--> out    (optionally gated by sigmoid(z))
 *   pages --gdn_attn_cache_read--> k, v                           (dense rows)
 *
 * Positions.  Sequence n has kv_lens[n] positions in its cache, its new tokens (the rows
 * cu_seqlens[n] .. cu_seqlens[n+1]-1 of the call) among them as the last ones: new token i of q_len
 * has position p = kv_lens[n] - q_len + i.  cu_seqlens NULL means one token for every sequence
 * (total_tokens = num_seqs, token n is sequence n's).  A token with p < 0 has no place in the cache:
 * gdn_attn_prepare writes none of it there, and no key is visible to it.  A sequence with
 * kv_lens[n] = 0 (an unused slot of a fixed-size batch) is thus allowed, whatever its table row
 * holds.  Rows from cu_seqlens[num_seqs] on are left as they were.
 *
 * Pages.  Position p of sequence n lies in page block_table[n * max_pages + p / page_size], row
 * p % page_size.  Pages may be shared by sequences that only read them; two tokens of one call must
 * not write the same row.  Device-side faults -- a page that is needed and lies outside
 * [0, num_pages), kv_lens[n] outside [0, max_pages * page_size] or above 2^31 - 256, bad cu_seqlens -- set
 * GDN_ERR_DEVICE_ARGUMENT in the device error word; nothing is written for those tokens by
 * gdn_attn_prepare, and the rows of such a sequence are unspecified in the other calls.
 *
 * This build supports head_dim 128 and 256, num_q_heads a multiple of num_kv_heads with at most 64
 * query heads to a key head, at most 256 query heads, and pages of 16, 32, 64 or 128 rows. */
typedef struct {
  int32_t num_q_heads;  /* Hq: query head h reads key head h / (Hq / Hkv) */
  int32_t num_kv_heads; /* Hkv */
  int32_t head_dim;     /* D: 128 or 256 */
} gdn_attn_geometry;

#define GDN_CACHE_BF16 0 /* bf16 rows                                                          */
#define GDN_CACHE_E4M3 1 /* e4m3 codes with one power of two for each row of a key head         */

/* The page pool of one layer.  An e4m3 row x of D values is held as codes c and a byte b with
 * x ~ c * 2^(b - 127): with a the row's largest finite magnitude, 2^(b - 127) is the least power of
 * two (2^-117 or more) with a <= 448 * 2^(b - 127), and c is x * 2^(127 - b) rounded to the nearest
 * e4m3 (ties to even).  Values that are not finite become NaN.  The value of a code is exact in
 * bf16 (one that was rounded up to 2^128, from a magnitude above 1.9375 * 2^127, reads as an infinity). */
typedef struct {
  int32_t type;      /* GDN_CACHE_BF16 or GDN_CACHE_E4M3 */
  int32_t page_size; /* rows of a page: 16, 32, 64 or 128 */
  int32_t num_pages;
  void* k;           /* [num_pages, Hkv, page_size, D] bf16 or e4m3 (16-byte aligned) */
  void* v;           /* the same */
  uint8_t* k_scale;  /* [num_pages, Hkv, page_size] exponent bytes (E4M3, 16-byte aligned; NULL for BF16) */
  uint8_t* v_scale;  /* the same */
} gdn_kv_cache;

/* Position rotation of the first rot_dim values of a head (0: none): with theta_j = p * freqs[j],
 * j < rot_dim / 2, and the pair (a, b) = (x_j, x_{j + rot_dim/2}), or (x_{2j}, x_{2j+1}) when
 * interleaved, becomes (a c - b s, b c + a s) with c = magnitude * cos theta, s = magnitude * sin theta. */
typedef struct {
  int32_t rot_dim;     /* a multiple of 16, at most D */
  int32_t interleaved; /* 0: halves, 1: neighbours */
  float magnitude;
  const double* freqs; /* [rot_dim / 2] radians for each position (device, 8-byte aligned, finite, |f| <= 2 pi) */
} gdn_rope;

#define GDN_ROPE_PLAIN 0  /* f_j = base^(-2j / rot_dim)                                                       */
#define GDN_ROPE_LINEAR 1 /* f_j / factor: positions interpolated                                             */
#define GDN_ROPE_BASE 2   /* the plain f_j of base * factor^(rot_dim / (rot_dim - 2)): the lowest is f / factor */
#define GDN_ROPE_RAMP 3   /* by the turns r_j = original_positions * f_j / (2 pi): f_j where r_j >= high,
                             f_j / factor where r_j <= low, between them in proportion to r_j; the
                             magnitude is 0.1 ln(factor) + 1 (1 for factor <= 1) */
typedef struct {
  int32_t kind;
  double base, factor;
  double original_positions, low, high; /* GDN_ROPE_RAMP */
} gdn_rope_scaling;

/* Host function: fills freqs[rot_dim / 2] and *magnitude (host memory) for gdn_rope.  rot_dim is
 * positive and even (at least 4 for GDN_ROPE_BASE), base > 0, factor > 0, low < high. */
GDN_API gdn_status gdn_attn_rope_frequencies(int32_t rot_dim, const gdn_rope_scaling* scaling, double* freqs,
                                             double* magnitude);

/*
 * What the attention reads, from the projections, in one pass: every query and key head normalised
 * and rotated, the queries written to q_out and the keys and values to the sequences' pages.
 *   y = x * (mean_d x^2 + rms_eps)^(-1/2) * w   (y = x when w is NULL), then the rotation of gdn_rope,
 * computed in fp32 and rounded once to bf16; an e4m3 cache quantises the rounded keys and the values.
 *   q          Hq heads of D bf16 for each token, head h of token t at q + t * q_token_stride +
 *              h * q_head_stride (elements, multiples of 8); NULL: keys and values alone
 *   k, v       Hkv heads each, the same way
 *   q_norm_w, k_norm_w  [D] bf16, or NULL for no norm
 *   rope       NULL or rot_dim 0: no rotation.  Angles are formed to about 2^-23 turns at positions below
 *              2^24 (2^-18 at any) without fp64 arithmetic in the token loop
 *   q_out      [total_tokens, Hq, D] bf16; may be q itself where q has that layout, and overlaps nothing
 *              else that the call reads or writes
 */
GDN_API gdn_status gdn_attn_prepare(const gdn_attn_geometry* geo, const gdn_bf16* q, int64_t q_token_stride,
                                    int64_t q_head_stride, const gdn_bf16* k, int64_t k_token_stride,
                                    int64_t k_head_stride, const gdn_bf16* v, int64_t v_token_stride,
                                    int64_t v_head_stride, const gdn_bf16* q_norm_w,
                                    const gdn_bf16* k_norm_w, float rms_eps, const gdn_rope* rope,
                                    const gdn_kv_cache* cache, const int32_t* block_table,
                                    int32_t max_pages, const int32_t* kv_lens, const int32_t* cu_seqlens,
                                    int32_t num_seqs, int32_t total_tokens, gdn_bf16* q_out, void* stream);

/*
 * Rows of the cache as dense bf16 (exact for both cache types): output rows cu_seqlens[n] ..
 * cu_seqlens[n+1]-1 receive positions starts[n], starts[n] + 1, ... of sequence n (starts NULL: 0).
 *   k_out, v_out  [total_tokens, Hkv, D] bf16; must not overlap each other or the cache
 * Positions outside [0, max_pages * page_size) or on a bad page set GDN_ERR_DEVICE_ARGUMENT; their
 * rows are left as they were.
 */
GDN_API gdn_status gdn_attn_cache_read(const gdn_attn_geometry* geo, const gdn_kv_cache* cache,
                                       const int32_t* block_table, int32_t max_pages,
                                       const int32_t* starts, const int32_t* cu_seqlens, int32_t num_seqs,
                                       int32_t total_tokens, gdn_bf16* k_out, gdn_bf16* v_out, void* stream);

/* Bytes of device workspace of the two attention calls (0 for an unsupported geometry); it needs no
 * initialisation and is dead when the call's kernels finish. */
GDN_API size_t gdn_attn_workspace_size(const gdn_attn_geometry* geo);

/*
 * Causal attention of the new tokens of packed sequences over their caches (which hold the new tokens
 * too: gdn_attn_prepare first).  With p the token's position and j = 0 .. p:
 *   s_j = softmax_scale * q . k_j,   o = sum_j e^(s_j) v_j / sum_j e^(s_j)   (0 when p < 0),
 *   out = o, or o * sigmoid(z) where z is given; softmax_scale is positive, at most 1e38.
 * A key or value that is not finite reaches the tokens that see its position, and no others.
 * Scores and sums are fp32 with a running maximum; the weights e^(s_j - max) are rounded to bf16
 * for the product with v.  Beside an e4m3 cache the matrix operands are binary16, which holds every code
 * exactly: the queries are rounded to it (divided by a power of two), and the weights.  Few query heads and one
 * token a sequence: the weights times the power of two of v_j, relative to the largest of 16 or 32 keys (2^-31
 * of the largest value there is lost at most).  Otherwise: keys and values relative to the largest power of
 * two of a block of 128; rows up to 2^22 below it are exact, and rows 2^32 or more below it count as zero
 * (less than 2^-30 of the block's largest key or value).
 *   q          [total_tokens, Hq, D] bf16
 *   z          Hq heads of D bf16 for each token, head h of token t at z + t * z_token_stride +
 *              h * z_head_stride (elements, multiples of 8), or NULL
 *   out        [total_tokens, Hq, D] bf16; must not overlap q, z or the cache
 *   workspace  256-byte aligned device memory of gdn_attn_workspace_size() bytes; calls that may
 *              overlap on the GPU (other streams, graphs replayed together) need one each
 */
GDN_API gdn_status gdn_attn_prefill(const gdn_attn_geometry* geo, const gdn_bf16* q, const gdn_kv_cache* cache,
                                    const int32_t* block_table, int32_t max_pages, const int32_t* kv_lens,
                                    const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                                    float softmax_scale, const gdn_bf16* z, int64_t z_token_stride,
                                    int64_t z_head_stride, gdn_bf16* out, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* The same for one new token of each of `batch` sequences: q, out [batch, Hq, D], row n is sequence n's. */
GDN_API gdn_status gdn_attn_decode_step(const gdn_attn_geometry* geo, const gdn_bf16* q,
                                        const gdn_kv_cache* cache, const int32_t* block_table,
                                        int32_t max_pages, const int32_t* kv_lens, int32_t batch,
                                        float softmax_scale, const gdn_bf16* z, int64_t z_token_stride,
                                        int64_t z_head_stride, gdn_bf16* out, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * What stands around the layers in 8 bits: the projections' products and the expert layers (Qwen3.8 kernel
 * architecture and TDD ledger, "Current dense-27B kernel map": 8-bit projections; spark_model layer_struct.rs: per-group
 * activation quantisation, 8-bit products; GLM-5.3-Flash and Flash-Next ledgers: expert layers).
 *
 *   x --gdn_fp8_quantize--> codes, scales --gdn_fp8_matmul--> rows of the product
 *   x --gdn_moe_step--> the expert layer's rows, for a few tokens
 *
 * A matrix in 8 bits is e4m3 codes with an fp32 scale for each block of GDN_FP8_BLOCK columns and 1 row (activations) or
 * GDN_FP8_BLOCK rows (weights); the last blocks of a row or column may be narrower.  An element's value is
 * code * scale. */
#define GDN_FP8_BLOCK 128

/*
 * Codes and scales of bf16 rows.  Over each block of block_rows x 128 elements
 *   scale = max(max |x| / 448, 2^-126),   code = x / scale rounded to the nearest e4m3 (ties to even), at most 448,
 * in IEEE fp32 divisions.  A block with a NaN has the scale NaN; one with an infinity the scale infinity, and the
 * infinity's code is NaN: a product with it is NaN in that row, and in that row alone.
 *   x            rows x cols bf16, row r at x + r * x_row_stride (elements, any stride >= cols)
 *   block_rows   1 or GDN_FP8_BLOCK
 *   codes        row r at codes + r * codes_row_stride (bytes, a multiple of 16, >= cols); the bytes between cols and
 *                the stride are left as they were
 *   scales       [ceil(rows / block_rows), ceil(cols / 128)] fp32
 * The outputs overlap neither x nor one another.  rows == 0 is a no-op that returns GDN_OK; cols >= 1.
 */
GDN_API gdn_status gdn_fp8_quantize(const gdn_bf16* x, int64_t x_row_stride, int32_t rows, int32_t cols,
                                    int32_t block_rows, uint8_t* codes, int64_t codes_row_stride, float* scales,
                                    void* stream);

#define GDN_OUT_BF16 0
#define GDN_OUT_F32 1

/*
 * Activations times weights, both in 8 bits:
 *   out[t, j] = sum_b x_scale[t, b] w_scale[j / 128, b] sum_{i in block b} x[t, i] w[j, i]
 * Each block's products are summed in fp32 on the tensor cores, scaled by the product of the two scales in fp32, and added
 * up in fp32; the sum is rounded once to bf16, or not at all.  The order of the sums depends on the sizes alone.
 *   x        tokens rows of k codes, x_row_stride bytes apart (a multiple of 16, >= k)
 *   x_scale  [tokens, ceil(k / 128)] fp32
 *   w        n rows of k codes, w_row_stride bytes apart (a multiple of 16, >= k)
 *   w_scale  [ceil(n / 128), ceil(k / 128)] fp32
 *   out      tokens rows of n bf16 or fp32 values, out_row_stride elements apart (>= n, any); overlaps no input.  What
 *            lies between n and the stride is left as it was
 * A code or a scale that is NaN makes the rows and columns it belongs to NaN, and a scale that is infinite makes them
 * infinite or NaN; no others change.
 * tokens == 0 or n == 0 is a no-op that returns GDN_OK; k >= 1.
 */
GDN_API gdn_status gdn_fp8_matmul(const uint8_t* x, int64_t x_row_stride, const float* x_scale, const uint8_t* w,
                                  int64_t w_row_stride, const float* w_scale, int32_t tokens, int32_t n, int32_t k,
                                  int32_t out_type, void* out, int64_t out_row_stride, void* stream);

/* The sizes of an expert layer: H, I and Is multiples of 16, at most GDN_MOE_MAX_WIDTH; Is = 0: no shared expert. */
typedef struct {
  int32_t hidden;       /* H  */
  int32_t inter;        /* I, of an expert */
  int32_t num_experts;  /* E, at most GDN_MOE_MAX_EXPERTS */
  int32_t shared_inter; /* Is, of the expert that every token passes */
} gdn_moe_geometry;
#define GDN_MOE_MAX_WIDTH 16384
#define GDN_MOE_MAX_EXPERTS 1024
#define GDN_MOE_MAX_TOKENS 64
#define GDN_MOE_MAX_TOP_K 16

#define GDN_WEIGHT_BF16 0
#define GDN_WEIGHT_E4M3 1 /* with a scale for each block of 128 x 128 of every [I, H] or [H, I] matrix */

/* A NaN or an infinity among an expert's matrices or scales makes the rows of the tokens that pass the expert not finite, in
 * the columns whose sums it enters, and changes no other row. */
typedef struct {
  int32_t type;                      /* of the experts' matrices, GDN_WEIGHT_* */
  const gdn_bf16* router;            /* [E, H] */
  const float* router_bias;          /* [E] added to the scores for the choice alone, or NULL */
  const void* gate_up;               /* [E, 2, I, H]: the gate's matrix, then the up projection's */
  const void* down;                  /* [E, H, I] */
  const float* gate_up_scale;        /* [E, 2, ceil(I / 128), ceil(H / 128)] (E4M3), else NULL */
  const float* down_scale;           /* [E, ceil(H / 128), ceil(I / 128)] */
  const void* shared_gate_up;        /* [2, Is, H], or NULL without a shared expert */
  const void* shared_down;           /* [H, Is] */
  const float* shared_gate_up_scale; /* [2, ceil(Is / 128), ceil(H / 128)] */
  const float* shared_down_scale;    /* [ceil(H / 128), ceil(Is / 128)] */
  const gdn_bf16* shared_gate;       /* [H]: its output is multiplied by sigmoid(x . shared_gate); NULL: by 1 */
} gdn_moe_weights;

#define GDN_SCORE_SOFTMAX 0 /* over all E experts */
#define GDN_SCORE_SIGMOID 1
typedef struct {
  int32_t top_k;       /* at most GDN_MOE_MAX_TOP_K and E */
  int32_t scoring;     /* GDN_SCORE_* */
  int32_t renormalise; /* nonzero: a token's chosen scores are divided by their sum */
  float scale;         /* multiplies the weights; finite */
} gdn_moe_routing;

/* Bytes of device workspace of the two calls for this many tokens and experts a token (0 for an unsupported geometry);
 * it needs no initialisation and is dead when the call's kernels finish. */
GDN_API size_t gdn_moe_workspace_size(const gdn_moe_geometry* geo, int32_t tokens, int32_t top_k);

/*
 * A whole mixture-of-experts layer for at most GDN_MOE_MAX_TOKENS tokens (a decode step, a speculative one):
 *   logits = x router^T;   s = softmax(logits) or sigmoid(logits);   chosen: the top_k largest s + router_bias (the
 *   logits themselves without a bias), ties to the lowest index, NaN last;   weight_e = s_e, or s_e / sum of the
 *   chosen s, times scale;
 *   f_e(x) = down_e (silu(gate_e x) * up_e x);
 *   out = sum over the chosen weight_e f_e(x) + sigmoid(x . shared_gate) f_shared(x).
 * Logits, sums and an expert's h = silu(gate) * up are fp32, and out is rounded once to bf16.  Beside GDN_WEIGHT_E4M3 an h
 * enters the down projection off by at most 2^-23 of itself or 2^-39 of the largest one of its token and expert, and a
 * token's values pass through binary16, relative to its largest finite one: those of at least 2^-32 of it are exact, and
 * smaller ones change by at most 2^-40 of it.
 * The order of the sums depends on the call's arguments alone: two calls give the same bits.
 *   x        tokens rows of H bf16, x_row_stride elements apart (a multiple of 8)
 *   ids      [tokens, top_k] int32, receives the chosen experts, largest first, or NULL
 *   weights  [tokens, top_k] fp32, receives their weights, or NULL
 *   out      [tokens, H] bf16; overlaps neither x, the weights, ids nor weights
 *   workspace  256-byte aligned device memory of gdn_moe_workspace_size() bytes; calls that may overlap on the GPU
 *              (other streams, graphs replayed together) need one each
 * A token whose x is not finite has a row that is not finite, and changes no other row.  tokens == 0 is a no-op.
 */
GDN_API gdn_status gdn_moe_step(const gdn_moe_geometry* geo, const gdn_moe_weights* w, const gdn_moe_routing* routing,
                                const gdn_bf16* x, int64_t x_row_stride, int32_t tokens, int32_t* ids, float* weights,
                                gdn_bf16* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same with the routing given: token t passes the experts ids[t, 0 .. top_k-1] with weights[t, 0 .. top_k-1].  A
 * negative id stands for no expert (one that another device has, or none: the row is the shared expert's alone, or 0);
 * an expert named twice counts with the sum of its weights.  An id >= E counts as none and sets
 * GDN_ERR_DEVICE_ARGUMENT in the device error word.  router and router_bias are not read and may be NULL.
 */
GDN_API gdn_status gdn_moe_step_routed(const gdn_moe_geometry* geo, const gdn_moe_weights* w, const int32_t* ids,
                                       const float* weights, int32_t top_k, const gdn_bf16* x, int64_t x_row_stride,
                                       int32_t tokens, gdn_bf16* out, void* workspace, size_t workspace_bytes,
                                       void* stream);

/*
 * Waits for `stream`, then reads and clears the library's device error word.  Returns GDN_OK,
 * GDN_ERR_DEVICE_ARGUMENT (a kernel skipped a sequence with bad cu_seqlens entries, or a bad page or
 * length of a paged cache, or an expert that is not there),
 * GDN_ERR_TIMEOUT (a bounded in-kernel wait ran out) or GDN_ERR_CUDA.  The word is per device
 * and shared by all streams; the kernels only ever set bits in it.
 */
GDN_API gdn_status gdn_check_device_errors(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
