/*
 * mk.h -- C ABI of the single-launch decode engine for hybrid
 * Gated-DeltaNet + full-attention language models on NVIDIA B200 (sm_100a).
 *
 * The operation behind every entry point is one token's (or a few tokens')
 * forward pass of the hybrid stack described in the launch post "OS
 * Megakernel that match M5 Max Tok/w at 2x the Throughput on RTX 3090"
 * (paragraph "Why nobody had done this yet?": DeltaNet layers with a
 * learned recurrence interleaved with full-attention layers; the kernel
 * bullet list: one dispatch for the whole forward pass, bf16 weights,
 * fp32 accumulation, fused QKV + RoPE + causal softmax + output
 * projection; the post synchronises the grid between layers, this engine
 * lets each CTA wait for exactly the data it needs instead).  The
 * recurrence is the gated delta rule of "Gated Delta Networks" (Yang,
 * Kautz & Hatamizadeh, ICLR 2025).
 *
 * Conventions shared by all entry points
 *  - Every pointer documented as "device" must point to memory of the CUDA
 *    device that was current when mk_create ran; "host" pointers are read
 *    before the call returns.
 *  - Calls are asynchronous on the stream given to mk_create unless stated.
 *  - Nothing throws across the ABI.  Every call returns an mk_status code;
 *    MK_OK is 0.  A device-side failure (a wait for another CTA's data or
 *    a pipeline wait that ran out of time) is recorded in a device error
 *    word and reported by mk_sync() until mk_reset() clears it; results of
 *    calls made after such an error are undefined until then.  mk_reset()
 *    clears the error, the recurrent state and the KV cache.
 *  - Tensors are row-major.  bf16 values are IEEE bfloat16 bit patterns.
 */
#ifndef MK_H
#define MK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MK_MAX_LAYERS 64

typedef enum {
  MK_OK = 0,
  MK_ERR_ARG = 1,          /* bad argument, shape, alignment or NULL        */
  MK_ERR_CTX_OVERFLOW = 2, /* the call would write past max_ctx             */
  MK_ERR_STATE = 3,        /* call not valid in the engine's current state  */
  MK_ERR_LAUNCH = 4,       /* cooperative launch impossible / failed        */
  MK_ERR_TIMEOUT = 5,      /* a device-side wait gave up (error word set)   */
  MK_ERR_CUDA = 6,         /* another CUDA runtime error                    */
  MK_ERR_UNSUPPORTED = 7,  /* shape outside what the kernels implement      */
  MK_ERR_RANGE = 8         /* a decode partial sum left the fixed-point range
                              of the split-K reduction (|value| >= 8192)     */
} mk_status;

/* Model shape.  Layer l is full attention when layer_is_attn[l] != 0 and a
 * Gated-DeltaNet layer otherwise.  Shapes the decode kernel is built for:
 * hidden % 256 == 0 and <= 2048; conv_k == 4; mlp % 8 == 0 and <= 4096; the embedding
 * tied to the LM head; q_heads == 4 * kv_heads; and (dn_dk == dn_dv,
 * head_dim) one of (64, 64), (128, 128), (128, 256); mlp and
 * q_heads * head_dim divisible by dn_heads (the decode groups' K blocks,
 * each a multiple of 8 and the attention block at most 256 wide); at least
 * one SM per DeltaNet head.  mk_create returns MK_ERR_UNSUPPORTED otherwise
 * (also when a CTA's share of a phase exceeds the kernel's shared-memory
 * staging). */
typedef struct {
  int32_t n_layers;
  uint8_t layer_is_attn[MK_MAX_LAYERS];
  int32_t hidden, vocab, mlp;
  int32_t dn_heads, dn_dk, dn_dv, conv_k;
  int32_t q_heads, kv_heads, head_dim;
  float rope_theta, rms_eps;
  int32_t max_ctx;     /* KV-cache capacity in positions                    */
  int32_t max_verify;  /* most tokens one mk_verify call may carry (<= 8)   */
} mk_config;

/* Device pointers of one layer's weights.  bf16 matrices are [out][in];
 * every pointer must be 16-byte aligned.  Members of the other layer kind
 * are ignored and may be NULL.
 *   attn_norm [H], mlp_norm [H]            pre-mixer / pre-MLP RMSNorm gains
 *   in_proj   [2*nh*dk + 2*nh*dv + 2*nh][H] DeltaNet rows q | k | v | z | b | a
 *   conv_w    [2*nh*dk + nh*dv][conv_k]    causal conv taps of q | k | v
 *   A_log, dt_bias [nh] (float32)          decay parameters
 *   out_norm  [dv]                         gated-RMSNorm gain (shared by heads)
 *   out_proj  [H][nh*dv]                   DeltaNet output projection
 *   w_q [q_heads*hd][H], w_k, w_v [kv_heads*hd][H], w_o [H][q_heads*hd]
 *   w_gate, w_up [mlp][H], w_down [H][mlp] SwiGLU MLP                      */
typedef struct {
  const void *attn_norm;
  const void *in_proj, *conv_w;
  const float *A_log, *dt_bias;
  const void *out_norm, *out_proj;
  const void *w_q, *w_k, *w_v, *w_o;
  const void *mlp_norm;
  const void *w_gate, *w_up, *w_down;
} mk_layer_weights;

/* embed [vocab][H] bf16 (also the LM head: tied), final_norm [H] bf16,
 * layers: host array of n_layers entries. */
typedef struct {
  const void *embed;
  const void *final_norm;
  const mk_layer_weights *layers;
} mk_weights;

typedef struct mk_engine mk_engine;

/* Bytes of device workspace mk_create needs for this config (recurrent
 * state buffers, verify records, KV cache, activations, exchange words, and the
 * decode kernel's copies of the layer weights, see mk_create).
 * Returns 0 for an invalid config. */
size_t mk_workspace_bytes(const mk_config *cfg);

/* Create an engine on the current CUDA device for the hybrid stack of the
 * launch post "OS Megakernel that match M5 Max Tok/w at 2x the Throughput on
 * RTX 3090" (kernel bullet list: the whole forward pass of one token in one
 * dispatch).  `workspace` (device, at
 * least mk_workspace_bytes(cfg) bytes, 256-byte aligned) and the weights
 * stay owned by the caller and must outlive the engine; the engine only
 * keeps pointers.  `cuda_stream` (a cudaStream_t, may be NULL for the
 * legacy stream) is the stream every later call runs on.  Checks that one
 * CTA of the decode kernel fits on every SM (cooperative co-residency) and
 * returns MK_ERR_LAUNCH otherwise.  Copies weights into the workspace in
 * the layouts the decode kernel's CTA groups read (one group per DeltaNet
 * head): each attention layer's w_q, w_k and w_v as one [q|k|v][hidden]
 * matrix, each DeltaNet head's in_proj rows (q|k|v|z|b|a of that head) as
 * one block, and every out_proj, w_o and w_down split into dn_heads column
 * blocks; later changes to the caller's weights need a new engine.  Zeroes
 * the state (as mk_reset). */
int mk_create(const mk_config *cfg, const mk_weights *w, void *workspace,
              size_t ws_bytes, void *cuda_stream, mk_engine **out);

/* Destroy the host handle (NULL is allowed).  Does not free caller memory. */
void mk_destroy(mk_engine *e);

/* Zero the DeltaNet and conv states, empty the KV cache, clear a device
 * error, any pending verify and any accepted positions not yet replayed:
 * the start of a new sequence (launch post,
 * "Why nobody had done this yet?": the DeltaNet layers carry a recurrent
 * state and the attention layers a KV cache from token to token).  Weights
 * are untouched. */
int mk_reset(mk_engine *e);

/* Run n prompt tokens (host array, values in [0, vocab)) through the stack
 * at positions pos .. pos+n-1 and leave the state and KV cache as n decode
 * steps would, up to rounding (launch post "OS Megakernel that match M5 Max
 * Tok/w at 2x the Throughput on RTX 3090", results table: prompt processing
 * "pp520" beside decode).  When n-1 >= 8 the first n-1 positions run as
 * chunks of up to 1024 positions: every projection one tensor-core GEMM
 * (bf16 weights; each fp32 activation as a bf16 hi + lo pair; fp32
 * accumulation), the causal conv and gated delta rule scanned position by
 * position, causal attention over cache + chunk.  The last position is
 * always one decode step, so its logits and greedy argmax come from the
 * decode kernel.  If logits_out (device, float32 [vocab]) is not NULL it
 * receives the logits of the last prompt position.  n == 0 is a no-op.
 * The host array is copied before the call returns (pageable copies
 * synchronise with the stream).  Errors: MK_ERR_ARG (token out of range),
 * MK_ERR_CTX_OVERFLOW when pos+n > max_ctx, MK_ERR_STATE while a verify is
 * pending, MK_ERR_LAUNCH / MK_ERR_CUDA on launch failures. */
int mk_prefill(mk_engine *e, const int32_t *tokens_host, int n,
               float *logits_out);

/* One decode step: the whole forward pass of `token` at the current
 * position in one cooperative launch of the persistent kernel (launch post
 * "OS Megakernel that match M5 Max Tok/w at 2x the Throughput on RTX 3090",
 * kernel bullet list: one dispatch per token instead of ~100 launches).
 * logits_out (device, float32 [vocab]) may be NULL.  The greedy argmax of
 * the step is kept on the device (see mk_generate) and can be read with
 * mk_last_argmax.  Does not synchronise the host.  Errors: MK_ERR_ARG
 * (token out of range), MK_ERR_CTX_OVERFLOW at max_ctx, MK_ERR_STATE while
 * a verify is pending, MK_ERR_LAUNCH / MK_ERR_CUDA on launch failures. */
int mk_decode_step(mk_engine *e, int32_t token, float *logits_out);

/* Greedy generation with no host round trip between tokens (the tg128
 * decode of the launch post's results table): n decode launches, the first
 * fed `first_token` (or, when first_token == -1, the device-side argmax of
 * the last decode launch, which must be at the current position: the last
 * prefill position or the last decode / generate step; MK_ERR_STATE after
 * mk_create, mk_reset, mk_set_state or mk_verify), each later one fed the
 * device-side argmax of the launch before it.  tokens_out (device, int32 [n]) receives the n argmax tokens;
 * logits_out (device, float32 [n][vocab]) may be NULL.  Other errors as
 * mk_decode_step. */
int mk_generate(mk_engine *e, int32_t first_token, int n, int32_t *tokens_out,
                float *logits_out);

/* Verify n tokens at once (1 <= n <= max_verify), the speculative-decoding
 * shape (several draft tokens checked by one forward pass, with the
 * recurrent state kept recoverable for rollback; the follow-up post
 * "업데이트: 단일 RTX 3090에서 Qwen 3.8 27B를 140 tok/s로 구동 (Megakernel:
 * KL divergence", speed list: four draft tokens checked for the cost of one
 * forward pass, greedy output unchanged): the stack runs over positions
 * pos .. pos+n-1 as one chunk -- every projection one pass over its weights
 * for the n positions, the conv and the gated delta rule advanced position
 * by position -- and writes the logits of every position to logits_out
 * (device, float32 [n][vocab], not NULL) and K/V of the n positions to the
 * cache.  Instead of the state after every position it records, per
 * DeltaNet layer and position, the normalised key, the value, alpha, beta
 * and the conv inputs (a few KB).  Positions kept by the previous
 * mk_accept are applied to the state first, inside this call.  Results
 * equal n decode steps up to rounding.  The position does not advance until
 * mk_accept.  MK_ERR_STATE while a verify is pending. */
int mk_verify(mk_engine *e, const int32_t *tokens_host, int n,
              float *logits_out);

/* Keep the first n_keep (1..n) positions of the last mk_verify and advance
 * the position by n_keep (the rollback of rejected draft tokens that exact
 * greedy speculative decoding needs; same follow-up post, accuracy
 * paragraph: greedy output stays the main model's greedy choice).  No work
 * is launched: the next call that reads the state (verify, decode,
 * generate, prefill, mk_get_state) first replays the n_keep recorded
 * positions on it, so the state after a rejected position is never
 * written.  (Without the chunk path, mk_verify falls back to one decode
 * launch per position with a full state copy after each, and mk_accept
 * selects the copy.)  MK_ERR_STATE if no verify is pending. */
int mk_accept(mk_engine *e, int n_keep);

/* Current position (number of tokens consumed). */
int mk_position(const mk_engine *e);

/* Synchronise the stream and report a recorded device-side error. */
int mk_sync(mk_engine *e);

/* Host copy of the packed argmax of the last decode/generate step:
 * the token id, or -1.  Synchronises the stream. */
int32_t mk_last_argmax(mk_engine *e);

/* Engine state I/O (checkpoint / resume and tests).  All buffers are device
 * pointers in these layouts:
 *   dn_state   [n_dn][dn_heads][dv][dk] float32
 *   conv_state [n_dn][2*nh*dk + nh*dv][conv_k-1] float32
 *   k_cache, v_cache [n_attn][kv_heads][pos][head_dim] bf16
 * mk_set_state installs a state as if `pos` tokens had been consumed;
 * mk_get_state copies the current one out (k/v caches may be NULL). */
int mk_set_state(mk_engine *e, int pos, const float *dn_state,
                 const float *conv_state, const void *k_cache,
                 const void *v_cache);
int mk_get_state(mk_engine *e, float *dn_state, float *conv_state,
                 void *k_cache, void *v_cache);

/* Residual stream after every layer for the last position processed by a
 * decode, generate or prefill call: device float32 [n_layers][hidden]. */
int mk_get_hidden(mk_engine *e, float *hidden_out);

/* Launch statistics: number of kernels the engine launched so far. */
int64_t mk_launch_count(const mk_engine *e);

/* Debug: device-side wait limit in nanoseconds (default 2e9).  A pipeline
 * wait or a wait for another CTA's data that exceeds it records
 * MK_ERR_TIMEOUT and the kernel returns early.  `fail_phase` >= 0 makes the
 * next decode launch wait, in that phase (0-based index of the launch's
 * phase sequence: five phases per layer, then the LM head), for data
 * tagged with a value no phase ever writes (or a split-K sum with one
 * contribution more than any phase adds), so the wait must run out (tests
 * of the timeout path only). */
int mk_debug_set_wait_limit(mk_engine *e, int64_t limit_ns, int fail_phase);

/* ------------------------------------------------------------------------
 * Isolated gated delta-rule step (no engine).  One launch advances B
 * sequences x heads of the recurrence by one token, in place:
 *   S <- alpha S (I - beta k k^T) + beta v k^T ,   o = S q
 * (Gated Delta Networks, the gated delta rule).
 *   S     device float32 [B][heads][dv][dk]   state, read and written
 *   q, k  device bf16    [B][heads][dk]       used as given (no renorm)
 *   v     device bf16    [B][heads][dv]
 *   alpha, beta device float32 [B][heads]
 *   o     device float32 [B][heads][dv]
 * dk == dv in {64, 128}.  `stream` is a cudaStream_t (may be NULL). */
int mk_delta_step(float *S, const void *q, const void *k, const void *v,
                  const float *alpha, const float *beta, float *o, int B,
                  int heads, int dk, int dv, void *stream);

/* The gated delta rule over a whole sequence of T positions in the
 * chunkwise-parallel form the prompt path uses ("Gated Delta Networks",
 * the WY / UT representation of a chunk of delta-rule updates: chunks of 64
 * positions prepared independently, then one pass over the chunks per slice
 * of state rows), no engine.  Results equal T consecutive steps of
 * mk_delta_step up to rounding.
 *   S      device float32 [heads][dv][dk], read and written
 *   q, k   device float32 [heads][T][dk], used as given (no renormalisation)
 *   v      device float32 [heads][T][dv]
 *   alpha, beta device float32 [heads][T]
 *   o      device float32 [heads][T][dv]   (o_t = S_t q_t)
 *   workspace device scratch, 16-byte aligned, at least
 *          mk_delta_chunked_ws_bytes(T, heads, dk) bytes (caller-owned)
 * dk == dv in {64, 128} (else MK_ERR_UNSUPPORTED); MK_ERR_ARG on NULL,
 * misaligned or short arguments.  Asynchronous on `stream`. */
size_t mk_delta_chunked_ws_bytes(int T, int heads, int dk);
int mk_delta_chunked(float *S, const float *q, const float *k, const float *v,
                     const float *alpha, const float *beta, float *o, int T,
                     int heads, int dk, int dv, void *workspace, size_t ws_bytes,
                     void *stream);

/* Debug: the prompt path's tensor-core GEMM on its own, asynchronous on
 * `stream` (a cudaStream_t, may be NULL):
 *   C[t][n] = sum_k (X_hi[t][k] + X_lo[t][k]) * W[n][k]
 *   W device bf16 [n_out][K]; X device bf16 [2][T][K], the hi operands of
 *   the activations then their lo residuals (an fp32 x is split as
 *   hi = bf16(x), lo = bf16(x - hi)); C device float32 [T][n_out]; all
 *   16-byte aligned, K a multiple of 64.
 * MK_ERR_ARG on bad sizes, MK_ERR_UNSUPPORTED if the TMA descriptors cannot
 * be encoded.  The first call on a device allocates a 4-byte device word
 * (kept for the life of the process) where a device-side wait that runs
 * out is recorded.  Every call clears that word first (stream-ordered), and
 * if a tile's wait runs out, all of C is set to NaN: the call returns
 * before the GPU runs it, so a timed-out call shows in its output, never as
 * silently wrong values. */
int mk_debug_gemm(const void *W, const void *X, float *C, int n_out, int T,
                  int K, void *stream);

/* The same GEMM as mk_debug_gemm, for callers that must not allocate device
 * memory (the pages have no counterpart): a process whose device memory is
 * fully budgeted up front, or a host loop that may not call cudaMalloc or an
 * allocating library between steps.  It allocates nothing: K is split over
 * the SMs and the ranges' partial sums go to a static device scratch array
 * of 2^21 floats (8 MiB) inside libmk.so, then are summed in a fixed order
 * into C.  T * n_out must not exceed 2^21 (else MK_ERR_ARG); other argument
 * rules and layouts as mk_debug_gemm.  The first call on a device (made
 * with that device current) looks up the scratch address with
 * cudaGetSymbolAddress; make that first call before any stream capture.
 * No partial needs to start at zero: every partial is written before it is
 * read.  The private wait-error word (also static) is cleared by every call
 * with cudaMemsetAsync before its kernels; if a range's wait runs out it is
 * set, and the reduction writes NaN to all of C instead of the sums.  Calls
 * share the scratch, so calls that overlap (other streams or threads
 * without ordering) race; serialise them. */
int mk_debug_gemm_noalloc(const void *W, const void *X, float *C, int n_out,
                          int T, int K, void *stream);

/* ---- 4-bit weights ------------------------------------------------------
 * The tag page "RTX 3090" (item on a custom engine for a 27B-class model
 * on one RTX 3090: 4-bit weights with 16-bit activations, "W4A16") credits
 * 4-bit weights for its speed, since a batch-1 decoder streams every weight
 * once per token.  Format (the page names none; this is the plain
 * group-wise symmetric reading): groups of 64 consecutive weights of a row
 * share one fp32 scale s = max|w| / 7 (0 for an all-zero group); each weight
 * is stored as the nibble q + 8 with q = clamp(rint(w / s), -7, 7) (IEEE
 * fp32 division, round half to even); weight k of a row lives in byte k / 2
 * of the row, the even weight in the low nibble.  A row of `cols` weights
 * takes cols / 2 bytes of codes and cols / 16 bytes of scales. */

/* Quantise W (device, bf16 [rows][cols], 16-byte aligned) into codes
 * (device, uint8 [rows][cols / 2], 16-byte aligned) and scales (device,
 * float32 [rows][cols / 64], 16-byte aligned).  cols must be a multiple of
 * 64 (else MK_ERR_ARG).  Asynchronous on `stream` (a cudaStream_t or NULL);
 * nothing is allocated. */
int mk_quantize_w4(const void *W, int rows, int cols, void *codes, float *scales,
                   void *stream);

/* y[t][n] = sum_k s(n, k / 64) * q(n, k) * x[t][k] for t < T, with fp32
 * activations and fp32 accumulation: every code row is read once for all T
 * rows of x.  codes / scales as mk_quantize_w4 writes them; x (device,
 * float32 [T][cols], 16-byte aligned); y (device, float32 [T][rows]).
 * 1 <= T <= 8 and cols a multiple of 64 (else MK_ERR_ARG); T * cols * 4
 * bytes must fit in 220 KB of shared memory (else MK_ERR_UNSUPPORTED).
 * Asynchronous on `stream`; allocates nothing.  The first call per device
 * and T (and any call that needs more shared memory than the earlier ones)
 * raises the kernel's shared-memory limit: serialise those calls when
 * several host threads use the library. */
int mk_gemv_w4(const void *codes, const float *scales, const float *x, int T,
               int rows, int cols, float *y, void *stream);

/* ---- an attention layer over a paged cache --------------------------------
 * Five operators for callers that serve many sequences at once (the launch
 * post's engine holds one): norm and rotation of query and key heads, writing
 * and reading a paged cache, attention of a few or many new tokens over that
 * cache, and attention of whole packed prompts.  No engine is needed.  All are
 * asynchronous on `stream` (a cudaStream_t or NULL), allocate nothing, may be
 * captured into a CUDA graph, and run on the device that is current, which
 * must hold every pointer.
 *
 * Rows are [token][head][dim] with the dims of a head side by side; `ts` and
 * `hs` are the distances between tokens and between heads in values (>= 0),
 * so that a slice of a fused projection's output is a valid argument, and with
 * a distance of 0 an input whose tokens or heads share rows (but for what the
 * attention calls say of it).  Rows that a call writes do not overlap: between
 * several tokens or heads of an output (an input turned in place is one) the
 * distance is head_dim or more (else MK_ERR_ARG).  Rows
 * start on 16-byte boundaries (base pointers and both distances; else
 * MK_ERR_ARG).  head_dim is 64, 128 or 256 (else MK_ERR_UNSUPPORTED).  A call
 * with no tokens (or an empty batch) does nothing. */
typedef enum { MK_BF16 = 0, MK_FP16 = 1, MK_FP32 = 2, MK_E4M3 = 3 } mk_dtype;

typedef enum {
  MK_ROPE_NONE = 0,   /* f_i = theta^(-2i / rot_dim)                          */
  MK_ROPE_LINEAR = 1, /* f_i / factor                                        */
  MK_ROPE_NTK = 2,    /* theta * factor^(rot_dim / (rot_dim - 2)) for theta   */
  MK_ROPE_YARN = 3,   /* f_i / factor for the pairs that turn less than `low`
                         times over original_ctx positions, f_i for those that
                         turn more than `high` times, a linear ramp over the
                         pair index between; rotations 0.1 ln(factor) + 1 long */
  MK_ROPE_BANDED = 4  /* the same two ends, the share of f_i between them
                         linear in the number of turns: (turns - low) /
                         (high - low); rotations of length 1                 */
} mk_rope_scaling;

/* How positions turn a head, filled by mk_rope_init: host memory that the
 * caller keeps and passes to mk_qk_norm_rope. */
typedef struct {
  int32_t rot_dim;      /* rotated values at the front of a head            */
  int32_t interleaved;  /* pairs (2i, 2i + 1); else (i, i + rot_dim / 2)     */
  float magnitude;      /* length of the rotation                            */
  uint64_t turns[128];  /* turns per position of pair i, f_i / 2 pi, in 2^-64 */
} mk_rope;

/* Fill *r (host).  rot_dim a multiple of 16, at most 256 (else
 * MK_ERR_UNSUPPORTED); theta > 1; factor >= 1 where `scaling` uses it;
 * original_ctx >= 1 and 0 < low < high for YARN and BANDED (else MK_ERR_ARG).
 * Arguments that `scaling` does not use are ignored. */
int mk_rope_init(mk_rope *r, int rot_dim, int interleaved, double theta,
                 int scaling, double factor, double original_ctx, double low,
                 double high);

/* RMSNorm of every query and key head over its head_dim values, then the
 * rotation of its first rot_dim values by the token's position (launch post,
 * kernel bullet list: "fused QKV + RoPE"; head norms as an option):
 *   y = x rsqrt(mean(x^2) + eps) gain;  (y_a, y_b) of pair i turned by
 *   positions[token] * turns[i] 2^-64 turns
 * in fp32, the angle in 64-bit fixed point; rounded once, on the way out.
 *   q, q_out [tokens][q_heads][head_dim], k, k_out [tokens][kv_heads][head_dim]
 *   device, of `dtype` (MK_BF16, MK_FP16 or MK_FP32); an output may be its
 *   input (the same pointer and distances), and must not overlap otherwise;
 *   q_gain, k_gain device [head_dim] of `dtype`, 16-byte aligned; NULL: no
 *   norm of that side.  kv_heads == 0: k and k_out are ignored.
 *   positions device int32 [tokens], of any sign.
 * rot_dim must not exceed head_dim (MK_ERR_ARG). */
int mk_qk_norm_rope(const mk_rope *rope, const void *q, int64_t q_ts,
                    int64_t q_hs, const void *k, int64_t k_ts, int64_t k_hs,
                    const void *q_gain, const void *k_gain,
                    const int32_t *positions, void *q_out, int64_t qo_ts,
                    int64_t qo_hs, void *k_out, int64_t ko_ts, int64_t ko_hs,
                    int tokens, int q_heads, int kv_heads, int head_dim,
                    float eps, int dtype, void *stream);

/* A paged cache of keys and values: n_pages pages of page_size positions
 * (16, 32, 64, 128 or 256; else MK_ERR_UNSUPPORTED), device memory of the
 * caller.  The row of (page, head, position) starts page * page_stride +
 * head * head_stride + position * pos_stride values into k and into v, 16-byte
 * aligned; rows do not overlap.  dtype MK_BF16 or MK_FP16, or MK_E4M3 with one
 * float scale for each row in k_scale and v_scale (16-byte aligned),
 * [page][head][position] without gaps: a row's values are code * scale.
 * Scales are positive, normal numbers; mk_kv_write stores powers of two from
 * 2^-64 to 2^120.  An engine's
 * cache as mk_get_state copies it out is one sequence of such pages (page
 * stride page_size * head_dim, head stride pos * head_dim) when its length is
 * a multiple of the page. */
typedef struct {
  void *k, *v;
  float *k_scale, *v_scale;
  int64_t page_stride, head_stride, pos_stride;
  int32_t n_pages, page_size, kv_heads, head_dim, dtype;
} mk_kv_cache;

/* Write the rows of `tokens` tokens into a cache: token t goes to slot
 * slots[t] = page * page_size + position (device int64 [tokens]); a slot
 * outside the cache (-1 for padding) skips its token.  Slots of one call are
 * distinct: two tokens with one slot leave a mixture of their rows and scales
 * there, and nothing else is touched.  k, v device
 * [tokens][kv_heads][head_dim] of dtype MK_BF16, MK_FP16 or MK_FP32, rounded
 * to nearest even.  For an e4m3 cache the scale of a row is the least power of
 * two, 2^-64 at least, that brings its largest magnitude to 448 or below;
 * NaN stays NaN; a row with an infinity gets the scale 2^120, with which the
 * largest code reads back as infinity and small values as 0. */
int mk_kv_write(const mk_kv_cache *cache, const void *k, int64_t k_ts,
                int64_t k_hs, const void *v, int64_t v_ts, int64_t v_hs,
                const int64_t *slots, int tokens, int dtype, void *stream);

/* Read rows back by slot: k and v receive code * scale (or the stored value)
 * rounded to dtype; the rows of a slot outside the cache stay as they were.
 * A slot may be read more than once. */
int mk_kv_read(const mk_kv_cache *cache, const int64_t *slots, int tokens,
               void *k, int64_t k_ts, int64_t k_hs, void *v, int64_t v_ts,
               int64_t v_hs, int dtype, void *stream);

/* Bytes of device workspace (256-byte aligned) of the two attention calls
 * below for a head_dim; 0 for one that is not implemented.  It holds partial
 * results of one call: calls that may overlap (other streams, graphs that
 * replay at once) need one each.  Nothing is kept in it between calls and its
 * content does not matter. */
size_t mk_attn_ws_bytes(int head_dim);

/* Attention of new tokens over a paged cache (launch post, "Why nobody had
 * done this yet?": attention layers read a KV cache that grows by a token;
 * the follow-up post's draft tokens are chunks of a few): sequence b has its
 * new tokens in rows cu_q[b] .. cu_q[b + 1] - 1 of q and seq_lens[b] keys in
 * all, its new ones (already written) among them, in pages block_table[b][0],
 * [1], ...  New token t of T sees the keys 0 .. seq_lens[b] - T + t:
 *   out = sum_j softmax_j(scale * q . k_j) v_j
 * with products of 16-bit values and sums, maxima and exponentials in fp32;
 * the weights are rounded to 16 bits before they multiply the values.
 *   q, out [rows][q_heads][head_dim] device, dtype MK_BF16 or MK_FP16; query
 *     head h reads key head h / (q_heads / kv_heads); q_heads a multiple of
 *     the cache's kv_heads, 128 times at most (else MK_ERR_UNSUPPORTED); the
 *     cache of the same dtype or MK_E4M3; a distance of 0 between several
 *     tokens or heads of q only while q_heads / kv_heads times the new tokens
 *     of a sequence (rows / batch, rounded up) is 16 or less (else
 *     MK_ERR_UNSUPPORTED)
 *   block_table device int32 [batch][table_stride]; seq_lens device int32
 *     [batch], held to 0 .. table_stride * page_size (and to 2^30); a page
 *     number outside the cache stands for keys and values of zero
 *   cu_q device int32 [batch + 1], from 0, not decreasing, at most `rows`; batch
 *     at most 2^30 (else MK_ERR_UNSUPPORTED);
 *     rows from cu_q[batch] on are left as they were
 *   lse device float32 [rows][q_heads] or NULL: the natural logarithm of the
 *     sum of exp(scale * q . k_j)
 * A token that sees no key (seq_lens[b] < T - t) gets out = 0, lse = -inf.
 * What lies behind seq_lens[b] in a page is never part of a result, whatever
 * its bits; a key that a token does not see within seq_lens[b] must have
 * finite values.  out must not overlap an input.  Results do not depend on
 * timing: the same call gives the same bits.  One kernel, chosen by the mean
 * number of new tokens (rows / batch), serves the whole batch: a long chunk
 * beside many single tokens is faster as a call of its own.  Device-side waits
 * are bounded (2 s): rows of a tile whose wait runs out are set to NaN. */
int mk_attn_paged(const mk_kv_cache *cache, const void *q, int64_t q_ts,
                  int64_t q_hs, const int32_t *block_table, int table_stride,
                  const int32_t *seq_lens, const int32_t *cu_q, void *out,
                  int64_t o_ts, int64_t o_hs, float *lse, int rows, int batch,
                  int q_heads, float scale, int dtype, void *workspace,
                  size_t ws_bytes, void *stream);

/* Causal attention of whole prompts packed one after another (launch post,
 * results table: prompt processing; kernel bullet list: causal softmax):
 * sequence b has rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of q, k and v,
 * and its row t sees the rows 0 .. t.  k, v [rows][kv_heads][head_dim] device
 * of q's dtype; everything else as mk_attn_paged.  Heads of k and of v may share
 * their rows (k_hs or v_hs 0); tokens of k and v and tokens or heads of q that
 * do are MK_ERR_UNSUPPORTED. */
int mk_attn_packed(const void *q, int64_t q_ts, int64_t q_hs, const void *k,
                   int64_t k_ts, int64_t k_hs, const void *v, int64_t v_ts,
                   int64_t v_hs, const int32_t *cu_seqlens, void *out,
                   int64_t o_ts, int64_t o_hs, float *lse, int rows, int batch,
                   int q_heads, int kv_heads, int head_dim, float scale,
                   int dtype, void *workspace, size_t ws_bytes, void *stream);

/* Human-readable text of a status code. */
const char *mk_strerror(int status);

#ifdef __cplusplus
}
#endif
#endif /* MK_H */
