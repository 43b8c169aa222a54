/*
 * gdn.h -- C ABI of the B200 (sm_100a) gated-delta-rule token mixer.
 *
 * The mixer is the recurrent token mixer of the hybrid decoder described on
 * the Agnes-3.0-Flash pages: model card, "Architecture" table, row
 * "Delta-rule layers" (16 key heads / 48 value heads, head dim 128, a causal
 * conv of kernel 4 in front, a gated RMS-norm after, recurrent state in fp32);
 * "Agnes-3.0-Flash Deep Dive: A 33B Hybrid-Attention Multimodal Model",
 * section "Feed-Forward and Positional Encoding", paragraph on the Gated Delta
 * Rule (each step erases the key's old association and then writes the new
 * value, and a forget gate decays the memory).  Per value head h (key head h / (H_v / H_k)) and token t:
 *
 *   x_t      = [q | k | v] raw channels; y = SiLU(causal depthwise conv_4(x))
 *   q_t, k_t = per-head L2-normalised y (x / sqrt(sum x^2 + 1e-6)), q_t *= scale
 *   g_t      = -exp(A_log[h]) * softplus(a_t),  alpha_t = exp(g_t),  beta_t = sigmoid(b_t)
 *   S_t      = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T   (S: d_v x d_k, fp32)
 *   o_t      = S_t q_t
 *   out_t    = o_t / sqrt(mean(o_t^2) + 1e-6) * norm_w * SiLU(z_t)           (bf16, RNE)
 *
 * Conventions common to every call:
 *   - All tensor pointers are DEVICE pointers unless named *_host.  The caller
 *     owns every buffer; the library keeps no state between calls and
 *     allocates no memory (prefill scratch is the caller's `workspace`).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and never synchronise.  A returned GDN_OK means the work was
 *     validated and launched.
 *   - Head dim is fixed at 128 (GDN_HEAD_DIM), H_v % H_k == 0 and
 *     1 <= H_v / H_k <= 8.  Every tensor base pointer and every token stride
 *     (in bytes) must be a multiple of 16.
 *   - Layouts: q, k [T_tot][stride_q|k] with the H_k*128 head channels first;
 *     v, z [T_tot][stride_v|z] with H_v*128 channels; a, b [T_tot][stride_a|b]
 *     with H_v gate logits; out [T_tot][H_v][128] contiguous.  All bf16.
 *     conv_w bf16 [C_conv][4] with C_conv = (2 H_k + H_v) * 128 channels
 *     ordered q | k | v and tap 3 applied to the current token; A_log fp32
 *     [H_v]; norm_w bf16 [128] shared by all heads.
 *   - Recurrent state: fp32 [N][H_v][128 (d_v)][128 (d_k)], row-major.
 *     Conv state: bf16 [N][3][C_conv], the 3 most recent raw tokens, oldest first.
 *   - `err` (nullable) is a device int the kernels OR error bits into
 *     (1 = a bounded wait timed out, 2 = reserved,
 *     4 = cu_seqlens on the device disagreed with cu_seqlens_host, 8 = a decode
 *     state_slot outside the pool, 16 = an attention KV cache with no row left, 32 = an
 *     attention decode cache_len outside [0, cache_cap], 64 = (libgdn_debug.so only) a
 *     prefill kernel found a workspace access outside the workspace and skipped it, 128 = a
 *     tree's parent, an accepted node or a cache row of gdn_qk_norm_rope outside its range).
 *     It is never cleared by the library.  Read it after synchronising; gdn_err_status
 *     maps it to a gdn_status.
 *   - libgdn_debug.so exports the same calls, built with every workspace access of the
 *     prefill kernels checked against the workspace's bounds (a failed check sets bit 64
 *     and skips the access; nothing traps).  Same results as libgdn.so on valid calls.
 *   - With GDN_NVTX set in the environment (to anything but "0", read on the first
 *     call), every launching entry point pushes an NVTX range named after itself for
 *     its duration on the host (NVTX3, header-only: nothing is loaded unless a
 *     profiler injects its library).
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_HEAD_DIM 128
#define GDN_CHUNK 64
#define GDN_CONV_TAPS 4

typedef enum {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = 1,   /* null required pointer, bad count, bad shape */
  GDN_ERR_UNSUPPORTED = 2,   /* valid request this library does not implement */
  GDN_ERR_MISALIGNED = 3,    /* a pointer or stride is not 16-byte aligned */
  GDN_ERR_ALIAS = 4,         /* buffers that must be distinct overlap */
  GDN_ERR_CUDA = 5,          /* a CUDA launch failed */
  GDN_ERR_DEVICE_TIMEOUT = 6,/* a bounded device-side wait gave up (bit 1 of *err): every call is
                                asynchronous, so no call returns it; gdn_err_status maps the word */
  GDN_ERR_WORKSPACE = 7      /* workspace null or smaller than required */
} gdn_status;

/* Per-token inputs and per-layer parameters shared by all entry points. */
typedef struct {
  const void* q;          /* bf16 [T_tot] x stride_q, first H_k*128 channels used (pre-conv) */
  const void* k;          /* bf16 [T_tot] x stride_k (pre-conv) */
  const void* v;          /* bf16 [T_tot] x stride_v, first H_v*128 channels used (pre-conv) */
  const void* a;          /* bf16 [T_tot] x stride_a, H_v decay logits */
  const void* b;          /* bf16 [T_tot] x stride_b, H_v beta logits */
  const void* z;          /* bf16 [T_tot] x stride_z, H_v*128 output-gate channels */
  long long stride_q, stride_k, stride_v, stride_z, stride_a, stride_b; /* token strides, elements */
  const void* conv_w;     /* bf16 [C_conv][4] */
  const float* A_log;     /* fp32 [H_v] */
  const void* norm_w;     /* bf16 [128] */
  int H_k, H_v;
  float scale;            /* multiplies the normalised q; 1.0 = o_t = S_t q_t as written above */
  void* const* events;    /* optional timing hook (benchmarking and profiling; NULL in normal use -- an
                             addition to the plain tensor arguments of the mixer calls, kept in the
                             struct so that timing a call does not need a second entry point):
                             NULL, or caller-created cudaEvent_t handles that
                             the library records on `stream` around its kernels.  Prefill: 3 events,
                             [0] before the prep kernel, [1] between prep and scan, [2] after the
                             scan; when both phases run as one fused launch (see `schedule`), [1] is
                             recorded right after [0] and [2] after the launch.  Decode: 2 events,
                             before and after the decode kernel. */
  int schedule;           /* prefill launch plan.  1 = the chunk-parallel prep kernel, then the
                             sequential scan kernel.  2 = one launch that overlaps them chunk by
                             chunk (the scan on the launch's last CTAs, the prep on the others
                             publishing each chunk to the scan) whenever the scan's (sequence,
                             value head) units fit in half the SMs, else as 1.  0 = automatic: as 2 when the prep
                             also has at least 8 (chunk, key head) items per remaining SM, else
                             as 1.  "The SMs" are those the calling context may use (see
                             gdn_prefill_fused_plan).  Results are bitwise identical under every
                             plan. */
} gdn_inputs;

/*
 * The launch plan of a prefill: the number of scan CTAs of one overlapped launch, or 0 when
 * the prep and the scan run as two launches, for N sequences of n_chunks chunks in all, under
 * gdn_inputs.schedule `schedule`, on n_sm SMs.  The overlapped launch needs its scan CTAs
 * (N * H_v) to fit in half the SMs, so that the prep, which the scan waits for, always has SMs
 * of its own; the automatic plan (0) also wants at least 8 prep items (chunk, key head) per
 * remaining SM.  The prefill calls take n_sm from the calling context: the SMs of its SM
 * resource (a green context holds a partition of the device), scaled down by
 * CUDA_MPS_ACTIVE_THREAD_PERCENTAGE when that is set, else the device's count.  Pure host
 * function; 0 on bad arguments.
 */
int gdn_prefill_fused_plan(int H_k, int H_v, int N, long long n_chunks, int schedule, int n_sm);

/*
 * Bytes of device workspace gdn_prefill / gdn_prefill_varlen need for a batch
 * of N sequences that splits into n_chunks chunks of 64 tokens
 * (n_chunks = sum over sequences of ceil(L_n / 64)).  0 on bad arguments.
 */
size_t gdn_prefill_workspace_size(int H_k, int H_v, int N, long long n_chunks);

/*
 * Prefill of B sequences of T tokens each, packed as [B*T] tokens (sequence n
 * holds tokens n*T .. n*T+T-1).  Computes out for every token, and optionally
 * the final recurrent state and conv state of each sequence.
 * Departure from a launch that needs nothing but the tensors: the prefill takes a caller
 * `workspace`.  Its chunk-parallel phase (front end, triangular solve and the state-independent
 * products of every chunk, on all SMs at once) hands each chunk's operands to the sequential
 * phase through that scratch, which the library does not allocate itself (see
 * gdn_prefill_noalloc for callers that cannot provide one).  Both phases are described under
 * gdn_inputs.schedule.
 *   state_in   fp32 [B][H_v][128][128] or NULL (zero initial state)
 *   state_out  fp32 [B][H_v][128][128] or NULL; may equal state_in (in place)
 *   conv_in    bf16 [B][3][C_conv] or NULL (zero history)
 *   conv_out   bf16 [B][3][C_conv] or NULL; must not overlap conv_in
 *   out        bf16 [B*T][H_v][128]
 *   workspace  device scratch of gdn_prefill_workspace_size(H_k, H_v, B, B*ceil(T/64))
 *              bytes, 16-byte aligned; contents need no initialisation
 * B = 0 or T = 0 is a no-op apart from state_out = state_in and conv_out = conv_in history.
 */
gdn_status gdn_prefill(const gdn_inputs* in, int B, int T, const float* state_in, float* state_out,
                       const void* conv_in, void* conv_out, void* out, void* workspace,
                       size_t workspace_bytes, int* err, void* stream);

/*
 * gdn_prefill for tensors that live in host memory.  The per-token inputs q, k, v, a, b, z
 * of `in` (with its token strides), state_in, state_out, conv_in, conv_out and out are HOST
 * pointers, page-locked for the copies to run asynchronously; conv_w, A_log and norm_w stay
 * device pointers (the layer's weights live on the GPU).  On `stream`, in order: one copy
 * per input tensor into packed device copies held in `workspace` (after the prefill's own
 * scratch), gdn_prefill on them (the state updated in place on the device), one copy per
 * output back to the host.  Semantics, nullable arguments and errors as gdn_prefill; the
 * host buffers must stay valid and unmodified until the stream has passed the call.  Two
 * calls on two streams with two workspaces overlap one call's input copies with the other's
 * compute and output copies (the host link is full duplex).
 *   workspace  device memory of gdn_prefill_host_workspace_size(H_k, H_v, B, T) bytes,
 *              16-byte aligned, owned by the caller.
 */
size_t gdn_prefill_host_workspace_size(int H_k, int H_v, int B, int T);
gdn_status gdn_prefill_host(const gdn_inputs* in, int B, int T, const float* state_in, float* state_out,
                            const void* conv_in, void* conv_out, void* out, void* workspace,
                            size_t workspace_bytes, int* err, void* stream);

/*
 * Prefill of N variable-length sequences packed back to back.
 *   cu_seqlens       device int32 [N+1], cu[0] = 0, non-decreasing; sequence n is
 *                    tokens cu[n] .. cu[n+1]-1
 *   cu_seqlens_host  host copy of the same values (used to size the launch);
 *                    validated on the host.  The device copy is checked on the
 *                    device: cu[0] = 0, non-decreasing, and the same number of
 *                    chunks and total tokens as the host copy (otherwise nothing
 *                    is computed and *err gets bit 4)
 * Every sequence starts from its own state_in[n] / conv_in[n] (or zeros): state
 * and conv history never cross a cu_seqlens boundary.  Results for sequence n
 * are bitwise identical to a gdn_prefill of that sequence alone.  Other arguments as in gdn_prefill with leading dimension N; the
 * workspace size uses n_chunks = sum ceil((cu[n+1]-cu[n]) / 64).
 */
gdn_status gdn_prefill_varlen(const gdn_inputs* in, int N, const int* cu_seqlens,
                              const int* cu_seqlens_host, const float* state_in, float* state_out,
                              const void* conv_in, void* conv_out, void* out, void* workspace,
                              size_t workspace_bytes, int* err, void* stream);

/*
 * One decode step for N sequences, one new token each (token n of the inputs
 * belongs to sequence n, so T_tot = N).  Updates, in place,
 *   state       fp32 [N][H_v][128][128]
 *   conv_state  bf16 [N][3][C_conv]  (shifted by one token)
 * and writes out bf16 [N][H_v][128].  Inputs must not overlap state, conv_state or out.
 */
gdn_status gdn_decode_step(const gdn_inputs* in, int N, float* state, void* conv_state, void* out,
                           int* err, void* stream);

/*
 * The dense projections on either side of the mixer (hidden size 5120 -> q|k|v|z|a|b,
 * and 48*128 -> 5120; model card "Agnes-3.0-Flash Preview", "Architecture" table, rows
 * "Hidden size" and "Delta-rule layers"): C = A B^T on the tensor cores, bf16 in and out,
 * fp32 accumulation, one rounding to bf16 per output element.
 *   A  bf16 [M][lda], first K columns used        (activations, row-major)
 *   B  bf16 [N][ldb], first K columns used        (weights, one output channel per row)
 *   C  bf16 [M][ldc], first N columns written
 * K must be a multiple of 64 (GDN_ERR_UNSUPPORTED otherwise); every pointer and
 * leading dimension 16-byte aligned (GDN_ERR_MISALIGNED); C must not overlap A or
 * B (GDN_ERR_ALIAS).  M or N = 0 is a no-op.  Error bit 1 of *err: a wait inside
 * the kernel timed out.
 */
gdn_status gdn_gemm_bf16(const void* A, long long lda, const void* B, long long ldb, void* C, long long ldc, int M,
                         int N, int K, int* err, void* stream);

/*
 * One delta-rule layer around the mixer: y = out_proj(mixer(in_proj(x))) (model card
 * "Agnes-3.0-Flash Preview", "Architecture" table: hidden size 5120, delta-rule layers of
 * 16 key / 48 value heads of 128).  The pages give no layout for the projections; this
 * library's reading: the input projection's output channels are q (H_k*128) | k (H_k*128) |
 * v (H_v*128) | z (H_v*128) | a (H_v) | b (H_v), n_in of them in all; no biases.
 */
typedef struct {
  const void* w_in;       /* bf16 [n_in][ld_w_in], first `hidden` columns used */
  long long ld_w_in;
  const void* w_out;      /* bf16 [hidden][ld_w_out], first H_v*128 columns used */
  long long ld_w_out;
  const void* conv_w;     /* bf16 [C_conv][4] */
  const float* A_log;     /* fp32 [H_v] */
  const void* norm_w;     /* bf16 [128] */
  int H_k, H_v;
  int hidden;             /* model width; a multiple of 64 */
  float scale;            /* as gdn_inputs.scale */
  int schedule;           /* as gdn_inputs.schedule */
  void* const* events;    /* optional timing hook: NULL, or 4 caller-created cudaEvent_t recorded on
                             `stream` before the input projection, after it, after the mixer, and
                             after the output projection */
} gdn_layer;

/* Channels of the input projection's output: 2 H_k 128 + 2 H_v 128 + 2 H_v. */
long long gdn_layer_n_in(int H_k, int H_v);

/* Bytes of workspace gdn_layer_prefill needs for B sequences of T tokens: the
   projection output (bf16 [B T][n_in, padded to 8]), the mixer output (bf16 [B T][H_v 128])
   and the mixer's own workspace.  0 on bad arguments. */
size_t gdn_layer_workspace_size(int H_k, int H_v, int B, int T);

/*
 * Prefill of one delta-rule layer for B sequences of T tokens (packed [B*T]):
 *   x  bf16 [B*T][ldx], first `hidden` columns used;  y  bf16 [B*T][ldy], first `hidden` written.
 * state_in / state_out / conv_in / conv_out as in gdn_prefill.  Three launches
 * groups on `stream`: gdn_gemm_bf16 (in_proj), gdn_prefill on the projection's
 * columns (no copy: strided inputs), gdn_gemm_bf16 (out_proj).  Errors as those calls;
 * y must not overlap x or the workspace.
 */
gdn_status gdn_layer_prefill(const gdn_layer* L, int B, int T, const void* x, long long ldx, const float* state_in,
                             float* state_out, const void* conv_in, void* conv_out, void* y, long long ldy,
                             void* workspace, size_t workspace_bytes, int* err, void* stream);

/* Workspace bytes of gdn_layer_decode for N sequences of T new tokens (0 on bad arguments). */
size_t gdn_layer_decode_workspace_size(int H_k, int H_v, int N, int T);

/*
 * Decode of one delta-rule layer: T = 1 .. GDN_MAX_DECODE_TOKENS new tokens for each of N
 * sequences (x bf16 [N*T][ldx], token n*T + t = new token t of sequence n) -> y bf16
 * [N*T][ldy].  Three launch groups on `stream`: gdn_gemm_bf16 (in_proj), gdn_decode_multi on
 * the projection's columns (strided, no copy) with the states in place, gdn_gemm_bf16
 * (out_proj).  state, conv_state, state_slot and n_slots as in gdn_decode_multi (state_slot
 * NULL: sequence n uses slot n and n_slots is ignored).  A state left by gdn_layer_prefill
 * (state_out, conv_out) continues here unchanged: the handoff from prefill to decode is the
 * same buffers.  L->events, when set, gets 4 records as in gdn_layer_prefill.  Errors as
 * those calls; y must not overlap the workspace.
 */
gdn_status gdn_layer_decode(const gdn_layer* L, int N, int T, const void* x, long long ldx, float* state,
                            void* conv_state, const int* state_slot, int n_slots, void* y, long long ldy,
                            void* workspace, size_t workspace_bytes, int* err, void* stream);

/*
 * The global-attention layer of the hybrid decoder (the fourth layer of every four):
 * model card "Agnes-3.0-Flash Preview", "Architecture" table, rows "Global attention"
 * and "Positions"; "Agnes-3.0-Flash Deep Dive: A 33B Hybrid-Attention Multimodal Model",
 * section "Attention Layer Details".
 * 24 query heads / 4 KV heads of dimension 256, RMS-norm on q and k, rotary position
 * on the first 64 dims of each head (positions = token index within its sequence,
 * base 1e7, pairs (i, i + 32)), causal softmax attention, output * sigmoid(gate).
 * The input projection's output channels: q (24*256) | gate (24*256) | k (4*256) | v (4*256).
 */
#define GDN_ATTN_Q_HEADS 24
#define GDN_ATTN_KV_HEADS 4
#define GDN_ATTN_HEAD_DIM 256
#define GDN_ATTN_N_IN (2 * GDN_ATTN_Q_HEADS * GDN_ATTN_HEAD_DIM + 2 * GDN_ATTN_KV_HEADS * GDN_ATTN_HEAD_DIM)
typedef struct {
  const void* w_in;       /* bf16 [GDN_ATTN_N_IN][ld_w_in], first `hidden` columns used */
  long long ld_w_in;
  const void* w_out;      /* bf16 [hidden][ld_w_out], first 24*256 columns used */
  long long ld_w_out;
  const void* q_norm_w;   /* bf16 [256] */
  const void* k_norm_w;   /* bf16 [256] */
  int hidden;             /* a multiple of 64 */
  void* const* events;    /* optional timing hook: NULL or 4 cudaEvent_t, recorded before the input
                             projection, after it, after the attention, after the output projection */
} gdn_attn_layer;

/*
 * The attention itself, for B sequences of T tokens (packed [B*T]), on given operands:
 *   q_hat  bf16 [B*T][24][256]  normalised, rotated queries
 *   k, v   bf16 [B*T][4][256]   normalised, rotated keys and values (a KV cache)
 *   g      bf16, gate of head h of token t at g + t*ld_g + h*256
 *   out    bf16 [B*T][24*256] = softmax(q_hat k^T / 16, causal within each sequence) v * sigmoid(g),
 *          query head h reading KV head h / 6.
 * The probabilities enter the tensor cores as bf16 (relative error <= 2^-8 each).
 */
gdn_status gdn_attention_prefill(const void* q_hat, const void* k, const void* v, const void* g, long long ld_g,
                                 int B, int T, void* out, int* err, void* stream);

/* Workspace bytes of gdn_attn_layer_prefill for B sequences of T tokens. */
size_t gdn_attn_layer_workspace_size(int B, int T);

/*
 * Prefill of the attention layer for B sequences of T tokens each (packed [B*T]):
 *   x  bf16 [B*T][ldx] -> y bf16 [B*T][ldy] (first `hidden` columns);
 *   k_cache, v_cache  bf16 [B][cache_cap][4][256] (cache_cap = 0: T), rows 0 .. T-1 of each
 *   sequence written: the normalised, rotated keys and the values, i.e. the layer's KV
 *   cache after the prompt (gdn_attn_layer_decode_step continues from it).
 * Launches: gdn_gemm_bf16 (in_proj), the q/k norm + rotary kernel, the flash-attention
 * kernel (tcgen05, gate in its epilogue), gdn_gemm_bf16 (out_proj).  Errors as the
 * other entry points; y, the caches and the workspace must not overlap.  The workspace
 * holds, each from a 1 KiB boundary: the projection [B*T][GDN_ATTN_N_IN], q_hat
 * [B*T][24][256] and the attention output [B*T][24*256] (readable after the call).
 */
gdn_status gdn_attn_layer_prefill(const gdn_attn_layer* L, int B, int T, const void* x, long long ldx,
                                  void* k_cache, void* v_cache, int cache_cap, void* y, long long ldy,
                                  void* workspace, size_t workspace_bytes, int* err, void* stream);

/* Workspace bytes of gdn_attn_layer_decode_step for N sequences with caches of cache_cap rows. */
size_t gdn_attn_decode_workspace_size(int N, int cache_cap);

/*
 * One decode step of the attention layer: one new token per sequence, x bf16 [N][ldx] -> y.
 *   k_cache, v_cache  bf16 [N][cache_cap][4][256]; cache_len  device int32 [N], rows in use,
 *   0 <= cache_len[n] <= cache_cap (a value outside that range is treated like a full cache,
 *   but sets bit 32 of *err instead of 16).
 * The new token's normalised, rotated key and its value go to row cache_len[n] (its rotary
 * position), its queries attend to rows 0 .. cache_len[n], and cache_len[n] grows by one,
 * all on `stream`.  A full cache (cache_len[n] == cache_cap) gives that sequence a zero row of
 * y, leaves its cache and cache_len as they were, and sets bit 16 of *err.  The attention
 * is split over blocks of 512 cache rows and merged exactly; scores and weighted sums are
 * bf16 tensor-core products with fp32 accumulation, the weights entering as a bf16 pair
 * hi + lo (about 16 significant bits), the softmax in fp32.  Workspace: the projection
 * [N][GDN_ATTN_N_IN], q_hat, the attention output [N][24*256] (each from a 1 KiB boundary),
 * then the split partials.
 */
gdn_status gdn_attn_layer_decode_step(const gdn_attn_layer* L, int N, const void* x, long long ldx, void* k_cache,
                                      void* v_cache, int cache_cap, int* cache_len, void* y, long long ldy,
                                      void* workspace, size_t workspace_bytes, int* err, void* stream);

/*
 * T = 1 .. GDN_MAX_DECODE_TOKENS new tokens for each of N sequences in one call
 * (decode with several tokens per step, e.g. verifying drafted tokens), with
 * the states held in slots of a state pool.  Token n * T + t of the inputs is
 * new token t of sequence n (T_tot = N * T); out is bf16 [N * T][H_v][128].
 * The tokens of a sequence are applied in order exactly as T gdn_decode_step
 * calls would apply them (same arithmetic: results are bitwise equal), but each
 * state row is read from HBM once and written once for all T tokens.
 *   state       fp32 [n_slots][H_v][128][128], updated in place
 *   conv_state  bf16 [n_slots][3][C_conv], updated in place (the last 3 raw tokens)
 *   state_slot  device int32 [N]: the slot of sequence n, or NULL for slot n
 *               (then n_slots >= N).  Slots must be distinct within a call.  A slot
 *               outside [0, n_slots) leaves that sequence untouched and sets bit 8
 *               of *err.
 * Inputs must not overlap state, conv_state or out.
 */
#define GDN_MAX_DECODE_TOKENS 8
gdn_status gdn_decode_multi(const gdn_inputs* in, int N, int T, float* state, void* conv_state,
                            const int* state_slot, int n_slots, void* out, int* err, void* stream);

/*
 * Decoding with a TREE of drafted tokens: T = 1 .. GDN_MAX_TREE_NODES new tokens for each of N
 * sequences, which need not follow one another.  Node t of sequence n is token n * T + t of the
 * inputs, and
 *   parent  device int32 [N][T] (NULL: a chain, parent t - 1 for node t)
 * names the token it follows: -1 the last committed token, 0 .. t - 1 an earlier node of the
 * same sequence.  Below -1 there is no node: the padding of a batch whose trees differ in size.
 * A node whose parent is absent is absent too, and a parent >= t makes the node absent and sets
 * bit 128 of *err.  An absent node's inputs are not used and its output row is zeros.
 * Every node's result is that of decoding its path (its ancestors from the root on, then
 * itself) after the committed tokens.  A verification call changes no state and no cache; the
 * commit calls then take
 *   accepted  device int32 [N], the last node of the accepted path, or -1 to accept none
 * and advance the state or the cache along the path from the root to that node.  An accepted
 * node that is absent or outside [-1, T) sets bit 128 of *err and counts as -1.
 */
#define GDN_MAX_TREE_NODES 64

/*
 * The delta-rule mixer for a tree: out bf16 [N * T][H_v][128], every node's output after its own
 * path from the state and conv state as they stand (the causal conv runs along the path too).
 * With G_t the sum of the path's log decays and e^{G_t - G_j} the decay from node j to t,
 *   u_t = beta_t (v_t - e^{G_t} S k_t - sum over ancestors j of t: e^{G_t - G_j} (k_j . k_t) u_j)
 *   o_t = e^{G_t} S q_t + sum over j = t and its ancestors: e^{G_t - G_j} (k_j . q_t) u_j,
 * so the state is read once for all nodes.  The products run on the tensor cores with operands as
 * bf16 pairs hi + lo (about 16 significant bits) and fp32 accumulation.
 *   state       fp32 [n_slots][H_v][128][128], read
 *   conv_state  bf16 [n_slots][3][C_conv], read
 *   state_slot  as in gdn_decode_multi (NULL: sequence n uses slot n, n_slots >= N); slots may
 *               repeat here.  A slot outside [0, n_slots) gives that sequence zero rows and sets bit 8.
 * in->events, when set, gets 2 records as in decode.  N = 0 is a no-op.  out must not overlap the
 * inputs, state, conv_state, state_slot or parent.
 */
gdn_status gdn_decode_tree(const gdn_inputs* in, int N, int T, const int* parent, const float* state,
                           const void* conv_state, const int* state_slot, int n_slots, void* out, int* err,
                           void* stream);

/*
 * The commit of gdn_decode_tree: applies the tokens of the accepted path, in order, exactly as
 * gdn_decode_step calls would (same arithmetic: the states are bitwise those of decoding the
 * path token by token).  in, N, T, parent: as in the gdn_decode_tree call, with the contents that q, k, v, a
 * and b had there: the path's last raw rows of q, k and v become the conv state.  (z is not read, but has to
 * be a valid argument.)
 *   state_in, conv_in    the pools as in gdn_decode_tree, read
 *   state_out, conv_out  the pools written, the same slots; each either exactly its input (in place) or
 *                        without overlap.  Slots no sequence uses stay as they were.
 *   state_slot           slots must be distinct within a call
 * A sequence that accepts nothing keeps its state (copied when not in place).
 */
gdn_status gdn_decode_tree_commit(const gdn_inputs* in, int N, int T, const int* parent, const int* accepted,
                                  const float* state_in, float* state_out, const void* conv_in, void* conv_out,
                                  const int* state_slot, int n_slots, int* err, void* stream);

/*
 * gdn_decode_tree between the layer's projections, as gdn_layer_decode: x bf16 [N*T][ldx] ->
 * y bf16 [N*T][ldy].  The workspace keeps the projected inputs: pass it, unchanged, to
 * gdn_layer_tree_commit, which advances state and conv_state in place along the accepted paths
 * (one workspace per layer between the step and its commit).  state_slot NULL: sequence n uses slot n of
 * pools that hold at least N, and n_slots is ignored.  y must not overlap the workspace, the
 * state or the conv state.  L->events, when set, gets 4 records as in gdn_layer_prefill (the commit: none).
 */
size_t gdn_layer_tree_workspace_size(int H_k, int H_v, int N, int T);
gdn_status gdn_layer_decode_tree(const gdn_layer* L, int N, int T, const int* parent, const void* x, long long ldx,
                                 const float* state, const void* conv_state, const int* state_slot, int n_slots,
                                 void* y, long long ldy, void* workspace, size_t workspace_bytes, int* err,
                                 void* stream);
gdn_status gdn_layer_tree_commit(const gdn_layer* L, int N, int T, const int* parent, const int* accepted,
                                 float* state, void* conv_state, const int* state_slot, int n_slots,
                                 const void* workspace, size_t workspace_bytes, int* err, void* stream);

/*
 * Rotary positions: pair i (of rotary_dim / 2) turns by position * theta_i,
 *   layout   GDN_ROPE_HALF pairs dims (i, i + rotary_dim / 2), GDN_ROPE_INTERLEAVED (2 i, 2 i + 1);
 *            dims from rotary_dim on are not turned
 *   scaling  GDN_ROPE_NONE    theta_i = base^(-2 i / rotary_dim)
 *            GDN_ROPE_LINEAR  theta_i / factor (positions interpolated)
 *            GDN_ROPE_NTK     base * factor^(r / (r - 2)) in place of base, r = rotary_dim
 *            GDN_ROPE_YARN    theta_i (1 - ramp_i) + theta_i / factor * ramp_i with ramp_i rising from 0 to 1
 *                             between the pairs that turn beta_fast and beta_slow times within original_len
 *                             positions: ramp_i = min(max((i - low) / (high - low), 0), 1), low = max(floor(c(beta_fast)), 0),
 *                             high = min(ceil(c(beta_slow)), r - 1), c(b) = r ln(original_len / 2 pi b) / (2 ln base);
 *                             and cosine and sine times `amplitude`, 0.1 ln(factor) + 1
 * gdn_rope_init fills the table once; the struct is then only read.  (A checkpoint that scales cosine and sine by a
 * factor of its own: store that in `amplitude` after gdn_rope_init.)  turns[i] is theta_i / 2 pi in units of
 * 2^-64 turns, so that position * turns[i] modulo 2^64 is the angle whatever the position: no angle of a
 * far position loses bits before its reduction.  Positions may be any int32.
 * head_dim: a multiple of 8, 8 .. GDN_ROPE_MAX_HEAD_DIM; rotary_dim: a multiple of 16, 0 .. head_dim (0: no
 * rotation), else GDN_ERR_UNSUPPORTED; base > 1, factor >= 1 and finite, eps >= 0, and for YaRN original_len >= 1 and
 * beta_fast > beta_slow > 0, else GDN_ERR_INVALID_ARG.
 */
#define GDN_ROPE_MAX_HEAD_DIM 256
enum { GDN_ROPE_HALF = 0, GDN_ROPE_INTERLEAVED = 1 };
enum { GDN_ROPE_NONE = 0, GDN_ROPE_LINEAR = 1, GDN_ROPE_NTK = 2, GDN_ROPE_YARN = 3 };
typedef struct {
  int head_dim, rotary_dim;
  int layout;
  float eps;          /* of the norms */
  float amplitude;    /* factor on cosine and sine */
  unsigned long long turns[GDN_ROPE_MAX_HEAD_DIM / 2];
} gdn_rope;
gdn_status gdn_rope_init(gdn_rope* rope, int head_dim, int rotary_dim, int layout, int scaling, double base,
                         double factor, int original_len, double beta_fast, double beta_slow, float eps);

/*
 * RMS norm of each head of q and k, the rotation of their positions, and the placement of k and v,
 * in one pass over n_tok tokens:
 *   q_out = rope(q / sqrt(mean q^2 + eps) * q_norm_w), k_out likewise with k_norm_w, v_out = v.
 *   q, k, v        bf16 [n_tok][ld], heads of head_dim side by side (H_q, H_kv, H_kv of them); q may be
 *                  NULL with H_q = 0, k NULL with v NULL and H_kv = 0, v NULL alone (v_out NULL too)
 *   q_norm_w, k_norm_w   bf16 [head_dim], each NULL for no norm
 *   positions      device int32 [n_tok], NULL: 0, 1, ..
 *   rows           device int64 [n_tok], the row of k_out and v_out that token t goes to, NULL: row t (n_rows >= n_tok).
 *                  Negative: not stored.  A row >= n_rows is not stored and sets bit 128 of *err.  Rows
 *                  no token names stay as they were; two tokens that name one row race.
 *   q_out bf16 [n_tok][ld_qo]; k_out [n_rows][ld_ko], v_out [n_rows][ld_vo]
 * q_out may be exactly q with the same stride (in place), and without `rows` k_out exactly k; otherwise outputs
 * overlap neither inputs nor one another.  The sums and rotations are fp32, one rounding to bf16 per output element.
 */
gdn_status gdn_qk_norm_rope(const gdn_rope* rope, long long n_tok, int H_q, int H_kv, const void* q, long long ld_q,
                            const void* k, long long ld_k, const void* v, long long ld_v, const void* q_norm_w,
                            const void* k_norm_w, const int* positions, const long long* rows, long long n_rows,
                            void* q_out, long long ld_qo, void* k_out, long long ld_ko, void* v_out, long long ld_vo,
                            int* err, void* stream);

/*
 * Attention of a tree's nodes over a KV cache: node t of sequence n sees rows 0 .. cache_len[n] - 1 of its
 * cache and, among the nodes, its ancestors and itself:
 *   out = softmax(scale q K^T) V * sigmoid(g), query head h reading KV head h / (H_q / H_kv).
 *   q_hat           bf16 [N*T][ld_q], H_q heads of head_dim
 *   k_tree, v_tree  bf16 [N*T][ld_kt], [N*T][ld_vt], H_kv heads: the nodes' own keys and values
 *   k_cache, v_cache  bf16 [N][cache_cap][H_kv][head_dim]
 *   cache_len       device int32 [N], rows in use, 0 <= cache_len[n] <= cache_cap (outside: zero
 *                   rows for that sequence and bit 32 of *err)
 *   g               bf16 [N*T][ld_g], H_q heads, or NULL for no gate
 *   out             bf16 [N*T][H_q][head_dim]
 * What rows beyond cache_len, absent nodes and nodes off a node's path hold (infinities and NaN
 * included) does not reach its output.  head_dim is 128 or 256 and H_q / H_kv at most 16 (else
 * GDN_ERR_UNSUPPORTED); scale > 0 and finite.  The probabilities enter the tensor cores as bf16 (relative error
 * <= 2^-8 each, as in gdn_attention_prefill; gdn_attn_layer_decode_step takes pairs hi + lo), sums and statistics
 * are fp32.  A row that sees a score of NaN, +inf, or nothing but -inf is NaN.  Repeated calls give bitwise equal results.
 *   workspace  device scratch of gdn_attention_tree_workspace_size bytes, 16-byte aligned, not shared
 *              with a call that may run at the same time; contents need no initialisation
 */
size_t gdn_attention_tree_workspace_size(int H_q, int H_kv, int head_dim, int N, int T);
gdn_status gdn_attention_tree(const void* q_hat, long long ld_q, const void* k_tree, long long ld_kt,
                              const void* v_tree, long long ld_vt, const void* k_cache, const void* v_cache,
                              int cache_cap, const int* cache_len, const int* parent, const void* g, long long ld_g,
                              int H_q, int H_kv, int head_dim, float scale, int N, int T, void* out, void* workspace,
                              size_t workspace_bytes, int* err, void* stream);

/*
 * The commit of gdn_attention_tree: the keys and values of the accepted path's nodes go to rows cache_len[n],
 * cache_len[n] + 1, .. of the caches, and cache_len_out[n] becomes cache_len[n] plus their number.
 *   cache_len_out   device int32 [N]; may be exactly cache_len (in place)
 * A path that does not fit the cache is not appended at all (the length stays) and sets bit 16 of *err; a
 * cache_len outside [0, cache_cap] likewise, with bit 32.  Other arguments as in gdn_attention_tree.
 */
gdn_status gdn_attn_tree_commit(const void* k_tree, long long ld_kt, const void* v_tree, long long ld_vt, int H_kv,
                                int head_dim, int N, int T, const int* parent, const int* accepted, void* k_cache,
                                void* v_cache, int cache_cap, const int* cache_len, int* cache_len_out, int* err,
                                void* stream);

/*
 * The attention layer for a tree: in_proj, q/k norm and rotary (node at depth d of its tree: position cache_len[n] + d,
 * its root at cache_len[n]), attention over the cache and the tree, out_proj.  x bf16 [N*T][ldx] -> y bf16
 * [N*T][ldy]; the caches [N][cache_cap][4][256] and cache_len are read.  The workspace keeps the nodes'
 * keys and values: pass it, unchanged, to gdn_attn_layer_tree_commit, which appends the accepted paths to the caches and
 * advances cache_len in place.  Errors as the calls above and gdn_attn_layer_decode_step.
 */
size_t gdn_attn_layer_tree_workspace_size(int N, int T);
gdn_status gdn_attn_layer_decode_tree(const gdn_attn_layer* L, int N, int T, const int* parent, const void* x,
                                      long long ldx, const void* k_cache, const void* v_cache, int cache_cap,
                                      const int* cache_len, void* y, long long ldy, void* workspace,
                                      size_t workspace_bytes, int* err, void* stream);
gdn_status gdn_attn_layer_tree_commit(int N, int T, const int* parent, const int* accepted, void* k_cache,
                                      void* v_cache, int cache_cap, int* cache_len, const void* workspace,
                                      size_t workspace_bytes, int* err, void* stream);

/*
 * Allocation-free prefill.  The pages have no counterpart to this call; it
 * exists for callers that cannot allocate device memory (code running inside a
 * memory budget fixed by a host framework, an allocator hook that must not
 * re-enter the allocator, a runtime whose memory plan is frozen before its
 * first launch).  Same inputs, outputs and results as gdn_prefill, but no
 * workspace argument: the scratch is a file-scope device array of
 * GDN_NOALLOC_SCRATCH_BYTES inside libgdn.so, which every GPU that loads the
 * library holds until the process exits.
 *   - Limit: gdn_prefill_workspace_size(H_k, H_v, B, B*ceil(T/64)) must not
 *     exceed GDN_NOALLOC_SCRATCH_BYTES (64 MiB: e.g. up to 9 chunks of 64
 *     tokens in total at 16/48 heads, 88 at 2/6 heads); larger requests return
 *     GDN_ERR_WORKSPACE and launch nothing.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.  The address is kept per device index for
 *     the life of the process: do not use this call across a cudaDeviceReset
 *     (the reset ends the context the address belongs to).
 *   - Every call on a device shares the one array and it keeps the previous
 *     call's contents (nothing in it needs to start at zero).  Calls whose work
 *     overlaps on the GPU -- on different streams, or from different host
 *     threads without ordering -- race on it; order them on one stream.
 *   - Allocates nothing: no cudaMalloc, no cudaFree, no allocating library call.
 */
#define GDN_NOALLOC_SCRATCH_BYTES (64u << 20)
gdn_status gdn_prefill_noalloc(const gdn_inputs* in, int B, int T, const float* state_in,
                               float* state_out, const void* conv_in, void* conv_out, void* out,
                               int* err, void* stream);

/* Static description of a status code. */
const char* gdn_status_string(gdn_status status);

/*
 * The status that an `err` word (read back after synchronising the stream) stands for:
 * GDN_OK for 0, GDN_ERR_DEVICE_TIMEOUT when bit 1 is set, GDN_ERR_INVALID_ARG for any
 * other bit (device cu_seqlens, a state slot or a KV-cache length the call could not use).
 */
gdn_status gdn_err_status(int err_word);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
