/*
 * gdn.h -- C ABI of the MI355X (gfx950) gated-delta-rule forward library.
 *
 * One recurrence covers every model served here. With S in R^{dk x dv} (rows are
 * key channels) and per token (or per Householder sub-step) vectors a, b in R^dk,
 * w in R^dv and a forget vector alpha in (0,1]^dk:
 *
 *     S_t = (I - a_t b_t^T) Diag(alpha_t) S_{t-1} + a_t w_t^T,     o_t = S_t^T q_t
 *
 *   FG2-GDN   a = b = sqrt(beta) . k,  w = sqrt(beta) . v,  alpha per channel
 *             (FG2-GDN, "Enhancing Long-Context Gated Delta Networks with Doubly
 *             Fine-Grained Control": summary section 2, reading notes section 2.2,
 *             eq. (11)). With beta_v given: w = sqrt(beta_v) . v (FG2-GDN+, eq. (13)).
 *   KDA       a = b = sqrt(beta) k, w = sqrt(beta) v, beta scalar, alpha per channel
 *   GDN       as KDA with a scalar alpha (GDN2-stability page, "Problem Description")
 *   DELTAPRODUCT  n_h steps per token; step i: a = k_i, b = beta_i k_i, w = beta_i v_i;
 *             the scalar gate alpha acts once per token before step 1; q is read after
 *             step n_h (DeltaProduct summary, "Approach")
 *   ASYM      GDN2 / RWKV-7-style  S' = S' D (I - eta j k^T) + eta v k^T, o = S' q
 *             (GDN2-stability page, eq. (1)); the library state is S = S'^T, so
 *             a = k, b = eta j, w = eta v, alpha = D.
 *
 * Layouts: every array is row-major and contiguous; every pointer is a device
 * pointer aligned to 16 bytes.
 *   q, o                      [B, T, H, dk] / [B, T, H, dv]
 *   k, v (all but DP)         [B, T, H, dk] / [B, T, H, dv]
 *   k, v (DELTAPRODUCT)       [B, T, H, n_h, dk] / [B, T, H, n_h, dv]
 *   FG2   alpha, beta         [B, T, H, dk];  beta_v [B, T, H, dv] (optional)
 *   KDA   alpha [B, T, H, dk];  beta [B, T, H]
 *   GDN   alpha, beta         [B, T, H]
 *   DELTAPRODUCT  alpha (gate) [B, T, H];  beta [B, T, H, n_h]
 *   ASYM  alpha (= D) [B, T, H, dk];  j [B, T, H, dk];  eta [B, T, H]
 *   s0, s_final, state        [B, H, dk, dv] float32
 * dtype covers q, k, v, alpha, beta, beta_v, j, eta and o. The state is float32.
 *
 * Ownership: the caller owns every buffer, the workspace included. The library
 * allocates nothing on the device, keeps no state between calls and may be called
 * from several host threads at once.
 *
 * Semantics: calls are asynchronous and stream-ordered (stream is a hipStream_t;
 * NULL means the default stream); they return after enqueueing and never
 * synchronise the host. Results are bitwise deterministic for equal inputs and
 * launch parameters.
 *
 * Errors: 0 is success; negative codes below. Arguments are validated before
 * anything is enqueued: on an error nothing is launched and no output is touched.
 * Out-of-domain values (beta < 0, alpha outside (0, 1]) are not checked on the
 * device; they give NaN or Inf. Decay range of the chunked path: GDN and
 * DELTAPRODUCT (one decay per step) take any alpha in (0, 1]. The per-channel
 * decays (FG2, KDA, ASYM) are factored through reference points inside each
 * 16-step tile of a chunk, so the result stays in float32 range as long as no
 * channel decays by more than e^-87 over 8 consecutive steps (for instance,
 * alpha >= 1.9e-5 at every step); stronger decay over such a window can give NaN.
 * The recurrent entry point has no such limit.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 3

enum gdn_variant {
  GDN_VARIANT_FG2 = 0,
  GDN_VARIANT_KDA = 1,
  GDN_VARIANT_GDN = 2,
  GDN_VARIANT_DELTAPRODUCT = 3,
  GDN_VARIANT_ASYM = 4
};

enum gdn_dtype { GDN_DTYPE_F32 = 0, GDN_DTYPE_BF16 = 1 };

enum gdn_status {
  GDN_OK = 0,
  GDN_ERR_ARG = -1,         /* null pointer, bad shape, misaligned pointer     */
  GDN_ERR_UNSUPPORTED = -2, /* valid but not implemented (size, chunk, n_h)   */
  GDN_ERR_WORKSPACE = -3,   /* workspace missing or smaller than required     */
  GDN_ERR_HIP = -4          /* a HIP launch reported an error                 */
};

/* GDN2 stabilisers: gdn_asym_stabilize's mode, and gdn_args.stabilize. */
enum gdn_stabilize_mode { GDN_STABILIZE_CLIP_DECAY = 1, GDN_STABILIZE_PROJECT_J = 2 };

typedef struct gdn_args {
  int32_t variant;  /* enum gdn_variant */
  int32_t dtype;    /* enum gdn_dtype   */
  int64_t B, T, H;  /* batch, tokens (T >= 0), heads                          */
  int64_t dk, dv;   /* key and value head dims, each in {16, 32, 64, 128}     */
  int32_t chunk;    /* chunk length C in {16, 32, 64} (chunked entry points);
                       fp32 with dk = 128 runs 64 as 32 (same result up to
                       rounding, workspace sized for 32)                      */
  int32_t n_h;      /* Householder steps per token (DELTAPRODUCT, 1..8), else 1;
                       chunked entry points lay a token out as n_h steps, 4 for
                       n_h = 3 and 8 for n_h = 5..7 (the extra ones identity
                       steps) and need chunk / steps >= 8 output rows a chunk:
                       n_h 1..8 with chunk 64 (fp32 with dk = 128 runs 32-step
                       chunks: n_h 1..4), n_h 1..4 with chunk 32, n_h 1..2 with
                       chunk 16; GDN_ERR_UNSUPPORTED otherwise;
                       gdn_recurrent_step takes every n_h                     */
  const void* q;
  const void* k;
  const void* v;
  const void* alpha;
  const void* beta;   /* unused by ASYM */
  const void* beta_v; /* FG2 only, optional (NULL: the value uses beta)       */
  const void* j;      /* ASYM only */
  const void* eta;    /* ASYM only */
  const float* s0;    /* initial state, NULL means zero                        */
  float* s_final;     /* final state, NULL means not written; may alias s0     */
  void* o;            /* outputs; ignored by gdn_final_state                   */
  int32_t stabilize;  /* ASYM only: 0, or a gdn_stabilize_mode applied to every
                         token's D or j inside the pass (as gdn_asym_stabilize
                         would, without its extra pass over the inputs or the
                         rounding of D' / j' to the input dtype)                */
} gdn_args;

/* Bytes of device workspace gdn_chunk_fwd / gdn_final_state need for *args
 * (0 for an invalid argument set). */
size_t gdn_workspace_bytes(const gdn_args* args);

/* Chunkwise-parallel forward pass: writes o for all T tokens and, when
 * s_final != NULL, the state after token T. The sequence is cut into chunks of
 * `chunk` steps (tokens, or Householder sub-steps for DELTAPRODUCT, whose chunk
 * must then be a multiple of n_h); inside a chunk the work is parallel (the
 * WY/UT form of the FG2-GDN reading notes, section 2.4), between chunks the state
 * is carried. T = 0 copies s0 (or zeros) to s_final. ws must hold
 * gdn_workspace_bytes(args) bytes and be 256-byte aligned. */
int gdn_chunk_fwd(const gdn_args* args, void* ws, size_t ws_bytes, void* stream);

/* Same pass computing the final state only (o is not read or written;
 * s_final must be non-NULL): the state S_T the recurrence above reaches after T
 * tokens (FG2-GDN reading notes, section 2.2 eq. (11), the state a chunked
 * prefill hands to decoding). */
int gdn_final_state(const gdn_args* args, void* ws, size_t ws_bytes, void* stream);

/* The two stages of gdn_chunk_fwd, for callers that schedule them separately
 * (gdn_chunk_fwd is exactly prepare followed by scan on one stream).
 * gdn_chunk_prepare runs the chunk-local work (decay cumsum, masked Grams, the
 * UT inverse T = (I + M)^{-1}, W = T B+, U~ = T Wv; FG2-GDN reading notes,
 * section 2.4) into ws; gdn_chunk_scan carries the state across chunks and writes
 * o and s_final. Both take the same args, ws and ws_bytes; with args->o == NULL
 * the pair computes the final state only (as gdn_final_state). ws must not be
 * modified between the two calls. */
int gdn_chunk_prepare(const gdn_args* args, void* ws, size_t ws_bytes, void* stream);
int gdn_chunk_scan(const gdn_args* args, void* ws, size_t ws_bytes, void* stream);

/* Bytes of the device buffer gdn_chunk_fwd_static keeps on each device. */
#define GDN_STATIC_SCRATCH_BYTES ((size_t)64 << 20)

/* gdn_chunk_fwd without a workspace, for callers that cannot allocate device
 * memory: code under stream capture, serving loops that must not allocate, and
 * harnesses that forbid hipMalloc. The call itself allocates nothing. The chunk
 * records live in a buffer of GDN_STATIC_SCRATCH_BYTES inside the library, one per
 * device, created when the library's code is loaded on that device and held until
 * the process ends; its device address is looked up once per device, on the first
 * call made with that device current. The sequence runs in blocks of as many
 * chunks as the buffer holds for all B*H sequences (one prepare and one scan
 * launch per block, each block starting from the state the previous one left), so
 * o and s_final are bitwise equal to gdn_chunk_fwd's for the same args.
 * Arguments, layouts and errors are those of gdn_chunk_fwd, plus
 * GDN_ERR_UNSUPPORTED when one chunk's records for all B*H sequences, plus
 * B*H*dk*dv*4 bytes for the carried state when s_final is NULL, exceed the buffer
 * (bf16, dk = dv = 128, chunk 64: 72 KiB of records per sequence, so B*H <= 910
 * with s_final given, B*H <= 481 without).
 * All calls on one device share its buffer, and the buffer keeps the last call's
 * contents: calls that may overlap on one device (several streams or host threads)
 * race and must be serialised by the caller. */
int gdn_chunk_fwd_static(const gdn_args* args, void* stream);

/* Token-sequential recurrence: advances state_inout ([B, H, dk, dv] float32,
 * updated in place) by args->T tokens, writing o for each (T = 1 is one decode
 * step): the step above applied token by token, exactly as the FG2-GDN reading
 * notes write it (section 2.2 eq. (11); section 2.1 eq. (6) for the delta rule it
 * extends; GDN2-stability page eq. (1) for ASYM; DeltaProduct summary, "Approach",
 * for the n_h sub-steps). args->s0, args->s_final and args->chunk are ignored. No
 * workspace. */
int gdn_recurrent_step(const gdn_args* args, float* state_inout, void* stream);

/* GDN2 stabilisers: token-wise transforms of the ASYM inputs that bound the spectral norm of each step's transition D (I - eta j k^T)
 * (GDN2-stability page: "The Spectral Norm" gives rho = ||I - eta j k^T||_2 in closed
 * form; "Simple Strategy" clips D; "Modifying Itself" moves j). args is an ASYM
 * argument set (variant GDN_VARIANT_ASYM, shapes as for the forward pass); only k,
 * j, alpha (= D) and eta are read, in args->dtype, and out has the same dtype.
 * The page's unit-norm j and k are not required: their norms are folded into eta.
 *   GDN_STABILIZE_CLIP_DECAY  out [B, T, H, dk] = min(D, 1/rho) per channel; then
 *                             ||D' (I - eta j k^T)||_2 <= 1.
 *   GDN_STABILIZE_PROJECT_J   out [B, T, H, dk] = j' = s k + lam (j - s k) with
 *                             s = j^T k / ||k||^2: eta j'^T k = eta j^T k (the erase
 *                             rate c is kept) and, with g = max_i D_i and
 *                             tau = (c - 1) g + 1/g, ||I - eta j' k^T||_2 <= 1/g
 *                             whenever tau >= |c|. lam = min(1, sqrt((tau^2 - c^2) /
 *                             (eta^2 ||k||^2 ||j - s k||^2))); lam = 1 when that
 *                             denominator is 0; lam = 0 when tau^2 <= c^2 (no j'
 *                             reaches the bound; only c < 0 gets there).
 * args->stabilize is ignored here; setting it on the forward entry points applies
 * the same transform inside the pass instead. out must be 16-byte aligned; it may be
 * args->alpha (mode 1) or args->j (mode 2) for an in-place update, and must not
 * overlap any other input. k = 0 rows give
 * NaN in mode 2. T = 0 does nothing. Errors: GDN_ERR_ARG for a variant other than
 * ASYM, a mode outside the enum, or a null or misaligned k, j, alpha, eta or out. */
int gdn_asym_stabilize(const gdn_args* args, int mode, void* out, void* stream);

/* Gradient outputs of gdn_recurrent_bwd, all float32, laid out like the matching
 * input (dalpha like alpha, dbeta like beta, ...; ds0 like s0). Pointers for inputs
 * the variant does not take must be NULL; the others must be non-NULL and 16-byte
 * aligned, except ds0, which may be NULL (not written). */
typedef struct gdn_grads {
  float* dq;
  float* dk;
  float* dv;
  float* dalpha;
  float* dbeta;    /* FG2, KDA, GDN */
  float* dbeta_v;  /* FG2 with beta_v */
  float* dj;       /* ASYM */
  float* deta;     /* ASYM */
  float* ds0;
} gdn_grads;

/* Bytes of device workspace gdn_recurrent_bwd needs (0 for an invalid set). Per
 * token (or sub-step) and head: the float32 step operands (4 dk + 2 dv floats), the
 * records of the 16-step chunks ((80 dk + 32 dv + dk + 512) / 16 floats), the state
 * before every even chunk and the state gradient after every odd one (dk dv / 16
 * floats) and the row gradients (4 dk + dv floats); chunks are counted in pairs. 13.2
 * KiB per token and head at dk = dv = 128: 0.88 GB for 4,096 tokens x 16 heads. */
size_t gdn_bwd_workspace_bytes(const gdn_args* args);

/* Backward pass (reverse-mode gradients) of the token recurrence for every variant
 * (FG2, FG2+, KDA, GDN, ASYM, and DELTAPRODUCT through its Householder sub-steps,
 * DeltaProduct summary, "Approach"; dalpha is then the gate's gradient [B, T, H]).
 * The pages give the forward pass only; this is the derivative of the same recurrence
 * (FG2-GDN reading notes, section 2.2 eq. (11), section 2.3 eq. (13); GDN2-stability
 * page, eq. (1)), taken through the chunkwise WY / UT form of section 2.4 on 16-step
 * chunks. gdn_args.stabilize must be 0 (GDN_ERR_UNSUPPORTED otherwise), and
 * B * H * T * n_h may not exceed 2^33 (GDN_ERR_UNSUPPORTED). args as for the forward
 * pass (o, s_final and chunk are ignored; s0 NULL means zero); d_o [B, T, H, dv] in
 * args->dtype is dL/do; d_s_final [B, H, dk, dv] float32 is dL/dS_T (NULL: zero).
 * Gradients with respect to beta and beta_v are singular at 0 (their square roots
 * enter the step). ws must hold gdn_bwd_workspace_bytes(args) bytes, 256-byte
 * aligned. Decay factors span at most 8 steps of a chunk, so, as in the chunked
 * forward pass, results stay in float32 range while no channel decays by more than
 * e^-87 over 8 consecutive steps (alpha >= 1.9e-5 at every step suffices); beyond
 * that they can overflow. Every sum has a fixed order: results are deterministic. */
int gdn_recurrent_bwd(const gdn_args* args, const void* d_o, const float* d_s_final,
                      const gdn_grads* grads, void* ws, size_t ws_bytes, void* stream);

/* ---- Linear attention with one decay a head ----------------------------------------
 *
 * The recurrence above without the erase: with S in R^{dk x dv} per value head h and a
 * constant log decay g_h <= 0,
 *
 *     S_t = e^{g_h} S_{t-1} + k_t v_t^T,     o_t = S_t^T q_t
 *
 * Layouts (row-major; pointers aligned to 16 bytes):
 *   q, k                 [B, T, Hk, dk]   key head h / (H / Hk) serves value head h
 *   v, o                 [B, T, H, dv]
 *   log_decay            [H] float32; e^{g} below e^-128 is taken as 0 (-Inf included);
 *                        values above 0 are not checked (they grow the state)
 *   seq_lens             [B] int32 on the device, or NULL: T tokens each. Sequence b has
 *                        min(max(seq_lens[b], 0), T) tokens; rows of o behind them are
 *                        left as they were, and the states are those after its last token
 *   s0, s_final, state   [B, H, dk, dv] float32
 * q, k and v may be views of a larger array: *_stride is the distance in elements from
 * one token to the next (0: contiguous), a multiple of 16 bytes and at least one token's
 * heads; the heads of a token are contiguous, and a sequence starts T strides after the
 * one before. o is contiguous and must not overlap an input.
 * GDN_ERR_UNSUPPORTED above B = 2^20, H = 2^16, B * H = 2^24, B * T = 2^36, T = 2^31 - 2^16
 * or a stride of 2^24, and from B * H * max(dk, dv) = 2^30 on (the norms below: the same
 * without the last and with T = 2^31).
 * Ownership, asynchrony, determinism and errors as above; the current device must be
 * the stream's. States are float32 sums on either type; of bf16 inputs the scores q k^T and
 * the state as it meets q enter the chunked products to 2^-16, under the rounding of o.
 * A NaN or Inf in row t of k or v makes the rows of o from t on NaN or Inf (v: in its
 * column), at least as long as the row's weight e^{g (i - t)} is over 2^-127; one in q its
 * own row of o. It never reaches an earlier row, another head or another sequence. Behind
 * that weight nothing is promised: 0 times NaN is NaN where tokens go one by one and within
 * a segment of the chunked pass, while a segment does not read rows that weigh nothing, and
 * where segments begin goes by the sizes and by whether seq_lens is given. A finite s_final of a head that
 * forgets is no sign of finite inputs. In the gradients below the same holds along each
 * formula (in dk and dv from the row backwards). Of float32 inputs, magnitudes above
 * 3.3e38 count as Inf. */
typedef struct gdn_linear_args {
  int32_t dtype;          /* enum gdn_dtype: q, k, v and o                    */
  int32_t reserved;       /* must be 0                                        */
  int64_t B, T, H, Hk;    /* sequences, tokens (T >= 0), value heads, key heads (H % Hk == 0) */
  int64_t dk, dv;         /* head dims, each in {16, 32, 64, 128}             */
  int64_t q_stride, k_stride, v_stride;
  const void* q;
  const void* k;
  const void* v;
  const float* log_decay;
  const int32_t* seq_lens;
  const float* s0;        /* NULL means zero; ignored by the step             */
  float* s_final;         /* NULL means not written; may alias s0; ignored by the step */
  void* o;
} gdn_linear_args;

/* Bytes of device workspace gdn_linear_chunk_fwd needs (0 for an invalid set). */
size_t gdn_linear_workspace_bytes(const gdn_linear_args* args);

/* Chunked pass over prompts: o for every token, and the state after the last one. The
 * sequence is cut into segments that run in parallel: one pass adds up each segment's own
 * k v^T, a second carries the state over the segments, and a third computes the outputs
 * chunk by chunk from the state before each segment (one launch where a sequence is one
 * segment; up to eight tokens go one by one). ws must hold gdn_linear_workspace_bytes(args) bytes, 256-byte aligned. */
int gdn_linear_chunk_fwd(const gdn_linear_args* args, void* ws, size_t ws_bytes, void* stream);

/* The recurrence token by token on state_inout ([B, H, dk, dv] float32, updated in
 * place): T = 1 is one decode step. A sequence of length 0 (seq_lens) keeps its state and
 * its row of o. No workspace. */
int gdn_linear_recurrent_step(const gdn_linear_args* args, float* state_inout, void* stream);

/* Gradient outputs of gdn_linear_chunk_bwd, contiguous: dq, dk [B, T, Hk, dk] and dv
 * [B, T, H, dv] in args->dtype (dq and dk summed over the value heads of a key head);
 * ds0 [B, H, dk, dv] float32, NULL means not written; none may overlap an input or
 * d_s_final. Rows behind a sequence's length are written as zero. */
typedef struct gdn_linear_grads {
  void* dq;
  void* dk;
  void* dv;
  float* ds0;
} gdn_linear_grads;

/* Bytes of device workspace gdn_linear_chunk_bwd needs (0 for an invalid set). */
size_t gdn_linear_bwd_workspace_bytes(const gdn_linear_args* args);

/* Gradients of o and s_final with respect to q, k, v and s0 (log_decay is a constant of
 * the model): with d_o [B, T, H, dv] in args->dtype (contiguous) and d_s_final
 * [B, H, dk, dv] float32 (NULL: zero),
 *     G_n = d_s_final + q_n do_n^T,  G_t = e^{g} G_{t+1} + q_t do_t^T  (t < n),
 *     dq_t = S_t do_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  ds0 = e^{g} G_1,
 * n the sequence's tokens; ds0 = d_s_final where n = 0.
 * args->o and args->s_final are ignored. Rows of d_o behind a sequence's length are not
 * used. ws must hold gdn_linear_bwd_workspace_bytes(args) bytes, 256-byte aligned. */
int gdn_linear_chunk_bwd(const gdn_linear_args* args, const void* d_o, const float* d_s_final,
                         const gdn_linear_grads* grads, void* ws, size_t ws_bytes, void* stream);

/* ---- Norms of queries and keys a head, with the position rotation --------------------
 *
 * The delta-rule and linear entry points take q and k as they are (keys of unit norm
 * where the method asks for them); this pass makes them from a projection's output. Per
 * token and head, with x a row of d channels:
 *     n = x r w,   r = (sum x^2 / d + eps)^{-1/2} (RMS) or (sum x^2 + eps)^{-1/2} (L2)
 * then channels 0 .. rot-1 of n are rotated by the token's position p in pairs (a, b),
 *     a' = a cos[p][i] - b sin[p][i],   b' = b cos[p][i] + a sin[p][i],
 * where pair i is channels (i, i + rot/2), or (2i, 2i + 1) when interleaved; queries are
 * multiplied by q_scale. Sums and products are float32, rounded once.
 *   q, k          [B, T, Hq, d], [B, T, Hk, d]; strides as for the linear entry points
 *   wq, wk        [d] float32, NULL means ones
 *   cos, sin      [n_pos, rot/2] float32 (NULL when rot == 0)
 *   positions     [B, T] int32, NULL means 0 .. T-1 (then n_pos >= T). A position outside
 *                 [0, n_pos) gives a row of NaN; nothing is read out of bounds
 *   q_out, k_out  contiguous; may be q / k themselves when those are contiguous */
enum gdn_norm { GDN_NORM_RMS = 1, GDN_NORM_L2 = 2 };

typedef struct gdn_qk_norm_args {
  int32_t dtype;        /* enum gdn_dtype: q, k, q_out, k_out                  */
  int32_t norm;         /* enum gdn_norm                                       */
  int64_t B, T, Hq, Hk; /* Hq, Hk >= 1                                         */
  int64_t d;            /* head dim in {16, 32, 64, 128}                       */
  int64_t q_stride, k_stride;
  int64_t rot;          /* rotated channels: 0, or a multiple of 8 up to d     */
  int64_t n_pos;        /* rows of cos and sin                                 */
  int32_t interleaved;  /* 0 or 1                                              */
  float eps;            /* >= 0                                                */
  float q_scale;
  int32_t reserved;     /* must be 0                                           */
  const void* q;
  const void* k;
  const float* wq;
  const float* wk;
  const float* cos;
  const float* sin;
  const int32_t* positions;
  void* q_out;
  void* k_out;
} gdn_qk_norm_args;

int gdn_qk_norm_fwd(const gdn_qk_norm_args* args, void* stream);

/* Gradients: dq_out, dk_out (contiguous, grad_dtype: args->dtype, or GDN_DTYPE_F32 as
 * gdn_recurrent_bwd returns them) in; dq, dk (contiguous, args->dtype) and dwq, dwk [d]
 * float32 (NULL: not written) out. args->q_out and k_out are ignored. The weight sums run
 * in a fixed order. */
typedef struct gdn_qk_norm_grads {
  int32_t grad_dtype;
  int32_t reserved; /* must be 0 */
  const void* dq_out;
  const void* dk_out;
  void* dq;
  void* dk;
  float* dwq;
  float* dwk;
} gdn_qk_norm_grads;

/* Bytes of device workspace gdn_qk_norm_bwd needs (0 for an invalid set). */
size_t gdn_qk_norm_bwd_workspace_bytes(const gdn_qk_norm_args* args);
int gdn_qk_norm_bwd(const gdn_qk_norm_args* args, const gdn_qk_norm_grads* grads, void* ws,
                    size_t ws_bytes, void* stream);

/* ---- Gated norm of a layer's outputs ----------------------------------------------------
 *
 * Per token and head, y = x (sum x^2 / d + eps)^{-1/2} w act(gate), act(z) = z / (1 + e^-z)
 * (SILU) or 1 / (1 + e^-z) (SIGMOID): what follows o in a gated layer.
 *   x, gate    [B, T, H, d]; strides as for the linear entry points
 *   weight     [d] float32, NULL means ones
 *   y          contiguous; may be x or gate when that is contiguous */
enum gdn_activation { GDN_ACT_SILU = 1, GDN_ACT_SIGMOID = 2 };

typedef struct gdn_gated_norm_args {
  int32_t dtype;      /* enum gdn_dtype: x, gate, y   */
  int32_t activation; /* enum gdn_activation          */
  int64_t B, T, H;
  int64_t d;          /* head dim in {16, 32, 64, 128} */
  int64_t x_stride, gate_stride;
  float eps;          /* >= 0 */
  int32_t reserved;   /* must be 0 */
  const void* x;
  const void* gate;
  const float* weight;
  void* y;
} gdn_gated_norm_args;

int gdn_gated_norm_fwd(const gdn_gated_norm_args* args, void* stream);

/* Gradients: dy (contiguous, args->dtype) in; dx, dgate (contiguous, args->dtype) and
 * dweight [d] float32 (NULL: not written) out. args->y is ignored. */
typedef struct gdn_gated_norm_grads {
  const void* dy;
  void* dx;
  void* dgate;
  float* dweight;
} gdn_gated_norm_grads;

/* Bytes of device workspace gdn_gated_norm_bwd needs (0 for an invalid set). */
size_t gdn_gated_norm_bwd_workspace_bytes(const gdn_gated_norm_args* args);
int gdn_gated_norm_bwd(const gdn_gated_norm_args* args, const gdn_gated_norm_grads* grads, void* ws,
                       size_t ws_bytes, void* stream);

/* ---- Gated recurrence a channel ----------------------------------------------------------
 *
 * A state of one number a channel instead of a matrix a head:
 *
 *     h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t,     elementwise over C channels
 *
 *   LOG      a = e^f, m = 1 (f <= 0 forgets; above 0 the state grows, as far as float32 holds it and
 *            e^f itself; long stretches of either may follow each other)
 *   SIGMOID  a = sigmoid(f), m = 1 - a
 *   POWER    a = e^{-decay_c sigmoid(f)} (decay [C] >= 0), m = sqrt(1 - a^2)
 * and without i its factor is 1. 1 - a is computed as it is, not as a difference, so that
 * channels that keep many tokens keep their last bits.
 *   x, f, i      [B, T, C], C a multiple of 8; views of a larger array by *_stride as for the
 *                linear entry points (at least C elements from token to token)
 *   h            [B, T, C], contiguous, in the inputs' type; may be x, f or i itself where that is
 *                contiguous, and must not overlap an input otherwise (GDN_ERR_ARG)
 *   seq_lens     as for the linear entry points: rows of h behind a length stay as they were
 *   h0, h_final  [B, C] float32
 *   checkpoints  [B, ceil(T / GDN_SCAN_SPAN), C] float32: the state before every span of
 *                GDN_SCAN_SPAN tokens (spans behind a length: not written). The forward pass
 *                writes them if given; the gradients read them if given, and otherwise run
 *                over x, f and i once more to get them.
 * GDN_ERR_UNSUPPORTED above C = 2^16, B * C = 2^24, and the limits of B, T, B * T and strides
 * of the linear entry points. The state is float32; a sequence's tokens are joined in a tree that
 * goes by the sizes alone. A NaN or Inf in row t makes its channel of h NaN or Inf from t on, at
 * least as long as its weight, the product of the a's since (and from any row since, where LOG has
 * a's over 1), is over 2^-127, and nothing else; behind that weight nothing is promised (0 times
 * NaN is NaN within a part of the sequence, while rows that weigh nothing are not read from the
 * next). The same holds along the gradients'
 * formulas, from a row backwards. */
enum gdn_scan_gate { GDN_SCAN_LOG = 1, GDN_SCAN_SIGMOID = 2, GDN_SCAN_POWER = 3 };
#define GDN_SCAN_SPAN 64

typedef struct gdn_scan_args {
  int32_t dtype;     /* enum gdn_dtype: x, f, i and h  */
  int32_t gate;      /* enum gdn_scan_gate             */
  int64_t B, T, C;   /* T >= 0                         */
  int64_t x_stride, f_stride, i_stride;
  const void* x;
  const void* f;
  const void* i;        /* NULL: no input gate         */
  const float* decay;   /* [C], POWER only             */
  const int32_t* seq_lens;
  const float* h0;      /* NULL means zero; ignored by the step               */
  float* h_final;       /* NULL: not written; may alias h0; ignored by the step */
  float* checkpoints;   /* ignored by the step         */
  void* h;
} gdn_scan_args;

/* Bytes of device workspace gdn_gated_scan_fwd needs (0 for an invalid set). */
size_t gdn_gated_scan_workspace_bytes(const gdn_scan_args* args);

/* h for every token and the state after the last one. ws must hold
 * gdn_gated_scan_workspace_bytes(args) bytes, 256-byte aligned. */
int gdn_gated_scan_fwd(const gdn_scan_args* args, void* ws, size_t ws_bytes, void* stream);

/* The recurrence token by token on state_inout ([B, C] float32, in place): T = 1 is one
 * decode step. A sequence of length 0 keeps its state and its row of h. No workspace. */
int gdn_gated_scan_step(const gdn_scan_args* args, float* state_inout, void* stream);

/* Gradient outputs of gdn_gated_scan_bwd: dx, df, di [B, T, C] contiguous in args->dtype
 * (di NULL without i), zero behind a sequence's length; ddecay [C] float32 (POWER only;
 * NULL: not written) and dh0 [B, C] float32 (NULL: not written). dx, df or di may be x, f, i or d_h
 * itself where that is contiguous; otherwise none may overlap an input (GDN_ERR_ARG for rows, and for
 * dh0 over d_h_final). */
typedef struct gdn_scan_grads {
  void* dx;
  void* df;
  void* di;
  float* ddecay;
  float* dh0;
} gdn_scan_grads;

/* Bytes of device workspace gdn_gated_scan_bwd needs (0 for an invalid set); fewer with checkpoints. */
size_t gdn_gated_scan_bwd_workspace_bytes(const gdn_scan_args* args);

/* Gradients of h and h_final: with d_h [B, T, C] in args->dtype (contiguous; rows behind a
 * length are not used) and d_h_final [B, C] float32 (NULL: zero),
 *     l_n = d_h_n + d_h_final,  l_t = d_h_t + a_{t+1} l_{t+1},
 *     d a_t = l_t h_{t-1},  d (m sigmoid(i) x)_t = l_t,  dh0 = a_1 l_1,
 * h recomputed in float32. args->h and args->h_final are ignored. In POWER, m has no slope
 * at a = 1 (decay or sigmoid(f) 0): its part is taken as 0 there, the limit for f. The sums
 * for ddecay run in a fixed order. */
int gdn_gated_scan_bwd(const gdn_scan_args* args, const void* d_h, const float* d_h_final, const gdn_scan_grads* grads,
                       void* ws, size_t ws_bytes, void* stream);

/* ---- Short causal convolution a channel ----------------------------------------------------
 *
 *     z_t = bias + sum_{j < W} w[c][j] x_{t - W + 1 + j},     y_t = z_t / (1 + e^{-z_t}) or z_t
 *
 * what mixes a few neighbouring tokens before a recurrence's inputs. The rows before the
 * first token are those of a state, the last W - 1 inputs so far, oldest first.
 *   x, y             [B, T, C], C a multiple of 8; x a view by x_stride, y contiguous. y must not
 *                    overlap x (GDN_ERR_ARG), but may be x itself where that is contiguous and T at
 *                    most 8
 *   w                [C, W] float32, bias [C] float32 (NULL: zero)
 *   seq_lens         as above: rows of y behind a length stay as they were
 *   s0, s_final      [B, W - 1, C] in the inputs' type
 * Limits as for the gated recurrence. A NaN or Inf in a row reaches the W rows that read it. */
typedef struct gdn_conv_args {
  int32_t dtype;       /* enum gdn_dtype: x, y and the states  */
  int32_t activation;  /* 0: none, or GDN_ACT_SILU             */
  int64_t B, T, C;
  int64_t W;           /* 2, 3 or 4                            */
  int64_t x_stride;
  const void* x;
  const float* w;
  const float* bias;
  const int32_t* seq_lens;
  const void* s0;      /* NULL means zero; ignored by the step                 */
  void* s_final;       /* NULL: not written; may alias s0; ignored by the step */
  void* y;
} gdn_conv_args;

/* y for every token, and the state after the last one. No workspace. */
int gdn_short_conv_fwd(const gdn_conv_args* args, void* stream);

/* The same with one state, read and then replaced ([B, W - 1, C] in args->dtype). */
int gdn_short_conv_step(const gdn_conv_args* args, void* state_inout, void* stream);

/* Gradient outputs of gdn_short_conv_bwd: dx [B, T, C] contiguous and ds0 [B, W - 1, C]
 * (NULL: not written) in args->dtype, zero behind a sequence's length; dw [C, W] and dbias
 * [C] float32 (NULL: not written). None may overlap an input (GDN_ERR_ARG for dx over x or d_y and
 * for ds0 over a state). */
typedef struct gdn_conv_grads {
  void* dx;
  float* dw;
  float* dbias;
  void* ds0;
} gdn_conv_grads;

/* Bytes of device workspace gdn_short_conv_bwd needs (0 for an invalid set). */
size_t gdn_short_conv_bwd_workspace_bytes(const gdn_conv_args* args);

/* Gradients of y and s_final: d_y [B, T, C] in args->dtype (contiguous; rows behind a length
 * are not used), d_s_final [B, W - 1, C] in args->dtype (NULL: zero). args->y and
 * args->s_final are ignored. The sums for dw and dbias run in a fixed order. */
int gdn_short_conv_bwd(const gdn_conv_args* args, const void* d_y, const void* d_s_final, const gdn_conv_grads* grads,
                       void* ws, size_t ws_bytes, void* stream);

/* ---- Norms around a block, with its gate and residual scale ---------------------------------
 *
 * What stands between one block's output y and the next block's input, in one pass:
 *     u  = y (sum y^2 / C + eps)^{-1/2} post_weight   (post_norm), or y
 *     r' = residual_scale r + scale act(gate) u
 *     n  = r' (sum r'^2 / C + eps)^{-1/2} weight
 * with r the residual stream; the sums and n are of r' before it is rounded. Sums of squares are
 * float32: a row whose sum passes 3.4e38 (values of 1.8e19 / sqrt(C), 1.4e17 at C = 16,384) has a
 * norm of zeros; with eps = 0 values under 1e-19 lose bits, and a row of zeros is 0 times infinity.
 *   r, residual_out   [B, T, C] in residual_dtype; C a multiple of 8 up to 16,384
 *   y, gate, out      [B, T, C] in dtype. gate NULL: act(gate) is 1. y NULL (then gate, scale and
 *                     post_weight are NULL and post_norm 0): u = 0, the norm before a first block
 *   scale, post_weight, weight   [C] float32, NULL means ones
 * r, y and gate may be views by their strides; residual_out and out are contiguous, at least
 * one is given, and each may be r, y or gate itself where that is contiguous and of its type; they
 * must not overlap each other or an input otherwise (GDN_ERR_ARG).
 * Other limits as for the gated recurrence. */
typedef struct gdn_block_norm_args {
  int32_t dtype;           /* enum gdn_dtype: y, gate, out                            */
  int32_t residual_dtype;  /* GDN_DTYPE_F32 or dtype: r, residual_out                 */
  int32_t activation;      /* enum gdn_activation (of the gate)                       */
  int32_t post_norm;       /* 0 or 1                                                  */
  int64_t B, T, C;
  int64_t r_stride, y_stride, gate_stride;
  float eps;               /* >= 0 */
  float residual_scale;
  const void* r;
  const void* y;
  const void* gate;
  const float* scale;
  const float* post_weight;
  const float* weight;
  void* residual_out;
  void* out;
} gdn_block_norm_args;

int gdn_block_norm_fwd(const gdn_block_norm_args* args, void* stream);

/* Gradients: d_residual_out (residual_dtype) and d_out (dtype), contiguous, at least one of
 * them given (NULL: zero), in; dr (residual_dtype), dy and dgate (dtype), contiguous, NULL:
 * not written, and dscale, dpost_weight, dweight [C] float32 (NULL: not written) out. What an
 * absent input would have as a gradient must be NULL. args->residual_out and out are ignored.
 * dr, dy and dgate may each be a [B, T, C] input itself where that is contiguous and of its type (dr
 * d_residual_out), and must not overlap one otherwise (GDN_ERR_ARG). The weight sums run in a fixed
 * order. */
typedef struct gdn_block_norm_grads {
  const void* d_residual_out;
  const void* d_out;
  void* dr;
  void* dy;
  void* dgate;
  float* dscale;
  float* dpost_weight;
  float* dweight;
} gdn_block_norm_grads;

/* Bytes of device workspace gdn_block_norm_bwd needs (0 for an invalid set). */
size_t gdn_block_norm_bwd_workspace_bytes(const gdn_block_norm_args* args);
int gdn_block_norm_bwd(const gdn_block_norm_args* args, const gdn_block_norm_grads* grads, void* ws, size_t ws_bytes,
                       void* stream);

/* Static text for a status code. */
const char* gdn_status_str(int status);

/* GDN_ABI_VERSION of the loaded library. */
int gdn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
