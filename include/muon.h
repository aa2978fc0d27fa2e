/*
 * libmuon — one Muon optimizer step for a list of 2-D weight matrices on an
 * AMD Instinct MI355X (gfx950).  C ABI: plain pointers and sizes only.
 *
 * What a step computes, per matrix, follows "Muon: An optimizer for hidden
 * layers in neural networks" (synthesis note on papers.chlience.com),
 * section 4, the algorithm definition:
 *
 *   B  <- mu * B + G                        momentum accumulation
 *   M  =  B            (nesterov == 0)      input of the orthogonalisation
 *   M  =  G + mu * B   (nesterov != 0)      Nesterov-style reading
 *   X  =  M / (||M||_F + eps)               Frobenius normalisation
 *   X  =  X^T when rows > cols              smaller Gram matrix
 *   repeat ns_steps times (default 5):
 *       A = X X^T;  P = b A + c A A;  X = a X + P X
 *       (a, b, c) = (3.4445, -4.7750, 2.0315)
 *   O  =  X, transposed back when rows > cols
 *   W  <- W - lr * scale * O                parameter update
 *   W  <- W - lr * (lambda * W + scale * O)  with decoupled weight decay
 *                                            lambda (hp->weight_decay)
 *
 * Precision: G is float32 or bfloat16; W and B are float32 and updated in
 * place in float32.  For a Gram side m > 64 every matrix product of the
 * iteration runs on bf16 matrix cores with float32 accumulation; A and P are
 * stored as bf16; the iterate X is carried as a pair of bf16 values (high
 * part and rounding residual) so that the linear term a*X keeps ~16
 * significant bits.  The pair first holds M itself and the first
 * iteration applies 1 / (||M||_F + eps) in its float32 epilogues (the Gram
 * product scaled by its square), unless ||M||_F lies outside [2^-50, 2^50],
 * where the pair holds the normalised M instead.  For m <= 64 (few singular
 * values, where bf16 operand rounding does not average out and the work is
 * small) the iteration runs in float32 throughout.
 *
 * Memory: every pointer passed to the step calls is a DEVICE pointer on the
 * current HIP device, except the descriptor arrays themselves (mats, hp and
 * the pointer/size arrays of muon_orthogonalize), which are HOST memory read
 * only during the call.  All device memory is owned by the caller; the
 * library allocates no device memory and keeps no pointer after a call
 * returns (it keeps a small pinned host staging area for the descriptor
 * table it uploads into the workspace).
 *
 * Ordering: work is enqueued on `stream` (a hipStream_t; NULL = the default
 * stream) and the call returns without waiting.  Results are visible after
 * the caller synchronises the stream.  The caller keeps every buffer alive
 * until then.  Two calls that share a workspace must be ordered on one
 * stream (or synchronised) — the workspace holds the call's descriptor table
 * and intermediates.
 *
 * Errors: all arguments are validated on the host before anything is
 * enqueued, so an error return has no side effects.  A failing HIP launch
 * returns MUON_ERR_HIP; muon_last_error() then holds the HIP message.
 * Faults inside kernels surface at the caller's next synchronisation.
 * NaN or Inf in G propagates into B, W; it is not masked.
 */
#ifndef MUON_H_
#define MUON_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_ABI_VERSION 7

typedef enum muon_status {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = -1, /* null pointer, size < 1, bad hyper-parameter   */
  MUON_ERR_UNSUPPORTED = -2, /* shape beyond the supported maximum            */
  MUON_ERR_WORKSPACE = -3,   /* workspace missing, too small or misaligned    */
  MUON_ERR_ALIAS = -4,       /* W/G/B/workspace ranges overlap                */
  MUON_ERR_ALIGN = -5,       /* a matrix base pointer is not 16-byte aligned  */
  MUON_ERR_HIP = -6          /* a HIP runtime call or launch failed           */
} muon_status_t;

typedef enum muon_dtype { MUON_F32 = 0, MUON_BF16 = 1 } muon_dtype_t;

/* One weight matrix.  W, G, B are dense row-major rows x cols arrays
 * (leading dimension = cols), each 16-byte aligned, pairwise disjoint and
 * disjoint from every other matrix's arrays and from the workspace.
 * G has the dtype given by muon_hparams_t.g_dtype; W and B are float32.
 * `scale` multiplies the learning rate for this matrix (the per-parameter
 * update scale of the synthesis note's Moonlight results section; the
 * pages give no formula, so the caller supplies it; 1.0 = plain Muon). */
typedef struct muon_matrix {
  float* W;
  const void* G;
  float* B;
  int64_t rows;
  int64_t cols;
  float scale;
} muon_matrix_t;

/* Hyper-parameters shared by every matrix of a call.
 * mu: momentum (finite); lr: learning rate (finite);
 * eps: added to the Frobenius norm (finite, >= 0; 1e-7 is customary);
 * ns_steps: Newton-Schulz iterations, 0..MUON_MAX_NS_STEPS (5 is the usual);
 * nesterov: 0 = orthogonalise the momentum buffer, 1 = G + mu * B;
 * g_dtype: MUON_F32 or MUON_BF16;
 * weight_decay: decoupled ("AdamW-style") weight decay lambda of the
 *   Moonlight results section of the synthesis note (finite; 0 = none):
 *   W <- W - lr * (lambda * W + scale * O), formed as
 *   fma(-lr*scale, O, fma(-lr*lambda, W, W)) with lr*scale and lr*lambda
 *   rounded to float32 on the host. */
typedef struct muon_hparams {
  float mu;
  float lr;
  float eps;
  int32_t ns_steps;
  int32_t nesterov;
  int32_t g_dtype;
  float weight_decay;
} muon_hparams_t;

#define MUON_MAX_NS_STEPS 64
/* Largest supported dimension of a matrix (rows and cols each). */
#define MUON_MAX_DIM 65536
/* Largest supported short side (the Gram dimension min(rows, cols)). */
#define MUON_MAX_GRAM 16384

/* Bytes of device workspace muon_step needs for this list (0 if n == 0).
 * Returns 0 and sets muon_last_error() when the arguments are invalid.
 * The workspace must be 256-byte aligned. */
size_t muon_workspace_bytes(const muon_matrix_t* mats, int64_t n, const muon_hparams_t* hp);

/* One Muon step on `n` matrices (section 4 of the synthesis note, as above).
 * Updates W and B in place; G is read only.  All matrices are processed by
 * the same sequence of grouped launches (one launch per stage for the whole
 * list), so same-shape matrices such as separate Q, K and V share each
 * dispatch.  n == 0 is a no-op returning MUON_OK. */
muon_status_t muon_step(const muon_matrix_t* mats, int64_t n, const muon_hparams_t* hp,
                        void* workspace, size_t workspace_bytes, void* stream);

/* muon_step for callers that cannot allocate device memory (serving loops
 * and harnesses that forbid hipMalloc): the same kernels and the same bits
 * as muon_step, with the workspace in a static device array of the library
 * instead of a caller's buffer.  The array holds MUON_STATIC_WORKSPACE_BYTES
 * (64 MiB) on every GPU the library runs on, from the first use on that GPU
 * until the process ends; a call whose workspace (muon_workspace_bytes)
 * exceeds it returns MUON_ERR_WORKSPACE before anything is enqueued.  The
 * call allocates nothing: no device memory and no pinned host memory (its
 * descriptor table is copied from the call's own host memory, which the
 * copy has consumed when the call returns; so this entry point is not for
 * stream capture).  Every call on one GPU shares that GPU's array, which
 * keeps the last call's contents (every byte a call reads it writes first):
 * calls that overlap on one GPU (other threads, other streams) race and
 * must be ordered by the caller.  The address of the array is looked up once
 * per device, with that device current. */
#define MUON_STATIC_WORKSPACE_BYTES (64u * 1024u * 1024u)
muon_status_t muon_step_static(const muon_matrix_t* mats, int64_t n, const muon_hparams_t* hp, void* stream);

/* A recorded step, for training loops that run the same step many times on
 * the same buffers (the case where launching ~20 kernels per step from the
 * host costs more than the kernels themselves, e.g. a single 256 x 256
 * matrix).  muon_plan_create validates the call exactly as muon_step does,
 * binds its device buffers, uploads the descriptor table into the workspace
 * (synchronously, on `stream`) and records the step's launch sequence into
 * a HIP graph; each muon_plan_step replays it on `stream` as one graph
 * launch.  A replay is one Muon step on the bound buffers: it reads G's
 * current contents (the caller writes each step's gradient into the bound
 * G buffers) and updates W and B in place, with the hyper-parameters given
 * at creation (create a new plan to change mu, lr, eps, ns_steps, nesterov,
 * weight decay or any scale).  Results are bit-identical to muon_step on
 * the same inputs.  The caller keeps every bound buffer, the workspace
 * included, alive and otherwise untouched until muon_plan_destroy has
 * returned (it waits for the last replay); replays of one plan are ordered
 * one after another by the library, and other work on the bound buffers
 * must be ordered against them by the caller.  A plan belongs
 * to the device current at creation; muon_plan_step on another device is
 * MUON_ERR_INVALID_ARG.  n must be >= 1.  The graph holds no memset node
 * (the per-step counter is zeroed by a kernel). */
typedef struct muon_plan_s* muon_plan_t;
muon_status_t muon_plan_create(const muon_matrix_t* mats, int64_t n, const muon_hparams_t* hp, void* workspace,
                               size_t workspace_bytes, void* stream, muon_plan_t* out);
/* A replay on `stream` is ordered after the plan's previous replay,
 * whichever stream that ran on. */
muon_status_t muon_plan_step(muon_plan_t plan, void* stream);
/* Waits for the plan's last replay to end, then frees its graph (NULL is a
 * no-op); afterwards the caller may release the bound buffers. */
muon_status_t muon_plan_destroy(muon_plan_t plan);

/* Per-matrix diagnostics of one step: the layer-wise quantities that the
 * practice checklist of the synthesis note asks a Muon run to record
 * (item 4 of its local-discussion part: update RMS per matrix shape,
 * weight RMS, norm dynamics), plus a
 * non-finite flag.  With N = rows * cols:
 *   momentum_norm  ||M||_F, M the Newton-Schulz input (section 4), from the
 *                  same float32 block sums as the normalisation
 *   direction_rms  ||O||_F / sqrt(N), O the orthogonalised direction as the
 *                  update applies it, before lr and scale
 *   update_rms     ||W_new - W_old||_F / sqrt(N), the step actually applied
 *                  (decay included), each difference formed in float32
 *   weight_rms     ||W_new||_F / sqrt(N)
 *   nonfinite      bit 0: M holds a NaN or an infinity; bit 1: W_new does
 * The sums of squares are accumulated in float32 per lane and in float64
 * across lanes and work-groups, in a fixed order (repeatable bit for bit).
 * 32 bytes per entry; reserved words are written as 0. */
typedef struct muon_diag {
  float momentum_norm;
  float direction_rms;
  float update_rms;
  float weight_rms;
  int32_t nonfinite;
  int32_t reserved[3];
} muon_diag_t;

/* muon_step plus diagnostics: identical W and B results, and diag[i]
 * (DEVICE memory, n entries, 4-byte aligned, caller-owned, disjoint from
 * every other buffer of the call) describes matrix i once the stream
 * reaches the end of the call.  Needs the same workspace as muon_step; one
 * extra launch (stage MUON_STAGE_DIAG).  diag == NULL is MUON_ERR_INVALID_ARG. */
muon_status_t muon_step_diag(const muon_matrix_t* mats, int64_t n, const muon_hparams_t* hp,
                             muon_diag_t* diag, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Orthogonalisation alone: O[i] = NS(M[i]) for float32 row-major inputs
 * M[i] (rows[i] x cols[i]) into float32 outputs O[i] of the same shape,
 * with the same normalisation, transpose rule and iteration as muon_step.
 * For tests and measurement of the Newton-Schulz stage.  M and O are arrays
 * of n device pointers held in host memory. */
size_t muon_orthogonalize_workspace_bytes(const int64_t* rows, const int64_t* cols, int64_t n,
                                          int32_t ns_steps);
muon_status_t muon_orthogonalize(const float* const* M, float* const* O, const int64_t* rows,
                                 const int64_t* cols, int64_t n, int32_t ns_steps, float eps,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* Host-only description of how a call would be executed (no GPU needed).
 * Fills `info`; if `per_matrix` is non-NULL it must hold n entries. */
typedef struct muon_plan_info {
  int64_t workspace_bytes;
  int64_t launches;          /* kernel launches per call                    */
  int64_t gram_tiles;        /* work-groups of one Gram launch              */
  int64_t poly_tiles;        /* work-groups of one polynomial launch        */
  int64_t bx_tiles;          /* work-groups of one BX + aX launch           */
  int64_t ew_blocks;         /* work-groups of the momentum/norm launch     */
  int32_t tile;              /* symmetric tile edge of the first group      */
  int32_t reserved;
} muon_plan_info_t;

typedef struct muon_matrix_plan {
  int32_t transposed;   /* 1 when rows > cols: the iteration runs on M^T          */
  int32_t m;            /* Gram side min(rows, cols)                              */
  int32_t n;            /* long side max(rows, cols)                              */
  int32_t m_pad;        /* padded Gram side of the iterate buffers (zeros)        */
  int32_t n_pad;        /* padded long side of the iterate buffers (zeros)        */
  int32_t tile;         /* tile edge of the symmetric products; 0 = float32 path  */
  int32_t bx_tile_rows; /* Gram-side tile height of the BX product (0 on float32) */
  int32_t bx_tile_cols; /* long-side tile width of the BX product (0 on float32)  */
  int32_t fused_update; /* 1: the last BX launch writes W (or O) itself, from the  */
                        /* float32 accumulator; 0: a separate update pass reads   */
                        /* the final iterate pair (hi + lo)                       */
  int32_t xcd_edges;    /* bit s (s = 0 Gram, 1 polynomial, 2 BX) set when one of */
                        /* the 8 XCDs starts its share of that grouped launch     */
                        /* inside (or at the first tile of) this matrix's tiles   */
  int64_t x_offset;     /* byte offset of the iterate buffers in the workspace    */
} muon_matrix_plan_t;

muon_status_t muon_plan_query(const muon_matrix_t* mats, int64_t n, const muon_hparams_t* hp,
                              muon_plan_info_t* info, muon_matrix_plan_t* per_matrix);

/* Stage timing.  When enabled (per process), every launch of a step is
 * bracketed by HIP events on the stream it is launched on;
 * muon_profile_read waits for the recorded events, adds their elapsed times
 * per stage to `ms` and the launch counts to `launches` (arrays of
 * MUON_STAGE_COUNT entries, caller-owned host memory), and clears them. */
typedef enum muon_stage {
  MUON_STAGE_MOMENTUM = 0, /* momentum, Frobenius partial sums and the */
                           /* unnormalised bf16 pair (first iteration  */
                           /* applies the normalisation)               */
  MUON_STAGE_NORM = 1,     /* per-matrix norm reduction                */
  MUON_STAGE_PREP = 2,     /* normalised iterate, only for matrices    */
                           /* that cannot fold it (m <= 64, ns_steps 0,*/
                           /* ||M||_F outside [2^-50, 2^50])           */
  MUON_STAGE_GRAM = 3,     /* A = X X^T (upper tiles + mirror)         */
  MUON_STAGE_POLY = 4,     /* P = b A + c A A (upper tiles + mirror)   */
  MUON_STAGE_BX = 5,       /* X = a X + P X                            */
  MUON_STAGE_UPDATE = 6,   /* W -= lr * scale * O (or O store)         */
  MUON_STAGE_UPLOAD = 7,   /* descriptor table copy                    */
  MUON_STAGE_BX_UPDATE = 8, /* last X = a X + P X with W -= lr*scale*O  */
                            /* applied in the same launch (wide tiles)  */
  MUON_STAGE_DIAG = 9,      /* per-matrix diagnostics (muon_step_diag)  */
  MUON_STAGE_COUNT = 10
} muon_stage_t;

muon_status_t muon_profile_enable(int32_t on);
muon_status_t muon_profile_read(double* ms, int64_t* launches);

/* QK-Clip: after a step, rescale attention query and key projections head by
 * head from each head's max logit, to keep attention logits from growing
 * without bound.  The synthesis note's results section (result 3, Kimi K2's
 * MuonClip) describes this rescale after the Muon step without a formula or
 * threshold; the reading implemented: rows h*head_dim .. (h+1)*head_dim-1
 * of W belong to head h (the (out, in) layout of a projection), and when
 * max_logit[h] > tau they are multiplied by sqrt(tau / max_logit[h])
 * (float32 division and square root, correctly rounded; one rounding per
 * element).  Clipping the query and the key projection of one attention
 * layer with the same max_logit array scales every logit of a clipped head
 * by tau / max_logit[h], so its max logit becomes tau; heads at or below
 * tau (or with a NaN max logit) are not touched.  An infinite max logit
 * zeroes the head's rows.
 *   That holds where logits are linear in both projections (rotary positions
 * keep them so).  Behind a norm of queries and keys (muon_qk_norm_rotate with
 * norm != 0) they do not depend on the projections' size, and clipping W_q and
 * W_k would shrink them at every step for nothing: there the norm's weights
 * take their place, each as one head (rows = head_dim, cols = 1), with the
 * largest max logit of the heads that share them.
 *   W          DEVICE, rows x cols float32 row-major, 16-byte aligned,
 *              updated in place; disjoint from every other W of the call
 *   rows, cols >= 1, <= MUON_MAX_DIM; rows a multiple of head_dim
 *   head_dim   >= 1
 *   max_logit  DEVICE, rows / head_dim float32 entries, 4-byte aligned,
 *              read only (Q and K of one layer may share it)
 * tau: finite, > 0.  mats is HOST memory read during the call.  One launch
 * per 48 matrices (the descriptors travel as kernel arguments; no
 * workspace); a head whose factor is 1 costs one read.  Stream-ordered:
 * call it after muon_step on the same stream. */
typedef struct muon_qk_clip_matrix {
  float* W;
  int64_t rows;
  int64_t cols;
  int32_t head_dim;
  int32_t reserved;
  const float* max_logit;
} muon_qk_clip_matrix_t;
muon_status_t muon_qk_clip(const muon_qk_clip_matrix_t* mats, int64_t n, float tau, void* stream);

/* ---------------------------------------------------------------- training-step
 * operators next to the Muon step: what produces the arguments of muon_step
 * and muon_qk_clip in a training step.  Attention gives each head's largest
 * logit (QK-Clip's input); a saved 8-bit activation and the upstream
 * gradient give a projection's G.  They were added within
 * MUON_ABI_VERSION 7, since no earlier entry point changed: a caller that
 * loads the library at run time looks for muon_packing_create by name (and, for
 * windowed attention, norms and rotations and clipping, which came after the
 * rest, for muon_grad_norm).
 *
 * As for the step calls: host structures are read only during the call,
 * device memory is the caller's, everything is validated before anything is
 * enqueued, work is enqueued on `stream` and the call returns without
 * waiting.  Apart from muon_packing_create the calls may be captured into a
 * HIP graph.  Results are the same bits in every run. */

/* A packing: sequences of the given lengths laid end to end in the first
 * sum(lengths) rows of the token dimension.  muon_packing_create checks the
 * lengths (each 0 .. MUON_MAX_SEQUENCE; sum <= MUON_MAX_TOKENS) and writes the kernels' work
 * list into `table` (DEVICE, muon_packing_bytes bytes, 256-byte aligned)
 * through `stream`, which it synchronises; the handle may then be used on any
 * stream of that device, by any number of calls at once.  The caller keeps
 * `table` alive and untouched until the last call that uses the handle has
 * finished on the device; muon_packing_destroy frees host memory only and
 * does not wait.  Zero sequences, and empty ones, are allowed.
 * muon_packing_bytes returns 0 on invalid lengths. */
#define MUON_MAX_TOKENS 1073741824
#define MUON_MAX_SEQUENCE 16777216
typedef struct muon_packing_s* muon_packing_t;
size_t muon_packing_bytes(const int64_t* lengths, int64_t n);
muon_status_t muon_packing_create(const int64_t* lengths, int64_t n, void* table, size_t table_bytes, void* stream,
                                  muon_packing_t* out);
muon_status_t muon_packing_destroy(muon_packing_t packing);

/* A (tokens, heads, head_dim) bfloat16 tensor in DEVICE memory: element
 * (t, h, d) at data[t * token_stride + h * head_stride + d].  data is 16-byte
 * aligned, the strides (in elements) are multiples of 8, >= 0 and at most
 * MUON_MAX_TOKEN_STRIDE (token) so that views into a fused projection output
 * work as they are.  Tensors that a call writes must not overlap themselves
 * or any other tensor of the call; interleaved views of one buffer that
 * share no element are fine. */
#define MUON_MAX_TOKEN_STRIDE 4194304
typedef struct muon_heads {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} muon_heads_t;

/* Causal self-attention over a packing.  Row i of a sequence attends to rows
 * 0..i of the same sequence; query head h uses key and value head
 * h / (heads / kv_heads):
 *   s_ij = scale * q_i . k_j,  lse_i = log sum_{j<=i} exp(s_ij),
 *   o_i = sum_{j<=i} exp(s_ij - lse_i) v_j
 * Products of bfloat16 with float32 accumulation; softmax in float32; the
 * unnormalised probabilities are rounded to bfloat16 for the product with v,
 * o to bfloat16 once.
 *   q, o       heads query heads; k, v: kv_heads heads; o is written
 *   lse        heads rows of lse_stride (>= the packing's tokens) float32,
 *              4-byte aligned, written
 *   max_logit  NULL, or logit_heads float32 entries, read and written:
 *              entry g becomes max(entry, s_ij over every visible pair of its
 *              heads g * heads / logit_heads ...), so that one array collects
 *              the maximum over the calls of an optimizer step (the caller
 *              starts it at -infinity).  logit_heads is heads or kv_heads:
 *              the latter is what muon_qk_clip takes for a grouped layout
 *              (query projection with head_dim * heads / kv_heads rows per
 *              entry, key projection with head_dim).  A NaN logit gives
 *              NaN, +infinity where the row's largest logit is that; an entry
 *              that is NaN stays NaN.
 *   heads      a multiple of kv_heads >= 1, at most MUON_MAX_HEADS; times the
 *              128-row pieces of the packing's sequences (the last of each may
 *              be shorter) below MUON_MAX_ATTENTION_ITEMS
 *   head_dim   a multiple of 8, 8..128 (others: MUON_ERR_UNSUPPORTED)
 *   scale      finite, > 0; scale * log2(e) finite too (others:
 *              MUON_ERR_UNSUPPORTED)
 * Logits from 2^128 / log2(e) on, in magnitude, count as infinite in o and lse.
 * Rows of o and lse behind the packing's last sequence are left as they
 * were, and rows of q, k, v there are not read.  Sequences do not mix: a NaN
 * or infinity in a sequence reaches rows of that sequence only (there it
 * may reach rows before it too: 0 * NaN is NaN). */
#define MUON_MAX_HEADS 4096
#define MUON_MAX_ATTENTION_ITEMS 8388608
typedef struct muon_attention {
  muon_heads_t q, k, v, o;
  float* lse;
  int64_t lse_stride;
  float* max_logit;
  int32_t logit_heads;
  int32_t heads;
  int32_t kv_heads;
  int32_t head_dim;
  float scale;
} muon_attention_t;
muon_status_t muon_attention(const muon_attention_t* args, muon_packing_t packing, void* stream);

/* Backward pass of muon_attention: from q, k, v, the forward's o and lse and
 * the upstream gradient d_o,
 *   p_ij = exp(s_ij - lse_i),  delta_i = d_o_i . o_i,
 *   dv_j = sum_i p_ij d_o_i,  ds_ij = p_ij (d_o_i . v_j - delta_i),
 *   dq_i = scale * sum_j ds_ij k_j,  dk_j = scale * sum_i ds_ij q_i
 * (dk and dv summed over the query heads of a group), written as bfloat16,
 * each rounded once from float32; p and ds are rounded to bfloat16 for the
 * products.  No atomics.  Rows behind the last sequence are left as they
 * were.  Workspace: DEVICE, 256-byte aligned, muon_attention_backward_workspace_bytes
 * bytes (0 and muon_last_error() on invalid arguments; data pointers are not
 * looked at). */
typedef struct muon_attention_grad {
  muon_heads_t q, k, v, o, d_o;
  const float* lse;
  int64_t lse_stride;
  muon_heads_t dq, dk, dv;
  int32_t heads;
  int32_t kv_heads;
  int32_t head_dim;
  float scale;
} muon_attention_grad_t;
size_t muon_attention_backward_workspace_bytes(const muon_attention_grad_t* args, muon_packing_t packing);
muon_status_t muon_attention_backward(const muon_attention_grad_t* args, muon_packing_t packing, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* Attention with a sliding window and first tokens that stay visible: as
 * muon_attention, but row i of a sequence sees its row j <= i where i - j <
 * window, or j < sinks.
 *   window  >= 1: the row itself and the window - 1 before it.  A window that
 *           hides no key of the packing gives muon_attention's bits
 *   sinks   0 .. MUON_MAX_SINKS first rows of each sequence
 * max_logit is over visible pairs.  A NaN or infinity in a sequence may reach
 * rows of it that do not see it, as there.  The forward workspace (DEVICE,
 * 256-byte aligned) may be NULL; with muon_window_attention_workspace_bytes
 * bytes (4 for each 128-row piece of a sequence and head; 0 where it makes no
 * difference, which muon_last_error() being empty tells from an error; of
 * args' pointers only max_logit being NULL is looked at) max_logit is raised
 * with fewer atomics.  The backward workspace holds,
 * beside muon_attention_backward's, 8 * head_dim * kv_heads * sinks bytes for
 * every 256 rows (or fewer) of a sequence, where the window hides any, and up to
 * 1024 * head_dim * heads for every 128 (or fewer) where that makes few key
 * heads or rows faster. */
#define MUON_MAX_SINKS 128
size_t muon_window_attention_workspace_bytes(const muon_attention_t* args, int64_t window, int64_t sinks,
                                             muon_packing_t packing);
muon_status_t muon_window_attention(const muon_attention_t* args, int64_t window, int64_t sinks, muon_packing_t packing,
                                    void* workspace, size_t workspace_bytes, void* stream);
size_t muon_window_attention_backward_workspace_bytes(const muon_attention_grad_t* args, int64_t window, int64_t sinks,
                                                      muon_packing_t packing);
muon_status_t muon_window_attention_backward(const muon_attention_grad_t* args, int64_t window, int64_t sinks,
                                             muon_packing_t packing, void* workspace, size_t workspace_bytes,
                                             void* stream);

/* Norms of queries and keys per head with rotary positions in the same pass,
 * between the projections and attention.  Per token and head:
 *   y_d = x_d * w_d / sqrt(mean over the head of x^2 + eps)   (norm == 0: y = x)
 *   pair i < rotary_dim / 2 of elements (l, h): (i, rotary_dim / 2 + i), or
 *   (2 i, 2 i + 1) where interleaved, is turned by u = position * frequency[i]:
 *   z_l = y_l cos u - y_h sin u,  z_h = y_h cos u + y_l sin u
 *   z_d = y_d for d >= rotary_dim
 * Float32 throughout, z rounded to bfloat16 once.  Angles are exact modulo a
 * turn up to 2^-64 turns a position where |frequency| < 1 (far positions stay as
 * good as near ones).
 * A token has one position per axis (time, height, width of a video, say), and
 * each pair goes by one axis.
 *   rotary.rotary_dim   a multiple of 8, 0 (no rotation) .. head_dim
 *   rotary.axes         1 .. MUON_MAX_AXES
 *   rotary.frequency    HOST, rotary_dim / 2 radians per position, each of
 *                       magnitude <= MUON_MAX_FREQUENCY
 *   rotary.axis         HOST, each pair's axis (0 .. axes - 1), or NULL: 0
 *   positions  DEVICE, axes rows of position_stride (>= the packing's tokens, or
 *              0: one row for every axis) integers of position_bits (32 or 64),
 *              of any sign and size; or NULL: each token's index in its
 *              sequence, on every axis
 *   weights    DEVICE, head_dim float32, or NULL: ones (and so without a norm)
 *   eps        finite, >= 2^-126 (norm only)
 *   heads, kv_heads  1 .. MUON_MAX_HEADS each; head_dim as for attention
 * q_out may be q itself and k_out k (the same data and strides).  Rows behind
 * the packing's last sequence are neither read nor written.  For QK-Clip of a
 * layer with these norms see muon_qk_clip. */
#define MUON_MAX_AXES 4
#define MUON_MAX_FREQUENCY 1024
typedef struct muon_rotary {
  int32_t rotary_dim;
  int32_t interleaved;
  int32_t axes;
  int32_t reserved;
  const double* frequency;
  const int32_t* axis;
} muon_rotary_t;
typedef struct muon_qk_rotate {
  muon_heads_t q, k, q_out, k_out;
  const float* q_weight;
  const float* k_weight;
  const void* positions;
  int64_t position_stride;
  int32_t position_bits;
  int32_t heads;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t norm;
  float eps;
  muon_rotary_t rotary;
} muon_qk_rotate_t;
muon_status_t muon_qk_norm_rotate(const muon_qk_rotate_t* args, muon_packing_t packing, void* stream);

/* Backward pass of muon_qk_norm_rotate: from the forward's q, k (its inputs;
 * not looked at without a norm), weights, positions and rotary, and the
 * gradients d_q_out and d_k_out of its outputs, with g the upstream gradient
 * turned back and n = x / sqrt(mean x^2 + eps),
 *   dx_d = (w_d g_d - n_d mean(w g n)) / sqrt(mean x^2 + eps)   (norm == 0: g)
 *   dw_d = sum over tokens and heads of g_d n_d
 * args->q_out and k_out take dq and dk (bfloat16, rounded once; they may be
 * d_q_out and d_k_out, or q and k, themselves); d_q_weight and d_k_weight
 * DEVICE, head_dim float32 each, written; NULL: not formed (and NULL where the
 * weight is).  No atomics.  Workspace, where one of them is formed: DEVICE,
 * 256-byte aligned, muon_qk_norm_rotate_backward_workspace_bytes(head_dim)
 * bytes (0 for a head_dim that is not supported). */
size_t muon_qk_norm_rotate_backward_workspace_bytes(int32_t head_dim);
muon_status_t muon_qk_norm_rotate_backward(const muon_qk_rotate_t* args, const muon_heads_t* d_q_out,
                                           const muon_heads_t* d_k_out, float* d_q_weight, float* d_k_weight,
                                           muon_packing_t packing, void* workspace, size_t workspace_bytes, void* stream);

/* 8-bit activation checkpoints: a layer's input x (tokens x cols, row-major)
 * kept from the forward to the backward pass in half the bytes of bfloat16.
 * Blocks of 32 tokens x 32 columns share the exponent e, the smallest integer
 * >= -117 with max |x| <= 448 * 2^e over the block's finite values; each
 * value is held as the 8-bit number (4 exponent and 3 mantissa bits, e4m3)
 * nearest to x * 2^-e, ties to even, and stands for that number times 2^e:
 * off by at most 2^-4 of x, or by 2^(e-10) where |x| < 2^(e-6).  Magnitudes
 * above 1.875 * 2^127 are held as that (the next such number would be 2^128),
 * NaN and infinities as NaN.  A held value is exact in bfloat16.
 *   x         DEVICE, element (t, c) at x[t * x_stride + c], dtype MUON_F32 or
 *             MUON_BF16, aligned to its element; x_stride >= cols, at most 2^40,
 *             and tokens * x_stride at most 2^56
 *   data      DEVICE, 256-byte aligned, muon_checkpoint_bytes(tokens, cols)
 *             bytes (cols and tokens rounded up to 32, plus 1 / 1024); an
 *             opaque layout, made for muon_checkpoint_grad
 *   tokens    >= 0, <= MUON_MAX_TOKENS; cols: 1 .. MUON_MAX_DIM; to write and
 *             read, ceil(tokens / 32) * ceil(cols / 256) < 2^24
 * muon_checkpoint_write fills every item's data from its x;
 * muon_checkpoint_read writes the held values to x (each exact in bfloat16),
 * for backward passes that need the input itself.  One launch per 32 items;
 * buffers that a call writes overlap nothing else of the call (a strided x
 * counts from its first to its last element). */
typedef struct muon_checkpoint {
  void* x;
  int64_t x_stride;
  int32_t x_dtype;
  int32_t reserved;
  void* data;
  int64_t tokens;
  int64_t cols;
} muon_checkpoint_t;
size_t muon_checkpoint_bytes(int64_t tokens, int64_t cols); /* 0 on invalid arguments */
muon_status_t muon_checkpoint_write(const muon_checkpoint_t* items, int64_t n, void* stream);
muon_status_t muon_checkpoint_read(const muon_checkpoint_t* items, int64_t n, void* stream);

/* Weight gradients from checkpoints, G of muon_step: for a projection y = x W^T
 * with W outs x cols,
 *   G[o][c] = sum_t dy[t][o] * x^[t][c]      (accumulate: added to G)
 * with x^ the checkpoint's held values: exact bfloat16 products, float32
 * sums, one rounding to G's type.
 *   dy    DEVICE bfloat16, element (t, o) at dy[t * dy_stride + o], 2-byte
 *         aligned, dy_stride >= outs and <= MUON_MAX_TOKEN_STRIDE (a 16-byte
 *         aligned dy with a stride that is a multiple of 8 is read fastest;
 *         there, with outs odd, the four aligned bytes that hold dy's last
 *         element are read whole)
 *   data  a checkpoint of (tokens, cols); matrices of a call may share it
 *   G     DEVICE, outs x cols row-major, MUON_F32 or MUON_BF16, 16-byte
 *         aligned, overlapping nothing else of the call
 *   accumulate  0: G is written; 1: the sum is added to it in float32
 * All matrices share launches (24 per launch).  tokens == 0 gives zeros
 * (or leaves G with accumulate).  Workspace: DEVICE, 256-byte aligned,
 * muon_checkpoint_grad_workspace_bytes bytes; may be 0 (then workspace may
 * be NULL), which muon_last_error() being empty tells from an error. */
typedef struct muon_checkpoint_grad {
  const void* dy;
  int64_t dy_stride;
  const void* data;
  int64_t tokens;
  int64_t cols;
  void* G;
  int64_t outs;
  int32_t g_dtype;
  int32_t accumulate;
} muon_checkpoint_grad_t;
size_t muon_checkpoint_grad_workspace_bytes(const muon_checkpoint_grad_t* mats, int64_t n);
muon_status_t muon_checkpoint_grad(const muon_checkpoint_grad_t* mats, int64_t n, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Global norm of a step's gradients, and clipping by it.
 *   norm  = sqrt of the sum of g^2 over every element of every tensor
 *   out   = g * factor, factor = max_norm / norm where norm > max_norm and
 *           norm is finite, else 1
 * Squares, their sums, norm and factor in float64 (no square overflows or
 * vanishes), g * factor rounded to float32 and from there to out's type.  A
 * norm that is NaN or infinite (a gradient holds such a value) leaves the
 * values as they are: they reach the step unmasked, and norm tells.
 *   g      DEVICE, count elements (0 .. MUON_MAX_GRADIENT) without gaps,
 *          MUON_F32 or MUON_BF16, aligned to its element (16 bytes are fastest)
 *   out    DEVICE, likewise; g itself (of one dtype) to clip in place.  Not
 *          looked at by muon_grad_norm
 *   norm   DEVICE, one float64.  muon_grad_norm writes it.  muon_grad_clip
 *          reads it where norm_given != 0 (what a program made of several
 *          calls' norms, or of several devices'), else forms and writes it
 *   max_norm  finite, > 0
 * Buffers that a call writes overlap nothing else of it; muon_grad_norm may
 * be given a tensor twice.  n == 0 gives the norm 0.  Two launches (and one
 * each for every further 96 tensors); workspace: DEVICE, 256-byte aligned,
 * muon_grad_norm_workspace_bytes() bytes (a constant); not used, and may be
 * NULL, where norm_given != 0. */
#define MUON_MAX_GRADIENT 1099511627776
typedef struct muon_gradient {
  const void* g;
  void* out;
  int64_t count;
  int32_t g_dtype;
  int32_t out_dtype;
} muon_gradient_t;
size_t muon_grad_norm_workspace_bytes(void);
muon_status_t muon_grad_norm(const muon_gradient_t* items, int64_t n, double* norm, void* workspace,
                             size_t workspace_bytes, void* stream);
muon_status_t muon_grad_clip(const muon_gradient_t* items, int64_t n, double max_norm, double* norm, int32_t norm_given,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Bandwidth yardstick for the HBM-bound stages (the measurement side of the
 * boundary, not part of a step): copies `bytes` from src to dst (DEVICE
 * memory, 16-byte aligned, bytes a multiple of 16, disjoint) with a plain
 * streaming kernel that reads and writes every byte once, on `stream`.
 * variant 0..MUON_COPY_PROBE_VARIANTS-1: bit 0 selects nontemporal loads and
 * stores, bits 1-2 the grid (1024, 4096 or 16384 work-groups of 256 lanes,
 * each lane with four 16-byte loads in flight).  A benchmark times the
 * variants and takes the fastest as the measured copy ceiling. */
#define MUON_COPY_PROBE_VARIANTS 6
muon_status_t muon_copy_probe(const void* src, void* dst, size_t bytes, int32_t variant, void* stream);

const char* muon_status_string(muon_status_t status);
/* Message of the last error on the calling thread ("" if none). */
const char* muon_last_error(void);
int32_t muon_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MUON_H_ */
