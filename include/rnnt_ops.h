/*
 * rnnt_ops.h -- C ABI of the operators around the transducer loss in
 * librnnt_gb300.so: what a training step does between the batch and rnnt_fwd
 * and between rnnt_bwd and the updated weights.
 *
 *   rnnt_embed_*  the prediction network's label embedding: the rows hL that
 *                 rnnt_fwd reads, and the table's gradient from dhL;
 *   rnnt_norm_*   group norm with an activation over the encoder's frames,
 *                 channels last, ragged lengths: the rows hA, and the frames'
 *                 gradient from dhA;
 *   rnnt_ln_*     layer norm of rows (frames or label rows), and its gradients;
 *   rnnt_orth     the orthogonalised update of a weight matrix (Newton-Schulz
 *                 products, as the Muon optimiser takes of hidden matrices such
 *                 as W^A and W^L; it leaves input and output layers, and so W^O,
 *                 to another method);
 *   rnnt_clip     the norm of all gradients together, and their clipping;
 *   rnnt_adamw    the AdamW update of many tensors (W^O, the label table, biases
 *                 and norms, or everything), with the clipping's scale.
 *
 * Conventions are those of rnnt.h: tensor pointers are device pointers, the
 * dims structs host memory; calls are asynchronous on `stream`, never
 * synchronize, allocate no device memory and can be captured into a CUDA
 * graph; the caller owns every buffer; host-checkable problems return an
 * error before anything is launched.  Calls that share a workspace must not
 * run concurrently.  Workspaces must be 256-byte aligned; their contents mean
 * nothing between calls.  Tensors need only their element's alignment (16
 * bytes and sizes that keep rows 16-byte aligned run faster).
 *
 * `status` (every call but rnnt_clip and rnnt_adamw; may be NULL): one device int32 that the caller
 * cleared; the kernels OR bit k into it when a problem with rnnt_status code
 * k is found, and nothing clears it.  Read it with rnnt_ops_status.
 *
 * Outputs must not overlap inputs or one another (but as rnnt_clip and rnnt_adamw
 * say).
 *
 * Sums run in fp32 (rnnt_orth's products as described there, its norm in fp64)
 * without atomics on values: the same inputs, sizes, strides, alignment of the
 * pointers and device give the same bits.  The last three can choose another
 * kernel or grid, and with it another order of a sum.
 */
#ifndef RNNT_GB300_OPS_H
#define RNNT_GB300_OPS_H

#include "rnnt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Synchronize `stream` and read the status word: RNNT_OK or the first recorded
 * code among RNNT_ERR_LENGTH_RANGE, RNNT_ERR_LABEL_RANGE, RNNT_ERR_TIMEOUT;
 * `word` (if not NULL) receives the raw bits. */
rnnt_status rnnt_ops_status(const int32_t* status, rnnt_stream stream, int32_t* word);

/* ---- label embedding ------------------------------------------------------
 *   hL[b,u,:] = scale * E[id(b,u),:]       u <= U_len[b], else 0
 *   dE[v,:]   = scale * sum over (b,u) with id(b,u) = v, u <= U_len[b] of dhL[b,u,:]
 * id(b,u) = ids[b,u], except id(b,0) = blank when sos != 0 (labels as rnnt_fwd
 * takes them: column 0 is the prepended blank and is never read).  sos = 0
 * reads every id (one decoding step: U1 = 1).  U_len NULL: every row exists.
 * An id outside [0,V) on an existing row sets RNNT_ERR_LABEL_RANGE, its row of
 * hL is zero and it has no gradient; a U_len outside [0,U1-1] sets
 * RNNT_ERR_LENGTH_RANGE and its sample has no rows.  Rows that do not exist
 * are never read (their ids and their dhL may hold anything).
 * B*U1 <= 2^30, D <= 2^20; scale finite.
 */
typedef struct {
  int B, U1, V, D;
  int blank;
  int sos;
  int table_dtype;    /* E: RNNT_F32 or RNNT_BF16 (dE is fp32 always) */
  int row_dtype;      /* hL and dhL: RNNT_F32 or RNNT_BF16 */
  float scale;
  long long ld_table; /* row stride of E and of dE, elements >= D (0: D) */
  long long ld_rows;  /* row stride of hL and of dhL, elements >= D (0: D) */
} rnnt_embed_dims;

/* Workspace of rnnt_embed_bwd (rnnt_embed_fwd needs none); 0: invalid dims. */
size_t rnnt_embed_workspace_bytes(const rnnt_embed_dims* dims);

rnnt_status rnnt_embed_fwd(const rnnt_embed_dims* dims, const int32_t* ids, const int32_t* U_len,
                           const void* table, void* rows, int32_t* status, rnnt_stream stream);

/* dtable [V] rows of fp32 is overwritten (rows of labels that do not occur: 0). */
rnnt_status rnnt_embed_bwd(const rnnt_embed_dims* dims, const int32_t* ids, const int32_t* U_len,
                           const void* drows, float* dtable, void* ws, size_t ws_bytes,
                           int32_t* status, rnnt_stream stream);

/* ---- group norm with an activation, channels last -------------------------
 * x [B,T,C]; group g holds channels [g C/G, (g+1) C/G).  Over the frames
 * t < T_len[b] and the channels of a group:
 *   xh = (x - mean) * rstd, rstd = 1 / sqrt(var + eps) (var over n, not n-1)
 *   u = gamma_c xh + beta_c,  y = act(u)
 * Backward, g = dy act'(u):
 *   dgamma_c = sum_{b,t} g xh,  dbeta_c = sum_{b,t} g
 *   dx = rstd (gamma g - mean(gamma g) - xh mean(gamma g xh))
 * act' of relu at 0 is 0.  Frames t >= T_len[b] are never read; their y and dx
 * are 0.  T_len NULL: every frame exists; T_len[b] = 0 is an empty sample; one
 * outside [0,T] sets RNNT_ERR_LENGTH_RANGE and counts as 0.
 * C divisible by G; T <= 2^20, C <= 2^28, B*G <= 2^27.
 * Statistics, sums and the activation's sigmoid (relative error about 2^-21) are
 * fp32; only y and dx are rounded to dtype.  A group's statistics run over all
 * frames of its sample: frames handed over one at a time are normalised each by
 * itself.
 */
typedef enum { RNNT_ACT_NONE = 0, RNNT_ACT_SILU = 1, RNNT_ACT_RELU = 2 } rnnt_act;

typedef struct {
  int B, T, C, G;
  int act;             /* rnnt_act */
  int dtype;           /* x, y, dy, dx: RNNT_F32 or RNNT_BF16 */
  float eps;
  long long x_frame, x_batch;  /* strides of x and dx, elements (0: C, T * x_frame) */
  long long y_frame, y_batch;  /* strides of y and dy, elements (0: C, T * y_frame) */
} rnnt_norm_dims;

/* Bytes of `saved` (fp32 mean and rstd of every sample and group) and of the
 * workspace of either call; 0: invalid dims. */
size_t rnnt_norm_saved_bytes(const rnnt_norm_dims* dims);
size_t rnnt_norm_workspace_bytes(const rnnt_norm_dims* dims);

/* gamma, beta: fp32 [C], either may be NULL (1 and 0). */
rnnt_status rnnt_norm_fwd(const rnnt_norm_dims* dims, const void* x, const float* gamma,
                          const float* beta, const int32_t* T_len, void* y, void* saved, void* ws,
                          size_t ws_bytes, int32_t* status, rnnt_stream stream);

/* saved: as rnnt_norm_fwd wrote it for the same x and T_len.  dgamma, dbeta:
 * fp32 [C], overwritten; either may be NULL. */
rnnt_status rnnt_norm_bwd(const rnnt_norm_dims* dims, const void* x, const void* dy,
                          const float* gamma, const float* beta, const int32_t* T_len,
                          const void* saved, void* dx, float* dgamma, float* dbeta, void* ws,
                          size_t ws_bytes, int32_t* status, rnnt_stream stream);

/* ---- layer norm of rows ------------------------------------------------------
 * x [B,T,C]; each row (b,t) that exists is normalised by itself:
 *   xh = (x - mean) * rstd, rstd = 1 / sqrt(var + eps) (var over C, not C-1)
 *   y = gamma_c xh + beta_c
 * Backward, a = gamma dy:
 *   dgamma_c = sum_{b,t} dy xh,  dbeta_c = sum_{b,t} dy
 *   dx = rstd (a - mean(a) - xh mean(a xh))
 * Rows that exist: t < lengths[b] for frames (label_rows = 0, lengths in [0,T]),
 * t <= lengths[b] for label rows as rnnt_embed_fwd makes them (label_rows = 1,
 * lengths in [0,T-1]).  The others are never read; their y and dx are 0.  lengths
 * NULL: every row exists; a length out of its range sets RNNT_ERR_LENGTH_RANGE and
 * its sample has no rows.  One streamed frame or one decoding step: T = 1.
 * Statistics and sums are fp32, the variance taken about the mean (a row whose
 * squares leave fp32's range gives NaN); only y and dx are rounded to their types.  B*T <= 2^30, C <= 2^20.  Strides may put samples
 * after one another or frames after one another (time-major), without overlap.
 */
typedef struct {
  int B, T, C;
  int label_rows;
  int x_dtype;                 /* x and dx: RNNT_F32 or RNNT_BF16 */
  int y_dtype;                 /* y and dy: RNNT_F32 or RNNT_BF16 */
  float eps;                   /* >= 0; a constant row with eps = 0 gives NaN */
  long long x_frame, x_batch;  /* strides of x and dx, elements (0: C, T * x_frame) */
  long long y_frame, y_batch;  /* strides of y and dy, elements (0: C, T * y_frame) */
} rnnt_ln_dims;

/* Bytes of `saved` (fp32 mean and rstd of every row) and of the workspace of
 * rnnt_ln_bwd (rnnt_ln_fwd needs none); 0: invalid dims. */
size_t rnnt_ln_saved_bytes(const rnnt_ln_dims* dims);
size_t rnnt_ln_workspace_bytes(const rnnt_ln_dims* dims);

/* gamma, beta: fp32 [C], either may be NULL (1 and 0).  saved may be NULL when no
 * gradient will be asked for. */
rnnt_status rnnt_ln_fwd(const rnnt_ln_dims* dims, const void* x, const float* gamma,
                        const float* beta, const int32_t* lengths, void* y, void* saved,
                        int32_t* status, rnnt_stream stream);

/* saved: as rnnt_ln_fwd wrote it for the same x and lengths.  dgamma, dbeta: fp32
 * [C], overwritten; either may be NULL. */
rnnt_status rnnt_ln_bwd(const rnnt_ln_dims* dims, const void* x, const void* dy,
                        const float* gamma, const int32_t* lengths, const void* saved, void* dx,
                        float* dgamma, float* dbeta, void* ws, size_t ws_bytes, int32_t* status,
                        rnnt_stream stream);

/* ---- orthogonalised update -------------------------------------------------
 * For each of `batch` matrices G [rows,cols]:
 *   X = G / (|G|_F + eps), then `steps` times
 *   S = X X^T (rows <= cols; X^T X otherwise), X <- a X + (b S + c S S) X
 * with (a, b, c) = (3.4445, -4.7750, 2.0315), the quintic of the Muon
 * optimiser; O = X.  The singular values move towards 1 and the singular
 * vectors stay: O is near the closest (semi-)orthogonal matrix to G.  A matrix
 * of zeros gives zeros; a NaN or an infinity gives NaN throughout its matrix, and
 * finite entries of any size are fine.
 * Numbers: X and S are held in 22 bits at a fixed scale, so an entry of G below
 * about 2^-39 |G|_F counts as 0, and rows far smaller than the rest keep fewer
 * digits of their own.  A product is three of fp16 halves (22 bits), added in
 * fp32, when O is fp32, when rows or cols is at most 256, or when steps > 5; a
 * bf16 O of larger matrices takes one term (11 bits) where the rounding averages
 * out, which leaves it 1.7 to 2.9e-3 off in all over a range of spectra (relative
 * 2-norm), of which the rounding to bf16 alone is 1.7e-3.  For bf16 storage of an
 * exact result, ask for fp32 and round.  An error of the first step grows by up
 * to 3.4445 a step, and after about eight steps singular values no longer settle
 * but cycle between 0.68 and 1.13: more steps than that are bound to amplify
 * rounding, here as in fp32.
 * rows * cols <= 2^31 - 1 per matrix, batch <= 65535.  O must not overlap G.
 * A wait inside the kernel that gives up sets RNNT_ERR_TIMEOUT; O is then
 * undefined.
 */
typedef struct {
  int rows, cols, batch;
  int in_dtype, out_dtype;        /* RNNT_F32 or RNNT_BF16 */
  int steps;                      /* 1 to 32 */
  float eps;
  long long in_ld, in_batch;      /* strides of G, elements (0: cols, rows * in_ld) */
  long long out_ld, out_batch;    /* strides of O, elements (0: cols, rows * out_ld) */
} rnnt_orth_dims;

size_t rnnt_orth_workspace_bytes(const rnnt_orth_dims* dims); /* 0: invalid dims */

rnnt_status rnnt_orth(const rnnt_orth_dims* dims, const void* G, void* O, void* ws,
                      size_t ws_bytes, int32_t* status, rnnt_stream stream);

/* ---- gradient clipping ---------------------------------------------------------
 * Over all elements of n tensors together:
 *   norm = sqrt(sum g^2),  scale = min(1, max_norm / (norm + eps)),  into = scale g
 * Squares are added in fp64 (fp32 in groups of 32, fp64 where that would leave the
 * range), in an order that follows from the list, the gradients' places modulo 16
 * bytes and the device; entries of any size add up.  The norm is given in fp32: one
 * past its range is infinite, as one of an infinite entry.  An infinite norm gives
 * scale 0, whatever the limit, NaN gives NaN, and `into` is the product (0 times an
 * infinite entry: NaN) all the same; rnnt_adamw leaves such an update out.
 */
typedef struct {
  int n;                   /* tensors, 0 to 2^16 */
  const long long* count;  /* host [n]: elements of each, dense, 0 allowed */
  const int* dtype;        /* host [n]: RNNT_F32 or RNNT_BF16 each; NULL: fp32 */
} rnnt_grad_list;          /* read before a call returns */

size_t rnnt_clip_workspace_bytes(const rnnt_grad_list* list); /* 0: invalid list */

/* grads, into: host [n] of device pointers (a tensor of 0 elements: anything), read
 * before the call returns.  into NULL: the norm alone; into[i] = grads[i]: in place
 * (nothing is written there when scale is 1); otherwise `into` overlaps nothing.
 * clip: fp32 [2] on the device, (norm, scale).  max_norm >= 0 (infinity: scale 1
 * while the norm is finite), eps >= 0. */
rnnt_status rnnt_clip(const rnnt_grad_list* list, const void* const* grads, void* const* into,
                      float max_norm, float eps, float* clip, void* ws, size_t ws_bytes,
                      rnnt_stream stream);

/* ---- AdamW update ---------------------------------------------------------------
 * For every element of n tensors, t the number of this update (from 1), s = clip's
 * scale (1 without clip):
 *   m <- beta1 m + (1 - beta1) s g,   v <- beta2 v + (1 - beta2) (s g)^2
 *   p <- p - lr (decay p + (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps))
 *   low <- p in bf16, where a copy is wanted
 * p, m, v are fp32, updated in place; g is read only, fp32 or bf16 by the list.
 * With clip, an update whose norm is not finite changes nothing and is not counted;
 * neither is one of a list without elements.
 */
typedef struct {
  double beta1, beta2;  /* [0,1) */
  float eps;            /* >= 0 (0: an element whose v is 0 gives NaN) */
  float lr;             /* used when the call's lr is NULL */
  float decay;          /* used when decays is NULL */
  const float* decays;  /* host [n], read before a call returns, or NULL */
} rnnt_adamw_opts;

/* params, grads, m, v, low: host [n] of device pointers, read before the call
 * returns (a tensor of 0 elements: anything).  low NULL, or an entry NULL: no bf16
 * copy.  The 5 n tensors do not overlap, but for gradients among themselves (the
 * same parameter twice is refused).  lr: one device fp32 or NULL; clip: rnnt_clip's
 * (norm, scale) or NULL.  steps: device int32 [2]: the updates taken so far, which
 * the call reads and adds 1 to (up to 2^31 - 1, where the count stays), and a word
 * that is 0 between calls; the caller clears both once.  So a captured call counts
 * its replays. */
rnnt_status rnnt_adamw(const rnnt_grad_list* list, const rnnt_adamw_opts* opts,
                       float* const* params, const void* const* grads, float* const* m,
                       float* const* v, void* const* low, const float* lr, const float* clip,
                       int32_t* steps, rnnt_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* RNNT_GB300_OPS_H */
