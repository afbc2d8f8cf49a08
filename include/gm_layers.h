/*
 * gm_layers.h -- what makes the rows H of gm_losses.h from other rows, on one GB300:
 * a matrix product with bias, activation and residual in its epilogue, and the norms
 * around a residual with its gate and scale. Forward and backward.
 *
 *   product   z = X W^T + b,   y = r + act(z)
 *             dz = g * act'(z),  dX = dz W,  dW = dz^T X,  db = sum of dz's rows; r's gradient is g
 *   norms     p = n(f) * after + after_bias      (f itself without after)
 *             x' = x + scale * gate * p
 *             y = n(x') * before + before_bias   (not computed without before)
 *             n(v) = v / sqrt(mean(v^2) + eps), or with the row's mean taken off v first
 *             backward, from gx and gy, the gradients by x' and y: with c the mean of a row,
 *               d = gy * before,  dx = gx + (d - n(x') c(d n(x')) - [layer] c(d)) / size(x')
 *               dp = scale * gate * dx,  dgate = scale * dx * p,  e = dp * after,
 *               df = (e - n(f) c(e n(f)) - [layer] c(e)) / size(f)
 *               dafter = sum dp * n(f), dafter_bias = sum dp, dbefore = sum gy * n(x'),
 *               dbefore_bias = sum gy; sums over rows, as is dgate of a gate that is a vector
 *
 * Conventions common to every call
 *   - All arrays are device memory of the current CUDA device; descriptors are host memory and
 *     only read during the call. Matrices have rows of consecutive elements, ld elements apart.
 *     Every array of a call has the descriptor's type, stats apart. Results do not overlap each
 *     other or any input, but where said.
 *   - Work is queued on `stream`; no call waits for it. Workspace is the caller's
 *     (gm_layer_config.workspace) or comes through gm_set_allocator's hooks, in stream order.
 *   - Every call returns a gm_status; nothing is thrown across the ABI.
 *   - Arithmetic and sums are fp32, results are rounded once, but: dz is rounded to a 16-bit
 *     operand type before the two products that read it (db is summed before that); f16's is scaled
 *     by a power of two first, so that its steps are at most 2^-37 of the largest finite gradient by y where
 *     they are not a rounding of dz itself. The slope
 *     of an activation is taken at z as it was kept, rounded to the operand type. Products on the
 *     tensor cores, forward and backward, add up to 1024 elements of 16 bits 16 at a time, each sum cut, not
 *     rounded, to 24 bits; such parts are added in fp32. f32 operands are three bf16 parts each, 64 elements
 *     at a time. No value is added atomically: results do not depend on the launch.
 */
#ifndef GM_LAYERS_H
#define GM_LAYERS_H

#include "gm_losses.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace of a call; NULL, or a NULL workspace: the hooks. */
typedef struct gm_layer_config {
  void* workspace;         /* 256-byte aligned; may be reused once the call's work on the stream is done */
  int64_t workspace_bytes; /* at least gm_linear_workspace's or gm_norm_workspace's answer               */
} gm_layer_config;

/* ---- product with bias, activation and residual -------------------------------------------- */

#define GM_ACT_NONE 0
#define GM_ACT_RELU 1      /* max(z, 0), slope 0 at 0                                    */
#define GM_ACT_GELU 2      /* z (1 + erf(z / sqrt 2)) / 2                                */
#define GM_ACT_GELU_TANH 3 /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2          */
#define GM_ACT_SILU 4      /* z / (1 + exp(-z))                                          */

typedef struct gm_linear {
  int64_t n_rows; /* 0 .. 2^31 - 256                       */
  int64_t dim;    /* 1 .. 2^24, elements of a row of X, W  */
  int64_t n_outs; /* 1 .. 2^24, rows of W, columns of y    */
  const void* x;
  int64_t x_ld;
  const void* w;
  int64_t w_ld;
  int32_t type;       /* GM_LOSS_F32, _BF16, _F16          */
  int32_t activation; /* GM_ACT_*                          */
} gm_linear;

/* bias: n_outs elements, or NULL; residual: n_rows x n_outs, or NULL. y: n_rows x n_outs; it may be
 * the residual (same address and ld). z: NULL, or n_rows x n_outs for X W^T + b as the backward call wants it.
 * Errors: GM_ERR_INVALID_ARG (null or misaligned pointer, size out of range, ld shorter than a row,
 * unknown type or activation), GM_ERR_INDEX_OVERFLOW (a size above its limit), GM_ERR_OOM, GM_ERR_WORKSPACE (the caller's
 * workspace is too small), GM_ERR_CUDA (a launch failed, or a CUDA error from earlier
 * work was still pending: left pending, nothing queued). A bounded wait that gives up leaves results incomplete; gm_loss_status
 * tells of it. */
gm_status gm_linear_forward(const gm_linear* p, const gm_layer_config* cfg, void* stream, const void* bias,
                            const void* residual, int64_t residual_ld, void* y, int64_t y_ld, void* z, int64_t z_ld);

/* grad: n_rows x n_outs, the gradient by y. z: gm_linear_forward's, NULL without activation. dx: n_rows x dim,
 * dw: n_outs x dim, dbias: n_outs; overwritten; each may be NULL (not computed), not all.
 * Errors: those of gm_linear_forward. */
gm_status gm_linear_backward(const gm_linear* p, const gm_layer_config* cfg, void* stream, const void* grad,
                             int64_t grad_ld, const void* z, int64_t z_ld, void* dx, int64_t dx_ld, void* dw,
                             int64_t dw_ld, void* dbias);

/* Bytes of workspace that suffice for a call (host only); backward: 0 or 1. Errors: those of the call's
 * arguments in p, GM_ERR_INVALID_ARG for a NULL bytes. */
gm_status gm_linear_workspace(const gm_linear* p, int32_t backward, int64_t* bytes);

/* ---- norms around a residual ------------------------------------------------------------------ */

#define GM_NORM_RMS 0
#define GM_NORM_LAYER 1
#define GM_GATE_NONE 0
#define GM_GATE_VECTOR 1 /* dim elements, the same for every row */
#define GM_GATE_MATRIX 2 /* n_rows x dim                         */

typedef struct gm_norm {
  int64_t n_rows; /* 0 .. 2^31 - 256 */
  int64_t dim;    /* 1 .. 2^24       */
  int32_t type;   /* GM_LOSS_*       */
  int32_t norm;   /* GM_NORM_*       */
  int32_t gate_kind;
  float scale;    /* finite          */
  float eps;      /* finite, >= 0; a row of zeros has a norm of zeros where eps > 0 */
  const void* x;
  int64_t x_ld;
  const void* f; /* NULL: x' = x; then after, after_bias are NULL and there is no gate */
  int64_t f_ld;
  const void* after; /* dim elements each; a bias only with its weight */
  const void* after_bias;
  const void* gate;
  int64_t gate_ld;
  const void* before;
  const void* before_bias;
} gm_norm;

/* x_out: x', may be x itself (same address and ld); NULL only without f. y: with before, else NULL. Either x_out or
 * y is wanted. stats: 4 floats a row, 16-byte aligned, for the backward call (mean and 1 / size of f, of x'; mean 0 of
 * GM_NORM_RMS), or NULL. y is of x' before it is rounded. Errors: those of gm_linear_forward; no workspace is used. */
gm_status gm_norm_forward(const gm_norm* n, void* stream, void* x_out, int64_t x_out_ld, void* y, int64_t y_ld,
                          float* stats);

/* What gm_norm_backward computes: NULL members are not computed, those of inputs that the call does not have are NULL. */
typedef struct gm_norm_grads {
  void* x; /* n_rows x dim */
  int64_t x_ld;
  void* f; /* n_rows x dim */
  int64_t f_ld;
  void* gate; /* as the gate */
  int64_t gate_ld;
  void* after; /* dim elements each */
  void* after_bias;
  void* before;
  void* before_bias;
} gm_norm_grads;

/* n: as in the forward call, x as it was before it. stats: the forward call's. gx: gradient by x', or NULL (zeros); gy: by y, with before (NULL: zeros).
 * Errors: those of gm_linear_forward. */
gm_status gm_norm_backward(const gm_norm* n, const gm_layer_config* cfg, void* stream, const float* stats,
                           const void* gx, int64_t gx_ld, const void* gy, int64_t gy_ld, const gm_norm_grads* grads);

/* Bytes of workspace that suffice for gm_norm_backward (host only). Errors: those of its arguments in n,
 * GM_ERR_INVALID_ARG for a NULL bytes. */
gm_status gm_norm_workspace(const gm_norm* n, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* GM_LAYERS_H */
