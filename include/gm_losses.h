/*
 * gm_losses.h -- losses over a large class table on one GB300: softmax cross
 * entropy and distillation from a teacher's top entries, forward and backward.
 *
 * Both work on logits that are a product and are never stored,
 *
 *   Z = H W^T,   H: n_rows x dim (states),   W: n_classes x dim (class table),
 *
 * in pieces of the classes where what is kept of their size would pass a bound. The teacher of the distillation is a CSR matrix of
 * n_rows x n_classes (gm_csr, as gm_spgemm writes it: columns ascending in a row),
 * so rows of a sparse product C = A * B serve as one without conversion.
 *
 *   cross entropy   lse_i  = log sum_j exp(z_ij)
 *                   loss_i = lse_i - z_i,t(i)
 *   distillation    q_i    = softmax of row i's stored values / T
 *                   lse_t_i = log sum_j exp(z_ij / T)
 *                   kl_i   = sum_k q_ik (log q_ik - z_ik / T + lse_t_i)
 *   gradient        G_ij   = (g_loss_i + g_lse_i) exp(z_ij - lse_i) - g_loss_i [j = t(i)]
 *                            + g_kl_i / T (exp(z_ij / T - lse_t_i) - q_ij)
 *                   dH = G W,  dW = G^T H
 *
 * Conventions common to every call
 *   - All arrays are device memory of the current CUDA device; descriptors
 *     (gm_logits, gm_labels, gm_csr, gm_loss_config) are host memory and only read
 *     during the call.
 *   - Work is queued on `stream`; a call does not wait for it unless
 *     GM_LOSS_CHECK is set. Workspace is the caller's (gm_loss_config.workspace), or
 *     comes through gm_set_allocator's hooks, in stream order, and is given back
 *     before the call returns.
 *   - Every call returns a gm_status; nothing is thrown across the ABI.
 *   - One row, or up to 8 of f32, of dim up to 4096: fp32 arithmetic throughout, G too.
 *     Others: products on the tensor cores with fp32 sums, which are cut, not rounded,
 *     to 24 bits for up to 1024 elements at a time; bf16 and f16 operands as they are, f32
 *     operands as three bf16 parts each. Before the gradient products G is rounded to
 *     the operands' 16-bit type; with at most 128 rows the remainder is kept beside it in that
 *     type, and f32's G is three bf16 parts. Maxima, sums of exponentials and losses
 *     are fp32; dH and dW are rounded once, from fp32 sums. The results do not depend
 *     on the launch (no atomics on values).
 *   - A row of H is read even when its target is the ignored one: such a row's
 *     values must be finite for dW to be, but they do not change any result.
 */
#ifndef GM_LOSSES_H
#define GM_LOSSES_H

#include "gm_spgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of H, W and of their gradients. */
#define GM_LOSS_F32 0
#define GM_LOSS_BF16 1
#define GM_LOSS_F16 2

/* The logits Z = H W^T. Rows of H and W are dim consecutive elements, ld elements
 * apart (ld >= dim). 16-bit rows that start on 16-byte boundaries are read in place;
 * others, and f32 ones, are laid out in workspace first. */
typedef struct gm_logits {
  int64_t n_rows;    /* 0 .. 2^31 - 256                    */
  int64_t n_classes; /* 1 .. 2^31 - 256                    */
  int64_t dim;       /* 1 .. 2^24                          */
  const void* h;     /* device, n_rows rows                */
  int64_t h_ld;
  const void* w;     /* device, n_classes rows             */
  int64_t w_ld;
  int32_t type;      /* GM_LOSS_*                          */
} gm_logits;

/* The class each row should have. Rows with ignore_index have loss 0 and no
 * gradient by it; grad_lse, the derivative by their lse, counts. A target outside
 * [0, n_classes) that is not ignore_index gives loss NaN, no gradient by loss or lse,
 * and GM_ERR_BAD_INDEX from gm_loss_status. */
typedef struct gm_labels {
  const void* target;   /* device, n_rows int64 (int32 with target32) */
  int64_t ignore_index;
  int32_t target32;     /* 1: targets are int32                       */
} gm_labels;

#define GM_LOSS_CHECK 1 /* wait for the work and return what this call met (as gm_loss_status would, which then
                           does not tell of it); other calls' reports stay where they are */

/* Tuning; zero selects the automatic value. NULL is the same as all zeros. */
typedef struct gm_loss_config {
  int64_t workspace_cap_bytes; /* bound on the piece of G a backward call holds; 0 = 512 MiB, f16 (which
                                  may keep G at two scales) 1 GiB; the narrowest piece has 256 classes.
                                  A forward call's row statistics, 16 bytes a row and 128 classes (f32 of at
                                  most 128 rows: 64), keep to 512 MiB in pieces of two such at least */
  int32_t flags;               /* GM_LOSS_CHECK                                                  */
  void* workspace;             /* device memory for the call, 256-byte aligned (NULL: the hooks); it
                                  may be reused once the call's work on the stream is done       */
  int64_t workspace_bytes;     /* at least gm_loss_workspace's answer for the same call          */
} gm_loss_config;

/* Bytes of workspace a call needs (host only): of gm_xent_* with teacher_nnz < 0, of
 * gm_distill_* with the teacher's entries; backward: 0 for a forward call, 1 for a
 * backward one. For callers that own the memory, for example while work is captured
 * into a CUDA graph. Errors: those of the call's arguments in z and cfg (whose flags and
 * workspace do not matter), GM_ERR_INVALID_ARG for a NULL bytes. */
gm_status gm_loss_workspace(const gm_logits* z, int64_t teacher_nnz, int32_t backward, const gm_loss_config* cfg,
                            int64_t* bytes);

/* loss and lse: device, n_rows floats, both written.
 * Errors: GM_ERR_INVALID_ARG (null or misaligned pointer, size out of range, ld < dim,
 * unknown type or flag), GM_ERR_INDEX_OVERFLOW (n_rows, n_classes or dim above its
 * limit), GM_ERR_OOM, GM_ERR_WORKSPACE (the caller's workspace is too
 * small), GM_ERR_CUDA (a launch failed, or a CUDA error from earlier work was still pending: left pending, nothing queued); with GM_LOSS_CHECK those of
 * gm_loss_status. */
gm_status gm_xent_forward(const gm_logits* z, const gm_labels* labels, const gm_loss_config* cfg, void* stream,
                          float* loss, float* lse);

/* lse: gm_xent_forward's. grad_loss, grad_lse: device, n_rows floats, the derivatives of
 * the caller's objective by loss and lse (grad_lse may be NULL: zeros). dh: n_rows rows of
 * dim elements of z->type, dh_ld apart; dw: n_classes rows, dw_ld apart; both are
 * overwritten; either may be NULL (not computed), not both.
 * Errors: those of gm_xent_forward. */
gm_status gm_xent_backward(const gm_logits* z, const gm_labels* labels, const gm_loss_config* cfg, void* stream,
                           const float* lse, const float* grad_loss, const float* grad_lse, void* dh, int64_t dh_ld,
                           void* dw, int64_t dw_ld);

/* teacher: n_rows x n_classes; value_type (GM_VALUE_*) and index_type (GM_INDEX_*) say
 * its arrays' types. Columns of a row ascend strictly. A value of -inf has probability 0;
 * a row without entries, or with nothing but -inf, has kl 0 and no gradient. A row with a
 * column out of range or out of order, or row pointers that decrease or leave [0, nnz],
 * or that starts before the end of an earlier row, has kl NaN, no gradient, and
 * GM_ERR_BAD_INDEX from gm_loss_status; other rows are as they would be without it. temperature: finite,
 * above 0 (log2(e) / T is finite too: T from 4.3e-39). labels: NULL, or the rows' targets, whose cross entropy (at temperature 1) the
 * same pass then returns in loss and lse (both NULL without labels).
 * Errors: those of gm_xent_forward, and GM_ERR_DIM_MISMATCH when the teacher's sizes are
 * not n_rows x n_classes. */
gm_status gm_distill_forward(const gm_logits* z, const gm_csr* teacher, int32_t value_type, int32_t index_type,
                             float temperature, const gm_labels* labels, const gm_loss_config* cfg, void* stream,
                             float* kl, float* lse_t, float* loss, float* lse);

/* lse_t and, with labels, lse: gm_distill_forward's. grad_kl: derivatives by kl;
 * grad_loss and grad_lse as in gm_xent_backward, read with labels only.
 * Errors: those of gm_distill_forward. */
gm_status gm_distill_backward(const gm_logits* z, const gm_csr* teacher, int32_t value_type, int32_t index_type,
                              float temperature, const gm_labels* labels, const gm_loss_config* cfg, void* stream,
                              const float* lse_t, const float* grad_kl, const float* lse, const float* grad_loss,
                              const float* grad_lse, void* dh, int64_t dh_ld, void* dw, int64_t dw_ld);

/* Waits for the stream and returns what the losses' calls of this device, on any stream, have met
 * since the last gm_loss_status, calls with GM_LOSS_CHECK apart: GM_ERR_DEVICE_TIMEOUT (a bounded wait in a
 * kernel gave up: that call's losses and what it summed of dh are NaN, other gradients of it
 * incomplete; other calls are not touched), GM_ERR_BAD_INDEX (a bad target or teacher row), GM_ERR_CUDA,
 * GM_ERR_OOM (4 bytes could not be had; nothing is cleared), or GM_OK. Reading clears; a report that
 * arrives meanwhile is told now or next time. */
gm_status gm_loss_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GM_LOSSES_H */
