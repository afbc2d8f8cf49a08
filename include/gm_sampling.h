/*
 * gm_sampling.h -- a class drawn from each row of logits over a class table on one GB300, by a
 * temperature, top-k, top-p and min-p, from given random numbers.
 *
 * For a row z of n_classes logits, with classes ordered by logit from the largest down, equal ones (0 and -0
 * are equal) from the lowest class up, and w_j = exp((z_j - max z) / T):
 *   top-k  keeps the first top_k classes (0: all);
 *   top-p  of these, the shortest run from the first whose sum of w reaches top_p times the sum of all of
 *          them, at least one class (1: all);
 *   min-p  of these, the classes with w_j >= min_p (0: all).
 *   The class drawn is the first, in class order, at which the sum of the kept w up to and with it is more than u
 *   times the sum of all kept w.
 * A logit of -inf is never kept. Where the largest is +inf, w is 1 there and 0 elsewhere. T = 0 keeps the largest alone.
 *
 * The weights are within 2^-28 of w relatively (or 2^-40 of the largest, up to 2^22 classes) and are summed exactly, as
 * 64-bit integers: a border between two classes is met to more than eight digits, and results do not depend on the launch.
 * z_j - max z is formed in fp32: a difference past 3.4e38 counts as infinite.
 */
#ifndef GM_SAMPLING_H
#define GM_SAMPLING_H

#include "gm_losses.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One value a row (device; NULL: the value for all rows beside it). */
typedef struct gm_draw_rule {
  const float* temperature; /* 0, or finite with log2(e) / T finite: T from 4.3e-39 */
  const int32_t* top_k;     /* >= 0    */
  const float* top_p;       /* 0 .. 1  */
  const float* min_p;       /* 0 .. 1  */
  float all_temperature;
  int32_t all_top_k;
  float all_top_p;
  float all_min_p;
} gm_draw_rule;

/* logits: device, n_rows (0 .. 2^31 - 256) rows of n_classes (1 .. 2^24) elements of type (GM_LOSS_*), ld apart. u: device, n_rows
 * floats in [0, 1). index, logprob, kept: device, n_rows each: the class; the log of its share of the kept
 * weights; how many classes were kept. A row that cannot be drawn from (a NaN, nothing but -inf, u or a value of the row's
 * rule out of range) has index -1, logprob NaN, kept 0. Work is queued on `stream`; the call does not wait and
 * needs no workspace. index, logprob and kept overlap nothing.
 * Errors: GM_ERR_INVALID_ARG (null or misaligned pointer, size out of range, ld < n_classes, unknown type, a value for all
 * rows out of range), GM_ERR_INDEX_OVERFLOW (a size above its limit), GM_ERR_CUDA (a launch failed, or a CUDA error from earlier work was
 * still pending: left pending, nothing queued). */
gm_status gm_draw(const void* logits, int64_t n_rows, int64_t n_classes, int64_t ld, int32_t type,
                  const gm_draw_rule* rule, const float* u, void* stream, int64_t* index, float* logprob, int32_t* kept);

#ifdef __cplusplus
}
#endif

#endif /* GM_SAMPLING_H */
