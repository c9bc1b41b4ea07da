/*
 * lstm_block.h -- C ABI of the block operators on MI355X (gfx950): what a deep
 * recurrent network has between and beside its stacks (lstm_fwd.h), and after
 * their gradients (lstm_bwd.h).
 *
 *   lstm_norm_fwd, lstm_norm_bwd   layer norm of a residual sum, and its gradients
 *   lstm_glr_fwd, lstm_glr_bwd     gated linear recurrence over a sequence (one
 *                                  step or many), and its gradients
 *   lstm_clip                      the norm of many tensors' values together, and
 *                                  the tensors scaled to a largest norm
 *
 * ---- sequences ------------------------------------------------------------
 * Tensors [B][T][width] by strides in elements (sentence, step); the values of a
 * step are contiguous.  Both the recurrence's [T][B][H] outputs and [B][T][H]
 * tensors are read in place, and so are parts of a wider tensor.  Addresses and
 * strides need no alignment beyond the element's; the steps of an output must not
 * overlap.  lengths [B] int32 (NULL: T
 * each) leaves the steps t >= lengths[b] out: below 0 counts as 0, above T as T.
 * What stands in an input there is never used, infinities and NaN change
 * nothing; outputs and gradients are 0 there.
 *
 * ---- layer norm -----------------------------------------------------------
 * For every step of every sentence, over its N values:
 *     s = x + r          (rounded to dtype and stored; s = x without r)
 *     mean = sum s / N ,  rstd = 1 / sqrt(sum (s - mean)^2 / N + eps)
 *     y = w (s - mean) rstd + b          (w, b [N] dtype; NULL: 1 and 0)
 * and with n = (s - mean) rstd, g = w dy:
 *     dx = rstd (g - sum g / N - n sum(g n) / N) + ds        (ds NULL: 0)
 *     dw = sum dy n ,  db = sum dy           over all steps of all sentences
 * ds is the gradient that reaches s past the norm; dx is the gradient of x and
 * of r alike.  mean, rstd [B][T] fp32.  The mean is rounded to fp32 before it is
 * subtracted (twice at widths above 1024), so a row whose spread is not much more
 * than 2^-24 of its mean is normalised as accurately as that; rows of one value give
 * y = b.  Sums and squares are fp32: values' sums have to stay below 2^128, and so
 * do those of their squared distances to the mean.
 *
 * ---- gated linear recurrence ----------------------------------------------
 * For every channel of every sentence, c_{-1} = c0 (NULL: 0):
 *     a_t = sigmoid(f_t) ,  z_t = u_t or tanh(u_t)
 *     c_t = a_t c_{t-1} + (1 - a_t) z_t
 *     y_t = c_t, or sigmoid(o_t) c_t where o is given
 *     cT  = c after the sentence's last step (c0 if it has none)
 * f, u and o do not depend on c (a projection of the layer's input makes them),
 * so the steps are joined by a scan.  Gradients, with dy_t of y_t, dcT of cT:
 *     d_t = sigmoid(o_t) dy_t + a_{t+1} d_{t+1}     (dcT at the last step)
 *     df = a (1 - a) (c_{t-1} - z) d ,  du = (1 - a) d (1, or 1 - z^2)
 *     do = sigmoid(o) (1 - sigmoid(o)) c dy ,  dc0 = a_0 d_0
 * c0, cT, dcT, dc0 [B][H] fp32, dense.  a and 1 - a are formed apart, each within
 * 7 x 2^-24 of itself, of bf16 f within (6 + 1.3 |f|) 2^-24 (but not below 2^-126), so
 * gates that are almost shut or open keep their accuracy.  tanh of fp32 u is within
 * 12 x 2^-24 of itself, of bf16 u within 2^-17.  An infinity or NaN in u or f reaches
 * later steps as infinity or NaN.
 * A sentence's stretches of steps are worked on side by side and wait for one
 * another's states.  Every wait ends by itself; one that passes wait_timeout_us all
 * the same leaves NaN in what depends on it, and lstm_glr_last_error reports it (the
 * call does not sync).
 *
 * ---- clipping -------------------------------------------------------------
 *     norm = sqrt(sum over all tensors of x^2) ,  coef = min(1, max_norm / (norm + eps))
 *     dst = coef src       for every tensor (a NULL dst is left out of this)
 * dst may be src.  Sums are taken in 64 bits, so no square overflows; a NaN makes
 * coef NaN, an infinity makes it 0, as the formula says.  With an infinite max_norm
 * coef is 1 whatever the norm, and where norm + eps is 0.  out holds norm and coef.
 *
 * ---- all ------------------------------------------------------------------
 * dtype is an lstm_dtype_t; arithmetic and statistics are fp32 or wider, each
 * output is rounded once.  grad_dtype is the type of the sequences' gradients (dy,
 * ds, dx, df, du, do): LSTM_F32, which lstm_bwd takes and gives, or with bf16
 * tensors also LSTM_BF16; dw, db, dcT and dc0 are fp32.  All sums are taken in a
 * fixed order, so results are deterministic.  Outputs must not overlap
 * inputs or each other, but for s, which may be x or r with its strides, and dst,
 * which may be its own src (those that begin at one address are refused, dst apart).
 * Limits: N at most 16384; B*T and B*H at most 2^31 - 65536, B*T*H at most
 * 2^42; eps > 0.
 * Ownership, streams and errors as in lstm_fwd.h: every tensor pointer is a
 * device pointer owned by the caller, workspaces and tables hold the size
 * functions' bytes, 256-byte aligned, work is enqueued on `stream`, arguments
 * are checked on the host before anything is enqueued, and nothing throws.
 */
#ifndef LSTM_BLOCK_H
#define LSTM_BLOCK_H

#include "../lstm_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Strides in elements: sentence, step. */
typedef struct {
  int64_t b, t;
} lstm_seq_stride_t;

/* Descriptions.  Zero-initialise and set what you need. */
typedef struct {
  int32_t B, T, N;
  int32_t dtype, grad_dtype;
  float eps;
  lstm_seq_stride_t x, r, s, y; /* r with a residual only; s: of what is normalised (the backward
                                   reads it: without a residual, x's) */
  lstm_seq_stride_t dy, ds, dx; /* lstm_norm_bwd only */
} lstm_norm_desc_t;

/* Checks of a description without a call (host only): the status that
 * lstm_norm_fwd (train = 0) or lstm_norm_bwd (train = 1) would return for it,
 * pointers aside. */
lstm_status_t lstm_norm_validate(const lstm_norm_desc_t *d, int train);

/* Bytes of the workspace of lstm_norm_bwd; 0 if `d` is invalid or unsupported. */
size_t lstm_norm_bwd_workspace_size(const lstm_norm_desc_t *d);

/* y, and where given s (needs r), mean and rstd (the backward needs both). */
lstm_status_t lstm_norm_fwd(const lstm_norm_desc_t *d, const void *x, const void *r, const void *w, const void *b,
                            const int32_t *lengths, void *s, void *y, float *mean, float *rstd, hipStream_t stream);

/* dx, and where given dw and db, from the s (x without a residual), mean and rstd of
 * lstm_norm_fwd. */
lstm_status_t lstm_norm_bwd(const lstm_norm_desc_t *d, const void *s, const void *w, const int32_t *lengths,
                            const float *mean, const float *rstd, const void *dy, const void *ds, void *dx, float *dw,
                            float *db, void *ws, hipStream_t stream);

typedef enum { LSTM_GLR_LINEAR = 0, LSTM_GLR_TANH = 1 } lstm_glr_cand_t;

typedef struct {
  int32_t B, T, H;
  int32_t dtype, grad_dtype;
  int32_t cand;                         /* lstm_glr_cand_t: what z is of u */
  lstm_seq_stride_t f, u, o, y;         /* o with an output gate only */
  lstm_seq_stride_t dy, df, du, dout_o; /* lstm_glr_bwd only; dout_o: of do */
  int64_t wait_timeout_us;              /* limit of a wait for the state before a stretch of steps, in
                                           microseconds of the kernel's own running; 0 selects the default
                                           (2 s); negative makes every wait that is not already satisfied
                                           fail at once (exercises the timeout path without waiting) */
} lstm_glr_desc_t;

lstm_status_t lstm_glr_validate(const lstm_glr_desc_t *d, int train);

/* Bytes of the reserve that lstm_glr_fwd fills for lstm_glr_bwd (states between
 * stretches of steps); 0 if `d` is invalid or unsupported. */
size_t lstm_glr_reserve_size(const lstm_glr_desc_t *d);

/* Bytes of the workspace of lstm_glr_fwd and lstm_glr_bwd; 0 if `d` is invalid or unsupported. */
size_t lstm_glr_workspace_size(const lstm_glr_desc_t *d);

/* y, and where given cT and reserve.  o, c0 and lengths may each be NULL. */
lstm_status_t lstm_glr_fwd(const lstm_glr_desc_t *d, const void *f, const void *u, const void *o, const float *c0,
                           const int32_t *lengths, void *y, float *cT, void *reserve, void *ws, hipStream_t stream);

/* df, du, and do where o is given, dc0 where it is given, from dy and dcT (may be
 * NULL) and the reserve of lstm_glr_fwd on the same inputs. */
lstm_status_t lstm_glr_bwd(const lstm_glr_desc_t *d, const void *f, const void *u, const void *o, const float *c0,
                           const int32_t *lengths, const void *reserve, const void *dy, const float *dcT, void *df,
                           void *du, void *dout_o, float *dc0, void *ws, hipStream_t stream);

/*
 * Waits for `stream`, then reads the error word that the last lstm_glr_fwd
 * (train = 0) or lstm_glr_bwd (train = 1) of this description left in `ws`, if it
 * was the last call on it: LSTM_OK or LSTM_ERR_BARRIER_TIMEOUT.
 */
lstm_status_t lstm_glr_last_error(const lstm_glr_desc_t *d, int train, const void *ws, hipStream_t stream);

/* One tensor: `count` contiguous elements. */
typedef struct {
  const void *src;
  void *dst;
  int64_t count; /* may be 0 */
  int32_t dtype; /* of src and dst */
  int32_t reserved;
} lstm_clip_tensor_t;

/* Bytes of the table of n tensors (at least 1, at most 2^20, 2^42 elements in all);
 * 0 if the list is invalid. */
size_t lstm_clip_table_size(const lstm_clip_tensor_t *tensors, int32_t n);

/* Writes the table (device memory) that lstm_clip reads: once for a list of
 * tensors, however often they are clipped. */
lstm_status_t lstm_clip_table(const lstm_clip_tensor_t *tensors, int32_t n, void *table, hipStream_t stream);

/* Clips the tensors of the table, which lstm_clip_table has written from the same
 * list; out [2] fp32: norm and coef.  The table holds the call's partial sums too,
 * so calls that overlap need one each. */
lstm_status_t lstm_clip(const lstm_clip_tensor_t *tensors, int32_t n, void *table, double max_norm, double eps,
                        float *out, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LSTM_BLOCK_H */
