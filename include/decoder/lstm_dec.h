/*
 * lstm_dec.h -- C ABI of the decoder operators on MI355X (gfx950): what an
 * encoder-decoder recurrent network needs beside its stacks (lstm_fwd.h,
 * lstm_bwd.h).
 *
 *   lstm_attn_fwd, lstm_attn_bwd   attention of a decoder's outputs over an
 *                                  encoder's outputs, and its gradients
 *   lstm_beam_step                 one step of beam search: selection over
 *                                  beams and vocabulary, reordering of the
 *                                  recurrent states
 *
 * ---- attention ------------------------------------------------------------
 * For sentence b, query step t, query head h (it reads key head h / (Hq/Hkv)):
 *     z_s  = scale * <q[b,t,h], k[b,s,h']>              s in keys(b)
 *     lse  = log sum_s exp(z_s) ,   p_s = exp(z_s - lse)
 *     o[b,t,h] = sum_s p_s v[b,s,h']
 * keys(b) = { s < kv_len[b] (if given) and key_mask[b][s] != 0 (if given) }.
 * A kv_len below 0 counts as 0, one above S as S.  What stands in k and v at
 * other positions is never used: infinities and NaN there change nothing.
 * Where keys(b) is empty (or S is 0), o = 0, lse = -inf and every gradient is 0,
 * whatever q and dout hold.
 * Gradients, with dP_s = <do, v_s> and delta = <do, o>:
 *     dv_s = sum p_s do ,  dz_s = p_s (dP_s - delta)
 *     dq = scale sum_s dz_s k_s ,  dk_s = scale sum dz_s q
 * (the sums of dk and dv run over the steps and over the query heads that share
 * the key head; both are 0 at positions outside keys(b)).
 *
 * Layouts: q, o [B][Tq][Hq][D], k, v [B][S][Hkv][D] by strides in elements
 * (sentence, step, head); the D values of a head are contiguous, so both the
 * recurrence's [T][B][H] outputs and [B][T][H] tensors are read in place.
 * The gradients have strides of their own.  lse [B][Hq][Tq] fp32, dense.
 * kv_len [B] int32, key_mask [B][S] bytes, dense.  Products take dtype operands
 * (bf16: p and dz enter theirs as the sum of two bf16 values, within 2^-16) and
 * accumulate in fp32; softmax statistics, lse and delta are fp32.  delta is taken
 * from the o that is handed in and, for bf16, from what o's rounding left where
 * o_rest is given: the forward writes it there, the backward reads it.  An infinity
 * in v at a key or in dout reaches o and the gradients as an infinity or NaN.  All
 * sums are taken in a fixed order, so results are deterministic.
 *
 * Limits: D a multiple of 8, 8 ... 256; Hq a multiple of Hkv; q, k, v, o, dout
 * and the gradients aligned to 16 bytes and every stride a multiple of 16 bytes,
 * kv_len and lse aligned to 4; scale > 0 and at most 2.3e38 (0 selects
 * 1/sqrt(D)); B*Hq*Tq and B*S at most 2^31 - 4096, for the gradients also
 * B*Hkv*(ceil(Tq*Hq/(64*Hkv)) + ceil(S/64)).  Byte offsets are 64-bit.
 *
 * ---- beam search ----------------------------------------------------------
 * Sentence b holds K beams.  A beam that is not finished proposes every token v:
 *     cand = scores[b,k] + logits[b,k,v] - log sum_w exp(logits[b,k,w])
 *     rank = cand / ((5 + n) / 6)^alpha ,   n = lengths[b,k] + 1
 * A finished beam proposes eos only, with cand = scores[b,k], n = lengths[b,k].
 * The K best of all proposals by rank are taken, ties to the lowest k*V + v;
 * proposals of rank -inf (also every other token of a finished beam) count as
 * last, in that order.  Within a beam the order by rank is the order by logits.
 * A beam whose logits hold NaN or +inf, or are all -inf, or whose score is no
 * finite number, proposes nothing but rank -inf.  Outputs, best first:
 *     tokens, parents (the beam k), scores_out (cand), lengths_out (n),
 *     finished_out = finished[b,parent] or token == eos
 * and the states of the chosen beams: for n_states layers,
 *     h_out[l, b*K + i] = h[l, b*K + parents[b,i]] ,  c likewise.
 * cand and rank are computed in 64 bits, since proposals of different beams may
 * lie closer together than fp32 tells apart.  The log-sum-exp takes the largest
 * logits' exponentials and all sums beyond 8 values in 64 bits, the other
 * exponentials in fp32: it is within 2^-19 at worst (every rounding one way), 2^-26
 * to 2^-29 for logits of a normal distribution, and proposals of different beams
 * that lie closer together than that may change places.  cand is at most scores[b,k].
 *
 * Layouts: logits [B][K][V] dtype, dense rows of V with beam stride
 * logits_stride (elements, 0 selects V); scores, scores_out [B][K] fp32;
 * finished(_out) [B][K] bytes; lengths(_out), tokens, parents [B][K] int32;
 * h [L][B*K][H] dtype, c [L][B*K][H] fp32 (each may be NULL, with its output).
 * Outputs must not overlap inputs.
 * Limits: K 1 ... 16, K <= V <= 2^20, B*K < 2^24, L*H < 2^23,
 * L*B*K < 2^31.
 *
 * ---- all ------------------------------------------------------------------
 * Ownership, streams and errors as in lstm_fwd.h: every tensor pointer is a
 * device pointer owned by the caller, `ws` holds the size function's bytes,
 * 256-byte aligned (contents
 * on entry ignored), work is enqueued on `stream`, arguments are checked on the
 * host before anything is enqueued, and nothing throws.
 */
#ifndef LSTM_DEC_H
#define LSTM_DEC_H

#include "../lstm_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Strides in elements: sentence, step, head. */
typedef struct {
  int64_t b, t, h;
} lstm_attn_stride_t;

/* Problem description.  Zero-initialise and set what you need. */
typedef struct {
  int32_t B, Tq, S, Hq, Hkv, D; /* S may be 0 */
  int32_t dtype;                /* lstm_dtype_t of every tensor but lse */
  float scale;                  /* 0: 1/sqrt(D) */
  lstm_attn_stride_t q, k, v, o;
  lstm_attn_stride_t dout, dq, dk, dv; /* lstm_attn_bwd only */
  void *o_rest;                 /* NULL, or B*Tq*Hq*D bf16 values on the device, aligned to 16 bytes: what o's
                                   rounding leaves (training; not used for fp32) */
} lstm_attn_desc_t;

/* Checks of a description without a call (host only): the status that
 * lstm_attn_fwd (train = 0) or lstm_attn_bwd (train = 1) would return for it,
 * pointers aside. */
lstm_status_t lstm_attn_validate(const lstm_attn_desc_t *d, int train);

/* Bytes of the workspace of lstm_attn_fwd and lstm_attn_bwd; 0 if `d` is
 * invalid or unsupported. */
size_t lstm_attn_workspace_size(const lstm_attn_desc_t *d);
size_t lstm_attn_bwd_workspace_size(const lstm_attn_desc_t *d);

/* o and lse (lse may be NULL).  kv_len and key_mask may each be NULL. */
lstm_status_t lstm_attn_fwd(const lstm_attn_desc_t *d, const void *q, const void *k, const void *v,
                            const int32_t *kv_len, const uint8_t *key_mask, void *o, float *lse, void *ws,
                            hipStream_t stream);

/* dq, dk, dv from dout and from the o and lse of lstm_attn_fwd on the same inputs. */
lstm_status_t lstm_attn_bwd(const lstm_attn_desc_t *d, const void *q, const void *k, const void *v,
                            const int32_t *kv_len, const uint8_t *key_mask, const void *o, const float *lse,
                            const void *dout, void *dq, void *dk, void *dv, void *ws, hipStream_t stream);

typedef struct {
  int32_t B, K, V;
  int32_t dtype;         /* lstm_dtype_t of logits and h */
  int32_t eos;           /* 0 ... V-1 */
  float alpha;           /* exponent of the length penalty, >= 0 */
  int32_t L, H;          /* states: layers and width (both 0 without states) */
  int64_t logits_stride; /* elements from one beam's logits to the next; 0: V */
} lstm_beam_desc_t;

/* Bytes of the workspace of lstm_beam_step; 0 if `d` is invalid or unsupported. */
size_t lstm_beam_workspace_size(const lstm_beam_desc_t *d);

/* One step.  Any of h, c may be NULL (then its output is ignored). */
lstm_status_t lstm_beam_step(const lstm_beam_desc_t *d, const void *logits, const float *scores,
                             const uint8_t *finished, const int32_t *lengths, int32_t *tokens, int32_t *parents,
                             float *scores_out, uint8_t *finished_out, int32_t *lengths_out, const void *h,
                             const float *c, void *h_out, float *c_out, void *ws, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LSTM_DEC_H */
