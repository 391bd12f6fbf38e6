/*
 * per_train.h -- C ABI of the operators a learner that replays sequences runs
 * next to the sum tree of per.h (libper.so, MI355X gfx950):
 *
 *   - an 8-bit row store: rows are quantised as they are written to the
 *     ring's slots and read back as sequences behind the sampled slots;
 *   - a gated linear recurrence over those sequences: forward, backward, and
 *     one step for an actor;
 *   - the distillation loss against a teacher's stored top logits, with its
 *     gradient; its per-row losses are the TD errors per_update takes.
 *
 * Conventions are those of per.h: pointers prefixed d_ are device pointers
 * owned by the caller, work is enqueued on the caller's stream without
 * waiting, nothing is allocated, all checks happen on the host before
 * anything is enqueued, and PER_EINVAL / PER_ENOSPC / PER_EHIP come with a
 * text in per_last_error().  There is no handle: every call takes the arrays
 * it works on.  Calls that share no writable array may overlap on different
 * streams.  The tensors belong to the current device.  A call whose largest
 * launch would take 2^32 work-items or more (its rows times the threads that a
 * row takes, at most 1024) is refused with PER_EINVAL; it can be made in pieces.
 *
 * Element types are PER_F32, PER_BF16 and PER_F16; strides count elements.
 * Sums, softmax statistics, scales and recurrent states are f32 or wider;
 * what is returned in 16 bits is rounded once, to nearest even.  Results do
 * not depend on the order in which workgroups run.
 */
#ifndef PER_TRAIN_H
#define PER_TRAIN_H

#include "per.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define PER_F32 0
#define PER_BF16 1
#define PER_F16 2

/* 8-bit formats of the row store */
#define PER_E4M3 0 /* 4 exponent and 3 mantissa bits, largest value 448, no infinities */
#define PER_I8 1   /* signed integers in [-127, 127] */

#define PER_MAX_ROW_DIM (1LL << 20)
#define PER_MAX_TOP 1024
#define PER_MAX_VOCAB (1LL << 24)
#define PER_SCAN_CHUNK 64

/*
 * The row store.  Row r of a store of `capacity` rows of `dim` values holds
 * dim codes at d_codes + r * codes_stride (bytes) and, for each group of
 * `group` neighbouring columns (32, 64, 128, or 0: the whole row; the last
 * group may be shorter), one f32 scale at d_scales + r * scales_stride
 * (floats).  A row's scales may lie behind its codes in one record.
 *
 * Quantising: a = the largest |x| of the group over its finite values, at
 * least 2^-100; scale = a * f32(1 / M) with M = 448 (e4m3) or 127 (i8); code =
 * x * f32(1 / scale) rounded to the nearest value of the format, ties to
 * even.  +-Inf becomes the code of +-M; NaN stays NaN in e4m3 and becomes 0
 * in i8.  Reading back: code * scale in f32, rounded to the output's type.
 *
 * per_rows_write: row j of d_src ([count x dim] of `type`, src_stride >= dim
 *   elements between rows) goes to slot (first + j) mod capacity, the slots
 *   of per_add with first = per_cursor before it.  count in [0, capacity],
 *   first in [0, capacity).
 * per_rows_write_at: row j goes to slot d_slots[j]; slots outside
 *   [0, capacity) are skipped, and of a slot given more than once the last
 *   position wins, as in per_update.  d_claims: [capacity] u32, all zero
 *   before the first call and zero again after each; calls that share it must
 *   be ordered.  count in [0, 2^31).
 * per_rows_read: output row b * window + s, for s in [0, window), is the row
 *   of slot (d_idx[b] + s) mod capacity; all zeros where d_idx[b] is outside
 *   [0, capacity).  d_out: [B * window x dim] of `type`, out_stride >= dim.
 *   B * window < 2^31.
 * Codes, scales, source and output must not overlap.
 */
int per_rows_write(int64_t capacity, int64_t dim, int32_t format, int32_t group, uint8_t* d_codes,
                   int64_t codes_stride, float* d_scales, int64_t scales_stride, int64_t count,
                   int64_t first, const void* d_src, int32_t type, int64_t src_stride,
                   hipStream_t stream);
int per_rows_write_at(int64_t capacity, int64_t dim, int32_t format, int32_t group,
                      uint8_t* d_codes, int64_t codes_stride, float* d_scales,
                      int64_t scales_stride, int64_t count, const int64_t* d_slots,
                      uint32_t* d_claims, const void* d_src, int32_t type, int64_t src_stride,
                      hipStream_t stream);
int per_rows_read(int64_t capacity, int64_t dim, int32_t format, int32_t group,
                  const uint8_t* d_codes, int64_t codes_stride, const float* d_scales,
                  int64_t scales_stride, int64_t B, const int64_t* d_idx, int64_t window,
                  void* d_out, int32_t type, int64_t out_stride, hipStream_t stream);

/*
 * The gated linear recurrence.  With f = 1 / (1 + exp(-g)), for each sequence
 * b and channel d
 *     h_t = f_t * h'_{t-1} + (1 - f_t) * x_t,
 * h' = 0 where d_reset[b, t] is not 0 (an episode begins at t) and the state
 * before it elsewhere; the state before t = 0 is h0 (0 when NULL).  A
 * sequence ends after d_length[b] steps (T when NULL; values outside [0, T]
 * are clamped): outputs and gradients past its end are 0, and what x, g and
 * dy hold there is not used.
 *
 * x, g, y, dy, dx and dg are [B x T x D] of `type` with unit channel stride
 * and their own strides between sequences (_sb) and steps (_st), so the two
 * halves of one projection can be taken in place.  d_reset: [B x T] u8, dense.
 * States (h0, h_last, dh_last, dh0) are dense [B x D] f32.
 *
 * per_scan_forward writes y, d_h_last (or NULL), the state after the last
 *   step of each sequence, and d_carries (or NULL), [B x ceil(T / 64) x D]
 *   f32: the state before each chunk of PER_SCAN_CHUNK steps, for the backward
 *   pass.  d_h_last may be d_h0.
 * per_scan_backward takes those carries, dy, and d_dh_last, the gradient of
 *   h_last (or NULL), and writes dx, dg and d_dh0 (or NULL).  States inside a
 *   chunk are computed again in f32 from its carry.
 * per_scan_workspace_bytes: device workspace both calls need (0 when the
 *   batch fills the chip without splitting the time axis), 16-byte aligned.
 *   Its contents are scratch of one call.
 * per_scan_step: one step of B sequences: x, g, y are [B x D] with the given
 *   row strides, d_reset [B] u8 or NULL, d_h_out may be d_h.
 */
int per_scan_workspace_bytes(int64_t B, int64_t T, int64_t D, size_t* out);
int per_scan_forward(int64_t B, int64_t T, int64_t D, int32_t type, const void* d_x, int64_t x_sb,
                     int64_t x_st, const void* d_g, int64_t g_sb, int64_t g_st,
                     const uint8_t* d_reset, const int64_t* d_length, const float* d_h0, void* d_y,
                     int64_t y_sb, int64_t y_st, float* d_h_last, float* d_carries, void* d_ws,
                     size_t ws_bytes, hipStream_t stream);
int per_scan_backward(int64_t B, int64_t T, int64_t D, int32_t type, const void* d_x, int64_t x_sb,
                      int64_t x_st, const void* d_g, int64_t g_sb, int64_t g_st,
                      const uint8_t* d_reset, const int64_t* d_length, const float* d_carries,
                      const void* d_dy, int64_t dy_sb, int64_t dy_st, const float* d_dh_last,
                      void* d_dx, int64_t dx_sb, int64_t dx_st, void* d_dg, int64_t dg_sb,
                      int64_t dg_st, float* d_dh0, void* d_ws, size_t ws_bytes,
                      hipStream_t stream);
int per_scan_step(int64_t B, int64_t D, int32_t type, const void* d_x, int64_t x_stride,
                  const void* d_g, int64_t g_stride, const uint8_t* d_reset, const float* d_h,
                  float* d_h_out, void* d_y, int64_t y_stride, hipStream_t stream);

/*
 * Distillation from a teacher's top logits.  Row n has student logits z over
 * V tokens and K teacher entries (token d_tidx[n, k], logit t_k); entries
 * whose token is outside [0, V) are absent.  With temperature tau,
 * q = softmax(z / tau) and
 *   without d_tlse: p = softmax(t / tau) over the entries present;
 *   with d_tlse [N] f32, the teacher's log-sum-exp of its logits / tau over
 *     its whole vocabulary: p_k = exp(t_k / tau - tlse), and the rest
 *     p_r = max(0, 1 - sum p_k) stands against the student's
 *     q_r = 1 - (the q of the distinct tokens present),
 *   loss_n = tau^2 [sum_k p_k (log p_k - log q_k) + p_r (log p_r - log q_r)],
 * where a term with p = 0 is 0, and so is the rest's when q_r = 0 (no token of
 * the rest, or all of them at -Inf).  log q_r is taken from the rest's own largest
 * logit, so it holds as well where q_r is too small for f32.  The gradient by z_j,
 * scaled by w_n, is tau w_n (q_j - p_j) with p_j the sum of the entries for token
 * j, or in place of p_j, for the tokens of the rest, p_r q_j / q_r.  A row has
 * loss 0 and gradient 0 when no entry is present (without d_tlse) or every student
 * logit is -Inf; NaN and +Inf logits give NaN.
 *
 * d_logits: [N x V] of `type`, stride >= V elements between rows; d_tidx:
 * dense [N x K] i32; d_tlogit: dense [N x K] of tlogit_type; 1 <= K <=
 * PER_MAX_TOP; 2^-20 <= tau <= 2^6.  The loss is tau^2 times a difference of
 * logarithms of sums, so its error grows as tau^2 whatever its own size: sums are
 * f32 within a thread and f64 from there on, which leaves about 2^-31 tau^2.
 *
 * per_distill: loss and gradient in one call.  d_weight: [N] f32 or NULL (1);
 *   the losses are not weighted, the gradient is; a row of weight 0 gets loss 0
 *   and gradient 0 whatever its logits and entries hold.  d_grad may be d_logits
 *   (with the same stride).
 * per_distill_forward: the losses, and d_saved [N x (4 + K)] f32 (or NULL):
 *   largest logit m, S = sum of exp((z - m) / tau) (0 for a row without loss),
 *   largest logit m_r of the rest, C = exp((m_r - m) / tau) / S - p_r / (sum of
 *   exp((z - m_r) / tau) over the rest), and the K probabilities p_k.  Without
 *   d_tlse, or where the rest has no mass, m_r = m and C = 1 / S or 0.
 * per_distill_backward: the gradient from d_saved, weighted by d_gloss [N]
 *   f32, the gradient by each row's loss; d_grad may be d_logits.
 * per_distill_workspace_bytes: device workspace of per_distill and
 *   per_distill_forward (0 for short rows), 16-byte aligned, scratch of one
 *   call.  per_distill does not look at it where a workgroup holds a whole row.
 */
int per_distill_workspace_bytes(int64_t N, int64_t V, int64_t K, int32_t type, size_t* out);
int per_distill(int64_t N, int64_t V, int64_t K, int32_t type, const void* d_logits,
                int64_t stride, const int32_t* d_tidx, const void* d_tlogit, int32_t tlogit_type,
                const float* d_tlse, double temperature, const float* d_weight, float* d_loss,
                void* d_grad, int64_t grad_stride, void* d_ws, size_t ws_bytes,
                hipStream_t stream);
int per_distill_forward(int64_t N, int64_t V, int64_t K, int32_t type, const void* d_logits,
                        int64_t stride, const int32_t* d_tidx, const void* d_tlogit,
                        int32_t tlogit_type, const float* d_tlse, double temperature,
                        float* d_loss, float* d_saved, void* d_ws, size_t ws_bytes,
                        hipStream_t stream);
int per_distill_backward(int64_t N, int64_t V, int64_t K, int32_t type, const void* d_logits,
                         int64_t stride, const int32_t* d_tidx, const void* d_tlogit,
                         int32_t tlogit_type, const float* d_tlse, double temperature,
                         const float* d_saved, const float* d_gloss, void* d_grad,
                         int64_t grad_stride, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* PER_TRAIN_H */
