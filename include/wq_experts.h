/*
 * wq_experts.h -- C ABI of the experts' routing (MI355X, gfx950): which experts
 * a token meets and with what weight, the order that sorts all choices by
 * expert (what wq_block_grouped_linear and wq_int8_grouped_linear take), and the
 * weighted sum that brings the experts' rows back to their tokens.
 *
 * Conventions are those of wq.h: device pointers owned by the caller, row-major
 * tensors, bf16 as uint16 bit patterns, stream-ordered calls that neither wait
 * nor allocate, every check on the host before anything is enqueued,
 * wq_last_error() for the reason.  Pointers are aligned to their type, those of
 * bf16 tensors with N % 8 == 0 to 16 bytes.
 */
#ifndef WQ_EXPERTS_H
#define WQ_EXPERTS_H

#include "wq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WQ_MAX_EXPERTS 1024
#define WQ_MAX_TOP 32
#define WQ_MAX_EXPERT_GROUPS 64

/* Scores of a token's logits l_e. */
enum {
  WQ_SCORE_SOFTMAX = 0, /* exp(l_e - max) / sum over all E experts of exp(l - max) */
  WQ_SCORE_SIGMOID = 1  /* 1 / (1 + exp(-l_e)) */
};

/*
 * Route M tokens to `top` of E experts each.
 *   choice c_e = score s_e + bias_e; without a bias (and without pairs) experts
 *   are compared by their logits, which order them alike.  An expert is never
 *   picked whose logit, or choice, is -infinity.
 *   With `groups` > 1 (a divisor of E) only experts of the `keep` best groups of
 *   E / groups consecutive experts are picked.  A group's value is its largest
 *   choice, or with `pairs` the sum of its two largest (of one, if it has no two
 *   that can be picked).
 *   The `top` largest choices are picked in their order, and their weights are
 *     w_e = scale * s_e                                        (renormalize == 0)
 *     w_e = scale * (s_e / sum of the picked s), 0 if that is 0 (otherwise)
 *   Ties go to the lowest index, of experts and of groups; a NaN is larger than
 *   any number, and equal to any NaN.  A softmax over a NaN or +infinity is NaN
 *   throughout.
 *   Scores, their sums and weights' ratios are held in fp64; a weight is rounded
 *   once.  Choices are compared in all their bits, whatever M.  (A softmax's
 *   scores are within 2^-48 of themselves: the order of its sum goes by M and E.)
 *
 *   logits   : fp32 (logit_bits 32) or bf16 (16), row m at logits + m * ld elements, E <= ld < 2^22
 *   bias     : fp32 [E] or NULL
 *   valid    : uint8 [M] or NULL; a token with 0 gets no expert
 *   ids      : int32 [M][top]; -1 where fewer than `top` can be picked
 *   weights  : fp32 [M][top]; 0 there
 *   offsets  : int32 [E + 1]; sorted choices of expert e are offsets[e] <= t < offsets[e + 1]
 *   rows     : int32 [M * top]; rows[t] = token of sorted choice t, tokens of an
 *              expert in their order; not written from offsets[E] on
 *   places   : int32 [M][top]; t of each choice, -1 where there is none
 *   workspace: wq_experts_route_workspace(M, E) bytes, 4-byte aligned (NULL where
 *              that is 0), no contents kept between calls; one for M tokens and E
 *              experts serves fewer of either, calls that may run concurrently need
 *              different ones
 * 1 <= E <= 1024, 1 <= top <= min(E, 32), 1 <= keep <= groups <= 64, M * top < 2^30
 * (WQ_EUNSUPPORTED above).  With M == 0 the offsets are written, all zero.
 * The outputs overlap neither each other nor the inputs.
 */
size_t wq_experts_route_workspace(int64_t M, int64_t E);
wq_status wq_experts_route(const void* logits, int logit_bits, int64_t ld, int64_t M, int64_t E, int64_t top, int score,
                           const float* bias, int64_t groups, int64_t keep, int pairs, int renormalize, float scale,
                           const void* valid, int32_t* ids, float* weights, int32_t* offsets, int32_t* rows,
                           int32_t* places, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Weighted sum of each token's rows:
 *   out[m] = bf16( sum_j weights[m][j] * Y[places[m][j]] (+ base[m]) )
 * in fp32, j in order, rounded once.  A choice whose place is outside [0, T)
 * counts as none, whatever its weight.
 *   Y       : bf16 [T][N]
 *   places  : int32 [M][top]
 *   weights : fp32 [M][top]
 *   base    : bf16 [M][N] or NULL (a shared expert's rows, a residual)
 *   out     : bf16 [M][N]; may be `base`, no other overlap
 * Any N; 0 <= top <= 1024.
 */
wq_status wq_experts_combine(const void* Y, int64_t T, int64_t N, const int32_t* places, const float* weights,
                             int64_t M, int64_t top, const void* base, void* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WQ_EXPERTS_H */
