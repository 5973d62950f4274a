/*
 * wq_int8.h -- C ABI of the 8-bit integer operators (MI355X, gfx950).
 *
 * Rows in 8-bit integers hold codes int8 in [-127, 127] and one fp32 scale a
 * row: value = code * scale.
 *   activations X[M][K]:    codes [M][K],    scales float [M]      (one a token)
 *   weights     W[E][N][K]: codes [E][N][K], scales float [E][N]   (one an output channel; a plain Linear is E = 1)
 * The quantizer, for a row of fp32 values y:
 *   s    = max(amax / 127, 2^-126), amax = max |y|, one IEEE fp32 division
 *   code = y / s to the nearest whole number, ties to even; the fp32 quotient is
 *          within one ulp of IEEE division's
 * The floor 2^-126 keeps 1 / s finite: a row of zeros has that scale and codes 0.
 * A row that holds a NaN or an infinity has the scale NaN and codes 0: no finite
 * value is made up for it, and all that is computed from it is NaN.
 *
 * Conventions are those of wq.h: device pointers owned by the caller, row-major
 * tensors, bf16 as uint16 bit patterns, stream-ordered calls that neither wait
 * nor allocate, every check on the host before anything is enqueued,
 * wq_last_error() for the reason.  Base pointers of codes and bf16 tensors must
 * be 16-byte aligned (a bias 2-byte), the other pointers aligned to their type.
 * K % 16 == 0 everywhere (WQ_ESHAPE otherwise) and K < 2^17 (WQ_EUNSUPPORTED
 * otherwise): a sum of so many products of any two int8 codes fits an int32.
 * The quantizers write nothing where there are no rows, or rows of no elements
 * (K == 0), scales neither; the products refuse K == 0 (WQ_EUNSUPPORTED).
 * A call has fewer rows, or tiles, than a launch holds (some 2^22 to 2^26;
 * WQ_EUNSUPPORTED otherwise).
 */
#ifndef WQ_INT8_H
#define WQ_INT8_H

#include "wq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Quantize bf16 weights W[E][N][K] (contiguous) to codes and one scale for each of the E N rows. */
wq_status wq_int8_quantize_weight(const void* W, int64_t E, int64_t N, int64_t K, void* codes, float* scales,
                                  void* stream);

/*
 * Quantize bf16 rows X[M][K] (row m at X + m * ldx elements; ldx >= K,
 * ldx % 8 == 0) to codes Xq[M][K] and scales Xs[M].
 */
wq_status wq_int8_quantize_act(const void* X, int64_t ldx, int64_t M, int64_t K, void* Xq, float* Xs, void* stream);

/*
 * Gated activation with a quantized result: GU holds rows of 2 K bf16 values
 * (row m at GU + m * ldg elements; ldg >= 2 K, ldg % 8 == 0), gate first;
 *   y[k] = silu(GU[m][k]) * GU[m][K + k],  silu(g) = g / (1 + exp(-g))
 * in fp32, y within 10 * 2^-24 of itself (or of 2^-126), as far as exp(-g) is a number in fp32;
 * beyond (g < -88.72) it is -0, as the fp32 formula has it.  Infinite gates spoil
 * their row: y is an infinity or a NaN.  Xq/Xs receive y quantized.
 */
wq_status wq_int8_silu_mul_quantize(const void* GU, int64_t ldg, int64_t M, int64_t K, void* Xq, float* Xs,
                                    void* stream);

/*
 * Linear:
 *   Y[m][n] = bf16( float(sum_k Xq[m][k] Wq[n][k]) * Xs[m] * Ws[n] (+ bias[n]) )
 * The sum is exact (int32); from there on fp32, each operation rounded by itself:
 * the sum is rounded to 24 bits, multiplied by Xs, then by Ws, the bias is added,
 * and the result rounded to bf16.  A row's bits do not go by the other rows or
 * their number.  bias: bf16 [N] or NULL.  Any M and N.  No workspace.
 */
wq_status wq_int8_linear(const void* Xq, const float* Xs, int64_t M, int64_t K, const void* Wq, const float* Ws,
                         const void* bias, int64_t N, void* Y, void* stream);

/*
 * The same product for E experts over rows sorted by expert:
 *   Y[t] = X[rows[t]] . W[e]^T   for offsets[e] <= t < offsets[e + 1]
 *   Xq, Xs  : M rows of codes and scales, M >= 1 where T >= 1
 *   rows    : int32 [T] on the device, each in [0, M) (a row of another value
 *             is read as zeros), or NULL: sorted row t reads X[t], and M == T
 *   offsets : int32 [E + 1] on the device, nondecreasing from offsets[0] = 0;
 *             an expert may have no rows.  Rows of Y from offsets[E] on are not
 *             written, so T may be a buffer's capacity.
 *   Wq, Ws  : weights of the E experts
 *   Y       : bf16 [T][N]
 * Nothing is read back to the host: T and E alone decide the launch.  Entries
 * of offsets are clamped to [0, T] and the tiles they make to those launched, so
 * no value of them reaches outside Y or the operands (out of order, which rows
 * are written by which expert is not defined).
 * M * K < 2^32 with rows, E <= 2^20 (WQ_EUNSUPPORTED otherwise).
 */
wq_status wq_int8_grouped_linear(const void* Xq, const float* Xs, int64_t M, int64_t K, const int32_t* rows,
                                 const int32_t* offsets, int64_t T, int64_t E, const void* Wq, const float* Ws,
                                 int64_t N, void* Y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WQ_INT8_H */
