// C ABI of the block-scaled FP8 operators (include/wq_block.h): argument checks
// and dispatch to the launchers.  Host-side checks run before any HIP call.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "wq_block.h"
#include "wq_block_internal.hpp"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxGrid = 65535;  // workgroups along y and z
// Scale blocks of a row operator's result: at most 32 threads for each (64 for
// a row of one), and a launch holds fewer than 2^32.
constexpr int64_t kMaxBlocks = (int64_t)1 << 27;

wq_status fail(wq_status st, const char* fmt, ...) {
  char text[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  return wq::api_error(st, text);
}

wq_status launched(hipError_t e, const char* what) {
  if (e == hipErrorInvalidConfiguration) return fail(WQ_EUNSUPPORTED, "%s: more tiles than a launch holds", what);
  return e == hipSuccess ? wq::api_ok() : fail(WQ_EHIP, "%s launch: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// sizes every call has: `what` names the entry point in messages
wq_status check_sizes(const char* what, int64_t M, int64_t K) {
  if (M < 0 || K < 0) return fail(WQ_EINVAL, "%s: negative size", what);
  if (K % 16) return fail(WQ_ESHAPE, "%s: needs K %% 16 == 0 (K=%lld)", what, (long long)K);
  if (M > kMaxDim || K > kMaxDim) return fail(WQ_EUNSUPPORTED, "%s: dimension above 2^30", what);
  return WQ_OK;
}

int64_t blocks(int64_t n) { return (n + WQ_BLOCK - 1) / WQ_BLOCK; }

wq_status quant_rows(const char* what, bool gate, const void* X, int64_t ldx, int64_t M, int64_t K, void* Xq,
                     float* Xs, void* stream) {
  wq_status st = check_sizes(what, M, K);
  if (st != WQ_OK) return st;
  if (M == 0 || K == 0) return wq::api_ok();
  if (!X || !Xq || !Xs) return fail(WQ_EINVAL, "%s: null pointer", what);
  if (ldx < (gate ? 2 * K : K)) return fail(WQ_EINVAL, "%s: row stride %lld is shorter than a row", what, (long long)ldx);
  if (ldx % 8) return fail(WQ_EALIGN, "%s: row stride %lld is not a multiple of 8", what, (long long)ldx);
  if (!aligned(X, 16) || !aligned(Xq, 16)) return fail(WQ_EALIGN, "%s: input and codes must be 16-byte aligned", what);
  if (!aligned(Xs, 4)) return fail(WQ_EALIGN, "%s: scales must be 4-byte aligned", what);
  if (M * blocks(K) >= kMaxBlocks) return fail(WQ_EUNSUPPORTED, "%s: 2^27 scale blocks or more", what);
  return launched(wq::launch_block_quant_rows(gate, (const uint16_t*)X, ldx, M, K, (uint8_t*)Xq, Xs,
                                              (hipStream_t)stream),
                  what);
}

// What both products check.  `rows_y`: rows of Y.  *empty: nothing to launch.
wq_status check_gemm(const char* what, const void* Xq, const float* Xs, int64_t M, int64_t K, const void* Wq,
                     const float* Ws, int64_t N, int64_t E, const void* Y, int64_t rows_y, bool* empty) {
  *empty = false;
  wq_status st = check_sizes(what, M, K);
  if (st != WQ_OK) return st;
  if (N < 0 || E < 0 || rows_y < 0) return fail(WQ_EINVAL, "%s: negative size", what);
  if (N > kMaxDim || rows_y > kMaxDim || E > (1 << 20)) return fail(WQ_EUNSUPPORTED, "%s: dimension too large", what);
  if (rows_y == 0 || N == 0) {
    *empty = true;
    return wq::api_ok();
  }
  if (K == 0) return fail(WQ_EUNSUPPORTED, "%s: K == 0", what);
  // a tile's rows are addressed with 32-bit offsets from the tile's start
  if (K >= (int64_t)1 << 22) return fail(WQ_EUNSUPPORTED, "%s: K of 2^22 or more", what);
  if (!Xq || !Xs || !Wq || !Ws || !Y) return fail(WQ_EINVAL, "%s: null pointer", what);
  if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(Y, 16))
    return fail(WQ_EALIGN, "%s: codes and Y must be 16-byte aligned", what);
  if (!aligned(Xs, 4) || !aligned(Ws, 4)) return fail(WQ_EALIGN, "%s: scales must be 4-byte aligned", what);
  return WQ_OK;
}

}  // namespace

extern "C" {

wq_status wq_block_quantize_weight(const void* W, int64_t E, int64_t N, int64_t K, void* codes, float* scales,
                                   void* stream) {
  const char* what = "wq_block_quantize_weight";
  wq_status st = check_sizes(what, N, K);
  if (st != WQ_OK) return st;
  if (E < 0) return fail(WQ_EINVAL, "%s: negative size", what);
  if (E == 0 || N == 0 || K == 0) return wq::api_ok();
  if (!W || !codes || !scales) return fail(WQ_EINVAL, "%s: null pointer", what);
  if (!aligned(W, 16) || !aligned(codes, 16)) return fail(WQ_EALIGN, "%s: W and codes must be 16-byte aligned", what);
  if (!aligned(scales, 4)) return fail(WQ_EALIGN, "%s: scales must be 4-byte aligned", what);
  if (E > kMaxGrid || blocks(N) > kMaxGrid)
    return fail(WQ_EUNSUPPORTED, "%s: more than 65535 matrices or blocks along N", what);
  return launched(wq::launch_block_quant_weight((const uint16_t*)W, E, N, K, (uint8_t*)codes, scales,
                                                (hipStream_t)stream),
                  what);
}

wq_status wq_block_quantize_act(const void* X, int64_t ldx, int64_t M, int64_t K, void* Xq, float* Xs, void* stream) {
  return quant_rows("wq_block_quantize_act", false, X, ldx, M, K, Xq, Xs, stream);
}

wq_status wq_block_silu_mul_quantize(const void* GU, int64_t ldg, int64_t M, int64_t K, void* Xq, float* Xs,
                                     void* stream) {
  return quant_rows("wq_block_silu_mul_quantize", true, GU, ldg, M, K, Xq, Xs, stream);
}

wq_status wq_block_add_rmsnorm_quantize(const void* X, int64_t ldx, const void* residual, const void* gain, float eps,
                                        int64_t M, int64_t K, void* Xq, float* Xs, void* residual_out, void* y_out,
                                        void* stream) {
  const char* what = "wq_block_add_rmsnorm_quantize";
  wq_status st = check_sizes(what, M, K);
  if (st != WQ_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(WQ_EINVAL, "%s: eps must be finite and not negative", what);
  if (K > wq::kNormMaxK) return fail(WQ_EUNSUPPORTED, "%s: K above %lld", what, (long long)wq::kNormMaxK);
  if (M == 0 || K == 0) return wq::api_ok();
  if (M * (blocks(K) > 1 ? blocks(K) : 2) >= kMaxBlocks) return fail(WQ_EUNSUPPORTED, "%s: 2^27 scale blocks or more", what);
  if (!X || !gain || !Xq || !Xs) return fail(WQ_EINVAL, "%s: null pointer", what);
  if (ldx < K) return fail(WQ_EINVAL, "%s: row stride %lld is shorter than a row", what, (long long)ldx);
  if (ldx % 8) return fail(WQ_EALIGN, "%s: row stride %lld is not a multiple of 8", what, (long long)ldx);
  if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(gain, 16) || !aligned(Xq, 16) ||
      !aligned(residual_out, 16) || !aligned(y_out, 16))
    return fail(WQ_EALIGN, "%s: bf16 tensors and codes must be 16-byte aligned", what);
  if (!aligned(Xs, 4)) return fail(WQ_EALIGN, "%s: scales must be 4-byte aligned", what);
  if (residual_out && residual_out == X && ldx != K)
    return fail(WQ_EINVAL, "%s: residual_out may be X only where X is contiguous", what);
  wq::BlockNormArgs a{};
  a.X = (const uint16_t*)X;
  a.residual = (const uint16_t*)residual;
  a.gain = (const uint16_t*)gain;
  a.Xq = (uint8_t*)Xq;
  a.Xs = Xs;
  a.residual_out = (uint16_t*)residual_out;
  a.y_out = (uint16_t*)y_out;
  a.ldx = ldx;
  a.M = (int)M;
  a.K = (int)K;
  a.eps = eps;
  return launched(wq::launch_block_norm(a, (hipStream_t)stream), what);
}

wq_status wq_block_linear(const void* Xq, const float* Xs, int64_t M, int64_t K, const void* Wq, const float* Ws,
                          const void* bias, int64_t N, void* Y, void* stream) {
  const char* what = "wq_block_linear";
  bool empty;
  wq_status st = check_gemm(what, Xq, Xs, M, K, Wq, Ws, N, 1, Y, M, &empty);
  if (st != WQ_OK || empty) return st;
  if (!aligned(bias, 2)) return fail(WQ_EALIGN, "%s: bias must be 2-byte aligned", what);
  wq::BlockGemmArgs a{};
  a.Xq = (const uint8_t*)Xq;
  a.Xs = Xs;
  a.Wq = (const uint8_t*)Wq;
  a.Ws = Ws;
  a.bias = (const uint16_t*)bias;
  a.Y = (uint16_t*)Y;
  a.M = a.T = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.E = 1;
  return launched(wq::launch_block_gemm(a, (hipStream_t)stream), what);
}

wq_status wq_block_grouped_linear(const void* Xq, const float* Xs, int64_t M, int64_t K, const int32_t* rows,
                                  const int32_t* offsets, int64_t T, int64_t E, const void* Wq, const float* Ws,
                                  int64_t N, void* Y, void* stream) {
  const char* what = "wq_block_grouped_linear";
  bool empty;
  wq_status st = check_gemm(what, Xq, Xs, M, K, Wq, Ws, N, E, Y, T, &empty);
  if (st != WQ_OK || empty) return st;
  if (E == 0) return wq::api_ok();
  if (!offsets) return fail(WQ_EINVAL, "%s: null offsets", what);
  if (!aligned(offsets, 4) || !aligned(rows, 4))
    return fail(WQ_EALIGN, "%s: offsets and rows must be 4-byte aligned", what);
  if (M == 0) return fail(WQ_EINVAL, "%s: %lld rows from none", what, (long long)T);
  if (!rows && M != T) return fail(WQ_EINVAL, "%s: without rows M must be T (M=%lld T=%lld)", what, (long long)M, (long long)T);
  if (rows && M * K >= (int64_t)1 << 32) return fail(WQ_EUNSUPPORTED, "%s: 2^32 codes or more behind rows", what);
  wq::BlockGemmArgs a{};
  a.Xq = (const uint8_t*)Xq;
  a.Xs = Xs;
  a.Wq = (const uint8_t*)Wq;
  a.Ws = Ws;
  a.rows = rows;
  a.offsets = offsets;
  a.Y = (uint16_t*)Y;
  a.M = (int)M;
  a.T = (int)T;
  a.N = (int)N;
  a.K = (int)K;
  a.E = (int)E;
  return launched(wq::launch_block_gemm(a, (hipStream_t)stream), what);
}

}  // extern "C"
