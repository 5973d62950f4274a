// C ABI of the 8-bit integer operators (include/wq_int8.h): argument checks and
// dispatch to the launchers.  Host-side checks run before any HIP call.
#include <hip/hip_runtime_api.h>

#include "wq_api_checks.hpp"
#include "wq_int8.h"
#include "wq_int8_internal.hpp"

namespace {

using namespace wq::api;

// sizes every call has: `what` names the entry point in messages
wq_status check_sizes(const char* what, int64_t M, int64_t K) {
  if (M < 0 || K < 0) return fail(WQ_EINVAL, "%s: negative size", what);
  if (K % 16) return fail(WQ_ESHAPE, "%s: needs K %% 16 == 0 (K=%lld)", what, (long long)K);
  if (M > kMaxDim || K > kMaxDim) return fail(WQ_EUNSUPPORTED, "%s: dimension above 2^30", what);
  if (K >= wq::kInt8MaxK) return fail(WQ_EUNSUPPORTED, "%s: K of 2^17 or more", what);
  return WQ_OK;
}

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
  return launched(wq::launch_int8_quant_rows(gate, (const uint16_t*)X, ldx, M, K, (uint8_t*)Xq, Xs, (hipStream_t)stream),
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
  if (!Xq || !Xs || !Wq || !Ws || !Y) return fail(WQ_EINVAL, "%s: null pointer", what);
  if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(Y, 16))
    return fail(WQ_EALIGN, "%s: codes and Y must be 16-byte aligned", what);
  if (!aligned(Xs, 4) || !aligned(Ws, 4)) return fail(WQ_EALIGN, "%s: scales must be 4-byte aligned", what);
  return WQ_OK;
}

}  // namespace

extern "C" {

wq_status wq_int8_quantize_weight(const void* W, int64_t E, int64_t N, int64_t K, void* codes, float* scales,
                                  void* stream) {
  const char* what = "wq_int8_quantize_weight";
  wq_status st = check_sizes(what, N, K);
  if (st != WQ_OK) return st;
  if (E < 0) return fail(WQ_EINVAL, "%s: negative size", what);
  if (E > kMaxDim || E * N > kMaxDim) return fail(WQ_EUNSUPPORTED, "%s: more than 2^30 rows", what);
  return quant_rows(what, false, W, K, E * N, K, codes, scales, stream);
}

wq_status wq_int8_quantize_act(const void* X, int64_t ldx, int64_t M, int64_t K, void* Xq, float* Xs, void* stream) {
  return quant_rows("wq_int8_quantize_act", false, X, ldx, M, K, Xq, Xs, stream);
}

wq_status wq_int8_silu_mul_quantize(const void* GU, int64_t ldg, int64_t M, int64_t K, void* Xq, float* Xs,
                                    void* stream) {
  return quant_rows("wq_int8_silu_mul_quantize", true, GU, ldg, M, K, Xq, Xs, stream);
}

wq_status wq_int8_linear(const void* Xq, const float* Xs, int64_t M, int64_t K, const void* Wq, const float* Ws,
                          const void* bias, int64_t N, void* Y, void* stream) {
  const char* what = "wq_int8_linear";
  bool empty;
  wq_status st = check_gemm(what, Xq, Xs, M, K, Wq, Ws, N, 1, Y, M, &empty);
  if (st != WQ_OK || empty) return st;
  if (!aligned(bias, 2)) return fail(WQ_EALIGN, "%s: bias must be 2-byte aligned", what);
  wq::Int8GemmArgs a{};
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
  return launched(wq::launch_int8_gemm(a, (hipStream_t)stream), what);
}

wq_status wq_int8_grouped_linear(const void* Xq, const float* Xs, int64_t M, int64_t K, const int32_t* rows,
                                  const int32_t* offsets, int64_t T, int64_t E, const void* Wq, const float* Ws,
                                  int64_t N, void* Y, void* stream) {
  const char* what = "wq_int8_grouped_linear";
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
  wq::Int8GemmArgs a{};
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
  return launched(wq::launch_int8_gemm(a, (hipStream_t)stream), what);
}

}  // extern "C"
