// Internal launch interface of the 8-bit integer operators (wq_int8_api.hip to
// wq_int8_quant.hip and wq_int8_gemm.hip).  Launchers assume their arguments
// were validated by the ABI layer.
#pragma once

#include "wq_block_internal.hpp"

namespace wq {

constexpr int64_t kInt8MaxK = (int64_t)1 << 17;  // from here on a sum of products of codes may leave an int32

// gate = false: Xq/Xs = quantized rows of X[M][K]; true: of silu(X[:, :K]) * X[:, K:]
hipError_t launch_int8_quant_rows(bool gate, const uint16_t* X, int64_t ldx, int64_t M, int64_t K, uint8_t* Xq,
                                  float* Xs, hipStream_t s);

struct Int8GemmArgs {
  const uint8_t* Xq;       // codes [M][K]
  const float* Xs;         // scales [M]
  const uint8_t* Wq;       // codes [E][N][K]
  const float* Ws;         // scales [E][N]
  const uint16_t* bias;    // bf16 [N] or null
  const int32_t* rows;     // grouped: source row of each sorted row, or null
  const int32_t* offsets;  // grouped: [E + 1], null for a plain Linear
  uint16_t* Y;             // bf16 [M or T][N]
  int M, N, K, T, E;       // T: rows of Y (M for a plain Linear)
};
hipError_t launch_int8_gemm(const Int8GemmArgs& a, hipStream_t s);

// Kernel forms of the products: dot products for single rows (by a wave's columns), streams of the weights for few
// (by columns x rows of a workgroup; deep: two blocks of a wave under way), LDS tiles for more.
enum Int8Form {
  kI8Dot2, kI8Dot4, kI8Dot8, kI8Stream16, kI8Stream16Deep, kI8Stream32, kI8Stream16x32,
  kI8Tile256, kI8Tile256x128, kI8Tile128, kI8Tile128x64, kI8Tile64, kI8Tile32x64, kI8Forms
};
// The form of T rows of Y over E experts (a plain Linear: grouped false), chosen on the host (wq_int8_plan.cpp).
Int8Form int8_form(bool grouped, int T, int E, int N, int K);

}  // namespace wq

// The form's name, for tests (E = 0: a plain Linear).
extern "C" const char* wq_int8_form(int64_t T, int64_t E, int64_t N, int64_t K);
