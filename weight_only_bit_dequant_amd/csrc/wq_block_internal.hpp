// Internal launch interface of the block-scaled FP8 operators
// (wq_block_api.hip to wq_block_quant.hip and wq_block_gemm.hip).  Launchers
// assume their arguments were validated by the ABI layer.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "wq.h"

namespace wq {

constexpr int kBlk = 128;  // K elements (and weight rows) per scale

// Status of a call and the text of wq_last_error() (defined in wq_api.hip,
// which holds the thread's message).
wq_status api_error(wq_status st, const char* message);
wq_status api_ok();

// Enqueue a kernel.  (hipLaunchKernel itself: the <<<>>> form first stores the
// configuration and takes it back, 0.25 of its 3.65 us on the host.)
template <typename... P, typename... A>
hipError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, hipStream_t s, const A&... a) {
  static_assert(sizeof...(P) == sizeof...(A), "one argument for each parameter");
  return [&](P... p) {
    void* args[] = {(void*)&p...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), args, smem, s);
  }(a...);
}

constexpr int64_t kNormMaxK = 32768;  // 16 waves x 64 lanes x 4 chunks of 8

struct BlockNormArgs {
  const uint16_t* X;         // bf16 rows, ldx elements apart
  const uint16_t* residual;  // bf16 [M][K] or null
  const uint16_t* gain;      // bf16 [K]
  uint8_t* Xq;               // codes [M][K]
  float* Xs;                 // scales [M][KB]
  uint16_t* residual_out;    // bf16 [M][K] or null
  uint16_t* y_out;           // bf16 [M][K] or null
  int64_t ldx;
  int M, K;
  float eps;
};
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t s);

// gate = false: Xq/Xs = quantized rows of X[M][K]; true: of silu(X[:, :K]) * X[:, K:]
hipError_t launch_block_quant_rows(bool gate, const uint16_t* X, int64_t ldx, int64_t M, int64_t K, uint8_t* Xq,
                                   float* Xs, hipStream_t s);
hipError_t launch_block_quant_weight(const uint16_t* W, int64_t E, int64_t N, int64_t K, uint8_t* codes,
                                     float* scales, hipStream_t s);

struct BlockGemmArgs {
  const uint8_t* Xq;       // codes [M][K]
  const float* Xs;         // scales [M][KB]
  const uint8_t* Wq;       // codes [E][N][K]
  const float* Ws;         // scales [E][NB][KB]
  const uint16_t* bias;    // bf16 [N] or null
  const int32_t* rows;     // grouped: source row of each sorted row, or null
  const int32_t* offsets;  // grouped: [E + 1], null for a plain Linear
  uint16_t* Y;             // bf16 [M or T][N]
  int M, N, K, T, E;       // T: rows of Y (M for a plain Linear)
};
hipError_t launch_block_gemm(const BlockGemmArgs& a, hipStream_t s);

// A round of the chip in tiles, and the largest rest of one that is split into smaller ones (wq_block_tiles.hpp).
constexpr int kRound = 256, kMostRest = kRound / 2;

// Kernel forms of the products, by columns x rows of a workgroup: streams of the weights for few rows (deep: two
// blocks of a wave under way; eight: waves, where the others of 32 columns have four), LDS tiles for more (one:
// 64 x 64 without K split).
enum BlockForm {
  kStream16, kStream16Deep, kStream32Eight, kStream32, kStream32x32, kStream64,
  kTile256, kTile256x128, kTile128, kTile128x64, kTile64, kTile64One, kBlockForms
};
// The form of T rows of Y over E experts (a plain Linear: grouped false), chosen on the host (wq_block_plan.cpp).
BlockForm block_form(bool grouped, int T, int E, int N, int K);

}  // namespace wq

// The form's name, for tests (E = 0: a plain Linear).
extern "C" const char* wq_block_form(int64_t T, int64_t E, int64_t N, int64_t K);
