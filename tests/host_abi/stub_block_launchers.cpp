// Host-only stand-ins for the block-scaled operators' launchers (see
// stub_launchers.cpp): every launcher fails as on a machine without a GPU.
#include <hip/hip_runtime_api.h>

#include "wq_block_internal.hpp"

namespace wq {
hipError_t launch_block_norm(const BlockNormArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_block_quant_rows(bool, const uint16_t*, int64_t, int64_t, int64_t, uint8_t*, float*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_block_quant_weight(const uint16_t*, int64_t, int64_t, int64_t, uint8_t*, float*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_block_gemm(const BlockGemmArgs&, hipStream_t) { return hipErrorNoDevice; }
}  // namespace wq
