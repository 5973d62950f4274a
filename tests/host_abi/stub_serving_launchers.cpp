// Host-only stand-ins for the launchers of the 8-bit integer operators and the
// experts' routing (see stub_launchers.cpp): every launcher fails as on a
// machine without a GPU.
#include <hip/hip_runtime_api.h>

#include "wq_experts_internal.hpp"
#include "wq_int8_internal.hpp"

namespace wq {
hipError_t launch_int8_quant_rows(bool, const uint16_t*, int64_t, int64_t, int64_t, uint8_t*, float*, hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_int8_gemm(const Int8GemmArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_route(const RouteArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_combine(const CombineArgs&, hipStream_t) { return hipErrorNoDevice; }
}  // namespace wq
