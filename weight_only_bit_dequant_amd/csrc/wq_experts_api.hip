// C ABI of the experts' routing (include/wq_experts.h): argument checks and
// dispatch to the launchers.  Host-side checks run before any HIP call.
#include <hip/hip_runtime_api.h>

#include "wq_api_checks.hpp"
#include "wq_experts.h"
#include "wq_experts_internal.hpp"

using namespace wq::api;

extern "C" {

size_t wq_experts_route_workspace(int64_t M, int64_t E) {
  if (M <= wq::kFewSpan || E <= 0 || M > kMaxDim || E > WQ_MAX_EXPERTS) return 0;
  // no less than fewer tokens need, which have more stretches up to a point
  const int few = wq::stretches(M < wq::kWaves * wq::kMaxStretches ? M : wq::kWaves * wq::kMaxStretches).count, count = wq::stretches(M).count;
  return (size_t)(count > few ? count : few) * (size_t)wq::counts_pitch((int)E) * sizeof(uint16_t);
}

wq_status wq_experts_route(const void* logits, int logit_bits, int64_t ld, int64_t M, int64_t E, int64_t top, int score,
                           const float* bias, int64_t groups, int64_t keep, int pairs, int renormalize, float scale,
                           const void* valid, int32_t* ids, float* weights, int32_t* offsets, int32_t* rows,
                           int32_t* places, void* workspace, size_t workspace_bytes, void* stream) {
  const char* what = "wq_experts_route";
  if (M < 0 || E < 1 || top < 1 || groups < 1 || keep < 1)
    return fail(WQ_EINVAL, "%s: M must not be negative, E, top, groups and keep at least 1", what);
  if (logit_bits != 16 && logit_bits != 32) return fail(WQ_EINVAL, "%s: logits of 16 or 32 bits (got %d)", what, logit_bits);
  if (score != WQ_SCORE_SOFTMAX && score != WQ_SCORE_SIGMOID) return fail(WQ_EINVAL, "%s: unknown score %d", what, score);
  if (E > WQ_MAX_EXPERTS || top > WQ_MAX_TOP || groups > WQ_MAX_EXPERT_GROUPS)
    return fail(WQ_EUNSUPPORTED, "%s: more than %d experts, %d of a token or %d groups", what, WQ_MAX_EXPERTS, WQ_MAX_TOP,
                WQ_MAX_EXPERT_GROUPS);
  if (top > E) return fail(WQ_EINVAL, "%s: %lld of %lld experts", what, (long long)top, (long long)E);
  if (E % groups) return fail(WQ_ESHAPE, "%s: %lld experts in %lld groups", what, (long long)E, (long long)groups);
  if (keep > groups) return fail(WQ_EINVAL, "%s: %lld of %lld groups", what, (long long)keep, (long long)groups);
  if (M >= kMaxDim / top) return fail(WQ_EUNSUPPORTED, "%s: 2^30 choices or more", what);
  if (!offsets) return fail(WQ_EINVAL, "%s: null pointer", what);
  if (!aligned(offsets, 4)) return fail(WQ_EALIGN, "%s: pointers must be aligned to their type", what);
  if (M > 0) {
    if (!logits || !ids || !weights || !rows || !places) return fail(WQ_EINVAL, "%s: null pointer", what);
    if (ld >= 1 << 22) return fail(WQ_EUNSUPPORTED, "%s: row stride of 2^22 or more", what);
    if (ld < E) return fail(WQ_EINVAL, "%s: row stride %lld is shorter than a row", what, (long long)ld);
    if (!aligned(logits, logit_bits / 8) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(rows, 4) || !aligned(places, 4) || !aligned(workspace, 4))
      return fail(WQ_EALIGN, "%s: pointers must be aligned to their type", what);
    const size_t need = wq_experts_route_workspace(M, E);
    if (need && (!workspace || workspace_bytes < need))
      return fail(WQ_EWORKSPACE, "%s: needs %zu bytes of workspace (got %zu)", what, need, workspace ? workspace_bytes : 0);
  }
  wq::RouteArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.bias = bias;
  a.valid = (const uint8_t*)valid;
  a.ids = ids;
  a.weights = weights;
  a.offsets = offsets;
  a.rows = rows;
  a.places = places;
  a.counts = (uint16_t*)workspace;
  a.M = (int)M;
  a.E = (int)E;
  a.top = (int)top;
  a.groups = (int)groups;
  a.keep = (int)keep;
  a.scale = scale;
  a.half = logit_bits == 16;
  a.sigmoid = score == WQ_SCORE_SIGMOID;
  a.pairs = pairs && groups > 1;
  a.renormalize = renormalize != 0;
  return launched(wq::launch_route(a, (hipStream_t)stream), what);
}

wq_status wq_experts_combine(const void* Y, int64_t T, int64_t N, const int32_t* places, const float* weights,
                             int64_t M, int64_t top, const void* base, void* out, void* stream) {
  const char* what = "wq_experts_combine";
  if (T < 0 || N < 0 || M < 0 || top < 0) return fail(WQ_EINVAL, "%s: negative size", what);
  if (T > kMaxDim || N > kMaxDim || M > kMaxDim || top > 1024) return fail(WQ_EUNSUPPORTED, "%s: dimension too large", what);
  if (M == 0 || N == 0) return wq::api_ok();
  if (!out || (T > 0 && !Y) || (top > 0 && (!places || !weights))) return fail(WQ_EINVAL, "%s: null pointer", what);
  const uintptr_t to = N % 8 ? 2 : 16;
  if (!aligned(Y, to) || !aligned(base, to) || !aligned(out, to))
    return fail(WQ_EALIGN, "%s: bf16 tensors must be %d-byte aligned", what, (int)to);
  if (!aligned(places, 4) || !aligned(weights, 4)) return fail(WQ_EALIGN, "%s: places and weights must be 4-byte aligned", what);
  wq::CombineArgs a{};
  a.Y = (const uint16_t*)Y;
  a.places = places;
  a.weights = weights;
  a.base = (const uint16_t*)base;
  a.out = (uint16_t*)out;
  a.N = N;
  a.T = (int)T;
  a.M = (int)M;
  a.top = (int)top;
  return launched(wq::launch_combine(a, (hipStream_t)stream), what);
}

}  // extern "C"
