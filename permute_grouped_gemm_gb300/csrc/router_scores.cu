// The router's choice by score + bias (see pgg_route_choose.cuh): a translation unit of its own, so
// that the forms of the two choices compile side by side.
//
// Fewer sizes than of the choice by the logits: the scores, an exponential and a quotient a logit,
// are what it costs, not the slots past the last expert (65536 tokens, 256 experts, k 8, bf16, whole
// call: sigmoid 50 us, softmax 59, by the logits 30; 13500 x 60: 12.6 and 12.0).

#include "pgg_route_choose.cuh"

namespace pgg {
namespace {

template <int DT>
cudaError_t launch_scores_d(const RouteArgs& a, cudaStream_t stream) {
  if (a.k <= 8 && a.G <= 64) return launch_route_t<DT, 8, 8, true>(a, stream);
  if (a.k <= 8 && a.G <= 256) return launch_route_t<DT, 32, 8, true>(a, stream);
  if (a.k <= 16 && a.G <= 512) return launch_route_t<DT, 32, 16, true>(a, stream);
  return launch_route_t<DT, 32, 32, true>(a, stream);
}

}  // namespace

cudaError_t launch_route_scores(int dtype, const RouteArgs& a, cudaStream_t stream) {
  if (dtype == PGG_F32) return launch_scores_d<PGG_F32>(a, stream);
  if (dtype == PGG_F16) return launch_scores_d<PGG_F16>(a, stream);
  if (dtype == PGG_BF16) return launch_scores_d<PGG_BF16>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pgg
