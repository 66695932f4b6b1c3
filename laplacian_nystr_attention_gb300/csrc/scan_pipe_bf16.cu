// scan_pipe_bf16.cu -- scan_pipe.cuh's kernels for bf16 inputs.
#include "scan_pipe.cuh"

namespace lapl {
namespace scan {
namespace pipe {
namespace {

constexpr bool kIn16 = true;
constexpr int V = kIn16 ? 2 : 1, kElem = kIn16 ? 2 : 4;

template <bool kOut16, bool kSig, int kLanes>
Pick forward() {
  constexpr int kStages = 2;
  return {scan_forward_pipe_kernel<kIn16, kOut16, kSig, kLanes, kStages, kForwardTeams, kForwardWarps>,
          kForwardTeams, kForwardWarps,
          layout_of<V, kLanes>(kForwardTeams, kForwardWarps, 2 * Tile<kLanes, V * kElem>::kWarp, kStages)};
}
template <bool kGrad16, bool kSig, int kLanes>
Pick backward() {
  constexpr int kStages = 2;
  return {scan_backward_pipe_kernel<kIn16, kGrad16, kSig, kLanes, kStages, kBackwardTeams, kBackwardWarps>,
          kBackwardTeams, kBackwardWarps,
          layout_of<V, kLanes>(kBackwardTeams, kBackwardWarps, 2 * Tile<kLanes, V * kElem>::kWarp +
                                  Tile<kLanes, V * (kGrad16 ? 2 : 4)>::kWarp, kStages)};
}
template <bool kOther16, bool kSig, bool kBackward>
Pick pick(int lanes) {
  if constexpr (kBackward)
    return lanes == 32 ? backward<kOther16, kSig, 32>()
           : lanes == 16 ? backward<kOther16, kSig, 16>() : backward<kOther16, kSig, 8>();
  else
    return lanes == 32 ? forward<kOther16, kSig, 32>()
           : lanes == 16 ? forward<kOther16, kSig, 16>() : forward<kOther16, kSig, 8>();
}

}  // namespace

Pick forward_bf16(bool out16, bool sig, int lanes) {
  return out16 ? (sig ? pick<true, true, false>(lanes) : pick<true, false, false>(lanes))
               : (sig ? pick<false, true, false>(lanes) : pick<false, false, false>(lanes));
}
Pick backward_bf16(bool grad16, bool sig, int lanes) {
  return grad16 ? (sig ? pick<true, true, true>(lanes) : pick<true, false, true>(lanes))
                : (sig ? pick<false, true, true>(lanes) : pick<false, false, true>(lanes));
}

}  // namespace pipe
}  // namespace scan
}  // namespace lapl
