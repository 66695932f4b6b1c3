// scan_few.cuh -- what scan.cu launches of scan_few.cu.
#pragma once

#include "scan.cuh"

namespace lapl {
namespace scan {
namespace few {

constexpr int kTokens = 4;           // read at once
constexpr int kBackwardTokens = 8;   // the most the backward takes
constexpr int kThreads = 256;        // of a CTA: lanes across the channels, the rest sequences

using Kernel = void (*)(Args);
// v: channels of a thread, 4 or 1.
Kernel forward(bool in16, bool out16, bool sig, int v, int tokens);
// v: 4 up to kTokens, then 2; or 1.
Kernel backward(bool in16, bool grad16, bool sig, int v, int tokens);

}  // namespace few
}  // namespace scan
}  // namespace lapl
