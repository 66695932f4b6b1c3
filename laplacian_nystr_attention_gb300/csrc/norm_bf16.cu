// norm_bf16.cu -- residual addition + root-mean-square norm with bf16 outputs (norm_kernels.cuh).
#include "norm_kernels.cuh"

namespace lapl {
namespace norm {

Kernel forward_bf16(bool x16, bool r16, Cut cut, int nv) {
  return forward_for<kBf16>(x16, r16, cut, nv);
}

}  // namespace norm
}  // namespace lapl
