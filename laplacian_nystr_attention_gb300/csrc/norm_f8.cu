// norm_f8.cu -- residual addition + root-mean-square norm with e4m3 outputs (norm_kernels.cuh).
#include "norm_kernels.cuh"

namespace lapl {
namespace norm {

Kernel forward_f8(bool x16, bool r16, Cut cut, int nv) {
  return forward_for<kF8>(x16, r16, cut, nv);
}

}  // namespace norm
}  // namespace lapl
