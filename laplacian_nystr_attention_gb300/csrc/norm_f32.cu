// norm_f32.cu -- residual addition + root-mean-square norm with fp32 outputs (norm_kernels.cuh).
#include "norm_kernels.cuh"

namespace lapl {
namespace norm {

Kernel forward_f32(bool x16, bool r16, Cut cut, int nv) {
  return forward_for<kF32>(x16, r16, cut, nv);
}

}  // namespace norm
}  // namespace lapl
