// Which kernels a packed-weight operator takes, and its workspace.
#include "w4_internal.h"

namespace awq {

size_t w4_workspace(W4Op op, const W4Args& a) {
  switch (op) {
    case kOpLinear:
    case kOpGated:
      return w4_skinny_fits(a) ? 0 : w4_gemm_workspace(op, a);
    case kOpInputGrad:
    case kOpGatedBackward:
      return w4_input_grad_workspace(a);
    case kOpParamGrad:
      return w4_param_grad_workspace(a);
  }
  return 0;
}

hipError_t launch_w4(W4Op op, const W4Args& a, hipStream_t stream) {
  switch (op) {
    case kOpLinear:
    case kOpGated:
      return w4_skinny_fits(a) ? launch_w4_skinny(op, a, stream) : launch_w4_gemm(op, a, stream);
    case kOpInputGrad:
    case kOpGatedBackward:
      return launch_w4_input_grad(op, a, stream);
    case kOpParamGrad:
      return launch_w4_param_grad(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace awq
