// The packed-weight operators' host side, and the element-wise half of the
// gated block's backward pass.
#include "w4_internal.h"

namespace awq {

// dG = dH U act'(G), dU = dH act(G), each rounded once.
template <typename T, int ACT>
__global__ void __launch_bounds__(256)
k_gated_grad(const T* __restrict__ dH, const T* __restrict__ pre, int64_t n, int F,
             T* __restrict__ dpre) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += stride) {
    const int64_t t = e / F;
    const int64_t at = t * 2 * F + (e - t * F);
    const float g = to_f32(pre[at]), u = to_f32(pre[at + F]), d = to_f32(dH[e]);
    float slope;
    const float a = act_value<ACT>(g, &slope);
    dpre[at] = from_f32<T>(d * u * slope);
    dpre[at + F] = from_f32<T>(d * a);
  }
}

template <typename T>
static hipError_t launch_gated_grad(const W4Args& a, hipStream_t stream) {
  const int64_t n = a.N * (a.O / 2), want = (n + 255) / 256;
  const dim3 grid((unsigned)(want < 8192 ? want : 8192));
  if (a.act == kActSilu)
    hipLaunchKernelGGL((k_gated_grad<T, kActSilu>), grid, dim3(256), 0, stream, (const T*)a.in0,
                       (const T*)a.in1, n, (int)(a.O / 2), (T*)a.out1);
  else
    hipLaunchKernelGGL((k_gated_grad<T, kActGelu>), grid, dim3(256), 0, stream, (const T*)a.in0,
                       (const T*)a.in1, n, (int)(a.O / 2), (T*)a.out1);
  return hipGetLastError();
}

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
      return launch_w4_input_grad(a, a.in0, stream);
    case kOpGatedBackward: {
      const hipError_t e = a.type == kF16 ? launch_gated_grad<_Float16>(a, stream)
                                          : launch_gated_grad<__bf16>(a, stream);
      return e != hipSuccess ? e : launch_w4_input_grad(a, a.out1, stream);
    }
    case kOpParamGrad:
      return launch_w4_param_grad(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace awq
