// Products with packed 4-bit weights beyond awq_w4a16_matmul's form: Y = X W^T
// and the gated feed-forward product H = act(X Wg^T) * (X Wu^T), with
// W[o, k] = (q[o, k] - z[o, g]) step[o, g], g = k / group, and their gradients.
// Source: dev.to "AWQ: How Activation-Aware Quantization Saves 4-bit LLMs",
// "What do you actually deploy" (W4A16, group size).
//
// One tile kernel serves every product: a block forms 64 x 128 sums in fp32
// from operands widened to fp32 in LDS, 16 steps of the reduction at a time,
// lays the sums out in LDS and applies the operator's epilogue.
#include "awq_internal.h"
#include "w4_device.h"
#include "w4_internal.h"

namespace awq {

enum W4Mode { kW4Linear, kW4Gated, kW4InputGrad, kW4ParamGrad };

struct W4Layer {
  const uint32_t* q;
  const _Float16* step;
  const _Float16* zero;
  int K, O, group;
};

__device__ __forceinline__ float code_at(const W4Layer& w, int o, int k) {
  return (float)((w.q[(size_t)o * (w.K >> 3) + (k >> 3)] >> (4 * (k & 7))) & 15u);
}
__device__ __forceinline__ float weight_at(const W4Layer& w, int o, int k) {
  const size_t g = (size_t)o * (w.K / w.group) + k / w.group;
  return (float)(_Float16)(code_at(w, o, k) - (float)w.zero[g]) * (float)w.step[g];
}

constexpr int kTI = 64, kTJ = 128, kTK = 16;

template <typename T, int MODE, int ACT, typename TY>
__global__ void __launch_bounds__(256)
k_w4_tile(const T* __restrict__ A, const T* __restrict__ B, W4Layer w, int N, TY* __restrict__ Y,
          T* __restrict__ pre, float* __restrict__ dstep, float* __restrict__ dzero) {
  __shared__ float sa[kTK][kTI + 1], sb[kTK][kTJ + 1];
  __shared__ float sd[kTI][kTJ + 1];
  const int tid = threadIdx.x, ti = tid / 16, tj = tid % 16;
  const int F = w.O / 2;
  const int i0 = blockIdx.y * kTI, j0 = blockIdx.x * (MODE == kW4Gated ? kTJ / 2 : kTJ);
  const int ni = MODE == kW4ParamGrad ? w.O : N;
  const int nr = MODE == kW4InputGrad ? w.O : MODE == kW4ParamGrad ? N : w.K;
  float acc[4][8] = {};
  for (int r0 = 0; r0 < nr; r0 += kTK) {
    for (int e = tid; e < kTI * kTK; e += 256) {
      const int i = e / kTK, r = e % kTK;
      float v = 0.0f;
      if (i0 + i < ni && r0 + r < nr) {
        if (MODE == kW4ParamGrad)
          v = to_f32(A[(size_t)(r0 + r) * w.O + i0 + i]);
        else
          v = to_f32(A[(size_t)(i0 + i) * nr + r0 + r]);
      }
      sa[r][i] = v;
    }
    for (int e = tid; e < kTJ * kTK; e += 256) {
      const int j = e % kTJ, r = e / kTJ;
      float v = 0.0f;
      if (r0 + r < nr) {
        if (MODE == kW4ParamGrad)
          v = to_f32(B[(size_t)(r0 + r) * w.K + j0 + j]);
        else if (MODE == kW4InputGrad)
          v = weight_at(w, r0 + r, j0 + j);
        else if (MODE == kW4Gated) {
          const int f = j0 + j % (kTJ / 2);
          if (f < F) v = weight_at(w, f + (j < kTJ / 2 ? 0 : F), r0 + r);
        } else if (j0 + j < w.O)
          v = weight_at(w, j0 + j, r0 + r);
      }
      sb[r][j] = v;
    }
    __syncthreads();
    for (int r = 0; r < kTK; ++r)
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 8; ++b) acc[a][b] = fmaf(sa[r][ti + 16 * a], sb[r][tj + 16 * b], acc[a][b]);
    __syncthreads();
  }
  for (int a = 0; a < 4; ++a)
    for (int b = 0; b < 8; ++b) sd[ti + 16 * a][tj + 16 * b] = acc[a][b];
  __syncthreads();
  if (MODE == kW4ParamGrad) {
    const int per = kTJ / w.group, ng = w.K / w.group;
    for (int e = tid; e < kTI * per; e += 256) {
      const int i = e / per, gl = e % per, o = i0 + i;
      if (o >= w.O) continue;
      const size_t at = (size_t)o * ng + j0 / w.group + gl;
      const float z = (float)w.zero[at];
      float ds = 0.0f, dz = 0.0f;
      for (int j = gl * w.group; j < (gl + 1) * w.group; ++j) {
        ds = fmaf(sd[i][j], (float)(_Float16)(code_at(w, o, j0 + j) - z), ds);
        dz += sd[i][j];
      }
      dstep[at] = ds;
      dzero[at] = -(float)w.step[at] * dz;
    }
    return;
  }
  const int cols = MODE == kW4Gated ? kTJ / 2 : kTJ;
  const int nj = MODE == kW4Gated ? F : MODE == kW4InputGrad ? w.K : w.O;
  for (int e = tid; e < kTI * cols; e += 256) {
    const int i = e / cols, j = e % cols;
    if (i0 + i >= N || j0 + j >= nj) continue;
    float v = sd[i][j];
    if (MODE == kW4Gated) {
      const float u = sd[i][j + kTJ / 2];
      if (pre) {
        pre[(size_t)(i0 + i) * w.O + j0 + j] = from_f32<T>(v);
        pre[(size_t)(i0 + i) * w.O + F + j0 + j] = from_f32<T>(u);
      }
      v = act_value<ACT>(v, nullptr) * u;
    }
    Y[(size_t)(i0 + i) * nj + j0 + j] = from_f32<TY>(v);
  }
}

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

template <typename T, int MODE, int ACT, typename TY>
static void launch_tile(const void* A, const void* B, const W4Layer& w, int64_t N, int64_t ni,
                        int64_t nj, void* Y, void* pre, float* ds, float* dz, hipStream_t stream) {
  const int tj = MODE == kW4Gated ? kTJ / 2 : kTJ;
  const dim3 grid((unsigned)((nj + tj - 1) / tj), (unsigned)((ni + kTI - 1) / kTI));
  hipLaunchKernelGGL((k_w4_tile<T, MODE, ACT, TY>), grid, dim3(256), 0, stream, (const T*)A,
                     (const T*)B, w, (int)N, (TY*)Y, (T*)pre, ds, dz);
}

static W4Layer layer_of(const W4Args& a) {
  return W4Layer{(const uint32_t*)a.qweight, (const _Float16*)a.step16, (const _Float16*)a.zero16,
                 (int)a.K, (int)a.O, a.group};
}

size_t w4_workspace(W4Op op, const W4Args& a) {
  if (op == kOpLinear || op == kOpGated) return w4_skinny_fits(a) ? 0 : w4_gemm_workspace(a);
  if (op == kOpInputGrad || op == kOpGatedBackward) return w4_input_grad_workspace(a);
  return 0;
}

template <typename T>
static hipError_t w4_launch(W4Op op, const W4Args& a, hipStream_t stream) {
  const W4Layer w = layer_of(a);
  const int64_t F = a.O / 2;
  switch (op) {
    case kOpLinear:
      if (a.y_type == kF32)
        launch_tile<T, kW4Linear, 0, float>(a.in0, nullptr, w, a.N, a.N, a.O, a.out0, nullptr,
                                            nullptr, nullptr, stream);
      else
        launch_tile<T, kW4Linear, 0, T>(a.in0, nullptr, w, a.N, a.N, a.O, a.out0, nullptr, nullptr,
                                        nullptr, stream);
      break;
    case kOpGated:
      if (a.act == kActSilu)
        launch_tile<T, kW4Gated, kActSilu, T>(a.in0, nullptr, w, a.N, a.N, F, a.out0, a.out1,
                                              nullptr, nullptr, stream);
      else
        launch_tile<T, kW4Gated, kActGelu, T>(a.in0, nullptr, w, a.N, a.N, F, a.out0, a.out1,
                                              nullptr, nullptr, stream);
      break;
    case kOpInputGrad:
      return launch_w4_input_grad(a, a.in0, stream);
    case kOpGatedBackward: {
      const int64_t n = a.N * F;
      const int64_t want = (n + 255) / 256;
      const dim3 grid((unsigned)(want < 8192 ? want : 8192));
      if (a.act == kActSilu)
        hipLaunchKernelGGL((k_gated_grad<T, kActSilu>), grid, dim3(256), 0, stream,
                           (const T*)a.in0, (const T*)a.in1, n, (int)F, (T*)a.out1);
      else
        hipLaunchKernelGGL((k_gated_grad<T, kActGelu>), grid, dim3(256), 0, stream,
                           (const T*)a.in0, (const T*)a.in1, n, (int)F, (T*)a.out1);
      return launch_w4_input_grad(a, a.out1, stream);
    }
    case kOpParamGrad:
      launch_tile<T, kW4ParamGrad, 0, T>(a.in0, a.in1, w, a.N, a.O, a.K, nullptr, nullptr,
                                         (float*)a.out0, (float*)a.out1, stream);
      break;
  }
  return hipGetLastError();
}

hipError_t launch_w4(W4Op op, const W4Args& a, hipStream_t stream) {
  if ((op == kOpLinear || op == kOpGated) && w4_skinny_fits(a))
    return launch_w4_skinny(op, a, stream);
  if (op == kOpLinear || op == kOpGated) return launch_w4_gemm(op, a, stream);
  return a.type == kF16 ? w4_launch<_Float16>(op, a, stream) : w4_launch<__bf16>(op, a, stream);
}

}  // namespace awq
