// Y = X W^T and H = act(X Wg^T) * (X Wu^T) on packed weights for up to 64
// tokens: the weights stream from HBM once and bound the call.
//
// A block owns RT tiles of 16 packed rows (gated: RT/2 of the gate and the
// same features' RT/2 of the up projection) and all tokens; its W wavefronts
// take the blocks of 128 columns in turn (wavefront w blocks w, w + W, ..), so
// that neighbours read the two halves of a line at the same time, and add
// their sums through LDS in a fixed order.
//   * Lane l holds row l % 16 of each tile; a 16-byte load brings 32 codes of
//     its row, and four lane swaps put them so that MFMA j takes columns
//     32 j .. 32 j + 31.  That keeps every MFMA inside one group for groups
//     of 32, 64 and 128, so a group's sum of exact products (q - z) x is
//     formed by itself and enters the output with one fp32 fma by its step.
//   * Steps and zeros of the block's rows are contiguous; they are copied to
//     LDS once, laid out by group, while the first codes are on their way.
//   * bf16 activations: differences are brought to bf16, exactly for integer
//     zeros up to 240 in magnitude; where a wavefront sees others it multiplies
//     the remainders too.
#include "awq_internal.h"
#include "w4_device.h"

namespace awq {

template <typename T, int GROUP, bool GATED, int ACT, int MT, int RT, int W, typename TY>
__global__ void __launch_bounds__(W * 64)
k_w4_skinny(const T* __restrict__ X, int M, int K, int O, const uint32_t* __restrict__ qw,
            const _Float16* __restrict__ step16, const _Float16* __restrict__ zero16,
            TY* __restrict__ Y, T* __restrict__ pre) {
  constexpr int R = 16 * RT;        // packed rows per block
  constexpr int GPB = 128 / GROUP;  // groups per block of 128 columns
  constexpr int JG = 4 / GPB;       // MFMAs per group
  constexpr int RP = R + 1;         // padded row count of the LDS sums
  extern __shared__ uint32_t lds[];  // [ng][R] (step, zero) pairs, then the wavefronts' sums
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int nkb = K >> 7, ng = K / GROUP, F = O >> 1;
  const int rb = blockIdx.x * (GATED ? R / 2 : R);  // first output of the block
  const int rows = GATED ? F : O;                   // outputs
  // packed row of row i of the block; rows past the end repeat the last one
  auto row_of = [&](int i) {
    if (GATED) return min(rb + i % (R / 2), F - 1) + (i < R / 2 ? 0 : F);
    return min(rb + i, O - 1);
  };
  const uint32_t* qrow[RT];
#pragma unroll
  for (int u = 0; u < RT; ++u) qrow[u] = qw + (size_t)row_of(16 * u + r16) * (K >> 3) + 4 * q4;
  const T* xrow[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) xrow[m] = X + (size_t)min(16 * m + r16, M - 1) * K + 8 * q4;

  uint4 cw[RT];
  auto load_codes = [&](int kb) {
#pragma unroll
    for (int u = 0; u < RT; ++u) cw[u] = *(const uint4*)(qrow[u] + 16 * kb);
  };
  uint4 xv[MT][4];
  auto load_x = [&](int kb) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) xv[m][j] = *(const uint4*)(xrow[m] + 128 * kb + 32 * j);
  };
  if (wave < nkb) {
    load_codes(wave);
    load_x(wave);
  }
  // (step, zero) of row i, group g at lds[g * R + i]
  for (int e = tid; e < R * ng; e += W * 64) {
    const int i = e / ng, g = e - i * ng;
    const size_t at = (size_t)row_of(i) * ng + g;
    lds[g * R + i] = (uint32_t)__builtin_bit_cast(uint16_t, step16[at]) |
                     ((uint32_t)__builtin_bit_cast(uint16_t, zero16[at]) << 16);
  }
  __syncthreads();

  floatx4 acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int u = 0; u < RT; ++u) acc[m][u] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = wave; kb < nkb; kb += W) {
    uint4 c[RT], x[MT][4];
#pragma unroll
    for (int u = 0; u < RT; ++u) c[u] = cw[u];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[m][j] = xv[m][j];
    // the next block's operands are on their way during this block's products
    const int next = min(kb + W, nkb - 1);
    load_codes(next);
    load_x(next);
#pragma unroll
    for (int u = 0; u < RT; ++u) {
      transpose_words(c[u]);
#pragma unroll
      for (int g = 0; g < GPB; ++g) {
        const uint32_t sz = lds[(kb * GPB + g) * R + 16 * u + r16];
        const _Float16 z = __builtin_bit_cast(_Float16, (uint16_t)(sz >> 16));
        const uint32_t nz = neg_zero_pair(z);
        const float st = f16_lo(sz) * kCodeScale;
        floatx4 t[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) t[m] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        uint4 b[JG];
#pragma unroll
        for (int j = 0; j < JG; ++j) b[j] = dequant_word(word_of(c[u], g * JG + j), nz);
        if constexpr (!__is_same(T, _Float16)) {
          const float zf = (float)z;
          const bool odd = !(fabsf(zf) <= 240.0f) || zf != __builtin_rintf(zf);
          uint4 d[JG];
#pragma unroll
          for (int j = 0; j < JG; ++j) {
            d[j] = b[j];
            b[j] = make_uint4(half2_to_bf16x2(d[j].x), half2_to_bf16x2(d[j].y),
                              half2_to_bf16x2(d[j].z), half2_to_bf16x2(d[j].w));
          }
          if (__any(odd)) {
#pragma unroll
            for (int j = 0; j < JG; ++j) {
              const uint4 e = make_uint4(
                  half2_minus_bf16x2(d[j].x, b[j].x), half2_minus_bf16x2(d[j].y, b[j].y),
                  half2_minus_bf16x2(d[j].z, b[j].z), half2_minus_bf16x2(d[j].w, b[j].w));
#pragma unroll
              for (int m = 0; m < MT; ++m) t[m] = mfma16<T>(x[m][g * JG + j], e, t[m]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < JG; ++j)
#pragma unroll
          for (int m = 0; m < MT; ++m) t[m] = mfma16<T>(x[m][g * JG + j], b[j], t[m]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][u][r] = fmaf(st, t[m][r], acc[m][u][r]);
      }
    }
  }

  // the wavefronts' sums, 16 tokens at a time: register r of lane l is token
  // 4 (l / 16) + r, row 16 u + l % 16
  float* const red = (float*)lds;  // [W][16][RP]
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    __syncthreads();
#pragma unroll
    for (int u = 0; u < RT; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[(wave * 16 + 4 * q4 + r) * RP + 16 * u + r16] = acc[m][u][r];
    __syncthreads();
    constexpr int C = GATED ? R / 2 : R;
    for (int e = tid; e < 16 * C; e += W * 64) {
      const int t = e / C, i = e - t * C, token = 16 * m + t;
      if (token >= M || rb + i >= rows) continue;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[(w * 16 + t) * RP + i];
      if (GATED) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += red[(w * 16 + t) * RP + C + i];
        if (pre) {
          pre[(size_t)token * O + rb + i] = from_f32<T>(s);
          pre[(size_t)token * O + F + rb + i] = from_f32<T>(v);
        }
        s = act_value<ACT>(s, nullptr) * v;
      }
      Y[(size_t)token * rows + rb + i] = from_f32<TY>(s);
    }
  }
}

template <typename T, int GROUP, bool GATED, int ACT, int MT, int RT, int W, typename TY>
static hipError_t launch(const W4Args& a, hipStream_t stream) {
  constexpr int R = 16 * RT;
  const int64_t outs = GATED ? a.O / 2 : a.O;
  const int per = GATED ? R / 2 : R;
  const size_t params = (size_t)R * (a.K / GROUP) * 4;
  const size_t sums = (size_t)W * 16 * (R + 1) * 4;
  const size_t lds = params > sums ? params : sums;
  auto* kernel = &k_w4_skinny<T, GROUP, GATED, ACT, MT, RT, W, TY>;
  // above 64 KiB the runtime wants to be told
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)((outs + per - 1) / per)), dim3(W * 64), lds, stream,
                     (const T*)a.in0, (int)a.N, (int)a.K, (int)a.O, (const uint32_t*)a.qweight,
                     (const _Float16*)a.step16, (const _Float16*)a.zero16, (TY*)a.out0,
                     (T*)a.out1);
  return hipGetLastError();
}

#ifndef AWQ_SKINNY_RT
#define AWQ_SKINNY_RT 4
#define AWQ_SKINNY_W 8
#endif

template <typename T, int GROUP, bool GATED, int ACT, typename TY>
static hipError_t by_tokens(const W4Args& a, hipStream_t stream) {
  constexpr int RT = AWQ_SKINNY_RT, W = AWQ_SKINNY_W;
  if (a.N <= 16) return launch<T, GROUP, GATED, ACT, 1, RT, W, TY>(a, stream);
  if (a.N <= 32) return launch<T, GROUP, GATED, ACT, 2, RT, W, TY>(a, stream);
  if (a.N <= 48) return launch<T, GROUP, GATED, ACT, 3, RT, W, TY>(a, stream);
  return launch<T, GROUP, GATED, ACT, 4, RT, W, TY>(a, stream);
}

template <typename T, int GROUP>
static hipError_t by_op(W4Op op, const W4Args& a, hipStream_t stream) {
  if (op == kOpGated)
    return a.act == kActSilu ? by_tokens<T, GROUP, true, kActSilu, T>(a, stream)
                             : by_tokens<T, GROUP, true, kActGelu, T>(a, stream);
  return a.y_type == kF32 ? by_tokens<T, GROUP, false, 0, float>(a, stream)
                          : by_tokens<T, GROUP, false, 0, T>(a, stream);
}

// The steps and zeros of a block's rows have to fit its LDS.
bool w4_skinny_fits(const W4Args& a) {
  return a.N <= 64 && (size_t)16 * AWQ_SKINNY_RT * (a.K / a.group) * 4 <= 160 * 1024;
}

hipError_t launch_w4_skinny(W4Op op, const W4Args& a, hipStream_t stream) {
  if (a.type == kF16) {
    if (a.group == 128) return by_op<_Float16, 128>(op, a, stream);
    if (a.group == 64) return by_op<_Float16, 64>(op, a, stream);
    return by_op<_Float16, 32>(op, a, stream);
  }
  if (a.group == 128) return by_op<__bf16, 128>(op, a, stream);
  if (a.group == 64) return by_op<__bf16, 64>(op, a, stream);
  return by_op<__bf16, 32>(op, a, stream);
}

}  // namespace awq
