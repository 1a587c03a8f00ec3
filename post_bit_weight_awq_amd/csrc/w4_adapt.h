// Adapters of rank R beside a packed product: for each token t of adapter a
//   low[t, r] = sum_k X[t, k] A[a, r, k],   Y[t, o] += scale[a] low[t] . B[a, o]
// low comes from k_adapt_low (w4_adapt.hip); the products add the second term to
// their sums before they leave a block.
#pragma once

#include "w4_internal.h"

namespace awq {

// What a product's kernel sees.  The tiled kernels read `parts`: scale low as
// sums of 16-bit values (fp16: two, in units of 2^up[t]; bf16: two, three for
// fp32 outputs), [N, width], value p of rank r at p R + r, zeros behind; the
// streaming kernel reads `low`, [splits, N, R] in fp32, and the scales.
struct Adapters {
  static constexpr bool on = true;
  const int32_t* ids;
  const char* mat;  // [count, columns, R]
  const char* parts;
  const int* up;
  const float *low, *scale;
  int count, rank, width, nparts, splits;
};
struct NoAdapters {
  static constexpr bool on = false;
};

// One token in a tile of 16 has its adapter by itself: all 16 rows are multiplied
// with an adapter that any has and only its own rows take the result, so that
// what another token or adapter holds stays out of a token's sums.
// acc: tiles of 16 tokens from t0 by the columns col_of(n), in units of
// 2^-back[t].
template <int MT, typename ColOf>
__device__ __forceinline__ void add_adapters(floatx4 (&acc)[MT][4], const Adapters& ad, int type,
                                             const int* back, ColOf col_of, int cols, int t0, int N,
                                             int lane) {
  const int r16 = lane & 15, q4 = lane >> 4;
  const int rb = ad.rank >> 3, blocks = ad.nparts * rb;  // of eight ranks
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    // a tile's loads stay behind the one before it: the sums fill the registers
    asm volatile("" ::: "memory");
    const int t = t0 + 16 * m + r16;
    const int v = t < N ? ad.ids[t] : -1;
    const int id = v < ad.count ? v : -1;
    const char* u = ad.parts + (int64_t)min(t, N - 1) * ad.width * 2 + 16 * q4;
    uint64_t wait = __ballot(id >= 0);
    while (wait) {
      const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(wait));
      wait &= ~__ballot(id == a);
      const char* mat = ad.mat + (int64_t)a * cols * ad.rank * 2;
      floatx4 d[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) d[n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int c = 0; c < ad.width >> 5; ++c) {
        const uint4 x = *(const uint4*)(u + 64 * c);
        const int e = 4 * c + q4;
        const int r = e - (int)((uint32_t)e / (uint32_t)rb) * rb;
        uint4 b[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          b[n] = *(const uint4*)(mat + ((int64_t)col_of(n) * rb + r) * 16);
          if (e >= blocks) b[n] = make_uint4(0, 0, 0, 0);
        }
        if (type == kF16) {
#pragma unroll
          for (int n = 0; n < 4; ++n) d[n] = mfma16<_Float16>(x, b[n], d[n]);
        } else {
#pragma unroll
          for (int n = 0; n < 4; ++n) d[n] = mfma16<__bf16>(x, b[n], d[n]);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tr = min(t0 + 16 * m + 4 * q4 + r, N - 1);
        const int sh = (ad.up ? ad.up[tr] : 0) - (back ? back[tr] : 0);
        const bool mine = __shfl(id, 4 * q4 + r) == a;
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[m][n][r] += mine ? ldexpf(d[n][r], sh) : 0.0f;
      }
    }
  }
}

// w4_gemm.hip, w4_input_grad.hip, w4_skinny.hip with adapters: `a` as for the
// plain product, its workspace at a.ws.
hipError_t launch_w4_gemm_adapted(const W4Args& a, const Adapters& ad, hipStream_t stream);
hipError_t launch_w4_input_grad_adapted(const W4Args& a, const Adapters& ad, hipStream_t stream);
bool w4_skinny_fits_adapted(const W4Args& a, int rank);
hipError_t launch_w4_skinny_adapted(const W4Args& a, const Adapters& ad, hipStream_t stream);

}  // namespace awq
