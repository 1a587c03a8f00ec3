// What the packed-weight kernels share beyond w4_device.h: tile order, output
// stores, and the launchers that call one another.
#pragma once

#include "awq_internal.h"
#include "w4_device.h"

namespace awq {

// Block b runs on XCD b % 8.  Each XCD takes a contiguous share of the tiles
// in an order that walks strips of four output tiles through all token tiles,
// so the 32 blocks it holds at a time cover about eight token tiles by four
// output tiles and share both operands in its L2.
struct TileUnit {
  int t, o;
};
__device__ __forceinline__ TileUnit tile_unit(int b, int nt, int no) {
  const int total = nt * no, x = b & 7, i = b >> 3;
  // XCD x has total / 8 tiles, one more for the first total % 8
  const int per = total >> 3, rest = total & 7;
  const int u = x * per + min(x, rest) + i;
  const int strip = u / (4 * nt), in = u - strip * 4 * nt;
  const int wide = min(4, no - 4 * strip);
  TileUnit r;
  r.t = in / wide;
  r.o = 4 * strip + in - r.t * wide;
  return r;
}

// Up to eight values of one row, rounded once: `n` are left in the row; whole
// 16-byte stores where rows begin on such a boundary.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int n, bool aligned) {
  if (aligned && n >= 8) {
    if constexpr (sizeof(T) == 4) {
      *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
      *(float4*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = (uint32_t)__builtin_bit_cast(uint16_t, from_f32<T>(v[2 * e])) |
               ((uint32_t)__builtin_bit_cast(uint16_t, from_f32<T>(v[2 * e + 1])) << 16);
      *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = from_f32<T>(v[e]);
  }
}

hipError_t launch_rows_to_half(const void* in, int64_t rows, int64_t cols, int64_t ld_out, void* out,
                               int* back, hipStream_t stream);
size_t w4_gemm_workspace(const W4Args& a);
hipError_t launch_w4_gemm(W4Op op, const W4Args& a, hipStream_t stream);

}  // namespace awq
