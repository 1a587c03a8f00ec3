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
__device__ __forceinline__ TileUnit tile_unit(int b, int nt, int no, int total) {
  const int x = b & 7, i = b >> 3;
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

// A launch runs its tiles in rounds of one per compute unit.  The tiles of a
// last, partial round are split along the sum into parts that fill the chip;
// the parts' sums go to the workspace in fp32 and a second launch adds them in
// order.  `full` tiles run whole, `left` in `parts` parts.
struct TileSplit {
  int nt, no, steps, full, left, parts;
};
constexpr int kCUs = 256;

// Microseconds of a tile of 32 mt tokens by 256 (mt = 2, 4, 6, 8) per
// iteration of its kernel, which takes `per` steps of the sum; the rest is
// common to all.
struct TileCosts {
  float step[4];
  int per[4];
};
constexpr float kTileStart = 5.0f;            // a tile's first loads and its epilogue
constexpr float kJoinStart = 4.0f;            // the second launch
constexpr float kPartRate = 6.0e6f;           // bytes per microsecond of parts, written and read

// Tile height and split with the least estimated time; `scale` multiplies the
// steps' cost.
inline void choose_tiles(int64_t N, int no, int all_steps, const TileCosts& c, float scale, int* mt_out,
                         TileSplit* out) {
  float best = 0.0f;
  for (int i = 0; i < 4; ++i) {
    const int mt = 2 * (i + 1), steps = (all_steps + c.per[i] - 1) / c.per[i];
    const int nt = (int)((N + 32 * mt - 1) / (32 * mt));
    const int total = nt * no, left = total % kCUs;
    const float step = scale * c.step[i], tile = step * steps + kTileStart;
    for (int parts = 1; parts <= 32 && parts <= steps; ++parts) {
      if (parts > 1 && left == 0) break;
      const int whole = total - left;
      float t = (float)(whole / kCUs) * tile;
      if (left) {
        const int rounds = (left * parts + kCUs - 1) / kCUs;
        t += (float)rounds * (step * (float)((steps + parts - 1) / parts) + kTileStart);
        if (parts > 1) t += kJoinStart + 2.0f * left * parts * mt * 32768.0f / kPartRate;
      }
      // low tiles read the weights more often: in more than two rounds they took
      // a tenth longer than that (4096 x 5120 <- 27648: 1.17 against 1.11 ms on
      // 256-token tiles)
      if (mt <= 4 && total > 2 * kCUs) t *= 1.1f;
      if (best == 0.0f || t < best) {
        best = t;
        *mt_out = mt;
        *out = parts > 1 ? TileSplit{nt, no, steps, whole, left, parts}
                         : TileSplit{nt, no, steps, total, 0, 1};
      }
    }
  }
}
// Measured with one tile per unit on 512 x 4096 x 4096, 1024 x 13824 -> 5120
// for the products (w4_gemm.hip, 128 columns a step) and 128 x 4096 <- 11008
// for the input gradient (w4_input_grad.hip, 64 packed rows a step).
constexpr TileCosts kGemmCosts = {{2.2f, 3.05f, 2.4f, 2.95f}, {2, 2, 1, 1}};
constexpr TileCosts kDxCosts = {{1.15f, 1.42f, 1.25f, 1.45f}, {2, 2, 1, 1}};

struct SplitUnit {
  int t, o, s0, s1, parts, slot;  // steps s0 .. s1 - 1
};
__device__ __forceinline__ SplitUnit split_unit(int b, const TileSplit& s) {
  SplitUnit r;
  const int i = b - s.full;
  const bool whole = i < 0;
  const int tile = whole ? b : s.full + i / s.parts, part = whole ? 0 : i % s.parts;
  const TileUnit u = tile_unit(tile, s.nt, s.no, s.full + s.left);
  r.t = u.t;
  r.o = u.o;
  r.parts = whole ? 1 : s.parts;
  r.s0 = (int)((int64_t)s.steps * part / r.parts);
  r.s1 = (int)((int64_t)s.steps * (part + 1) / r.parts);
  r.slot = i;
  return r;
}

// The sum, in order, of a split tile's parts for tiles 2 mp and 2 mp + 1 of
// wavefront `wave`'s mt x 4; parts are kept as the wavefronts' registers.
__device__ __forceinline__ void join_parts(const float* parts, const TileSplit& sp, int left, int wave,
                                           int mt, int mp, int lane, floatx4 (&v)[2][4]) {
  const size_t tile = (size_t)mt * 4 * 64;
  const floatx4* p = (const floatx4*)parts + ((size_t)left * sp.parts * 8 + wave) * tile +
                     mp * 8 * 64 + lane;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = p[i * 64];
  // four parts' loads in flight at a time (past the end the last part's,
  // which are not added)
  for (int k = 1; k < sp.parts; k += 4) {
    floatx4 t[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] = p[(size_t)min(k + j, sp.parts - 1) * 8 * tile + i * 64];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k + j < sp.parts)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] += t[j][i];
  }
}

// What the last step of a product does with its sums.
struct Epilogue {
  const int* back;  // a token's exponent, or NULL
  void *y, *pre;
  int N, O, y_type, type, act;
};

// Direct loads to LDS: 16 (or 4) bytes per lane from base + off to l + 16 (4)
// times the lane.  l goes to M0 as an operand, so that the compiler writes the
// register and knows it; the load needs a wait state behind that.
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t l) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "{m0}"(l) : "memory");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t l) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" : : "v"(off), "s"(base), "{m0}"(l) : "memory");
}
// All but the wavefront's last N vector memory operations have ended.
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
}

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

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

// One launch before the tiled kernels (w4_prepare.hip).
struct Prepare {
  const _Float16 *step16, *zero16;
  int O, ng;
  void* prm;
  int* big;     // input gradient
  int* parted;  // products: one per 32 rows x 32 groups
  float* lows;  // products: [ng, O]
  float* sums;  // products: [rows, ng], each row's sums over groups of 2^shift
  int shift;
  // rows: cols values of in0 (gated: cols / 2 of dH in in0 and cols of pre in
  // in1, giving dpre) to out, ld_out apart; out may be NULL with gated
  const void *in0, *in1;
  void* dpre;
  int cols, ld_out, act;
  void* out;
  int* back;
  int param_blocks;
};
// params: 0 none, 1 the products', 2 the input gradient's; gated with 2 alone
hipError_t launch_w4_prepare(const Prepare& p, int type, int params, bool gated, int64_t rows,
                             hipStream_t stream);

// linear and gated (w4_gemm.hip), input gradient and gated backward
// (w4_input_grad.hip), parameter gradients (w4_param_grad.hip)
size_t w4_gemm_workspace(W4Op op, const W4Args& a);
hipError_t launch_w4_gemm(W4Op op, const W4Args& a, hipStream_t stream);
size_t w4_input_grad_workspace(const W4Args& a);
hipError_t launch_w4_input_grad(W4Op op, const W4Args& a, hipStream_t stream);
size_t w4_param_grad_workspace(const W4Args& a);
hipError_t launch_w4_param_grad(const W4Args& a, hipStream_t stream);

}  // namespace awq
