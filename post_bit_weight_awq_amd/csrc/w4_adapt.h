// Adapters of rank R beside a packed product: for each token t of adapter a
//   low[t, r] = sum_k X[t, k] A[a, r, k],   Y[t, o] += scale[a] low[t] . B[a, o]
// Tiled products: low comes from k_adapt_low (w4_adapt.hip), and they add the
// second term to their sums before they leave a block.  Streaming product: further
// blocks of its launch sum low, and k_adapt_add adds the second term behind it.
#pragma once

#include <type_traits>

#include "w4_internal.h"

namespace awq {

// What a tiled product's kernel sees: `parts`, scale low as sums of 16-bit values
// (fp16: two, in units of 2^up[t]; bf16: two, three for fp32 outputs), [N, width],
// value p of rank r at p R + r, zeros behind.
struct Adapters {
  static constexpr bool on = true;
  const int32_t* ids;
  const char* mat;  // [count, columns, R]
  const char* parts;
  const int* up;
  int count, rank, width, nparts;
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

// An unaligned 16-byte load of eight values, those from `left` on as 0.
__device__ __forceinline__ uint4 load8(const uint16_t* p, int left) {
  typedef uint16_t u16x8 __attribute__((ext_vector_type(8), aligned(2)));
  if (left >= 8) return __builtin_bit_cast(uint4, *(const u16x8*)p);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kLowWaves = 8;

struct LowArgs {
  const uint16_t *X, *A;  // [N, K] dense; [count][rank][lda]
  const int32_t* ids;
  const float* scale;  // of the parts
  float* low;          // [splits, N, rank]
  float* out;          // [N, rank] or NULL
  uint16_t* parts;
  int* up;  // fp16's parts
  int N, K, lda, count, rank, width, nparts, splits;
  int scaled;  // out takes the scale too
};

// Tile of 16 MT tokens by 16 RT ranks, eight wavefronts along piece `split` of the
// sum.  Single tokens (SLOTS): a block takes the slot-th adapter of its tile and
// 16 ranks from r0 on; else all of both, one adapter after another.  Pieces' sums
// lie in `low` one behind the other.  FULL: K is a multiple of 32, so rows are
// aligned and no step needs a check: a wavefront then has U steps' loads in
// flight.
// Bound by what a compute unit gets from L2 (about 30 bytes a ns here): high tiles
// read A less often, pieces keep all units busy (4096 tokens, 15360 columns, rank
// 64: 83 us with 16 tokens and whole sums, 40 with 64 and quarters).
template <typename T, int MT, int RT, int U, bool SLOTS, bool FULL>
__device__ __forceinline__ void sum_low(const LowArgs& a, float* red, int split, int tile, int slot, int r0) {
  constexpr int R = 16 * RT, RP = R + 1, M = 16 * MT, W = kLowWaves;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int t0 = tile * M, ranks = SLOTS ? min(16, a.rank - r0) : a.rank;
  int id = -1;
  if (lane < M && t0 + lane < a.N) id = a.ids[t0 + lane];
  if (id >= a.count) id = -1;
  uint64_t wait = __ballot(id >= 0);
  float* const low = a.low + (size_t)split * a.N * a.rank;
  // tokens without an adapter have zeros
  if (!SLOTS)
    for (int e = tid; e < M * a.rank; e += 64 * W) {
      const int t = e / a.rank;
      if (t0 + t < a.N && !((wait >> t) & 1)) low[(size_t)t0 * a.rank + e] = 0.0f;
    }
  if (SLOTS) {
    for (int z = slot; z > 0 && wait; --z) {
      const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(wait));
      wait &= ~__ballot(id == one);
    }
    if (!wait) return;
  }
  const int steps = (a.K + 31) >> 5;
  const int s0 = (int)((int64_t)steps * split / a.splits), s1 = (int)((int64_t)steps * (split + 1) / a.splits);
  const uint16_t* x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) x[m] = a.X + (int64_t)min(t0 + 16 * m + r16, a.N - 1) * a.K + 8 * q4;
  while (wait) {
    const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(wait));
    const uint64_t mine = __ballot(id == one);
    wait = SLOTS ? 0 : wait & ~mine;
    floatx4 acc[MT][RT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < RT; ++n) acc[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint16_t* w[RT];
#pragma unroll
    for (int n = 0; n < RT; ++n)
      w[n] = a.A + ((int64_t)one * a.rank + min(r0 + 16 * n + r16, a.rank - 1)) * a.lda + 8 * q4;
    auto take = [&](int s, auto count) {
      constexpr int C = decltype(count)::value;
      uint4 xv[C][MT], wv[C][RT];
#pragma unroll
      for (int h = 0; h < C; ++h) {
        const int c = 32 * (s + h), left = a.K - c - 8 * q4;
#pragma unroll
        for (int m = 0; m < MT; ++m) xv[h][m] = FULL ? *(const uint4*)(x[m] + c) : load8(x[m] + c, left);
#pragma unroll
        for (int n = 0; n < RT; ++n) wv[h][n] = FULL ? *(const uint4*)(w[n] + c) : load8(w[n] + c, left);
      }
#pragma unroll
      for (int h = 0; h < C; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < RT; ++n) acc[m][n] = mfma16<T>(xv[h][m], wv[h][n], acc[m][n]);
    };
    // U neighbouring steps of 32 columns at a time
    for (int s = s0 + U * wave; s < s1; s += U * W) {
      if (s + U <= s1)
        take(s, std::integral_constant<int, U>{});
      else
        for (int h = s; h < s1; ++h) take(h, std::integral_constant<int, 1>{});
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m > 0) __syncthreads();
#pragma unroll
      for (int n = 0; n < RT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[(wave * 16 + 4 * q4 + r) * RP + 16 * n + r16] = acc[m][n][r];
      __syncthreads();
      for (int e = tid; e < 16 * ranks; e += 64 * W) {
        const int t = e / ranks, r = e - t * ranks;
        if (!((mine >> (16 * m + t)) & 1)) continue;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) v += red[(i * 16 + t) * RP + r];
        low[(size_t)(t0 + 16 * m + t) * a.rank + r0 + r] = v;
      }
    }
    if (!SLOTS) __syncthreads();
  }
}

// Blocks behind the streaming product's own, for single tokens: all pieces, tiles,
// adapters of a tile and rank tiles.
struct LowBlocks {
  static constexpr bool on = true;
  LowArgs a;
  int first, tiles, slots, ranks;
  __host__ __device__ int blocks() const { return a.splits * tiles * slots * ranks; }
  template <typename T>
  __device__ __forceinline__ void run(int b, float* red) const {
    const int split = b % a.splits;
    b /= a.splits;
    const int r = b % ranks;
    b /= ranks;
    sum_low<T, 1, 1, 4, true, true>(a, red, split, b / slots, b % slots, 16 * r);
  }
};

// w4_gemm.hip, w4_input_grad.hip with adapters, w4_skinny.hip with blocks for low
// beside it: `a` as for the plain product, its workspace at a.ws.
hipError_t launch_w4_gemm_adapted(const W4Args& a, const Adapters& ad, hipStream_t stream);
hipError_t launch_w4_input_grad_adapted(const W4Args& a, const Adapters& ad, hipStream_t stream);
hipError_t launch_w4_skinny_low(const W4Args& a, const LowBlocks& low, hipStream_t stream);

}  // namespace awq
