// Low-rank adapters beside a packed product, for tokens that each may have
// another one: what the products' kernels (w4_adapt.h) do not do themselves.
//
//   k_adapt_low    low[t] = X[t] A[a_t]^T, or v[t] = scale dY[t] B[a_t]: tiles of
//                  tokens, the wavefronts of a block share the sum's columns.
//                  Bound by reading X once; for single tokens by latency, so
//                  each adapter of a tile and parts of the sum get a block.
//   k_adapt_order  the backward pass's copies A^T and B^T, whose rows are what the
//                  products read, and each adapter's tokens in order
//   k_adapt_grad   dA[a] = sum over a's tokens of v[t]^T X[t], dB[a] likewise of dY
//                  and low: the left side's fp32 values as sums of 16-bit parts,
//                  the right side transposed in registers; a long list of tokens is
//                  taken in chunks, k_adapt_join adds them in order
#include "w4_adapt.h"

namespace awq {

constexpr int kOrder = 256;

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

// v as a sum of 16-bit values, the first the nearest.  What is not finite is the
// first one alone.
template <typename T, int P>
__device__ __forceinline__ void split_parts(float v, uint16_t (&out)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const T h = from_f32<T>(v);
    out[p] = __builtin_bit_cast(uint16_t, h);
    v = fabsf(v) < INFINITY ? v - to_f32(h) : 0.0f;
  }
}
// Exponent that brings a largest magnitude to 2^14 .. 2^15, 0 for 0 and what is
// not finite: fp16's parts then lose nothing above 2^-39 of it.
__device__ __forceinline__ int up_of(float top) {
  if (!(top > 0.0f) || !(top < INFINITY)) return 0;
  int e;
  frexpf(top, &e);
  return e - 15;
}

struct LowArgs {
  const uint16_t *X, *A;  // [N, K] dense; [count][rank][lda]
  const int32_t* ids;
  const float* scale;  // of the parts
  float* low;          // [splits, N, rank] or NULL
  uint16_t* parts;     // or NULL
  int* up;             // fp16's parts
  int N, K, lda, count, rank, width, nparts, splits;
  int scaled;          // low takes the scale too
};

constexpr int kLowWaves = 8;

// Tile of 16 MT tokens by 16 RT ranks (all).  SLOTS: block z takes the z-th
// adapter of its tile and every splits-th piece of the sum; else a block takes
// all of them one by one and leaves parts.
template <typename T, int MT, int RT, bool SLOTS>
__global__ void __launch_bounds__(64 * kLowWaves)
k_adapt_low(LowArgs a) {
  constexpr int R = 16 * RT, RP = R + 1, M = 16 * MT;
  extern __shared__ float red[];  // [wavefront][M][RP]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int t0 = blockIdx.y * M;
  int id = -1;
  if (lane < M && t0 + lane < a.N) id = a.ids[t0 + lane];
  if (id >= a.count) id = -1;
  const int split = SLOTS ? blockIdx.x : 0;
  uint64_t wait = __ballot(id >= 0);
  // tokens without an adapter have zeros
  const bool first = !SLOTS || blockIdx.z == 0;
  auto leave = [&](int t, float v0, float v1) {  // ranks lane and lane + 64
    const int token = t0 + t;
    if (a.low) {
      float* p = a.low + ((size_t)split * a.N + token) * a.rank;
      if (lane < a.rank) p[lane] = v0;
      if (lane + 64 < a.rank) p[lane + 64] = v1;
    }
  };
  if (first)
    for (int t = wave; t < M && t0 + t < a.N; t += kLowWaves)
      if (!((wait >> t) & 1)) leave(t, 0.0f, 0.0f);
  if (SLOTS) {
    for (int z = blockIdx.z; z > 0 && wait; --z) {
      const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(wait));
      wait &= ~__ballot(id == one);
    }
    if (!wait) return;
  }
  const int steps = (a.K + 31) >> 5;
  const int s0 = (int)((int64_t)steps * split / a.splits), s1 = (int)((int64_t)steps * (split + 1) / a.splits);
  while (wait) {
    const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(wait));
    const uint64_t mine = __ballot(id == one);
    wait = SLOTS ? 0 : wait & ~mine;
    floatx4 acc[MT][RT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < RT; ++n) acc[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint16_t* x[MT];
    const uint16_t* w[RT];
#pragma unroll
    for (int m = 0; m < MT; ++m) x[m] = a.X + (int64_t)min(t0 + 16 * m + r16, a.N - 1) * a.K + 8 * q4;
#pragma unroll
    for (int n = 0; n < RT; ++n)
      w[n] = a.A + ((int64_t)one * a.rank + min(16 * n + r16, a.rank - 1)) * a.lda + 8 * q4;
    // two neighbouring steps of 32 columns at a time
    for (int s = s0 + 2 * wave; s < s1; s += 2 * kLowWaves) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = s + h;
        const int left = c < s1 ? a.K - 32 * c - 8 * q4 : 0;
        uint4 xv[MT], wv[RT];
#pragma unroll
        for (int m = 0; m < MT; ++m) xv[m] = load8(x[m] + 32 * c, left);
#pragma unroll
        for (int n = 0; n < RT; ++n) wv[n] = load8(w[n] + 32 * c, left);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < RT; ++n) acc[m][n] = mfma16<T>(xv[m], wv[n], acc[m][n]);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < RT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          red[(wave * M + 16 * m + 4 * q4 + r) * RP + 16 * n + r16] = acc[m][n][r];
    __syncthreads();
    const float scale = a.scale[one];
    for (int t = wave; t < M; t += kLowWaves) {
      if (!((mine >> t) & 1)) continue;
      float v[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kLowWaves; ++i) {
        if (lane < R) v[0] += red[(i * M + t) * RP + lane];
        if (lane + 64 < R) v[1] += red[(i * M + t) * RP + lane + 64];
      }
      const float k = a.scaled ? scale : 1.0f;
      leave(t, v[0] * k, v[1] * k);
      if (!SLOTS && a.parts) {
        v[0] = lane < a.rank ? v[0] * scale : 0.0f;
        v[1] = lane + 64 < a.rank ? v[1] * scale : 0.0f;
        uint16_t* p = a.parts + (int64_t)(t0 + t) * a.width;
        if constexpr (__is_same(T, _Float16)) {
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < 2; ++i) top = fmaxf(top, fabsf(v[i]) < INFINITY ? fabsf(v[i]) : 0.0f);
#pragma unroll
          for (int s = 1; s < 64; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
          const int e = up_of(top);
          if (lane == 0) a.up[t0 + t] = e;
          v[0] = ldexpf(v[0], -e);
          v[1] = ldexpf(v[1], -e);
        }
        uint16_t h[2][3];
        split_parts<T>(v[0], h[0]);
        split_parts<T>(v[1], h[1]);
        for (int i = 0; i < a.nparts; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (lane + 64 * j < a.rank)
              p[i * a.rank + lane + 64 * j] = i == 0 ? h[j][0] : i == 1 ? h[j][1] : h[j][2];
        const int end = a.nparts * a.rank;  // less than 32 zeros
        if (lane < a.width - end) p[end + lane] = 0;
      }
    }
    if (!SLOTS) __syncthreads();
  }
}

template <typename T, bool SLOTS>
static hipError_t launch_low(const LowArgs& a, hipStream_t stream) {
  const int rt = (a.rank + 15) / 16;
  auto go = [&](auto* kernel, int mt, int r) {
    const int M = 16 * mt, lds = kLowWaves * M * (16 * r + 1) * 4;
    if (lds > 65536) {
      const hipError_t e =
          hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
    }
    const unsigned tiles = (unsigned)((a.N + M - 1) / M);
    const dim3 grid(SLOTS ? a.splits : 1, tiles, SLOTS ? (unsigned)(a.N < 16 ? a.N : 16) : 1);
    hipLaunchKernelGGL(kernel, grid, dim3(64 * kLowWaves), lds, stream, a);
    return hipGetLastError();
  };
  constexpr int MT = SLOTS ? 1 : 2;
  if (rt == 1) return go(&k_adapt_low<T, MT, 1, SLOTS>, MT, 1);
  if (rt == 2) return go(&k_adapt_low<T, MT, 2, SLOTS>, MT, 2);
  if (rt <= 4) return go(&k_adapt_low<T, MT, 4, SLOTS>, MT, 4);
  return go(&k_adapt_low<T, MT, 8, SLOTS>, MT, 8);
}

// ------------------------------------------------------------ backward pass
struct OrderArgs {
  const uint16_t *A, *B;  // [count][rank][K], [count][O][rank]
  uint16_t *At, *Bt;      // [count][K][rank], [count][rank][ldb], zeros from O on
  const int32_t* ids;
  int32_t *order, *start;  // [N], [count + 1]
  int N, K, O, ldb, count, rank;
};

// Blocks 0 .. count - 1: the tokens of an adapter, in order.  The others: 64
// columns of A or B of an adapter, transposed through LDS.
__global__ void __launch_bounds__(kOrder)
k_adapt_order(OrderArgs a) {
  __shared__ uint16_t tile[64 * 129];
  __shared__ int wsum[kOrder / 64][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if ((int)blockIdx.x < a.count) {
    const int me = blockIdx.x;
    int less = 0, mine = 0;
    for (int t = tid; t < a.N; t += kOrder) {
      const int id = a.ids[t];
      less += id >= 0 && id < me;
      mine += id == me;
    }
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      less += __shfl_xor(less, s);
      mine += __shfl_xor(mine, s);
    }
    if (lane == 0) wsum[wave][0] = less, wsum[wave][1] = mine;
    __syncthreads();
    less = mine = 0;
    for (int i = 0; i < kOrder / 64; ++i) less += wsum[i][0], mine += wsum[i][1];
    __syncthreads();
    if (tid == 0) {
      a.start[me] = less;
      if (me == a.count - 1) a.start[a.count] = less + mine;
    }
    int at = less;
    if (!mine) return;
    // four neighbouring tokens per thread
    for (int b = 0; b < a.N; b += 4 * kOrder) {
      int hit = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = b + 4 * tid + i;
        if (t < a.N && a.ids[t] == me) hit |= 1 << i;
      }
      const int n = __popc(hit);
      int before = n;
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const int v = __shfl_up(before, s);
        if (lane >= s) before += v;
      }
      if (lane == 63) wsum[wave][0] = before;
      __syncthreads();
      int all = 0;
      before -= n;
#pragma unroll
      for (int i = 0; i < kOrder / 64; ++i) {
        if (i < wave) before += wsum[i][0];
        all += wsum[i][0];
      }
      __syncthreads();
      int p = at + before;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (hit >> i & 1) a.order[p++] = b + 4 * tid + i;
      at += all;
    }
    return;
  }
  const int ka = (a.K + 63) / 64, kb = (a.ldb + 63) / 64;
  const int64_t id = (int64_t)blockIdx.x - a.count;
  const int which = (int)(id % (ka + kb));
  const int64_t ad = id / (ka + kb);
  if (which < ka) {
    const int c0 = 64 * which;  // K is a multiple of 128
    const uint16_t* s = a.A + ad * a.rank * a.K + c0;
    for (int e = tid; e < 64 * a.rank; e += kOrder)
      tile[(e & 63) * 129 + (e >> 6)] = s[(int64_t)(e >> 6) * a.K + (e & 63)];
    __syncthreads();
    uint16_t* d = a.At + (ad * a.K + c0) * a.rank;
    for (int e = tid; e < 64 * a.rank; e += kOrder) d[e] = tile[(e / a.rank) * 129 + e % a.rank];
  } else {
    const int o0 = 64 * (which - ka);
    const uint16_t* s = a.B + (ad * a.O + o0) * a.rank;
    for (int e = tid; e < 64 * a.rank; e += kOrder)
      tile[(e / a.rank) * 129 + e % a.rank] = o0 + e / a.rank < a.O ? s[e] : (uint16_t)0;
    __syncthreads();
    uint16_t* d = a.Bt + ad * a.rank * a.ldb + o0;
    for (int e = tid; e < 64 * a.rank; e += kOrder)
      if (o0 + (e & 63) < a.ldb) d[(int64_t)(e >> 6) * a.ldb + (e & 63)] = tile[(e & 63) * 129 + (e >> 6)];
  }
}

struct GradArgs {
  const uint16_t *X, *dY;
  const float *v, *low, *scale;  // [N, rank]
  const int32_t *order, *start;
  float *dA, *dB;      // [count][rank][K], [count][O][rank]
  float *pA, *pB;      // of a unit
  int N, K, O, count, rank, chunk;
};
// Unit u: adapter a owns the units from start[a] / chunk + a on.
__device__ __forceinline__ int unit_base(const GradArgs& g, int a) { return g.start[a] / g.chunk + a; }

constexpr int kGradWaves = 4, kGradCols = 128;

// 16 RT ranks from 64 z on by 128 columns of X, then of dY; each wavefront takes
// every fourth 32 tokens of the chunk.
template <typename T, int RT>
__global__ void __launch_bounds__(64 * kGradWaves, 1)
k_adapt_grad(GradArgs g) {
  constexpr int R = 16 * RT, P = __is_same(T, _Float16) ? 2 : 3, CP = kGradCols + 4;
  extern __shared__ float red[];  // [2][R][CP]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int unit = blockIdx.y, r0 = 64 * blockIdx.z;
  int a = 0, hi = g.count;  // unit_base(a) <= unit < unit_base(hi)
  while (hi - a > 1) {
    const int mid = (a + hi) >> 1;
    if (unit_base(g, mid) <= unit)
      a = mid;
    else
      hi = mid;
  }
  const int begin = g.start[a], count = g.start[a + 1] - begin;
  const int piece = unit - unit_base(g, a);
  if (piece * g.chunk >= count) return;
  const int p0 = begin + piece * g.chunk, p1 = min(p0 + g.chunk, begin + count);
  const int ka = g.K / kGradCols;
  const bool right = (int)blockIdx.x >= ka;  // dB
  const int C = right ? g.O : g.K, c0 = kGradCols * (right ? blockIdx.x - ka : blockIdx.x);
  const uint16_t* Y = right ? g.dY : g.X;
  const float* L = right ? g.low : g.v;

  int up = 0;
  if constexpr (__is_same(T, _Float16)) {
    // fp16's parts are in units of the wavefront's largest value
    float top = 0.0f;
    const int per = min(R, g.rank - r0);
    for (int s = p0 + 32 * wave; s < p1; s += 32 * kGradWaves) {
      const int n = min(32, p1 - s) * per;
      for (int e = lane; e < n; e += 64) {
        const float v = fabsf(L[(int64_t)g.order[s + e / per] * g.rank + r0 + e % per]);
        top = fmaxf(top, v < INFINITY ? v : 0.0f);
      }
    }
#pragma unroll
    for (int s = 1; s < 64; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
    up = up_of(top);
  }
  floatx4 acc[RT][8];
#pragma unroll
  for (int m = 0; m < RT; ++m)
#pragma unroll
    for (int n = 0; n < 8; ++n) acc[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const int left = C - c0 - 8 * r16;  // columns from the lane's first on
  for (int s = p0 + 32 * wave; s < p1; s += 32 * kGradWaves) {
    uint4 y[8];
    float l[RT][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = s + 8 * q4 + i;
      const bool in = at < p1;
      const int64_t t = g.order[min(at, p1 - 1)];
      y[i] = load8(Y + t * C + c0 + 8 * r16, in ? left : 0);
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const int r = r0 + 16 * m + r16;
        const float v = L[t * g.rank + min(r, g.rank - 1)];
        l[m][i] = in && r < g.rank ? v : 0.0f;
      }
    }
    uint4 lp[RT][P];
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      uint16_t h[8][P];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        split_parts<T>(__is_same(T, _Float16) ? ldexpf(l[m][i], -up) : l[m][i], h[i]);
#pragma unroll
      for (int p = 0; p < P; ++p)
        lp[m][p] = make_uint4(h[0][p] | (uint32_t)h[1][p] << 16, h[2][p] | (uint32_t)h[3][p] << 16,
                              h[4][p] | (uint32_t)h[5][p] << 16, h[6][p] | (uint32_t)h[7][p] << 16);
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const uint32_t sel = n & 1 ? 0x07060302u : 0x05040100u;
      const uint4 b = make_uint4(__builtin_amdgcn_perm(word_of(y[1], n >> 1), word_of(y[0], n >> 1), sel),
                                 __builtin_amdgcn_perm(word_of(y[3], n >> 1), word_of(y[2], n >> 1), sel),
                                 __builtin_amdgcn_perm(word_of(y[5], n >> 1), word_of(y[4], n >> 1), sel),
                                 __builtin_amdgcn_perm(word_of(y[7], n >> 1), word_of(y[6], n >> 1), sel));
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int p = 0; p < P; ++p) acc[m][n] = mfma16<T>(lp[m][p], b, acc[m][n]);
    }
  }
  // tile n, lane l: ranks 4 (l / 16) + r, column 8 (l % 16) + n; the
  // wavefronts' sums in a tree of fixed order
  auto put = [&](float* p) {
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int n = 0; n < 8; ++n)
          p[(16 * m + 4 * q4 + r) * CP + 8 * r16 + n] = ldexpf(acc[m][n][r], up);
  };
  auto add = [&](const float* p) {
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int n = 0; n < 8; ++n)
          acc[m][n][r] = ldexpf(acc[m][n][r], up) + p[(16 * m + 4 * q4 + r) * CP + 8 * r16 + n];
    up = 0;
  };
  if (wave >= 2) put(red + (wave - 2) * R * CP);
  __syncthreads();
  if (wave < 2) add(red + wave * R * CP);
  __syncthreads();
  if (wave == 1) put(red);
  __syncthreads();
  if (wave == 0) {
    add(red);
    put(red);
  }
  __syncthreads();
  const int rows = min(R, g.rank - r0), cols = min(kGradCols, C - c0);
  const bool whole = count <= g.chunk;
  const float f = right && whole ? g.scale[a] : 1.0f;
  const int64_t to = whole ? a : unit;
  if (right) {
    float* d = (whole ? g.dB : g.pB) + (to * g.O + c0) * g.rank + r0;
    for (int e = tid; e < cols * rows; e += 64 * kGradWaves) {
      const int c = e / rows, r = e - c * rows;
      d[(int64_t)c * g.rank + r] = red[r * CP + c] * f;
    }
  } else {
    float* d = (whole ? g.dA : g.pA) + (to * g.rank + r0) * g.K + c0;
    for (int e = tid; e < rows * kGradCols; e += 64 * kGradWaves) {
      const int r = e / kGradCols, c = e % kGradCols;
      d[(int64_t)r * g.K + c] = red[r * CP + c];
    }
  }
}

// Adapters of several chunks: their sums, in order; of none: zeros.  Four values
// per thread.
__global__ void __launch_bounds__(256)
k_adapt_join(GradArgs g) {
  const int a = blockIdx.y;
  const int count = g.start[a + 1] - g.start[a];
  if (count > 0 && count <= g.chunk) return;
  const int64_t na = (int64_t)g.rank * g.K, nb = (int64_t)g.O * g.rank;
  const int64_t e = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (e >= na + nb) return;
  const bool right = e >= na;
  const int64_t at = right ? e - na : e, n = right ? nb : na;
  const float* p = (right ? g.pB : g.pA) + unit_base(g, a) * n + at;
  floatx4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = 0; i * g.chunk < count; ++i) s += *(const floatx4*)(p + i * n);
  if (right) {
    const float f = g.scale[a];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = count ? s[i] * f : 0.0f;
  }
  *(floatx4*)((right ? g.dB : g.dA) + a * n + at) = s;
}

// ------------------------------------------------------------------- plans
struct AdaptPlan {
  bool skinny;
  int splits, width, nparts, ldb, chunk, units;
  size_t off_low, off_parts, off_up, off_At, off_Bt, off_order, off_start, off_pA, off_pB, bytes;
};
static AdaptPlan adapt_plan(const W4Args& a, const W4Adapt& d, bool backward) {
  AdaptPlan p{};
  size_t at = backward ? w4_input_grad_workspace(a) : w4_workspace(kOpLinear, a);
  p.skinny = !backward && w4_skinny_fits_adapted(a, d.rank);
  if (!backward && !p.skinny) at = w4_gemm_workspace(kOpLinear, a);
  auto take = [&](size_t n) {
    const size_t r = align256(at);
    at = r + n;
    return r;
  };
  p.splits = 1;
  if (p.skinny) {
    // pieces of the sum of at least 256 columns, as many as give each unit a block;
    // a kept low is written whole
    const int64_t slots = (a.N + 15) / 16 * (a.N < 16 ? a.N : 16);
    int64_t n = kCUs / slots, most = a.K / 256;
    n = n > 16 ? 16 : n;
    n = n > most ? most : n;
    p.splits = d.low || n < 1 ? 1 : (int)n;
    p.off_low = take(d.low ? 0 : (size_t)p.splits * a.N * d.rank * 4);
  } else {
    p.nparts = a.type == kBF16 && a.y_type == kF32 ? 3 : 2;
    p.width = (p.nparts * d.rank + 31) & ~31;
    p.off_parts = take((size_t)a.N * p.width * 2);
    p.off_up = take((size_t)a.N * 4);
  }
  if (backward) {
    p.ldb = (int)((a.O + 31) & ~(int64_t)31);
    p.off_low = take((size_t)a.N * d.rank * 4);
    p.off_At = take((size_t)d.count * a.K * d.rank * 2);
    p.off_Bt = take((size_t)d.count * p.ldb * d.rank * 2);
    p.off_order = take((size_t)a.N * 4);
    p.off_start = take((size_t)(d.count + 1) * 4);
    // A chunk's sums are written and read in fp32: from eight tokens per rank on
    // they are at most half of what it reads; beyond that about four blocks per
    // unit.
    const int64_t tiles = (a.K + a.O + kGradCols - 1) / kGradCols * (d.rank > 64 ? 2 : 1);
    int64_t chunk = a.N * tiles / (4 * kCUs);
    if (chunk < 8 * d.rank) chunk = 8 * d.rank;
    p.chunk = (int)((chunk + 127) & ~(int64_t)127);
    p.units = (int)(a.N / p.chunk) + d.count;
    const bool many = a.N > p.chunk;  // else no adapter has two chunks
    p.off_pA = take(many ? (size_t)p.units * d.rank * a.K * 4 : 0);
    p.off_pB = take(many ? (size_t)p.units * d.rank * a.O * 4 : 0);
  }
  p.bytes = at;
  return p;
}
size_t w4_adapt_workspace(const W4Args& a, const W4Adapt& d, bool backward) {
  return adapt_plan(a, d, backward).bytes;
}

template <typename T>
static hipError_t forward(const W4Args& a, const W4Adapt& d, const AdaptPlan& p, hipStream_t stream) {
  char* ws = (char*)a.ws;
  LowArgs l{};
  l.X = (const uint16_t*)a.in0;
  l.A = (const uint16_t*)d.A;
  l.ids = d.ids;
  l.scale = d.scale;
  l.low = d.low ? d.low : p.skinny ? (float*)(ws + p.off_low) : nullptr;
  l.N = (int)a.N;
  l.K = l.lda = (int)a.K;
  l.count = d.count;
  l.rank = d.rank;
  l.splits = p.splits;
  Adapters ad{};
  ad.ids = d.ids;
  ad.mat = (const char*)d.B;
  ad.scale = d.scale;
  ad.count = d.count;
  ad.rank = d.rank;
  if (p.skinny) {
    ad.low = l.low;
    ad.splits = p.splits;
    const hipError_t e = launch_low<T, true>(l, stream);
    return e != hipSuccess ? e : launch_w4_skinny_adapted(a, ad, stream);
  }
  l.parts = (uint16_t*)(ws + p.off_parts);
  l.up = a.type == kF16 ? (int*)(ws + p.off_up) : nullptr;
  l.width = ad.width = p.width;
  l.nparts = ad.nparts = p.nparts;
  ad.parts = (const char*)l.parts;
  ad.up = l.up;
  const hipError_t e = launch_low<T, false>(l, stream);
  return e != hipSuccess ? e : launch_w4_gemm_adapted(a, ad, stream);
}

template <typename T>
static hipError_t backward(const W4Args& a, const W4Adapt& d, const AdaptPlan& p, hipStream_t stream) {
  char* ws = (char*)a.ws;
  OrderArgs o{};
  o.A = (const uint16_t*)d.A;
  o.B = (const uint16_t*)d.B;
  o.At = (uint16_t*)(ws + p.off_At);
  o.Bt = (uint16_t*)(ws + p.off_Bt);
  o.ids = d.ids;
  o.order = (int32_t*)(ws + p.off_order);
  o.start = (int32_t*)(ws + p.off_start);
  o.N = (int)a.N;
  o.K = (int)a.K;
  o.O = (int)a.O;
  o.ldb = p.ldb;
  o.count = d.count;
  o.rank = d.rank;
  const int64_t blocks = d.count * (1 + (a.K + 63) / 64 + (p.ldb + 63) / 64);
  hipLaunchKernelGGL(k_adapt_order, dim3((unsigned)blocks), dim3(kOrder), 0, stream, o);
  LowArgs l{};
  l.X = (const uint16_t*)a.in0;
  l.A = o.Bt;
  l.ids = d.ids;
  l.scale = d.scale;
  l.low = (float*)(ws + p.off_low);
  l.scaled = 1;
  l.parts = (uint16_t*)(ws + p.off_parts);
  l.up = a.type == kF16 ? (int*)(ws + p.off_up) : nullptr;
  l.N = (int)a.N;
  l.K = (int)a.O;
  l.lda = p.ldb;
  l.count = d.count;
  l.rank = d.rank;
  l.width = p.width;
  l.nparts = p.nparts;
  l.splits = 1;
  hipError_t e = launch_low<T, false>(l, stream);
  if (e != hipSuccess) return e;
  Adapters ad{};
  ad.ids = d.ids;
  ad.mat = (const char*)o.At;
  ad.parts = (const char*)l.parts;
  ad.up = l.up;
  ad.count = d.count;
  ad.rank = d.rank;
  ad.width = p.width;
  ad.nparts = p.nparts;
  e = launch_w4_input_grad_adapted(a, ad, stream);
  if (e != hipSuccess) return e;
  GradArgs g{};
  g.X = (const uint16_t*)a.in1;
  g.dY = (const uint16_t*)a.in0;
  g.v = l.low;
  g.low = d.low;
  g.scale = d.scale;
  g.order = o.order;
  g.start = o.start;
  g.dA = d.dA;
  g.dB = d.dB;
  g.pA = (float*)(ws + p.off_pA);
  g.pB = (float*)(ws + p.off_pB);
  g.N = (int)a.N;
  g.K = (int)a.K;
  g.O = (int)a.O;
  g.count = d.count;
  g.rank = d.rank;
  g.chunk = p.chunk;
  auto go = [&](auto* kernel, int rt, int z) {
    const int lds = 2 * 16 * rt * (kGradCols + 4) * 4;
    if (lds > 65536) {
      const hipError_t e =
          hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)(a.K / kGradCols + (a.O + kGradCols - 1) / kGradCols), p.units, z);
    hipLaunchKernelGGL(kernel, grid, dim3(64 * kGradWaves), lds, stream, g);
    return hipGetLastError();
  };
  e = d.rank <= 16   ? go(&k_adapt_grad<T, 1>, 1, 1)
      : d.rank <= 32 ? go(&k_adapt_grad<T, 2>, 2, 1)
                     : go(&k_adapt_grad<T, 4>, 4, d.rank > 64 ? 2 : 1);
  if (e != hipSuccess) return e;
  const int64_t quads = d.rank * (a.K + a.O) / 4;
  hipLaunchKernelGGL(k_adapt_join, dim3((unsigned)((quads + 255) / 256), d.count), dim3(256), 0, stream,
                     g);
  return hipGetLastError();
}

hipError_t launch_w4_adapt(const W4Args& a, const W4Adapt& d, bool back, hipStream_t stream) {
  const AdaptPlan p = adapt_plan(a, d, back);
  if (back) return a.type == kF16 ? backward<_Float16>(a, d, p, stream) : backward<__bf16>(a, d, p, stream);
  return a.type == kF16 ? forward<_Float16>(a, d, p, stream) : forward<__bf16>(a, d, p, stream);
}

}  // namespace awq
