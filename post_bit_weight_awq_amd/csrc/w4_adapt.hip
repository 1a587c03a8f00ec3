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
//                  and low: the left side's fp32 values as sums of 16-bit parts
//                  (k_adapt_left), the right side transposed in registers; a long
//                  list of tokens is taken in chunks, k_adapt_join adds them in
//                  order
#include "w4_adapt.h"

namespace awq {

constexpr int kOrder = 256;

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

template <typename T, int MT, int RT, int U, bool FULL>
__global__ void __launch_bounds__(64 * kLowWaves)
k_adapt_low(LowArgs a) {
  extern __shared__ float red[];  // [wavefront][16][16 RT + 1]
  sum_low<T, MT, RT, U, false, FULL>(a, red, blockIdx.x, blockIdx.y, 0, 0);
}

// A wavefront per token: the pieces' sums in order, as `out` (times the scale
// where `scaled`) and, times the scale, as parts.
template <typename T>
__global__ void __launch_bounds__(256)
k_adapt_parts(LowArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.N) return;
  int id = a.ids[t];
  if (id >= a.count) id = -1;
  const float scale = id < 0 ? 0.0f : a.scale[id];
  float v[2] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = lane + 64 * j;
    if (r >= a.rank) continue;
    const float* p = a.low + (size_t)t * a.rank + r;
    float s = 0.0f;
    for (int k = 0; k < a.splits; k += 4) {
      float y[4];  // past the end the last one, not added
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = p[(size_t)min(k + i, a.splits - 1) * a.N * a.rank];
#pragma unroll
      for (int i = 0; i < 4; ++i) s += k + i < a.splits ? y[i] : 0.0f;
    }
    v[j] = id < 0 ? 0.0f : s;
    if (a.out) a.out[(size_t)t * a.rank + r] = a.scaled ? v[j] * scale : v[j];
    v[j] *= scale;
  }
  uint16_t* p = a.parts + (int64_t)t * a.width;
  if constexpr (__is_same(T, _Float16)) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) top = fmaxf(top, fabsf(v[i]) < INFINITY ? fabsf(v[i]) : 0.0f);
#pragma unroll
    for (int s = 1; s < 64; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
    const int e = up_of(top);
    if (lane == 0) a.up[t] = e;
    v[0] = ldexpf(v[0], -e);
    v[1] = ldexpf(v[1], -e);
  }
  uint16_t h[2][3];
  split_parts<T>(v[0], h[0]);
  split_parts<T>(v[1], h[1]);
  for (int i = 0; i < a.nparts; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (lane + 64 * j < a.rank) p[i * a.rank + lane + 64 * j] = i == 0 ? h[j][0] : i == 1 ? h[j][1] : h[j][2];
  const int end = a.nparts * a.rank;  // less than 32 zeros
  if (lane < a.width - end) p[end + lane] = 0;
}

// Token tiles of the sum of low: 64 high where the ranks' registers allow it and
// there are enough tokens, and pieces of at least 512 columns until each unit has
// a block.
struct LowPlan {
  int mt, splits;
};
static LowPlan low_plan(int64_t N, int64_t K, int rank) {
  LowPlan p;
  p.mt = N <= 128 ? 1 : rank > 64 || N <= 512 ? 2 : 4;
  const int64_t tiles = (N + 16 * p.mt - 1) / (16 * p.mt);
  int64_t n = kCUs / tiles;
  if (n > K / 512) n = K / 512;
  p.splits = (int)(n < 1 ? 1 : n > 8 ? 8 : n);
  return p;
}

template <typename T, bool FULL>
static hipError_t launch_low(const LowArgs& a, int mt, hipStream_t stream) {
  constexpr int U = FULL ? 2 : 1;
  const int rt = (a.rank + 15) / 16;
  auto go = [&](auto* kernel, int r) {
    const int lds = kLowWaves * 16 * (16 * r + 1) * 4;
    if (lds > 65536) {
      const hipError_t e =
          hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
    }
    const dim3 grid(a.splits, (unsigned)((a.N + 16 * mt - 1) / (16 * mt)));
    hipLaunchKernelGGL(kernel, grid, dim3(64 * kLowWaves), lds, stream, a);
    return hipGetLastError();
  };
  if (mt == 4) {
    if (rt == 1) return go(&k_adapt_low<T, 4, 1, U, FULL>, 1);
    if (rt == 2) return go(&k_adapt_low<T, 4, 2, U, FULL>, 2);
    return go(&k_adapt_low<T, 4, 4, U, FULL>, 4);
  }
  if (mt == 2) {
    if (rt == 1) return go(&k_adapt_low<T, 2, 1, U, FULL>, 1);
    if (rt == 2) return go(&k_adapt_low<T, 2, 2, U, FULL>, 2);
    if (rt <= 4) return go(&k_adapt_low<T, 2, 4, U, FULL>, 4);
    return go(&k_adapt_low<T, 2, 8, 1, FULL>, 8);
  }
  if (rt == 1) return go(&k_adapt_low<T, 1, 1, U, FULL>, 1);
  if (rt == 2) return go(&k_adapt_low<T, 1, 2, U, FULL>, 2);
  if (rt <= 4) return go(&k_adapt_low<T, 1, 4, U, FULL>, 4);
  return go(&k_adapt_low<T, 1, 8, U, FULL>, 8);
}
template <typename T, bool FULL>
static hipError_t launch_parts(const LowArgs& a, int mt, hipStream_t stream) {
  const hipError_t e = launch_low<T, FULL>(a, mt, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_adapt_parts<T>), dim3((unsigned)((a.N + 3) / 4)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// Single tokens: y = round(base + scale low B[a]^T), base the streaming product's
// sums in fp32.  A block takes one token, a wavefront 64 outputs, whose rows of
// B[a] lie one behind the other: a team of lanes takes a row, eight ranks each.
// Bound by latency and the read of B.  In the streaming kernel's epilogue, whose
// few blocks have to read all of it, the second term cost 48 tokens, 13824 ->
// 5120, 25 adapters of rank 64, 28 us; here it takes 7.6.
struct AddArgs {
  const float *base, *low, *scale;  // low: [splits, N, rank]
  const int32_t* ids;
  const char* mat;  // [count, O, rank]
  void* y;
  float* out;  // low, kept, or NULL
  int N, O, count, rank, splits, y_type;
};
template <typename T>
__global__ void __launch_bounds__(256)
k_adapt_add(AddArgs a) {
  __shared__ float low[128], sums[4][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t = blockIdx.y, o0 = 64 * (4 * blockIdx.x + wave);
  int id = a.ids[t];
  if (id >= a.count) id = -1;
  const int o = o0 + lane;
  float v = o < a.O ? a.base[(size_t)t * a.O + o] : 0.0f;
  if (tid < a.rank) {
    float s = 0.0f;
    if (id >= 0) {
      float x[8];  // past the end the last piece's, not added
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = a.low[((size_t)min(k, a.splits - 1) * a.N + t) * a.rank + tid];
#pragma unroll
      for (int k = 0; k < 8; ++k) s += k < a.splits ? x[k] : 0.0f;
    }
    if (a.out && blockIdx.x == 0) a.out[(size_t)t * a.rank + tid] = s;
    low[tid] = id >= 0 ? s * a.scale[id] : 0.0f;
  }
  __syncthreads();
  if (o0 >= a.O) return;
  if (id >= 0) {
    const int rb = a.rank >> 3, rows = min(64, a.O - o0);
    int team = 1;
    while (team < rb) team *= 2;
    const int part = lane & (team - 1), first = lane / team, step = 64 / team;
    const char* b = a.mat + ((int64_t)id * a.O + o0) * a.rank * 2 + 16 * min(part, rb - 1);
    float u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = part < rb ? low[8 * part + k] : 0.0f;
    for (int i0 = 0; i0 < 64; i0 += 4 * step) {
      uint4 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = *(const uint4*)(b + (int64_t)min(i0 + j * step + first, rows - 1) * a.rank * 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * step + first;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          s = fmaf(u[k], to_f32(__builtin_bit_cast(T, (uint16_t)(word_of(w[j], k >> 1) >> (16 * (k & 1))))), s);
        s = part < rb ? s : 0.0f;
        for (int k = 1; k < team; k *= 2) s += __shfl_xor(s, k);
        if (part == 0 && i < 64) sums[wave][i] = s;
      }
    }
    // the wavefront's own writes
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    v += sums[wave][lane];
  }
  if (o >= a.O) return;
  if (a.y_type == kF32)
    ((float*)a.y)[(size_t)t * a.O + o] = v;
  else
    ((T*)a.y)[(size_t)t * a.O + o] = from_f32<T>(v);
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
  constexpr int kTileRow = 136;
  __shared__ __attribute__((aligned(16))) uint16_t tile[64 * kTileRow];
  __shared__ int wsum[kOrder / 64][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t block = grid_block();
  if (block < (uint32_t)a.count) {
    const int me = block;
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
  const int ka = a.K / 64, kb = (a.ldb + 63) / 64, rb = a.rank >> 3;
  const int64_t id = (int64_t)block - a.count;
  const int which = (int)(id % (ka + kb));
  const int64_t ad = id / (ka + kb);
  if (ad >= a.count) return;
  if (which < ka) {
    const int c0 = 64 * which;
    const uint16_t* s = a.A + ad * a.rank * a.K + c0;
    for (int e = tid; e < 8 * a.rank; e += kOrder) {  // eight columns of a rank
      const int r = e >> 3, c = 8 * (e & 7);
      const uint4 v = *(const uint4*)(s + (int64_t)r * a.K + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) tile[(c + i) * kTileRow + r] = (uint16_t)(word_of(v, i >> 1) >> (16 * (i & 1)));
    }
    __syncthreads();
    uint4* d = (uint4*)(a.At + (ad * a.K + c0) * a.rank);
    for (int e = tid; e < 64 * rb; e += kOrder) d[e] = *(const uint4*)(tile + (e / rb) * kTileRow + 8 * (e % rb));
  } else {
    const int o0 = 64 * (which - ka);
    const uint4* s = (const uint4*)(a.B + (ad * a.O + o0) * a.rank);
    for (int e = tid; e < 64 * rb; e += kOrder)
      *(uint4*)(tile + (e / rb) * kTileRow + 8 * (e % rb)) = o0 + e / rb < a.O ? s[e] : make_uint4(0, 0, 0, 0);
    __syncthreads();
    uint16_t* d = a.Bt + ad * a.rank * a.ldb + o0;
    for (int e = tid; e < 8 * a.rank; e += kOrder) {  // eight rows of a rank
      const int r = e >> 3, o = 8 * (e & 7);
      if (o0 + o >= a.ldb) continue;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = tile[(o + 2 * i) * kTileRow + r] | (uint32_t)tile[(o + 2 * i + 1) * kTileRow + r] << 16;
      *(uint4*)(d + (int64_t)r * a.ldb + o) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

struct GradArgs {
  const uint16_t *X, *dY;
  const float *v, *low, *scale;  // [N, rank]
  const int32_t *order, *start;
  uint16_t* left;  // [v, low][part][ranks][stride]: see k_adapt_left
  int* up;         // [unit][v, low][ranks], fp16
  float *dA, *dB;  // [count][rank][K], [count][O][rank]
  float *pA, *pB;  // of the units of adapters with more than one: part_of
  int64_t stride;
  int N, K, O, count, rank, ranks, chunk;  // ranks: rounded up to 16
};
// Unit u: adapter a owns the units from start[a] / chunk + a on.
__device__ __forceinline__ int unit_base(const GradArgs& g, int a) { return g.start[a] / g.chunk + a; }
// An adapter of c >= chunk tokens finds room for its ceil(c / chunk) units'
// sums: floor(2 c / chunk) is as many at least.
__device__ __forceinline__ int64_t part_of(const GradArgs& g, int a) { return 2 * (int64_t)g.start[a] / g.chunk; }
// The tokens p0 .. p1 - 1 of a unit in `order`; false where it has none.
struct GradUnit {
  int a, p0, p1, all;  // all: the adapter's tokens
  int piece;           // of them
};
__device__ __forceinline__ bool grad_unit(const GradArgs& g, int unit, GradUnit* u) {
  int a = 0, hi = g.count;  // unit_base(a) <= unit < unit_base(hi)
  while (hi - a > 1) {
    const int mid = (a + hi) >> 1;
    if (unit_base(g, mid) <= unit)
      a = mid;
    else
      hi = mid;
  }
  const int begin = g.start[a], end = g.start[a + 1];
  u->a = a;
  u->all = end - begin;
  u->piece = unit - unit_base(g, a);
  u->p0 = begin + u->piece * g.chunk;
  u->p1 = min(u->p0 + g.chunk, end);
  return u->p0 < end;
}
// Place of a unit's first token in the rows of `left`: adapters begin on 16 bytes.
__device__ __forceinline__ int64_t left_place(const GradArgs& g, const GradUnit& u) {
  return ((g.start[u.a] + 7) & ~7) + 8 * (int64_t)u.a + (int64_t)u.piece * g.chunk;
}

template <typename T>
constexpr int kLeftParts = __is_same(T, _Float16) ? 2 : 3;

// The left operands of the gradients once instead of in every block: v and low of
// a unit's tokens as 16-bit parts, a rank's tokens in a row.  fp16's are in units
// of the largest of the rank's tokens, which every block of 64 tokens looks for in its
// whole unit by itself: that costs no launch and nothing at 4096 tokens (5 us), but units
// grow with the tokens, so it grows with their square (65536 tokens, 5120 <- 5120, rank
// 64: 174 us of 4.7 ms, bf16 21).
template <typename T>
__global__ void __launch_bounds__(256)
k_adapt_left(GradArgs g) {
  constexpr int P = kLeftParts<T>;
  __shared__ float tile[16][68];
  __shared__ float tops[16][17];
  const int tid = threadIdx.x;
  const int unit = blockIdx.x, side = blockIdx.y & 1, r0 = 16 * (blockIdx.y >> 1);
  GradUnit u;
  if (!grad_unit(g, unit, &u)) return;
  const float* L = side ? g.low : g.v;
  const int ti = tid >> 2, tr = 4 * (tid & 3);  // one of 64 tokens, four ranks
  auto load = [&](int at) {  // of token p0 + at
    floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (u.p0 + at < u.p1 && r0 + tr < g.rank) v = *(const floatx4*)(L + (int64_t)g.order[u.p0 + at] * g.rank + r0 + tr);
    return v;
  };
  const int r = tid >> 4, i4 = 4 * (tid & 15);  // a rank, four tokens
  int e = 0;
  if constexpr (__is_same(T, _Float16)) {
    float top[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int at = ti; u.p0 + at < u.p1; at += 64) {
      const floatx4 v = load(at);
#pragma unroll
      for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], fabsf(v[i]) < INFINITY ? fabsf(v[i]) : 0.0f);
    }
    // of the 16 tokens that a wavefront has, then of the wavefronts
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int s = 4; s < 64; s *= 2) top[i] = fmaxf(top[i], __shfl_xor(top[i], s));
      if ((tid & 60) == 0) tops[tr + i][tid >> 6] = top[i];
    }
    __syncthreads();
    e = up_of(fmaxf(fmaxf(tops[r][0], tops[r][1]), fmaxf(tops[r][2], tops[r][3])));
    if (blockIdx.z == 0 && i4 == 0) g.up[(unit * 2 + side) * g.ranks + r0 + r] = e;
  }
  uint16_t* d = g.left + ((int64_t)side * P * g.ranks + r0 + r) * g.stride + left_place(g, u);
  const int n = u.p1 - u.p0;
  const int b = 64 * blockIdx.z;
  const floatx4 v = load(b + ti);
#pragma unroll
  for (int i = 0; i < 4; ++i) tile[tr + i][ti] = v[i];
  __syncthreads();
  uint16_t h[4][P];
#pragma unroll
  for (int i = 0; i < 4; ++i) split_parts<T>(ldexpf(tile[r][i4 + i], -e), h[i]);
  // up to seven places behind the last token are this adapter's too
  if (b + i4 < n)
#pragma unroll
    for (int p = 0; p < P; ++p)
      *(uint2*)(d + (int64_t)p * g.ranks * g.stride + b + i4) =
          make_uint2(h[0][p] | (uint32_t)h[1][p] << 16, h[2][p] | (uint32_t)h[3][p] << 16);
}

constexpr int kGradWaves = 4, kGradCols = 128;

// 16 RT ranks from 64 z on by 4 x 128 columns of X, then of dY, all tokens of a
// unit, 32 at a time.  A wavefront takes 128 columns; the left operands' fragments
// come through LDS, each wavefront brings a quarter of them by direct loads: a
// compute unit gets about 30 bytes a ns from L2, and read by each wavefront they
// were 60 % of that (4096 tokens, 5120 and 15360 columns, rank 64: 92 us instead of
// 72; with the tokens divided among the wavefronts and their sums added
// through LDS, 95).  The next step's operands are on the way while one is used.
template <typename T, int RT>
__global__ void __launch_bounds__(64 * kGradWaves, 2)
k_adapt_grad(GradArgs g) {
  constexpr int P = kLeftParts<T>, F = RT * P;
  __shared__ __attribute__((aligned(16))) char smem[2 * F * 1024];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int unit = blockIdx.y, r0 = 64 * blockIdx.z;
  GradUnit u;
  if (!grad_unit(g, unit, &u)) return;
  const int ba = (g.K / kGradCols + kGradWaves - 1) / kGradWaves;
  const bool right = (int)blockIdx.x >= ba;  // dB
  const int C = right ? g.O : g.K;
  const int c0 = kGradCols * (kGradWaves * (blockIdx.x - (right ? ba : 0)) + wave);
  const bool live = c0 < C;  // else it only brings its fragments
  const uint16_t* Y = (right ? g.dY : g.X) + (live ? c0 + 8 * r16 : 0);
  const char* L = (const char*)(g.left + ((int64_t)right * P * g.ranks + r0) * g.stride + left_place(g, u));
  const uint32_t at = (uint32_t)(r16 * g.stride * 2) + 16 * q4;
  const int m_last = (g.ranks - r0) / 16 - 1;  // tiles of ranks behind it repeat it
  floatx4 acc[RT][8];
#pragma unroll
  for (int m = 0; m < RT; ++m)
#pragma unroll
    for (int n = 0; n < 8; ++n) acc[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const int left = live ? C - c0 - 8 * r16 : 0;  // columns from the lane's first on
  const bool plain = live && C - c0 >= kGradCols && C % 8 == 0;
  int token[8];
  auto tokens = [&](int s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) token[i] = g.order[min(s + 8 * q4 + i, u.p1 - 1)];
  };
  uint4 y[8], yn[8];
  const uint32_t lds = (uint32_t)(uintptr_t)smem;
  auto request = [&](int s, int stage) {
    // fragment f = m P + p
#pragma unroll
    for (int f = 0; f < F; f += kGradWaves)
      if (f + wave < F) {
        const int m = (f + wave) / P, p = (f + wave) % P;
        dma16(L + ((int64_t)(p * g.ranks + 16 * min(m, m_last)) * g.stride + (s - u.p0)) * 2, at,
              lds + stage * F * 1024 + (f + wave) * 1024);
      }
    if (plain) {
#pragma unroll
      for (int i = 0; i < 8; ++i) yn[i] = *(const uint4*)(Y + (int64_t)token[i] * C);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) yn[i] = load8(Y + (int64_t)token[i] * C, left);
    }
  };
  tokens(u.p0);
  request(u.p0, 0);
  if (u.p0 + 32 < u.p1) tokens(u.p0 + 32);
  int stage = 0;
  for (int s = u.p0; s < u.p1; s += 32) {
    // this step's fragments have landed, and nobody reads the other stage
    wait_vm<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = yn[i];
    if (s + 32 < u.p1) request(s + 32, stage ^ 1);
    if (s + 64 < u.p1) tokens(s + 64);
    const char* st = smem + stage * F * 1024 + 16 * lane;
    // behind the unit's last token both sides are 0
    const int n_in = u.p1 - s - 8 * q4;
    const bool edge = s + 32 > u.p1;
    if (edge)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= n_in) y[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      uint4 lp[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        lp[p] = *(const uint4*)(st + (m * P + p) * 1024);
        if (edge) {
          lp[p].x &= 0 >= n_in ? 0u : 1 >= n_in ? 0xffffu : 0xffffffffu;
          lp[p].y &= 2 >= n_in ? 0u : 3 >= n_in ? 0xffffu : 0xffffffffu;
          lp[p].z &= 4 >= n_in ? 0u : 5 >= n_in ? 0xffffu : 0xffffffffu;
          lp[p].w &= 6 >= n_in ? 0u : 7 >= n_in ? 0xffffu : 0xffffffffu;
        }
      }
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const uint32_t sel = n & 1 ? 0x07060302u : 0x05040100u;
        const uint4 b = make_uint4(__builtin_amdgcn_perm(word_of(y[1], n >> 1), word_of(y[0], n >> 1), sel),
                                   __builtin_amdgcn_perm(word_of(y[3], n >> 1), word_of(y[2], n >> 1), sel),
                                   __builtin_amdgcn_perm(word_of(y[5], n >> 1), word_of(y[4], n >> 1), sel),
                                   __builtin_amdgcn_perm(word_of(y[7], n >> 1), word_of(y[6], n >> 1), sel));
#pragma unroll
        for (int p = 0; p < P; ++p) acc[m][n] = mfma16<T>(lp[p], b, acc[m][n]);
      }
    }
    stage ^= 1;
  }
  if (!live) return;
  // tile n, lane l: ranks 4 (l / 16) + r, column 8 (l % 16) + n
  const bool whole = u.all <= g.chunk;
  const float f = right && whole ? g.scale[u.a] : 1.0f;
  const int64_t to = whole ? u.a : part_of(g, u.a) + u.piece;
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    const int r = r0 + 16 * m + 4 * q4;  // four ranks; rank is a multiple of 8
    if (r >= g.rank) continue;
    if (g.up)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int up = g.up[(unit * 2 + right) * g.ranks + r + i];
#pragma unroll
        for (int n = 0; n < 8; ++n) acc[m][n][i] = ldexpf(acc[m][n][i], up);
      }
    if (right) {
      float* d = (whole ? g.dB : g.pB) + (to * g.O + c0 + 8 * r16) * g.rank + r;
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (n < left) *(floatx4*)(d + (int64_t)n * g.rank) = acc[m][n] * f;
    } else {
      float* d = (whole ? g.dA : g.pA) + (to * g.rank + r) * g.K + c0 + 8 * r16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *(floatx4*)(d + (int64_t)i * g.K) = floatx4{acc[m][0][i], acc[m][1][i], acc[m][2][i], acc[m][3][i]};
        *(floatx4*)(d + (int64_t)i * g.K + 4) = floatx4{acc[m][4][i], acc[m][5][i], acc[m][6][i], acc[m][7][i]};
      }
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
  const float* p = (right ? g.pB : g.pA) + part_of(g, a) * n + at;
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
  int mt, splits, width, nparts, ldb, ranks, chunk, units;
  int64_t stride;
  size_t off_low, off_base, off_v, off_parts, off_up, off_At, off_Bt, off_order, off_start, off_left, off_lup, off_pA, off_pB,
      bytes;
};
static AdaptPlan adapt_plan(const W4Args& a, const W4Adapt& d, bool backward) {
  AdaptPlan p{};
  size_t at = backward ? w4_input_grad_workspace(a) : w4_workspace(kOpLinear, a);
  p.skinny = !backward && w4_skinny_fits(a);
  auto take = [&](size_t n) {
    const size_t r = align256(at);
    at = r + n;
    return r;
  };
  p.splits = 1;
  if (p.skinny) {
    // pieces of the sum of at least 256 columns, until each unit has a block of
    // them (they run beside the product's own)
    const int64_t blocks = (a.N + 15) / 16 * (a.N < 16 ? a.N : 16) * ((d.rank + 15) / 16);
    int64_t n = kCUs / blocks, most = a.K / 256;
    n = n > 8 ? 8 : n;
    n = n > most ? most : n;
    p.splits = n < 1 ? 1 : (int)n;
    p.off_low = take((size_t)p.splits * a.N * d.rank * 4);
    p.off_base = take(a.y_type == kF32 ? 0 : (size_t)a.N * a.O * 4);
  } else {
    const LowPlan low = low_plan(a.N, backward ? a.O : a.K, d.rank);
    p.mt = low.mt;
    p.splits = low.splits;
    p.off_low = take((size_t)p.splits * a.N * d.rank * 4);
    p.nparts = a.type == kBF16 && a.y_type == kF32 ? 3 : 2;
    p.width = (p.nparts * d.rank + 31) & ~31;
    p.off_parts = take((size_t)a.N * p.width * 2);
    p.off_up = take((size_t)a.N * 4);
  }
  if (backward) {
    p.ldb = (int)((a.O + 31) & ~(int64_t)31);
    p.off_v = take((size_t)a.N * d.rank * 4);
    p.off_At = take((size_t)d.count * a.K * d.rank * 2);
    p.off_Bt = take((size_t)d.count * p.ldb * d.rank * 2);
    p.off_order = take((size_t)a.N * 4);
    p.off_start = take((size_t)(d.count + 1) * 4);
    // A chunk's sums are written and read in fp32: from eight tokens per rank on
    // they are at most half of what it reads; beyond that two blocks per unit.
    const int64_t tiles = (a.K + a.O + 4 * kGradCols - 1) / (4 * kGradCols) * (d.rank > 64 ? 2 : 1);
    int64_t chunk = a.N * tiles / (2 * kCUs);
    if (chunk < 8 * d.rank) chunk = 8 * d.rank;
    if (chunk > a.N) chunk = a.N;
    p.chunk = (int)((chunk + 63) & ~(int64_t)63);
    p.units = (int)(a.N / p.chunk) + d.count;
    p.ranks = (d.rank + 15) & ~15;
    // the adapters' tokens, each from a multiple of eight on, and what a last
    // step of 32 reads behind them
    p.stride = ((a.N + 7) & ~(int64_t)7) + 8 * (int64_t)d.count + 32;
    p.off_left = take((size_t)6 * p.ranks * p.stride * 2);
    p.off_lup = take((size_t)p.units * 2 * p.ranks * 4);
    const bool many = a.N > p.chunk;  // else no adapter has two chunks
    const size_t parts = many ? 2 * a.N / p.chunk + 1 : 0;
    p.off_pA = take(parts * d.rank * a.K * 4);
    p.off_pB = take(parts * d.rank * a.O * 4);
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
  l.low = (float*)(ws + p.off_low);
  l.out = d.low;
  l.N = (int)a.N;
  l.K = l.lda = (int)a.K;
  l.count = d.count;
  l.rank = d.rank;
  l.splits = p.splits;
  if (p.skinny) {
    LowBlocks low{l, 0, (int)((a.N + 15) / 16), (int)(a.N < 16 ? a.N : 16), (d.rank + 15) / 16};
    W4Args b = a;
    b.y_type = kF32;
    if (a.y_type != kF32) b.out0 = ws + p.off_base;
    const hipError_t e = launch_w4_skinny_low(b, low, stream);
    if (e != hipSuccess) return e;
    const AddArgs add{(const float*)b.out0, l.low, d.scale, d.ids, (const char*)d.B, a.out0, d.low,
                      (int)a.N, (int)a.O, d.count, d.rank, p.splits, a.y_type};
    hipLaunchKernelGGL((k_adapt_add<T>), dim3((unsigned)((a.O + 255) / 256), (unsigned)a.N), dim3(256), 0,
                       stream, add);
    return hipGetLastError();
  }
  Adapters ad{};
  ad.ids = d.ids;
  ad.mat = (const char*)d.B;
  ad.count = d.count;
  ad.rank = d.rank;
  l.parts = (uint16_t*)(ws + p.off_parts);
  l.up = a.type == kF16 ? (int*)(ws + p.off_up) : nullptr;
  l.width = ad.width = p.width;
  l.nparts = ad.nparts = p.nparts;
  ad.parts = (const char*)l.parts;
  ad.up = l.up;
  const hipError_t e = launch_parts<T, true>(l, p.mt, stream);
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
  hipLaunchKernelGGL(k_adapt_order, grid_of(blocks), dim3(kOrder), 0, stream, o);
  LowArgs l{};
  l.X = (const uint16_t*)a.in0;
  l.A = o.Bt;
  l.ids = d.ids;
  l.scale = d.scale;
  l.low = (float*)(ws + p.off_low);
  l.out = (float*)(ws + p.off_v);
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
  l.splits = p.splits;
  hipError_t e = a.O % 32 ? launch_parts<T, false>(l, p.mt, stream) : launch_parts<T, true>(l, p.mt, stream);
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
  g.v = l.out;
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
  g.ranks = p.ranks;
  g.stride = p.stride;
  g.left = (uint16_t*)(ws + p.off_left);
  g.up = a.type == kF16 ? (int*)(ws + p.off_lup) : nullptr;
  hipLaunchKernelGGL((k_adapt_left<T>), dim3(p.units, 2 * p.ranks / 16, p.chunk / 64), dim3(256), 0, stream, g);
  auto go = [&](auto* kernel, int z) {
    const int64_t wide = kGradCols * kGradWaves;
    const dim3 grid((unsigned)((a.K + wide - 1) / wide + (a.O + wide - 1) / wide), p.units, z);
    hipLaunchKernelGGL(kernel, grid, dim3(64 * kGradWaves), 0, stream, g);
    return hipGetLastError();
  };
  e = d.rank <= 16   ? go(&k_adapt_grad<T, 1>, 1)
      : d.rank <= 32 ? go(&k_adapt_grad<T, 2>, 1)
                     : go(&k_adapt_grad<T, 4>, d.rank > 64 ? 2 : 1);
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
