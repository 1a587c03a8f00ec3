// Gradients of a packed layer's steps and zeros: D = dY^T X is formed tile by
// tile and only its weighted sums over each group leave the chip,
//   dstep[o, g] = sum_{k in g} D[o, k] (q[o, k] - z[o, g])
//   dzero[o, g] = -step[o, g] sum_{k in g} D[o, k].
//
// Block tile 256 packed rows x 256 columns, eight wavefronts as 4 x 2, each
// 64 x 128 as 4 x 8 tiles of the 16x16x32 MFMA, 64 tokens a step.  Both
// operands lie with the token as the slow index, the MFMA wants eight
// consecutive tokens per lane: tiles move to LDS as they lie (direct loads,
// 512-byte rows) and fragments are read with the transposing LDS read, four
// tokens at a time.  The 32-byte piece u of token t's row sits at
// u ^ (t % 4 + 4 (t / 8 % 2)), so the eight row pieces of half a wavefront's
// read lie in different banks.
// Epilogue: 16 rows at a time through the wavefront's own LDS, each lane then
// takes 32 columns of a row with their four words of codes.  q - z is formed in
// fp32, for any fp16 zero.
// The result is linear in D, so a split tile's parts are split over tokens and
// write their group sums, 256 x groups pairs, which a second launch adds.
// Bound by MFMA issue: 4096 tokens, 13824 -> 5120, 0.49-0.52 ms over the cards
// measured (1.12-1.18 PFLOP/s); 512 tokens, 4096 x 4096, 22-24 us, eight steps
// between prologue and epilogue.
#include "w4_internal.h"

namespace awq {

constexpr int kPgXS = 3, kPgWS = 2;       // LDS stages of dY and X
constexpr int kPgTile = 64 * 256;         // halfs of a stage
constexpr int kPgEpRow = 132;             // floats per row in the epilogue
constexpr int kPgLds = (kPgXS + kPgWS) * kPgTile * 2;

typedef short short4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint2 read_tr(const _Float16* p) {
  const short4v v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) short4v*)(uint32_t)(uintptr_t)p);
  return __builtin_bit_cast(uint2, v);
}

template <typename T, int GROUP>
__global__ void __launch_bounds__(512, 2)
k_w4_param_grad(const _Float16* __restrict__ dY, int ldy, const _Float16* __restrict__ X, int N,
                int K, int O, const uint32_t* __restrict__ qw, const _Float16* __restrict__ step16,
                const _Float16* __restrict__ zero16, float* __restrict__ dstep,
                float* __restrict__ dzero, float* __restrict__ parts, TileSplit sp) {
  constexpr int MT = 4, NT = 8, LOADS = 4;
  constexpr int GT = 256 / GROUP;  // groups of a tile
  extern __shared__ __attribute__((aligned(16))) _Float16 sm[];
  _Float16* const sa = sm;
  _Float16* const sb = sm + kPgXS * kPgTile;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r16 = lane & 15, q4 = lane >> 4;
  const SplitUnit un = split_unit(blockIdx.x, sp);
  const int o0 = un.t * 256, k0 = un.o * 256;

  // load i of a wavefront: two tokens' rows of 512 bytes; pieces past the
  // row's end repeat the first
  uint32_t oa[LOADS], ob[LOADS];
  int tr[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int t = 2 * (wave * LOADS + i) + (lane >> 5);
    const int piece = (lane & 31) ^ (2 * ((t & 3) + 4 * ((t >> 3) & 1)));
    tr[i] = t;
    oa[i] = o0 + 8 * piece < ldy ? 16u * piece : 0u;
    ob[i] = k0 + 8 * piece < K ? 16u * piece : 0u;
  }
  auto load_y = [&](int s) {
    const uint32_t l = (uint32_t)(uintptr_t)(sa + (s % kPgXS) * kPgTile);
    const char* base = (const char*)(dY + (size_t)64 * s * ldy + o0);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const uint32_t t = (uint32_t)min(tr[i], N - 1 - 64 * s);
      dma16(base, t * (uint32_t)ldy * 2 + oa[i], l + (wave * LOADS + i) * 1024);
    }
  };
  auto load_x = [&](int s) {
    const uint32_t l = (uint32_t)(uintptr_t)(sb + (s % kPgWS) * kPgTile);
    const char* base = (const char*)(X + (size_t)64 * s * K + k0);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const uint32_t t = (uint32_t)min(tr[i], N - 1 - 64 * s);
      dma16(base, t * (uint32_t)K * 2 + ob[i], l + (wave * LOADS + i) * 1024);
    }
  };
  // fragment of 16 rows (columns) from c, 32 tokens of half h: lane l gives
  // the place of token 8 q + (l % 16) / 4 (+ 4), four values at 4 (l % 4)
  const int ft = 8 * q4 + (r16 >> 2);
  const int fx = (r16 >> 2) + 4 * (q4 & 1);  // the row's swizzle
  auto frag = [&](const _Float16* stage, int c, int h) -> uint4 {
    const _Float16* p = stage + (32 * h + ft) * 256 + 16 * ((c >> 4) ^ fx) + 4 * (r16 & 3);
    const uint2 a = read_tr(p), b = read_tr(p + 4 * 256);
    return make_uint4(a.x, a.y, b.x, b.y);
  };
  floatx4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  load_y(un.s0);
  load_x(un.s0);
  if (un.s0 + 1 < un.s1) load_y(un.s0 + 1);
  uint4 a0[MT], b0[NT], a1[MT], b1[NT];
  for (int s = un.s0; s < un.s1; ++s) {
    // this step's tiles have landed (dY's of the next step, issued last, may
    // be in flight), and no wavefront still reads the stages loaded next
    if (s + 1 < un.s1)
      wait_vm<LOADS>();
    else
      wait_vm<0>();
    __syncthreads();
    _Float16* ta = sa + (s % kPgXS) * kPgTile;
    _Float16* tb = sb + (s % kPgWS) * kPgTile;
    if (64 * s + 64 > N) {
      // tokens past the last one count as zero in both operands
      for (int e = tid; e < 64 * 32; e += 512)
        if (64 * s + (e >> 5) >= N) {
          *(uint4*)(ta + 8 * e) = make_uint4(0, 0, 0, 0);
          *(uint4*)(tb + 8 * e) = make_uint4(0, 0, 0, 0);
        }
      __syncthreads();
    }
    if (s + 1 < un.s1) load_x(s + 1);
#pragma unroll
    for (int m = 0; m < MT; ++m) a0[m] = frag(ta, wm * 64 + m * 16, 0);
#pragma unroll
    for (int n = 0; n < NT; ++n) b0[n] = frag(tb, wn * 128 + n * 16, 0);
#pragma unroll
    for (int m = 0; m < MT; ++m) a1[m] = frag(ta, wm * 64 + m * 16, 1);
#pragma unroll
    for (int n = 0; n < NT; ++n) b1[n] = frag(tb, wn * 128 + n * 16, 1);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = mfma16<T>(a0[m], b0[n], acc[m][n]);
    if (s + 2 < un.s1) {
      __builtin_amdgcn_sched_barrier(0);
      load_y(s + 2);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = mfma16<T>(a1[m], b1[n], acc[m][n]);
  }
  __syncthreads();

  // register r of lane l is row 4 (l / 16) + r, column l % 16 of its tile
  float* const ep = (float*)sm + wave * 16 * kPgEpRow;
  const int er = lane >> 2, ec = 32 * (lane & 3);
  const int kc = k0 + wn * 128 + ec;
  const int ng = K / GROUP;
  const int g = kc / GROUP;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int o = o0 + wm * 64 + m * 16 + er;
    const bool live = o < O && kc < K;
    uint4 w = make_uint4(0, 0, 0, 0);
    float z = 0.0f;
    if (live) {
      w = *(const uint4*)(qw + (size_t)o * (K >> 3) + (kc >> 3));
      z = (float)zero16[(size_t)o * ng + g];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) ep[(4 * q4 + r) * kPgEpRow + 16 * n + r16] = acc[m][n][r];
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the wavefront's own writes
    asm volatile("" ::: "memory");
    float ds = 0.0f, dz = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 lo = *(const float4*)(ep + er * kPgEpRow + ec + 8 * j);
      const float4 hi = *(const float4*)(ep + er * kPgEpRow + ec + 8 * j + 4);
      // even columns' codes in the bytes of one word, odd ones' in the other's
      const uint32_t even = word_of(w, j) & 0x0F0F0F0Fu, odd = (word_of(w, j) >> 4) & 0x0F0F0F0Fu;
      auto diff = [&](uint32_t codes, int b) { return (float)((codes >> (8 * b)) & 0xffu) - z; };
      ds = fmaf(diff(even, 0), lo.x, ds);
      ds = fmaf(diff(odd, 0), lo.y, ds);
      ds = fmaf(diff(even, 1), lo.z, ds);
      ds = fmaf(diff(odd, 1), lo.w, ds);
      ds = fmaf(diff(even, 2), hi.x, ds);
      ds = fmaf(diff(odd, 2), hi.y, ds);
      ds = fmaf(diff(even, 3), hi.z, ds);
      ds = fmaf(diff(odd, 3), hi.w, ds);
      dz += ((lo.x + lo.y) + (lo.z + lo.w)) + ((hi.x + hi.y) + (hi.z + hi.w));
    }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int d = 1; d < GROUP / 32; d *= 2) {
      ds += __shfl_xor(ds, d, 64);
      dz += __shfl_xor(dz, d, 64);
    }
    if (!live || (lane & (GROUP / 32 - 1))) continue;
    if (un.parts > 1) {
      float* p = parts + ((size_t)un.slot * 256 + wm * 64 + m * 16 + er) * (2 * GT) +
                 2 * ((wn * 128 + ec) / GROUP);
      p[0] = ds;
      p[1] = dz;
    } else {
      const size_t at = (size_t)o * ng + g;
      dstep[at] = ds;
      dzero[at] = -(float)step16[at] * dz;
    }
  }
}

// Sums of the split tiles' parts, in order.
template <int GROUP>
__global__ void __launch_bounds__(256)
k_param_join(const float* __restrict__ parts, int K, int O, const _Float16* __restrict__ step16,
             float* __restrict__ dstep, float* __restrict__ dzero, TileSplit sp) {
  constexpr int GT = 256 / GROUP;
  const int left = blockIdx.x / GT, e = (blockIdx.x % GT) * 256 + threadIdx.x;
  const TileUnit un = tile_unit(sp.full + left, sp.nt, sp.no, sp.full + sp.left);
  const int row = e / GT, o = un.t * 256 + row;
  const int ng = K / GROUP, g = un.o * GT + e % GT;
  if (o >= O || g >= ng) return;
  const float2* p = (const float2*)parts + ((size_t)left * sp.parts * 256 + row) * GT + e % GT;
  float2 s = p[0];
  for (int i = 1; i < sp.parts; ++i) {
    const float2 v = p[(size_t)i * 256 * GT];
    s.x += v.x;
    s.y += v.y;
  }
  const size_t at = (size_t)o * ng + g;
  dstep[at] = s.x;
  dzero[at] = -(float)step16[at] * s.y;
}

struct PgPlan {
  bool copy;
  int ldy;
  TileSplit sp;
  size_t off_y, off_parts, bytes;
};
static PgPlan pg_plan(const W4Args& a) {
  PgPlan p;
  p.copy = a.O % 8 != 0;
  p.ldy = (int)((a.O + 7) / 8 * 8);
  // the tiles of a last, partial round are split over tokens into parts that
  // fill the chip; their sums are small
  const int steps = (int)((a.N + 63) / 64);
  TileSplit s{(int)((a.O + 255) / 256), (int)((a.K + 255) / 256), steps, 0, 0, 1};
  const int total = s.nt * s.no, left = total % kCUs;
  if (left) s.parts = kCUs / left < steps / 2 ? kCUs / left : steps / 2;
  if (s.parts < 2) s.parts = 1;
  if (s.parts > 1) s.left = left;
  s.full = total - s.left;
  p.sp = s;
  size_t at = 0;
  p.off_y = at;
  if (p.copy) at += align256((size_t)a.N * p.ldy * 2);
  p.off_parts = at;
  if (p.sp.parts > 1) at += (size_t)p.sp.left * p.sp.parts * 256 * (256 / a.group) * 8;
  p.bytes = at;
  return p;
}
size_t w4_param_grad_workspace(const W4Args& a) { return pg_plan(a).bytes; }

template <typename T, int GROUP>
static hipError_t launch(const W4Args& a, const PgPlan& p, hipStream_t stream) {
  auto* kernel = &k_w4_param_grad<T, GROUP>;
  const hipError_t e =
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kPgLds);
  if (e != hipSuccess) return e;
  char* ws = (char*)a.ws;
  float* parts = (float*)(ws + p.off_parts);
  const _Float16* st = (const _Float16*)a.step16;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(p.sp.full + p.sp.left * p.sp.parts)), dim3(512), kPgLds,
                     stream, (const _Float16*)(p.copy ? ws + p.off_y : a.in0), p.ldy,
                     (const _Float16*)a.in1, (int)a.N, (int)a.K, (int)a.O,
                     (const uint32_t*)a.qweight, st, (const _Float16*)a.zero16, (float*)a.out0,
                     (float*)a.out1, parts, p.sp);
  if (p.sp.parts > 1)
    hipLaunchKernelGGL(k_param_join<GROUP>, dim3((unsigned)(p.sp.left * (256 / GROUP))), dim3(256), 0,
                       stream, parts, (int)a.K, (int)a.O, st, (float*)a.out0, (float*)a.out1, p.sp);
  return hipGetLastError();
}

template <typename T>
static hipError_t by_group(const W4Args& a, const PgPlan& p, hipStream_t stream) {
  if (a.group == 128) return launch<T, 128>(a, p, stream);
  if (a.group == 64) return launch<T, 64>(a, p, stream);
  return launch<T, 32>(a, p, stream);
}

hipError_t launch_w4_param_grad(const W4Args& a, hipStream_t stream) {
  const PgPlan p = pg_plan(a);
  char* ws = (char*)a.ws;
  if (p.copy) {
    // the bits as they are, rows padded to whole 16-byte pieces
    Prepare q{};
    q.in0 = a.in0;
    q.cols = (int)a.O;
    q.ld_out = p.ldy;
    q.out = ws + p.off_y;
    const hipError_t e = launch_w4_prepare(q, kF16, 0, false, a.N, stream);
    if (e != hipSuccess) return e;
  }
  return a.type == kF16 ? by_group<_Float16>(a, p, stream) : by_group<__bf16>(a, p, stream);
}

}  // namespace awq
