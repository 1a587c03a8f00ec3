// dX = dY W on packed weights: W[o, k] = (q[o, k] - z[o, g]) step[o, g], the
// sum running over the packed rows o.
//
// Block tile of up to 256 tokens x 256 columns, eight wavefronts as 2 x 4
// (columns), each 16 MT x 64 as MT x 4 tiles of v_mfma_f32_16x16x32_f16, 64
// packed rows a step.  For tiles of 192 and 256 tokens the two halves of the
// wavefronts take half of the tokens each; for 64 and 128 both take all, each
// every second step (SPLIT), and add their sums through LDS at the end: a
// wavefront then converts codes for twice as many tokens.  One
// 64- or 128-token tile per unit, 512 x 4096 <- 4096: 53 and 59 us against 67
// and 83 with halved tokens.  dY, the codes and the group parameters move to LDS by
// direct loads, two (codes: three) steps ahead.
//   * An MFMA needs eight consecutive rows of one column per lane, while a
//     word holds eight columns of one row.  So lane l reads the word l % 16 of
//     each of its eight rows (8 (l / 16) ..), pairs the rows' halves with one
//     byte permute, and each nibble position of the pair is the fragment of
//     another column tile: tile c of a wavefront is the columns 8 j + 4 h + c,
//     j = 0..15, h the wavefront's half of the words.  No transpose, and a
//     lane's four tiles are four neighbouring columns of dX.
//   * The step changes along the sum, so it has to enter the operand: weights
//     are formed as fp16((q - z) step), 15 operations per eight.  A block with
//     weights that fp16 may not hold sums in fp32 without the matrix units (512
//     x 4096 <- 4096, all blocks: 0.4 ms against 40 us): no layer that is packed
//     from ordinary weights has one.
//   * The LDS rows of the codes are ordered (row % 8, row / 8) and every
//     second pair swaps its 64-byte halves: the 64 words of a read then lie
//     in 64 banks.
//   * dY in bf16, or of a width that is no multiple of 64, is copied to fp16
//     rows of a padded width first (w4_prepare.hip; zeros behind the row's end
//     meet weights of 0).
// Bound by the issue of MFMAs and conversions: 4096 x 5120 <- 27648 takes
// 0.95-1.03 ms (1.13-1.22 PFLOP/s over the cards measured) of 1.13-1.18 with its
// row scaling, 2048 x 4096 <- 12288 203-222 us of which 27 are the scaling.
#include "w4_internal.h"

namespace awq {

// An iteration is one step, or two (SPLIT), whose operands lie side by side.
// Three stages of dY and four of codes and parameters, three where four do not
// fit.
template <int MT, bool SPLIT>
struct DxLds {
  static constexpr int kA = 32 * MT * 128;            // bytes of dY per stage
  static constexpr int kC = (SPLIT ? 2 : 1) * 64 * 128;  // codes
  static constexpr int kP = (SPLIT ? 2 : 1) * 2048;      // group parameters
  static constexpr int kNC = SPLIT && MT == 8 ? 3 : 4;
  static constexpr int kOffC = 3 * kA, kOffP = kOffC + kNC * kC;
  static constexpr int kBytes = kOffP + kNC * kP;
  static_assert(kBytes <= 160 * 1024);
};

// Values of one token's four neighbouring columns per lane, tile by tile.
template <typename T, int MT>
__device__ __forceinline__ void store_dx(const floatx4 (&acc)[MT][4], const int* back, int N, int K,
                                         int t0, int col, int lane, T* dX) {
  if (col >= K) return;
  typedef T Tx4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = t0 + 16 * m + 4 * (lane >> 4) + r;
      if (t >= N) continue;
      const int x = back ? back[t] : 0;
      Tx4 v;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = from_f32<T>(back ? ldexpf(acc[m][c][r], x) : acc[m][c][r]);
      *(Tx4*)(dX + (size_t)t * K + col) = v;
    }
}

// A part's sums to the workspace as they lie, a whole tile's values to dX.
template <typename T, int MT>
__device__ __forceinline__ void leave(const floatx4 (&acc)[MT][4], float* parts, const SplitUnit& un,
                                      int wave, const int* back, int N, int K, int t0, int col,
                                      int lane, T* dX) {
  if (un.parts > 1) {
    floatx4* p = (floatx4*)parts + ((size_t)un.slot * 8 + wave) * (MT * 4 * 64) + lane;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < 4; ++c) p[(m * 4 + c) * 64] = acc[m][c];
    return;
  }
  store_dx<T, MT>(acc, back, N, K, t0, col, lane, dX);
}

template <typename T, int GROUP, int MT, bool SPLIT>
__global__ void __launch_bounds__(512, 2)
k_w4_dx(const _Float16* __restrict__ A, int lda, const int* __restrict__ back, int N, int K, int O,
        const char* __restrict__ qw, const char* __restrict__ prm, const int* __restrict__ big,
        T* __restrict__ dX, float* __restrict__ parts, TileSplit sp) {
  using L = DxLds<MT, SPLIT>;
  constexpr int BM = (SPLIT ? 16 : 32) * MT;
  constexpr int AL = MT / 2;           // direct loads of dY per wavefront and iteration
  constexpr int CL = SPLIT ? 2 : 1;    // of codes
  constexpr int PB = CL * 8192 / GROUP;  // parameter bytes per wavefront and iteration
  constexpr int PL = PB > 256 ? 2 : 1;   // their loads
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3, wb = wn >> 1, half = wn & 1;
  const int r16 = lane & 15, q4 = lane >> 4;
  const SplitUnit un = split_unit(blockIdx.x, sp);
  const int t0 = un.t * BM, k0 = un.o * 256;
  const int ng = K / GROUP, steps = (O + 63) >> 6;
  // With SPLIT wavefronts 0-3 load and take the even steps, 4-7 the odd ones;
  // an odd one past the end loads the last step, which is not used.
  auto step_of = [&](int it) {
    return SPLIT ? __builtin_amdgcn_readfirstlane(min(2 * it + wm, steps - 1)) : it;
  };
  const int lw = SPLIT ? wn : wave;  // the wavefront among those that load a step

  // dY: load i brings 8 rows of 128 bytes; 16-byte piece p of row r at p ^ (r % 8)
  uint32_t oa[AL];
#pragma unroll
  for (int i = 0; i < AL; ++i) {
    const int r = 8 * (lw * AL + i) + (lane >> 3);
    oa[i] = 2u * ((uint32_t)(min(t0 + r, N - 1) - t0) * (uint32_t)lda + 8 * ((lane & 7) ^ (r & 7)));
  }
  const char* a0 = (const char*)(A + (size_t)t0 * lda);
  // codes: a load brings 8 LDS rows of 128 bytes; LDS row 32 c + 4 i + q is
  // packed row 32 c + 8 q + i of the step
  int crow[CL];
  uint32_t oc[CL];
#pragma unroll
  for (int i = 0; i < CL; ++i) {
    const int lr = 8 * (lw * CL + i) + (lane >> 3);
    crow[i] = 32 * (lr >> 5) + 8 * (lr & 3) + ((lr & 31) >> 2);
    int piece = (lane & 7) ^ (((lr >> 1) & 1) << 2);
    if (k0 + 32 * piece >= K) piece -= 4;  // a last tile of 128 columns
    oc[i] = (uint32_t)(k0 / 2 + 16 * piece);
  }
  // parameters: PB bytes of the block's groups per wavefront
  uint32_t op[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int at = lw * PB + 256 * i + 4 * lane;
    op[i] = (uint32_t)min(k0 / GROUP + at / 256, ng - 1) * 256u + (at & 255);
  }

  const uint32_t lds = (uint32_t)(uintptr_t)smem;
  auto load_a = [&](int it) {
    const char* base = a0 + step_of(it) * 128;
#pragma unroll
    for (int i = 0; i < AL; ++i)
      dma16(base, oa[i], lds + (it % 3) * L::kA + (wave * AL + i) * 1024);
  };
  auto load_c = [&](int it) {
    const int s = step_of(it);
    // each lane's row, the last one where the step passes the end
#pragma unroll
    for (int i = 0; i < CL; ++i)
      dma16(qw + (size_t)(64 * s) * (K / 2),
            (uint32_t)(min(64 * s + crow[i], O - 1) - 64 * s) * (uint32_t)(K / 2) + oc[i],
            lds + L::kOffC + (it % L::kNC) * L::kC + (wave * CL + i) * 1024);
    const char* p = prm + (size_t)s * ng * 256;
    const uint32_t l = lds + L::kOffP + (it % L::kNC) * L::kP + (SPLIT ? wm * 2048 : 0) + lw * PB;
    if (PB >= 256) {
#pragma unroll
      for (int i = 0; i < PL; ++i) dma4(p, op[i], l + 256 * i);
    } else if (lane < PB / 4) {
      dma4(p, op[0], l);
    }
  };

  floatx4 acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[m][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const int cbase = (SPLIT ? wm * 8192 : 0) + q4 * 128 + ((wb ^ (q4 >> 1)) * 64) + 4 * r16;
  const int gl = (128 * wb + 8 * r16) / GROUP;  // the lane's group among the block's
  const uint32_t sel = half ? 0x07060302u : 0x05040100u;

  const int send = un.s1;
  load_c(un.s0);
  load_a(un.s0);
  if (un.s0 + 1 < send) {
    load_c(un.s0 + 1);
    load_a(un.s0 + 1);
  }
  if (L::kNC == 4 && un.s0 + 2 < send) load_c(un.s0 + 2);
  // weights that fp16 may not hold among the block's: it takes them in fp32
  int over = 0;
  const int gb = (ng + 31) / 32, gb0 = k0 / GROUP / 32, gb1 = min(k0 + 255, K - 1) / GROUP / 32;
  for (int s = CL * un.s0 + tid; s < min(CL * un.s1, steps); s += 512)
    over |= big[s * gb + gb0] | big[s * gb + gb1];
  over = __syncthreads_or(over);
  // the iteration's dY and the next one's codes have landed (what was
  // requested after them may be in flight), and no wavefront still reads the
  // stages that are requested next
  auto landed = [&](int s) {
    if (L::kNC == 4 && s + 2 < send && s > un.s0)
      wait_vm<AL + CL + PL>();
    else if (L::kNC == 3 && s + 1 < send && s > un.s0)
      wait_vm<AL>();
    else
      wait_vm<0>();
    __syncthreads();
  };
  auto request = [&](int s) {
    if (s + L::kNC - 1 < send) load_c(s + L::kNC - 1);
    if (s + 2 < send) load_a(s + 2);
  };
  // Half a step (32 packed rows) at a time; while one half multiplies, the
  // next one's codes are read and converted a row pair after each few
  // fragments, so that the conversion fills the gaps between MFMAs.
  auto sum = [&]() {
    uint32_t w[8];
    uint4 zv, sv, b[4];
    uint32_t bn[4][4];
    auto read_codes = [&](int s, int ch) {
      const char* pc = smem + L::kOffC + (s % L::kNC) * L::kC + cbase + ch * 4096;
      const char* pp = smem + L::kOffP + (s % L::kNC) * L::kP + (SPLIT ? wm * 2048 : 0) +
                       gl * 256 + 16 * q4 + ch * 64;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = *(const uint32_t*)(pc + i * 512);
      zv = *(const uint4*)pp;
      sv = *(const uint4*)(pp + 128);
    };
    // rows 2 p and 2 p + 1 of the lane's eight: both halves of a dword in each
    // of the four tiles' fragments
    auto convert = [&](int p) {
      const uint32_t t = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], sel);
      const uint32_t t8 = t >> 8;
      const half2v z = __builtin_bit_cast(half2v, word_of(zv, p));
      const half2v s1 = __builtin_bit_cast(half2v, word_of(sv, p));
      const half2v m0 = {(_Float16)32768.0f, (_Float16)32768.0f};
      const half2v m1 = {(_Float16)2048.0f, (_Float16)2048.0f};
      const half2v k512 = {(_Float16)512.0f, (_Float16)512.0f};
      const half2v s5 = s1 * k512;
      const uint32_t n[4] = {t & 0x000F000Fu, t & 0x00F000F0u, t8 & 0x000F000Fu, t8 & 0x00F000F0u};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const half2v d =
            __builtin_elementwise_fma(__builtin_bit_cast(half2v, n[c]), c & 1 ? m1 : m0, z);
        bn[c][p] = __builtin_bit_cast(uint32_t, d * s5);
      }
    };
    auto take = [&]() {
#pragma unroll
      for (int c = 0; c < 4; ++c) b[c] = make_uint4(bn[c][0], bn[c][1], bn[c][2], bn[c][3]);
    };
    wait_vm<0>();
    __syncthreads();
    read_codes(un.s0, 0);
#pragma unroll
    for (int p = 0; p < 4; ++p) convert(p);
    take();
    for (int s = un.s0; s < send; ++s) {
      landed(s);
      // the odd step past the last one
      const bool live = !SPLIT || 2 * s + wm < steps;
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        if (live) {
          const char* ta = smem + (s % 3) * L::kA + (wm * MT * 16 + r16) * 128 +
                           16 * ((4 * ch + q4) ^ (r16 & 7));
          // past the end the stage holds old values: read, not used
          read_codes(s + ch, 1 - ch);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint4 a = *(const uint4*)(ta + m * 2048);
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[m][c] = mfma16<_Float16>(a, b[c], acc[m][c]);
#pragma unroll
            for (int p = 0; p < 4; ++p)
              if (m == 1 + p * (MT - 1) / 4) convert(p);
          }
          take();
        }
        // between the halves the requests delay the MFMAs least
        if (ch == 0) request(s);
      }
    }
  };
  // The same sums a packed row at a time, one product per weight and token: a
  // register of a lane is token 4 (l / 16) + r of its tile.
  auto sum_fp32 = [&]() {
    for (int s = un.s0; s < send; ++s) {
      landed(s);
      if (!SPLIT || 2 * s + wm < steps) {
        const char* pc = smem + L::kOffC + (s % L::kNC) * L::kC + (SPLIT ? wm * 8192 : 0) + 4 * r16;
        const char* pp = smem + L::kOffP + (s % L::kNC) * L::kP + (SPLIT ? wm * 2048 : 0) + gl * 256;
        const char* ta = smem + (s % 3) * L::kA + (wm * MT * 16 + 4 * q4) * 128;
#pragma unroll 1
        for (int row = 0; row < 64; ++row) {
          const int q = (row >> 3) & 3;
          const uint32_t w = *(const uint32_t*)(pc + (32 * (row >> 5) + 4 * (row & 7) + q) * 128 +
                                                ((wb ^ (q >> 1)) * 64)) >> (16 * half);
          const float nz = (float)*(const _Float16*)(pp + 2 * row) * kCodeScale;
          const float st = (float)*(const _Float16*)(pp + 128 + 2 * row);
          float v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = ((float)((w >> (4 * c)) & 15u) + nz) * st;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int t = 4 * q4 + r;  // of the tile; its rows are multiples of 8
              const float a = (float)*(const _Float16*)(ta + (16 * m + r) * 128 +
                                                        16 * ((row >> 3) ^ (t & 7)) + 2 * (row & 7));
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[m][c][r] = fmaf(a, v[c], acc[m][c][r]);
            }
        }
      }
      request(s);
    }
  };
  if (over)
    sum_fp32();
  else
    sum();
  const int col = k0 + 128 * wb + 8 * r16 + 4 * half;
  if constexpr (!SPLIT) {
    leave<T, MT>(acc, parts, un, wave, back, N, K, t0 + wm * MT * 16, col, lane, dX);
  } else {
    // each half of the wavefronts hands half of its tokens' sums to the other
    constexpr int H = MT / 2;
    floatx4 keep[H][4];
    floatx4* const mine = (floatx4*)smem + wave * (H * 4 * 64) + lane;
    const floatx4* const other = (const floatx4*)smem + (wave ^ 4) * (H * 4 * 64) + lane;
    __syncthreads();
#pragma unroll
    for (int m = 0; m < H; ++m)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mine[(m * 4 + c) * 64] = wm ? acc[m][c] : acc[H + m][c];
        keep[m][c] = wm ? acc[H + m][c] : acc[m][c];
      }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < H; ++m)
#pragma unroll
      for (int c = 0; c < 4; ++c) keep[m][c] += other[(m * 4 + c) * 64];
    leave<T, H>(keep, parts, un, wave, back, N, K, t0 + wm * H * 16, col, lane, dX);
  }
}

// Sums of a split tile's parts, in order; a block takes 32 tokens of one
// wavefront's columns.
template <typename T>
__global__ void __launch_bounds__(64)
k_dx_join(const float* __restrict__ parts, const int* __restrict__ back, int N, int K,
          T* __restrict__ dX, TileSplit sp, int mt) {
  const int lane = threadIdx.x;
  const int mp = blockIdx.x % (mt / 2), wave = blockIdx.x / (mt / 2) % 8, left = blockIdx.x / (mt * 4);
  const TileUnit un = tile_unit(sp.full + left, sp.nt, sp.no, sp.full + sp.left);
  floatx4 v[2][4];
  join_parts(parts, sp, left, wave, mt, mp, lane, v);
  const int wm = wave >> 2, wn = wave & 3;
  store_dx<T, 2>(v, back, N, K, un.t * 32 * mt + wm * mt * 16 + 32 * mp,
                 un.o * 256 + 128 * (wn >> 1) + 8 * (lane & 15) + 4 * (wn & 1), lane, dX);
}

struct DxPlan {
  int mt, steps, lda;
  bool copy;
  TileSplit sp;
  size_t off_prm, off_big, off_a, off_back, off_parts, bytes;
};
static DxPlan dx_plan(const W4Args& a) {
  DxPlan p;
  p.steps = (int)((a.O + 63) / 64);
  p.copy = a.type == kBF16 || a.O % 64;
  p.lda = p.copy ? p.steps * 64 : (int)a.O;
  choose_tiles(a.N, (int)((a.K + 255) / 256), p.steps, kDxCosts, 1.0f, &p.mt, &p.sp);
  size_t at = 0;
  p.off_prm = at;
  at += align256((size_t)p.steps * 64 * (a.K / a.group) * 4);
  p.off_big = at;
  at += align256((size_t)p.steps * ((a.K / a.group + 31) / 32) * 4);
  p.off_a = at;
  if (p.copy) at += align256((size_t)a.N * p.lda * 2);
  p.off_back = at;
  if (p.copy) at += align256((size_t)a.N * 4);
  p.off_parts = at;
  if (p.sp.parts > 1) at += (size_t)p.sp.left * p.sp.parts * p.mt * 32 * 256 * 4;
  p.bytes = at;
  return p;
}
size_t w4_input_grad_workspace(const W4Args& a) { return dx_plan(a).bytes; }

// The tile is 32 MT tokens high.
template <typename T, int GROUP, int MT>
static hipError_t launch(const W4Args& a, const void* dY, const DxPlan& p, hipStream_t stream) {
  constexpr bool SPLIT = MT <= 4;
  constexpr int W = SPLIT ? 2 * MT : MT;  // token tiles of a wavefront
  auto* kernel = &k_w4_dx<T, GROUP, W, SPLIT>;
  const int lds = DxLds<W, SPLIT>::kBytes;
  hipError_t e =
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  char* ws = (char*)a.ws;
  const int* back = a.type == kBF16 ? (const int*)(ws + p.off_back) : nullptr;
  float* parts = (float*)(ws + p.off_parts);
  hipLaunchKernelGGL(kernel, dim3((unsigned)(p.sp.full + p.sp.left * p.sp.parts)), dim3(512), lds,
                     stream, p.copy ? (const _Float16*)(ws + p.off_a) : (const _Float16*)dY, p.lda,
                     back, (int)a.N, (int)a.K, (int)a.O, (const char*)a.qweight, ws + p.off_prm,
                     (const int*)(ws + p.off_big), (T*)a.out0, parts, p.sp);
  if (p.sp.parts > 1)
    hipLaunchKernelGGL((k_dx_join<T>), dim3((unsigned)(p.sp.left * 4 * MT)), dim3(64), 0, stream,
                       parts, back, (int)a.N, (int)a.K, (T*)a.out0, p.sp, MT);
  return hipGetLastError();
}

template <typename T, int GROUP>
static hipError_t by_tokens(const W4Args& a, const void* dY, const DxPlan& p, hipStream_t stream) {
  if (p.mt == 2) return launch<T, GROUP, 2>(a, dY, p, stream);
  if (p.mt == 4) return launch<T, GROUP, 4>(a, dY, p, stream);
  if (p.mt == 6) return launch<T, GROUP, 6>(a, dY, p, stream);
  return launch<T, GROUP, 8>(a, dY, p, stream);
}

template <typename T>
static hipError_t by_group(const W4Args& a, const void* dY, const DxPlan& p, hipStream_t stream) {
  if (a.group == 128) return by_tokens<T, 128>(a, dY, p, stream);
  if (a.group == 64) return by_tokens<T, 64>(a, dY, p, stream);
  return by_tokens<T, 32>(a, dY, p, stream);
}

// Of a gated block the preparing launch forms dpre on the way.
hipError_t launch_w4_input_grad(W4Op op, const W4Args& a, hipStream_t stream) {
  const bool gated = op == kOpGatedBackward;
  const DxPlan p = dx_plan(a);
  char* ws = (char*)a.ws;
  Prepare q{};
  q.step16 = (const _Float16*)a.step16;
  q.zero16 = (const _Float16*)a.zero16;
  q.O = (int)a.O;
  q.ng = (int)(a.K / a.group);
  q.prm = ws + p.off_prm;
  q.big = (int*)(ws + p.off_big);
  q.in0 = a.in0;
  q.in1 = a.in1;
  q.dpre = a.out1;
  q.cols = (int)a.O;
  q.ld_out = p.lda;
  q.act = a.act;
  q.out = p.copy ? ws + p.off_a : nullptr;
  q.back = (int*)(ws + p.off_back);
  const hipError_t e =
      launch_w4_prepare(q, a.type, 2, gated, p.copy || gated ? a.N : 0, stream);
  if (e != hipSuccess) return e;
  const void* dY = gated ? a.out1 : a.in0;
  return a.type == kF16 ? by_group<_Float16>(a, dY, p, stream) : by_group<__bf16>(a, dY, p, stream);
}

}  // namespace awq
