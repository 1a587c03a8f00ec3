// Y = X W^T and H = act(X Wg^T) * (X Wu^T) on packed weights for many tokens:
// a tiled MFMA product that reads the codes as they are packed.
//
// Block tile of up to 256 tokens x 256 packed rows (gated: 128 rows of the gate
// and the same features' 128 up rows), eight wavefronts as 2 x 4 (rows), each
// 16 MT x 64 as MT x 4 tiles of v_mfma_f32_16x16x32_f16.  For tiles of 192 and
// 256 tokens the two halves of the wavefronts take half of the tokens each; for
// 64 and 128 both take all, each every second block of 128 columns (SPLIT), and
// add their sums through LDS at the end: each weight is then converted once per
// block.  One 64- or 128-token tile per unit, 512 x 4096 -> 4096: 48 and 61 us
// against 58 and 75 with halved tokens.
//   * Activations move to LDS 64 columns at a time, codes and group parameters
//     128 columns at a time, by direct loads up to two steps ahead; 16-byte
//     pieces are permuted by row so that reads hit every bank once.
//   * Codes become (q - z) 2^-9 in fp16 in registers, exactly, ten operations
//     per eight: four bits per weight through LDS instead of sixteen.
//   * The step enters in fp32.  The accumulators of a row are kept in units
//     of the present group's step: where a group begins they are multiplied
//     by (last step / this step), and by the last group's step at the end.
//     So the MFMAs accumulate in place and no product is rounded to 16 bits.
//     Ratios are rounded to nearest: 1 between equal steps, so that a row of
//     them keeps its first sums (a reciprocal's rounding, always to one side,
//     took 5e-5 of them in 432 groups).
//   * A zero is taken as a high part, which the differences hold exactly, and a
//     low one, 0 for the zeros that packing writes: where there are others, fp32
//     MFMAs behind the loop add the low parts times the tokens' group sums (333
//     tokens, 4096 -> 11008 in groups of 64: 69 and 80 us; 4096 tokens, gated
//     5120 -> 2 x 13824: 1.03 and 1.18 ms).
//   * A group whose step is 0 leaves the unit as it is and takes codes and
//     zero as 0.
// bf16 activations are first brought to fp16 by a power of two per row
// (w4_prepare.hip), which the epilogue takes back.
// Bound by the issue of MFMAs and of the conversions beside them: 4096 tokens,
// gated 5120 -> 2 x 13824 with [G | U] kept, 1.02-1.11 ms over the cards
// measured (up to 1.13 PFLOP/s; with the codes converted where they are used 4 %
// more); 333 tokens, 4096 -> 11008 in groups of 64, 68-70 us.
#include "w4_adapt.h"
#include "w4_internal.h"

namespace awq {

constexpr int kBN = 256;    // packed rows per block
constexpr int kEpRow = 68;  // floats per token of a wavefront's 64 columns in the epilogue's LDS
constexpr int kEpWave = 32 * kEpRow;

template <bool GATED, typename T>
__device__ __forceinline__ void store_outputs(const Epilogue& e, int token, int o, int outs,
                                              float (&v)[8], const float (&u)[8], T* y) {
  if constexpr (GATED) {
    const int F = outs;
    if (e.pre) {
      T* pre = (T*)e.pre + (size_t)token * 2 * F + o;
      store8(pre, v, F - o, (F & 7) == 0);
      store8(pre + F, u, F - o, (F & 7) == 0);
    }
    if (e.act == kActSilu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_value<kActSilu>(v[i], nullptr) * u[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_value<kActGelu>(v[i], nullptr) * u[i];
    }
  }
  store8(y + (size_t)token * outs + o, v, outs - o, (outs & 7) == 0);
}

// 32 tokens from t0 of a wavefront's 64 columns (gated: 32 of the gate, then
// their 32 up columns), through the wavefront's own LDS: eight columns of a
// token per lane then, stored as whole 16-byte pieces.  Register r of lane l
// is token 4 (l / 16) + r, column l % 16 of its tile.
template <bool GATED>
__device__ __forceinline__ void finish32(const floatx4 (&v0)[4], const floatx4 (&v1)[4], float* ep,
                                         const Epilogue& e, int t0, int ob, int lane) {
  constexpr int CW = GATED ? 32 : 64, LPT = CW / 8;
  const int r16 = lane & 15, q4 = lane >> 4;
  const int outs = GATED ? e.O / 2 : e.O;
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      ep[(4 * q4 + r) * kEpRow + 16 * n + r16] = v0[n][r];
      ep[(16 + 4 * q4 + r) * kEpRow + 16 * n + r16] = v1[n][r];
    }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the wavefront's own writes
  asm volatile("" ::: "memory");
#pragma unroll
  for (int it = 0; it < 32 * LPT / 64; ++it) {
    const int tl = it * (64 / LPT) + lane / LPT, c8 = 8 * (lane % LPT);
    const int token = t0 + tl, o = ob + c8;
    float v[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = ep[tl * kEpRow + c8 + i];
      u[i] = GATED ? ep[tl * kEpRow + 32 + c8 + i] : 0.0f;
    }
    if (token >= e.N || o >= outs) continue;
    if (e.back) {
      const int x = e.back[token];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = ldexpf(v[i], x);
        if (GATED) u[i] = ldexpf(u[i], x);
      }
    }
    if (!GATED && e.y_type == kF32)
      store_outputs<GATED>(e, token, o, outs, v, u, (float*)e.y);
    else if (e.type == kF16)
      store_outputs<GATED>(e, token, o, outs, v, u, (_Float16*)e.y);
    else
      store_outputs<GATED>(e, token, o, outs, v, u, (__bf16*)e.y);
  }
  asm volatile("" ::: "memory");
}

// A part's sums to the workspace as they lie, a whole tile's values to the
// outputs through LDS once no wavefront reads it any more.
template <bool GATED, int MT>
__device__ __forceinline__ void leave(const floatx4 (&acc)[MT][4], float* parts, const SplitUnit& un,
                                      int wave, float* own, const Epilogue& ep, int t0, int ob,
                                      int lane) {
  if (un.parts > 1) {
    floatx4* p = (floatx4*)parts + ((size_t)un.slot * 8 + wave) * (MT * 4 * 64) + lane;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n) p[(m * 4 + n) * 64] = acc[m][n];
    return;
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; m += 2) finish32<GATED>(acc[m], acc[m + 1], own, ep, t0 + 16 * m, ob, lane);
}

// Three stages of the activations and of the codes; the codes of 128 columns
// (SPLIT: 64 of each of two blocks of 128), parameters three (two) stages.
template <int GROUP, int MT, bool SPLIT>
struct GemmLds {
  static constexpr int kA = 32 * MT * 128;                           // 64 columns of activations
  static constexpr int kC = kBN * 64;                                // codes
  static constexpr int kP1 = kBN * 4 * (128 / GROUP);                // parameters of 128 columns
  static constexpr int kP = (SPLIT ? 2 : 1) * kP1, kNP = SPLIT ? 2 : 3;
  static constexpr int kOffC = 3 * kA, kOffP = kOffC + 3 * kC;
  static constexpr int kMain = kOffP + kNP * kP;
  static constexpr int kBytes = kMain > 8 * kEpWave * 4 ? kMain : 8 * kEpWave * 4;
  static_assert(kBytes <= 160 * 1024);
};

// The zeros' low parts: they multiply the tokens' sums over each group, as fp32
// matrix products over the groups g0 .. g1 - 1, from what the preparing launch
// left of the sums.
struct Lows {
  const float* sums;  // [N, ng], and as far behind as a last lane's four loads reach
  const int* parted;  // per 32 rows x 32 groups: whether `lows` holds them
  const float* lows;  // [ng, O]
};
template <int MT, typename RowOf>
__device__ __forceinline__ void add_lows(floatx4 (&acc)[MT][4], const Lows& l, RowOf row_of, int N, int O,
                                         int ng, int g0, int g1, int t0, int lane) {
  typedef float float4u __attribute__((ext_vector_type(4), aligned(4)));
  const int r16 = lane & 15, q4 = lane >> 4;
  // 16 groups' loads at a time, four neighbours per lane
#pragma unroll 1
  for (int gb = g0; gb < g1; gb += 16) {
    const int g = gb + 4 * q4;
    float c[4][4];
    float4u s[MT];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int row = row_of(16 * n + r16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // loaded in any case, so that no load waits for the other
        const int at = min(g + i, ng - 1);
        const float v = l.lows[(size_t)at * O + row];
        const int there = l.parted[(at >> 5) * ((O + 31) >> 5) + (row >> 5)];
        c[i][n] = g + i < g1 && there ? v : 0.0f;
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      s[m] = *(const float4u*)(l.sums + (size_t)min(t0 + 16 * m + r16, N - 1) * ng + g);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[m][i] = g + i < g1 ? s[m][i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(s[m][i], c[i][n], acc[m][n], 0, 0, 0);
  }
}

// AD: Adapters, whose term the part with the first columns adds, or none.
template <int GROUP, bool GATED, int MT, bool SPLIT, typename AD>
__global__ void __launch_bounds__(512, 2)
k_w4_gemm(const _Float16* __restrict__ A, int K, const char* __restrict__ qw,
          const char* __restrict__ prm, Lows lows, float* __restrict__ parts, TileSplit sp,
          Epilogue ep, AD ad) {
  using L = GemmLds<GROUP, MT, SPLIT>;
  constexpr int BM = (SPLIT ? 16 : 32) * MT;
  constexpr int GPB = 128 / GROUP, JG = 4 / GPB;
  constexpr int AL = MT / 2;  // direct loads of activations per wavefront and half
  // of group parameters per iteration
  constexpr int PL = SPLIT ? GPB : GPB == 4 ? 2 : 1;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int r16 = lane & 15, q4 = lane >> 4;
  const SplitUnit un = split_unit(blockIdx.x, sp);
  const int N = ep.N, O = ep.O, F = O >> 1;
  const int t0 = un.t * BM, rb = un.o * (GATED ? kBN / 2 : kBN);
  const uint32_t lds = (uint32_t)(uintptr_t)smem;
  // An iteration takes 128 columns, or two such blocks (SPLIT), of which
  // wavefronts 0-3 load and take the even ones and 4-7 the odd ones; an odd one
  // past the end loads the last block, which is not used.
  const int nkb = K >> 7;
  auto block_of = [&](int it) {
    return SPLIT ? __builtin_amdgcn_readfirstlane(min(2 * it + wm, nkb - 1)) : it;
  };
  const int lw = SPLIT ? wn : wave;  // the wavefront among those that load a block

  // activations: load i brings 8 rows of 128 bytes; 16-byte piece p of row r
  // at p ^ (r % 8)
  uint32_t oa[AL];
#pragma unroll
  for (int i = 0; i < AL; ++i) {
    const int r = 8 * (lw * AL + i) + (lane >> 3);
    oa[i] = 2u * ((uint32_t)(min(t0 + r, N - 1) - t0) * (uint32_t)K + 8 * ((lane & 7) ^ (r & 7)));
  }
  const char* a0 = (const char*)(A + (size_t)t0 * K);
  auto load_a = [&](int s) {  // half s & 1 of iteration s / 2
    // halves follow each other where blocks do
    const int col = SPLIT ? 2 * block_of(s >> 1) + (s & 1) : s;
    const char* base = a0 + col * 128;
#pragma unroll
    for (int i = 0; i < AL; ++i)
      dma16(base, oa[i], lds + (s % 3) * L::kA + (wave * AL + i) * 1024);
  };
  // Block row i: wavefront column i / 64; gated, its first 32 rows are the
  // gate's and the next 32 the same features' up rows.  Past the end the last
  // row is repeated.
  auto packed_row = [&](int i) {
    if (GATED) return min(rb + 32 * (i >> 6) + (i & 31), F - 1) + (i & 32 ? F : 0);
    return min(rb + i, O - 1);
  };
  // codes: a load brings 16 rows of 64 bytes, 16-byte piece p of row r at
  // p ^ (r / 4 % 4); or 32 rows of 32 bytes, at p ^ (r / 8 % 2).  A load's rows
  // lie in one half of the packed rows.
  constexpr int RB = SPLIT ? 32 : 64, RL = 1024 / RB;  // bytes of a row, rows of a load
  uint32_t oc[2];
  const char* c0[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = RL * (2 * lw + i), row = packed_row(r);
    const int at = SPLIT ? (lane & 1) ^ ((lane >> 4) & 1) : (lane & 3) ^ ((lane >> 4) & 3);
    c0[i] = qw + (size_t)row * (K >> 1);
    oc[i] = (uint32_t)(packed_row(r + lane / (RB / 16)) - row) * (uint32_t)(K >> 1) + 16 * at;
  }
  auto load_c = [&](int s) {  // SPLIT: of a half; else of iteration s
    const int off = SPLIT ? 64 * block_of(s >> 1) + 32 * (s & 1) : 64 * s;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      dma16(c0[i] + off, oc[i], lds + L::kOffC + (s % 3) * L::kC + (2 * wave + i) * 1024);
  };
  // parameters: 64 rows of one group (32 with one group and all wavefronts)
  constexpr bool PHALF = !SPLIT && GPB == 1;
  uint32_t op[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int at = PHALF ? 32 * wave + (lane & 31) : 64 * (lw * PL + i) + lane;
    op[i] = 4u * ((uint32_t)(at / kBN) * (uint32_t)O + (uint32_t)packed_row(at % kBN));
  }
  auto load_p = [&](int it) {
    const char* p = prm + (size_t)block_of(it) * GPB * O * 4;
    const uint32_t l = lds + L::kOffP + (it % L::kNP) * L::kP + (SPLIT ? wm * L::kP1 : 0);
    if (PHALF) {
      if (lane < 32) dma4(p, op[0], l + wave * 128);
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i) dma4(p, op[i], l + (lw * PL + i) * 256);
    }
  };

  floatx4 acc[MT][4];
  float unit[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    unit[n] = 1.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // One set of 32 columns at a time; while set j multiplies, the next one's
  // codes (its group's parameters where it begins one) are read and converted
  // after each few fragments, so that the conversion fills the gaps between
  // MFMAs.
  uint4 b[4];
  uint32_t w[4], pv[4], nz[4], factors[4];
  float ratio[4], next_ratio[4];
  auto read_codes = [&](int it, int j) {
    const char* pc = smem + L::kOffC + (64 * wn + r16) * RB + 4 * q4;
#pragma unroll
    for (int n = 0; n < 4; ++n)
      w[n] = SPLIT ? *(const uint32_t*)(pc + (2 * it + (j >> 1)) % 3 * L::kC + wm * 8192 + n * 512 +
                                        16 * ((j & 1) ^ (r16 >> 3)))
                   : *(const uint32_t*)(pc + it % 3 * L::kC + n * 1024 + 16 * (j ^ (r16 >> 2)));
    const char* pp = smem + L::kOffP + (it % L::kNP) * L::kP + (SPLIT ? wm * L::kP1 : 0) +
                     (64 * wn + r16) * 4;
    if (j % JG == 0)
#pragma unroll
      for (int n = 0; n < 4; ++n)
        pv[n] = *(const uint32_t*)(pp + (j / JG) * (kBN * 4) + n * 64);
  };
  // of tile column n; `more` false: behind the last set the unit stays
  auto take_params = [&](int n, bool more) {
    const bool none = (pv[n] & 0x7fffu) == 0;
    nz[n] = none ? 0 : (pv[n] >> 16) | (pv[n] & 0xffff0000u);
    factors[n] = none ? 0 : kNibbleFactors;
    const float st = none || !more ? unit[n] : f16_lo(pv[n]);
    // unit / st to the nearest: 1 where the unit stays, as 1 / st times it is not
    const float inv = __builtin_amdgcn_rcpf(st);
    const float q = unit[n] * inv;
    next_ratio[n] = fmaf(fmaf(-q, st, unit[n]), inv, q);
    unit[n] = st;
  };
  // Does a zero of this wavefront's columns and groups have a low part?  Its 64
  // columns begin on a multiple of 32 rows, but for the up rows' 32.  The first
  // answers are requested here and looked at behind the loop.
  const int ow = rb + (GATED ? 32 : 64) * wn;
  const int ng = K / GROUP, g0 = (SPLIT ? 2 : 1) * un.s0 * GPB;
  const int g1 = min((SPLIT ? 2 : 1) * un.s1 * GPB, ng);
  const int first = 4 * (g0 >> 5) + lane, last = 4 * ((g1 + 31) >> 5);
  auto flag = [&](int e) {
    const int j = e & 3;
    const int row = GATED ? min(ow, F - 1) + (j & 1 ? F : 0) : ow + 32 * (j & 1);
    const int off = GATED && j == 3 ? 31 : 0;
    return lows.parted[(e >> 2) * ((O + 31) >> 5) + (min(row + off, O - 1) >> 5)];
  };
  int low = flag(min(first, last - 1));
  const int end = un.s1, send = 2 * end;
  if constexpr (SPLIT) {
    load_p(un.s0);
    load_c(2 * un.s0);
    load_a(2 * un.s0);
    load_c(2 * un.s0 + 1);
    load_a(2 * un.s0 + 1);
    wait_vm<2 * AL + 2>();  // the first parameters and codes
  } else {
    load_c(un.s0);
    load_p(un.s0);
    load_a(2 * un.s0);
    if (un.s0 + 1 < end) {
      load_c(un.s0 + 1);
      load_p(un.s0 + 1);
    }
    load_a(2 * un.s0 + 1);
    if (un.s0 + 1 < end)
      wait_vm<2 * AL + 2 + PL>();
    else
      wait_vm<2 * AL>();
  }
  __syncthreads();
  read_codes(un.s0, 0);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    take_params(n, true);
    b[n] = dequant_word(w[n], nz[n], factors[n]);
    ratio[n] = next_ratio[n];
  }
  for (int it = un.s0; it < end; ++it) {
    // whether this wavefront has this block and another one
    const bool live = !SPLIT || 2 * it + wm < nkb;
    const bool more = it + 1 < end && (!SPLIT || 2 * it + 2 + wm < nkb);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int s = 2 * it + h;
      // This half's activations have landed, and the codes and parameters that
      // its last set reads ahead.  What may be in flight was requested after
      // them: the next half's activations, without SPLIT also one block's
      // codes, as far as there are any.  No wavefront still reads the stages
      // requested next.
      if constexpr (SPLIT) {
        if (s + 1 < send && s > 2 * un.s0)
          wait_vm<AL>();
        else
          wait_vm<0>();
      } else {
        if (it + 1 + h < end)
          wait_vm<AL + 2 + PL>();
        else if (it + h < end)
          wait_vm<AL>();
        else
          wait_vm<0>();
      }
      __syncthreads();
      const char* ta = smem + (s % 3) * L::kA + (wm * MT * 16 + r16) * 128;
#pragma unroll
      for (int j2 = 0; j2 < 2; ++j2) {
        const int j = 2 * h + j2, jn = (j + 1) & 3;
        if (live) {
          // past the last block the stage holds an old one: read, not used
          read_codes(j == 3 ? it + 1 : it, jn);
          uint4 bn[4];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint4 a = *(const uint4*)(ta + m * 2048 + 16 * ((4 * j2 + q4) ^ (r16 & 7)));
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              if (j % JG == 0)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[m][n][r] *= ratio[n];
              acc[m][n] = mfma16<_Float16>(a, b[n], acc[m][n]);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
              if (m == 1 + n * (MT - 1) / 4) {
                if (jn % JG == 0) take_params(n, j != 3 || more);
                bn[n] = dequant_word(w[n], nz[n], factors[n]);
              }
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            b[n] = bn[n];
            if (jn % JG == 0) ratio[n] = next_ratio[n];
          }
        }
        // between a half's two sets the requests delay the MFMAs least
        if (j2 == 0) {
          if constexpr (SPLIT) {
            if (h == 0 && it + 1 < end) load_p(it + 1);
            if (s + 2 < send) {
              load_c(s + 2);
              load_a(s + 2);
            }
          } else if (it + 1 < end) {
            load_a(s + 2);
            if (h == 0 && it + 2 < end) {
              load_c(it + 2);
              load_p(it + 2);
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[m][n][r] *= unit[n] * kCodeScale;
  for (int e = first + 64; e < last; e += 64) low |= flag(e);
  low = __any(low);
  auto row_of = [&](int i) { return packed_row(64 * wn + i); };
  if constexpr (!SPLIT) {
    if (low) add_lows(acc, lows, row_of, N, O, ng, g0, g1, t0 + wm * MT * 16, lane);
    if constexpr (AD::on)
      if (un.s0 == 0)
        add_adapters<MT>(acc, ad, ep.type, ep.back, [&](int n) { return row_of(16 * n + r16); }, O,
                         t0 + wm * MT * 16, N, lane);
    leave<GATED, MT>(acc, parts, un, wave, (float*)smem + wave * kEpWave, ep, t0 + wm * MT * 16, ow,
                     lane);
  } else {
    // each half of the wavefronts hands half of its tokens' sums to the other
    __syncthreads();
    constexpr int H = MT / 2;
    floatx4 keep[H][4];
    floatx4* const mine = (floatx4*)smem + wave * (H * 4 * 64) + lane;
    const floatx4* const other = (const floatx4*)smem + (wave ^ 4) * (H * 4 * 64) + lane;
#pragma unroll
    for (int m = 0; m < H; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        mine[(m * 4 + n) * 64] = wm ? acc[m][n] : acc[H + m][n];
        keep[m][n] = wm ? acc[H + m][n] : acc[m][n];
      }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < H; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n) keep[m][n] += other[(m * 4 + n) * 64];
    if (low) add_lows(keep, lows, row_of, N, O, ng, g0, g1, t0 + wm * H * 16, lane);
    if constexpr (AD::on)
      if (un.s0 == 0)
        add_adapters<H>(keep, ad, ep.type, ep.back, [&](int n) { return row_of(16 * n + r16); }, O,
                        t0 + wm * H * 16, N, lane);
    leave<GATED, H>(keep, parts, un, wave, (float*)smem + wave * kEpWave, ep, t0 + wm * H * 16, ow,
                    lane);
  }
}

// Sums of a split tile's parts, in order; a block takes 32 tokens of one
// wavefront's columns.
template <bool GATED>
__global__ void __launch_bounds__(64)
k_gemm_join(const float* __restrict__ parts, TileSplit sp, Epilogue ep, int mt) {
  __shared__ float lds[kEpWave];
  const int lane = threadIdx.x;
  const int mp = blockIdx.x % (mt / 2), wave = blockIdx.x / (mt / 2) % 8, left = blockIdx.x / (mt * 4);
  const TileUnit un = tile_unit(sp.full + left, sp.nt, sp.no, sp.full + sp.left);
  floatx4 v[2][4];
  join_parts(parts, sp, left, wave, mt, mp, lane, v);
  finish32<GATED>(v[0], v[1], lds, ep, un.t * 32 * mt + (wave >> 2) * mt * 16 + 32 * mp,
                  un.o * (GATED ? kBN / 2 : kBN) + (GATED ? 32 : 64) * (wave & 3), lane);
}

struct GemmPlan {
  int mt;
  TileSplit sp;
  size_t off_prm, off_parted, off_lows, off_sums, off_a, off_back, off_parts, bytes;
};
static GemmPlan gemm_plan(W4Op op, const W4Args& a) {
  GemmPlan p;
  const int64_t outs = op == kOpGated ? a.O / 2 : a.O, per = op == kOpGated ? kBN / 2 : kBN;
  // groups of 64 and 32 change the unit two and four times per 128 columns:
  // a step takes 1.2 and 1.5 times as long (512 x 4096 x 4096)
  const float scale = a.group == 128 ? 1.0f : a.group == 64 ? 1.2f : 1.5f;
  choose_tiles(a.N, (int)((outs + per - 1) / per), (int)(a.K / 128), kGemmCosts, scale, &p.mt,
               &p.sp);
  size_t at = 0;
  p.off_prm = at;
  at += align256((size_t)a.O * (a.K / a.group) * 4);
  p.off_parted = at;
  at += align256((size_t)((a.O + 31) / 32) * ((a.K / a.group + 31) / 32) * 4);
  p.off_lows = at;
  at += align256((size_t)a.O * (a.K / a.group) * 4);
  p.off_sums = at;
  at += align256((size_t)a.N * (a.K / a.group) * 4 + 64);
  p.off_a = p.off_back = at;
  if (a.type == kBF16) {
    at += align256((size_t)a.N * a.K * 2);
    p.off_back = at;
    at += align256((size_t)a.N * 4);
  }
  p.off_parts = at;
  if (p.sp.parts > 1) at += (size_t)p.sp.left * p.sp.parts * p.mt * 32 * kBN * 4;
  p.bytes = at;
  return p;
}
size_t w4_gemm_workspace(W4Op op, const W4Args& a) { return gemm_plan(op, a).bytes; }

// The tile is 32 MT tokens high.
template <int GROUP, bool GATED, int MT, typename AD>
static hipError_t launch(const W4Args& a, const AD& ad, const GemmPlan& p, hipStream_t stream) {
  constexpr bool SPLIT = MT <= 4;
  constexpr int W = SPLIT ? 2 * MT : MT;  // token tiles of a wavefront
  auto* kernel = &k_w4_gemm<GROUP, GATED, W, SPLIT, AD>;
  const int lds = GemmLds<GROUP, W, SPLIT>::kBytes;
  const hipError_t e =
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  char* ws = (char*)a.ws;
  const bool bf = a.type == kBF16;
  const Epilogue ep{bf ? (const int*)(ws + p.off_back) : nullptr,
                    a.out0, a.out1, (int)a.N, (int)a.O, a.y_type, a.type, a.act};
  const Lows lows{(const float*)(ws + p.off_sums), (const int*)(ws + p.off_parted),
                  (const float*)(ws + p.off_lows)};
  float* parts = (float*)(ws + p.off_parts);
  hipLaunchKernelGGL(kernel, dim3((unsigned)(p.sp.full + p.sp.left * p.sp.parts)), dim3(512), lds,
                     stream, bf ? (const _Float16*)(ws + p.off_a) : (const _Float16*)a.in0, (int)a.K,
                     (const char*)a.qweight, ws + p.off_prm, lows, parts, p.sp, ep, ad);
  if (p.sp.parts > 1)
    hipLaunchKernelGGL(k_gemm_join<GATED>, dim3((unsigned)(p.sp.left * 4 * MT)), dim3(64), 0, stream,
                       parts, p.sp, ep, MT);
  return hipGetLastError();
}

template <int GROUP, bool GATED, typename AD>
static hipError_t by_tile(const W4Args& a, const AD& ad, const GemmPlan& p, hipStream_t stream) {
  if (p.mt == 2) return launch<GROUP, GATED, 2>(a, ad, p, stream);
  if (p.mt == 4) return launch<GROUP, GATED, 4>(a, ad, p, stream);
  if (p.mt == 6) return launch<GROUP, GATED, 6>(a, ad, p, stream);
  return launch<GROUP, GATED, 8>(a, ad, p, stream);
}

template <bool GATED, typename AD>
static hipError_t by_group(const W4Args& a, const AD& ad, const GemmPlan& p, hipStream_t stream) {
  if (a.group == 128) return by_tile<128, GATED>(a, ad, p, stream);
  if (a.group == 64) return by_tile<64, GATED>(a, ad, p, stream);
  return by_tile<32, GATED>(a, ad, p, stream);
}

static hipError_t prepare(const W4Args& a, const GemmPlan& p, hipStream_t stream) {
  char* ws = (char*)a.ws;
  Prepare q{};
  q.step16 = (const _Float16*)a.step16;
  q.zero16 = (const _Float16*)a.zero16;
  q.O = (int)a.O;
  q.ng = (int)(a.K / a.group);
  q.prm = ws + p.off_prm;
  q.parted = (int*)(ws + p.off_parted);
  q.lows = (float*)(ws + p.off_lows);
  q.sums = (float*)(ws + p.off_sums);
  q.shift = __builtin_ctz((unsigned)a.group);
  q.in0 = a.in0;
  q.cols = q.ld_out = (int)a.K;
  q.out = ws + p.off_a;
  q.back = (int*)(ws + p.off_back);
  return launch_w4_prepare(q, a.type, 1, false, a.N, stream);
}

hipError_t launch_w4_gemm(W4Op op, const W4Args& a, hipStream_t stream) {
  const GemmPlan p = gemm_plan(op, a);
  const hipError_t e = prepare(a, p, stream);
  if (e != hipSuccess) return e;
  return op == kOpGated ? by_group<true>(a, NoAdapters{}, p, stream)
                        : by_group<false>(a, NoAdapters{}, p, stream);
}

hipError_t launch_w4_gemm_adapted(const W4Args& a, const Adapters& ad, hipStream_t stream) {
  const GemmPlan p = gemm_plan(kOpLinear, a);
  const hipError_t e = prepare(a, p, stream);
  if (e != hipSuccess) return e;
  return by_group<false>(a, ad, p, stream);
}

}  // namespace awq
