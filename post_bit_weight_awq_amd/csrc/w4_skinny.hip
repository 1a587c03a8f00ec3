// Y = X W^T and H = act(X Wg^T) * (X Wu^T) on packed weights for up to 64
// tokens: the weights are read once (one token, 5120 -> 15360 in fp16: 42 MB,
// 10.6 us a call from the 256 MB cache, 11.8 us or 3.5 TB/s from HBM; 48 tokens,
// gated 5120 -> 2 x 13824 in bf16: 34 and 38 us).  Beside that stream VALU
// issue bounds it: 0.6 of the busy units' cycles.
//
// A block of eight wavefronts owns 32 WR packed rows (gated: 16 WR of the gate
// and the same features' 16 WR up rows) and all tokens.  The wavefronts are KS
// groups of WR: group g takes the blocks of 128 columns g, g + KS, ..; within
// it each wavefront takes two tiles of 16 rows and all share the activations.
// The groups' sums are added through LDS in a fixed order.
//   * Codes and activations move to LDS by direct loads of whole 64- and
//     256-byte row pieces, one iteration ahead, so the bytes in flight
//     do not cost registers.  With WR = 1 a wavefront loads only for itself
//     and the loop has no barrier.  More stages measured slower (one token,
//     5120 -> 15360: 11.0, 12.0 and 15.6 us with two, three and four): what
//     counts is blocks per compute unit, which they cost.
//   * Word 4 j + q of a row's 16 goes to lane group q for MFMA j, which thus
//     takes columns 32 j .. 32 j + 31: every MFMA lies inside one group for
//     groups of 32, 64 and 128, a group's sum of exact products (q - z) x is
//     formed by itself and enters the output with one fp32 fma by its step.
//   * Steps and zeros of the block's rows are contiguous; they are copied to
//     LDS once, laid out by group, behind the first codes.
//   * A zero is taken as a high part, from which the codes' differences are
//     exact (in bf16 for bf16 activations), and a low one, 0 for the zeros that
//     packing writes.  A block that has any other runs a second form of the
//     loop, which adds the tokens' sums over the group, one MFMA by ones for
//     both tiles, times the low parts (16 tokens, 13824 -> 5120 in bf16: 18.7
//     us with whole zeros, 21.4 with fractional ones; one token, 5120 -> 15360
//     in fp16: 10.5 and 12.3).  The ones are 2^-9, the
//     differences' unit: a sum of 128 finite values stays finite.  One that is
//     not holds an infinity or a NaN, which the product of the high parts has
//     whole, and is left out.
#include <type_traits>

#include "w4_internal.h"

namespace awq {

constexpr int kSkinnyLds = 160 * 1024;

struct SkinnyPlan {
  int lds;       // bytes
  int off_ring;  // of the two stages, behind the (step, zero) pairs
};
static SkinnyPlan skinny_plan(int64_t N, int64_t K, int group, int KS) {
  const int WR = 8 / KS, rows = 32 * WR, MT = (int)((N + 15) / 16);
  const int64_t params = ((int64_t)rows * (K / group) * 4 + 1023) & ~1023;
  const int64_t sums = (int64_t)KS * 16 * MT * (rows + 1) * 4;
  const int64_t ring = params + 2 * (KS * (N <= 4 ? 1024 : MT * 4096) + 8 * 2048);
  SkinnyPlan p;
  p.off_ring = (int)params;
  p.lds = ring > kSkinnyLds ? 0 : (int)(ring > sums ? ring : sums);
  return p;
}

template <typename T, int GROUP, bool GATED, int MT, int KS, bool FEW>
__global__ void __launch_bounds__(512, 2)
k_w4_skinny(const T* __restrict__ X, int M, int K, int O, const char* __restrict__ qw,
            const _Float16* __restrict__ step16, const _Float16* __restrict__ zero16, Epilogue ep,
            int off_ring) {
  constexpr bool BF = !__is_same(T, _Float16);
  constexpr int WR = 8 / KS, R = 32 * WR;  // packed rows per block
  constexpr int GPB = 128 / GROUP;         // groups per block of 128 columns
  constexpr int JG = 4 / GPB;              // MFMAs per group
  constexpr int RP = R + 1;                // padded row count of the sums
  constexpr int XB = FEW ? 1024 : MT * 4096;  // bytes of a group's activations per stage
  constexpr int STAGE = KS * XB + 8 * 2048;
  // activation loads of a wavefront per stage; up to four tokens are one load,
  // which every wavefront of the group issues
  constexpr int XW = FEW ? 1 : 4 * MT / WR;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  uint32_t* const pairs = (uint32_t*)smem;  // [ng][R] (step, zero)
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = wave / WR, wr = wave % WR;
  const int r16 = lane & 15, q4 = lane >> 4;
  const int nkb = K >> 7, ng = K / GROUP, F = O >> 1;
  const int rb = blockIdx.x * (GATED ? R / 2 : R);  // first output of the block
  const int rows = GATED ? F : O;                   // outputs
  // packed row of row i of the block, past the end the last one: of a
  // wavefront's 32 rows the first 16 are the gate's, the others the up rows
  auto row_of = [&](int i) {
    if (GATED) return min(rb + 16 * (i >> 5) + (i & 15), F - 1) + (i & 16 ? F : 0);
    return min(rb + i, O - 1);
  };
  // codes: two loads of 16 rows of 64 bytes, 16-byte piece p of row r at
  // p ^ (r / 4 % 4)
  uint32_t oc[2];
  const char* c0[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 32 * wr + 16 * i, row = row_of(r);
    c0[i] = qw + (size_t)row * (K >> 1);
    oc[i] = (uint32_t)(row_of(r + (lane >> 2)) - row) * (uint32_t)(K >> 1) +
            16 * ((lane & 3) ^ ((lane >> 4) & 3));
  }
  // activations: a load brings 4 tokens of 256 bytes, 16-byte piece p of
  // token t at p ^ (t % 16); past the end the last token is repeated
  uint32_t ox[XW];
#pragma unroll
  for (int i = 0; i < XW; ++i) {
    const int t = FEW ? q4 : 4 * (wr + i * WR) + q4;
    ox[i] = 2u * ((uint32_t)min(t, M - 1) * (uint32_t)K + 8 * (r16 ^ (t & 15)));
  }
  const uint32_t ring = (uint32_t)(uintptr_t)smem + off_ring;
  const int its = (nkb + KS - 1) / KS;
  auto load = [&](int it) {
    const int kb = min(it * KS + kg, nkb - 1);
    const uint32_t l = ring + (it & 1) * STAGE;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      dma16(c0[i] + 64 * kb, oc[i], l + KS * XB + (2 * wave + i) * 1024);
#pragma unroll
    for (int i = 0; i < XW; ++i)
      dma16((const char*)X + 256 * kb, ox[i], l + kg * XB + (FEW ? 0 : (wr + i * WR) * 1024));
  };
  load(0);
  uint16_t part = 0;  // of the zeros: bits of what they have behind the point,
  _Float16 top = 0;   // and the largest magnitude
  const int di = 512 / ng, dg = 512 - di * ng;
  for (int e = tid, i = tid / ng, g = tid - i * ng; e < R * ng; e += 512) {
    const size_t at = (size_t)row_of(i) * ng + g;
    const _Float16 z = zero16[at];
    part |= __builtin_bit_cast(uint16_t, (_Float16)(z - __builtin_floorf16(z)));
    top = __builtin_fmaxf16(top, __builtin_fabsf16(z));
    pairs[g * R + i] = (uint32_t)__builtin_bit_cast(uint16_t, step16[at]) |
                       ((uint32_t)__builtin_bit_cast(uint16_t, z) << 16);
    i += di;
    g += dg;
    if (g >= ng) {
      g -= ng;
      ++i;
    }
  }
  // whether any of the block is to be taken apart: each wavefront's answer goes
  // through its own codes of the second stage, requested behind the loop's
  // first barrier or, without one, this one
  const bool odd = __any(part != 0 || !((float)top <= (BF ? 240.0f : 2032.0f)));
  int* const seen = (int*)(smem + off_ring + STAGE + KS * XB);
  if (lane == 0) seen[512 * wave] = odd;
  __syncthreads();
  int apart = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) apart |= seen[512 * i];
  apart = __builtin_amdgcn_readfirstlane(apart);
  if (WR == 1) __syncthreads();

  floatx4 acc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int u = 0; u < 2; ++u) acc[m][u] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  auto sum = [&](auto parted) {
    for (int it = 0; it < its; ++it) {
      // the stage has landed, and every wavefront of the group has read the
      // other one (with WR = 1 its own reads have returned)
      wait_vm<0>();
      if (WR > 1)
        __syncthreads();
      else
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (it + 1 < its) load(it + 1);
      const int kb = it * KS + kg;
      const char* st = smem + off_ring + (it & 1) * STAGE;
      if (kb >= nkb) continue;
      const int tx = FEW ? r16 & 3 : r16;  // rows past the fourth repeat it
      const char* px = st + kg * XB + tx * 256;
      const char* pc = st + KS * XB + wave * 2048 + r16 * 64 + 4 * q4;
      uint32_t w[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[u][j] = *(const uint32_t*)(pc + u * 1024 + 16 * (j ^ (r16 >> 2)));
      uint4 x[4][MT];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          x[j][m] = *(const uint4*)(px + m * 4096 + 16 * ((4 * j + q4) ^ tx));
#pragma unroll
      for (int g = 0; g < GPB; ++g) {
        float stp[2];
        _Float16 z[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t sz = pairs[(kb * GPB + g) * R + 32 * wr + 16 * u + r16];
          z[u] = __builtin_bit_cast(_Float16, (uint16_t)(sz >> 16));
          stp[u] = f16_lo(sz) * kCodeScale;
        }
        if constexpr (parted) {
          constexpr uint32_t kOnes = BF ? 0x3b003b00u : 0x18001800u;  // 2^-9
          const uint4 ones = make_uint4(kOnes, kOnes, kOnes, kOnes);
          float low[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const ZeroParts p = split_zero<BF>((float)z[u]);
            z[u] = (_Float16)p.high;
            low[u] = -p.low * stp[u];
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            floatx4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < JG; ++j) s = mfma16<T>(x[g * JG + j][m], ones, s);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float v = fabsf(s[r]) < INFINITY ? s[r] : 0.0f;
#pragma unroll
              for (int u = 0; u < 2; ++u) acc[m][u][r] = fmaf(low[u], v, acc[m][u][r]);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t nz = neg_zero_pair(z[u]);
          floatx4 t[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) t[m] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
          uint4 b[JG];
#pragma unroll
          for (int j = 0; j < JG; ++j) {
            b[j] = dequant_word(w[u][g * JG + j], nz);
            if constexpr (BF)
              b[j] = make_uint4(half2_to_bf16x2(b[j].x), half2_to_bf16x2(b[j].y),
                                half2_to_bf16x2(b[j].z), half2_to_bf16x2(b[j].w));
          }
#pragma unroll
          for (int j = 0; j < JG; ++j)
#pragma unroll
            for (int m = 0; m < MT; ++m) t[m] = mfma16<T>(x[g * JG + j][m], b[j], t[m]);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[m][u][r] = fmaf(stp[u], t[m][r], acc[m][u][r]);
        }
      }
    }
  };
  if (apart)
    sum(std::true_type{});
  else
    sum(std::false_type{});
  __syncthreads();

  // the groups' sums: register r of lane l is token 4 (l / 16) + r, row l % 16
  // of its tile; the two tiles of wavefront wr are rows 16 wr and (gated: its
  // up rows at R / 2 + 16 wr) of the sums
  float* const red = (float*)smem;  // [KS][16 MT][RP]
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[(kg * 16 * MT + 16 * m + 4 * q4 + r) * RP +
            (GATED ? u * (R / 2) + 16 * wr : 32 * wr + 16 * u) + r16] = acc[m][u][r];
  __syncthreads();
  constexpr int C = GATED ? R / 2 : R;
  for (int e = tid; e < M * C; e += 512) {
    const int t = e / C, i = e - t * C;
    if (rb + i >= rows) continue;
    float s = 0.0f, v = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      s += red[(k * 16 * MT + t) * RP + i];
      if (GATED) v += red[(k * 16 * MT + t) * RP + C + i];
    }
    const size_t at = (size_t)t * rows + rb + i;
    if (GATED) {
      if (ep.pre) {
        ((T*)ep.pre)[(size_t)t * O + rb + i] = from_f32<T>(s);
        ((T*)ep.pre)[(size_t)t * O + F + rb + i] = from_f32<T>(v);
      }
      s = (ep.act == kActSilu ? act_value<kActSilu>(s, nullptr) : act_value<kActGelu>(s, nullptr)) * v;
    }
    if (!GATED && ep.y_type == kF32)
      ((float*)ep.y)[at] = s;
    else
      ((T*)ep.y)[at] = from_f32<T>(s);
  }
}

template <typename T, int GROUP, bool GATED, int MT, int KS, bool FEW>
static hipError_t launch(const W4Args& a, hipStream_t stream) {
  const SkinnyPlan p = skinny_plan(a.N, a.K, a.group, KS);
  const int per = GATED ? 16 * (8 / KS) : 32 * (8 / KS);
  const int64_t outs = GATED ? a.O / 2 : a.O;
  auto* kernel = &k_w4_skinny<T, GROUP, GATED, MT, KS, FEW>;
  if (p.lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(
        (const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, p.lds);
    if (e != hipSuccess) return e;
  }
  const Epilogue ep{nullptr, a.out0, a.out1, (int)a.N, (int)a.O, a.y_type, a.type, a.act};
  hipLaunchKernelGGL(kernel, dim3((unsigned)((outs + per - 1) / per)), dim3(512), p.lds, stream,
                     (const T*)a.in0, (int)a.N, (int)a.K, (int)a.O, (const char*)a.qweight,
                     (const _Float16*)a.step16, (const _Float16*)a.zero16, ep, p.off_ring);
  return hipGetLastError();
}

// Groups of wavefronts along the columns; 0 where the call goes to the tiled
// kernel.  Fewer groups share the activations among more rows but leave fewer
// blocks.  Measured (us, two / four / eight groups): one token 5120 -> 15360
// 22.2 / 13.3 / 11.0, gated 4096 -> 2 x 11008 20.7 / 16.2 / 12.9; 8 tokens
// 5120 -> 15360 22.2 / 13.8 / 14.7, 16 tokens 5120 -> 5120 21.2 / 12.4 / 8.0,
// gated 5120 -> 2 x 13824 29.2 / 24.5 / 36.0; 32 tokens, the same, 31.8 / 37.6,
// 48 tokens 5120 -> 15360 32.5 / 22.2, gated 42.8 / 50.4.
static int skinny_ks(const W4Args& a) {
  auto fits = [&](int ks) { return skinny_plan(a.N, a.K, a.group, ks).lds > 0; };
  if (a.N > 64) return 0;
  int ks = 8;
  if (a.N > 16)
    ks = a.O >= 192 * 128 ? 2 : 4;
  else if (a.N > 4 && a.O >= 224 * 64)
    ks = 4;
  if (a.N > 48) {
    // only two groups fit; below 160 blocks the tiled kernel, whose parts fill
    // the chip, is faster (64 tokens, 4096 -> 4096: 24 against 30 us)
    if (a.O < 160 * 128) return 0;
    ks = 2;
  }
  if (fits(ks)) return ks;
  // long rows of small groups: eight groups hold the fewest rows' parameters,
  // two the least activations
  return fits(8) ? 8 : fits(4) ? 4 : fits(2) ? 2 : 0;
}

// The groups that a token count can take: up to four tokens take eight (which
// fit wherever fewer do), up to 16 eight or four; LDS holds no more than four
// with 17 to 48 tokens and two with more.
template <typename T, int GROUP, bool GATED, int MT, bool FEW>
static hipError_t by_ks(const W4Args& a, hipStream_t stream) {
  const int ks = skinny_ks(a);
  if constexpr (MT == 1)
    if (ks == 8) return launch<T, GROUP, GATED, MT, 8, FEW>(a, stream);
  if constexpr (!FEW && MT <= 3)
    if (ks == 4) return launch<T, GROUP, GATED, MT, 4, FEW>(a, stream);
  if constexpr (MT >= 2)
    if (ks == 2) return launch<T, GROUP, GATED, MT, 2, FEW>(a, stream);
  return hipErrorInvalidValue;
}

template <typename T, int GROUP, bool GATED>
static hipError_t by_tokens(const W4Args& a, hipStream_t stream) {
  if (a.N <= 4) return by_ks<T, GROUP, GATED, 1, true>(a, stream);
  if (a.N <= 16) return by_ks<T, GROUP, GATED, 1, false>(a, stream);
  if (a.N <= 32) return by_ks<T, GROUP, GATED, 2, false>(a, stream);
  if (a.N <= 48) return by_ks<T, GROUP, GATED, 3, false>(a, stream);
  return by_ks<T, GROUP, GATED, 4, false>(a, stream);
}

template <typename T, int GROUP>
static hipError_t by_op(W4Op op, const W4Args& a, hipStream_t stream) {
  return op == kOpGated ? by_tokens<T, GROUP, true>(a, stream)
                        : by_tokens<T, GROUP, false>(a, stream);
}

bool w4_skinny_fits(const W4Args& a) { return skinny_ks(a) != 0; }

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
