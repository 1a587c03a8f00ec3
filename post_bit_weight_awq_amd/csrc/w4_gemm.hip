// Y = X W^T and H = act(X Wg^T) * (X Wu^T) on packed weights for many tokens:
// a tiled MFMA product that reads the codes as they are packed.
//
// Block tile 32 MT tokens x 256 packed rows (gated: 128 rows of the gate and
// the same features' 128 up rows), eight wavefronts as 2 (tokens) x 4 (rows),
// each 16 MT x 64 as MT x 4 tiles of v_mfma_f32_16x16x32_f16.
//   * Activations move to LDS 128 columns at a time by direct loads, two
//     stages; the 16-byte piece p of row r sits at p ^ (r % 16), so fragment
//     reads hit every bank once.
//   * Codes go from memory to registers (16 bytes per lane, row and step, one
//     step ahead) and become (q - z) 2^-9 in fp16 there, exactly, ten
//     operations per eight: no LDS traffic and a quarter of the load bytes of
//     16-bit weights.
//   * The step enters in fp32.  The accumulators of a row are kept in units
//     of the present group's step: where a group begins they are multiplied
//     by (last step / this step), and the last group's step by the epilogue.
//     So the MFMAs accumulate in place and no product is rounded to 16 bits.
//   * A group whose step is 0 leaves the unit as it is and takes codes and
//     zero as 0.
// bf16 activations are first brought to fp16 by a power of two per row
// (k_rows_to_half), which the epilogue takes back.
#include "awq_internal.h"
#include "w4_device.h"
#include "w4_internal.h"

namespace awq {

// (step, -zero 2^-9) as fp16 pairs by group: prm[g * O + row].
__global__ void __launch_bounds__(256)
k_w4_params(const uint16_t* __restrict__ step16, const uint16_t* __restrict__ zero16, int O, int ng,
            uint32_t* __restrict__ prm) {
  __shared__ uint32_t tile[32][33];
  const int r0 = blockIdx.x * 32, g0 = blockIdx.y * 32;
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    const int row = r0 + r + i, g = g0 + c;
    if (row < O && g < ng) {
      const size_t at = (size_t)row * ng + g;
      const uint32_t nz = neg_zero_pair(__builtin_bit_cast(_Float16, zero16[at]));
      tile[r + i][c] = (uint32_t)step16[at] | (nz & 0xffff0000u);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    const int row = r0 + c, g = g0 + r + i;
    if (row < O && g < ng) prm[(size_t)g * O + row] = tile[c][r + i];
  }
}

// Rows padded to ld_out with zeros; fp16 rows as they are, back = 0.  Rows of
// bf16 become fp16 times 2^e, e chosen by the row's largest finite
// magnitude (which lands in [2^14, 2^15)); back[row] = 2^-e as an exponent.
// Values down to 2^-32 of the largest stay exact, smaller ones are rounded at
// 2^-40 of it.
template <bool BF16>
__global__ void __launch_bounds__(256)
k_rows_to_half(const uint16_t* __restrict__ in, int cols, int ld_out, _Float16* __restrict__ out,
               int* __restrict__ back) {
  __shared__ uint32_t red[4];
  const size_t row = blockIdx.x;
  const uint16_t* src = in + row * cols;
  const bool vec = (cols & 7) == 0;
  _Float16* dst = out + row * ld_out;
  for (int c = cols + threadIdx.x; c < ld_out; c += 256) dst[c] = (_Float16)0.0f;
  if constexpr (!BF16) {
    if (vec)
      for (int c = threadIdx.x * 8; c < cols; c += 2048) *(uint4*)(dst + c) = *(const uint4*)(src + c);
    else
      for (int c = threadIdx.x; c < cols; c += 256) dst[c] = __builtin_bit_cast(_Float16, src[c]);
    if (threadIdx.x == 0) back[row] = 0;
    return;
  }
  uint32_t top = 0;  // largest finite magnitude, as bits
  auto look = [&](uint32_t b) {
    b &= 0x7fffu;
    if (b < 0x7f80u && b > top) top = b;
  };
  if (vec) {
    for (int c = threadIdx.x * 8; c < cols; c += 2048) {
      const uint4 v = *(const uint4*)(src + c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        look(w[e]);
        look(w[e] >> 16);
      }
    }
  } else {
    for (int c = threadIdx.x; c < cols; c += 256) look(src[c]);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, d, 64);
    top = o > top ? o : top;
  }
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
  __syncthreads();
  top = max(max(red[0], red[1]), max(red[2], red[3]));
  // the largest is in [2^(x - 1), 2^x): x from frexp, also for subnormals
  int x = 0;
  if (top) (void)frexpf(__uint_as_float(top << 16), &x);
  const int e = top ? 15 - x : 0;
  if (threadIdx.x == 0) back[row] = -e;
  auto half = [&](uint32_t b) -> uint32_t {
    return __builtin_bit_cast(uint16_t, (_Float16)ldexpf(__uint_as_float(b << 16), e));
  };
  if (vec) {
    for (int c = threadIdx.x * 8; c < cols; c += 2048) {
      const uint4 v = *(const uint4*)(src + c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = half(w[i] & 0xffffu) | (half(w[i] >> 16) << 16);
      *(uint4*)(dst + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
    for (int c = threadIdx.x; c < cols; c += 256)
      dst[c] = __builtin_bit_cast(_Float16, (uint16_t)half(src[c]));
  }
}

hipError_t launch_rows_to_half(const void* in, int type, int64_t rows, int64_t cols, int64_t ld_out, void* out,
                               int* back, hipStream_t stream) {
  if (type == kBF16)
    hipLaunchKernelGGL(k_rows_to_half<true>, dim3((unsigned)rows), dim3(256), 0, stream,
                       (const uint16_t*)in, (int)cols, (int)ld_out, (_Float16*)out, back);
  else
    hipLaunchKernelGGL(k_rows_to_half<false>, dim3((unsigned)rows), dim3(256), 0, stream,
                       (const uint16_t*)in, (int)cols, (int)ld_out, (_Float16*)out, back);
  return hipGetLastError();
}

constexpr int kBN = 256;   // packed rows per block
constexpr int kEpRow = 68;  // floats per token of a wavefront's 64 columns in the epilogue's LDS
constexpr int kEpBytes = 8 * 32 * kEpRow * 4;

template <typename T, int GROUP, bool GATED, int ACT, int MT, typename TY>
__global__ void __launch_bounds__(512, 2)
k_w4_gemm(const _Float16* __restrict__ A, const int* __restrict__ back, int N, int K, int O,
          const uint32_t* __restrict__ qw, const uint32_t* __restrict__ prm, TY* __restrict__ Y,
          T* __restrict__ pre, int nt, int no) {
  constexpr int BM = 32 * MT;
  constexpr int GPB = 128 / GROUP, JG = 4 / GPB;
  constexpr int STAGE = BM * 128;  // halfs
  extern __shared__ __attribute__((aligned(16))) _Float16 smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int r16 = lane & 15, q4 = lane >> 4;
  const TileUnit un = tile_unit(blockIdx.x, nt, no, nt * no);
  const int F = O >> 1;
  const int t0 = un.t * BM, rb = un.o * (GATED ? kBN / 2 : kBN);
  const int outs = GATED ? F : O;
  const int nkb = K >> 7;

  // direct loads of the activations: load i brings 4 rows of 256 bytes
  uint32_t oa[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = 4 * (wave * MT + i) + q4;
    oa[i] = 2u * ((uint32_t)(min(t0 + r, N - 1) - t0) * (uint32_t)K + 8 * (r16 ^ (r & 15)));
  }
  const _Float16* a0 = A + (size_t)t0 * K;
  auto load_a = [&](int s) {
    const _Float16* base = a0 + s * 128;
    const _Float16* d = smem + (s & 1) * STAGE + wave * MT * 512;
#pragma unroll
    for (int i = 0; i < MT; ++i) dma16(base, oa[i], (uint32_t)(uintptr_t)(d + i * 512));
  };
  // row of tile n (16 rows each) for this lane, past the end the last one
  int prow[4];
  uint32_t oq[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    if (GATED)
      prow[n] = min(rb + 32 * wn + 16 * (n & 1) + r16, F - 1) + (n < 2 ? 0 : F);
    else
      prow[n] = min(rb + 64 * wn + 16 * n + r16, O - 1);
  }
  // codes relative to the block's first row (of the gate's or the up rows)
  const uint32_t* q0 = qw + (size_t)rb * (K >> 3);
  const uint32_t* q1 = GATED ? q0 + (size_t)F * (K >> 3) : q0;
#pragma unroll
  for (int n = 0; n < 4; ++n)
    oq[n] = (uint32_t)(prow[n] - rb - (GATED && n >= 2 ? F : 0)) * (uint32_t)(K >> 3) + 4 * q4;
  uint4 cn[4];
  uint32_t pn[4][GPB];
  auto load_w = [&](int s) {
#pragma unroll
    for (int n = 0; n < 4; ++n) cn[n] = *(const uint4*)((n < 2 ? q0 : q1) + oq[n] + 16 * s);
#pragma unroll
    for (int g = 0; g < GPB; ++g)
#pragma unroll
      for (int n = 0; n < 4; ++n) pn[n][g] = prm[(size_t)(s * GPB + g) * O + prow[n]];
  };

  floatx4 acc[MT][4];
  float unit[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    unit[n] = 1.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  load_w(0);
  load_a(0);
  for (int s = 0; s < nkb; ++s) {
    // this step's operands have landed, and no wavefront still reads the
    // other stage
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __syncthreads();
    uint4 c[4];
    uint32_t p[4][GPB];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      c[n] = cn[n];
#pragma unroll
      for (int g = 0; g < GPB; ++g) p[n][g] = pn[n][g];
    }
    if (s + 1 < nkb) {
      load_w(s + 1);
      load_a(s + 1);
    }
    if (GPB > 1)
#pragma unroll
      for (int n = 0; n < 4; ++n) transpose_words(c[n]);
    const _Float16* ta = smem + (s & 1) * STAGE + (wm * MT * 16 + r16) * 128;
#pragma unroll
    for (int g = 0; g < GPB; ++g) {
      float ratio[4];
      uint32_t nz[4];
      bool none = false;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const uint32_t w = p[n][g];
        nz[n] = (w >> 16) | (w & 0xffff0000u);
        none |= (w & 0x7fffu) == 0;
      }
      if (__any(none)) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if ((p[n][g] & 0x7fffu) == 0) {
            // nothing of this group counts: its codes and zero are 0
            nz[n] = 0;
#pragma unroll
            for (int j = 0; j < JG; ++j) {
              const int at = g * JG + j;
              if (at == 0) c[n].x = 0;
              if (at == 1) c[n].y = 0;
              if (at == 2) c[n].z = 0;
              if (at == 3) c[n].w = 0;
            }
          }
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float st = (p[n][g] & 0x7fffu) == 0 ? unit[n] : f16_lo(p[n][g]);
        // 1 / st to the last bit by one Newton step
        const float r = __builtin_amdgcn_rcpf(st);
        ratio[n] = unit[n] * fmaf(fmaf(-st, r, 1.0f), r, r);
        unit[n] = st;
      }
#pragma unroll
      for (int j = 0; j < JG; ++j) {
        const int at = g * JG + j;
        const int piece = GPB > 1 ? 4 * at + q4 : 4 * q4 + at;
        uint4 b[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) b[n] = dequant_word(word_of(c[n], at), nz[n]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint4 a = *(const uint4*)(ta + m * 2048 + 8 * (piece ^ r16));
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            if (j == 0)
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[m][n][r] *= ratio[n];
            acc[m][n] = mfma16<_Float16>(a, b[n], acc[m][n]);
          }
        }
      }
    }
  }
  __syncthreads();

  // epilogue, 32 tokens of the wavefront at a time through its own LDS: tokens
  // by columns, then eight columns of a token per lane
  float* const ep = (float*)smem + wave * 32 * kEpRow;
  const int tw = t0 + wm * MT * 16;
  constexpr int CW = GATED ? 32 : 64;  // outputs of the wavefront
  const int ob = rb + CW * wn;
#pragma unroll
  for (int h = 0; h < MT / 2; ++h) {
#pragma unroll
    for (int mm = 0; mm < 2; ++mm)
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          ep[(16 * mm + 4 * q4 + r) * kEpRow + 16 * n + r16] =
              acc[2 * h + mm][n][r] * (unit[n] * kCodeScale);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the wavefront's own writes
    asm volatile("" ::: "memory");
    constexpr int LPT = CW / 8;  // lanes per token
#pragma unroll
    for (int it = 0; it < 32 * LPT / 64; ++it) {
      const int tl = it * (64 / LPT) + lane / LPT, c8 = 8 * (lane % LPT);
      const int token = tw + 32 * h + tl, o = ob + c8;
      float v[8], u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = ep[tl * kEpRow + c8 + e];
        if (GATED) u[e] = ep[tl * kEpRow + 32 + c8 + e];
      }
      if (token >= N || o >= outs) continue;
      if (back) {
        const int x = back[token];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = ldexpf(v[e], x);
          if (GATED) u[e] = ldexpf(u[e], x);
        }
      }
      if (GATED) {
        if (pre) {
          store8(pre + (size_t)token * O + o, v, outs - o, (F & 7) == 0);
          store8(pre + (size_t)token * O + F + o, u, outs - o, (F & 7) == 0);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = act_value<ACT>(v[e], nullptr) * u[e];
      }
      store8(Y + (size_t)token * outs + o, v, outs - o, (outs & 7) == 0);
    }
    asm volatile("" ::: "memory");
  }
}

struct GemmPlan {
  size_t off_prm, off_a, off_back, bytes;
};
static GemmPlan gemm_plan(const W4Args& a) {
  GemmPlan p;
  size_t at = 0;
  p.off_prm = at;
  at += align256((size_t)a.O * (a.K / a.group) * 4);
  p.off_a = p.off_back = at;
  if (a.type == kBF16) {
    at += align256((size_t)a.N * a.K * 2);
    p.off_back = at;
    at += align256((size_t)a.N * 4);
  }
  p.bytes = at;
  return p;
}
size_t w4_gemm_workspace(const W4Args& a) { return gemm_plan(a).bytes; }

template <typename T, int GROUP, bool GATED, int ACT, int MT, typename TY>
static hipError_t launch(const W4Args& a, const GemmPlan& p, hipStream_t stream) {
  constexpr int BM = 32 * MT;
  const int64_t outs = GATED ? a.O / 2 : a.O;
  const int nt = (int)((a.N + BM - 1) / BM);
  const int no = (int)((outs + (GATED ? kBN / 2 : kBN) - 1) / (GATED ? kBN / 2 : kBN));
  const size_t lds = 2 * BM * 256 > kEpBytes ? 2 * BM * 256 : kEpBytes;
  auto* kernel = &k_w4_gemm<T, GROUP, GATED, ACT, MT, TY>;
  const hipError_t e = hipFuncSetAttribute((const void*)kernel,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  char* ws = (char*)a.ws;
  const bool bf = a.type == kBF16;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(nt * no)), dim3(512), lds, stream,
                     bf ? (const _Float16*)(ws + p.off_a) : (const _Float16*)a.in0,
                     bf ? (const int*)(ws + p.off_back) : nullptr, (int)a.N, (int)a.K, (int)a.O,
                     (const uint32_t*)a.qweight, (const uint32_t*)(ws + p.off_prm), (TY*)a.out0,
                     (T*)a.out1, nt, no);
  return hipGetLastError();
}

template <typename T, int GROUP, bool GATED, int ACT, typename TY>
static hipError_t by_tokens(const W4Args& a, const GemmPlan& p, hipStream_t stream) {
  if (a.N <= 128) return launch<T, GROUP, GATED, ACT, 4, TY>(a, p, stream);
  return launch<T, GROUP, GATED, ACT, 8, TY>(a, p, stream);
}

template <typename T, int GROUP>
static hipError_t by_op(W4Op op, const W4Args& a, const GemmPlan& p, hipStream_t stream) {
  if (op == kOpGated)
    return a.act == kActSilu ? by_tokens<T, GROUP, true, kActSilu, T>(a, p, stream)
                             : by_tokens<T, GROUP, true, kActGelu, T>(a, p, stream);
  return a.y_type == kF32 ? by_tokens<T, GROUP, false, 0, float>(a, p, stream)
                          : by_tokens<T, GROUP, false, 0, T>(a, p, stream);
}

template <typename T>
static hipError_t by_group(W4Op op, const W4Args& a, const GemmPlan& p, hipStream_t stream) {
  if (a.group == 128) return by_op<T, 128>(op, a, p, stream);
  if (a.group == 64) return by_op<T, 64>(op, a, p, stream);
  return by_op<T, 32>(op, a, p, stream);
}

hipError_t launch_w4_gemm(W4Op op, const W4Args& a, hipStream_t stream) {
  const GemmPlan p = gemm_plan(a);
  char* ws = (char*)a.ws;
  const int ng = (int)(a.K / a.group);
  hipLaunchKernelGGL(k_w4_params, dim3((unsigned)((a.O + 31) / 32), (unsigned)((ng + 31) / 32)),
                     dim3(256), 0, stream, (const uint16_t*)a.step16, (const uint16_t*)a.zero16,
                     (int)a.O, ng, (uint32_t*)(ws + p.off_prm));
  if (a.type == kBF16) {
    const hipError_t e = launch_rows_to_half(a.in0, a.type, a.N, a.K, a.K, ws + p.off_a,
                                             (int*)(ws + p.off_back), stream);
    if (e != hipSuccess) return e;
    return by_group<__bf16>(op, a, p, stream);
  }
  return by_group<_Float16>(op, a, p, stream);
}

}  // namespace awq
