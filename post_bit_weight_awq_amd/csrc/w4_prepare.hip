// What the tiled packed-weight kernels want before they run, in one launch:
// the group parameters in the order of their loads, and rows of activations or
// gradients in fp16.  Bound by HBM: each element is read once (a scaled row's
// second pass comes from L2) and written once (4096 tokens of a gated block's
// gradient, 2 x 13824 wide, 158 us, 5 TB/s).
#include "w4_internal.h"

namespace awq {

// 32 rows x 32 groups as (step, -zero 2^-9) fp16 pairs by group, of the zeros
// their high parts: prm[g * O + row]; parted[block]: whether any has a low one,
// and then lows[g * O + row], -low times the step.
__device__ __forceinline__ void product_params(const Prepare& a, int block) {
  __shared__ uint32_t tile[32][33];
  __shared__ float lows[32][33];
  const int nr = (a.O + 31) / 32, r0 = block % nr * 32, g0 = block / nr * 32;
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  int parted = 0;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    const int row = r0 + r + i, g = g0 + c;
    if (row < a.O && g < a.ng) {
      const size_t at = (size_t)row * a.ng + g;
      const ZeroParts z = split_zero<false>((float)a.zero16[at]);
      const uint32_t nz = neg_zero_pair((_Float16)z.high);
      parted |= z.low != 0.0f;
      lows[r + i][c] = -z.low * (float)a.step16[at];
      tile[r + i][c] = (uint32_t)__builtin_bit_cast(uint16_t, a.step16[at]) | (nz & 0xffff0000u);
    }
  }
  parted = __syncthreads_or(parted);
  if (threadIdx.x == 0) a.parted[block] = parted;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    const int row = r0 + c, g = g0 + r + i;
    if (row < a.O && g < a.ng) {
      ((uint32_t*)a.prm)[(size_t)g * a.O + row] = tile[c][r + i];
      if (parted) a.lows[(size_t)g * a.O + row] = lows[c][r + i];
    }
  }
}

// 64 packed rows (a step of the input gradient) x 32 groups:
// prm[(s * ng + g) * 128 + ..] as 64 halfs -zero 2^-9 and 64 halfs of the step,
// 0 for rows past the end; big[s * blocks of 32 groups + block]: whether a step
// is 128 or more (512 of them leave fp16) or a weight may leave it.
__device__ __forceinline__ void gradient_params(const Prepare& a, int block) {
  __shared__ uint32_t tile[64][33];
  const int gb = (a.ng + 31) / 32, s = block / gb, o0 = s * 64, g0 = block % gb * 32;
  int over = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = threadIdx.x + 256 * i;
    const int r = e >> 5, c = e & 31;
    uint32_t v = 0;
    if (o0 + r < a.O && g0 + c < a.ng) {
      const size_t at = (size_t)(o0 + r) * a.ng + g0 + c;
      v = (neg_zero_pair(a.zero16[at]) & 0xffffu) |
          ((uint32_t)__builtin_bit_cast(uint16_t, a.step16[at]) << 16);
      const float st = fabsf((float)a.step16[at]), z = fabsf((float)a.zero16[at]);
      over |= !(st < 128.0f && st * (z + 15.0f) < 65504.0f);
    }
    tile[r][c] = v;
  }
  over = __syncthreads_or(over);
  if (threadIdx.x == 0) a.big[block] = over;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = threadIdx.x + 256 * i;
    const int c = e >> 6, r = e & 63;
    if (g0 + c >= a.ng) continue;
    _Float16* p = (_Float16*)a.prm + ((size_t)s * a.ng + g0 + c) * 128;
    p[r] = __builtin_bit_cast(_Float16, (uint16_t)(tile[r][c] & 0xffffu));
    p[64 + r] = __builtin_bit_cast(_Float16, (uint16_t)(tile[r][c] >> 16));
  }
}

// The bits of n (8 or 1) 16-bit values from p; n is 8 where rows lie on
// 16-byte boundaries.
template <int N>
__device__ __forceinline__ void load_bits(const uint16_t* p, uint32_t (&v)[8]) {
  if constexpr (N == 8) {
    const uint4 w = *(const uint4*)p;
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = d[i] & 0xffffu;
      v[2 * i + 1] = d[i] >> 16;
    }
  } else {
    v[0] = *p;
  }
}
template <int N>
__device__ __forceinline__ void store_bits(uint16_t* p, const uint32_t (&v)[8]) {
  if constexpr (N == 8)
    *(uint4*)p = make_uint4(v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16),
                            v[6] | (v[7] << 16));
  else
    *p = (uint16_t)v[0];
}
template <typename T>
__device__ __forceinline__ float bits_to_f32(uint32_t b) {
  return to_f32(__builtin_bit_cast(T, (uint16_t)b));
}
template <typename T>
__device__ __forceinline__ uint32_t f32_to_bits(float v) {
  return __builtin_bit_cast(uint16_t, from_f32<T>(v));
}

// The sum over a group of a row's fp16 values, 0 where it is not finite, from
// eight values of each of the group's lanes.
__device__ __forceinline__ void sum_group(const Prepare& a, int row, int col, const uint32_t (&v)[8]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += bits_to_f32<_Float16>(v[i]);
  for (int d = 1; d < (1 << a.shift) / 8; d *= 2) s += __shfl_xor(s, d, 64);
  if ((col & ((1 << a.shift) - 1)) == 0)
    a.sums[(size_t)row * a.ng + (col >> a.shift)] = fabsf(s) < INFINITY ? s : 0.0f;
}

// One row.  GATED: dG = dH U act'(G), dU = dH act(G), each rounded once, into
// dpre; the row that follows is dpre's.  Then, where `out` is given, the row as
// fp16 with zeros behind it up to ld_out: fp16 as it is; bf16 times 2^e, e
// from the row's largest finite magnitude (which lands in [2^14, 2^15)) and
// back[row] = -e.  Values down to 2^-31 of the largest stay exact,
// smaller ones may be off by 2^-39 of it (half of fp16's last place, 2^-25).
// SUMS: also sums[row, g] of what `out` gets, or of an fp16 row left in place.
template <typename T, bool GATED, int N, bool SUMS>
__device__ __forceinline__ void prepare_row(const Prepare& a, int row) {
  constexpr bool SCALE = !__is_same(T, _Float16);
  __shared__ uint32_t red[4];
  const int cols = a.cols;
  uint32_t top = 0;  // largest finite magnitude, as bits
  auto look = [&](const uint32_t (&v)[8]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t b = v[i] & 0x7fffu;
      if (b < 0x7f80u && b > top) top = b;
    }
  };
  const uint16_t* src = (const uint16_t*)(GATED ? a.dpre : a.in0) + (size_t)row * cols;
  if constexpr (GATED) {
    const int F = cols / 2;
    const uint16_t* dh = (const uint16_t*)a.in0 + (size_t)row * F;
    const uint16_t* pre = (const uint16_t*)a.in1 + (size_t)row * cols;
    uint16_t* dpre = (uint16_t*)a.dpre + (size_t)row * cols;
    for (int c = threadIdx.x * N; c < F; c += 256 * N) {
      uint32_t d[8], g[8], u[8], dg[8], du[8];
      load_bits<N>(dh + c, d);
      load_bits<N>(pre + c, g);
      load_bits<N>(pre + F + c, u);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x = bits_to_f32<T>(g[i]), e = bits_to_f32<T>(d[i]);
        float slope;
        const float y = a.act == kActSilu ? act_value<kActSilu>(x, &slope)
                                          : act_value<kActGelu>(x, &slope);
        const float w = bits_to_f32<T>(u[i]);
        float z = e * w * slope;
        // dH U may leave binary32 where the slope, below 1 then, brings it back
        if (SCALE && !(fabsf(e * w) < INFINITY) && fabsf(e) < INFINITY && fabsf(w) < INFINITY)
          z = e * slope * w;
        dg[i] = f32_to_bits<T>(z);
        du[i] = f32_to_bits<T>(e * y);
      }
      store_bits<N>(dpre + c, dg);
      store_bits<N>(dpre + F + c, du);
      if (SCALE) {
        look(dg);
        look(du);
      }
    }
    if (!a.out) return;
  } else if constexpr (SCALE) {
    for (int c = threadIdx.x * N; c < cols; c += 256 * N) {
      uint32_t v[8];
      load_bits<N>(src + c, v);
      look(v);
    }
  }
  int e = 0;
  if constexpr (SCALE) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(red[0], red[1]), max(red[2], red[3]));
    // the largest is in [2^(x - 1), 2^x): x from frexp, also for subnormals
    int x = 0;
    if (top) (void)frexpf(__uint_as_float(top << 16), &x);
    e = top ? 15 - x : 0;
    if (threadIdx.x == 0) a.back[row] = -e;
  }
  if constexpr (SUMS && !SCALE) {
    // four pieces' loads in flight
    for (int c = threadIdx.x * N; c < cols; c += 4 * 256 * N) {
      uint4 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = *(const uint4*)(src + min(c + j * 256 * N, cols - N));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (c + j * 256 * N >= cols) break;
        uint32_t v[8];
        load_bits<N>((const uint16_t*)&w[j], v);
        sum_group(a, row, c + j * 256 * N, v);
      }
    }
    return;
  }
  uint16_t* dst = (uint16_t*)a.out + (size_t)row * a.ld_out;
  auto copy = [&](int from, int to) {
    for (int c = from + threadIdx.x * N; c < to; c += 256 * N) {
      uint32_t v[8];
      load_bits<N>(src + c, v);  // of dpre: what this thread has written
      if constexpr (SCALE)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = f32_to_bits<_Float16>(ldexpf(bits_to_f32<T>(v[i]), e));
      store_bits<N>(dst + c, v);
      if constexpr (SUMS) sum_group(a, row, c, v);
    }
  };
  if constexpr (GATED) {
    copy(0, cols / 2);
    copy(cols / 2, cols);
  } else {
    copy(0, cols);
  }
  for (int c = cols + threadIdx.x; c < a.ld_out; c += 256) dst[c] = 0;
}

// First the blocks of the parameters (PARAMS: 0 none, 1 the products', 2 the
// input gradient's), then one block per row.
template <typename T, bool GATED, int PARAMS>
__global__ void __launch_bounds__(256) k_w4_prepare(Prepare a) {
  const int block = (int)blockIdx.x;
  if (PARAMS && block < a.param_blocks) {
    if (PARAMS == 1)
      product_params(a, block);
    else
      gradient_params(a, block);
    return;
  }
  const int row = block - (PARAMS ? a.param_blocks : 0);
  // whole 16-byte pieces where both halves of a row begin on a boundary, as the
  // products' rows always do
  if constexpr (PARAMS == 1)
    prepare_row<T, GATED, 8, true>(a, row);
  else if ((a.cols & (GATED ? 15 : 7)) == 0)
    prepare_row<T, GATED, 8, false>(a, row);
  else
    prepare_row<T, GATED, 1, false>(a, row);
}

hipError_t launch_w4_prepare(const Prepare& p, int type, int params, bool gated, int64_t rows,
                             hipStream_t stream) {
  Prepare a = p;
  a.param_blocks = params == 0   ? 0
                   : params == 1 ? ((a.O + 31) / 32) * ((a.ng + 31) / 32)
                                 : ((a.O + 63) / 64) * ((a.ng + 31) / 32);
  const dim3 grid((unsigned)(a.param_blocks + rows));
  if (params == 1) {
    if (type == kF16)
      hipLaunchKernelGGL((k_w4_prepare<_Float16, false, 1>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((k_w4_prepare<__bf16, false, 1>), grid, dim3(256), 0, stream, a);
  } else if (params == 2) {
    if (type == kF16 && gated)
      hipLaunchKernelGGL((k_w4_prepare<_Float16, true, 2>), grid, dim3(256), 0, stream, a);
    else if (type == kF16)
      hipLaunchKernelGGL((k_w4_prepare<_Float16, false, 2>), grid, dim3(256), 0, stream, a);
    else if (gated)
      hipLaunchKernelGGL((k_w4_prepare<__bf16, true, 2>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((k_w4_prepare<__bf16, false, 2>), grid, dim3(256), 0, stream, a);
  } else {
    // rows of any 16-bit type as they are
    hipLaunchKernelGGL((k_w4_prepare<_Float16, false, 0>), grid, dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace awq
