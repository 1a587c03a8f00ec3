// Writing keys and values into the 4-bit cache and reading them back.
//
// A group of G columns of a token's head is kept as
//   step = fp16((hi - lo) / 15), offset = fp16(lo),
//   code = clamp(rint((x - offset) / step), 0, 15), 0 where step is 0,
// all in binary32 with IEEE division, so a value is off by half a step and the
// roundings of step and offset.  The offset takes the place of the packed
// weights' zero: keys have channels that stand far from 0, where a zero of the
// fp16 step's multiples would leave fp16, and a group of equal values is kept
// as it is.  Finite values are brought into fp16's range first; a group with
// an infinity or a NaN has NaN as its offset and reads as NaN.
// One thread takes eight columns, G / 8 neighbouring threads a group.  Bound by
// the bytes moved (and by the launch for a step of decoding).
#include "kv4_device.h"

namespace awq {

template <typename T, int D, int G>
__global__ void __launch_bounds__(256)
k_kv4_append(Kv4 c, Kv4Rows rows, const int32_t* __restrict__ slots, int64_t threads) {
  constexpr int W = D / 8, L = G / 8;  // threads of a token's head and of a group
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= threads) return;  // a whole head's threads end together
  const bool values = blockIdx.y;
  const int cb = (int)(at % W);
  const int64_t row = at / W;
  const int head = (int)(row % c.heads);
  const int64_t t = row / c.heads;
  const int32_t slot = slots[t];
  if (slot < 0 || (slot >> c.shift) >= c.pages) return;
  const T* x = (const T*)(values ? rows.v : rows.k) +
               t * (values ? rows.v_token : rows.k_token) +
               head * (values ? rows.v_head : rows.k_head) + 8 * cb;
  const uint4 raw = *(const uint4*)x;
  float v[8];
  float lo = INFINITY, hi = -INFINITY;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint16_t h = (uint16_t)(word_of(raw, i >> 1) >> (16 * (i & 1)));
    v[i] = to_f32(__builtin_bit_cast(T, h));
    odd |= !(fabsf(v[i]) < INFINITY);
    v[i] = med3(v[i], -65504.0f, 65504.0f);
    lo = fminf(lo, v[i]);
    hi = fmaxf(hi, v[i]);
  }
  int any = odd;
#pragma unroll
  for (int s = 1; s < L; s *= 2) {
    lo = fminf(lo, __shfl_xor(lo, s));
    hi = fmaxf(hi, __shfl_xor(hi, s));
    any |= __shfl_xor(any, s);
  }
  const _Float16 step16 = (_Float16)((hi - lo) / 15.0f), off16 = (_Float16)lo;
  const float step = (float)step16, off = (float)off16;
  uint32_t w = 0;
  if (step > 0.0f && !any) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = med3(__builtin_rintf((v[i] - off) / step), 0.0f, 15.0f);
      w |= (uint32_t)q << (4 * i);
    }
  }
  const int64_t token = kv4_token(c, slot >> c.shift, head, slot & ((1 << c.shift) - 1));
  if (values)
    c.v_codes[kv4_v_word<D>(token, cb)] = w;
  else
    c.k_codes[kv4_k_word<D>(token, cb)] = w;
  if (cb % L == 0) {
    const uint32_t p = any ? 0x7e000000u
                           : (uint32_t)__builtin_bit_cast(uint16_t, step16) |
                                 ((uint32_t)__builtin_bit_cast(uint16_t, off16) << 16);
    (values ? c.v_params : c.k_params)[token * (D / G) + cb / L] = p;
  }
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(256)
k_kv4_gather(Kv4 c, const int32_t* __restrict__ slots, T* __restrict__ k, T* __restrict__ v,
             int64_t threads) {
  constexpr int W = D / 8, L = G / 8;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= threads) return;
  const bool values = blockIdx.y;
  const int cb = (int)(at % W);
  const int64_t row = at / W;
  const int head = (int)(row % c.heads);
  const int32_t slot = slots[row / c.heads];
  uint32_t o[4] = {0, 0, 0, 0};
  if (slot >= 0 && (slot >> c.shift) < c.pages) {
    const int64_t token = kv4_token(c, slot >> c.shift, head, slot & ((1 << c.shift) - 1));
    const uint32_t w = values ? c.v_codes[kv4_v_word<D>(token, cb)] : c.k_codes[kv4_k_word<D>(token, cb)];
    const uint32_t p = (values ? c.v_params : c.k_params)[token * (D / G) + cb / L];
    const float step = f16_lo(p), off = f16_hi(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the product is exact (4 by 11 bits): one rounding, then T's
      const T x = from_f32<T>(fmaf((float)((w >> (4 * i)) & 15u), step, off));
      o[i >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, x) << (16 * (i & 1));
    }
  }
  *(uint4*)((values ? v : k) + at * 8) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename T, int D, int G>
static hipError_t run(bool append, const Kv4& c, const Kv4Rows& rows, int64_t tokens,
                      const int32_t* slots, void* k, void* v, hipStream_t stream) {
  const int64_t threads = tokens * c.heads * (D / 8);
  const dim3 grid((unsigned)((threads + 255) / 256), 2);
  if (append)
    hipLaunchKernelGGL((k_kv4_append<T, D, G>), grid, dim3(256), 0, stream, c, rows, slots, threads);
  else
    hipLaunchKernelGGL((k_kv4_gather<T, D, G>), grid, dim3(256), 0, stream, c, slots, (T*)k, (T*)v,
                       threads);
  return hipGetLastError();
}
template <typename T>
static hipError_t by_size(bool append, const Kv4& c, const Kv4Rows& rows, int64_t tokens,
                          const int32_t* slots, void* k, void* v, hipStream_t stream) {
  if (c.dim == 128) {
    if (c.group == 128) return run<T, 128, 128>(append, c, rows, tokens, slots, k, v, stream);
    if (c.group == 64) return run<T, 128, 64>(append, c, rows, tokens, slots, k, v, stream);
    return run<T, 128, 32>(append, c, rows, tokens, slots, k, v, stream);
  }
  if (c.group == 64) return run<T, 64, 64>(append, c, rows, tokens, slots, k, v, stream);
  return run<T, 64, 32>(append, c, rows, tokens, slots, k, v, stream);
}

hipError_t launch_kv4_append(const Kv4& c, const Kv4Rows& rows, int type, int64_t tokens,
                             const int32_t* slots, hipStream_t stream) {
  return type == kF16 ? by_size<_Float16>(true, c, rows, tokens, slots, nullptr, nullptr, stream)
                      : by_size<__bf16>(true, c, rows, tokens, slots, nullptr, nullptr, stream);
}
hipError_t launch_kv4_gather(const Kv4& c, int64_t tokens, const int32_t* slots, void* k, void* v,
                             int type, hipStream_t stream) {
  return type == kF16 ? by_size<_Float16>(false, c, Kv4Rows{}, tokens, slots, k, v, stream)
                      : by_size<__bf16>(false, c, Kv4Rows{}, tokens, slots, k, v, stream);
}

}  // namespace awq
