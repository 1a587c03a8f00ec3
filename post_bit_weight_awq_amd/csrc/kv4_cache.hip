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
//
// A block takes one head of neighbouring tokens, a thread eight columns of one, G /
// 8 threads a group.  The codes of V pass through LDS, so that 16 tokens that fill
// a tile of the cache write (or read) its words in whole lines; a prompt's tokens
// do.  A code is rint of the product with 1 / step, which is within 2^-18 of the
// quotient, and where that lies so near a tie the quotient itself.  4095 tokens, 40
// heads of 128 in groups of 32 are 84 MB of rows and 26 MB of cache: gather, bound
// by these bytes, takes 23 us (4.7 TB/s); append, bound by VALU issue (about 25
// operations a value; 96 % of the busy cycles issue one, in groups of 128 too), 36 us (3.1
// TB/s).  A step of decoding (32 tokens, 8 heads) is a launch: 3.3 and 2.9 us.
#include "kv4_device.h"
#include "w4_internal.h"

namespace awq {

constexpr int kCacheThreads = 256;

template <int D>
struct CacheBlock {
  static constexpr int W = D / 8, kTokens = kCacheThreads / W;  // threads of a token's head
  int64_t t0;
  int head;
  // the thread's token and column block, and those whose word of V it moves
  int i, cb, vi, vcb;
  __device__ __forceinline__ CacheBlock(const Kv4& c, int heads)  // of a block
      : t0((int64_t)(grid_block() / (c.heads / heads)) * kTokens),
        head(grid_block() % (c.heads / heads) * heads), i(threadIdx.x / W),
        cb(threadIdx.x % W), vi(threadIdx.x % kTokens), vcb(threadIdx.x / kTokens) {}
};
// Token of a slot, -1 for none.
__device__ __forceinline__ int64_t slot_token(const Kv4& c, int32_t slot, int head) {
  return slot < 0 || (slot >> c.shift) >= c.pages
             ? -1
             : kv4_token(c, slot >> c.shift, head, slot & ((1 << c.shift) - 1));
}

typedef short short2v __attribute__((ext_vector_type(2)));
// Two 16-bit values as integers of the same order (and back: it is its own
// inverse): negative ones have their other bits turned.
__device__ __forceinline__ short2v sortable(uint32_t w) {
  const short2v x = __builtin_bit_cast(short2v, w);
  const short2v sign = x >> 15;
  return x ^ (sign & (short2v){0x7fff, 0x7fff});
}
__device__ __forceinline__ uint32_t sortable_bits(short a, short b) {
  return __builtin_bit_cast(uint32_t, sortable(__builtin_bit_cast(uint32_t, (short2v){a, b})));
}

// H heads one after another, all of whose values are requested first: with one a
// block of a prompt waits longer than it works (4095 tokens, 40 heads of 128,
// groups of 32: 40 us, 36 with four).
template <typename T, int D, int G, int H>
__global__ void __launch_bounds__(kCacheThreads)
k_kv4_append(Kv4 c, Kv4Rows rows, const int32_t* __restrict__ slots, int64_t tokens) {
  using B = CacheBlock<D>;
  constexpr int L = G / 8;  // threads of a group
  __shared__ uint32_t words[H][B::W][B::kTokens + 1];
  const B b(c, H);
  if (b.t0 >= tokens) return;
  const bool values = blockIdx.z;
  const int64_t t = b.t0 + b.i, vt = b.t0 + b.vi;
  uint4 raw[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    raw[h] = make_uint4(0, 0, 0, 0);
    if (t < tokens)
      raw[h] = *(const uint4*)((const T*)(values ? rows.v : rows.k) +
                               t * (values ? rows.v_token : rows.k_token) +
                               (b.head + h) * (values ? rows.v_head : rows.k_head) + 8 * b.cb);
  }
  const int32_t slot = t < tokens ? slots[t] : -1;
  const int32_t vslot = values && vt < tokens ? slots[vt] : -1;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t token = slot_token(c, slot, b.head + h);
    // least and largest as 16-bit integers of the same order, two at a time
    short2v least = sortable(raw[h].x), most = least;
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      const short2v x = sortable(word_of(raw[h], i));
      least = __builtin_elementwise_min(least, x);
      most = __builtin_elementwise_max(most, x);
    }
    short2v ends = {least.x < least.y ? least.x : least.y, (short)~(most.x > most.y ? most.x : most.y)};
#pragma unroll
    for (int s = 1; s < L; s *= 2)
      ends = __builtin_elementwise_min(
          ends, __builtin_bit_cast(short2v, __shfl_xor(__builtin_bit_cast(int, ends), s)));
    const uint32_t back = sortable_bits(ends.x, (short)~ends.y);
    constexpr short kInf = __is_same(T, _Float16) ? 0x7c00 : 0x7f80;
    // infinities and NaN lie behind all finite values
    const bool any = ends.x <= (short)~kInf || (short)~ends.y >= kInf;
    const float lo = med3(to_f32(__builtin_bit_cast(T, (uint16_t)back)), -65504.0f, 65504.0f);
    const float hi = med3(to_f32(__builtin_bit_cast(T, (uint16_t)(back >> 16))), -65504.0f, 65504.0f);
    float v[8];  // beyond fp16's range: a code at the end like that of its limit
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = to_f32(__builtin_bit_cast(T, (uint16_t)(word_of(raw[h], i >> 1) >> (16 * (i & 1)))));
    const _Float16 step16 = (_Float16)((hi - lo) / 15.0f), off16 = (_Float16)lo;
    const float step = (float)step16, off = (float)off16;
    uint32_t w = 0;
    if (step > 0.0f && !any) {
      const float inv = 1.0f / step;  // finite: step is 2^-24 or more
      float near = 0.0f;              // the largest distance from a code
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = (v[i] - off) * inv, r = __builtin_rintf(q);
        near = fmaxf(near, fabsf(q - r));
        w |= (uint32_t)med3(r, 0.0f, 15.0f) << (4 * i);
      }
      // quotients beyond the codes' range are clamped either way
      if (near > 0.5f - 0x1p-17f) {
        w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w |= (uint32_t)med3(__builtin_rintf((v[i] - off) / step), 0.0f, 15.0f) << (4 * i);
      }
    }
    if (token >= 0 && b.cb % L == 0) {
      const uint32_t p = any ? 0x7e000000u
                             : (uint32_t)__builtin_bit_cast(uint16_t, step16) |
                                   ((uint32_t)__builtin_bit_cast(uint16_t, off16) << 16);
      (values ? c.v_params : c.k_params)[token * (D / G) + b.cb / L] = p;
    }
    if (values)
      words[h][b.cb][b.i] = w;
    else if (token >= 0)
      c.k_codes[kv4_k_word<D>(token, b.cb)] = w;
  }
  if (!values) return;
  __syncthreads();
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t to = slot_token(c, vslot, b.head + h);
    if (to >= 0) c.v_codes[kv4_v_word<D>(to, b.vcb)] = words[h][b.vcb][b.vi];
  }
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kCacheThreads)
k_kv4_gather(Kv4 c, const int32_t* __restrict__ slots, T* __restrict__ k, T* __restrict__ v,
             int64_t tokens) {
  using B = CacheBlock<D>;
  constexpr int L = G / 8;
  __shared__ uint32_t words[B::W][B::kTokens + 1];
  const B b(c, 1);
  if (b.t0 >= tokens) return;
  const bool values = blockIdx.z;
  const int64_t t = b.t0 + b.i;
  const int64_t token = t < tokens ? slot_token(c, slots[t], b.head) : -1;
  uint32_t w = 0, p = 0;
  if (token >= 0) {
    p = (values ? c.v_params : c.k_params)[token * (D / G) + b.cb / L];
    if (!values) w = c.k_codes[kv4_k_word<D>(token, b.cb)];
  }
  if (values) {
    const int64_t vt = b.t0 + b.vi, from = vt < tokens ? slot_token(c, slots[vt], b.head) : -1;
    if (from >= 0) words[b.vcb][b.vi] = c.v_codes[kv4_v_word<D>(from, b.vcb)];
    __syncthreads();
    if (token >= 0) w = words[b.cb][b.i];
  }
  if (t >= tokens) return;
  uint32_t o[4] = {0, 0, 0, 0};
  if (token >= 0) {
    const float step = f16_lo(p), off = f16_hi(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the product is exact (4 by 11 bits): one rounding, then T's
      const T x = from_f32<T>(fmaf((float)((w >> (4 * i)) & 15u), step, off));
      o[i >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, x) << (16 * (i & 1));
    }
  }
  *(uint4*)((values ? v : k) + (t * c.heads + b.head) * D + 8 * b.cb) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename T, int D, int G>
static hipError_t run(bool append, const Kv4& c, const Kv4Rows& rows, int64_t tokens,
                      const int32_t* slots, void* k, void* v, hipStream_t stream) {
  constexpr int N = CacheBlock<D>::kTokens;
  const int64_t blocks = (tokens + N - 1) / N * c.heads;
  // four heads a block where that still leaves each unit four blocks
  if (append && c.heads % 4 == 0 && blocks >= 8 * kCUs)
    hipLaunchKernelGGL((k_kv4_append<T, D, G, 4>), grid_of(blocks / 4, 2), dim3(kCacheThreads), 0, stream,
                       c, rows, slots, tokens);
  else if (append)
    hipLaunchKernelGGL((k_kv4_append<T, D, G, 1>), grid_of(blocks, 2), dim3(kCacheThreads), 0, stream, c, rows, slots,
                       tokens);
  else
    hipLaunchKernelGGL((k_kv4_gather<T, D, G>), grid_of(blocks, 2), dim3(kCacheThreads), 0, stream, c, slots,
                       (T*)k, (T*)v, tokens);
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
