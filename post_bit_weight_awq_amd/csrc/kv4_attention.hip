// Attention over the 4-bit cache: for every query t and head h
//   O[t, h] = sum_j p_j V[j],  p = softmax_j(scale Q[t, h] . K[j])
// over the keys j of t's sequence up to t's own place, K and V = step code +
// offset of their groups, never rounded.
//
// One pass with a running maximum m and sum l (binary32, powers of 2).  A
// wavefront takes 32 keys at a time for 16 rows; a row is one token and one of
// the heads that share a kv head.
//   * Scores: MFMA 16x16x32 of codes (keys by columns) with Q.  Two operations
//     per pair put a nibble at the top of the mantissa below the exponent of 16,
//     so the operand is 16 + code, exactly; the sums begin at -16 sum Q.  Steps
//     and offsets enter behind them, per group, in binary32.
//   * A lane then holds keys 4 q .. 4 q + 3 of both tiles of 16 for one row:
//     as the second operand of O^T = V^T P^T these are its eight of 32 keys, if
//     V's codes are read for the same keys.  So P never leaves its lane.  Eight
//     words of V hold eight columns of eight keys: byte permutes pair the keys
//     and each nibble position is another tile of columns; no transpose.
//   * P step, the operand, is held as two bf16 parts (16 bits): in one, or in
//     fp16, it would add as much error as the output's rounding or leave the
//     type's range.  With at most 8 rows the parts lie in lanes r and r + 8 of
//     one MFMA.  -16 of V's codes is taken back from the same rounded parts (one
//     more MFMA), so a part's error meets the code and not 16 + code.  The
//     offsets' part, sum P offset, is summed per lane.
// Single tokens (k_kv4_decode): a block of four wavefronts takes 16 rows, each
// wavefront every fourth 32 keys through two stages of LDS of its own, filled by
// direct loads; they are joined through LDS.  A long axis is split over blocks
// and k_kv4_join joins the splits in order.  Bound by the stream of codes on long
// caches (64 ragged sequences of up to 4096 keys, 40 heads of 128: 182 us, 4.4
// TB/s, with 82 % of the busy cycles issuing vector operations; with the tiles in
// registers, at half the wavefronts in flight, 200), by the way to the first keys and
// the join on short ones (one sequence of 777: 10.3 us).  Heads of 128 in groups of 64
// take 198 us and in groups of 32 257 (4.3 and 3.7 TB/s): more parameters to work
// off, and in groups of 32 four to eight registers are spilled, whose reload in a tile
// waits for the stages asked for ahead as well.
// Runs of tokens (k_kv4_chunk): a block of eight wavefronts takes 128 rows; they
// prepare a tile's operands in LDS together, each an eighth.  Bound by VALU issue
// (about 175 vector operations for a tile's 26 MFMAs: 62 % of the busy cycles issue one,
// in 35 % the matrix units work) and the barrier of each tile and, with few sequences,
// by the longest one: 4 x 256 to 512 tokens behind 512 to 4096 keys, 32
// heads on 8: 149 us, 411 TFLOP/s, 16 such sequences 458 us, 513 TFLOP/s; heads of 128
// in groups of 64 215 and 725 us, of 32 289 and 985: their registers leave one block a
// unit.  (On the card where parts took 165 us, whole units: 200 us; each wavefront by
// itself, for two row tiles, then 268; four wavefronts of two row tiles 204; of 64 rows
// 197, and 16 sequences 509 for 464; products a tile ahead 255.)
#include "kv4_device.h"
#include "w4_internal.h"

namespace awq {

struct AttnArgs {
  Kv4 c;
  const void* q;
  void* out;
  int heads, per_kv;  // query heads, and those that share a kv head
  int64_t q_token, q_head;
  int tokens, seqs, per_seq;
  const int32_t *starts, *table, *lens;
  float scale, slack;  // scale: |scale| log2(e) (bf16: times kUnit); slack: 8 / scale
  int flip;            // the scale is negative: Q changes sign
  int splits, per;    // blocks of a unit, the keys of each
  uint32_t units;     // tiles of rows over all sequences, by kv heads
  int rows;           // of a tile that k_kv4_join looks at
  float* parts;  // [unit][split][row][D + 4]: the sums, maximum, sum of weights
};

// Rows row0 .. of one sequence and kv head, `rows` of them in the sequence.
struct Unit {
  int seq, head, first, run, row0, rows, len;
};
// Tile t of R rows.  Ragged runs: sequence s owns the tiles from
// floor(starts[s] per_kv / R) + s on, which leaves room for all of its own.
template <int R>
__device__ __forceinline__ Unit unit_of(const AttnArgs& a, int tile, int head) {
  Unit u;
  u.head = head;
  if (a.starts == nullptr) {
    const int per = (a.per_kv + R - 1) / R;
    u.seq = tile / per;
    u.first = u.seq;
    u.run = 1;
    u.row0 = (tile - u.seq * per) * R;
  } else {
    auto start = [&](int s) { return min(max(a.starts[s], 0), a.tokens); };
    auto base = [&](int s) { return (int)((int64_t)start(s) * a.per_kv / R) + s; };
    int lo = 0, hi = a.seqs;  // base(lo) <= tile < base(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (base(mid) <= tile)
        lo = mid;
      else
        hi = mid;
    }
    u.seq = lo;
    u.first = start(lo);
    u.run = max(start(lo + 1) - u.first, 0);
    // the last rows, which see the most keys, begin first
    const int at = max(tile - base(lo), 0), tiles = (u.run * a.per_kv + R - 1) / R;
    u.row0 = (at < tiles ? tiles - 1 - at : at) * R;
  }
  u.rows = u.run * a.per_kv;
  u.len = min(max(a.lens[u.seq], 0), a.per_seq << a.c.shift);
  return u;
}

// The keys of a unit: `end` that its last row sees, in parts of `per` each.
// One part alone goes to the output, more meet in the join.
struct Keys {
  int end, per;
  __device__ __forceinline__ bool one() const { return end <= per; }
  __device__ __forceinline__ int parts() const { return (end + per - 1) / per; }
};
template <int R>
__device__ __forceinline__ Keys keys_of(const AttnArgs& a, const Unit& u) {
  constexpr int kStep = R == 16 ? 128 : 32;  // what a block takes at a time
  Keys k;
  k.end = min(max(u.len - u.run + (min(u.row0 + R, u.rows) - 1) / a.per_kv + 1, 0), u.len);
  k.per = max(((k.end + a.splits - 1) / a.splits + kStep - 1) & -kStep, a.per);
  return k;
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}

// What a wavefront keeps of 16 rows: lane l has row l % 16.
template <int D, int G>
struct Rows {
  static constexpr int J = D / 32, NG = D / G, JG = G / 32, N = D / 16, TG = G / 16;
  uint4 q[J];
  float qs[NG];  // sum of Q over a group
  float m, l, off[NG];
  floatx4 o[N];   // O^T: tile n, columns 4 (l / 16) + r, see column()
  floatx4 c[NG];  // -16 sum of the operand P step
  int lim;        // keys that the row sees
};

// Column of register r of tile n in lane group q: the word 4 q + r of a group
// of 16 (8, 4) words, which gives 8 (4, 2) of its nibbles to as many tiles.
template <int G>
__device__ __forceinline__ int column(int n, int i) {
  constexpr int TG = G / 16, WG = G / 8;
  return (n / TG) * G + 8 * (i % WG) + TG * (i / WG) + n % TG;
}

// Two bf16 values in units of 2^32: any finite query is then below 2^96, and
// neither 16 + code times a row's sum nor a score (codes 15 and steps and offsets of
// fp16's largest: below 2^126) leaves binary32.  A power of two changes no bit above
// 2^-94; what is cut below costs less than 2^-34 of a weight at the largest scale.
constexpr float kUnit = 0x1p32f;
__device__ __forceinline__ uint32_t lower(uint32_t w) {
  return __builtin_amdgcn_perm(__float_as_uint(__uint_as_float(w & 0xffff0000u) * (1.0f / kUnit)),
                               __float_as_uint(__uint_as_float(w << 16) * (1.0f / kUnit)), 0x07060302u);
}

// Returns the keys that all 16 rows see.
template <typename T, int D, int G>
__device__ __forceinline__ int load_rows(const AttnArgs& a, const Unit& u, int row0, int lane, Rows<D, G>& w) {
  using R = Rows<D, G>;
  const uint32_t sign = a.flip ? 0x80008000u : 0u;
  const int r16 = lane & 15, q4 = lane >> 4;
  const int row = min(row0 + r16, u.rows - 1);
  const int t = row / a.per_kv;
  const T* p = (const T*)a.q + (int64_t)(u.first + t) * a.q_token +
               (int64_t)(u.head * a.per_kv + row - t * a.per_kv) * a.q_head;
  w.lim = min(max(u.len - u.run + t + 1, 0), u.len);
#pragma unroll
  for (int j = 0; j < R::J; ++j) {
    uint4 v = *(const uint4*)(p + 32 * j + 8 * q4);
    v.x ^= sign, v.y ^= sign, v.z ^= sign, v.w ^= sign;
    if constexpr (!__is_same(T, _Float16)) v.x = lower(v.x), v.y = lower(v.y), v.z = lower(v.z), v.w = lower(v.w);
    // columns 0 4, 1 5, 2 6, 3 7, as the words' nibbles come
    w.q[j] = make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u),
                        __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                        __builtin_amdgcn_perm(v.w, v.y, 0x05040100u),
                        __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
  }
#pragma unroll
  for (int g = 0; g < R::NG; ++g) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < R::JG; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        s += to_f32(
            __builtin_bit_cast(T, (uint16_t)(word_of(w.q[g * R::JG + j], i >> 1) >> (16 * (i & 1)))));
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    w.qs[g] = s;
    w.off[g] = 0.0f;
    w.c[g] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  w.m = -INFINITY;
  w.l = 0.0f;
#pragma unroll
  for (int n = 0; n < R::N; ++n) w.o[n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  int low = w.lim;
#pragma unroll
  for (int s = 1; s < 16; s *= 2) low = min(low, __shfl_xor(low, s));
  return __builtin_amdgcn_readfirstlane(low);
}

// First of the 16 keys from `key` on, which lie in one page.
__device__ __forceinline__ int64_t key_token(const Kv4& c, int page, int head, int key) {
  return kv4_token(c, max(page, 0), head, key & ((1 << c.shift) - 1));
}
// An address in scalar registers: lanes add 32 bits.
__device__ __forceinline__ const char* uniform(const void* p) {
  const uint64_t v = (uint64_t)p;
  return (const char*)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}
// Codes and parameters of 32 keys in a wavefront's own LDS, moved there by
// direct loads: they are in flight for two tiles' time and cost no registers.
template <int D, int G>
struct Stage {
  static constexpr int NG = D / G, kCodes = 32 * D / 2, kParams = 32 * NG * 4;
  static constexpr int kK = 0, kV = kCodes, kKp = 2 * kCodes, kVp = kKp + kParams;
  static constexpr int kBytes = kVp + kParams;
  static constexpr int kLoads = (D == 128 ? 4 : 2) + NG;
};
// Direct loads from each lane's own address.
__device__ __forceinline__ void dma16_from(const char* p, uint32_t l) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(p), "{m0}"(l) : "memory");
}
__device__ __forceinline__ void dma4_from(const char* p, uint32_t l) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" : : "v"(p), "{m0}"(l) : "memory");
}
template <int D, int G>
__device__ __forceinline__ void load_stage(const Kv4& c, const int (&page)[2], int head, int key, uint32_t lane,
                                           uint32_t lds) {
  using S = Stage<D, G>;
  const char *k[2], *v[2], *kp[2], *vp[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t token = key_token(c, page[u], head, key + 16 * u);
    k[u] = uniform(c.k_codes + token * (D / 8));
    v[u] = uniform(c.v_codes + token * (D / 8));
    kp[u] = uniform(c.k_params + token * S::NG);
    vp[u] = uniform(c.v_params + token * S::NG);
  }
  if constexpr (D == 128) {
    // lane l fetches what it will read: 16 bytes l % 16, l / 16 of the 16 x 64
    const uint32_t at = (lane & 15) * 64 + (lane >> 4) * 16;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      dma16(k[u], at, lds + S::kK + 1024 * u);
      dma16(v[u], at, lds + S::kV + 1024 * u);
    }
  } else {
    const uint32_t at = (lane & 31) * 16;  // twice 512 bytes as they lie
    dma16_from((lane & 32 ? k[1] : k[0]) + at, lds + S::kK);
    dma16_from((lane & 32 ? v[1] : v[0]) + at, lds + S::kV);
  }
  if constexpr (S::NG == 1) {
    const char* x = lane & 32 ? (lane & 16 ? vp[1] : vp[0]) : lane & 16 ? kp[1] : kp[0];
    dma4_from(x + 4 * (lane & 15), lds + S::kKp);
  } else if constexpr (S::NG == 2) {
    dma4_from((lane & 32 ? kp[1] : kp[0]) + 4 * (lane & 31), lds + S::kKp);
    dma4_from((lane & 32 ? vp[1] : vp[0]) + 4 * (lane & 31), lds + S::kVp);
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      dma4(kp[u], 4 * lane, lds + S::kKp + 256 * u);
      dma4(vp[u], 4 * lane, lds + S::kVp + 256 * u);
    }
  }
}
// Parameters of keys 4 q .. 4 q + 3 of both 16: [key][group].
template <int NG>
__device__ __forceinline__ void read_params(const char* base, uint32_t q4, uint32_t (&p)[2][4 * NG]) {
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint4 y = *(const uint4*)(base + 64 * NG * u + 16 * NG * q4 + 16 * g);
      p[u][4 * g] = y.x, p[u][4 * g + 1] = y.y, p[u][4 * g + 2] = y.z, p[u][4 * g + 3] = y.w;
    }
}

// The mask of a nibble below the exponent and the exponent of 16, for T's
// pairs, in a scalar and a vector register whose values the compiler does not
// see: "and, or" is then one operation (it takes no constants, and one scalar).
template <typename T>
struct Sixteen {
  uint32_t mask, exponent;
  __device__ __forceinline__ Sixteen() {
    if constexpr (__is_same(T, _Float16)) {
      asm("s_mov_b32 %0, 0x03c003c0" : "=s"(mask));
      asm("v_mov_b32 %0, 0x4c004c00" : "=v"(exponent));
    } else {
      asm("s_mov_b32 %0, 0x00780078" : "=s"(mask));
      asm("v_mov_b32 %0, 0x41804180" : "=v"(exponent));
    }
  }
  // Nibble n (0 to 3) of both halves of w as 16 + code.
  __device__ __forceinline__ uint32_t pair(uint32_t w, int n) const {
    constexpr int up = __is_same(T, _Float16) ? 6 : 3;
    const int by = up - 4 * n;
    return ((by >= 0 ? w << by : w >> -by) & mask) | exponent;
  }
  // Eight nibbles: pairs 0 4, 1 5, 2 6, 3 7.
  __device__ __forceinline__ uint4 word(uint32_t w) const {
    return make_uint4(pair(w, 0), pair(w, 1), pair(w, 2), pair(w, 3));
  }
};

// Scores of 32 keys, in units of the scale and less the row's maximum so far, in
// two steps: the groups' products, whose sums begin at -16 sum Q, which takes the
// codes' 16 back, and what steps and offsets make of them.  The maximum is taken
// off before the scale: its own product with it would be rounded, by more than
// exp2 holds where scores are beyond 2^30.  kf(u, j): columns 32 j .. of keys 16 u ..
template <typename T, int D, int G, typename KF>
__device__ __forceinline__ void products(const Rows<D, G>& w, KF kf, floatx4 (&acc)[2][D / G]) {
  using R = Rows<D, G>;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int g = 0; g < R::NG; ++g) {
      const float z = -16.0f * w.qs[g];
      acc[u][g] = floatx4{z, z, z, z};
#pragma unroll
      for (int j = 0; j < R::JG; ++j)
        acc[u][g] = mfma16<T>(kf(u, g * R::JG + j), w.q[g * R::JG + j], acc[u][g]);
    }
}
template <int D, int G>
__device__ __forceinline__ void scores(const Rows<D, G>& w, const uint32_t (&p)[2][4 * (D / G)],
                                       const floatx4 (&acc)[2][D / G], float (&s)[8]) {
  constexpr int NG = D / G;
  const float base = w.m == -INFINITY ? 0.0f : -w.m;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t x = p[u][r * NG + g];
        float& y = s[4 * u + r];
        y = fmaf(f16_hi(x), w.qs[g], g == 0 ? base : y);  // one operation of mixed types
        y = fmaf(f16_lo(x), acc[u][g][r], y);
      }
}

// Whether a lane's row sees its key i of the 32 from `key` on.
__device__ __forceinline__ bool sees(int lim, const int (&page)[2], int key, int q4, int i) {
  return page[i >> 2] >= 0 && key + 16 * (i >> 2) + 4 * q4 + (i & 3) < lim;
}
// The scores of keys that are not seen become -inf, their values' parameters 0,
// whatever lies there.
template <int N>
__device__ __forceinline__ void hide(int lim, const int (&page)[2], int key, int q4, float (&s)[8],
                                     uint32_t (&p)[2][N]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool v = sees(lim, page, key, q4, i);
    s[i] = v ? s[i] : -INFINITY;
#pragma unroll
    for (int g = 0; g < N / 4; ++g) {
      uint32_t& x = p[i >> 2][(i & 3) * (N / 4) + g];
      x = v ? x : 0u;
    }
  }
}

// Scores to weights.  The maximum follows only when a score passes it by more
// than 2^8 in the weights (which binary32 and bf16 hold), so most tiles need no
// exchange between the lane groups.
template <int D, int G>
__device__ __forceinline__ void weigh(Rows<D, G>& w, float scale, float slack, float (&s)[8]) {
  using R = Rows<D, G>;
  float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
  const bool first = w.m == -INFINITY;
  if (__any(top > (first ? -INFINITY : slack))) {
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float up = first ? (top == -INFINITY ? 0.0f : top) : fmaxf(top, 0.0f);
    const float a = first ? (top == -INFINITY ? 1.0f : 0.0f) : __builtin_amdgcn_exp2f(-up * scale);
    w.m = first ? top : w.m + up;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] -= up;
    w.l *= a;
#pragma unroll
    for (int g = 0; g < R::NG; ++g) {
      w.off[g] *= a;
#pragma unroll
      for (int r = 0; r < 4; ++r) w.c[g][r] *= a;
    }
#pragma unroll
    for (int n = 0; n < R::N; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) w.o[n][r] *= a;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = __builtin_amdgcn_exp2f(s[i] * scale);
    w.l += s[i];
  }
}

// P step of a group as two bf16 parts; PAIR: lanes 8 to 15 take the second.
struct Parts {
  uint4 hi, lo;
};
template <int NG, bool PAIR>
__device__ __forceinline__ Parts parts_of(const uint32_t (&p)[2][4 * NG], int g, const float (&s)[8], float& off,
                                          int r16) {
  float ps[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = p[i >> 2][(i & 3) * NG + g];
    ps[i] = fmaf(s[i], f16_lo(x), 0.0f);
    off = fmaf(s[i], f16_hi(x), off);
  }
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_bf16(ps[2 * i], ps[2 * i + 1]);
    l[i] = pack_bf16(ps[2 * i] - __uint_as_float(h[i] << 16),
                     ps[2 * i + 1] - __uint_as_float(h[i] & 0xffff0000u));
    if (PAIR) h[i] = r16 & 8 ? l[i] : h[i];
  }
  return {make_uint4(h[0], h[1], h[2], h[3]), make_uint4(l[0], l[1], l[2], l[3])};
}

// Adds the values of 32 keys, a group of columns after another.  vf.group(g),
// then vf(n): tile n of the group's columns.
template <int D, int G, bool PAIR, typename VF>
__device__ __forceinline__ void gather(Rows<D, G>& w, const uint32_t (&p)[2][4 * (D / G)], const float (&s)[8],
                                       VF& vf, int r16) {
  using R = Rows<D, G>;
  const uint4 ones = make_uint4(0xc180c180u, 0xc180c180u, 0xc180c180u, 0xc180c180u);  // -16
#pragma unroll
  for (int g = 0; g < R::NG; ++g) {
    vf.group(g);
    const Parts x = parts_of<R::NG, PAIR>(p, g, s, w.off[g], r16);
    w.c[g] = mfma16<__bf16>(ones, x.hi, w.c[g]);
    if (!PAIR) w.c[g] = mfma16<__bf16>(ones, x.lo, w.c[g]);
#pragma unroll
    for (int n = 0; n < R::TG; ++n) {
      const uint4 b = vf(n);
      floatx4& o = w.o[g * R::TG + n];
      o = mfma16<__bf16>(b, x.hi, o);
      if (!PAIR) o = mfma16<__bf16>(b, x.lo, o);
      if (VF::kTight && (n & 1)) __builtin_amdgcn_sched_barrier(0);  // few codes wait at a time
    }
  }
}

// A lane's words of V (see column()) from a stage: eight keys' words, paired,
// and of these the halves or bytes that hold the lane's columns.
template <int D, int G>
struct ValueWords {
  static constexpr int WG = G / 8, HG = G == 128 ? 2 : 1;
  static constexpr bool kTight = true;
  const char* base;
  Sixteen<__bf16> v16;
  int lane;
  uint32_t h[HG][4];
  __device__ __forceinline__ void group(int g) {
    const uint32_t r16 = lane & 15, q4 = lane >> 4, word = g * WG + r16 % WG;
    uint4 x[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      x[u] = D == 128 ? *(const uint4*)(base + 1024 * u + 16 * (word + 16 * q4))
                      : *(const uint4*)(base + 512 * u + 64 * word + 16 * q4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = i & 1 ? x[i >> 1].z : x[i >> 1].x, b = i & 1 ? x[i >> 1].w : x[i >> 1].y;
      if constexpr (G == 128) {
        h[0][i] = __builtin_amdgcn_perm(b, a, 0x05040100u);
        h[1][i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
      } else {
        h[0][i] = __builtin_amdgcn_perm(
            b, a, G == 64 ? (r16 & 8 ? 0x07060302u : 0x05040100u) : 0x0c040c00u + (r16 >> 2) * 0x00010001u);
      }
    }
  }
  __device__ __forceinline__ uint4 operator()(int n) const {
    const uint32_t(&p)[4] = h[HG > 1 ? n >> 2 : 0];
    return make_uint4(v16.pair(p[0], n & 3), v16.pair(p[1], n & 3), v16.pair(p[2], n & 3), v16.pair(p[3], n & 3));
  }
};

// A sequence's pages, 64 entries of its table at a time, one per lane: a load
// for each tile would be waited for with the tile's reads of LDS.
struct Pages {
  const int32_t* table;
  int len, shift, first, held;
  int64_t pages;
  __device__ __forceinline__ Pages(const AttnArgs& a, const Unit& u)
      : table(a.table + (int64_t)u.seq * a.per_seq), len(u.len), shift(a.c.shift), first(-64), held(0),
        pages(a.c.pages) {}
  // The pages of keys key .. key + 31; -1 where there is none or a bad one.
  __device__ __forceinline__ void of(int key, int lane, int (&page)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = key + 16 * u, i = k >> shift;
      page[u] = -1;
      if (k >= len) continue;
      if (i - first >= 64) {  // keys rise
        first = i;
        const int at = i + lane, last = (len - 1) >> shift;
        const int p = table[min(at, last)];
        held = p < pages ? max(p, -1) : -1;
      }
      page[u] = __builtin_amdgcn_readlane(held, i - first);
    }
  }
};

// Keys k0, k0 + stride, .. below k1 (32 at a time) for 16 rows, through two
// stages from `lds` on.
template <typename T, int D, int G, bool PAIR>
__device__ __forceinline__ void walk(const AttnArgs& a, const Unit& u, Rows<D, G>& w, int low,
                                     int k0, int k1, int stride, int lane, const char* smem) {
  using S = Stage<D, G>;
  if (k0 >= k1) return;
  Pages pages(a, u);
  const uint32_t lds = (uint32_t)(uintptr_t)smem;
  const float scale = a.scale, slack = a.slack;
  const Sixteen<T> k16;
  const uint32_t r16 = lane & 15, q4 = (uint32_t)lane >> 4;
  int page[2], next[2], after[2];
  pages.of(k0, lane, page);
  pages.of(k0 + stride, lane, next);
  load_stage<D, G>(a.c, page, u.head, k0, lane, lds);
  if (k0 + stride < k1) load_stage<D, G>(a.c, next, u.head, k0 + stride, lane, lds + S::kBytes);
  pages.of(k0 + 2 * stride, lane, after);
  int at = 0;
  for (int key = k0; key < k1; key += stride) {
    if (key + stride < k1)
      wait_vm<S::kLoads>();
    else
      wait_vm<0>();
    asm volatile("" ::: "memory");
    const char* st = smem + at;
    float s[8];
    uint32_t p[2][4 * S::NG];
    floatx4 acc[2][S::NG];
    products<T>(w, [&](int v, int j) {
      const char* x = st + S::kK + (D == 128 ? 1024 * v + 16 * lane : 512 * v + 32 * r16 + 8 * q4);
      return k16.word(*(const uint32_t*)(x + 4 * j));
    }, acc);
    read_params<S::NG>(st + S::kKp, q4, p);
    scores(w, p, acc, s);
    read_params<S::NG>(st + S::kVp, q4, p);
    if (key + 32 > low || (page[0] | page[1]) < 0) hide(w.lim, page, key, q4, s, p);
    weigh(w, scale, slack, s);
    __builtin_amdgcn_sched_barrier(0);
    ValueWords<D, G> vf{st + S::kV, {}, lane};
    gather<D, G, PAIR>(w, p, s, vf, r16);
    // the stage has been read
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (key + 2 * stride < k1) load_stage<D, G>(a.c, after, u.head, key + 2 * stride, lane, lds + at);
    at ^= S::kBytes;
#pragma unroll
    for (int i = 0; i < 2; ++i) page[i] = next[i], next[i] = after[i];
    pages.of(key + 3 * stride, lane, after);
  }
}

// The lane groups' shares of l and the offsets, and the parts of O together.
template <int D, int G>
__device__ __forceinline__ void finish_sums(Rows<D, G>& w) {
  w.l += __shfl_xor(w.l, 16);
  w.l += __shfl_xor(w.l, 32);
#pragma unroll
  for (int g = 0; g < D / G; ++g) {
    w.off[g] += __shfl_xor(w.off[g], 16);
    w.off[g] += __shfl_xor(w.off[g], 32);
#pragma unroll
    for (int n = 0; n < G / 16; ++n) w.o[g * (G / 16) + n] += w.c[g];
  }
}

template <typename T, int D>
__device__ __forceinline__ T* out_row(const AttnArgs& a, const Unit& u, int row) {
  const int t = row / a.per_kv;
  return (T*)a.out + ((int64_t)(u.first + t) * a.heads + u.head * a.per_kv + row - t * a.per_kv) * D;
}

constexpr int kDecodeRows = 16, kDecodeWaves = 4;

template <typename T, int D, int G, bool PAIR>
__global__ void __launch_bounds__(64 * kDecodeWaves, D / G == 4 ? 3 : 4)
k_kv4_decode(AttnArgs a) {
  using S = Stage<D, G>;
  constexpr int P = D + 4;  // of a row in LDS
  constexpr int ROWS = PAIR ? 8 : 16;
  constexpr int kRing = 2 * S::kBytes, kSums = ROWS * P * 4;
  // a wavefront's stages, then its sums
  constexpr int kOwn = kRing > kSums ? kRing : kSums;
  __shared__ __attribute__((aligned(16))) char smem[kDecodeWaves * kOwn];
  __shared__ float sm[kDecodeWaves][16], sl[kDecodeWaves][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t block = grid_block(), split = block % a.splits, id = block / a.splits;
  if (id >= a.units) return;
  const Unit u = unit_of<kDecodeRows>(a, id / a.c.heads, id % a.c.heads);
  if (u.row0 >= u.rows) return;
  const int count = min(u.rows - u.row0, 16);
  const Keys keys = keys_of<kDecodeRows>(a, u);
  const int from = (int)min((int64_t)split * keys.per, (int64_t)keys.end), to = min(from + keys.per, keys.end);
  Rows<D, G> w;
  // PAIR: rows of lanes 8 to 15 are those of 0 to 7
  const int low = load_rows<T>(a, u, PAIR ? u.row0 - (lane & 8) : u.row0, lane, w);
  if (split && from >= keys.end) return;  // not before Q is on its way
  walk<T, D, G, PAIR>(a, u, w, low, from + 32 * wave, to, 32 * kDecodeWaves, lane, smem + wave * kOwn);
  finish_sums(w);
  const int r16 = lane & 15, q4 = lane >> 4;
  if constexpr (PAIR) {
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r)  // of lane l ^ 8
        w.o[n][r] += __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(w.o[n][r]), 0x128, 0xf, 0xf, false));
  }
  if (q4 == 0) {
    sm[wave][r16] = w.m;
    sl[wave][r16] = w.l;
  }
  if (r16 < count) {
    float* so = (float*)(smem + wave * kOwn) + r16 * P;
#pragma unroll
    for (int n = 0; n < D / 16; n += 2)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *(float2*)(so + column<G>(n, 4 * q4 + r)) =
            make_float2(w.o[n][r] + w.off[n / (G / 16)], w.o[n + 1][r] + w.off[n / (G / 16)]);
  }
  __syncthreads();
  // a thread takes eight columns of a row
  for (int e = tid; e < count * (D / 8); e += 64 * kDecodeWaves) {
    const int row = e / (D / 8), c = 8 * (e % (D / 8));
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kDecodeWaves; ++i) m = fmaxf(m, sm[i][row]);
    float l = 0.0f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kDecodeWaves; ++i) {
      // a wavefront without keys has -inf, 0 and zeros; one with NaN sums keeps them
      const float f = sm[i][row] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((sm[i][row] - m) * a.scale);
      const float* so = (const float*)(smem + i * kOwn) + row * P + c;
      l = fmaf(f, sl[i][row], l);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = fmaf(f, so[k], v[k]);
    }
    if (!keys.one()) {
      float* p = a.parts + ((int64_t)block * 16 + row) * (D + 4);
      *(float4*)(p + c) = make_float4(v[0], v[1], v[2], v[3]);
      *(float4*)(p + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
      if (c == 0) {
        p[D] = m;
        p[D + 1] = l;
      }
    } else {
      const float f = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= f;
      store8(out_row<T, D>(a, u, u.row0 + row) + c, v, 8, true);
    }
  }
}

// Single tokens: a row per block: thread groups take every 256 / (D / 8)-th part
// each, with four in flight, and are joined through LDS, all in fixed order.
template <typename T, int D>
__global__ void __launch_bounds__(256)
k_kv4_join(AttnArgs a) {
  constexpr int C = D / 8, N = 256 / C;  // threads of a row's columns, groups
  __shared__ float sm[128], sl[N], so[N][D + 4];
  const int tid = threadIdx.x, c = 8 * (tid % C), part = tid / C;
  const int row = blockIdx.x % a.rows;
  const int id = blockIdx.x / a.rows;
  constexpr int R = kDecodeRows;
  const Unit u = unit_of<R>(a, id / a.c.heads, id % a.c.heads);
  if (u.row0 + row >= u.rows) return;
  const float* p = a.parts + ((int64_t)id * a.splits * R + row) * (D + 4);
  constexpr int64_t S = R * (D + 4);
  // requested before it is known how many of them were written
  const float top = p[min(tid, a.splits - 1) * S + D];
  const Keys keys = keys_of<R>(a, u);
  if (keys.one()) return;
  const int parts = keys.parts();
  if (tid < 128) sm[tid] = tid < parts ? top : -INFINITY;
  __syncthreads();
  float m = -INFINITY;
  for (int s = 0; s < parts; ++s) m = fmaxf(m, sm[s]);
  float l = 0.0f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int s = part; s < a.splits; s += 4 * N) {
    float4 y[4], z[4];
    float f[4], w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = s + i * N, at = min(k, a.splits - 1);
      const float* x = p + at * S;
      y[i] = *(const float4*)(x + c), z[i] = *(const float4*)(x + c + 4);
      w[i] = x[D + 1];
      f[i] = sm[at] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((sm[at] - m) * a.scale);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s + i * N >= parts) break;
      l = fmaf(f[i], w[i], l);
      v[0] = fmaf(f[i], y[i].x, v[0]), v[1] = fmaf(f[i], y[i].y, v[1]);
      v[2] = fmaf(f[i], y[i].z, v[2]), v[3] = fmaf(f[i], y[i].w, v[3]);
      v[4] = fmaf(f[i], z[i].x, v[4]), v[5] = fmaf(f[i], z[i].y, v[5]);
      v[6] = fmaf(f[i], z[i].z, v[6]), v[7] = fmaf(f[i], z[i].w, v[7]);
    }
  }
  if (c == 0) sl[part] = l;
#pragma unroll
  for (int k = 0; k < 8; ++k) so[part][c + k] = v[k];
  __syncthreads();
  if (tid >= D) return;
  l = 0.0f;
  float o = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    l += sl[i];
    o += so[i][tid];
  }
  out_row<T, D>(a, u, u.row0 + row)[tid] = from_f32<T>(l == 0.0f ? 0.0f : o * (1.0f / l));
}

// Runs: eight columns of a row per thread, part after part, four in flight.
template <typename T, int D, int R>
__global__ void __launch_bounds__(256)
k_kv4_join_runs(AttnArgs a) {
  constexpr int C = D / 8, N = 256 / C;  // rows of a block
  const uint32_t block = grid_block(), id = block / (R / N);
  const int c = 8 * (threadIdx.x % C), row = block % (R / N) * N + threadIdx.x / C;
  if (id >= a.units) return;
  const Unit u = unit_of<R>(a, id / a.c.heads, id % a.c.heads);
  if (u.row0 + row >= u.rows) return;
  const Keys keys = keys_of<R>(a, u);
  if (keys.one()) return;
  const int parts = keys.parts();
  const float* p = a.parts + ((int64_t)id * a.splits * R + row) * (D + 4);
  constexpr int64_t S = R * (D + 4);
  float m = -INFINITY, l = 0.0f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int s = 0; s < parts; s += 4) {
    float4 y[4], z[4];
    float2 w[4];  // maximum, sum of weights
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* x = p + min(s + i, parts - 1) * S;
      y[i] = *(const float4*)(x + c), z[i] = *(const float4*)(x + c + 4);
      w[i] = *(const float2*)(x + D);
    }
    const float was = m;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, w[i].x);
    // -inf has no keys, or sums that are NaN: they keep their weight
    const float f = was == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((was - m) * a.scale);
    l *= f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s + i >= parts) break;
      const float g = w[i].x == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((w[i].x - m) * a.scale);
      l = fmaf(g, w[i].y, l);
      v[0] = fmaf(g, y[i].x, v[0]), v[1] = fmaf(g, y[i].y, v[1]);
      v[2] = fmaf(g, y[i].z, v[2]), v[3] = fmaf(g, y[i].w, v[3]);
      v[4] = fmaf(g, z[i].x, v[4]), v[5] = fmaf(g, z[i].y, v[5]);
      v[6] = fmaf(g, z[i].z, v[6]), v[7] = fmaf(g, z[i].w, v[7]);
    }
  }
  const float f = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= f;
  store8(out_row<T, D>(a, u, u.row0 + row) + c, v, 8, true);
}

constexpr int kChunkWaves = 8, kChunkRows = 16 * kChunkWaves;

// Operands of 32 keys for the wavefronts of a block, in LDS: fragments of keys
// and values as 16 + code, 1 KB each in the lanes' order, and parameters.
template <int D, int G>
struct Shared {
  static constexpr int NG = D / G, J = D / 32, N = D / 16;
  static constexpr int kK = 0, kV = 2 * J * 1024, kKp = kV + N * 1024, kVp = kKp + 128 * NG;
  static constexpr int kBytes = kVp + 128 * NG;
};
// A wavefront's share of them on the way.  Heads of 128: a word of one of the 16
// keys of a half, and the eight keys' words of V that give one tile of columns;
// of 64: wavefronts 0 to 3 have a word of keys, 4 to 7 a tile of columns.
template <int D, int G>
struct Share {
  uint32_t k, p;
  uint4 v[2];
};
template <int D, int G>
__device__ __forceinline__ void load_share(const Kv4& c, const int (&page)[2], int head, int key, int wave,
                                           uint32_t lane, Share<D, G>& q) {
  constexpr uint32_t NG = D / G, TG = G / 16, WG = G / 8, J = D / 32;
  const uint32_t r16 = lane & 15, q4 = lane >> 4;
  const int64_t token[2] = {key_token(c, page[0], head, key), key_token(c, page[1], head, key + 16)};
  if (D == 128 || wave < 4) {
    const int u = wave / J, j = wave % J;
    q.k = *(const uint32_t*)(uniform(c.k_codes + (u ? token[1] : token[0]) * (D / 8)) +
                             (r16 * (D / 2) + q4 * (D / 8) + 4u * j));
  }
  if (D == 128 || wave >= 4) {
    const uint32_t n = D == 128 ? wave : wave - 4, word = n / TG * WG + r16 % WG;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      q.v[u] = *(const uint4*)(uniform(c.v_codes + token[u] * (D / 8)) + (64 * word + 16 * q4));
  }
  // parameters: threads 0 .. 32 NG - 1 the keys', as many behind them the values'
  const uint32_t tid = 64 * wave + lane, i = tid % (32 * NG);
  if (tid < 64 * NG) {
    const uint32_t* base = tid < 32 * NG ? c.k_params : c.v_params;
    q.p = base[(i < 16 * NG ? token[0] : token[1]) * NG + i % (16 * NG)];
  }
}
template <typename T, int D, int G>
__device__ __forceinline__ void store_share(const Share<D, G>& q, int wave, uint32_t lane, char* st,
                                            const Sixteen<T>& k16, const Sixteen<__bf16>& v16) {
  using S = Shared<D, G>;
  constexpr uint32_t TG = G / 16;
  const uint32_t r16 = lane & 15;
  if (D == 128 || wave < 4) *(uint4*)(st + S::kK + wave * 1024 + 16 * lane) = k16.word(q.k);
  if (D == 128 || wave >= 4) {
    const int tile = D == 128 ? wave : wave - 4;
    const uint32_t n = tile % TG;  // in its group: nibble n of the lane's halves or bytes
    const uint32_t sel = G == 128  ? (n & 4 ? 0x07060302u : 0x05040100u)
                         : G == 64 ? (r16 & 8 ? 0x07060302u : 0x05040100u)
                                   : 0x0c040c00u + (r16 >> 2) * 0x00010001u;
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4& x = q.v[i >> 1];
      h[i] = v16.pair(__builtin_amdgcn_perm(i & 1 ? x.w : x.y, i & 1 ? x.z : x.x, sel) >> (4 * (n & 3)), 0);
    }
    *(uint4*)(st + S::kV + tile * 1024 + 16 * lane) = make_uint4(h[0], h[1], h[2], h[3]);
  }
  const uint32_t tid = 64 * wave + lane;
  if (tid < 64 * S::NG) *(uint32_t*)(st + S::kKp + 4 * tid) = q.p;
}
template <int D, int G>
struct ValueFragments {
  static constexpr bool kTight = false;
  const char* base;  // of the lane
  int g;
  __device__ __forceinline__ void group(int i) { g = i; }
  __device__ __forceinline__ uint4 operator()(int n) const {
    return *(const uint4*)(base + (g * (G / 16) + n) * 1024);
  }
};

template <typename T, int D, int G>
__global__ void __launch_bounds__(64 * kChunkWaves, 2)
k_kv4_chunk(AttnArgs a) {
  using S = Shared<D, G>;
  __shared__ __attribute__((aligned(16))) char smem[2 * S::kBytes];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t block = grid_block(), split = block % a.splits, id = block / a.splits;
  if (id >= a.units) return;
  const Unit u = unit_of<kChunkRows>(a, id / a.c.heads, id % a.c.heads);
  if (u.row0 >= u.rows) return;
  auto seen_by = [&](int row) { return min(max(u.len - u.run + row / a.per_kv + 1, 0), u.len); };
  const Keys keys = keys_of<kChunkRows>(a, u);
  const int from = (int)min((int64_t)split * keys.per, (int64_t)keys.end), to = min(from + keys.per, keys.end);
  if (split && from >= keys.end) return;
  // a wavefront behind the sequence's rows prepares its share alone
  const int row0 = u.row0 + 16 * wave;
  const bool live = row0 < u.rows;
  const int mine = live ? min(to, seen_by(min(row0 + 16, u.rows) - 1)) : 0;
  Rows<D, G> w;
  const int low = load_rows<T>(a, u, row0, lane, w);
  const Sixteen<T> k16;
  const Sixteen<__bf16> v16;
  Pages pages(a, u);
  const uint32_t q4 = (uint32_t)lane >> 4;
  const float scale = a.scale, slack = a.slack;
  int page[3][2];
  Share<D, G> share;
  if (from < to) {
    pages.of(from, lane, page[0]);
    pages.of(from + 32, lane, page[1]);
    pages.of(from + 64, lane, page[2]);
    load_share(a.c, page[0], u.head, from, wave, lane, share);
    store_share(share, wave, lane, smem, k16, v16);
    if (from + 32 < to) load_share(a.c, page[1], u.head, from + 32, wave, lane, share);
  }
  int at = 0;
  for (int key = from; key < to; key += 32) {
    // this tile's operands are there, and nobody reads the other stage any more
    __syncthreads();
    if (key + 32 < to) {
      store_share(share, wave, lane, smem + (at ^ S::kBytes), k16, v16);
      if (key + 64 < to) load_share(a.c, page[2], u.head, key + 64, wave, lane, share);
    }
    if (key < mine) {
      const char* st = smem + at;
      float s[8];
      floatx4 acc[2][S::NG];
      uint32_t p[2][4 * S::NG];
      products<T>(w, [&](int v, int j) { return *(const uint4*)(st + S::kK + (v * S::J + j) * 1024 + 16 * lane); }, acc);
      read_params<S::NG>(st + S::kKp, q4, p);
      scores(w, p, acc, s);
      read_params<S::NG>(st + S::kVp, q4, p);
      if (key + 32 > low || (page[0][0] | page[0][1]) < 0) hide(w.lim, page[0], key, q4, s, p);
      weigh(w, scale, slack, s);
      ValueFragments<D, G> vf{st + S::kV + 16 * lane, 0};
      gather<D, G, false>(w, p, s, vf, 0);
    }
    at ^= S::kBytes;
#pragma unroll
    for (int i = 0; i < 2; ++i) page[i][0] = page[i + 1][0], page[i][1] = page[i + 1][1];
    pages.of(key + 96, lane, page[2]);
  }
  if (!live) return;
  finish_sums(w);
  const int row = row0 + (lane & 15);
  if (row >= u.rows) return;
  constexpr int TG = G / 16;
  if (!keys.one()) {
    float* x = a.parts + ((int64_t)block * kChunkRows + row - u.row0) * (D + 4);
#pragma unroll
    for (int n = 0; n < D / 16; n += 2)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *(float2*)(x + column<G>(n, 4 * q4 + r)) = make_float2(w.o[n][r] + w.off[n / TG], w.o[n + 1][r] + w.off[n / TG]);
    if (q4 == 0) {
      x[D] = w.m;
      x[D + 1] = w.l;
    }
    return;
  }
  T* x = out_row<T, D>(a, u, row);
  const float f = w.l == 0.0f ? 0.0f : 1.0f / w.l;
#pragma unroll
  for (int g = 0; g < D / G; ++g)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      typedef T Tx __attribute__((ext_vector_type(TG)));
      Tx v;  // neighbouring columns
#pragma unroll
      for (int n = 0; n < TG; ++n) v[n] = from_f32<T>((w.o[g * TG + n][r] + w.off[g]) * f);
      *(Tx*)(x + column<G>(g * TG, 4 * q4 + r)) = v;
    }
}

// Few rows for each sequence go to the decoding kernel: it splits the keys of
// 16 rows among wavefronts and blocks, where the other would leave rows empty.
static bool takes_decode(const Kv4Attention& a) {
  const int per = a.heads / a.cache.heads;
  return a.starts == nullptr || a.tokens * per <= 16 * a.seqs;
}
static int64_t row_tiles(const Kv4Attention& a, int rows) {
  const int64_t per = a.heads / a.cache.heads;
  return a.starts == nullptr ? a.seqs * ((per + rows - 1) / rows) : a.tokens * per / rows + a.seqs;
}
// A unit's keys go to `splits` blocks, `per` or more to each.
struct Split {
  int rows, splits, per;
};
static Split split_of(const Kv4Attention& a) {
  const bool decode = takes_decode(a);
  Split s;
  s.rows = decode ? kDecodeRows : kChunkRows;
  const int64_t units = row_tiles(a, s.rows) * a.cache.heads;
  const int64_t keys = a.per_seq << a.cache.shift;
  // Single tokens: four blocks of four wavefronts fit a compute unit (three with four
  // groups a head).  Where the
  // units fill them by themselves a part costs more than it hides: 64 x 500 keys,
  // 8 kv heads: 12.0 us whole, 16.6 in two; one sequence of 8192, 8 kv heads: 10.5
  // us in parts of 256, 12.4 of 192 and 11.9 of 512.  Runs: two blocks of eight fit
  // with heads of 64 and with groups of 128 (147 and 192 registers leave one with heads
  // of 128 in groups of 64 and 32, where nothing else was measured); half as many again even
  // out sequences of different lengths (4 x 256 to 512 tokens behind 512 to 4096 keys,
  // 32 heads on 8 in groups of 128: 165 us, 200 in whole; 8 x 256 behind up to 8192: 310
  // and 393), parts of 1024 keys too few (217).
  const int64_t target = decode ? 4 * kCUs : 3 * kCUs;
  s.per = !decode ? 512 : units < kCUs ? 256 : 320;
  int64_t n = (target + units / 2) / units, most = keys / s.per;
  if (n > most) n = most;
  s.splits = (int)(n > 128 ? 128 : n < 1 ? 1 : n);
  return s;
}
size_t kv4_attention_workspace(const Kv4Attention& a) {
  const Split s = split_of(a);
  return s.splits == 1 ? 0 : (size_t)row_tiles(a, s.rows) * a.cache.heads * s.splits * s.rows * (a.cache.dim + 4) * 4;
}

template <typename T, int D, int G>
static hipError_t run(const Kv4Attention& k, hipStream_t stream) {
  AttnArgs a{};
  a.c = k.cache;
  a.q = k.q;
  a.out = k.out;
  a.heads = k.heads;
  a.per_kv = k.heads / k.cache.heads;
  a.q_token = k.q_token;
  a.q_head = k.q_head;
  a.tokens = (int)k.tokens;
  a.seqs = (int)k.seqs;
  a.per_seq = (int)k.per_seq;
  a.starts = k.starts;
  a.table = k.table;
  a.lens = k.lens;
  // at the least value scores' products are below 2^-23 (so all weights 1 at scale 0),
  // and -inf, a hidden key's score, keeps its product
  a.scale = fmaxf(fabsf(k.scale) * (__is_same(T, _Float16) ? 1.0f : kUnit) * 1.4426950408889634f, 0x1p-149f);
  a.slack = 8.0f / a.scale;
  a.flip = k.scale < 0.0f;
  a.parts = (float*)k.ws;
  const Split split = split_of(k);
  a.splits = split.splits;
  a.per = split.per;
  // below 2^31, with splits below 2^18
  const int64_t units = row_tiles(k, split.rows) * a.c.heads;
  a.units = (uint32_t)units;
  const dim3 grid = grid_of(units * a.splits);
  // rows of a tile at most
  a.rows = k.starts == nullptr && a.per_kv < split.rows ? a.per_kv : split.rows;
  if (!takes_decode(k))
    hipLaunchKernelGGL((k_kv4_chunk<T, D, G>), grid, dim3(64 * kChunkWaves), 0, stream, a);
  else if (a.rows <= 8)
    hipLaunchKernelGGL((k_kv4_decode<T, D, G, true>), grid, dim3(64 * kDecodeWaves), 0, stream, a);
  else
    hipLaunchKernelGGL((k_kv4_decode<T, D, G, false>), grid, dim3(64 * kDecodeWaves), 0, stream, a);
  if (a.splits > 1 && takes_decode(k))
    hipLaunchKernelGGL((k_kv4_join<T, D>), dim3((unsigned)(units * a.rows)), dim3(256), 0, stream, a);
  else if (a.splits > 1)
    hipLaunchKernelGGL((k_kv4_join_runs<T, D, kChunkRows>), grid_of(units * (kChunkRows * D / 2048)), dim3(256), 0,
                       stream, a);
  return hipGetLastError();
}
template <typename T>
static hipError_t by_size(const Kv4Attention& a, hipStream_t stream) {
  if (a.cache.dim == 128) {
    if (a.cache.group == 128) return run<T, 128, 128>(a, stream);
    if (a.cache.group == 64) return run<T, 128, 64>(a, stream);
    return run<T, 128, 32>(a, stream);
  }
  if (a.cache.group == 64) return run<T, 64, 64>(a, stream);
  return run<T, 64, 32>(a, stream);
}
hipError_t launch_kv4_attention(const Kv4Attention& a, hipStream_t stream) {
  return a.type == kF16 ? by_size<_Float16>(a, stream) : by_size<__bf16>(a, stream);
}

}  // namespace awq
