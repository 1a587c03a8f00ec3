// Attention over the 4-bit cache: for every query t and head h
//   O[t, h] = sum_j p_j V[j],  p = softmax_j(scale Q[t, h] . K[j])
// over the keys j of t's sequence up to t's own place, K and V = step code +
// offset of their groups, never rounded.
//
// One pass with a running maximum m and sum l (binary32, powers of 2).  A
// wavefront takes 32 keys at a time for 16 MT rows; a row is one token and
// one of the heads that share a kv head.
//   * Scores: MFMA 16x16x32 of codes (keys by columns) with Q.  Four operations
//     shift nibbles to the top of the mantissa below the exponent of 16, so the
//     operand is 16 + code, exactly; it is step S + (offset - 16 step) sum Q
//     per group, S the group's product, in binary32.  Q's columns are put in
//     the nibbles' order once.
//   * A lane then holds keys 4 q .. 4 q + 3 of both tiles of 16 for one row:
//     as the second operand of O^T = V^T P^T these are its eight of 32 keys, if
//     V's codes are read for the same keys.  So P never leaves its lane.  Eight
//     words of V hold eight columns of eight keys: byte permutes pair the keys
//     and each nibble position is another tile of columns; no transpose.
//   * P step, the operand, is held as two bf16 parts (16 bits): in one, or in
//     fp16, it would add as much error as the output's rounding or leave the
//     type's range.  With at most 8 rows the parts lie in lanes r and r + 8 of
//     one MFMA.  The offsets' part, sum P (offset - 16 step), is summed per
//     lane.
// Single tokens (k_kv4_decode): a block of four wavefronts takes 16 rows, each
// wavefront every fourth 32 keys, and joins them through LDS; a long axis is
// split over blocks and k_kv4_join joins the splits in order.  Runs of tokens
// (k_kv4_chunk): a block takes 64 MT rows, each wavefront 16 MT of them and
// all keys.
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
  float scale;  // times log2(e)
  int splits, tiles;  // tiles: of rows, over all sequences
  float* parts;  // [unit][split][16][D + 2]
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
    u.row0 = max(tile - base(lo), 0) * R;
  }
  u.rows = u.run * a.per_kv;
  u.len = min(max(a.lens[u.seq], 0), a.per_seq << a.c.shift);
  return u;
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}

// What a wavefront keeps of 16 MT rows: lane l has row l % 16 of each tile.
template <int D, int G, int MT>
struct Rows {
  static constexpr int J = D / 32, NG = D / G, JG = G / 32, N = D / 16;
  uint4 q[MT][J];
  float qs[MT][NG];  // sum of Q over a group
  float m[MT], l[MT], off[MT][NG];
  floatx4 o[MT][N];  // O^T: tile n, columns 4 (l / 16) + r, see column()
  int lim[MT];       // keys that the row sees
};

// Column of register r of tile n in lane group q: the word 4 q + r of a group
// of 16 (8, 4) words, which gives 8 (4, 2) of its nibbles to as many tiles.
template <int G>
__device__ __forceinline__ int column(int n, int i) {
  constexpr int TG = G / 16, WG = G / 8;
  return (n / TG) * G + 8 * (i % WG) + TG * (i / WG) + n % TG;
}

template <typename T, int D, int G, int MT>
__device__ __forceinline__ void load_rows(const AttnArgs& a, const Unit& u, int row0, int lane,
                                          Rows<D, G, MT>& w, int* rlim) {
  using R = Rows<D, G, MT>;
  const int r16 = lane & 15, q4 = lane >> 4;
  int low = 0x7fffffff;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = min(row0 + 16 * m + r16, u.rows - 1);
    const int t = row / a.per_kv;
    const T* p = (const T*)a.q + (int64_t)(u.first + t) * a.q_token +
                 (int64_t)(u.head * a.per_kv + row - t * a.per_kv) * a.q_head;
    w.lim[m] = min(max(u.len - u.run + t + 1, 0), u.len);
    low = min(low, w.lim[m]);
#pragma unroll
    for (int j = 0; j < R::J; ++j) {
      const uint4 v = *(const uint4*)(p + 32 * j + 8 * q4);
      // columns 0 4, 1 5, 2 6, 3 7, as the words' nibbles come
      w.q[m][j] = make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u),
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
          s += to_f32(__builtin_bit_cast(
              T, (uint16_t)(word_of(w.q[m][g * R::JG + j], i >> 1) >> (16 * (i & 1)))));
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      w.qs[m][g] = s;
      w.off[m][g] = 0.0f;
    }
    w.m[m] = -INFINITY;
    w.l[m] = 0.0f;
#pragma unroll
    for (int n = 0; n < R::N; ++n) w.o[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  }
#pragma unroll
  for (int s = 1; s < 16; s *= 2) low = min(low, __shfl_xor(low, s));
  *rlim = __builtin_amdgcn_readfirstlane(low);
}

// Codes and parameters of 32 keys as a lane takes them.
template <int D, int G>
struct Tile {
  static constexpr int J = D / 32, NG = D / G, WG = G / 8;
  uint32_t k[2][J];
  uint4 v[2][NG];
  uint32_t kp[2][4 * NG], vp[2][4 * NG];  // keys 4 q .., [key][group]
};
template <int D, int G>
__device__ __forceinline__ void load_tile(const Kv4& c, const int (&page)[2], int head, int key,
                                          int lane, Tile<D, G>& t) {
  using X = Tile<D, G>;
  const int r16 = lane & 15, q4 = lane >> 4;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = (key + 16 * u) & ((1 << c.shift) - 1);
    const int64_t token = kv4_token(c, max(page[u], 0), head, i);  // a multiple of 16
    const uint32_t* pk = c.k_codes + token * (D / 8) + r16 * (D / 8) + q4 * X::J;
    if constexpr (X::J == 4) {
      const uint4 w = *(const uint4*)pk;
      t.k[u][0] = w.x, t.k[u][1] = w.y, t.k[u][2] = w.z, t.k[u][3] = w.w;
    } else {
      const uint2 w = *(const uint2*)pk;
      t.k[u][0] = w.x, t.k[u][1] = w.y;
    }
#pragma unroll
    for (int g = 0; g < X::NG; ++g)
      t.v[u][g] = *(const uint4*)(c.v_codes + token * (D / 8) + 16 * (g * X::WG + r16 % X::WG) + 4 * q4);
    const uint4* pp = (const uint4*)(c.k_params + (token + 4 * q4) * X::NG);
    const uint4* pv = (const uint4*)(c.v_params + (token + 4 * q4) * X::NG);
#pragma unroll
    for (int g = 0; g < X::NG; ++g) {
      const uint4 x = pp[g], y = pv[g];
      t.kp[u][4 * g] = x.x, t.kp[u][4 * g + 1] = x.y, t.kp[u][4 * g + 2] = x.z, t.kp[u][4 * g + 3] = x.w;
      t.vp[u][4 * g] = y.x, t.vp[u][4 * g + 1] = y.y, t.vp[u][4 * g + 2] = y.z, t.vp[u][4 * g + 3] = y.w;
    }
  }
}

// Eight nibbles of a word as 16 + code: pairs 0 4, 1 5, 2 6, 3 7.
template <typename T>
__device__ __forceinline__ uint4 codes16(uint32_t w) {
  if constexpr (__is_same(T, _Float16)) {
    constexpr uint32_t M = 0x03C003C0u, E = 0x4C004C00u;
    return make_uint4(((w << 6) & M) | E, ((w << 2) & M) | E, ((w >> 2) & M) | E, ((w >> 6) & M) | E);
  } else {
    constexpr uint32_t M = 0x00780078u, E = 0x41804180u;
    return make_uint4(((w << 3) & M) | E, ((w >> 1) & M) | E, ((w >> 5) & M) | E, ((w >> 9) & M) | E);
  }
}

// 32 keys for all rows.  MASK: some rows do not see all of them.  PAIR: the two
// parts of P in lanes r and r + 8 (rows r, twice).
template <typename T, int D, int G, int MT, bool PAIR, bool MASK>
__device__ __forceinline__ void take(Rows<D, G, MT>& w, const Tile<D, G>& t, const int (&page)[2],
                                     int key, float scale, int lane) {
  using R = Rows<D, G, MT>;
  const int q4 = lane >> 4, r16 = lane & 15;
  float s[MT][2][4];
  uint32_t seen[MT];
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int g = 0; g < R::NG; ++g) {
      floatx4 acc[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < R::JG; ++j) {
        const uint4 kc = codes16<T>(t.k[u][g * R::JG + j]);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = mfma16<T>(kc, w.q[m][g * R::JG + j], acc[m]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t p = t.kp[u][r * R::NG + g];
        const float step = f16_lo(p) * scale, off = fmaf(f16_hi(p), scale, -16.0f * step);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float x = off * w.qs[m][g];
          s[m][u][r] = g == 0 ? fmaf(step, acc[m][r], x) : fmaf(step, acc[m][r], x + s[m][u][r]);
        }
      }
    }
  uint4 hi[MT], lo[MT];  // P step of the group at hand
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float top = -INFINITY;
    seen[m] = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (MASK) {
          const bool v = page[u] >= 0 && key + 16 * u + 4 * q4 + r < w.lim[m];
          seen[m] |= (uint32_t)v << (4 * u + r);
          s[m][u][r] = v ? s[m][u][r] : -INFINITY;
        }
        top = fmaxf(top, s[m][u][r]);
      }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__any(top > w.m[m])) {
      const float now = fmaxf(w.m[m], top);
      const float a = w.m[m] == now ? 1.0f : __builtin_amdgcn_exp2f(w.m[m] - now);
      w.m[m] = now;
      w.l[m] *= a;
#pragma unroll
      for (int g = 0; g < R::NG; ++g) w.off[m][g] *= a;
#pragma unroll
      for (int n = 0; n < R::N; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) w.o[m][n][r] *= a;
    }
    const float base = MASK && w.m[m] == -INFINITY ? 0.0f : w.m[m];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[m][u][r] = __builtin_amdgcn_exp2f(s[m][u][r] - base);
        w.l[m] += s[m][u][r];
      }
  }
#pragma unroll
  for (int g = 0; g < R::NG; ++g) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float ps[8];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t p = t.vp[u][r * R::NG + g];
          const float step = f16_lo(p), off = fmaf(step, -16.0f, f16_hi(p));
          float a = s[m][u][r] * step, b = s[m][u][r] * off;
          if (MASK && !((seen[m] >> (4 * u + r)) & 1)) a = b = 0.0f;  // whatever lies there
          ps[4 * u + r] = a;
          w.off[m][g] += b;
        }
      uint32_t h[4], l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = pack_bf16(ps[2 * i], ps[2 * i + 1]);
        l[i] = pack_bf16(ps[2 * i] - __uint_as_float(h[i] << 16),
                         ps[2 * i + 1] - __uint_as_float(h[i] & 0xffff0000u));
        if (PAIR) h[i] = r16 & 8 ? l[i] : h[i];
      }
      hi[m] = make_uint4(h[0], h[1], h[2], h[3]);
      lo[m] = make_uint4(l[0], l[1], l[2], l[3]);
    }
    // V's codes of the group: key pairs of the lane's words
    constexpr uint32_t M = 0x00780078u, E = 0x41804180u;
    constexpr int TG = G / 16;
    uint32_t c[TG][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4& x = t.v[i >> 1][g];
      const uint32_t a = i & 1 ? x.z : x.x, b = i & 1 ? x.w : x.y;
      if constexpr (G == 128) {
        const uint32_t p0 = __builtin_amdgcn_perm(b, a, 0x05040100u);
        const uint32_t p1 = __builtin_amdgcn_perm(b, a, 0x07060302u);
        c[0][i] = ((p0 << 3) & M) | E;
        c[1][i] = ((p0 >> 1) & M) | E;
        c[2][i] = ((p0 >> 5) & M) | E;
        c[3][i] = ((p0 >> 9) & M) | E;
        c[4][i] = ((p1 << 3) & M) | E;
        c[5][i] = ((p1 >> 1) & M) | E;
        c[6][i] = ((p1 >> 5) & M) | E;
        c[7][i] = ((p1 >> 9) & M) | E;
      } else if constexpr (G == 64) {
        const uint32_t p0 = __builtin_amdgcn_perm(b, a, r16 & 8 ? 0x07060302u : 0x05040100u);
        c[0][i] = ((p0 << 3) & M) | E;
        c[1][i] = ((p0 >> 1) & M) | E;
        c[2][i] = ((p0 >> 5) & M) | E;
        c[3][i] = ((p0 >> 9) & M) | E;
      } else {
        const uint32_t p0 = __builtin_amdgcn_perm(b, a, 0x0c040c00u + (uint32_t)(r16 >> 2) * 0x00010001u);
        c[0][i] = ((p0 << 3) & M) | E;
        c[1][i] = ((p0 >> 1) & M) | E;
      }
    }
#pragma unroll
    for (int n = 0; n < TG; ++n) {
      const uint4 b = make_uint4(c[n][0], c[n][1], c[n][2], c[n][3]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        floatx4& o = w.o[m][g * TG + n];
        o = mfma16<__bf16>(b, hi[m], o);
        if (!PAIR) o = mfma16<__bf16>(b, lo[m], o);
      }
    }
  }
}

// The pages of keys key .. key + 31; -1 where there is none or a bad one.
__device__ __forceinline__ void pages_of(const AttnArgs& a, const int32_t* table, int key, int len,
                                         int (&page)[2]) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int k = key + 16 * u;
    int p = k < len ? table[k >> a.c.shift] : -1;
    if (p >= a.c.pages) p = -1;
    page[u] = __builtin_amdgcn_readfirstlane(max(p, -1));
  }
}

// Keys k0, k0 + stride, .. below k1 (32 at a time) for all rows.
template <typename T, int D, int G, int MT, bool PAIR>
__device__ __forceinline__ void walk(const AttnArgs& a, const Unit& u, Rows<D, G, MT>& w, int low,
                                     int k0, int k1, int stride, int lane) {
  const int32_t* table = a.table + (int64_t)u.seq * a.per_seq;
  int page[2], next[2];
  Tile<D, G> t, tn;
  if (k0 >= k1) return;
  pages_of(a, table, k0, u.len, page);
  load_tile(a.c, page, u.head, k0, lane, t);
  pages_of(a, table, k0 + stride, u.len, next);
  for (int key = k0; key < k1; key += stride) {
    int after[2] = {-1, -1};
    if (key + stride < k1) {
      load_tile(a.c, next, u.head, key + stride, lane, tn);
      pages_of(a, table, key + 2 * stride, u.len, after);
    }
    if (key + 32 <= low && page[0] >= 0 && page[1] >= 0)
      take<T, D, G, MT, PAIR, false>(w, t, page, key, a.scale, lane);
    else
      take<T, D, G, MT, PAIR, true>(w, t, page, key, a.scale, lane);
    t = tn;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      page[i] = next[i];
      next[i] = after[i];
    }
  }
}

// The lane groups' shares of l and the offsets.
template <int D, int G, int MT>
__device__ __forceinline__ void finish_sums(Rows<D, G, MT>& w) {
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    w.l[m] += __shfl_xor(w.l[m], 16);
    w.l[m] += __shfl_xor(w.l[m], 32);
#pragma unroll
    for (int g = 0; g < D / G; ++g) {
      w.off[m][g] += __shfl_xor(w.off[m][g], 16);
      w.off[m][g] += __shfl_xor(w.off[m][g], 32);
    }
  }
}

template <typename T, int D>
__device__ __forceinline__ T* out_row(const AttnArgs& a, const Unit& u, int row) {
  const int t = row / a.per_kv;
  return (T*)a.out + ((int64_t)(u.first + t) * a.heads + u.head * a.per_kv + row - t * a.per_kv) * D;
}

constexpr int kDecodeRows = 16, kDecodeWaves = 4, kSplitKeys = 256;

template <typename T, int D, int G, bool PAIR>
__global__ void __launch_bounds__(64 * kDecodeWaves)
k_kv4_decode(AttnArgs a) {
  constexpr int P = D + 4;  // of a row in LDS
  __shared__ float so[kDecodeWaves][16][P];
  __shared__ float sm[kDecodeWaves][16], sl[kDecodeWaves][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = blockIdx.x % a.splits, id = blockIdx.x / a.splits;
  const Unit u = unit_of<kDecodeRows>(a, id / a.c.heads, id % a.c.heads);
  if (u.row0 >= u.rows) return;
  const int count = min(u.rows - u.row0, 16);
  // the last row sees the most keys
  const int end = min(max(u.len - u.run + (u.row0 + count - 1) / a.per_kv + 1, 0), u.len);
  const int per = (max((end + a.splits - 1) / a.splits, kSplitKeys) + 31) & ~31;
  const int from = min((int64_t)split * per, (int64_t)end), to = min(from + per, end);
  Rows<D, G, 1> w;
  int low;
  // PAIR: rows of lanes 8 to 15 are those of 0 to 7
  load_rows<T>(a, u, PAIR ? u.row0 - (lane & 8) : u.row0, lane, w, &low);
  walk<T, D, G, 1, PAIR>(a, u, w, low, from + 32 * wave, to, 32 * kDecodeWaves, lane);
  finish_sums(w);
  const int r16 = lane & 15, q4 = lane >> 4;
  if constexpr (PAIR) {
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) w.o[0][n][r] += __shfl_xor(w.o[0][n][r], 8);
  }
  if (q4 == 0) {
    sm[wave][r16] = w.m[0];
    sl[wave][r16] = w.l[0];
  }
#pragma unroll
  for (int n = 0; n < D / 16; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      so[wave][r16][column<G>(n, 4 * q4 + r)] = w.o[0][n][r] + w.off[0][n / (G / 16)];
  __syncthreads();
  // a thread takes eight columns of a row
  for (int e = tid; e < 16 * (D / 8); e += 64 * kDecodeWaves) {
    const int row = e / (D / 8), c = 8 * (e % (D / 8));
    if (row >= count) continue;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kDecodeWaves; ++i) m = fmaxf(m, sm[i][row]);
    float l = 0.0f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kDecodeWaves; ++i) {
      // a wavefront without keys has -inf, 0 and zeros; one with NaN sums keeps them
      const float f = sm[i][row] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(sm[i][row] - m);
      l = fmaf(f, sl[i][row], l);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = fmaf(f, so[i][row][c + k], v[k]);
    }
    if (a.splits > 1) {
      float* p = a.parts + ((int64_t)blockIdx.x * 16 + row) * (D + 4);
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

// One row per D / 8 threads: its splits, in order.
template <typename T, int D>
__global__ void __launch_bounds__(256)
k_kv4_join(AttnArgs a) {
  const int per = 256 / (16 * (D / 8));  // units of a block
  const int row = threadIdx.x / (D / 8) % 16, c = 8 * (threadIdx.x % (D / 8));
  const int64_t id = (int64_t)blockIdx.x * per + threadIdx.x / (16 * (D / 8));
  if (id >= (int64_t)a.tiles * a.c.heads) return;
  const Unit u = unit_of<kDecodeRows>(a, (int)(id / a.c.heads), (int)(id % a.c.heads));
  if (u.row0 + row >= u.rows) return;
  const float* p = a.parts + (id * a.splits * 16 + row) * (D + 4);
  float m = -INFINITY;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, p[(int64_t)s * 16 * (D + 4) + D]);
  float l = 0.0f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int s = 0; s < a.splits; ++s) {
    const float* x = p + (int64_t)s * 16 * (D + 4);
    const float f = x[D] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(x[D] - m);
    l = fmaf(f, x[D + 1], l);
    const float4 y = *(const float4*)(x + c), z = *(const float4*)(x + c + 4);
    v[0] = fmaf(f, y.x, v[0]), v[1] = fmaf(f, y.y, v[1]), v[2] = fmaf(f, y.z, v[2]), v[3] = fmaf(f, y.w, v[3]);
    v[4] = fmaf(f, z.x, v[4]), v[5] = fmaf(f, z.y, v[5]), v[6] = fmaf(f, z.z, v[6]), v[7] = fmaf(f, z.w, v[7]);
  }
  const float f = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= f;
  store8(out_row<T, D>(a, u, u.row0 + row) + c, v, 8, true);
}

constexpr int kChunkTiles = 2, kChunkRows = 4 * 16 * kChunkTiles;

template <typename T, int D, int G>
__global__ void __launch_bounds__(256)
k_kv4_chunk(AttnArgs a) {
  constexpr int MT = kChunkTiles;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Unit u = unit_of<kChunkRows>(a, blockIdx.x / a.c.heads, blockIdx.x % a.c.heads);
  const int row0 = u.row0 + 16 * MT * wave;
  if (row0 >= u.rows) return;
  const int last = min(row0 + 16 * MT, u.rows) - 1;
  const int end = min(max(u.len - u.run + last / a.per_kv + 1, 0), u.len);
  Rows<D, G, MT> w;
  int low;
  load_rows<T>(a, u, row0, lane, w, &low);
  walk<T, D, G, MT, false>(a, u, w, low, 0, end, 32, lane);
  finish_sums(w);
  const int r16 = lane & 15, q4 = lane >> 4;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = row0 + 16 * m + r16;
    if (row >= u.rows) continue;
    T* p = out_row<T, D>(a, u, row);
    const float f = w.l[m] == 0.0f ? 0.0f : 1.0f / w.l[m];
    constexpr int TG = G / 16;
#pragma unroll
    for (int g = 0; g < D / G; ++g)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        typedef T Tx __attribute__((ext_vector_type(TG)));
        Tx v;  // neighbouring columns
#pragma unroll
        for (int n = 0; n < TG; ++n)
          v[n] = from_f32<T>((w.o[m][g * TG + n][r] + w.off[m][g]) * f);
        *(Tx*)(p + column<G>(g * TG, 4 * q4 + r)) = v;
      }
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
static int decode_splits(const Kv4Attention& a) {
  const int64_t units = row_tiles(a, kDecodeRows) * a.cache.heads;
  const int64_t keys = a.per_seq << a.cache.shift;
  const int64_t most = (keys + kSplitKeys - 1) / kSplitKeys;
  int64_t n = (4 * kCUs + units - 1) / units;
  n = n < most ? n : most;
  return (int)(n < 1 ? 1 : n > 128 ? 128 : n);
}
size_t kv4_attention_workspace(const Kv4Attention& a) {
  if (!takes_decode(a)) return 0;
  const int s = decode_splits(a);
  return s == 1 ? 0 : (size_t)row_tiles(a, kDecodeRows) * a.cache.heads * s * 16 * (a.cache.dim + 4) * 4;
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
  a.scale = k.scale * 1.4426950408889634f;
  a.splits = 1;
  a.parts = (float*)k.ws;
  if (takes_decode(k)) {
    a.splits = decode_splits(k);
    a.tiles = (int)row_tiles(k, kDecodeRows);
    const int64_t units = (int64_t)a.tiles * a.c.heads;
    const dim3 grid((unsigned)(units * a.splits));
    // a unit has at most per_kv rows where each sequence has one token
    if (k.starts == nullptr && a.per_kv <= 8)
      hipLaunchKernelGGL((k_kv4_decode<T, D, G, true>), grid, dim3(64 * kDecodeWaves), 0, stream, a);
    else
      hipLaunchKernelGGL((k_kv4_decode<T, D, G, false>), grid, dim3(64 * kDecodeWaves), 0, stream, a);
    if (a.splits > 1) {
      const int per = 256 / (16 * (D / 8));
      hipLaunchKernelGGL((k_kv4_join<T, D>), dim3((unsigned)((units + per - 1) / per)), dim3(256), 0,
                         stream, a);
    }
    return hipGetLastError();
  }
  a.tiles = (int)row_tiles(k, kChunkRows);
  hipLaunchKernelGGL((k_kv4_chunk<T, D, G>), dim3((unsigned)((int64_t)a.tiles * a.c.heads)), dim3(256), 0,
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
