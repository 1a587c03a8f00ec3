// Order of the 4-bit cache in memory.  A page holds 2^shift tokens (16 to 128)
// of every head; a token's head is D = 64 or 128 columns in D / G groups.
//   k_codes  [page][head][token][D/8]: word J q + j (J = D / 32) holds columns
//            8 (4 j + q) ..: a lane group q of a 16x16x32 MFMA finds its eight
//            columns of every product, each of which lies inside one group of
//            32 or more, in J neighbouring words
//   v_codes  [page][head][token / 16][D/8][token % 16]: word c holds columns
//            8 c ..; the sum runs over tokens, of which a lane takes four
//            neighbours in 16 bytes
//   k_params, v_params [page][head][token][D/G]: fp16 step, fp16 offset above
// value = step * code + offset; column 8 c + i is nibble i.
#pragma once

#include "kv4_internal.h"
#include "w4_device.h"

namespace awq {

// Token i of page p, head h.
__device__ __forceinline__ int64_t kv4_token(const Kv4& c, int64_t page, int head, int i) {
  return ((page * c.heads + head) << c.shift) + i;
}
// Word of column block cb (columns 8 cb ..) of a token.
template <int D>
__device__ __forceinline__ int64_t kv4_k_word(int64_t token, int cb) {
  return token * (D / 8) + (cb & 3) * (D / 32) + (cb >> 2);
}
template <int D>
__device__ __forceinline__ int64_t kv4_v_word(int64_t token, int cb) {
  return (token & ~(int64_t)15) * (D / 8) + 16 * cb + (token & 15);
}

}  // namespace awq
