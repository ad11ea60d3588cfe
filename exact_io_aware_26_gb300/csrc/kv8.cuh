// kv8.cuh -- the 8-bit cache's block: 16 tokens of one head,
//   key codes [16][D] int8 | value codes [D / 4][4][4][4] int8 | Kv8Tail (16 bytes).
// A code times its side's scale, a power of two (or 0), is the value.  Keys stand token by token,
// at D = 128 with the halves of odd tokens' rows in each other's place, so that the lanes of a
// product's fragment (neighbouring tokens, 16 bytes each) read shared memory without conflicts.
// Values stand in cells of 4 channels by 4 tokens, channel c of token j at
// [c / 4][j / 4][c % 4][j % 4]: a word is four tokens of one channel, which are neighbours along
// the contraction of P V.
#pragma once
#include <cstdint>

#include "kv4.cuh"

namespace fa {

// Scales of the keys and the values; bit j of a mark: token j's key (value) holds a NaN (its codes
// are 0 then).
struct Kv8Tail {
  float ks, vs;
  uint16_t k_nan, v_nan;
  uint32_t zero;
};

template <int D_>
struct Kv8Block {
  static constexpr int D = D_, bits = 8;
  static constexpr int row = D;               // bytes of a token's key codes
  static constexpr int half = kKvBlock * D;   // keys, then values
  static constexpr int tail = 2 * half;
  static constexpr int bytes = tail + 16;
  static_assert(sizeof(Kv8Tail) == 16, "the tail");
};

// The place of 16-byte chunk c of token j's key codes in its row.
template <int D>
__host__ __device__ constexpr int kv8_key_chunk(int j, int c) { return D == 128 ? c ^ ((j & 1) << 2) : c; }

// Scales' exponents; values below half of the least scale are 0.
constexpr int kKv8LeastExp = -64;

}  // namespace fa
