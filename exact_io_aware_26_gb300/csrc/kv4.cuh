// kv4.cuh -- the 4-bit cache's block: 16 tokens of one head,
//   key codes [16][D / 2] bytes | key pairs [16][D / 32] half2 (scale, base) |
//   value codes | value pairs.
// A block is contiguous, so that a single bulk copy brings it, whatever the page size (two
// blocks side by side, a unit of the attention kernel, in one).  Code c stands for
// fp16(base + scale * (1 + c / 16)): 1 + c / 16 is the fp16 number with bits
// 0x3C00 | c << 6, so that a mask and one half2 fused multiply-add give two values.
#pragma once
#include <cstdint>

namespace fa {

constexpr int kKvBlock = 16;  // tokens
constexpr int kKvGroup = 32;  // channels of a pair
constexpr float kKvSaturate = 16384.f;

template <int D>
struct KvBlock {
  static constexpr int row = D / 2;                 // bytes of a token's codes
  static constexpr int groups = D / kKvGroup;       // pairs of a token
  static constexpr int codes = kKvBlock * row;
  static constexpr int pairs = kKvBlock * groups * 4;
  static constexpr int half = codes + pairs;        // keys, then values
  static constexpr int bytes = 2 * half;
};

}  // namespace fa
