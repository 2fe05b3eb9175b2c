// The position rotation shared by attn_rope.cu (rotation, cache append) and
// attn_decode.cu (the query rotated on the way).
//
// A pair (x, y) of one head is turned by its angle a = p * f, p the token's
// position on the pair's axis and f the pair's frequency:
//   (x, y) -> (x cos a - y sin a, x sin a + y cos a),
// and its gradient by -a. Angles are kept as fixed point fractions of a turn:
// f / (2 pi) mod 1 is held as a 64-bit integer (attn_rope_t.turns, off by one unit
// at most), the product with the integer position wraps modulo a whole turn by
// itself, and its top 32 bits, read as a signed number, are the angle in
// [-1/2, 1/2) turns, off by 2^31 units of 2^-64 and the bits cut off: less than
// 2^-31 turns, whatever the position. What the sine and cosine take is that rounded
// to fp32, 2^-26 turns. A float product would be off by p f 2^-24 radians
// (6e-2 at position 10^6), and the double product that avoids this costs far
// more here (FP64 runs at about 1/60 of the FP32 rate) than the three integer
// multiply-adds it takes.
#pragma once

#include "cache_kernels.h"
#include "common.cuh"
#include "kernels.h"

namespace eba {

// cos and sin of the angle of position p at `turns` (negated for sign < 0).
__device__ __forceinline__ void rope_cs(int p, unsigned long long turns, float sign, float& c,
                                        float& s) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(p)) * turns;
  const int hi = static_cast<int>(t >> 32);
  sincospif(static_cast<float>(hi) * 0x1p-31f, &s, &c);  // half turns: [-1, 1)
  s *= sign;
}

// (x, y) turned; the products and the sum in fp32, rounded by the caller.
__device__ __forceinline__ void rope_turn(float& x, float& y, float c, float s) {
  const float a = x * c - y * s;
  y = x * s + y * c;
  x = a;
}

}  // namespace eba
