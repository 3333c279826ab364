// page_turn.cuh -- a frequency as a fraction of a turn, and a position's angle, for
// lbx_qk_norm_rope.
#pragma once

#include <cstdint>

namespace lbx {
namespace paged {

// f / (2 pi) modulo 1 of a finite f (its bits), in units of 2^-64, to the nearest: f's 24
// digits times 128 bits of 1 / (2 pi), of which the exponent says which 64 are wanted (the
// reduction of Payne and Hanek). 1 / (2 pi) is off by less than 2^-129, a turn by less than f
// times that.
__host__ __device__ inline uint64_t turns_of(uint32_t f) {
  const int exponent = f >> 23 & 255, right = 214 - (exponent ? exponent : 1);
  const uint64_t m = (f & 0x7fffffu) | (exponent ? 0x800000u : 0u);
  // m / (2 pi) = (w[2] 2^128 + w[1] 2^64 + w[0]) 2^-128, and f = m 2^(64 - right)
  const uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;
  const uint64_t a = m * (kLo & 0xffffffffu), b = m * (kLo >> 32) + (a >> 32);
  const uint64_t c = m * (kHi & 0xffffffffu) + (b >> 32), d = m * (kHi >> 32) + (c >> 32);
  const uint64_t w0 = b << 32 | (a & 0xffffffffu), w1 = d << 32 | (c & 0xffffffffu), w2 = d >> 32;
  uint64_t turns;
  if (right <= 0) {
    turns = right > -64 ? w0 << -right : 0;
  } else {
    // bits right .. right + 63, and the one below
    const uint64_t lo = right < 64 ? w0 : right < 128 ? w1 : right < 192 ? w2 : 0;
    const uint64_t hi = right < 64 ? w1 : right < 128 ? w2 : 0;
    const int under = right - 1, by = right & 63;
    const uint64_t below = under < 64 ? w0 : under < 128 ? w1 : under < 192 ? w2 : 0;
    turns = (by ? lo >> by | hi << (64 - by) : lo) + (below >> (under & 63) & 1);
  }
  return f >> 31 ? 0 - turns : turns;
}

// pos times a frequency (by_pos, of turns_of) as halves of a turn, -1 .. 1: the product modulo a
// turn is exact, and all 64 bits of it go into one conversion, so that an angle has fp32's 24
// digits however small it is.
__host__ __device__ inline float half_turns(int32_t pos, uint64_t by_pos) {
  return (float)(int64_t)((uint64_t)(int64_t)pos * by_pos) * 1.0842021724855044e-19f;  // 2^-63
}

}  // namespace paged
}  // namespace lbx
