// Angles of rotary positions in fixed point, shared by the kernels that append rows to a cache.
//
// inv_freq / (2 pi) becomes a 64-bit fraction of a turn, its product with the integer position
// wraps modulo one turn exactly, and the top 32 bits go to sincospi.
#pragma once

#include "common.cuh"

namespace rapid {

// inv_freq / (2 pi) modulo one turn as a fraction of 2^64.  |f| = m 2^(e - 23) with m a
// 24-bit integer, and 1 / (2 pi) = C 2^-66 to 64 bits, so the fraction is m C 2^(e - 25).
RAPID_DEVICE uint64_t turns_per_position(float f) {
    constexpr uint64_t kInvTwoPi = 0xa2f9836e4e441529ull;   // 2^66 / (2 pi), rounded down
    const uint32_t bits = __float_as_uint(f);
    const int field = (int)((bits >> 23) & 0xff);
    if (field == 0xff) return 0;                            // inf or NaN: no rotation is defined
    const uint64_t m = (bits & 0x7fffffu) | (field ? 0x800000u : 0u);
    const int right = 25 - ((field ? field : 1) - 127);     // fraction = (hi : lo) >> right
    const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
    uint64_t x;
    if (right >= 128) x = 0;
    else if (right >= 64) x = hi >> (right - 64);
    else if (right > 0) x = (lo >> right) | (hi << (64 - right));
    else x = right > -64 ? lo << -right : 0;
    return (bits >> 31) ? 0 - x : x;
}

RAPID_DEVICE void sincos_turn(uint64_t per_pos, int64_t pos, float* s, float* c) {
    const uint64_t t = per_pos * (uint64_t)pos;             // modulo one turn
    const int32_t top = (int32_t)((t + 0x80000000ull) >> 32);
    sincospif((float)top * 4.656612873077392578125e-10f, s, c);   // top 2^-31 half turns
}

}  // namespace rapid
