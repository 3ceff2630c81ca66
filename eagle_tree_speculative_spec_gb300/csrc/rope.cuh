// Rotary positions as turns: what eagle3_rope and eagle3_append_kv share.
#pragma once

#include "common.cuh"
#include "eagle3_kv.h"

namespace e3 {

// cos and sin, times amplitude, of position pos for a pair whose position step is `step` / 2^64 turns.  The
// product mod 2^64 is exact; its upper half, taken as signed, is the angle in [-1/2, 1/2) turns to 2^-33 turns
// (1.5e-9 radians, a hundredth of what fp32's cosine resolves).
E3_DEV float2 turned(int pos, uint64_t step, float amplitude) {
    const int32_t phase = (int32_t)(((uint64_t)(int64_t)pos * step + 0x80000000ull) >> 32);
    // the nearest quarter turn, exactly, and the angle t from there, at most pi / 4; Taylor's series to t^9 and t^8, whose
    // next terms are below 2^-29 and 2^-25 there
    const uint32_t quarter = ((uint32_t)phase + 0x20000000u) >> 30;
    const float t = (float)(int32_t)((uint32_t)phase - (quarter << 30)) * (6.283185307179586f * 0x1p-32f), x = t * t;
    const float s = fmaf(t * x, fmaf(x, fmaf(x, fmaf(x, 1.0f / 362880.0f, -1.0f / 5040.0f), 1.0f / 120.0f), -1.0f / 6.0f), t);
    const float c = fmaf(x, fmaf(x, fmaf(x, fmaf(x, 1.0f / 40320.0f, -1.0f / 720.0f), 1.0f / 24.0f), -0.5f), 1.0f);
    // turned on by the quarters: (c, s), (-s, c), (-c, -s), (s, -c)
    const uint32_t cos_sign = (quarter + 1u) << 30 & 0x80000000u, sin_sign = quarter << 30 & 0x80000000u;
    const float a = quarter & 1u ? s : c, b = quarter & 1u ? c : s;
    return make_float2(__uint_as_float(__float_as_uint(a) ^ cos_sign) * amplitude,
                       __uint_as_float(__float_as_uint(b) ^ sin_sign) * amplitude);
}

inline bool rope_dims_ok(int rotary_dim, int head_dim) {
    return rotary_dim >= 2 && rotary_dim % 2 == 0 && rotary_dim <= head_dim;
}

}  // namespace e3
