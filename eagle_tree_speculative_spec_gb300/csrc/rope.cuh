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
    float s, c;
    sincospif((float)phase * 0x1p-31f, &s, &c);
    return make_float2(c * amplitude, s * amplitude);
}

inline bool rope_dims_ok(int rotary_dim, int head_dim) {
    return rotary_dim >= 2 && rotary_dim % 2 == 0 && rotary_dim <= head_dim;
}

}  // namespace e3
