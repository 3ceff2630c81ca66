// e4m3 codes and power-of-two scale bytes of the 8-bit cache.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace e3 {

// 2^(127 - s) of a scale byte, NaN of 255
E3_DEV float inverse_scale(int s) {
    return __int_as_float(s == 255 ? 0x7fc00000 : s == 254 ? 0x400000 : (254 - s) << 23);
}

// the least byte s >= 1 with m <= 448 * 2^(s - 127) of a finite m >= 0 (448 = 1.75 * 2^8)
E3_DEV int scale_byte(float m) {
    const uint32_t u = __float_as_uint(m);
    return max(1, (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0));
}

E3_DEV uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
E3_DEV float2 from_e4m3x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// the same as packed fp16
E3_DEV uint32_t e4m3x2_f16(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}

// what a scale byte stands for
E3_DEV float scale_of(int byte) {
    return __int_as_float(byte == 255 ? 0x7fc00000 : byte == 0 ? 0x400000 : byte << 23);
}

}  // namespace e3
