// The 8-bit cache's numbers.  A row (one entry, one cached head; K or V) is D
// e4m3 codes and an exponent byte s: code * 2^(s - 127), s = 255: NaN.
// Powers of two make every scaling exact (of a query's products, of a softmax
// weight), so a value is rounded once, when it is written; a finer scale would add
// no precision, e4m3 having an exponent of its own, but to values 2^14 below the
// row's largest.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace specv {

// s of a row whose largest magnitude is `amax`: the smallest with amax <= 448 *
// 2^(s - 127) (448 = 1.75 * 2^8, the largest code), at least 1; 255 if not finite.
__device__ __forceinline__ unsigned kv8_scale(float amax) {
    const unsigned bits = __float_as_uint(amax);
    if (bits >= 0x7f800000u) return 255u;
    const int s = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (unsigned)max(s, 1);
}
// 2^(s - 127), NaN for 255 (0: 2^-127, a subnormal number)
__device__ __forceinline__ float kv8_power(unsigned s) {
    return s == 0u ? __uint_as_float(0x00400000u) : s == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(s << 23);
}
// 2^(127 - s) of kv8_scale's s <= 254
__device__ __forceinline__ float kv8_inverse(unsigned s) { return __uint_as_float((254u - s) << 23); }

// two e4m3 codes, the first in the low byte
__device__ __forceinline__ uint32_t kv8_code2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float2 kv8_value2(uint32_t codes) {  // of the low 16 bits
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    float2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h));
    return r;
}
__device__ __forceinline__ float4 kv8_value4(uint32_t codes) {
    const float2 a = kv8_value2(codes & 0xffffu), b = kv8_value2(codes >> 16);
    return make_float4(a.x, a.y, b.x, b.y);
}

// whether one of four codes is NaN
__device__ __forceinline__ bool kv8_nan4(uint32_t codes) { return (((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u; }

}  // namespace specv
