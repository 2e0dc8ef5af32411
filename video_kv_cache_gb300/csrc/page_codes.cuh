// 8-bit cache codes widened to the 16-bit operands of the tensor cores, exactly, and bf16 rows
// brought into fp16 beside them.
#pragma once

#include "internal.cuh"

namespace qvg {

// Four codes as four fp16 values: the E4M3 conversion instruction, or 1024 + (code + 128) - 1152.
template <bool E4M3>
__device__ __forceinline__ uint2 codes_to_f16(uint32_t w) {
    if constexpr (E4M3) {
        uint2 r;
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}\n"
            : "=r"(r.x), "=r"(r.y)
            : "r"(w));
        return r;
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t t0 = __byte_perm(u, 0x64646464u, 0x4140), t1 = __byte_perm(u, 0x64646464u, 0x4342);
        const uint32_t k = 0x64806480u;
        const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&t0), *reinterpret_cast<const __half2 *>(&k));
        const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&t1), *reinterpret_cast<const __half2 *>(&k));
        return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
}

// Eight bf16 values of a row that LANES neighbouring lanes hold, as fp16 values of the row
// divided by mul, the power of two that brings its largest to 1 .. 2.  A bf16 number has eight
// significant bits, so nothing is lost down to 2^-14 of that, and 2^-25 of it below.  A row with
// a NaN or an infinity keeps mul = 1 and stays one.
__device__ __forceinline__ float bf16_pow2(uint32_t bits) {  // 2^(exponent of the largest)
    const uint32_t e = bits >> 7;
    return e == 255u || e == 0u ? 1.f : __uint_as_float(e << 23);
}
__device__ __forceinline__ uint32_t bf16x2_max_bits(const uint4 &w) {
    const uint32_t a = __vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), c = __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu);
    const uint32_t m = __vmaxu2(a, c);
    return max(m & 0xFFFFu, m >> 16);
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float inv) {
    const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xFFFF0000u) * inv);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint4 normalised_f16(const uint4 &w, float &mul, int lanes) {
    uint32_t m = bf16x2_max_bits(w);
    for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    mul = bf16_pow2(m);
    const float inv = 1.f / mul;
    return make_uint4(bf16x2_to_f16x2(w.x, inv), bf16x2_to_f16x2(w.y, inv), bf16x2_to_f16x2(w.z, inv),
                      bf16x2_to_f16x2(w.w, inv));
}

}  // namespace qvg
