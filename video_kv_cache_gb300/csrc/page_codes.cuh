// 8-bit cache codes widened to the 16-bit operands of the tensor cores, exactly.
#pragma once

#include <cuda_fp8.h>

#include "internal.cuh"

namespace qvg {

// Four codes (one 32-bit word) as four bf16 values.
//   E4M3: sign, exponent and mantissa moved into a bf16's fields give the value times 2^-120
//   (the exponent biases are 7 and 127; subnormal codes become subnormal bf16), and one exact
//   multiplication by 2^120 undoes it.
//   INT8: the low seven bits under the exponent of 128 are 128 + low; the sign bit under it is
//   128 or 256; their difference is the code.
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool E4M3>
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w) {
    if constexpr (E4M3) {
        const uint32_t t0 = __byte_perm(w, 0u, 0x1404), t1 = __byte_perm(w, 0u, 0x3424);
        const uint32_t r0 = (t0 & 0x80008000u) | ((t0 >> 4) & 0x07F007F0u);
        const uint32_t r1 = (t1 & 0x80008000u) | ((t1 >> 4) & 0x07F007F0u);
        return make_uint2(bf16x2_mul(r0, 0x7B807B80u), bf16x2_mul(r1, 0x7B807B80u));
    } else {
        const uint32_t t0 = __byte_perm(w, 0x43434343u, 0x4140), t1 = __byte_perm(w, 0x43434343u, 0x4342);
        return make_uint2(bf16x2_sub(t0 & 0xFF7FFF7Fu, t0 & 0xFF80FF80u),
                          bf16x2_sub(t1 & 0xFF7FFF7Fu, t1 & 0xFF80FF80u));
    }
}
// Four codes as four fp16 values: the E4M3 conversion instruction, or 1024 + (code + 128) - 1152.
template <bool E4M3>
__device__ __forceinline__ uint2 codes_to_f16(uint32_t w) {
    if constexpr (E4M3) {
        const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
        const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
        return make_uint2((uint32_t)a.x | (uint32_t)a.y << 16, (uint32_t)b.x | (uint32_t)b.y << 16);
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t t0 = __byte_perm(u, 0x64646464u, 0x4140), t1 = __byte_perm(u, 0x64646464u, 0x4342);
        const uint32_t k = 0x64806480u;
        const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&t0), *reinterpret_cast<const __half2 *>(&k));
        const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&t1), *reinterpret_cast<const __half2 *>(&k));
        return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
}

}  // namespace qvg
