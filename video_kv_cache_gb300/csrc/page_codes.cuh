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

// 4-bit codes times their group's scale, as fp16: a code has at most three significant bits and an
// E4M3 scale four, and with scales up to 64 the product stays below 448, so it is exact.
//
// A group's scale, twice, from its E4M3 byte; of two bytes, a pair.
__device__ __forceinline__ uint32_t group_pair(uint32_t two_bytes) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo;\n\t"
        "cvt.u16.u32 lo, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}\n"
        : "=r"(r)
        : "r"(two_bytes));
    return r;
}
__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b),
                              *reinterpret_cast<const __half2 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// What the widening of a group multiplies by: E2M1 codes are converted and multiplied.  INT4 codes
// n - 8 become 64 + n by putting n = code ^ 8 into a mantissa; (64 + n) t - 72 t is one fused
// operation, and exact (72 t has seven significant bits).
template <int FMT>
struct GroupScale {
    uint32_t t, off;
    __device__ __forceinline__ explicit GroupScale(uint32_t t2) : t(t2) {
        if constexpr (FMT == PF_INT4) off = h2mul(t2, 0xD480D480u);  // -72
    }
};
// Eight codes of a word.  E2M1: the fp16 pairs of neighbouring channels (2i, 2i + 1); INT4: pairs
// (i, i + 4), which need no bytes moved.
template <int FMT>
__device__ __forceinline__ void widen4(uint32_t w, const GroupScale<FMT> &s, uint32_t h[4]) {
    if constexpr (FMT == PF_E2M1) {
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w));
#pragma unroll
        for (int i = 0; i < 4; i++) h[i] = h2mul(h[i], s.t);
    } else {
        const uint32_t m = 0x00F000F0u, one = 0x54805480u;  // bits of 64 + n at 2^4 a step, n = code ^ 8
        h[0] = h2fma(((w << 4) & m) ^ one, s.t, s.off);
        h[1] = h2fma((w & m) ^ one, s.t, s.off);
        h[2] = h2fma(((w >> 4) & m) ^ one, s.t, s.off);
        h[3] = h2fma(((w >> 8) & m) ^ one, s.t, s.off);
    }
}
// Channel of the low and high half of pair i of widen4, of eight.
template <int FMT>
__device__ __forceinline__ constexpr int pair_channel(int i, int half) {
    return FMT == PF_INT4 ? i + 4 * half : 2 * i + half;
}
// Eight fp16 or bf16 channels in the order of widen4's pairs.
template <int FMT>
__device__ __forceinline__ uint4 in_pair_order(const uint4 &w) {
    if constexpr (FMT != PF_INT4) return w;
    return make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632), __byte_perm(w.y, w.w, 0x5410),
                      __byte_perm(w.y, w.w, 0x7632));
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
