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
// E4M3 scale four, and with scales up to 64 the product stays below 448, so it is exact.  INT4 codes come
// out at half that size (kWiden): what multiplies them next makes up for it.
//
// What bounds widening is the pipe of integer, logic and conversion instructions, which issues every
// other cycle: a word of eight codes takes four of them in E2M1 and five in INT4, and four
// multiplications.
template <int FMT>
constexpr float kWiden = FMT == PF_INT4 ? 0.5f : 1.f;  // what widen4 gives, over scale times code

// Two group scales from their E4M3 bytes.
__device__ __forceinline__ uint32_t group_pair(uint32_t two_bytes) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo;\n\t"
        "cvt.u16.u32 lo, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}\n"
        : "=r"(r)
        : "r"(two_bytes));
    return r;
}
__device__ __forceinline__ __half2 as_half2(uint32_t a) { return *reinterpret_cast<const __half2 *>(&a); }
__device__ __forceinline__ uint32_t as_word(__half2 a) { return *reinterpret_cast<const uint32_t *>(&a); }
// (a & mask) ^ c in one instruction, which holds one constant: c has to be in a register that the
// compiler does not know the value of.
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t mask, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(a), "r"(mask), "r"(c));
    return r;
}
// (a & mask) | (b & ~mask)
__device__ __forceinline__ uint32_t bit_select(uint32_t a, uint32_t mask, uint32_t b) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xe2;" : "=r"(r) : "r"(a), "r"(mask), "r"(b));
    return r;
}

// What widens a group's codes: its scale t, twice (or those of two keys).
//   E2M1: codes are converted, and multiplied by t.
//   INT4: n = code ^ 8 = code + 8 is put into the mantissa of 512 (bits 0 - 3: 512 + n / 2) or of 64
//   (bits 4 - 7: 64 + n); (512 + n / 2) t - 516 t and (64 + n) t / 2 - 36 t are one fused operation each,
//   and exact: 516 = 4 * 129, and 129 times four bits has eleven.
template <int FMT>
struct GroupScale {
    __half2 t;
    __device__ __forceinline__ explicit GroupScale(__half2 t2) : t(t2) {}
};
template <>
struct GroupScale<PF_INT4> {
    __half2 t, half, off_low, off_high;
    __device__ __forceinline__ explicit GroupScale(__half2 t2)
        : t(t2), half(__hmul2(t2, as_half2(0x38003800u))), off_low(__hmul2(t2, as_half2(0xE008E008u))),
          off_high(__hmul2(t2, as_half2(0xD080D080u))) {}
};
// The exponents that INT4 codes are put under, with their topmost bit flipped.
struct CodeBits {
    uint32_t low, high;
    // zero: a number that is 0 and that the compiler cannot know
    __device__ __forceinline__ explicit CodeBits(uint32_t zero) : low(0x60086008u ^ zero), high(0x54805480u ^ zero) {}
};
// Eight codes of a word.  E2M1: the fp16 pairs of neighbouring channels (2i, 2i + 1); INT4: pairs
// (i, i + 4), which need no bytes moved.
template <int FMT>
__device__ __forceinline__ void widen4(uint32_t w, const GroupScale<FMT> &s, const CodeBits &bits, uint32_t h[4]) {
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
        for (int i = 0; i < 4; i++) h[i] = as_word(__hmul2(as_half2(h[i]), s.t));
    } else {
        const uint32_t v = w >> 8;
        h[0] = as_word(__hfma2(as_half2(and_xor(w, 0x000F000Fu, bits.low)), s.t, s.off_low));
        h[1] = as_word(__hfma2(as_half2(and_xor(w, 0x00F000F0u, bits.high)), s.half, s.off_high));
        h[2] = as_word(__hfma2(as_half2(and_xor(v, 0x000F000Fu, bits.low)), s.t, s.off_low));
        h[3] = as_word(__hfma2(as_half2(and_xor(v, 0x00F000F0u, bits.high)), s.half, s.off_high));
    }
}
// The same codes times any factor f (twice), rounded once: in INT4, code + 8 less 8 first, which is exact.
template <int FMT>
__device__ __forceinline__ void widen4_by(uint32_t w, __half2 f, const CodeBits &bits, uint32_t h[4]) {
    if constexpr (FMT == PF_E2M1) {
        widen4<FMT>(w, GroupScale<FMT>(f), bits, h);
    } else {
        const uint32_t v = w >> 8;
        const __half2 low = as_half2(0xE008E008u), high = as_half2(0xD480D480u);  // -516, -72
        const __half2 f2 = __hadd2(f, f);
        h[0] = as_word(__hmul2(__hadd2(as_half2(and_xor(w, 0x000F000Fu, bits.low)), low), f2));
        h[1] = as_word(__hmul2(__hadd2(as_half2(and_xor(w, 0x00F000F0u, bits.high)), high), f));
        h[2] = as_word(__hmul2(__hadd2(as_half2(and_xor(v, 0x000F000Fu, bits.low)), low), f2));
        h[3] = as_word(__hmul2(__hadd2(as_half2(and_xor(v, 0x00F000F0u, bits.high)), high), f));
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
