// A row of 128 channels held by 16 lanes, two pieces of four channels a lane: what the rotary
// and paged-cache kernels load, turn and store.
#pragma once

#include "internal.cuh"

namespace qvg {

// Channel of the first element of each of lane l's two pieces (l < 16).  Within the turned
// part each lane holds four whole pairs; the other lanes hold the channels behind it.
struct Pieces {
    int a, b;
    bool turned;
};
__device__ __forceinline__ Pieces pieces_of(int l, const Rotary &r) {
    Pieces c;
    c.turned = 8 * l < r.rot;
    const bool half = c.turned && !r.interleaved;
    c.a = half ? 4 * l : 8 * l;
    c.b = half ? r.rot / 2 + 4 * l : 8 * l + 4;
    return c;
}

template <int DT>
struct Raw4 {
    uint2 w;
};
template <>
struct Raw4<DT_F32> {
    float4 w;
};

template <int DT>
__device__ __forceinline__ Raw4<DT> load_raw4(const void *X, int64_t off) {
    Raw4<DT> r;
    if constexpr (DT == DT_F32)
        r.w = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(X) + off));
    else
        r.w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(X) + off));
    return r;
}
template <int DT>
__device__ __forceinline__ void unpack4(const Raw4<DT> &r, float v[4]) {
    if constexpr (DT == DT_F32) {
        v[0] = r.w.x; v[1] = r.w.y; v[2] = r.w.z; v[3] = r.w.w;
    } else if constexpr (DT == DT_BF16) {
        v[0] = __uint_as_float(r.w.x << 16);
        v[1] = __uint_as_float(r.w.x & 0xFFFF0000u);
        v[2] = __uint_as_float(r.w.y << 16);
        v[3] = __uint_as_float(r.w.y & 0xFFFF0000u);
    } else {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&r.w.x));
        const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&r.w.y));
        v[0] = p.x; v[1] = p.y; v[2] = q.x; v[3] = q.y;
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int DT>
__device__ __forceinline__ void store4(void *Y, int64_t off, const float v[4]) {
    if constexpr (DT == DT_F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(Y) + off) = make_float4(v[0], v[1], v[2], v[3]);
    else if constexpr (DT == DT_BF16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(Y) + off) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(Y) + off) =
            make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
}

// Both pieces of a lane: eight neighbouring channels in one access, or (SPLIT, the half layout)
// four and four.
template <int DT>
struct Raw8 {
    Raw4<DT> a, b;
};
template <int DT, bool SPLIT>
__device__ __forceinline__ Raw8<DT> load_raw8(const void *X, int64_t off, const Pieces &at) {
    Raw8<DT> r;
    if (DT == DT_F32 || SPLIT) {
        r.a = load_raw4<DT>(X, off + at.a);
        r.b = load_raw4<DT>(X, off + at.b);
    } else if constexpr (DT != DT_F32) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(X) + off + at.a));
        r.a.w = make_uint2(w.x, w.y);
        r.b.w = make_uint2(w.z, w.w);
    }
    return r;
}
template <int DT, bool SPLIT>
__device__ __forceinline__ void store8(void *Y, int64_t off, const Pieces &at, const float v[8]) {
    if (DT == DT_F32 || SPLIT) {
        store4<DT>(Y, off + at.a, v);
        store4<DT>(Y, off + at.b, v + 4);
    } else if constexpr (DT != DT_F32) {
        auto pk = [](float lo, float hi) { return DT == DT_BF16 ? pack_bf16(lo, hi) : pack_f16(lo, hi); };
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(Y) + off + at.a) =
            make_uint4(pk(v[0], v[1]), pk(v[2], v[3]), pk(v[4], v[5]), pk(v[6], v[7]));
    }
}

// Sine and cosine of 2 pi a / 2^32, each within 0.75 of a unit in the last place (a code is
// rounded after the turn, and an error of the angle moves it across more borders).  The nearest
// quarter turn is taken off in whole numbers; the rest, at most pi / 4, is the sum th + tl of
// two fp32 numbers (a 30-bit product with 2 pi / 2^32, itself in two parts).  Then the Taylor
// series, to th^9 and th^10 (what is left out is below 2^-29), with what rounding 1 - th^2 / 2
// loses added back.
__device__ __forceinline__ void sincos_turn(uint32_t a, float &s, float &c) {
    const uint32_t quarter = (a + 0x20000000u) >> 30;
    const int rest = (int)(a - (quarter << 30));
    const float hi = (float)rest, lo = (float)(rest - (int)hi);
    const float kC = 1.46291807926715969e-9f;                               // 2 pi / 2^32 in fp32
    const float kD = (float)(1.46291807926715968105e-9 - (double)kC);       // and what that leaves
    const float th = hi * kC, tl = __fmaf_rn(hi, kC, -th) + __fmaf_rn(hi, kD, lo * kC);
    const float z = th * th, zl = __fmaf_rn(th, th, -z);
    const float ps = z * (-1.f / 6 + z * (1.f / 120 + z * (-1.f / 5040 + z * (1.f / 362880))));
    const float sn = th + __fmaf_rn(th, ps, __fmaf_rn(-0.5f * z, tl, tl));
    const float h = 0.5f * z, one = 1.f - h, lost = (1.f - one) - h;
    const float pc = z * (1.f / 24 + z * (-1.f / 720 + z * (1.f / 40320 + z * (-1.f / 3628800))));
    const float cs = one + (lost + __fmaf_rn(z, pc, __fmaf_rn(-th, tl, -0.5f * zl)));
    const bool swap = quarter & 1u;
    s = swap ? cs : sn;
    c = swap ? sn : cs;
    if (quarter & 2u) s = -s;
    if ((quarter + 1u) & 2u) c = -c;
}

// The turn of a lane's four pairs for one token: sines and cosines times mscale.  position *
// frequency is exact modulo a turn in 64 bits, of which the upper 32 are taken (rounded).
struct Turn {
    float c[4], s[4];
};
__device__ __forceinline__ Turn turn_of(const Rotary &r, int64_t token, int l, float sign) {
    Turn t;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const int p = 4 * l + k;
        const int axis = (p >= r.end[0]) + (p >= r.end[1]) + (p >= r.end[2]);
        const uint64_t w = __ldg(reinterpret_cast<const unsigned long long *>(r.freqs) + p) *
                           (uint64_t)__ldg(reinterpret_cast<const long long *>(r.pos) + axis * r.pos_stride + token);
        float s, c;
        sincos_turn((uint32_t)((w + 0x80000000ull) >> 32), s, c);
        t.c[k] = c * r.mscale;
        t.s[k] = s * (r.mscale * sign);
    }
    return t;
}

__device__ __forceinline__ void turn_pair(float &x, float &y, float c, float s) {
    const float u = x * c - y * s, v = x * s + y * c;
    x = u;
    y = v;
}
// Applies the turn to a lane's pieces: pairs inside each piece, or across the two.
template <bool INTER>
__device__ __forceinline__ void apply_turn(float a[4], float b[4], const Turn &t) {
    if constexpr (INTER) {
        turn_pair(a[0], a[1], t.c[0], t.s[0]);
        turn_pair(a[2], a[3], t.c[1], t.s[1]);
        turn_pair(b[0], b[1], t.c[2], t.s[2]);
        turn_pair(b[2], b[3], t.c[3], t.s[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++) turn_pair(a[k], b[k], t.c[k], t.s[k]);
    }
}

}  // namespace qvg
