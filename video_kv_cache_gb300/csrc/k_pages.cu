// The paged cache: new rows written (keys turned by their positions on the way, rounded to 16
// bits or to 8-bit codes with a scale per row) and rows read back.
//
// Both are bound by memory, the 8-bit write nearly as much by instructions (about 25 a row and
// warp): sixteen lanes hold a row and take four heads' keys and values of a token, eight rows.
// The rows' largest magnitudes are maxima of bit patterns (so that a NaN or an infinity is the
// largest of all), reduced together: at each of four exchanges a lane gives away the rows that
// the other keeps, and ends with one row of the eight.  The pair of lanes that has a row then
// makes its two quotients, largest code / magnitude and magnitude / largest code, in one
// division for all eight rows.
// 32760 tokens of 12 heads in int8: 51 us written (301 MB, 5.9 TB/s), 48 us read back (6.3);
// 280800 in e4m3 read back: 384 us (6.8).
#include <cuda_fp8.h>

#include "rows.cuh"

namespace qvg {

namespace {
constexpr int kWriteHeads = 4;  // heads of one token that a half-warp writes, keys and values
// 24 warps an SM, 80 registers: 32760 x 12 heads in int8 take 51 us; 16 warps with all the
// registers they want 61, 32 with 64 registers 62.  Some registers spill at 80 too: 12 to 104 bytes
// a thread from 16-bit inputs, 160 from fp32 to 8 bits, 350 from fp32 to 16 bits.
constexpr int kWriteThreads = 128, kWriteCtas = 6;
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100: below it a row is stored as zeros

// Four codes of v * r.  INT8: adding 1.5 * 2^23 rounds to a whole number, half to even, whose
// low byte is the code (conversions to integers run at a quarter of the rate).
template <int FMT>
__device__ __forceinline__ uint32_t codes4(const float v[4], float r) {
    const float2 r2 = make_float2(r, r);
    float2 x = __fmul2_rn(make_float2(v[0], v[1]), r2), y = __fmul2_rn(make_float2(v[2], v[3]), r2);
    if constexpr (FMT == PF_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    } else {
        const float2 k = make_float2(12582912.f, 12582912.f);
        x = __fadd2_rn(x, k);
        y = __fadd2_rn(y, k);
        return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                           __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
    }
}

// Bits of the largest magnitude of a lane's eight channels, as fp32.
template <int DT>
__device__ __forceinline__ uint32_t raw_max(const Raw8<DT> &r) {
    if constexpr (DT == DT_F32) {
        const uint32_t k = 0x7FFFFFFFu;
        auto b = [&](float x) { return __float_as_uint(x) & k; };
        return max(max(max(b(r.a.w.x), b(r.a.w.y)), max(b(r.a.w.z), b(r.a.w.w))),
                   max(max(b(r.b.w.x), b(r.b.w.y)), max(b(r.b.w.z), b(r.b.w.w))));
    } else {
        const uint32_t k = 0x7FFF7FFFu;
        const uint32_t m = __vmaxu2(__vmaxu2(r.a.w.x & k, r.a.w.y & k), __vmaxu2(r.b.w.x & k, r.b.w.y & k));
        const uint32_t h = max(m & 0xFFFFu, m >> 16);
        if constexpr (DT == DT_BF16) return h << 16;
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
    }
}
__device__ __forceinline__ uint32_t float_max(const float v[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; k++) m = max(m, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    return m;
}
}  // namespace

// SPLIT: keys are turned in the half layout.
template <int DT, int FMT, bool SPLIT>
__global__ void __launch_bounds__(kWriteThreads, kWriteCtas) k_page_write(PWritePlan p) {
    pdl_begin();
    constexpr bool WIDE = FMT == PF_F16 || FMT == PF_BF16;
    const int l = threadIdx.x & 15;
    const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
    const int groups = (p.heads + kWriteHeads - 1) / kWriteHeads;
    const int64_t unit = (int64_t)blockIdx.x * (kWriteThreads / 16) + (threadIdx.x >> 4);
    const int64_t token = unit / groups;
    if (token >= p.n) return;
    const int h0 = (int)(unit - token * groups) * kWriteHeads, nh = min(p.heads - h0, kWriteHeads);
    const Pieces at = pieces_of(l, p.r);
    Pieces straight;
    straight.a = 8 * l;
    straight.b = 8 * l + 4;
    Raw8<DT> k[kWriteHeads], v[kWriteHeads];
#pragma unroll
    for (int u = 0; u < kWriteHeads; u++) {
        if (u < nh) {
            k[u] = load_raw8<DT, SPLIT>(p.K, token * p.kt + (h0 + u) * p.kh, at);
            v[u] = load_raw8<DT, false>(p.V, token * p.vt + (h0 + u) * p.vh, straight);
        } else {
            k[u] = Raw8<DT>{};
            v[u] = Raw8<DT>{};
        }
    }
    const int64_t slot = __ldg(reinterpret_cast<const long long *>(p.slots) + token);
    // positions and frequencies arrive beside the rows and the slot
    const bool turns = p.r.rot > 0;  // the same for every lane
    Turn t;
    if (turns && at.turned) t = turn_of(p.r, token, l, 1.f);
    if (slot < 0) return;
    const int shift = 31 - __clz(p.page);
    const int64_t page = slot >> shift;
    if (page >= p.n_pages) {
        if (l == 0 && h0 == 0) or_status(p.status, QVG_DEV_BAD_INDEX);
        return;
    }
    const int64_t row0 = ((page * p.heads + h0) << shift) + (slot & (p.page - 1));
    float kf[kWriteHeads][8];
    if (turns) {
#pragma unroll
        for (int u = 0; u < kWriteHeads; u++) {
            unpack4(k[u].a, kf[u]);
            unpack4(k[u].b, kf[u] + 4);
            if (at.turned) {
                if (SPLIT)
                    apply_turn<false>(kf[u], kf[u] + 4, t);
                else
                    apply_turn<true>(kf[u], kf[u] + 4, t);
            }
        }
    }
    auto key = [&](int u, float x[8]) {
        if (turns) {
#pragma unroll
            for (int c = 0; c < 8; c++) x[c] = kf[u][c];
        } else {
            unpack4(k[u].a, x);
            unpack4(k[u].b, x + 4);
        }
    };
    if constexpr (WIDE) {
        constexpr int OUT = FMT == PF_F16 ? DT_F16 : DT_BF16;
#pragma unroll
        for (int u = 0; u < kWriteHeads; u++) {
            if (u < nh) {
                const int64_t row = row0 + ((int64_t)u << shift);
                float x[8];
                key(u, x);
                store8<OUT, SPLIT>(p.k, row * kD, at, x);
                unpack4(v[u].a, x);
                unpack4(v[u].b, x + 4);
                store8<OUT, false>(p.v, row * kD, straight, x);
            }
        }
    } else {
        // rows 0-3: keys of the heads, 4-7: values; lanes 2r and 2r + 1 end with row r's maximum
        uint32_t m[8];
#pragma unroll
        for (int u = 0; u < kWriteHeads; u++) {
            m[u] = turns ? float_max(kf[u]) : raw_max(k[u]);
            m[4 + u] = raw_max(v[u]);
        }
#pragma unroll
        for (int w = 4; w > 0; w >>= 1) {
            const bool high = l & (2 * w);
#pragma unroll
            for (int r = 0; r < w; r++) {
                const uint32_t mine = high ? m[r + w] : m[r], theirs = high ? m[r] : m[r + w];
                m[r] = max(mine, __shfl_xor_sync(mask, theirs, 2 * w));
            }
        }
        const uint32_t bits = max(m[0], __shfl_xor_sync(mask, m[0], 1));
        const float top = FMT == PF_E4M3 ? 448.f : 127.f, amax = __uint_as_float(bits);
        const bool nonfinite = bits >= 0x7F800000u, zero = nonfinite || amax < kTiny, scale = l & 1;
        float f = zero ? 0.f : __fdiv_rn(scale ? amax : top, scale ? top : amax);
        if (scale) {
            const int r = l >> 1, u = r & 3;
            if (nonfinite) f = __uint_as_float(0x7FC00000u);
            if (u < nh) (r < 4 ? p.ks : p.vs)[row0 + ((int64_t)u << shift)] = f;
            if (nonfinite && u < nh) or_status(p.status, QVG_DEV_NONFINITE);
        }
        // a row of zeros, or one that is not finite, has the quotient 0 and every code 0 (the
        // products of infinities and NaN are made so)
#pragma unroll
        for (int r = 0; r < 8; r++) {
            const float q = __shfl_sync(mask, f, (threadIdx.x & 16) + 2 * r);
            const int u = r & 3;
            if (u < nh) {
                float x[8];
                if (r < 4) {
                    key(u, x);
                } else {
                    unpack4(v[u].a, x);
                    unpack4(v[u].b, x + 4);
                }
                uint2 w = make_uint2(codes4<FMT>(x, q), codes4<FMT>(x + 4, q));
                if (q == 0.f) w = make_uint2(0u, 0u);
                uint8_t *dst = static_cast<uint8_t *>(r < 4 ? p.k : p.v) + (row0 + ((int64_t)u << shift)) * kD;
                if (SPLIT && r < 4) {
                    *reinterpret_cast<uint32_t *>(dst + at.a) = w.x;
                    *reinterpret_cast<uint32_t *>(dst + at.b) = w.y;
                } else {
                    *reinterpret_cast<uint2 *>(dst + 8 * l) = w;
                }
            }
        }
    }
}

cudaError_t launch_page_write(const PWritePlan &p, cudaStream_t st) {
    if (four_bits(p.fmt)) return launch_page_write4(p, st);
    const int64_t units = p.n * ((p.heads + kWriteHeads - 1) / kWriteHeads);
    constexpr int per = kWriteThreads / 16;
    const dim3 grid((unsigned)((units + per - 1) / per));
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kWriteThreads), 0, st, p); };
    const bool split = p.r.rot > 0 && !p.r.interleaved;
    auto by_format = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        switch (p.fmt) {
            case PF_F16: return split ? go(k_page_write<DT, PF_F16, true>) : go(k_page_write<DT, PF_F16, false>);
            case PF_BF16: return split ? go(k_page_write<DT, PF_BF16, true>) : go(k_page_write<DT, PF_BF16, false>);
            case PF_E4M3: return split ? go(k_page_write<DT, PF_E4M3, true>) : go(k_page_write<DT, PF_E4M3, false>);
            default: return split ? go(k_page_write<DT, PF_INT8, true>) : go(k_page_write<DT, PF_INT8, false>);
        }
    };
    return p.dtype == DT_F32    ? by_format(std::integral_constant<int, DT_F32>{})
           : p.dtype == DT_BF16 ? by_format(std::integral_constant<int, DT_BF16>{})
                                : by_format(std::integral_constant<int, DT_F16>{});
}

// ------------------------------------------------------------------------------------

namespace {
constexpr int kReadRows = 4;    // rows of a half-warp in flight
constexpr int kReadTokens = 64; // tokens of a CTA: 16 half-warps x kReadRows
}  // namespace

// grid (token blocks, 2 * heads, sequences); sixteen lanes a row, eight channels a lane.
template <int FMT, int DT>
__global__ void __launch_bounds__(256) k_page_read(PReadPlan p) {
    pdl_begin();
    constexpr bool WIDE = FMT == PF_F16 || FMT == PF_BF16;
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4;
    const int tensor = blockIdx.y, b = blockIdx.z, h = tensor >> 1;
    const int shift = 31 - __clz(p.page);
    const int64_t cap = (int64_t)p.max_pages << shift;
    int64_t len = max(__ldg(p.lens + b), 0);
    if (len > cap) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && tensor == 0) or_status(p.status, QVG_DEV_BAD_INDEX);
        len = cap;
    }
    const uint8_t *pool = static_cast<const uint8_t *>((tensor & 1) ? p.v : p.k);
    const float *scales = (tensor & 1) ? p.vs : p.ks;
    uint4 raw[kReadRows];
    float s[kReadRows];
    const int64_t i0 = (int64_t)blockIdx.x * kReadTokens + hw;
#pragma unroll
    for (int u = 0; u < kReadRows; u++) {
        const int64_t t = p.first + i0 + 16 * u;  // token of the sequence
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        s[u] = 0.f;
        if (i0 + 16 * u < p.count && t < len) {
            const int64_t page = __ldg(p.table + (int64_t)b * p.max_pages + (t >> shift));
            if (page >= 0 && page < p.n_pages) {
                const int64_t row = ((page * p.heads + h) << shift) + (t & (p.page - 1));
                if constexpr (WIDE) {
                    raw[u] = __ldg(reinterpret_cast<const uint4 *>(pool + row * (2 * kD)) + l);
                } else {
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(pool + row * kD) + l);
                    raw[u].x = w.x;
                    raw[u].y = w.y;
                    s[u] = __ldg(scales + row);
                }
            } else if (l == 0) {
                or_status(p.status, QVG_DEV_BAD_INDEX);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kReadRows; u++) {
        if (i0 + 16 * u >= p.count) break;
        float v[8];
        if constexpr (WIDE) {
            constexpr int SRC = FMT == PF_F16 ? DT_F16 : DT_BF16;
            unpack4(Raw4<SRC>{make_uint2(raw[u].x, raw[u].y)}, v);
            unpack4(Raw4<SRC>{make_uint2(raw[u].z, raw[u].w)}, v + 4);
        } else {
            const uint32_t w[2] = {raw[u].x, raw[u].y};
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const uint32_t pair = w[k >> 2] >> (8 * (k & 3));
                if constexpr (FMT == PF_E4M3) {
                    const __half2_raw h2 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, __NV_E4M3);
                    const float2 f = __half22float2(__half2(h2));
                    v[k] = f.x * s[u];
                    v[k + 1] = f.y * s[u];
                } else {
                    v[k] = (float)(int8_t)(pair & 0xFFu) * s[u];
                    v[k + 1] = (float)(int8_t)(pair >> 8 & 0xFFu) * s[u];
                }
            }
        }
        const int64_t x = b * p.xs + tensor * p.xt + (i0 + 16 * u) * kD + 8 * l;
        if constexpr (DT == DT_F32) {
            store4<DT>(p.X, x, v);
            store4<DT>(p.X, x + 4, v + 4);
        } else {
            auto pk = [](float lo, float hi) { return DT == DT_BF16 ? pack_bf16(lo, hi) : pack_f16(lo, hi); };
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.X) + x) =
                make_uint4(pk(v[0], v[1]), pk(v[2], v[3]), pk(v[4], v[5]), pk(v[6], v[7]));
        }
    }
}

cudaError_t launch_page_read(const PReadPlan &p, cudaStream_t st) {
    if (four_bits(p.fmt)) return launch_page_read4(p, st);
    const dim3 grid((unsigned)((p.count + kReadTokens - 1) / kReadTokens), 2 * p.heads, p.B);
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(256), 0, st, p); };
    auto by_dtype = [&](auto fmt) {
        constexpr int FMT = decltype(fmt)::value;
        return p.dtype == DT_F32    ? go(k_page_read<FMT, DT_F32>)
               : p.dtype == DT_BF16 ? go(k_page_read<FMT, DT_BF16>)
                                    : go(k_page_read<FMT, DT_F16>);
    };
    switch (p.fmt) {
        case PF_F16: return by_dtype(std::integral_constant<int, PF_F16>{});
        case PF_BF16: return by_dtype(std::integral_constant<int, PF_BF16>{});
        case PF_E4M3: return by_dtype(std::integral_constant<int, PF_E4M3>{});
        default: return by_dtype(std::integral_constant<int, PF_INT8>{});
    }
}

}  // namespace qvg
