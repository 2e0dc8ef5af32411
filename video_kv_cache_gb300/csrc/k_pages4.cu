// The paged cache in 4 bits: new rows written (keys turned by their positions on the way) and rows
// read back.  With a a row's largest magnitude, a_g that of a group of 16 channels and TOP the largest
// code (6 or 7):
//   s = a / (64 TOP),  t = E4M3(64 a_g / a),  code = x 64 TOP / (a t) to 4 bits,  value = s t code.
//
// Sixteen lanes hold a row, eight neighbouring channels each, so that two lanes share a group; they
// take four heads' keys and values of a token, eight rows.  Keys that are turned in the half layout
// are worked on in split pieces (rows.cuh) and change places through shared memory.
// Halves are common among the quotients (x = a / 2 is 3.5 of INT4's codes) and have to come out as
// halves: x is multiplied by 64 TOP and the power of two that brings a to 1 .. 2, and a by t, both
// exact for rows that come in 16 bits, and the product with an approximate reciprocal is corrected once
// by its exact remainder (Markstein's division).  For fp32 rows and turned keys those two products are
// rounded, 2^-24 each, so that a quotient next to a half may become one.
//
// Bound by instructions, which issue in 77 % of the cycles: about 170 for two rows and a warp, with the
// turn, against 332 bytes of a row's traffic in bf16.  32760 tokens of 12 heads from bf16 to INT4 pages:
// 72 us turned on three axes (261 MB, 3.6 TB/s), 60 as they are; read back to bf16 44 us (5.9 TB/s).
#include <cuda_fp8.h>

#include "page_codes.cuh"
#include "rows.cuh"

namespace qvg {

namespace {
constexpr int kWriteHeads = 4;  // heads of one token that a half-warp writes, keys and values
// 24 warps an SM, 80 registers, as the other formats' writes (20 warps: 131 instead of 125 us, as this
// kernel was then).  Some registers spill from fp32 inputs, none from 16 bits.
constexpr int kWriteThreads = 128, kWriteCtas = 6;
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100: below it a row is stored as zeros
template <int FMT>
constexpr float kTop = FMT == PF_E2M1 ? 6.f : 7.f;

// Bits of the largest magnitude of eight channels, a NaN if there is one.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t bits_max(const float v[8]) {
    const float m = max_abs3(max_abs3(v[0], v[1], v[2]), v[3], v[4]);
    return __float_as_uint(max_abs3(m, max_abs3(v[5], v[6], v[7]), 0.f));
}
template <int DT>
__device__ __forceinline__ uint32_t bits_max(const Raw8<DT> &r) {
    if constexpr (DT == DT_F32) {
        const float v[8] = {r.a.w.x, r.a.w.y, r.a.w.z, r.a.w.w, r.b.w.x, r.b.w.y, r.b.w.z, r.b.w.w};
        return bits_max(v);
    } else if constexpr (DT == DT_BF16) {
        auto h = [](const uint32_t &w) { return __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w)); };
        const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h(r.a.w.x), h(r.a.w.y)), __hmax2_nan(h(r.b.w.x), h(r.b.w.y)));
        return __float_as_uint(__bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m))));
    } else {
        auto h = [](const uint32_t &w) { return __habs2(*reinterpret_cast<const __half2 *>(&w)); };
        const __half2 m = __hmax2_nan(__hmax2_nan(h(r.a.w.x), h(r.a.w.y)), __hmax2_nan(h(r.b.w.x), h(r.b.w.y)));
        return __float_as_uint(__half2float(__hmax_nan(__low2half(m), __high2half(m))));
    }
}
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// x / d with y about 1 / d, rounded correctly (but for a last place where y is at its worst; exact
// quotients come out exact).
__device__ __forceinline__ float2 quotient2(float2 x, float d, float y) {
    const float2 y2 = make_float2(y, y), q = __fmul2_rn(x, y2);
    return __ffma2_rn(__ffma2_rn(q, make_float2(-d, -d), x), y2, q);
}
// Eight codes of quotients.
template <int FMT>
__device__ __forceinline__ uint32_t codes8(float2 q[4], bool rough) {
    if constexpr (FMT == PF_E2M1) {
        uint32_t w;
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
            : "=r"(w)
            : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
        return w;
    } else {
        // a group's scale below E4M3's normal range may be well under a_g / 7: codes past 7
        if (rough) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                q[i] = make_float2(fminf(fmaxf(q[i].x, -7.f), 7.f), fminf(fmaxf(q[i].y, -7.f), 7.f));
        }
        // Adding and taking off 1.5 * 2^23 rounds to a whole number, half to even.  With 8 more for each,
        // 2^23 + low + 16 high has both codes, their topmost bits flipped, in its last byte.
        const float2 k = make_float2(12582912.f, 12582912.f), back = make_float2(8388608.f + 8.f - 12582912.f, 8.f - 12582912.f);
        uint32_t z[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 y = __fadd2_rn(__fadd2_rn(q[i], k), back);
            z[i] = __float_as_uint(__fmaf_rn(y.y, 16.f, y.x));
        }
        return __byte_perm(__byte_perm(z[0], z[1], 0x0040), __byte_perm(z[2], z[3], 0x0040), 0x5410) ^ 0x88888888u;
    }
}
}  // namespace

enum { TURN_NONE, TURN_PAIRS, TURN_HALVES };  // how keys are turned: not, neighbours, or in the half layout
template <int DT, int FMT, int TURN>
__global__ void __launch_bounds__(kWriteThreads, kWriteCtas) k_page_write4(PWritePlan p) {
    pdl_begin();
    constexpr bool SPLIT = TURN == TURN_HALVES;
    constexpr bool turns = TURN != TURN_NONE;
    __shared__ float4 s_turn[turns ? kWriteThreads / 16 : 1][16][2];
    __shared__ __align__(16) float s_k[SPLIT ? kWriteThreads / 16 : 1][kWriteHeads][kD];
    const int l = threadIdx.x & 15;
    const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
    const int groups = (p.heads + kWriteHeads - 1) / kWriteHeads;
    const int64_t unit = (int64_t)blockIdx.x * (kWriteThreads / 16) + (threadIdx.x >> 4);
    const int64_t token = unit / groups;
    // (a half-warp past the last token takes part in what the CTA shares)
    const bool live = token < p.n;
    const int h0 = (int)(unit - token * groups) * kWriteHeads, nh = min(p.heads - h0, kWriteHeads);
    const Pieces at = pieces_of(l, p.r);
    Pieces straight;
    straight.a = 8 * l;
    straight.b = 8 * l + 4;
    Raw8<DT> k[kWriteHeads], v[kWriteHeads];
#pragma unroll
    for (int u = 0; u < kWriteHeads; u++) {
        if (live && u < nh) {
            k[u] = load_raw8<DT, SPLIT>(p.K, token * p.kt + (h0 + u) * p.kh, at);
            v[u] = load_raw8<DT, false>(p.V, token * p.vt + (h0 + u) * p.vh, straight);
        } else {
            k[u] = Raw8<DT>{};
            v[u] = Raw8<DT>{};
        }
    }
    const int64_t slot = live ? __ldg(reinterpret_cast<const long long *>(p.slots) + token) : -1;
    // The turns of the CTA's tokens, each worked out by one half-warp for all that have its heads (each
    // for itself costs 2 us of the case above).
    if constexpr (turns) {
        const int64_t first = (int64_t)blockIdx.x * (kWriteThreads / 16) / groups, mine = first + (threadIdx.x >> 4);
        const int64_t last = ((int64_t)(blockIdx.x + 1) * (kWriteThreads / 16) - 1) / groups;
        if (mine <= last && mine < p.n && at.turned) {
            const Turn t = turn_of(p.r, mine, l, 1.f);
            float4 *to = s_turn[threadIdx.x >> 4][l];
            to[0] = make_float4(t.c[0], t.c[1], t.c[2], t.c[3]);
            to[1] = make_float4(t.s[0], t.s[1], t.s[2], t.s[3]);
        }
        __syncthreads();
    }
    if (slot < 0) return;
    const int shift = 31 - __clz(p.page);
    const int64_t page = slot >> shift;
    if (page >= p.n_pages) {
        if (l == 0 && h0 == 0) or_status(p.status, QVG_DEV_BAD_INDEX);
        return;
    }
    const int64_t row0 = ((page * p.heads + h0) << shift) + (slot & (p.page - 1));
    float kf[kWriteHeads][8];
    if constexpr (turns) {
        Turn t;
        if (at.turned) {
            const float4 *from = s_turn[token - (int64_t)blockIdx.x * (kWriteThreads / 16) / groups][l];
            const float4 c = from[0], s = from[1];
            t.c[0] = c.x; t.c[1] = c.y; t.c[2] = c.z; t.c[3] = c.w;
            t.s[0] = s.x; t.s[1] = s.y; t.s[2] = s.z; t.s[3] = s.w;
        }
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
    if constexpr (SPLIT) {  // to eight neighbouring channels a lane
        float(*mine)[kD] = s_k[threadIdx.x >> 4];
#pragma unroll
        for (int u = 0; u < kWriteHeads; u++) {
            *reinterpret_cast<float4 *>(mine[u] + at.a) = make_float4(kf[u][0], kf[u][1], kf[u][2], kf[u][3]);
            *reinterpret_cast<float4 *>(mine[u] + at.b) = make_float4(kf[u][4], kf[u][5], kf[u][6], kf[u][7]);
        }
        __syncwarp(mask);
#pragma unroll
        for (int u = 0; u < kWriteHeads; u++) {
            const float4 a = *reinterpret_cast<const float4 *>(mine[u] + 8 * l), b = *reinterpret_cast<const float4 *>(mine[u] + 8 * l + 4);
            kf[u][0] = a.x; kf[u][1] = a.y; kf[u][2] = a.z; kf[u][3] = a.w;
            kf[u][4] = b.x; kf[u][5] = b.y; kf[u][6] = b.z; kf[u][7] = b.w;
        }
    }
    auto row_of = [&](int r, float x[8]) {
        if (turns && r < kWriteHeads) {
#pragma unroll
            for (int c = 0; c < 8; c++) x[c] = kf[r][c];
        } else {
            const Raw8<DT> &raw = r < kWriteHeads ? k[r] : v[r - kWriteHeads];
            unpack4(raw.a, x);
            unpack4(raw.b, x + 4);
        }
    };
    // rows 0-3: keys of the heads, 4-7: values.  Largest magnitudes as bit patterns (a NaN or an
    // infinity is the largest): of a lane's channels, of its group, then of the rows together: at each
    // exchange a lane gives away the rows that the other keeps, and lanes 2r and 2r + 1 end with row r.
    uint32_t m[8], gm[8];
#pragma unroll
    for (int r = 0; r < 8; r++) {
        if (r < kWriteHeads && turns)
            m[r] = bits_max(kf[r]);
        else
            m[r] = bits_max(r < kWriteHeads ? k[r] : v[r - kWriteHeads]);
    }
#pragma unroll
    for (int r = 0; r < 8; r++) m[r] = gm[r] = max(m[r], __shfl_xor_sync(mask, m[r], 1));
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) {
        const bool high = l & (2 * w);
#pragma unroll
        for (int r = 0; r < w; r++) {
            const uint32_t mine = high ? m[r + w] : m[r], theirs = high ? m[r] : m[r + w];
            m[r] = max(mine, __shfl_xor_sync(mask, theirs, 2 * w));
        }
    }
    uint32_t bits = m[0];
    const bool nonfinite = bits >= 0x7F800000u;
    if (nonfinite || __uint_as_float(bits) < kTiny) bits = 0;
    {
        const int r = l >> 1, u = r & 3;
        if (!(l & 1) && u < nh) {
            const float s = nonfinite ? __uint_as_float(0x7FC00000u) : __fdiv_rn(__uint_as_float(bits), 64.f * kTop<FMT>);
            (r < 4 ? p.ks : p.vs)[row0 + ((int64_t)u << shift)] = s;
            if (nonfinite) or_status(p.status, QVG_DEV_NONFINITE);
        }
    }
    // Scales of the groups: the lanes of a pair share theirs, so the even one works them out for the
    // keys and the odd one for the values.
    const int64_t at0 = row0 * (kD / 2) + 4 * l, group0 = row0 * kGroups + (l >> 1);
    uint8_t *const codes[2] = {static_cast<uint8_t *>(p.k) + at0, static_cast<uint8_t *>(p.v) + at0};
    uint8_t *const scales = (l & 1 ? p.vg : p.kg) + group0;
#pragma unroll
    for (int u = 0; u < kWriteHeads; u++) {
        // a = a1 * 2^e, 64 * 2^-e (a row of zeros, or one that is not finite: codes and scales 0)
        const uint32_t ab = __shfl_sync(mask, bits, (threadIdx.x & 16) + 2 * u + (l & 1) * 8);
        const float a1 = __uint_as_float((ab & 0x007FFFFFu) | 0x3F800000u);
        const float p64 = __uint_as_float((260u - max(ab >> 23, 6u)) << 23);
        const float g = __uint_as_float(ab ? (l & 1 ? gm[4 + u] : gm[u]) : 0u) * p64;
        const uint32_t t8 = __nv_cvt_float_to_fp8(quotient2(make_float2(g, g), a1, fast_rcp(a1)).x, __NV_SATFINITE, __NV_E4M3);
        const float tg = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)t8, __NV_E4M3)));
        const float d = a1 * tg, y = tg > 0.f ? fast_rcp(d) : 0.f, c = kTop<FMT> * p64;
        const float d2 = __shfl_xor_sync(mask, d, 1), y2 = __shfl_xor_sync(mask, y, 1), c2 = __shfl_xor_sync(mask, c, 1);
        if (u < nh) {
            scales[(u << shift) * kGroups] = (uint8_t)t8;
#pragma unroll
            for (int v = 0; v < 2; v++) {
                const bool mine = v == (l & 1);
                const float dr = mine ? d : d2, yr = mine ? y : y2, cr = mine ? c : c2;
                float x[8];
                row_of(4 * v + u, x);
                float2 q[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 z = __fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(cr, cr));
                    q[i] = quotient2(z, dr, yr);
                }
                // t < 2^-6: a1 t is less than twice that
                uint32_t w = codes8<FMT>(q, dr < 0.03125f);
                if (yr == 0.f) w = 0u;
                *reinterpret_cast<uint32_t *>(codes[v] + (u << shift) * (kD / 2)) = w;
            }
        }
    }
}

cudaError_t launch_page_write4(const PWritePlan &p, cudaStream_t st) {
    const int64_t units = p.n * ((p.heads + kWriteHeads - 1) / kWriteHeads);
    constexpr int per = kWriteThreads / 16;
    const dim3 grid((unsigned)((units + per - 1) / per));
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kWriteThreads), 0, st, p); };
    auto by_turn = [&](auto dt, auto fmt) {
        constexpr int DT = decltype(dt)::value, FMT = decltype(fmt)::value;
        if (p.r.rot == 0) return go(k_page_write4<DT, FMT, TURN_NONE>);
        return p.r.interleaved ? go(k_page_write4<DT, FMT, TURN_PAIRS>) : go(k_page_write4<DT, FMT, TURN_HALVES>);
    };
    auto by_format = [&](auto dt) {
        if (p.fmt == PF_E2M1) return by_turn(dt, std::integral_constant<int, PF_E2M1>{});
        return by_turn(dt, std::integral_constant<int, PF_INT4>{});
    };
    return p.dtype == DT_F32    ? by_format(std::integral_constant<int, DT_F32>{})
           : p.dtype == DT_BF16 ? by_format(std::integral_constant<int, DT_BF16>{})
                                : by_format(std::integral_constant<int, DT_F16>{});
}

// ------------------------------------------------------------------------------------

namespace {
constexpr int kReadRows = 8;    // rows of a half-warp in flight
constexpr int kReadTokens = 16 * kReadRows; // tokens of a CTA: 16 half-warps x kReadRows
}  // namespace

// grid (token blocks, 2 * heads, sequences); sixteen lanes a row, eight channels a lane.
template <int FMT, int DT>
__global__ void __launch_bounds__(256) k_page_read4(PReadPlan p) {
    pdl_begin();
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4;
    const int tensor = blockIdx.y, b = blockIdx.z, h = tensor >> 1;
    const int shift = 31 - __clz(p.page);
    const int64_t cap = (int64_t)p.max_pages << shift;
    int64_t len = max(__ldg(p.lens + b), 0);
    if (len > cap) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && tensor == 0) or_status(p.status, QVG_DEV_BAD_INDEX);
        len = cap;
    }
    const uint8_t *pool = static_cast<const uint8_t *>((tensor & 1) ? p.v : p.k), *groups = (tensor & 1) ? p.vg : p.kg;
    const float *scales = (tensor & 1) ? p.vs : p.ks;
    uint32_t raw[kReadRows], t[kReadRows];
    float s[kReadRows];
    const int64_t i0 = (int64_t)blockIdx.x * kReadTokens + hw;
#pragma unroll
    for (int u = 0; u < kReadRows; u++) {
        const int64_t tok = p.first + i0 + 16 * u;  // token of the sequence
        raw[u] = t[u] = 0u;
        s[u] = 0.f;
        if (i0 + 16 * u < p.count && tok < len) {
            const int64_t page = __ldg(p.table + (int64_t)b * p.max_pages + (tok >> shift));
            if (page >= 0 && page < p.n_pages) {
                const int64_t row = ((page * p.heads + h) << shift) + (tok & (p.page - 1));
                raw[u] = __ldg(reinterpret_cast<const uint32_t *>(pool + row * (kD / 2)) + l);
                t[u] = __ldg(groups + row * kGroups + (l >> 1));
                s[u] = __ldg(scales + row);
            } else if (l == 0) {
                or_status(p.status, QVG_DEV_BAD_INDEX);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kReadRows; u++) {
        if (i0 + 16 * u >= p.count) break;
        uint32_t w[4];
        // (the code first, then its scale: exact for scales up to E4M3's largest, 448, where widen4's
        // offsets pass fp16's range from 128 on)
        widen4_by<FMT>(raw[u], __low2half2(as_half2(group_pair(t[u]))), CodeBits(0), w);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[pair_channel<FMT>(i, 0)] = f.x * s[u];
            v[pair_channel<FMT>(i, 1)] = f.y * s[u];
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

cudaError_t launch_page_read4(const PReadPlan &p, cudaStream_t st) {
    const dim3 grid((unsigned)((p.count + kReadTokens - 1) / kReadTokens), 2 * p.heads, p.B);
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(256), 0, st, p); };
    auto by_dtype = [&](auto fmt) {
        constexpr int FMT = decltype(fmt)::value;
        return p.dtype == DT_F32    ? go(k_page_read4<FMT, DT_F32>)
               : p.dtype == DT_BF16 ? go(k_page_read4<FMT, DT_BF16>)
                                    : go(k_page_read4<FMT, DT_F16>);
    };
    return p.fmt == PF_E2M1 ? by_dtype(std::integral_constant<int, PF_E2M1>{}) : by_dtype(std::integral_constant<int, PF_INT4>{});
}

}  // namespace qvg
