// The paged cache in 4 bits: new rows written (keys turned by their positions on the way) and rows
// read back.  With a a row's largest magnitude, a_g that of a group of 16 channels and TOP the largest
// code (6 or 7):
//   s = a / (64 TOP),  t = E4M3(64 a_g / a),  code = x 64 TOP / (a t) to 4 bits,  value = s t code.
//
// Sixteen lanes hold a row, eight neighbouring channels each, so that two lanes share a group; they
// take four heads' keys and values of a token, eight rows.  Keys that are turned in the half layout
// are worked on in split pieces (rows.cuh) and change places through shared memory.
// Quotients are rounded correctly, since halves are common among them (x = a / 2 is 3.5 of INT4's
// codes): x is multiplied by 64 TOP and the power of two that brings a to 1 .. 2, both exact in 16
// bits, and the product with an approximate reciprocal is corrected once by its exact remainder
// (Markstein's division).
#include <cuda_fp8.h>

#include "page_codes.cuh"
#include "rows.cuh"

namespace qvg {

namespace {
constexpr int kWriteHeads = 4;  // heads of one token that a half-warp writes, keys and values
constexpr int kWriteThreads = 128, kWriteCtas = 6;
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100: below it a row is stored as zeros
template <int FMT>
constexpr float kTop = FMT == PF_E2M1 ? 6.f : 7.f;

__device__ __forceinline__ uint32_t bits_max(const float v[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; k++) m = max(m, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    return m;
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
        // adding 1.5 * 2^23 rounds to a whole number, half to even, whose low four bits are the code
        const float2 k = make_float2(12582912.f, 12582912.f);
#pragma unroll
        for (int i = 0; i < 4; i++) q[i] = __fadd2_rn(q[i], k);
        auto low = [](float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040); };
        const uint32_t even = __byte_perm(low(q[0].x, q[1].x), low(q[2].x, q[3].x), 0x5410);
        const uint32_t odd = __byte_perm(low(q[0].y, q[1].y), low(q[2].y, q[3].y), 0x5410);
        return (even & 0x0F0F0F0Fu) | ((odd << 4) & 0xF0F0F0F0u);
    }
}
}  // namespace

// SPLIT: keys are turned in the half layout.
template <int DT, int FMT, bool SPLIT>
__global__ void __launch_bounds__(kWriteThreads, kWriteCtas) k_page_write4(PWritePlan p) {
    pdl_begin();
    __shared__ __align__(16) float s_k[SPLIT ? kWriteThreads / 16 : 1][kWriteHeads][kD];
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
#pragma unroll
    for (int u = 0; u < kWriteHeads; u++) {
        unpack4(k[u].a, kf[u]);
        unpack4(k[u].b, kf[u] + 4);
        if (turns && at.turned) {
            if (SPLIT)
                apply_turn<false>(kf[u], kf[u] + 4, t);
            else
                apply_turn<true>(kf[u], kf[u] + 4, t);
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
        if (r < kWriteHeads) {
#pragma unroll
            for (int c = 0; c < 8; c++) x[c] = kf[r][c];
        } else {
            unpack4(v[r - kWriteHeads].a, x);
            unpack4(v[r - kWriteHeads].b, x + 4);
        }
    };
    // rows 0-3: keys of the heads, 4-7: values.  Largest magnitudes as bit patterns (a NaN or an
    // infinity is the largest): of a lane's channels, of its group, then of the rows together: at each
    // exchange a lane gives away the rows that the other keeps, and lanes 2r and 2r + 1 end with row r.
    uint32_t m[8], gm[8];
#pragma unroll
    for (int r = 0; r < 8; r++) {
        float x[8];
        row_of(r, x);
        m[r] = bits_max(x);
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
#pragma unroll
    for (int r = 0; r < 8; r++) {
        const uint32_t ab = __shfl_sync(mask, bits, (threadIdx.x & 16) + 2 * r);
        const int u = r & 3;
        if (u < nh) {
            float x[8];
            row_of(r, x);
            // a = a1 * 2^e, 64 * 2^-e (a row of zeros, or one that is not finite: codes and scales 0)
            const float a1 = __uint_as_float((ab & 0x007FFFFFu) | 0x3F800000u);
            const float p64 = __uint_as_float((260u - max(ab >> 23, 6u)) << 23);
            const float g = __uint_as_float(ab ? gm[r] : 0u) * p64;
            const uint32_t t8 = __nv_cvt_float_to_fp8(quotient2(make_float2(g, g), a1, fast_rcp(a1)).x, __NV_SATFINITE, __NV_E4M3);
            const float tg = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)t8, __NV_E4M3)));
            const float d = a1 * tg, y = tg > 0.f ? fast_rcp(d) : 0.f, c = kTop<FMT> * p64;
            float2 q[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                q[i] = quotient2(__fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(c, c)), d, y);
            uint32_t w = codes8<FMT>(q, tg < 0.015625f);
            if (t8 == 0u) w = 0u;
            const int64_t row = row0 + ((int64_t)u << shift);
            *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(r < 4 ? p.k : p.v) + row * (kD / 2) + 4 * l) = w;
            if (!(l & 1)) (r < 4 ? p.kg : p.vg)[row * kGroups + (l >> 1)] = (uint8_t)t8;
        }
    }
}

cudaError_t launch_page_write4(const PWritePlan &p, cudaStream_t st) {
    const int64_t units = p.n * ((p.heads + kWriteHeads - 1) / kWriteHeads);
    constexpr int per = kWriteThreads / 16;
    const dim3 grid((unsigned)((units + per - 1) / per));
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kWriteThreads), 0, st, p); };
    const bool split = p.r.rot > 0 && !p.r.interleaved;
    auto by_format = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (p.fmt == PF_E2M1) return split ? go(k_page_write4<DT, PF_E2M1, true>) : go(k_page_write4<DT, PF_E2M1, false>);
        return split ? go(k_page_write4<DT, PF_INT4, true>) : go(k_page_write4<DT, PF_INT4, false>);
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
        widen4<FMT>(raw[u], GroupScale<FMT>(__low2half2(as_half2(group_pair(t[u])))), CodeBits(0), w);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[pair_channel<FMT>(i, 0)] = f.x * (1.f / kWiden<FMT>) * s[u];
            v[pair_channel<FMT>(i, 1)] = f.y * (1.f / kWiden<FMT>) * s[u];
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
