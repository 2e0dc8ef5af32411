// The paged cache: new rows written (keys turned by their positions on the way, rounded to 16
// bits or to 8-bit codes with a scale per row) and rows read back.
//
// Both are bound by memory.  Sixteen lanes hold a row; a row's largest magnitude, a maximum of
// bit patterns (so that a NaN or an infinity is the largest of all), takes four shuffles.
#include <cuda_fp8.h>

#include "rows.cuh"

namespace qvg {

namespace {
constexpr int kWriteHeads = 4;  // heads of one token that a half-warp writes, keys and values
constexpr float kTop8[2] = {448.f, 127.f};  // largest code: E4M3, INT8
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100: below it a row is stored as zeros

__device__ __forceinline__ uint32_t half_warp_max(uint32_t v, uint32_t mask) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(mask, v, o));
    return v;
}

template <int FMT>
__device__ __forceinline__ uint32_t codes4(const float v[4], float r) {
    if constexpr (FMT == PF_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * r, v[1] * r), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * r, v[3] * r), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    } else {
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 4; k++) w |= (uint32_t)(uint8_t)(int8_t)__float2int_rn(v[k] * r) << (8 * k);
        return w;
    }
}

// One row of one pool: pieces a and b of every lane, at row index `row`.
template <int FMT>
__device__ __forceinline__ void put_row(void *pool, float *scales, int64_t row, const Pieces &at, int l,
                                        const float a[4], const float b[4], uint32_t mask, bool &bad) {
    if constexpr (FMT == PF_F16 || FMT == PF_BF16) {
        constexpr int DT = FMT == PF_F16 ? DT_F16 : DT_BF16;
        store4<DT>(pool, row * kD + at.a, a);
        store4<DT>(pool, row * kD + at.b, b);
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 4; k++)
            m = max(m, max(__float_as_uint(a[k]) & 0x7FFFFFFFu, __float_as_uint(b[k]) & 0x7FFFFFFFu));
        m = half_warp_max(m, mask);
        const float top = FMT == PF_E4M3 ? kTop8[0] : kTop8[1];
        const float amax = __uint_as_float(m);
        const bool nonfinite = m >= 0x7F800000u, zero = nonfinite || amax < kTiny;
        const float r = zero ? 0.f : __fdiv_rn(top, amax);
        uint32_t wa = 0, wb = 0;
        if (!zero) {
            wa = codes4<FMT>(a, r);
            wb = codes4<FMT>(b, r);
        }
        uint8_t *dst = static_cast<uint8_t *>(pool) + row * kD;
        *reinterpret_cast<uint32_t *>(dst + at.a) = wa;
        *reinterpret_cast<uint32_t *>(dst + at.b) = wb;
        if (l == 0)
            scales[row] = nonfinite ? __uint_as_float(0x7FC00000u) : zero ? 0.f : __fdiv_rn(amax, top);
        bad |= nonfinite;
    }
}
}  // namespace

template <int DT, int FMT>
__global__ void __launch_bounds__(256) k_page_write(PWritePlan p) {
    pdl_begin();
    const int l = threadIdx.x & 15;
    const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
    const int groups = (p.heads + kWriteHeads - 1) / kWriteHeads;
    const int64_t unit = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int64_t token = unit / groups;
    if (token >= p.n) return;
    const int h0 = (int)(unit - token * groups) * kWriteHeads, nh = min(p.heads - h0, kWriteHeads);
    const Pieces at = pieces_of(l, p.r);
    Rotary straight = p.r;
    straight.rot = 0;
    const Pieces vat = pieces_of(l, straight);
    Raw4<DT> ka[kWriteHeads], kb[kWriteHeads], va[kWriteHeads], vb[kWriteHeads];
#pragma unroll
    for (int u = 0; u < kWriteHeads; u++) {
        if (u < nh) {
            const int64_t k = token * p.kt + (h0 + u) * p.kh, v = token * p.vt + (h0 + u) * p.vh;
            ka[u] = load_raw4<DT>(p.K, k + at.a);
            kb[u] = load_raw4<DT>(p.K, k + at.b);
            va[u] = load_raw4<DT>(p.V, v + vat.a);
            vb[u] = load_raw4<DT>(p.V, v + vat.b);
        }
    }
    const int64_t slot = __ldg(reinterpret_cast<const long long *>(p.slots) + token);
    if (slot < 0) return;
    const int shift = 31 - __clz(p.page);
    const int64_t page = slot >> shift;
    if (page >= p.n_pages) {
        if (l == 0 && h0 == 0) or_status(p.status, QVG_DEV_BAD_INDEX);
        return;
    }
    const int64_t row0 = ((page * p.heads + h0) << shift) + (slot & (p.page - 1));
    Turn t;
    if (at.turned) t = turn_of(p.r, token, l, 1.f);
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kWriteHeads; u++) {
        if (u < nh) {
            const int64_t row = row0 + ((int64_t)u << shift);
            float a[4], b[4];
            unpack4(ka[u], a);
            unpack4(kb[u], b);
            if (at.turned) {
                if (p.r.interleaved)
                    apply_turn<true>(a, b, t);
                else
                    apply_turn<false>(a, b, t);
            }
            put_row<FMT>(p.k, p.ks, row, at, l, a, b, mask, bad);
            unpack4(va[u], a);
            unpack4(vb[u], b);
            put_row<FMT>(p.v, p.vs, row, vat, l, a, b, mask, bad);
        }
    }
    if (bad && l == 0) or_status(p.status, QVG_DEV_NONFINITE);
}

cudaError_t launch_page_write(const PWritePlan &p, cudaStream_t st) {
    const int64_t units = p.n * ((p.heads + kWriteHeads - 1) / kWriteHeads);
    const dim3 grid((unsigned)((units + 15) / 16));
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(256), 0, st, p); };
    auto by_format = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        switch (p.fmt) {
            case PF_F16: return go(k_page_write<DT, PF_F16>);
            case PF_BF16: return go(k_page_write<DT, PF_BF16>);
            case PF_E4M3: return go(k_page_write<DT, PF_E4M3>);
            default: return go(k_page_write<DT, PF_INT8>);
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
