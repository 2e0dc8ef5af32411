// What the paged-attention kernels share: a sequence's geometry, what a query sees, and how a
// finished row is written.
#pragma once

#include <climits>

#include "page_codes.cuh"
#include "rows.cuh"
#include "tcgen.cuh"

namespace qvg {

struct SeqInfo {
    int64_t q0;  // first row of Q
    int qn;      // query tokens
    int len;     // cached tokens
};

// Sequence b's rows and length, cut to what the arguments allow.  One thread passes report =
// true to have what was cut reported.
__device__ __forceinline__ SeqInfo seq_info(const PAttnPlan &p, int b, bool report) {
    SeqInfo s;
    const int64_t cap = min((int64_t)p.max_pages * p.page, (int64_t)0x7FFFFF00);
    const int64_t len = __ldg(p.lens + b);
    s.len = (int)min(max(len, (int64_t)0), cap);
    int64_t q0 = b * p.max_q, q1 = q0 + p.max_q;
    if (p.cu) {
        q0 = __ldg(p.cu + b);
        q1 = __ldg(p.cu + b + 1);
    }
    const int64_t a = min(max(q0, (int64_t)0), p.total_q);
    const int64_t e = min(max(q1, a), min(p.total_q, a + p.max_q));
    s.q0 = a;
    s.qn = (int)(e - a);
    if (report && (s.len != len || a != q0 || e != q1)) or_status(p.status, QVG_DEV_BAD_INDEX);
    return s;
}

// Query token of a row (tokens x grouped heads).  r * (G * g_inv - 2^34) <= r * G < 2^34, so the
// quotient is exact.
__device__ __forceinline__ int token_of(const PAttnPlan &p, int r) { return (int)((uint64_t)(uint32_t)r * p.g_inv >> 34); }

// The item with this number among those of all sequences in a row (PAttnPlan::compact), for a whole
// warp: false if there are fewer.  A sequence's last rows come first.  With report, what is cut of
// any sequence is reported.
__device__ __forceinline__ bool compact_item(const PAttnPlan &p, int64_t number, bool report, int &b, int &h, int &pair) {
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < p.B; base += 32) {
        const int units = base + lane < p.B ? (seq_info(p, base + lane, report).qn * p.G + p.unit - 1) / p.unit : 0;
        int upto = units;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, x);
            if (lane >= x) upto += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, (int64_t)upto * p.H > number);
        if (past) {
            const int at = __ffs(past) - 1, n = __shfl_sync(0xffffffffu, units, at);
            const int in = (int)(number - (int64_t)(__shfl_sync(0xffffffffu, upto, at) - n) * p.H);
            b = base + at;
            h = in / n;
            pair = n - 1 - (in - h * n);
            return true;
        }
        number -= (int64_t)__shfl_sync(0xffffffffu, upto, 31) * p.H;
    }
    return false;
}

// Keys [lo, hi) that query i of the sequence sees (empty when lo >= hi).
__device__ __forceinline__ int seen_lo(const PAttnPlan &p, const SeqInfo &s, int i) {
    if (p.window <= 0) return 0;
    return (int)min(max((int64_t)s.len - s.qn + i + 1 - p.window, (int64_t)0), (int64_t)s.len);
}
__device__ __forceinline__ int seen_hi(const PAttnPlan &p, const SeqInfo &s, int i) {
    return p.causal ? max(s.len - s.qn + i + 1, 0) : s.len;
}

// Page of a token, checked against the pool.
__device__ __forceinline__ int64_t page_of(const PAttnPlan &p, int b, int token, int shift, bool &bad) {
    const int page = __ldg(p.table + (int64_t)b * p.max_pages + (token >> shift));
    if ((unsigned)page < (uint64_t)p.n_pages) return page;
    bad = true;
    return 0;
}

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLn2 = 0.6931471805599453f;

// The maximum a row's exponents are taken against: a row that has seen only -infinity (or
// nothing) takes 0, so that its weights are 2^-inf = 0 and not NaN.
__device__ __forceinline__ float exp_base(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ bool is_finite(float x) {
    return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

// A row may have to be computed once more by one warp, over the keys that it sees and no others,
// where a mask hides keys from some rows of a tile:
//   * 16-bit or E4M3 pages: a value that is NaN or infinite (a code that is NaN), multiplied by the
//     zero weight of a query that does not see its key, makes that query's row NaN.  Rows that did
//     not come out finite and shared a tile with such a key, which they do not see.  (Those that see one themselves are
//     what they should be.  Doing them again too, a key at a time, took seconds where a NaN is early
//     in a long cache: 44 us became 1600 for one query of four heads over 4096 keys.)
//   * 8-bit pages, many rows: a scale that the row does not see, far above all that it sees, has
//     taken its values' or keys' bits (k_page_attn_tc.cu).
// And, many rows, where scores are past 2^23.
__device__ __forceinline__ bool redo_possible(const PAttnPlan &p) { return p.causal || p.window > 0; }
__device__ __forceinline__ bool wide_pages(const PAttnPlan &p) { return p.fmt == PF_F16 || p.fmt == PF_BF16; }
__device__ __forceinline__ bool rows_to_check(const PAttnPlan &p) { return p.fmt != PF_INT8 && redo_possible(p); }
constexpr float kRedo = -1.f;  // in the place of a split's weight sum: the row is to be done again

// Of keys [x0, x1): those that only some of a tile's rows [first, last) see, [a0, a1) before and
// [z0, z1) behind what all of them see (if anything, then [a1, z0)).
struct KeySpans {
    int a0, a1, z0, z1;
};
__device__ __forceinline__ KeySpans key_spans(const PAttnPlan &p, const SeqInfo &s, int first, int last, int x0, int x1) {
    const int all_lo = seen_lo(p, s, token_of(p, last - 1)), all_hi = seen_hi(p, s, token_of(p, first));
    KeySpans k;
    k.a0 = x0;
    k.a1 = min(max(all_lo, x0), x1);
    k.z0 = min(max(all_hi, k.a1), x1);
    k.z1 = x1;
    return k;
}
// The largest finite scale of those spans' keys that this lane's row, which sees [a, z), sees, or
// top.  The lanes of a warp go through the same keys.
__device__ __forceinline__ float largest_scale(const PAttnPlan &p, const float *scales, int b, int h, KeySpans sp,
                                                   int a, int z, float top) {
    const int lane = threadIdx.x & 31, shift = 31 - __clz(p.page);
    for (int x = sp.a0; x < sp.z1; x += 32) {
        if (x >= sp.a1 && x < sp.z0) x = sp.z0;
        const int key = x + lane;
        float mine = 0.f;
        if (key < sp.z1) {
            bool bad = false;
            mine = __ldg(scales + ((page_of(p, b, key, shift, bad) * p.H + h) << shift) + (key & (p.page - 1)));
            mine = is_finite(mine) ? fabsf(mine) : 0.f;
        }
        for (int k = 0; k < 32; k++) {
            const float s = __shfl_sync(0xffffffffu, mine, k);
            if (x + k >= a && x + k < z) top = fmaxf(top, s);
        }
    }
    return top;
}

// Whether a scale of those spans lies too far (log2) above the largest that this lane's row sees: of
// `some`, the largest of the spans, and `all`, of the nearest keys that every row sees (bits); if
// those are too small, of as many more as it takes, in other splits too.  Of scales of zero only,
// nothing is lost.  The tile's first row is r0.
__device__ __forceinline__ bool too_far(uint32_t some, float seen, int limit) {
    return (int)(some >> 23) > (int)(__float_as_uint(seen) >> 23) + limit;
}
static __device__ __noinline__ bool sees_too_little(const PAttnPlan &p, const float *scales, int b, int h, const KeySpans &sp, int r0, int i,
                                                    uint32_t some, uint32_t all, int limit) {
    const SeqInfo s = seq_info(p, b, false);
    float v = largest_scale(p, scales, b, h, sp, seen_lo(p, s, i), seen_hi(p, s, i), __uint_as_float(all));
    if (__any_sync(0xffffffffu, v > 0.f && too_far(some, v, limit))) {
        const int shift = 31 - __clz(p.page);
        const int all_lo = seen_lo(p, s, token_of(p, min(s.qn * p.G, r0 + p.unit) - 1)), all_hi = seen_hi(p, s, token_of(p, r0));
        uint32_t most = 0;
        for (int x = all_hi; x > all_lo && too_far(some, __uint_as_float(most), limit); x -= 256) {
            float m = 0.f;
            for (int key = x - 1 - (threadIdx.x & 31); key >= max(all_lo, x - 256); key -= 32) {
                bool bad = false;
                const float y = __ldg(scales + ((page_of(p, b, key, shift, bad) * p.H + h) << shift) + (key & (p.page - 1)));
                m = fmaxf(m, is_finite(y) ? fabsf(y) : 0.f);
            }
            __syncwarp();
            most = max(most, __reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        }
        v = fmaxf(v, __uint_as_float(most));
    }
    return v > 0.f && too_far(some, v, limit);
}

// First and last of keys [from, to) with a value that is not finite, looked for by a whole warp;
// first > last where there is none.
struct BadKeys {
    int first, last;
};
__device__ __forceinline__ BadKeys bad_values(const PAttnPlan &p, int b, int h, int from, int to) {
    const int lane = threadIdx.x & 31, shift = 31 - __clz(p.page);
    const uint32_t ones = p.fmt == PF_F16 ? 0x7C007C00u : 0x7F807F80u;
    BadKeys k = {INT_MAX, -1};
#pragma unroll 4
    for (int key = from + (lane >> 4); key < to; key += 2) {  // 16 lanes a row
        bool bad = false;
        const int64_t row = ((page_of(p, b, key, shift, bad) * p.H + h) << shift) + (key & (p.page - 1));
        bool odd;
        if (p.fmt == PF_E4M3) {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(p.v) + row * kD) + (lane & 15));
            odd = __vcmpeq4(w.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(w.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        } else {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.v) + row * kD) + (lane & 15));
            odd = __vcmpeq2(w.x & ones, ones) | __vcmpeq2(w.y & ones, ones) | __vcmpeq2(w.z & ones, ones) | __vcmpeq2(w.w & ones, ones);
        }
        if (odd) {
            k.first = min(k.first, key);
            k.last = key;
        }
    }
    __syncwarp();
    k.first = __reduce_min_sync(0xffffffffu, k.first);
    k.last = __reduce_max_sync(0xffffffffu, k.last);
    return k;
}
// Eight channels of a row, as they lie in memory and as numbers (codes without their scale).
__device__ __forceinline__ uint4 load_cached8(const PAttnPlan &p, const void *pool, int64_t off) {
    if (wide_pages(p)) return __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(pool) + off));
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(pool) + off));
    return make_uint4(w.x, w.y, 0u, 0u);
}
__device__ __forceinline__ void unpack8(int fmt, uint4 w, float v[8]) {
    if (fmt == PF_BF16) {
        unpack4(Raw4<DT_BF16>{make_uint2(w.x, w.y)}, v);
        unpack4(Raw4<DT_BF16>{make_uint2(w.z, w.w)}, v + 4);
        return;
    }
    if (fmt != PF_F16) {
        const uint2 y = fmt == PF_E4M3 ? codes_to_f16<true>(w.x) : codes_to_f16<false>(w.x);
        const uint2 z = fmt == PF_E4M3 ? codes_to_f16<true>(w.y) : codes_to_f16<false>(w.y);
        w = make_uint4(y.x, y.y, z.x, z.y);
    }
    unpack4(Raw4<DT_F16>{make_uint2(w.x, w.y)}, v);
    unpack4(Raw4<DT_F16>{make_uint2(w.z, w.w)}, v + 4);
}
// Row (query i of sequence b, query head hq): lane l gets channels 4l .. 4l+3, unnormalised.  Half
// a warp takes a key, eight channels a lane, each half every other key with a maximum and sums of
// its own; the next keys are asked for before these are worked on, their pages looked up before that.
static __device__ __noinline__ void redo_row(const PAttnPlan &p, int b, int i, int hq, float o4[4], float &m4, float &l4) {
    const int lane = threadIdx.x & 31, part = lane & 15;
    const SeqInfo s = seq_info(p, b, false);
    const int shift = 31 - __clz(p.page), h = hq / p.G;
    const int lo = seen_lo(p, s, i), hi = seen_hi(p, s, i);
    const bool wide = wide_pages(p);
    float q[8], o[8] = {}, m = -INFINITY, l = 0.f;
    unpack8(p.q_dtype == DT_BF16 ? PF_BF16 : PF_F16,
            __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.Q) + (s.q0 + i) * p.qt + hq * p.qh + 8 * part)), q);
    auto row_of = [&](int key) {
        bool bad = false;
        return key < hi ? (int)(((page_of(p, b, key, shift, bad) * p.H + h) << shift) + (key & (p.page - 1))) : -1;
    };
    uint4 kn, vn;
    float ksn, vsn;
    auto ask = [&](int row) {
        kn = vn = make_uint4(0u, 0u, 0u, 0u);
        ksn = vsn = 1.f;
        if (row >= 0) {
            kn = load_cached8(p, p.k, (int64_t)row * kD + 8 * part);
            vn = load_cached8(p, p.v, (int64_t)row * kD + 8 * part);
            if (!wide) {
                ksn = __ldg(p.ks + row);
                vsn = __ldg(p.vs + row);
            }
        }
    };
    const int first = lo + (lane >> 4);
    ask(row_of(first));
    int next = row_of(first + 2);
    for (int key = first; key - (lane >> 4) < hi; key += 2) {
        float y[8], d = 0.f;
        unpack8(p.fmt, kn, y);
#pragma unroll
        for (int c = 0; c < 8; c++) d += q[c] * y[c];
        d *= ksn;
        const uint4 v = vn;
        const float vs = vsn;
        ask(next);
        next = row_of(key + 4);
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
        d = key < hi ? d * p.scale_log2 : -INFINITY;
        const float mn = fmaxf(m, d), base = exp_base(mn), corr = fast_exp2(m - base), w = fast_exp2(d - base);
        l = l * corr + w;
        unpack8(p.fmt, v, y);
#pragma unroll
        for (int c = 0; c < 8; c++) o[c] = o[c] * corr + w * (y[c] * vs);
        m = mn;
    }
    // the halves joined, and lane l's four channels from the lanes that have them
    m4 = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
    const float f = fast_exp2(m - exp_base(m4));
    l4 = l * f;
    l4 += __shfl_xor_sync(0xffffffffu, l4, 16);
#pragma unroll
    for (int c = 0; c < 8; c++) {
        float y = o[c] * f;
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        y = __shfl_sync(0xffffffffu, y, lane >> 1);
        if ((c >> 2) == (lane & 1)) o4[c & 3] = y;
    }
}

// Whether this lane's row (query i of head h) shares its tile, whose rows see keys [lo, hi), with a value
// that is not finite and that it does not see; the lanes' rows follow one another.
static __device__ __noinline__ bool spoilt(const PAttnPlan &p, int b, int h, int i, int lo, int hi) {
    const SeqInfo s = seq_info(p, b, false);
    const int a = seen_lo(p, s, i), z = seen_hi(p, s, i);
    const BadKeys before = bad_values(p, b, h, lo, min(__shfl_sync(0xffffffffu, a, 31), hi));
    const BadKeys behind = bad_values(p, b, h, max(__shfl_sync(0xffffffffu, z, 0), lo), hi);
    return before.first < a || behind.last >= max(z, 0);
}

// For a tile of rows [r0, r0 + p.unit).
static __device__ __noinline__ bool spoilt_in(const PAttnPlan &p, int b, int h, int i, int r0) {
    const SeqInfo s = seq_info(p, b, false);
    return spoilt(p, b, h, i, seen_lo(p, s, token_of(p, r0)), seen_hi(p, s, token_of(p, min(s.qn * p.G, r0 + p.unit) - 1)));
}

// The same if it must be, or if query i, in a tile of the sequence's queries [i0, i1], shares it with a
// value that is not finite and that it does not see.  Otherwise nothing changes.
static __device__ __noinline__ bool redo_if_shared(const PAttnPlan &p, int b, int i, int hq, int i0, int i1, bool must,
                                                   float o[4], float &m, float &l) {
    if (!must) {
        const SeqInfo s = seq_info(p, b, false);
        const int lo = seen_lo(p, s, i0), hi = seen_hi(p, s, i1);
        const int a = max(seen_lo(p, s, i), lo), z = max(seen_hi(p, s, i), a), h = hq / p.G;
        if (bad_values(p, b, h, lo, min(a, hi)).last < 0 && bad_values(p, b, h, z, hi).last < 0) return false;
    }
    redo_row(p, b, i, hq, o, m, l);
    return true;
}

__device__ __forceinline__ void store_out1(const PAttnPlan &p, int64_t off, float v) {
    if (p.out_dtype == DT_F32)
        static_cast<float *>(p.O)[off] = v;
    else if (p.out_dtype == DT_BF16)
        static_cast<__nv_bfloat16 *>(p.O)[off] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(p.O)[off] = __float2half_rn(v);
}
// Four consecutive channels of the output.
__device__ __forceinline__ void store_out4(const PAttnPlan &p, int64_t off, const float v[4]) {
    if (p.out_dtype == DT_F32)
        store4<DT_F32>(p.O, off, v);
    else if (p.out_dtype == DT_BF16)
        store4<DT_BF16>(p.O, off, v);
    else
        store4<DT_F16>(p.O, off, v);
}
__device__ __forceinline__ float row_lse(float m, float l) {
    return l > 0.f ? (m + fast_log2(l)) * kLn2 : (l == 0.f ? -INFINITY : l);  // NaN stays NaN
}

// Bounded wait on a phase: polls, and looks at the clock and the abort flag now and then.
constexpr uint64_t kPageWaitNs = 2000000000ull;  // a wait in the pipeline gives up after this
__device__ __forceinline__ bool page_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    if (mbar_try(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t n = 1; n < kSpinLimit; n++) {
        if (mbar_try(bar, parity)) return true;
        if ((n & 63u) == 0u) {
            if (*abort_flag) return false;
            const uint64_t now = global_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kPageWaitNs) break;
        }
    }
    *abort_flag = 1;
    return false;
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// The pool as rows of 128 channels, in boxes of `rows` rows that are 128 bytes wide (of a row
// of 8-bit codes, or of 64 channels in 16 bits), swizzled.
inline bool page_map(const PAttnPlan &p, const void *pool, int rows, CUtensorMap *map) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const bool wide = p.fmt == PF_F16 || p.fmt == PF_BF16;
    const CUtensorMapDataType dt = !wide              ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : p.fmt == PF_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)(p.n_pages * p.H * p.page)};
    const cuuint64_t strides[1] = {(cuuint64_t)(wide ? 2 * kD : kD)};
    const cuuint32_t box[2] = {wide ? 64u : (cuuint32_t)kD, (cuuint32_t)rows}, estr[2] = {1, 1};
    return enc(map, dt, 2, const_cast<void *>(pool), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Up to this many query rows (tokens x grouped heads) a sequence, attention is bound by reading
// the cache and runs on warp-level instructions (k_page_attn_rows.cu); above, on the tensor
// cores' own (k_page_attn_tc.cu).
constexpr int kRowsM = 16;
cudaError_t launch_page_attention_tc(const PAttnPlan &p, cudaStream_t st);

}  // namespace qvg
