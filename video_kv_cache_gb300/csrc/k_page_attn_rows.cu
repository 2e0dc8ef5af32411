// Attention of few query rows over paged keys and values: single new tokens, or a handful, of
// grouped query heads.
//   o = sum_j p_j v_j,  p = softmax over the visible keys j of scale * (q . k_j)
//
// Bound by memory: every cached byte is read once per key/value head and used for all rows
// (query tokens x grouped heads) of a 16-row tile, so the kernel is built around loads in
// flight.  A warp walks 16-key tiles with a running maximum and weight sum per row, straight
// from global memory to the registers of warp-level matrix instructions, with no pass through
// shared memory:
//   * scores: a dot product may take its channels in any order, so lane (g, q) = (lane / 4,
//     lane % 4) loads 16-byte chunks q, q + 4, ... of key g's row and feeds them to
//     successive 16-channel steps; Q is held in the same order.
//   * values: output channels may be numbered in any order, so column g of product tile t is
//     channel 8g + t (16g + t for 8-bit codes): lane (g, q) loads whole chunks of keys 2q,
//     2q + 1, 2q + 8 and 2q + 9 and pairs them up by byte permutations, and ends with whole
//     runs of channels to write.
// The keys of a row tile are cut into S splits (a CTA of four warps each, the warps taking
// alternate tiles); the warps' results are joined in shared memory, the splits' in
// k_page_combine.
#include "page_attn.cuh"

namespace qvg {

namespace {
constexpr int kRowsM = 16;      // query rows of a tile
constexpr int kRowsWarps = 4;   // warps of a CTA
constexpr int kRowsPad = 132;   // padded row of the join, floats

template <bool BF16>
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int w) {
    return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
}
}  // namespace

// grid (row tiles x splits, key/value heads, sequences).  QB: bf16 queries; FMT: the page
// format, the 16-bit ones (PF_F16 / PF_BF16) equal to the query's type.
template <bool QB, int FMT>
__global__ void __launch_bounds__(32 * kRowsWarps, 3) k_page_attn_rows(PAttnPlan p) {
    pdl_begin();
    constexpr bool WIDE = FMT == PF_F16 || FMT == PF_BF16;
    constexpr bool PVB = WIDE && QB;            // type of all operands; 8-bit pages: fp16
    constexpr int ROWB = WIDE ? 2 * kD : kD;    // bytes of a cached row
    constexpr int NCH = ROWB / 64;              // 16-byte chunks of a row per lane
    __shared__ float s_o[kRowsWarps][kRowsM][kRowsPad];
    __shared__ float s_m[kRowsWarps][kRowsM], s_l[kRowsWarps][kRowsM];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int rt = blockIdx.x / p.S, split = blockIdx.x - rt * p.S, h = blockIdx.y, b = blockIdx.z;
    const SeqInfo sq = seq_info(p, b, threadIdx.x == 0 && blockIdx.x == 0 && h == 0);
    const int rows = sq.qn * p.G, r0 = rt * kRowsM;
    if (r0 >= rows) return;
    const int shift = 31 - __clz(p.page);
    bool bad = false;

    // what this tile's rows see, this split's share of it
    const int i_first = r0 / p.G, i_last = (min(rows, r0 + kRowsM) - 1) / p.G;
    const int lo = seen_lo(p, sq, i_first), hi = seen_hi(p, sq, i_last);
    const int t_lo = lo >> 4, n_tiles = lo < hi ? ((hi + 15) >> 4) - t_lo : 0;
    const int per = (n_tiles + p.S - 1) / p.S;
    const int t0 = t_lo + split * per, t1 = t_lo + min(n_tiles, (split + 1) * per);
    // the two rows whose scores this lane holds
    int row_lo[2], row_hi[2];
#pragma unroll
    for (int x = 0; x < 2; x++) {
        const int i = min(r0 + g + 8 * x, rows - 1) / p.G;
        row_lo[x] = seen_lo(p, sq, i);
        row_hi[x] = seen_hi(p, sq, i);
    }

    // Q in the order the keys' chunks come in
    uint32_t qa[8][4];
    float qmul[2] = {1.f, 1.f};  // 8-bit pages: powers of two taken out of the rows of Q
    uint4 qraw[2][4];
#pragma unroll
    for (int x = 0; x < 2; x++) {
        const int r = r0 + g + 8 * x, i = r / p.G;
        const uint16_t *src = static_cast<const uint16_t *>(p.Q) + (sq.q0 + i) * p.qt + (int64_t)(h * p.G + r - i * p.G) * p.qh;
#pragma unroll
        for (int j = 0; j < 4; j++) {  // 8 channels: two steps
            const int ch = WIDE ? (j * 4 + q) * 8 : ((j >> 1) * 4 + q) * 16 + (j & 1) * 8;
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows) w = __ldg(reinterpret_cast<const uint4 *>(src + ch));
            if constexpr (!WIDE && QB) qraw[x][j] = w;
            qa[2 * j][x] = w.x;
            qa[2 * j][2 + x] = w.y;
            qa[2 * j + 1][x] = w.z;
            qa[2 * j + 1][2 + x] = w.w;
        }
    }

    if constexpr (!WIDE && QB) {
#pragma unroll
        for (int x = 0; x < 2; x++) {
            uint32_t big = 0;
#pragma unroll
            for (int j = 0; j < 4; j++) big = max(big, bf16x2_max_bits(qraw[x][j]));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            qmul[x] = bf16_pow2(big);
            const float inv = 1.f / qmul[x];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                qa[2 * j][x] = bf16x2_to_f16x2(qraw[x][j].x, inv);
                qa[2 * j][2 + x] = bf16x2_to_f16x2(qraw[x][j].y, inv);
                qa[2 * j + 1][x] = bf16x2_to_f16x2(qraw[x][j].z, inv);
                qa[2 * j + 1][2 + x] = bf16x2_to_f16x2(qraw[x][j].w, inv);
            }
        }
    }

    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int vexp = -100;  // exponent of the reference that the values' scales are taken against
#pragma unroll
    for (int t = 0; t < 16; t++) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

    const uint8_t *kp = static_cast<const uint8_t *>(p.k), *vp = static_cast<const uint8_t *>(p.v);
    auto row_of = [&](int t) {  // pool row of a tile's first key (a tile never leaves its page)
        return ((page_of(p, b, t * 16, shift, bad) * p.H + h) << shift) + ((t * 16) & (p.page - 1));
    };
    uint4 kr[2][NCH], vr[4][NCH / 2];
    float ksc[4], vsc[4];
    auto load_k = [&](int64_t row) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
#pragma unroll
            for (int c = 0; c < NCH; c++)
                kr[u][c] = __ldg(reinterpret_cast<const uint4 *>(kp + (row + u * 8 + g) * ROWB) + c * 4 + q);
            if constexpr (!WIDE) {
                const float2 f = __ldg(reinterpret_cast<const float2 *>(p.ks + row + u * 8 + 2 * q));
                ksc[2 * u] = f.x;
                ksc[2 * u + 1] = f.y;
            }
        }
    };
    auto load_v = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < 4; k++)
#pragma unroll
            for (int c = 0; c < NCH / 2; c++)
                vr[k][c] = __ldg(reinterpret_cast<const uint4 *>(
                    vp + (row + 2 * q + (k & 1) + (k >> 1) * 8) * ROWB) + c * 8 + g);
        if constexpr (!WIDE) {
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const float2 f = __ldg(reinterpret_cast<const float2 *>(p.vs + row + u * 8 + 2 * q));
                vsc[2 * u] = f.x;
                vsc[2 * u + 1] = f.y;
            }
        }
    };

    int t = t0 + warp;
    int64_t row = 0;
    if (t < t1) {
        row = row_of(t);
        load_k(row);
        load_v(row);
    }
    for (; t < t1; t += kRowsWarps) {
        const int64_t next = t + kRowsWarps < t1 ? row_of(t + kRowsWarps) : row;
        // scores of 16 keys: columns 8u + 2q, + 1 of rows g, g + 8
        float s[2][4] = {};
#pragma unroll
        for (int u = 0; u < 2; u++) {
#pragma unroll
            for (int c = 0; c < NCH; c++) {
                if constexpr (WIDE) {
                    mma16816<QB>(s[u], qa[2 * c], kr[u][c].x, kr[u][c].y);
                    mma16816<QB>(s[u], qa[2 * c + 1], kr[u][c].z, kr[u][c].w);
                } else {
#pragma unroll
                    for (int w = 0; w < 4; w++) {
                        const uint32_t codes = word_of(kr[u][c], w);
                        const uint2 k2 = codes_to_f16<FMT == PF_E4M3>(codes);
                        mma16816<PVB>(s[u], qa[4 * c + w], k2.x, k2.y);
                    }
                }
            }
        }
        const int key0 = t * 16 + 2 * q;
        const bool whole = t * 16 >= lo && t * 16 + 16 <= hi && sq.qn == 1;
#pragma unroll
        for (int u = 0; u < 2; u++) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float f = p.scale_log2;
                if constexpr (!WIDE) f *= ksc[2 * u + (e & 1)] * qmul[e >> 1];
                s[u][e] *= f;
                const int key = key0 + 8 * u + (e & 1), x = e >> 1;
                if (!whole && (key < row_lo[x] || key >= row_hi[x])) s[u][e] = -INFINITY;
            }
        }
        load_k(next);  // the keys are consumed: the next tile's are on their way meanwhile
        // 8-bit: the weights take in the values' scales relative to 2^vexp, an exponent that
        // follows the largest scale seen; times 2^8 they fill fp16's range
        float vmul = 0.f, vcorr = 1.f;
        if constexpr (!WIDE) {
            float big = 0.f;
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int key = key0 + (k & 1) + (k >> 1) * 8;
                if (key >= lo && key < hi) big = fmaxf(big, fabsf(vsc[k]));
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const int ve = max(vexp, min((int)(__float_as_uint(big) >> 23) - 127, 121));
            vcorr = __uint_as_float((uint32_t)max(127 + vexp - ve, 0) << 23);
            vmul = __uint_as_float((uint32_t)(127 + 8 - ve) << 23);
            vexp = ve;
        }
        float corr[2];
        uint32_t pa[4];
#pragma unroll
        for (int x = 0; x < 2; x++) {
            float mx = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx = fmaxf(m[x], mx);
            const float base = exp_base(mx);
            corr[x] = fast_exp2(m[x] - base);
            m[x] = mx;
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < 2; u++) {
                float w0 = fast_exp2(s[u][2 * x] - base), w1 = fast_exp2(s[u][2 * x + 1] - base);
                sum += w0 + w1;
                if constexpr (!WIDE) {  // a hidden key's scale may be NaN: its weight stays 0
                    w0 = s[u][2 * x] == -INFINITY ? 0.f : w0 * (vsc[2 * u] * vmul);
                    w1 = s[u][2 * x + 1] == -INFINITY ? 0.f : w1 * (vsc[2 * u + 1] * vmul);
                }
                pa[2 * u + x] = PVB ? pack_bf16(w0, w1) : pack_f16(w0, w1);
            }
            l[x] = l[x] * corr[x] + sum;
        }
        if constexpr (!WIDE) {
            corr[0] *= vcorr;
            corr[1] *= vcorr;
        }
        if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
            for (int n = 0; n < 16; n++) {
                o[n][0] *= corr[0];
                o[n][1] *= corr[0];
                o[n][2] *= corr[1];
                o[n][3] *= corr[1];
            }
        }
        // values that no row of the tile sees may hold anything
        if (t * 16 < lo || t * 16 + 16 > hi) {
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int key = key0 + (k & 1) + (k >> 1) * 8;
                if (key < lo || key >= hi)
#pragma unroll
                    for (int c = 0; c < NCH / 2; c++) vr[k][c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        if constexpr (WIDE) {
#pragma unroll
            for (int c = 0; c < 2; c++)
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    const uint32_t v0 = word_of(vr[0][c], w), v1 = word_of(vr[1][c], w),
                                   v2 = word_of(vr[2][c], w), v3 = word_of(vr[3][c], w);
                    mma16816<PVB>(o[c * 8 + 2 * w], pa, __byte_perm(v0, v1, 0x5410), __byte_perm(v2, v3, 0x5410));
                    mma16816<PVB>(o[c * 8 + 2 * w + 1], pa, __byte_perm(v0, v1, 0x7632), __byte_perm(v2, v3, 0x7632));
                }
        } else {
#pragma unroll
            for (int w = 0; w < 4; w++) {
                uint2 c[4];
#pragma unroll
                for (int k = 0; k < 4; k++) c[k] = codes_to_f16<FMT == PF_E4M3>(word_of(vr[k][0], w));
                mma16816<PVB>(o[4 * w], pa, __byte_perm(c[0].x, c[1].x, 0x5410), __byte_perm(c[2].x, c[3].x, 0x5410));
                mma16816<PVB>(o[4 * w + 1], pa, __byte_perm(c[0].x, c[1].x, 0x7632), __byte_perm(c[2].x, c[3].x, 0x7632));
                mma16816<PVB>(o[4 * w + 2], pa, __byte_perm(c[0].y, c[1].y, 0x5410), __byte_perm(c[2].y, c[3].y, 0x5410));
                mma16816<PVB>(o[4 * w + 3], pa, __byte_perm(c[0].y, c[1].y, 0x7632), __byte_perm(c[2].y, c[3].y, 0x7632));
            }
        }
        load_v(next);
        row = next;
    }
    if (bad) or_status(p.status, QVG_DEV_BAD_INDEX);

    // join the warps
    const float unit = WIDE ? 1.f : __uint_as_float((uint32_t)(127 + vexp - 8) << 23);
#pragma unroll
    for (int x = 0; x < 2; x++) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        if (q == 0) {
            s_m[warp][g + 8 * x] = m[x];
            s_l[warp][g + 8 * x] = l[x];
        }
#pragma unroll
        for (int n = 0; n < 16; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int col = 2 * q + e;
                const int ch = WIDE ? (n >> 3) * 64 + col * 8 + (n & 7) : col * 16 + n;
                s_o[warp][g + 8 * x][ch] = o[n][2 * x + e] * unit;
            }
    }
    __syncthreads();
    // eight lanes a row, 16 channels each (in runs of four, so that the lanes' reads and
    // writes are next to one another)
    const int r = threadIdx.x >> 3, part = threadIdx.x & 7;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kRowsWarps; w++) M = fmaxf(M, s_m[w][r]);
    const float base = exp_base(M);
    float L = 0.f, v[16] = {};
#pragma unroll
    for (int w = 0; w < kRowsWarps; w++) {
        const float f = fast_exp2(s_m[w][r] - base);
        L += f * s_l[w][r];
#pragma unroll
        for (int c = 0; c < 16; c++) v[c] += f * s_o[w][r][(c >> 2) * 32 + part * 4 + (c & 3)];
    }
    const int row_i = (r0 + r) / p.G, hq = h * p.G + (r0 + r) - row_i * p.G;
    const bool live = r0 + r < rows;
    if (p.S > 1) {
        if (!live) return;
        const int64_t at = ((int64_t)split * p.total_q + sq.q0 + row_i) * p.HQ + hq;
#pragma unroll
        for (int c = 0; c < 4; c++) store4<DT_F32>(p.part, at * kD + c * 32 + part * 4, v + 4 * c);
        if (part == 0) *reinterpret_cast<float2 *>(p.ml + 2 * at) = make_float2(M, L);
        return;
    }
    if (redo_possible(p)) {
        bool odd = false;
#pragma unroll
        for (int c = 0; c < 16; c++) odd |= !is_finite(v[c]);
        uint32_t todo = __ballot_sync(0xffffffffu, odd && live);
        while (todo) {
            const int first = (__ffs(todo) - 1) & ~7;  // the row's first lane
            todo &= ~(0xFFu << first);
            float ro[4], rm, rl;
            redo_row(p, b, __shfl_sync(0xffffffffu, row_i, first), __shfl_sync(0xffffffffu, hq, first), ro, rm, rl);
            // lane x has channels 4x ..: this thread's are those of lanes part + 8 c
#pragma unroll
            for (int c = 0; c < 16; c++) {
                const float y = __shfl_sync(0xffffffffu, ro[c & 3], (c >> 2) * 8 + part);
                if ((lane & ~7) == first) v[c] = y;
            }
            if ((lane & ~7) == first) {
                M = rm;
                L = rl;
            }
        }
    }
    if (!live) return;
    const float inv = L == 0.f ? 0.f : __fdiv_rn(1.f, L);
    const int64_t at = (sq.q0 + row_i) * p.ot + hq * p.oh;
#pragma unroll
    for (int c = 0; c < 16; c++) v[c] *= inv;
#pragma unroll
    for (int c = 0; c < 4; c++) store_out4(p, at + c * 32 + part * 4, v + 4 * c);
    if (p.lse && part == 0) p.lse[(sq.q0 + row_i) * p.HQ + hq] = row_lse(M, L);
}

// One warp per query row (of all sequences): the splits' partial rows rescaled to the largest
// maximum and summed.  Lane l writes channels 4l .. 4l+3.  Rows of no sequence are skipped.
__global__ void __launch_bounds__(256) k_page_combine(PAttnPlan p) {
    pdl_begin();
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (w >= p.total_q * p.HQ) return;
    const int64_t token = w / p.HQ;
    const int hq = (int)(w - token * p.HQ);
    // the row's sequence: the last one that starts at or before it
    int b;
    if (p.cu) {
        int a = 0, e = p.B;  // cu[a] <= token < cu[e], where the order of cu allows
        while (e - a > 1) {
            const int mid = (a + e) / 2;
            if (__ldg(p.cu + mid) <= token) a = mid; else e = mid;
        }
        b = a;
    } else {
        b = (int)min(token / p.max_q, (int64_t)p.B - 1);
    }
    const SeqInfo sq = seq_info(p, b, false);
    if (token < sq.q0 || token >= sq.q0 + sq.qn) return;
    const int64_t stride = p.total_q * p.HQ;
    float mx = -INFINITY;
    for (int s = lane; s < p.S; s += 32) mx = fmaxf(mx, p.ml[2 * (s * stride + w)]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float base = exp_base(mx);
    float l = 0.f, o[4] = {};
    constexpr int SB = 8;
    for (int s0 = 0; s0 < p.S; s0 += SB) {
        float2 ml[SB];
        float4 po[SB];
#pragma unroll
        for (int u = 0; u < SB; u++)
            if (s0 + u < p.S) {
                const int64_t at = (s0 + u) * stride + w;
                ml[u] = *reinterpret_cast<const float2 *>(p.ml + 2 * at);
                po[u] = *reinterpret_cast<const float4 *>(p.part + at * kD + 4 * lane);
            }
#pragma unroll
        for (int u = 0; u < SB; u++)
            if (s0 + u < p.S) {
                const float f = fast_exp2(ml[u].x - base);
                l += f * ml[u].y;
                o[0] += f * po[u].x;
                o[1] += f * po[u].y;
                o[2] += f * po[u].z;
                o[3] += f * po[u].w;
            }
    }
    if (redo_possible(p) &&
        __any_sync(0xffffffffu, !is_finite(o[0]) || !is_finite(o[1]) || !is_finite(o[2]) || !is_finite(o[3])))
        redo_row(p, b, (int)(token - sq.q0), hq, o, mx, l);
    const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
#pragma unroll
    for (int c = 0; c < 4; c++) o[c] *= inv;
    store_out4(p, token * p.ot + hq * p.oh + 4 * lane, o);
    if (p.lse && lane == 0) p.lse[token * p.HQ + hq] = row_lse(mx, l);
}

// Splits of the keys.  Few rows: enough CTAs to give every SM three of them (what their
// registers allow) about once, while each warp keeps at least four tiles.  Many rows: CTAs run
// one an SM, so the time is about the number of rounds times the tiles of one CTA; the split
// that makes it least is taken, counting a tile's worth of work for starting a CTA and the
// traffic of the partial results (two tiles for a pair of row tiles).
int page_attention_splits(const PAttnPlan &p) {
    const int64_t rows = p.max_q * p.G, cells = (int64_t)p.H * p.B;
    if (rows <= kRowsMost) {
        const int64_t want = (152 * 3 + cells - 1) / cells;
        const int64_t most = (p.max_kv + 16 * kRowsWarps * 4 - 1) / (16 * kRowsWarps * 4);
        return (int)std::max<int64_t>(1, std::min<int64_t>({want, most, 256}));
    }
    const int64_t pairs = (rows + 255) / 256 * cells, tiles = (p.max_kv + 127) / 128;
    int best = 1;
    double least = 1e300;
    for (int s = 1; s <= 64 && s <= std::max<int64_t>(1, tiles / 4); s++) {
        const double rounds = (double)((pairs * s + 151) / 152);
        const double t = rounds * ((double)((tiles + s - 1) / s) + 2.0) + (s > 1 ? 2.0 * s * pairs / 152 + 4.0 : 0.0);
        if (t < least * 0.97) {
            least = t;
            best = s;
        }
    }
    return best;
}

cudaError_t launch_page_attention_rows(const PAttnPlan &p, cudaStream_t st) {
    const int64_t rts = (p.max_q * p.G + kRowsM - 1) / kRowsM;
    const dim3 grid((unsigned)(rts * p.S), p.H, p.B);
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(32 * kRowsWarps), 0, st, p); };
    cudaError_t e;
    if (p.q_dtype == DT_BF16)
        e = p.fmt == PF_E4M3   ? go(k_page_attn_rows<true, PF_E4M3>)
            : p.fmt == PF_INT8 ? go(k_page_attn_rows<true, PF_INT8>)
                               : go(k_page_attn_rows<true, PF_BF16>);
    else
        e = p.fmt == PF_E4M3   ? go(k_page_attn_rows<false, PF_E4M3>)
            : p.fmt == PF_INT8 ? go(k_page_attn_rows<false, PF_INT8>)
                               : go(k_page_attn_rows<false, PF_F16>);
    return e;
}

cudaError_t launch_page_attention(const PAttnPlan &p, cudaStream_t st) {
    const cudaError_t e =
        p.max_q * p.G <= kRowsMost ? launch_page_attention_rows(p, st) : launch_page_attention_tc(p, st);
    if (e != cudaSuccess || p.S == 1) return e;
    return launch_kernel(k_page_combine, dim3((unsigned)((p.total_q * p.HQ + 7) / 8)), dim3(256), 0, st, p);
}

}  // namespace qvg
