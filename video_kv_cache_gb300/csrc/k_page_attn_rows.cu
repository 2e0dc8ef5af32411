// Attention of few query rows over paged keys and values: single new tokens, or a handful, of
// grouped query heads.
//   o = sum_j p_j v_j,  p = softmax over the visible keys j of scale * (q . k_j)
//
// Bound by memory: every cached byte is read once per key/value head and used for all rows
// (query tokens x grouped query heads, at most 16).  One warp of a CTA streams the keys' and
// values' pages by TMA into a ring of 64-key stages (about 100 KB in flight a CTA, two CTAs an
// SM: several times what the memory's latency needs); four warps take a 16-key tile of each
// stage, with a running maximum and weight sum per row, on warp-level matrix instructions:
//   * scores: a dot product may take its channels in any order, so lane (g, q) = (lane / 4,
//     lane % 4) reads 16-byte chunks q, q + 4, ... of key g's row and feeds them to successive
//     16-channel steps; Q is held in the same order.
//   * values: output channels may be numbered in any order, so column g of product tile t is
//     channel 8g + t (16g + t for 8-bit codes): lane (g, q) reads whole chunks of keys 2q,
//     2q + 1, 2q + 8 and 2q + 9, pairs them up by byte permutations, and ends with whole runs
//     of channels to write.  The stages are swizzled (128 bytes), which keeps these reads off
//     each other's banks.
// The keys are cut into S splits, a CTA each.  The warps' results are joined in shared memory;
// the splits', where there are at most eight, by a cluster of the S CTAs through each other's
// shared memory (one launch, no workspace), else through memory by k_page_combine.
#include "page_attn.cuh"
#include "tcgen.cuh"

namespace qvg {

namespace {
constexpr int kRowsWarps = 4;              // warps that compute
constexpr int kRowsThreads = 32 * (kRowsWarps + 1);
constexpr int kStageKeys = 16 * kRowsWarps;
constexpr int kRowsPad = 132;              // padded row of the join, floats
constexpr int kRowsCluster = 8;            // most splits joined by a cluster

template <int FMT>
struct RowsShape {
    static constexpr bool WIDE = FMT == PF_F16 || FMT == PF_BF16;
    static constexpr int STAGES = WIDE ? 3 : 6;
    static constexpr uint32_t TILE = kStageKeys * kD * (WIDE ? 2 : 1);  // keys or values of a stage
};
template <int FMT>
struct RowsShared {
    float ks[RowsShape<FMT>::STAGES][RowsShape<FMT>::WIDE ? 4 : kStageKeys];
    float vs[RowsShape<FMT>::STAGES][RowsShape<FMT>::WIDE ? 4 : kStageKeys];
    uint64_t full[RowsShape<FMT>::STAGES], empty[RowsShape<FMT>::STAGES];
    float m[kRowsWarps][kRowsM], l[kRowsWarps][kRowsM];
    float2 ml[kRowsM];  // this split's maximum and sum, for the cluster
    int abort;
};
// The join's rows take the ring's place once the keys are through.
template <int FMT>
constexpr size_t rows_smem() {
    constexpr size_t bytes = RowsShape<FMT>::STAGES * 2 * RowsShape<FMT>::TILE + sizeof(RowsShared<FMT>);
    static_assert(2 * (bytes + 1024) <= 228 * 1024, "two CTAs an SM");
    static_assert((kRowsWarps + 1) * kRowsM * kRowsPad * 4 <= RowsShape<FMT>::STAGES * 2 * RowsShape<FMT>::TILE, "join");
    return bytes;
}

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
__device__ __forceinline__ uint32_t cluster_addr(const void *p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
}  // namespace

// grid (splits, key/value heads, sequences).  QB: bf16 queries; FMT: the page format, the
// 16-bit ones (PF_F16 / PF_BF16) equal to the query's type.  joined: the splits are a cluster.
template <bool QB, int FMT>
__global__ void __launch_bounds__(kRowsThreads, 2)
    k_page_attn_rows(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ PAttnPlan p, int joined) {
    pdl_begin();
    using T = RowsShape<FMT>;
    constexpr bool WIDE = T::WIDE;
    constexpr bool PVB = WIDE && QB;            // type of all operands; 8-bit pages: fp16
    constexpr int ROWB = WIDE ? 2 * kD : kD;    // bytes of a cached row
    constexpr int NCH = ROWB / 64;              // 16-byte chunks of a row per lane
    constexpr int STAGES = T::STAGES;
    extern __shared__ __align__(1024) unsigned char sm[];
    RowsShared<FMT> &sh = *reinterpret_cast<RowsShared<FMT> *>(sm + STAGES * 2 * T::TILE);
    float(*s_o)[kRowsM][kRowsPad] = reinterpret_cast<float(*)[kRowsM][kRowsPad]>(sm);
    volatile int *abort_flag = &sh.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const SeqInfo sq = seq_info(p, b, threadIdx.x == 0 && blockIdx.x == 0 && h == 0);
    const int rows = sq.qn * p.G;
    if (rows == 0) return;
    const int shift = 31 - __clz(p.page);

    // what the rows see, this split's share of it, in stages of 64 keys
    const int lo = seen_lo(p, sq, 0), hi = seen_hi(p, sq, sq.qn - 1);
    int first = 0, n = 0;
    if (lo < hi) {
        const int s_lo = lo / kStageKeys, all = (hi + kStageKeys - 1) / kStageKeys - s_lo, per = (all + p.S - 1) / p.S;
        first = s_lo + split * per;
        n = max(0, min(per, all - split * per));
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), kRowsWarps);
        }
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int vexp = -100;  // exponent of the reference that the values' scales are taken against
    if (warp == kRowsWarps) {
        // -------------------------------------------------------------------- TMA loads
        const int box = min(p.page, kStageKeys), boxes = kStageKeys / box;
        bool bad = false, ok = true;
        int issued = 0;
        // the boxes of a stage that hold a key some row sees, a lane each; their pages are
        // looked up one stage ahead
        auto in_sight = [&](int k0) {
            const int token = k0 + lane * box;
            return lane < boxes && token < hi && token + box > lo;
        };
        auto row_of = [&](int k0) {
            const int token = k0 + lane * box;
            if (!in_sight(k0)) return 0;
            return (int)(((page_of(p, b, token, shift, bad) * p.H + h) << shift) + (token & (p.page - 1)));
        };
        int next = n > 0 ? row_of(first * kStageKeys) : 0;
        for (int it = 0; it < n; it++) {
            const int k0 = (first + it) * kStageKeys, s = it % STAGES, row = next;
            if (it + 1 < n) next = row_of(k0 + kStageKeys);
            ok = page_wait(smem_u32(&sh.empty[s]), (it / STAGES + 1) & 1, abort_flag);
            if (__any_sync(0xffffffffu, !ok)) break;
            const uint32_t bar = smem_u32(&sh.full[s]), count = __popc(__ballot_sync(0xffffffffu, in_sight(k0)));
            if (lane == 0) mbar_expect_tx(bar, count * box * 2 * (ROWB + (WIDE ? 0 : 4)));
            __syncwarp();
            if (in_sight(k0)) {
                const uint32_t at = smem_u32(sm) + s * 2 * T::TILE + lane * box * 128;
                tma_load_2d(at, &tmK, 0, row, bar);
                tma_load_2d(at + T::TILE, &tmV, 0, row, bar);
                if constexpr (WIDE) {
                    tma_load_2d(at + T::TILE / 2, &tmK, 64, row, bar);
                    tma_load_2d(at + T::TILE + T::TILE / 2, &tmV, 64, row, bar);
                } else {
                    bulk_g2s(smem_u32(&sh.ks[s][lane * box]), p.ks + row, box * 4, bar);
                    bulk_g2s(smem_u32(&sh.vs[s][lane * box]), p.vs + row, box * 4, bar);
                }
            }
            issued = it + 1;
        }
        if (bad) or_status(p.status, QVG_DEV_BAD_INDEX);
        // every copy lands before the CTA goes on to the join (or ends)
        for (int it = max(0, issued - STAGES); it < issued; it++)
            mbar_wait_final(smem_u32(&sh.full[it % STAGES]), (it / STAGES) & 1);
    } else {
        // -------------------------------------------------------------------- attention
        // the two rows whose scores this lane holds
        int row_lo[2], row_hi[2];
        // Q in the order the keys' chunks come in
        uint32_t qa[8][4];
        float qmul[2] = {1.f, 1.f};  // 8-bit pages: powers of two taken out of the rows of Q
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const int r = g + 8 * x, i = min(r, rows - 1) / p.G;
            row_lo[x] = seen_lo(p, sq, i);
            row_hi[x] = seen_hi(p, sq, i);
            const uint16_t *src = static_cast<const uint16_t *>(p.Q) + (sq.q0 + i) * p.qt + (int64_t)(h * p.G + r - i * p.G) * p.qh;
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {  // 8 channels: two steps
                const int ch = WIDE ? (j * 4 + q) * 8 : ((j >> 1) * 4 + q) * 16 + (j & 1) * 8;
                w[j] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(src + ch)) : make_uint4(0u, 0u, 0u, 0u);
            }
            if constexpr (!WIDE && QB) {
                uint32_t big = 0;
#pragma unroll
                for (int j = 0; j < 4; j++) big = max(big, bf16x2_max_bits(w[j]));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                qmul[x] = bf16_pow2(big);
                const float inv = 1.f / qmul[x];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    w[j] = make_uint4(bf16x2_to_f16x2(w[j].x, inv), bf16x2_to_f16x2(w[j].y, inv),
                                      bf16x2_to_f16x2(w[j].z, inv), bf16x2_to_f16x2(w[j].w, inv));
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                qa[2 * j][x] = w[j].x;
                qa[2 * j][2 + x] = w[j].y;
                qa[2 * j + 1][x] = w[j].z;
                qa[2 * j + 1][2 + x] = w[j].w;
            }
        }
#pragma unroll
        for (int t = 0; t < 16; t++) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

        // chunk c of row r of a swizzled tile of `rows of 128 bytes` (16 bits: two halves)
        auto chunk = [](const unsigned char *tile, int r, int c) {
            return *reinterpret_cast<const uint4 *>(tile + (c >> 3) * (T::TILE / 2) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
        };
        for (int it = 0; it < n; it++) {
            const int st = it % STAGES, t0 = (first + it) * kStageKeys + warp * 16;  // this warp's first key
            const bool ok = page_wait(smem_u32(&sh.full[st]), (it / STAGES) & 1, abort_flag);
            if (__any_sync(0xffffffffu, !ok)) break;
            if (t0 < hi && t0 + 16 > lo) {
                const unsigned char *kt = sm + st * 2 * T::TILE, *vt = kt + T::TILE;
                float s[2][4] = {};
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    uint4 kr[NCH];
#pragma unroll
                    for (int c = 0; c < NCH; c++) kr[c] = chunk(kt, warp * 16 + u * 8 + g, c * 4 + q);
#pragma unroll
                    for (int c = 0; c < NCH; c++) {
                        if constexpr (WIDE) {
                            mma16816<QB>(s[u], qa[2 * c], kr[c].x, kr[c].y);
                            mma16816<QB>(s[u], qa[2 * c + 1], kr[c].z, kr[c].w);
                        } else {
#pragma unroll
                            for (int w = 0; w < 4; w++) {
                                const uint2 k2 = codes_to_f16<FMT == PF_E4M3>(word_of(kr[c], w));
                                mma16816<false>(s[u], qa[4 * c + w], k2.x, k2.y);
                            }
                        }
                    }
                }
                // the values are on their way to registers during the softmax
                uint4 vr[4][NCH / 2];
#pragma unroll
                for (int k = 0; k < 4; k++)
#pragma unroll
                    for (int c = 0; c < NCH / 2; c++)
                        vr[k][c] = chunk(vt, warp * 16 + 2 * q + (k & 1) + (k >> 1) * 8, c * 8 + g);
                // columns 8u + 2q, + 1 of rows g, g + 8
                const int key0 = t0 + 2 * q;
                const bool edge = t0 < lo || t0 + 16 > hi;
                float vsc[4];
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    float2 f = make_float2(p.scale_log2, p.scale_log2);
                    if constexpr (!WIDE) {
                        const float2 k2 = *reinterpret_cast<const float2 *>(&sh.ks[st][warp * 16 + 8 * u + 2 * q]);
                        const float2 v2 = *reinterpret_cast<const float2 *>(&sh.vs[st][warp * 16 + 8 * u + 2 * q]);
                        f.x *= k2.x;
                        f.y *= k2.y;
                        vsc[2 * u] = v2.x;
                        vsc[2 * u + 1] = v2.y;
                    }
                    s[u][0] *= f.x * qmul[0];
                    s[u][1] *= f.y * qmul[0];
                    s[u][2] *= f.x * qmul[1];
                    s[u][3] *= f.y * qmul[1];
                    if (edge || sq.qn > 1) {
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const int key = key0 + 8 * u + (e & 1), x = e >> 1;
                            if (key < row_lo[x] || key >= row_hi[x]) s[u][e] = -INFINITY;
                        }
                    }
                }
                // 8-bit: the weights take in the values' scales relative to 2^vexp, an exponent
                // that follows the largest scale seen; times 2^8 they fill fp16's range
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
                    for (int k = 0; k < 16; k++) {
                        o[k][0] *= corr[0];
                        o[k][1] *= corr[0];
                        o[k][2] *= corr[1];
                        o[k][3] *= corr[1];
                    }
                }
                // values that no row sees may hold anything
                if (edge) {
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
                        // the codes of two keys interleaved, then widened pair by pair
                        const uint32_t v0 = word_of(vr[0][0], w), v1 = word_of(vr[1][0], w),
                                       v2 = word_of(vr[2][0], w), v3 = word_of(vr[3][0], w);
                        const uint2 a = codes_to_f16<FMT == PF_E4M3>(__byte_perm(v0, v1, 0x5140)),
                                    c = codes_to_f16<FMT == PF_E4M3>(__byte_perm(v0, v1, 0x7362)),
                                    d = codes_to_f16<FMT == PF_E4M3>(__byte_perm(v2, v3, 0x5140)),
                                    e = codes_to_f16<FMT == PF_E4M3>(__byte_perm(v2, v3, 0x7362));
                        mma16816<false>(o[4 * w], pa, a.x, d.x);
                        mma16816<false>(o[4 * w + 1], pa, a.y, d.y);
                        mma16816<false>(o[4 * w + 2], pa, c.x, e.x);
                        mma16816<false>(o[4 * w + 3], pa, c.y, e.y);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.empty[st]));
        }
    }

    // join the warps, in the ring's place
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) or_status(p.status, QVG_DEV_TIMEOUT);
    if (warp < kRowsWarps) {
        const float unit = WIDE ? 1.f : __uint_as_float((uint32_t)(127 + vexp - 8) << 23);
#pragma unroll
        for (int x = 0; x < 2; x++) {
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
            if (q == 0) {
                sh.m[warp][g + 8 * x] = m[x];
                sh.l[warp][g + 8 * x] = l[x];
            }
#pragma unroll
            for (int k = 0; k < 16; k++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int col = 2 * q + e;
                    const int ch = WIDE ? (k >> 3) * 64 + col * 8 + (k & 7) : col * 16 + k;
                    s_o[warp][g + 8 * x][ch] = o[k][2 * x + e] * unit;
                }
        }
    }
    __syncthreads();
    // eight lanes a row, 16 channels each (in runs of four, so that the lanes' reads and
    // writes are next to one another); the fifth warp only keeps the barriers
    const int r = threadIdx.x >> 3, part = threadIdx.x & 7;
    float M = -INFINITY, L = 0.f, v[16] = {};
    const bool mine = warp < kRowsWarps;
    if (mine) {
#pragma unroll
        for (int w = 0; w < kRowsWarps; w++) M = fmaxf(M, sh.m[w][r]);
        const float base = exp_base(M);
#pragma unroll
        for (int w = 0; w < kRowsWarps; w++) {
            const float f = fast_exp2(sh.m[w][r] - base);
            L += f * sh.l[w][r];
#pragma unroll
            for (int c = 0; c < 16; c++) v[c] += f * s_o[w][r][(c >> 2) * 32 + part * 4 + (c & 3)];
        }
    }
    const int row_i = min(r, rows - 1) / p.G, hq = h * p.G + min(r, rows - 1) - row_i * p.G;
    bool live = mine && r < rows;
    if (p.S > 1 && !joined) {
        if (!live) return;
        const int64_t at = ((int64_t)split * p.total_q + sq.q0 + row_i) * p.HQ + hq;
#pragma unroll
        for (int c = 0; c < 4; c++) store4<DT_F32>(p.part, at * kD + c * 32 + part * 4, v + 4 * c);
        if (part == 0) *reinterpret_cast<float2 *>(p.ml + 2 * at) = make_float2(M, L);
        return;
    }
    if (joined) {
        // each CTA of the cluster finishes the rows r with r % S its rank
        if (mine) {
#pragma unroll
            for (int c = 0; c < 4; c++)
                *reinterpret_cast<float4 *>(&s_o[kRowsWarps][r][c * 32 + part * 4]) =
                    make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            if (part == 0) sh.ml[r] = make_float2(M, L);
        }
        cluster_meet();
        live = live && r % p.S == split;
        if (live) {
            M = -INFINITY;
            for (int s = 0; s < p.S; s++) M = fmaxf(M, ld_cluster2(cluster_addr(&sh.ml[r], s)).x);
            const float base = exp_base(M);
            L = 0.f;
#pragma unroll
            for (int c = 0; c < 16; c++) v[c] = 0.f;
            for (int s = 0; s < p.S; s++) {
                const float2 ml = ld_cluster2(cluster_addr(&sh.ml[r], s));
                const float f = fast_exp2(ml.x - base);
                L += f * ml.y;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const float4 y = ld_cluster4(cluster_addr(&s_o[kRowsWarps][r][c * 32 + part * 4], s));
                    v[4 * c] += f * y.x;
                    v[4 * c + 1] += f * y.y;
                    v[4 * c + 2] += f * y.z;
                    v[4 * c + 3] += f * y.w;
                }
            }
        }
        cluster_meet();  // nobody leaves while its rows are read
    }
    if (!mine) return;
    if (redo_possible(p)) {
        bool odd = false;
#pragma unroll
        for (int c = 0; c < 16; c++) odd |= !is_finite(v[c]);
        uint32_t todo = __ballot_sync(0xffffffffu, odd && live);
        while (todo) {
            const int src = (__ffs(todo) - 1) & ~7;  // the row's first lane
            todo &= ~(0xFFu << src);
            float ro[4], rm, rl;
            redo_row(p, b, __shfl_sync(0xffffffffu, row_i, src), __shfl_sync(0xffffffffu, hq, src), ro, rm, rl);
            // lane x has channels 4x ..: this thread's are those of lanes part + 8 c
#pragma unroll
            for (int c = 0; c < 16; c++) {
                const float y = __shfl_sync(0xffffffffu, ro[c & 3], (c >> 2) * 8 + part);
                if ((lane & ~7) == src) v[c] = y;
            }
            if ((lane & ~7) == src) {
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

// Splits of the keys.  Few rows: enough CTAs to give every SM two of them (what their shared
// memory allows) about once, while each keeps at least four stages; not more than a cluster
// joins unless twice as many are wanted.  Many rows: CTAs run one an SM, so the time is about
// the number of rounds times the tiles of one CTA; the split that makes it least is taken,
// counting a few tiles' worth of work for starting a CTA and for the partial results.
int page_attention_splits(const PAttnPlan &p) {
    const int64_t rows = p.max_q * p.G, cells = (int64_t)p.H * p.B;
    if (rows <= kRowsM) {
        const int64_t want = (152 * 2 + cells - 1) / cells;
        const int64_t most = (p.max_kv + kStageKeys * 4 - 1) / (kStageKeys * 4);
        const int64_t s = std::max<int64_t>(1, std::min<int64_t>({want, most, 256}));
        return (int)(s > kRowsCluster && s < 2 * kRowsCluster ? kRowsCluster : s);
    }
    const int64_t pairs = (rows + 255) / 256 * cells, tiles = (p.max_kv + 127) / 128;
    int best = 1;
    double least = 1e300;
    for (int s = 1; s <= 64 && s <= std::max<int64_t>(1, tiles / 4); s++) {
        const double rounds = (double)((pairs * s + 151) / 152);
        const double t = rounds * ((double)((tiles + s - 1) / s) + 6.0) + (s > 1 ? 2.0 * s * pairs / 152 + 4.0 : 0.0);
        if (t < least * 0.97) {
            least = t;
            best = s;
        }
    }
    return best;
}
// Whether the splits go through memory (else there is one, or a cluster joins them).
bool page_attention_parts(const PAttnPlan &p) {
    return p.S > (p.max_q * p.G <= kRowsM ? kRowsCluster : 1);
}

namespace {
template <bool QB, int FMT>
cudaError_t launch_rows(const PAttnPlan &p, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st) {
    constexpr size_t smem = rows_smem<FMT>();
    const auto kernel = k_page_attn_rows<QB, FMT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int joined = p.S > 1 && p.S <= kRowsCluster;
    return launch_kernel_cluster(kernel, dim3((unsigned)p.S, p.H, p.B), dim3(kRowsThreads), smem, joined ? p.S : 1, st,
                                 mk, mv, p, joined);
}

cudaError_t launch_page_attention_rows(const PAttnPlan &p, cudaStream_t st) {
    CUtensorMap mk, mv;
    const int box = std::min(p.page, kStageKeys);
    if (!page_map(p, p.k, box, &mk) || !page_map(p, p.v, box, &mv)) return cudaErrorInvalidValue;
    if (p.q_dtype == DT_BF16)
        return p.fmt == PF_E4M3   ? launch_rows<true, PF_E4M3>(p, mk, mv, st)
               : p.fmt == PF_INT8 ? launch_rows<true, PF_INT8>(p, mk, mv, st)
                                  : launch_rows<true, PF_BF16>(p, mk, mv, st);
    return p.fmt == PF_E4M3   ? launch_rows<false, PF_E4M3>(p, mk, mv, st)
           : p.fmt == PF_INT8 ? launch_rows<false, PF_INT8>(p, mk, mv, st)
                              : launch_rows<false, PF_F16>(p, mk, mv, st);
}
}  // namespace

cudaError_t launch_page_attention(const PAttnPlan &p, cudaStream_t st) {
    const cudaError_t e =
        p.max_q * p.G <= kRowsM ? launch_page_attention_rows(p, st) : launch_page_attention_tc(p, st);
    if (e != cudaSuccess || !page_attention_parts(p)) return e;
    return launch_kernel(k_page_combine, dim3((unsigned)((p.total_q * p.HQ + 7) / 8)), dim3(256), 0, st, p);
}

}  // namespace qvg
