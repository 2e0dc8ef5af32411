// Attention of few query rows over paged keys and values: single new tokens, or a handful, of
// grouped query heads.
//   o = sum_j p_j v_j,  p = softmax over the visible keys j of scale * (q . k_j)
//
// Bound by memory: every cached byte is read once per key/value head and used for all rows
// (query tokens x grouped query heads, at most 16).  One warp of a CTA streams the keys' and
// values' pages by TMA into a ring of stages of 64 or 128 keys (about 100 KB in flight a CTA,
// two CTAs an SM: several times what the memory's latency needs).  One query of 32 sequences of
// 15000 tokens, 8 heads, back to back: bf16 278 us (7.1 TB/s), e4m3 and int8 161 us (6.1 TB/s; the
// latencies of widening and softmax, two computing warps a scheduler).  Of each stage four warps take a
// quarter, with a running maximum and weight sum per row, on warp-level matrix instructions (the
// tensor cores' own take 128 rows at a time, at most 16 of which would be in use):
//   * scores S^T = K Q^T: the keys are the product's 16 rows and the queries its columns, eight
//     at a time, so that one or two grouped heads' worth of rows wastes little.  A dot product
//     may take its channels in any order, so lane (g, q) = (lane / 4, lane % 4) reads 16-byte
//     chunks q, q + 4, ... of the rows of keys g and g + 8 and feeds them to successive
//     16-channel steps; Q is held in the same order.
//   * outputs O^T = V^T P^T: the weights turn from the scores' layout into an operand's by one
//     8 x 8 transposition instruction each.  Output channels may be numbered in any order, so
//     row g of product tile t is channel 8g + t and row g + 8 channel 64 + 8g + t (8-bit codes:
//     16g + t and 16g + 8 + t): lane (g, q) reads whole chunks of keys 2q, 2q + 1, 2q + 8 and
//     2q + 9, pairs them up by byte permutations, and ends with whole runs of channels to
//     write.  The stages are swizzled (128 bytes), which keeps these reads off each other's
//     banks.
// Scores, sums and outputs are fp32; the weights are rounded to the product's 16-bit type (fp16
// over 8-bit pages).
//
// The keys are cut into S splits, a CTA each.  The warps' results are joined in shared memory;
// the splits', where there are at most eight, by a cluster of the S CTAs through each other's
// shared memory (one launch, no workspace), else through memory by k_page_combine.  Or
// (SHARES) the keys of all heads, in a row, are cut into as many equal shares as CTAs run at
// once, each worked through item by item, the next one's loads running while the last one is
// joined; a head that more than one share has a part of is joined by k_page_combine.
#include "page_attn.cuh"
#include "tcgen.cuh"

namespace qvg {

namespace {
constexpr int kRowsWarps = 4;              // warps that compute
constexpr int kRowsThreads = 32 * (kRowsWarps + 1);
constexpr int kRowsShares = 152 * 2;       // CTAs that run at once
constexpr int kRowsPad = 132;              // padded row of the join, floats
constexpr int kRowsCluster = 8;            // most splits joined by a cluster
constexpr int kRowsShare = 4;              // stages of a share, at least

// RT: groups of eight query rows, one or two.
template <int FMT, int RT>
struct RowsShape {
    static constexpr bool WIDE = FMT == PF_F16 || FMT == PF_BF16;
    // 16-key tiles that a warp takes at a time: widening codes is a chain of short
    // instructions, which needs more of them side by side than feeding 16-bit rows does
    static constexpr int KT = WIDE ? 1 : 2;
    static constexpr int KEYS = 16 * KT * kRowsWarps;              // of a stage
    static constexpr int CTAS = 2;    // an SM
    static constexpr int STAGES = 3;  // 32 KB each; two stages and three CTAs, or smaller stages, are slower
    static constexpr uint32_t TILE = KEYS * kD * (WIDE ? 2 : 1);   // bytes of its keys, or values
};
// SHARES: see PAttnPlan::stream.
template <int FMT, int RT, bool SHARES>
struct RowsShared {
    using T = RowsShape<FMT, RT>;
    __align__(16) float ks[T::STAGES][T::WIDE ? 4 : T::KEYS];
    __align__(16) float vs[T::STAGES][T::WIDE ? 4 : T::KEYS];
    __align__(16) float o[SHARES ? 8 * RT : 1][kRowsPad];  // where the warps' results are joined
    uint64_t full[T::STAGES], empty[T::STAGES];
    float m[kRowsWarps][8 * RT], l[kRowsWarps][8 * RT];
    float2 ml[8 * RT];  // this split's maxima and sums, for the cluster
    int abort;
    int b0, share;              // the sequence that this CTA's share starts in,
    int64_t p0, g0, g1, total;  // the stages before it, the share itself, all stages (share: of how many)
};
template <int FMT, int RT, bool SHARES>
constexpr size_t rows_smem() {
    using T = RowsShape<FMT, RT>;
    constexpr size_t bytes = T::STAGES * 2 * T::TILE + sizeof(RowsShared<FMT, RT, SHARES>);
    static_assert(T::CTAS * (bytes + 1024) <= 228 * 1024, "CTAs of an SM");
    static_assert((kRowsWarps + 1) * 8 * RT * kRowsPad * 4 <= T::STAGES * 2 * T::TILE, "join");
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
// The 8 x 8 matrix of 16-bit values whose row g lane 4g .. 4g + 3 hold in pairs, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
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
// The warps that compute meet.
__device__ __forceinline__ void rows_meet() {
    __syncwarp();
    asm volatile("barrier.cta.sync.aligned 1, %0;" ::"n"(32 * kRowsWarps) : "memory");
}
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
}  // namespace

// A stretch of one key/value head's keys, in stages.
struct RowsItem {
    int b, h, first, n;
    SeqInfo sq;
    bool whole;  // all of the head's keys (of a share)
};
// Stages of a sequence's keys that its rows see, from s_lo on; at least one where there are rows.
template <int KEYS>
__device__ __forceinline__ int rows_stages(const PAttnPlan &p, const SeqInfo &sq, int &s_lo) {
    s_lo = 0;
    if (sq.qn == 0) return 0;
    const int lo = seen_lo(p, sq, 0), hi = seen_hi(p, sq, sq.qn - 1);
    if (lo >= hi) return 1;
    s_lo = lo / KEYS;
    return (hi + KEYS - 1) / KEYS - s_lo;
}

// QB: bf16 queries; FMT: the page format, the 16-bit ones (PF_F16 / PF_BF16) equal to the query's
// type.  SHARES: grid (shares), each an equal part of all heads' stages in a row; else grid
// (splits, key/value heads, sequences), joined: the splits are a cluster.
template <bool QB, int FMT, int RT, bool SHARES>
__global__ void __launch_bounds__(kRowsThreads, RowsShape<FMT, RT>::CTAS)
    k_page_attn_rows(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ PAttnPlan p, int joined) {
    pdl_begin();
    using T = RowsShape<FMT, RT>;
    constexpr bool WIDE = T::WIDE;
    constexpr bool PVB = WIDE && QB;            // type of all operands; 8-bit pages: fp16
    constexpr int ROWB = WIDE ? 2 * kD : kD;    // bytes of a cached row
    constexpr int NCH = ROWB / 64;              // 16-byte chunks of a row per lane
    constexpr int STAGES = T::STAGES, KT = T::KT, KEYS = T::KEYS, ROWS = 8 * RT;
    extern __shared__ __align__(1024) unsigned char sm[];
    RowsShared<FMT, RT, SHARES> &sh = *reinterpret_cast<RowsShared<FMT, RT, SHARES> *>(sm + STAGES * 2 * T::TILE);
    float(*s_o)[ROWS][kRowsPad] = reinterpret_cast<float(*)[ROWS][kRowsPad]>(sm);
    volatile int *abort_flag = &sh.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int shift = 31 - __clz(p.page);

    if (!SHARES && seq_info(p, blockIdx.z, false).qn == 0) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) seq_info(p, blockIdx.z, true);
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), kRowsWarps);
        }
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (SHARES && warp == 0) {
        // the stages of all heads, and where among them this CTA's share lies
        int s_lo;
        int64_t all = 0;
        for (int b = lane; b < p.B; b += 32) all += rows_stages<KEYS>(p, seq_info(p, b, blockIdx.x == 0), s_lo);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) all += __shfl_xor_sync(0xffffffffu, all, x);
        all *= p.H;
        const int64_t shares = max(min((int64_t)gridDim.x, all / kRowsShare), (int64_t)1), c = blockIdx.x;
        const int64_t g0 = c < shares ? c * all / shares : all, g1 = c < shares ? (c + 1) * all / shares : all;
        int64_t before = 0;
        int b0 = 0;
        for (int base = 0; g0 < g1 && base < p.B; base += 32) {
            const int b = base + lane;
            const int64_t own = b < p.B ? (int64_t)rows_stages<KEYS>(p, seq_info(p, b, false), s_lo) * p.H : 0;
            int64_t upto = own;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, upto, x);
                if (lane >= x) upto += y;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, before + upto > g0);
            if (past) {
                const int at = __ffs(past) - 1;
                b0 = base + at;
                before += __shfl_sync(0xffffffffu, upto - own, at);
                break;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (lane == 0) {
            sh.b0 = b0;
            sh.p0 = before;
            sh.g0 = g0;
            sh.g1 = g1;
            sh.share = (int)shares;
            sh.total = all;
        }
    }
    __syncthreads();

    // Calls work with each of this CTA's items (the same for all its warps) and the row of its
    // partial results.
    auto items = [&](auto &&work) {
        RowsItem x;
        int s_lo;
        if constexpr (!SHARES) {
            x.b = blockIdx.z;
            x.h = blockIdx.y;
            x.sq = seq_info(p, x.b, threadIdx.x == 0 && blockIdx.x == 0 && x.h == 0);
            const int all = rows_stages<KEYS>(p, x.sq, s_lo), per = (all + p.S - 1) / p.S;
            x.first = s_lo + blockIdx.x * per;
            x.n = max(0, min(per, all - (int)blockIdx.x * per));
            work(x, 0);  // (made again from the grid where it is needed, to keep registers free)
            return;
        }
        int64_t pos = sh.g0, before = sh.p0;
        const int64_t end = sh.g1;
        for (x.b = sh.b0; x.b < p.B && pos < end; x.b++) {
            x.sq = seq_info(p, x.b, false);
            const int all = rows_stages<KEYS>(p, x.sq, s_lo);
            for (x.h = all ? (int)((pos - before) / all) : p.H; x.h < p.H && pos < end; x.h++) {
                const int64_t start = before + (int64_t)x.h * all;
                x.first = s_lo + (int)(pos - start);
                x.n = (int)min(start + all - pos, end - pos);
                x.whole = x.n == all;
                // a part's place: the second of this CTA's two if the head begins with it
                const int slot = 2 * blockIdx.x + (pos == start);
                if (threadIdx.x == 0 && pos == start) {
                    // the share that the head's last stage lies in
                    const int last = x.whole ? (int)blockIdx.x : (int)(((start + all) * sh.share - 1) / sh.total);
                    p.spans[(int64_t)x.b * p.H + x.h] = make_int2(slot, last - (int)blockIdx.x);
                }
                pos += x.n;
                work(x, (int64_t)slot * kRowsM);
                __syncwarp();
            }
            before += (int64_t)all * p.H;
        }
    };

    if (warp == kRowsWarps) {
        // -------------------------------------------------------------------- TMA loads
        const int box = min(p.page, KEYS), boxes = KEYS / box;
        bool bad = false, ok = true;
        int issued = 0;
        items([&](const RowsItem &x, int64_t) {
            const int b = x.b, h = x.h, first = x.first, n = x.n;
            const int lo = seen_lo(p, x.sq, 0), hi = seen_hi(p, x.sq, x.sq.qn - 1);
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
            int next = n > 0 ? row_of(first * KEYS) : 0;
            for (int j = 0; ok && j < n; j++) {
                const int it = issued, k0 = (first + j) * KEYS, s = it % STAGES, row = next;
                if (j + 1 < n) next = row_of(k0 + KEYS);
                ok = page_wait(smem_u32(&sh.empty[s]), (it / STAGES + 1) & 1, abort_flag);
                ok = !__any_sync(0xffffffffu, !ok);
                if (!ok) break;
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
        });
        if (bad) or_status(p.status, QVG_DEV_BAD_INDEX);
        // every copy lands before the CTA ends
        for (int it = max(0, issued - STAGES); it < issued; it++)
            mbar_wait_final(smem_u32(&sh.full[it % STAGES]), (it / STAGES) & 1);
        if (joined) {
            cluster_meet();
            cluster_meet();
        }
    } else {
        // -------------------------------------------------------------------- attention
        int done = 0;  // stages of the items before
        bool ok = true;
        items([&](const RowsItem &item, int64_t part_row) {
            const int b = SHARES ? item.b : blockIdx.z, h = SHARES ? item.h : blockIdx.y, first = item.first, n = item.n;
            const SeqInfo sq = item.sq;
            const int rows = sq.qn * p.G, lo = seen_lo(p, sq, 0), hi = seen_hi(p, sq, sq.qn - 1);
            const int all_lo = seen_lo(p, sq, sq.qn - 1), all_hi = seen_hi(p, sq, 0);  // what every row sees
            float o[RT][8][4], m[RT][2], l[RT][2];
            // exponents of the references that the values' scales are taken against: a row's own, so
            // that no key which it does not see has a part in it
            int vexp[RT][2];
#pragma unroll
            for (int y = 0; y < RT; y++) {
                m[y][0] = m[y][1] = -INFINITY;
                l[y][0] = l[y][1] = 0.f;
                vexp[y][0] = vexp[y][1] = -100;
#pragma unroll
                for (int t = 0; t < 8; t++) o[y][t][0] = o[y][t][1] = o[y][t][2] = o[y][t][3] = 0.f;
            }
            // Q in the order the keys' chunks come in: lane (g, q) holds row g of each group
            uint32_t qb[RT][8][2];
            float qmul[RT][2];  // 8-bit pages: powers of two taken out of the rows whose scores this lane has
            int row_lo[RT][2], row_hi[RT][2];
#pragma unroll
            for (int y = 0; y < RT; y++) {
                const int r = 8 * y + g, i = token_of(p, min(r, rows - 1));
                const uint16_t *src = static_cast<const uint16_t *>(p.Q) + (sq.q0 + i) * p.qt +
                                      (int64_t)(h * p.G + r - i * p.G) * p.qh;
                uint4 w[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {  // 8 channels: two steps
                    const int ch = WIDE ? (j * 4 + q) * 8 : ((j >> 1) * 4 + q) * 16 + (j & 1) * 8;
                    w[j] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(src + ch)) : make_uint4(0u, 0u, 0u, 0u);
                }
                float mul = 1.f;
                if constexpr (!WIDE && QB) {
                    uint32_t big = 0;
#pragma unroll
                    for (int j = 0; j < 4; j++) big = max(big, bf16x2_max_bits(w[j]));
                    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    mul = bf16_pow2(big);
                    const float inv = 1.f / mul;
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        w[j] = make_uint4(bf16x2_to_f16x2(w[j].x, inv), bf16x2_to_f16x2(w[j].y, inv),
                                          bf16x2_to_f16x2(w[j].z, inv), bf16x2_to_f16x2(w[j].w, inv));
                }
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    qb[y][2 * j][0] = w[j].x;
                    qb[y][2 * j][1] = w[j].y;
                    qb[y][2 * j + 1][0] = w[j].z;
                    qb[y][2 * j + 1][1] = w[j].w;
                }
                // the scores' columns of this lane are rows 2q and 2q + 1
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    qmul[y][x] = __shfl_sync(0xffffffffu, mul, (2 * q + x) * 4) * p.scale_log2;
                    const int i = token_of(p, min(8 * y + 2 * q + x, rows - 1));
                    row_lo[y][x] = seen_lo(p, sq, i);
                    row_hi[y][x] = seen_hi(p, sq, i);
                }
            }

            // chunk c of row r of a swizzled tile (16 bits: two halves of 128-byte rows)
            auto chunk = [](const unsigned char *tile, int r, int c) {
                return *reinterpret_cast<const uint4 *>(tile + (c >> 3) * (T::TILE / 2) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            };
            // (a warp that gives up a wait keeps meeting the others)
            for (int j = 0; ok && j < n; j++) {
                const int it = done + j, st = it % STAGES;
                const int w0 = warp * 16 * KT, t0 = (first + j) * KEYS + w0;  // this warp's first key
                ok = page_wait(smem_u32(&sh.full[st]), (it / STAGES) & 1, abort_flag);
                ok = !__any_sync(0xffffffffu, !ok);
                if (!ok) break;
                if (t0 < hi && t0 + 16 * KT > lo) {
                    const unsigned char *kt = sm + st * 2 * T::TILE, *vt = kt + T::TILE;
                    // s[z][y][..]: keys t0 + 16 z + g (0, 1) and + 8 (2, 3), rows 8 y + 2 q, + 1
                    float s[KT][RT][4] = {};
#pragma unroll
                    for (int c = 0; c < NCH; c++) {
#pragma unroll
                        for (int z = 0; z < KT; z++) {
                            const uint4 ka = chunk(kt, w0 + z * 16 + g, c * 4 + q), kb = chunk(kt, w0 + z * 16 + g + 8, c * 4 + q);
                            if constexpr (WIDE) {
                                const uint32_t a0[4] = {ka.x, kb.x, ka.y, kb.y}, a1[4] = {ka.z, kb.z, ka.w, kb.w};
#pragma unroll
                                for (int y = 0; y < RT; y++) {
                                    mma16816<QB>(s[z][y], a0, qb[y][2 * c][0], qb[y][2 * c][1]);
                                    mma16816<QB>(s[z][y], a1, qb[y][2 * c + 1][0], qb[y][2 * c + 1][1]);
                                }
                            } else {
#pragma unroll
                                for (int w = 0; w < 4; w++) {
                                    const uint2 ua = codes_to_f16<FMT == PF_E4M3>(word_of(ka, w)),
                                                ub = codes_to_f16<FMT == PF_E4M3>(word_of(kb, w));
                                    const uint32_t a[4] = {ua.x, ub.x, ua.y, ub.y};
#pragma unroll
                                    for (int y = 0; y < RT; y++) mma16816<false>(s[z][y], a, qb[y][4 * c + w][0], qb[y][4 * c + w][1]);
                                }
                            }
                        }
                    }
                    const bool edge = t0 < lo || t0 + 16 * KT > hi;
                    float vsc[KT][2];
#pragma unroll
                    for (int z = 0; z < KT; z++) {
                        float k2[2] = {1.f, 1.f};
                        if constexpr (!WIDE) {
#pragma unroll
                            for (int e = 0; e < 2; e++) {
                                k2[e] = sh.ks[st][w0 + 16 * z + 8 * e + g];
                                vsc[z][e] = sh.vs[st][w0 + 16 * z + 8 * e + g];
                            }
                        }
#pragma unroll
                        for (int y = 0; y < RT; y++) {
                            s[z][y][0] *= qmul[y][0] * k2[0];
                            s[z][y][1] *= qmul[y][1] * k2[0];
                            s[z][y][2] *= qmul[y][0] * k2[1];
                            s[z][y][3] *= qmul[y][1] * k2[1];
                        }
                        if (edge || sq.qn > 1) {
#pragma unroll
                            for (int y = 0; y < RT; y++)
#pragma unroll
                                for (int e = 0; e < 4; e++) {
                                    const int key = t0 + 16 * z + 8 * (e >> 1) + g;
                                    if (key < row_lo[y][e & 1] || key >= row_hi[y][e & 1]) s[z][y][e] = -INFINITY;
                                }
                        }
                    }
                    // 8-bit: the weights take in the values' scales relative to 2^vexp, an exponent
                    // that follows the largest finite scale the row has seen; times 2^8 they fill
                    // fp16's range
                    float vcorr[RT][2], vmul[RT][2];
                    if constexpr (!WIDE) {
                        float big[RT][2] = {};
                        auto take = [&](float &to, float scale) { to = fmaxf(to, is_finite(scale) ? fabsf(scale) : 0.f); };
                        if (t0 >= all_lo && t0 + 16 * KT <= all_hi) {
#pragma unroll
                            for (int z = 0; z < KT; z++)
#pragma unroll
                                for (int e = 0; e < 2; e++) take(big[0][0], vsc[z][e]);
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) big[0][0] = fmaxf(big[0][0], __shfl_xor_sync(0xffffffffu, big[0][0], x));
#pragma unroll
                            for (int y = 0; y < RT; y++) big[y][0] = big[y][1] = big[0][0];
                        } else {
#pragma unroll
                            for (int y = 0; y < RT; y++)
#pragma unroll
                                for (int x = 0; x < 2; x++) {
#pragma unroll
                                    for (int z = 0; z < KT; z++)
#pragma unroll
                                        for (int e = 0; e < 2; e++)
                                            if (s[z][y][2 * e + x] != -INFINITY) take(big[y][x], vsc[z][e]);
#pragma unroll
                                    for (int d = 4; d < 32; d <<= 1) big[y][x] = fmaxf(big[y][x], __shfl_xor_sync(0xffffffffu, big[y][x], d));
                                }
                        }
#pragma unroll
                        for (int y = 0; y < RT; y++)
#pragma unroll
                            for (int x = 0; x < 2; x++) {
                                const int ve = max(vexp[y][x], min((int)(__float_as_uint(big[y][x]) >> 23) - 127, 121));
                                vcorr[y][x] = __uint_as_float((uint32_t)max(127 + vexp[y][x] - ve, 0) << 23);
                                vmul[y][x] = __uint_as_float((uint32_t)(127 + 8 - ve) << 23);
                                vexp[y][x] = ve;
                            }
                    }
                    uint32_t pb[KT][RT][2];
#pragma unroll
                    for (int y = 0; y < RT; y++) {
                        float corr[2], base[2], sum[2] = {0.f, 0.f};
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            float mx = m[y][x];
#pragma unroll
                            for (int z = 0; z < KT; z++) mx = fmax3(mx, s[z][y][x], s[z][y][2 + x]);
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                            base[x] = exp_base(mx);
                            corr[x] = fast_exp2(m[y][x] - base[x]);
                            m[y][x] = mx;
                        }
#pragma unroll
                        for (int z = 0; z < KT; z++)
#pragma unroll
                            for (int e = 0; e < 2; e++) {
                                float w0 = fast_exp2(s[z][y][2 * e] - base[0]), w1 = fast_exp2(s[z][y][2 * e + 1] - base[1]);
                                sum[0] += w0;
                                sum[1] += w1;
                                if constexpr (!WIDE) {
                                    w0 *= vsc[z][e] * vmul[y][0];
                                    w1 *= vsc[z][e] * vmul[y][1];
                                    if (edge || sq.qn > 1) {  // a hidden key's scale may be NaN: its weight stays 0
                                        if (s[z][y][2 * e] == -INFINITY) w0 = 0.f;
                                        if (s[z][y][2 * e + 1] == -INFINITY) w1 = 0.f;
                                    }
                                }
                                pb[z][y][e] = transpose8x8(PVB ? pack_bf16(w0, w1) : pack_f16(w0, w1));
                            }
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            l[y][x] = l[y][x] * corr[x] + sum[x];
                            if constexpr (!WIDE) corr[x] *= vcorr[y][x];
                        }
                        if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
                            for (int t = 0; t < 8; t++) {
                                o[y][t][0] *= corr[0];
                                o[y][t][1] *= corr[1];
                                o[y][t][2] *= corr[0];
                                o[y][t][3] *= corr[1];
                            }
                        }
                    }
#pragma unroll
                    for (int z = 0; z < KT; z++) {
                        uint4 vr[4][NCH / 2];  // keys 2q, 2q + 1, 2q + 8, 2q + 9
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const int at = 16 * z + 2 * q + (k & 1) + (k >> 1) * 8;
#pragma unroll
                            for (int c = 0; c < NCH / 2; c++) {
                                vr[k][c] = chunk(vt, w0 + at, c * 8 + g);
                                // values that no row sees may hold anything
                                if (edge && (t0 + at < lo || t0 + at >= hi)) vr[k][c] = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                        if constexpr (WIDE) {
#pragma unroll
                            for (int t = 0; t < 8; t++) {
                                const int w = t >> 1, sel = t & 1 ? 0x7632 : 0x5410;
                                const uint32_t a[4] = {__byte_perm(word_of(vr[0][0], w), word_of(vr[1][0], w), sel),
                                                       __byte_perm(word_of(vr[0][1], w), word_of(vr[1][1], w), sel),
                                                       __byte_perm(word_of(vr[2][0], w), word_of(vr[3][0], w), sel),
                                                       __byte_perm(word_of(vr[2][1], w), word_of(vr[3][1], w), sel)};
#pragma unroll
                                for (int y = 0; y < RT; y++) mma16816<PVB>(o[y][t], a, pb[z][y][0], pb[z][y][1]);
                            }
                        } else {
#pragma unroll
                            for (int w = 0; w < 2; w++) {
                                // the codes of two keys interleaved, then widened pair by pair:
                                // channels 4w .. 4w + 3 of the first and of the last eight
                                uint2 a[2][2][2];  // [first / last eight][keys 2q.. / 2q + 8..][channels 0, 1 / 2, 3]
#pragma unroll
                                for (int e = 0; e < 2; e++)
#pragma unroll
                                    for (int k = 0; k < 2; k++) {
                                        const uint32_t v0 = word_of(vr[2 * k][0], w + 2 * e), v1 = word_of(vr[2 * k + 1][0], w + 2 * e);
                                        a[e][k][0] = codes_to_f16<FMT == PF_E4M3>(__byte_perm(v0, v1, 0x5140));
                                        a[e][k][1] = codes_to_f16<FMT == PF_E4M3>(__byte_perm(v0, v1, 0x7362));
                                    }
#pragma unroll
                                for (int t = 0; t < 4; t++) {
                                    const int x = t >> 1;
                                    const uint32_t f[4] = {t & 1 ? a[0][0][x].y : a[0][0][x].x, t & 1 ? a[1][0][x].y : a[1][0][x].x,
                                                           t & 1 ? a[0][1][x].y : a[0][1][x].x, t & 1 ? a[1][1][x].y : a[1][1][x].x};
#pragma unroll
                                    for (int y = 0; y < RT; y++) mma16816<false>(o[y][4 * w + t], f, pb[z][y][0], pb[z][y][1]);
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.empty[st]));
            }
            if (SHARES) done += n;

            // join the warps relative to the largest of their maxima: through the ring, which is
            // through with its keys, or, where the next item's are on their way, one after another in
            // a place of its own
            if constexpr (!SHARES) rows_meet();
#pragma unroll
            for (int y = 0; y < RT; y++)
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    const int r = 8 * y + 2 * q + x;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[y][x] += __shfl_xor_sync(0xffffffffu, l[y][x], d);
                    if (g == 0) {
                        sh.m[warp][r] = m[y][x];
                        sh.l[warp][r] = l[y][x];
                    }
                }
            // this lane's channels (two runs of eight of each row), added to what is there or stored
            auto put = [&](float(*rows_o)[kRowsPad], bool add, bool relative) {
#pragma unroll
                for (int y = 0; y < RT; y++)
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        const int r = 8 * y + 2 * q + x;
                        const float unit = WIDE ? 1.f : __uint_as_float((uint32_t)(127 + vexp[y][x] - 8) << 23);
                        float f = 1.f;
                        if (relative) {
                            const float top = fmaxf(fmaxf(sh.m[0][r], sh.m[1][r]), fmaxf(sh.m[2][r], sh.m[3][r]));
                            f = fast_exp2(m[y][x] - exp_base(top));
                        }
#pragma unroll
                        for (int e = 0; e < 2; e++)
#pragma unroll
                            for (int k = 0; k < 8; k += 4) {
                                float4 *dst = reinterpret_cast<float4 *>(&rows_o[r][(WIDE ? 64 * e + 8 * g : 16 * g + 8 * e) + k]);
                                float4 v = make_float4(o[y][k][2 * e + x] * unit, o[y][k + 1][2 * e + x] * unit,
                                                       o[y][k + 2][2 * e + x] * unit, o[y][k + 3][2 * e + x] * unit);
                                if (relative) {
                                    const float4 a = add ? *dst : make_float4(0.f, 0.f, 0.f, 0.f);
                                    v = make_float4(a.x + f * v.x, a.y + f * v.y, a.z + f * v.z, a.w + f * v.w);
                                }
                                *dst = v;
                            }
                    }
            };
            if constexpr (SHARES) {
                rows_meet();
#pragma unroll 1
                for (int w = 0; w < kRowsWarps; w++) {
                    if (warp == w) put(sh.o, w > 0, true);
                    rows_meet();
                }
            } else {
                put(s_o[warp], false, false);
                rows_meet();
            }
            // eight lanes a row, 16 channels each (in runs of four, so that the lanes' reads and
            // writes are next to one another); the other warps only keep the barriers
            const int r = threadIdx.x >> 3, part = threadIdx.x & 7;
            float M = -INFINITY, L = 0.f, v[16] = {};
            const bool mine = r < ROWS;
            if (mine) {
#pragma unroll
                for (int w = 0; w < kRowsWarps; w++) M = fmaxf(M, sh.m[w][r]);
                const float base = exp_base(M);
#pragma unroll
                for (int w = 0; w < kRowsWarps; w++) {
                    const float f = fast_exp2(sh.m[w][r] - base);
                    L += f * sh.l[w][r];
#pragma unroll
                    for (int c = 0; c < 16; c++) {
                        const int at = (c >> 2) * 32 + part * 4 + (c & 3);
                        if constexpr (!SHARES)
                            v[c] += f * s_o[w][r][at];
                        else if (w == 0)
                            v[c] = sh.o[r][at];
                    }
                }
            }
            const int row_i = token_of(p, min(r, rows - 1)), hq = h * p.G + min(r, rows - 1) - row_i * p.G;
            bool live = mine && r < rows;
            if constexpr (SHARES) rows_meet();  // the join's rows are read: the next item's may follow
            if (SHARES ? !item.whole : p.S > 1 && !joined) {
                if (!live) return;
                const int64_t cell = (int64_t)blockIdx.z * p.H + blockIdx.y;
                const int64_t at = (SHARES ? part_row : (cell * p.S + blockIdx.x) * kRowsM) + r;
#pragma unroll
                for (int c = 0; c < 4; c++) store4<DT_F32>(p.part, at * kD + c * 32 + part * 4, v + 4 * c);
                if (part == 0) *reinterpret_cast<float2 *>(p.ml + 2 * at) = make_float2(M, L);
                return;
            }
            if (!SHARES && joined) {
                // each CTA of the cluster finishes the rows r with r % S its rank
                if (mine) {
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        *reinterpret_cast<float4 *>(&s_o[kRowsWarps][r][c * 32 + part * 4]) =
                            make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
                    if (part == 0) sh.ml[r] = make_float2(M, L);
                }
                cluster_meet();
                live = live && r % p.S == (int)blockIdx.x;
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
        if (rows_to_check(p)) {
            bool odd = false;
#pragma unroll
            for (int c = 0; c < 16; c++) odd |= !is_finite(v[c]);
            uint32_t todo = __ballot_sync(0xffffffffu, odd && live);
            while (todo) {
                const int src = (__ffs(todo) - 1) & ~7;  // the row's first lane
                todo &= ~(0xFFu << src);
                const int ri = __shfl_sync(0xffffffffu, row_i, src), rh = __shfl_sync(0xffffffffu, hq, src);
                float ro[4], rm, rl;
                if (!redo_if_shared(p, b, ri, rh, 0, sq.qn - 1, false, ro, rm, rl)) continue;
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
        });
        if (threadIdx.x == 0 && *abort_flag) or_status(p.status, QVG_DEV_TIMEOUT);
    }
}

// One warp per row of the items that were split: the splits' partial rows rescaled to the
// largest maximum and summed.  Lane l writes channels 4l .. 4l+3.
__global__ void __launch_bounds__(256) k_page_combine(PAttnPlan p) {
    pdl_begin();
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t t = w / p.unit, item = p.whole + t;
    if (item >= p.items) return;
    int cell = (int)(item / p.units), b = cell / p.H, h = cell - b * p.H, pair = p.units - 1 - (int)(item - (int64_t)cell * p.units);
    if (p.compact) {
        if (!compact_item(p, t, false, b, h, pair)) return;
        cell = b * p.H + h;
    }
    const int local = (int)(w - t * p.unit), r = pair * p.unit + local;
    const SeqInfo sq = seq_info(p, b, false);
    if (r >= sq.qn * p.G) return;
    const int i = token_of(p, r), hq = h * p.G + r - i * p.G;
    // the parts' rows: S of them, one unit after another, or (PAttnPlan::stream) the second
    // place of the share that the head begins in and the first places of those after it
    int S = p.S;
    int64_t at = t * p.S * p.unit + local, step = p.unit, skip = 0;
    if (p.stream) {
        const int2 span = p.spans[cell];
        S = span.y + 1;
        if (S == 1) return;  // whole, and written
        at = (int64_t)span.x * p.unit + local;
        step = 2 * p.unit;
        skip = -p.unit;
    }
    auto row = [&](int s) { return at + s * step + (int)(s > 0) * skip; };
    float mx = -INFINITY;
    for (int s = lane; s < S; s += 32) mx = fmaxf(mx, p.ml[2 * row(s)]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float base = exp_base(mx);
    float l = 0.f, o[4] = {};
    bool again = false;
    constexpr int SB = 8;
    for (int s0 = 0; s0 < S; s0 += SB) {
        float2 ml[SB];
        float4 po[SB];
#pragma unroll
        for (int k = 0; k < SB; k++)
            if (s0 + k < S) {
                const int64_t x = row(s0 + k);
                ml[k] = *reinterpret_cast<const float2 *>(p.ml + 2 * x);
                po[k] = *reinterpret_cast<const float4 *>(p.part + x * kD + 4 * lane);
            }
#pragma unroll
        for (int k = 0; k < SB; k++)
            if (s0 + k < S) {
                const float f = fast_exp2(ml[k].x - base);
                again |= ml[k].y == kRedo;
                l += f * ml[k].y;
                o[0] += f * po[k].x;
                o[1] += f * po[k].y;
                o[2] += f * po[k].z;
                o[3] += f * po[k].w;
            }
    }
    const bool odd = rows_to_check(p) &&
                     __any_sync(0xffffffffu, !is_finite(o[0]) || !is_finite(o[1]) || !is_finite(o[2]) || !is_finite(o[3]));
    if (again || odd) {  // (an item's rows end where the sequence's do)
        float y[4], ym, yl;
        if (redo_if_shared(p, b, i, hq, token_of(p, r - local), min(token_of(p, r - local + p.unit - 1), sq.qn - 1), again, y, ym, yl)) {
            o[0] = y[0]; o[1] = y[1]; o[2] = y[2]; o[3] = y[3];
            mx = ym;
            l = yl;
        }
    }
    const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
#pragma unroll
    for (int c = 0; c < 4; c++) o[c] *= inv;
    store_out4(p, (sq.q0 + i) * p.ot + hq * p.oh + 4 * lane, o);
    if (p.lse && lane == 0) p.lse[(sq.q0 + i) * p.HQ + hq] = row_lse(mx, l);
}

// How the work is cut.
//   Few rows: one item a key/value head and sequence.  As many splits as the SMs, two CTAs
//   each, hold at once: one round has the least latency (8 sequences of up to 2000 keys, 8
//   heads: 11.2 us with four splits, one round, 13.9 with eight).  Up to eight are joined by a
//   cluster; more than that, through memory, only if twice as many are wanted.  A split keeps
//   256 keys at least.  Where one round is fewer than four splits a head and 2048 keys or more
//   come to a CTA, sequences of different lengths have to even out:
//     8-bit pages: equal shares of all heads' keys, one round (8 heads, int8: 32 sequences of
//     9000 to 20000 155 us, four splits 167, one 197; 16 of 15000 each 86, four 92; 20 of 3000 to
//     30000 with four heads 60, six splits 79).  Up to two rounds of heads: more even out by
//     themselves, and each item costs a start and a join (300 sequences of up to 3000: 209 us
//     in shares, 160 without).
//     16 bits, where the memory's rate bounds and a start costs little beside it: a multiple of
//     one round's splits, four or more (bf16, the first of these: 267 us, in shares 281; seven
//     splits fill their rounds no better than four and keep slots of an SM waiting for whole
//     clusters).
//   Many rows: items of 256 rows, a CTA an SM.  Whole items fill whole rounds of the SMs, and
//   the last round's are split so that they fill it too: the split that takes the least time
//   is chosen, counting six key tiles' worth of time to start a CTA and four more to join.
//   (Splitting every item alike would write 57 MB of partial results for 4680 x 32760 x 12
//   heads, one and a half rounds, instead of 19.)  Sequences with different numbers of queries
//   leave items empty, and the last ones say nothing about the last round: there all items
//   are split alike, if they are too few for one round (only those that the sequences can have
//   get CTAs and room for partial results: 16 sequences that share 512 queries of 16 heads on 2
//   over up to 32768 keys ask for 60 MB, room for 512 of each for 477; with 2000 keys each, 65 ->
//   33 us); else, up to 16 sequences, the items of
//   those that see the most come first, so that the last round is one of short ones (four draws
//   of six prompts of 17 to 2000 queries over 500 to 9000 keys, 32 query heads on 8, bf16, causal,
//   on warm caches: 241 -> 211 us, 250 -> 220, 306 -> 281, 561 -> 521; the last but one in fp16
//   with a window of 4096, which makes the items more alike, 250 either way; thirty prompts even
//   out by themselves: 1999, 1640, 1735, 1570 us, in order 2000, 1640, 1725, 1575).
void page_attention_cut(PAttnPlan &p) {
    const int64_t rows = p.max_q * p.G, cells = (int64_t)p.H * p.B;
    p.whole = 0;
    p.items = cells;
    p.stream = p.by_length = p.compact = 0;
    if (rows <= kRowsM) {
        p.unit = kRowsM;
        p.units = 1;
        const int64_t most = std::max<int64_t>((p.max_kv + 255) / 256, 1), once = std::max<int64_t>(kRowsShares / cells, 1);
        int64_t want = std::min<int64_t>(once, 256);
        const bool wide = p.fmt == PF_F16 || p.fmt == PF_BF16;
        if (!wide && once < 4 && cells <= 2 * kRowsShares && cells * p.max_kv >= (int64_t)kRowsShares * 2048) {
            p.stream = 1;
            p.S = 1;
            return;
        }
        if (once < 2 * kRowsCluster) {
            while (want < 4 && (want + once) * cells <= 4 * kRowsShares && (want + once) * 2048 <= p.max_kv) want += once;
            want = std::min<int64_t>(want, kRowsCluster);
        }
        p.S = (int)std::min(want, most);
        return;
    }
    p.unit = 256;
    p.units = (int)((rows + 255) / 256);
    const int64_t items = p.units * cells, tiles = (p.max_kv + 127) / 128;
    const bool alike = p.total_q == p.max_q * p.B;
    const int64_t busy = alike ? items : std::min(items, p.total_q * p.G / 256 * p.H + cells);
    const int64_t rest = alike ? items % 152 : busy < 152 ? busy : 0, rounds = alike ? items / 152 : 0;
    p.whole = p.items = items;
    p.S = 1;
    double least = (double)((rounds + 1) * (tiles + 6));
    for (int s = 2; rest && s <= 64 && s <= tiles / 4; s++) {
        const double t = (double)(rounds * (tiles + 6)) +
                         (double)((rest * s + 151) / 152) * ((double)((tiles + s - 1) / s) + 6.0) + 4.0;
        if (t < least * 0.98) {
            least = t;
            p.S = s;
            p.whole = alike ? items - rest : 0;
        }
    }
    p.by_length = p.S == 1 && !alike && p.B <= 16;
    if (p.S > 1 && !alike && busy < items) {
        p.compact = 1;
        p.items = busy;
    }
}
int64_t page_attention_part_rows(const PAttnPlan &p) {
    if (p.stream) return 2 * (int64_t)kRowsShares * kRowsM;
    if (p.S == 1 || (p.unit == kRowsM && p.S <= kRowsCluster)) return 0;
    return (p.items - p.whole) * p.S * p.unit;
}

namespace {
template <bool QB, int FMT, int RT, bool SHARES>
cudaError_t launch_rows(const PAttnPlan &p, cudaStream_t st) {
    constexpr size_t smem = rows_smem<FMT, RT, SHARES>();
    const auto kernel = k_page_attn_rows<QB, FMT, RT, SHARES>;
    CUtensorMap mk, mv;
    const int box = std::min(p.page, RowsShape<FMT, RT>::KEYS);
    if (!page_map(p, p.k, box, &mk) || !page_map(p, p.v, box, &mv)) return cudaErrorInvalidValue;
    cudaError_t e = allow_smem<k_page_attn_rows<QB, FMT, RT, SHARES>>(smem);
    if (e != cudaSuccess) return e;
    const int joined = p.S > 1 && p.S <= kRowsCluster;
    const dim3 grid = SHARES ? dim3(kRowsShares) : dim3((unsigned)p.S, p.H, p.B);
    return launch_kernel_cluster(kernel, grid, dim3(kRowsThreads), smem, joined ? p.S : 1, st,
                                 mk, mv, p, joined);
}

template <bool QB, int FMT>
cudaError_t launch_rows(const PAttnPlan &p, cudaStream_t st) {
    const bool one = p.max_q * p.G <= 8;
    if constexpr (FMT == PF_E4M3 || FMT == PF_INT8)
        if (p.stream) return one ? launch_rows<QB, FMT, 1, true>(p, st) : launch_rows<QB, FMT, 2, true>(p, st);
    return one ? launch_rows<QB, FMT, 1, false>(p, st) : launch_rows<QB, FMT, 2, false>(p, st);
}

cudaError_t launch_page_attention_rows(const PAttnPlan &p, cudaStream_t st) {
    if (p.q_dtype == DT_BF16)
        return p.fmt == PF_E4M3   ? launch_rows<true, PF_E4M3>(p, st)
               : p.fmt == PF_INT8 ? launch_rows<true, PF_INT8>(p, st)
                                  : launch_rows<true, PF_BF16>(p, st);
    return p.fmt == PF_E4M3   ? launch_rows<false, PF_E4M3>(p, st)
           : p.fmt == PF_INT8 ? launch_rows<false, PF_INT8>(p, st)
                              : launch_rows<false, PF_F16>(p, st);
}
}  // namespace

cudaError_t launch_page_attention(const PAttnPlan &p, cudaStream_t st) {
    const cudaError_t e =
        p.max_q * p.G <= kRowsM ? launch_page_attention_rows(p, st) : launch_page_attention_tc(p, st);
    if (e != cudaSuccess || page_attention_part_rows(p) == 0) return e;
    const int64_t combined = p.stream ? (int64_t)p.B * p.H * kRowsM : page_attention_part_rows(p) / p.S;
    return launch_kernel(k_page_combine, dim3((unsigned)(combined / 8)), dim3(256), 0, st, p);
}

}  // namespace qvg
