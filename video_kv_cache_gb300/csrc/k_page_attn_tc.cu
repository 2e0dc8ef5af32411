// Attention of many query rows over paged keys and values, on the tensor cores (tcgen05 + TMEM
// + TMA).
//   O = softmax(scale Q K^T, over the visible keys) V
//
// Bound by the tensor cores: 4 * 128 operations per visible (query row, key) pair.  4680 queries
// of 12 heads over 32760 keys, every one seen: 601 us back to back on warm caches (1567 TFLOP/s),
// 643 us with cold ones; 4096 over 32768 of 32 heads, causal, warm: 1280 us (1610).  The tensor
// cores work 87 % of the cycles of the loop over the keys at the clocks that this load leaves
// (1.5 to 1.6 GHz);
// the rest is the start of a CTA (about 8000 cycles: TMEM, Q, the first tile) and the join of
// the last round's splits.  Shared memory is as busy as they are: a tile pair's products read
// 192 KB of it and the loads write 64, at 128 bytes a cycle the 2048 cycles of the products.
// A CTA takes two tiles of 128 rows (query tokens x grouped query heads of one key/value head)
// and walks the keys in tiles of 128; both row tiles use every key tile that is loaded.  One
// pass, with a running maximum and weight sum per row:
//   * one warp loads: a tile's pages by TMA into a ring of 32 KB slots (K and V alternate), in
//     the 128-byte swizzled layout that serves K as a K-major operand and V as an MN-major one;
//   * one warp issues S_t = Q_t K^T into TMEM, then O_t += P_t V with P_t read from TMEM;
//   * warps 0-7 and 8-15: the softmax of row tile 0 and 1, two threads a row with 64 scores
//     each (one would hold 128 in registers and spill, and its chain of latencies is what the
//     tensor cores wait for: 951 us with one, 734 with two): scores from TMEM, their maximum,
//     powers of two against the row's base, and the weights in 16 bits back into TMEM over the
//     scores.  While one tile's softmax runs, the tensor cores work on the other's.  A product
//     starts once the first 32 keys of either half have their weights.
// The running maximum is raised only when a row's scores pass it by more than 2^8: the weights
// stay below 2^8 and O_t in TMEM is rescaled (by the softmax warps themselves) a few times in
// all instead of once a tile, and only then the two threads of a row exchange their maxima; the
// result is the same, since numerator and weight sum share the base.
// Scores, weight sums and O are fp32; the weights are rounded to the values' 16-bit type (2^-8
// or 2^-11 of each at most), as the product's operands have to be.
// TMEM: S/P of the two row tiles (128 columns each; the weights take columns 0 - 31 and 64 - 95
// of their scores, so that each thread overwrites only scores that it has read), then O of the
// two (128 each): all 512 columns, one CTA an SM.
//
// 8-bit pages: eight more warps widen the codes to fp16 into the ring, from raw tiles of 64 keys
// that TMA brings (half a tile each: that leaves room for four slots of widened ones). bf16
// queries are made fp16 too, each row scaled by a power of two that brings its largest channel
// to 1 .. 2: what falls below fp16's range is 2^-25 of that. Where the output is bf16 and no
// log-sum-exp is asked for (FOLD), the keys' and values' scales are multiplied in while
// widening, relative to a power of two (of the tile's largest scale for keys; for values, whose
// sums outlive the tile, of the largest so far), and the product is rounded to fp16 once: 2^-11
// of each key and value, an eighth of what the output's own rounding is. Otherwise the scales
// multiply the scores and the weights in the softmax (the weights, in fp16, relative to the same
// power of two), which costs time: every thread then reads the scales of all keys from shared
// memory. The case above takes 908 us in e4m3 and 974 in int8 on warm caches, without folding 1097
// and 1152; 4096 over 32768 of 32 heads, causal, in e4m3 1913, with cold caches 1924.
// What costs is instructions: 10500 of a warp a tile pair against 5400 in 16 bits, which share
// the issue slots with the exponentials; with one factor instead of two (a scale rounded to
// fp16, an error that all channels of a key share) the first two took 20 and 34 us less.
//
// Masks: a tile that some row does not see whole is compared key by key; a weight that is
// hidden is 0.  Memory that no row sees (rows past the length) is not multiplied: the value
// product runs over the 16-key steps in sight, and the rest of the outer steps is zeroed.  What some
// rows of a tile see and others do not can still spoil those (page_attn.cuh says how); they are
// found at an item's end and computed once more, a key at a time.  For that the widening warps look,
// while the last tile is under way, at the scales of the keys that only some rows see.
#include "page_attn.cuh"

namespace qvg {

namespace {
constexpr int kTcM = 128;                  // rows of a row tile
constexpr int kTcN = 128;                  // keys of a key tile
constexpr uint32_t kHalf = kTcM * 128;     // 64 channels of 128 rows: 16 KB
constexpr uint32_t kSlot = 2 * kHalf;      // a whole 16-bit tile: 32 KB
constexpr int kRawKeys = 64;               // keys of a raw tile of 8-bit codes, half a key tile
constexpr uint32_t kRaw = kRawKeys * kD;   // 8 KB
constexpr int kValueShift = 4, kKeyShift = 6;  // 8-bit values and keys over their references, times 2^this
// How far (log2) a scale that a row does not see may lie above the largest that it sees before the
// row is done again.  Values: a weight times a scale over the reference 2^e is rounded by at most
// 2^-25 times 2^(e - kValueShift) and a code, 2^-25 of the largest value that the row sees if 2^e is
// at most kValueShift above it.  Folded values are rounded alone, by 2^-25 times 2^(e - kValueShift):
// the same of a largest value of 127 codes at least if 2^e is 2^7 further up.  Keys: channels by
// 2^-25 times 2^(e - kKeyShift), which is 2^-30 of the row's largest key, 127 codes of its scale at
// least, if 2^e is at most kKeyShift + 2 above.
constexpr int kValueFar = kValueShift, kFoldedFar = kValueShift + 7, kKeyFar = kKeyShift + 2;
constexpr float kLazy = 8.f;               // how far (log2) scores may pass the running maximum
// The largest score less its base, from the unrounded product, is what the base was rounded by: at
// most 1/2 up to here, and weights stay below fp16's largest.  Past it the row is done again.
constexpr float kHugeScore = 8388608.f;

template <int FMT>
struct TcShape {
    static constexpr bool WIDE = FMT == PF_F16 || FMT == PF_BF16;
    static constexpr int SLOTS = WIDE ? 5 : 4;       // ring of 16-bit tiles
    static constexpr int RAWS = 3;                   // ring of raw 8-bit tiles
    // 16 softmax warps; MMA, loads and two idle ones (registers move by groups of four warps);
    // 8-bit: four that widen keys and four that widen values (four for both keep the tensor
    // cores waiting)
    static constexpr int THREADS = WIDE ? 640 : 896;
    // registers at launch (65,536 over the warps of an SM quarter), and after they were shared
    // out anew: the groups' sum stays what the launch had
    static constexpr int REGS = WIDE ? 96 : 72, REGS_SOFTMAX = WIDE ? 104 : 80, REGS_REST = WIDE ? 64 : 56;
    static_assert(512 * REGS_SOFTMAX + (THREADS - 512) * REGS_REST <= THREADS * REGS, "register shares");
    static constexpr uint32_t SMEM_TILES = 2 * kSlot + SLOTS * kSlot + (WIDE ? 0 : RAWS * kRaw);
};

// Everything the roles share besides the tiles (the 16-bit formats have no scales).
template <int FMT>
struct TcShared {
    static constexpr bool WIDE = TcShape<FMT>::WIDE;
    uint64_t full[5], empty[5];         // ring of 16-bit tiles
    // raw tiles: keys and values share the places, but each has a barrier of its own for them.  A
    // phase is told by its parity, so whoever waits on a barrier has to wait for every phase of it.
    uint64_t raw_full[2][3], raw_empty[3];
    uint64_t s_full[2], p_full[2][2], o_done[2];
    uint64_t sc_full[2], sc_empty[2];   // scales of a key tile
    uint64_t q_full, edge, fin;
    uint32_t tmem;
    int abort;
    int vexp[2], kexp[2];               // exponents of the values' and keys' references, per tile parity
    __align__(16) uint32_t vnan[2][4];                // keys whose value scale is not finite, a bit each
    float wmax[2][4];                   // largest scales of the widening warps: keys', values'
    uint64_t sizes;
    uint32_t some[2], all[2];           // bits of the largest scale of keys, values that some rows see only, and of others
    float xmax[2][2][kTcM];             // the two threads of a row: their maxima; at the end their weight sums
    uint32_t odd[2][4][2];              // rows to be done again, a bit each: row tile, quarter, half
    uint32_t bad[2][4];                 // rows that see a value whose scale is not finite: their output is NaN, their weight sum is not
    __align__(16) float ks[2][WIDE ? 4 : kTcN];  // keys' scales times the softmax scale
    __align__(16) float vs[2][WIDE ? 4 : kTcN];  // values' scales over their reference
    uint2 kf[2][WIDE ? 1 : kTcN], vf[2][WIDE ? 1 : kTcN];  // scales over their references, see scale_pair
    float qmul[WIDE ? 4 : 2 * kTcM];             // powers of two taken out of the rows of Q
};

template <int FMT>
constexpr size_t tc_smem() {
    constexpr size_t bytes = TcShape<FMT>::SMEM_TILES + sizeof(TcShared<FMT>);
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    return bytes;
}

// One arrival where it holds; the lanes stay together, as the tensor-memory instructions around
// it need them.
__device__ __forceinline__ void mbar_arrive_if(uint32_t bar, bool holds) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}\n" ::"r"(bar),
        "r"((uint32_t)holds)
        : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r));
    return r != 0u;
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
}
// 16 consecutive columns of this thread's TMEM lane written / read.
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t r[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t r[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// The read of 32 columns in two steps: what it gives may be used after the second.
__device__ __forceinline__ void tc_ld32_start(uint32_t taddr, float v[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_ld32_wait(float v[32]) {
    asm volatile(
        "tcgen05.wait::ld.sync.aligned;"
        : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
          "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
          "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
          "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
        :
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptor of an MN-major operand (values: 64 channels of a key are one 128-byte row) in the
// 128-byte swizzled layout: 64-channel blocks kHalf apart, groups of 8 keys 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kHalf >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// fp32 accumulator, A and B bf16 or fp16, M = N = 128; B MN-major for the value product.
__device__ __forceinline__ uint32_t attn_idesc(bool bf16, bool b_mn) {
    const uint32_t f = bf16 ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(kTcN >> 3) << 17) |
           ((uint32_t)(kTcM >> 4) << 24);
}
// Meets the other threads of a named barrier; whether every one of them says so (the same
// answer for all).  Roles that meet at barriers decide together this way whether to go on.
template <int THREADS>
__device__ __forceinline__ bool meet(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.aligned.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "n"(THREADS)
        : "memory");
    return r != 0u;
}
// A scale as two fp16 numbers, high and low part, each twice; and fp16 pairs times it, rounded
// once (the low product's own rounding is 2^-22 of the result).
__device__ __forceinline__ uint2 scale_pair(float f) {
    const __half hi = __float2half_rn(f), lo = __float2half_rn(f - __half2float(hi));
    const __half2 h2 = __half2half2(hi), l2 = __half2half2(lo);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&h2), *reinterpret_cast<const uint32_t *>(&l2));
}
__device__ __forceinline__ uint32_t scaled(uint32_t y, const uint2 &f) {
    const __half2 v = *reinterpret_cast<const __half2 *>(&y), hi = *reinterpret_cast<const __half2 *>(&f.x),
                  lo = *reinterpret_cast<const __half2 *>(&f.y);
    const __half2 r = __hfma2(v, hi, __hmul2_rn(v, lo));
    return *reinterpret_cast<const uint32_t *>(&r);
}
template <int REGS>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
// 64 columns of this thread's TMEM lane multiplied by f.
__device__ __forceinline__ void rescale64(uint32_t at, float f) {
#pragma unroll
    for (int c = 0; c < 64; c += 16) {
        uint32_t w[16];
        tc_ld16(at + c, w);
#pragma unroll
        for (int k = 0; k < 16; k++) w[k] = __float_as_uint(__uint_as_float(w[k]) * f);
        tc_st16(at + c, w);
    }
    tc_wait_st();
}
}  // namespace

// grid (items taken whole + splits of the others), see page_attention_cut
// FOLD (8-bit): the scales are multiplied into keys and values, not scores and weights.
template <bool QB, int FMT, bool FOLD>
__global__ void __launch_bounds__(TcShape<FMT>::THREADS, 1)
    k_page_attn_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ PAttnPlan p) {
    pdl_begin();
    using T = TcShape<FMT>;
    constexpr bool WIDE = T::WIDE;
    constexpr bool BF = WIDE && QB;  // type of all operands; 8-bit pages: fp16
    constexpr int SLOTS = T::SLOTS;
    constexpr int MMA_WARP = 16, LOAD_WARP = 17, WIDEN_WARP = 20;
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char *sQ = sm, *sKV = sm + 2 * kSlot, *sRaw = sKV + SLOTS * kSlot;
    TcShared<FMT> &sh = *reinterpret_cast<TcShared<FMT> *>(sm + T::SMEM_TILES);
    volatile int *abort_flag = &sh.abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this CTA's item and split of it: one head's items after one another, so that those that
    // run together find its keys and values in L2 (152 CTAs that each read their own would take
    // the whole bandwidth of the memory), the longest first (under a causal mask the last rows
    // see the most)
    const bool whole_item = blockIdx.x < p.whole;
    const int64_t tail = whole_item ? 0 : (blockIdx.x - p.whole) / p.S;
    const int split = whole_item ? 0 : (int)((blockIdx.x - p.whole) - tail * p.S), S = whole_item ? 1 : p.S;
    const int64_t item = whole_item ? blockIdx.x : p.whole + tail;
    const int cell = (int)(item / p.units);
    int b = cell / p.H, h = cell - b * p.H, pair = p.units - 1 - (int)(item - (int64_t)cell * p.units);
    if (p.by_length) {
        // the sequences, a lane each, those whose last rows see the most first, and only the
        // items that they have
        SeqInfo s = {0, 0, 0};
        if (lane < p.B) s = seq_info(p, lane, blockIdx.x == 0 && warp == 0);
        const int units = (s.qn * p.G + 2 * kTcM - 1) / (2 * kTcM);
        const int seen = units ? seen_hi(p, s, s.qn - 1) - seen_lo(p, s, token_of(p, (units - 1) * 2 * kTcM)) : 0;
        int ahead = 0;
        for (int x = 0; x < p.B; x++) {
            const int their = __shfl_sync(0xffffffffu, seen, x), n = __shfl_sync(0xffffffffu, units, x);
            if (their > seen || (their == seen && x < lane)) ahead += n;
        }
        const int64_t in = blockIdx.x - (int64_t)ahead * p.H;
        const bool mine = in >= 0 && in < (int64_t)units * p.H;
        const uint32_t owner = __ballot_sync(0xffffffffu, mine);
        if (!owner) return;
        // (reductions leave their results in uniform registers, of which there are enough)
        const int n = (int)__reduce_max_sync(0xffffffffu, mine ? units : 0), at = (int)__reduce_max_sync(0xffffffffu, mine ? (int)in : 0);
        b = __ffs(owner) - 1;
        h = at / n;
        pair = n - 1 - (at - h * n);
    }
    if (p.compact && !compact_item(p, tail, blockIdx.x == 0 && warp == 0, b, h, pair)) return;
    const SeqInfo sq = seq_info(p, b, !p.by_length && !p.compact && threadIdx.x == 0 && pair == 0 && split == 0 && h == 0);
    const int rows = sq.qn * p.G, r0 = pair * 2 * kTcM;
    if (r0 >= rows) return;
    const int nt = rows - r0 > kTcM ? 2 : 1;  // row tiles in use
    const int lo = seen_lo(p, sq, token_of(p, r0)), hi = seen_hi(p, sq, token_of(p, min(rows, r0 + 2 * kTcM) - 1));
    int n = 0, j0 = 0;  // this split's key tiles
    if (lo < hi) {
        const int t_lo = lo / kTcN, all = (hi + kTcN - 1) / kTcN - t_lo, per = (all + S - 1) / S;
        j0 = t_lo + split * per;
        n = max(0, min(per, all - split * per));
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < SLOTS; s++) {
            mbar_init(smem_u32(&sh.full[s]), WIDE ? 1 : 4);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        for (int s = 0; s < T::RAWS; s++) {
            mbar_init(smem_u32(&sh.raw_full[0][s]), 1);
            mbar_init(smem_u32(&sh.raw_full[1][s]), 1);
            mbar_init(smem_u32(&sh.raw_empty[s]), 4);
        }
        for (int t = 0; t < 2; t++) {
            mbar_init(smem_u32(&sh.s_full[t]), 1);
            mbar_init(smem_u32(&sh.p_full[t][0]), 8);
            mbar_init(smem_u32(&sh.p_full[t][1]), 8);
            mbar_init(smem_u32(&sh.o_done[t]), 1);
            mbar_init(smem_u32(&sh.sc_full[t]), 8);
            mbar_init(smem_u32(&sh.sc_empty[t]), 8 * nt);
            for (int x = 0; x < 4; x++) sh.bad[t][x] = 0u;
        }
        mbar_init(smem_u32(&sh.q_full), 16);
        mbar_init(smem_u32(&sh.edge), 1);
        mbar_init(smem_u32(&sh.fin), 1);
        mbar_init(smem_u32(&sh.sizes), 8);
        sh.some[0] = sh.some[1] = sh.all[0] = sh.all[1] = 0u;
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    auto wait = [&](uint64_t &bar, uint32_t parity) { return page_wait(smem_u32(&bar), parity & 1u, abort_flag); };

    if (warp >= MMA_WARP) {
        regs_dec<T::REGS_REST>();
        if (warp == MMA_WARP) {
            // ---------------------------------------------------------------- MMA issuer
            // What this thread does between two batches of MMAs is time that the tensor cores
            // stand still, so a batch is as long as it can be (O_t += P_t V, then the next
            // tile's S_t) and follows one wait, that for P_t; the ring was waited for before.
            if (n > 0 && elect_one()) {
                const uint32_t id_qk = attn_idesc(BF, false), id_pv = attn_idesc(BF, true);
                const uint64_t q_desc = sw128_desc(smem_u32(sQ)), k_desc = sw128_desc(smem_u32(sKV)),
                               v_desc = sw128_mn_desc(smem_u32(sKV));
                auto scores = [&](int t, int slot) {
                    const uint64_t a = q_desc + (uint64_t)(t * (kSlot >> 4)), k = k_desc + (uint64_t)(slot * (kSlot >> 4));
#pragma unroll
                    for (int kk = 0; kk < 8; kk++) {
                        const uint64_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                        tc_mma(tmem + t * 128, a + off, k + off, id_qk, kk > 0);
                    }
                    tc_commit(smem_u32(&sh.s_full[t]));
                };
                bool ok = wait(sh.full[0], 0) && wait(sh.q_full, 0);
                if (ok) {
                    tc_fence_after();
                    for (int t = 0; t < nt; t++) scores(t, 0);
                    tc_commit(smem_u32(&sh.empty[0]));
                }
                for (int j = 0; ok && j < n; j++) {
                    const uint32_t iv = 2 * j + 1, ik = iv + 1;  // ring items: V of this tile, K of the next
                    const int sv = iv % SLOTS, sk = ik % SLOTS;
                    // the 16-key steps of the tile that some row sees
                    const int k0 = (j0 + j) * kTcN;
                    const int st0 = max(lo - k0, 0) >> 4, st1 = (min(hi - k0, kTcN) + 15) >> 4;
                    const uint64_t v = v_desc + (uint64_t)(sv * (kSlot >> 4));
                    const bool more = j + 1 < n;
                    ok = wait(sh.full[sv], iv / SLOTS) && (!more || wait(sh.full[sk], ik / SLOTS));
                    for (int t = 0; ok && t < nt; t++) {
                        ok = wait(sh.p_full[t][0], j);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t o = tmem + 256 + t * 128, w = tmem + t * 128;
                        auto product = [&](int s, bool accumulate) {
                            // (the two halves of the weights lie where their scores were)
                            tc_mma_ts(o, w + s * 8 + (s >= 4 ? 32 : 0), v + (uint64_t)((s * 2048) >> 4), id_pv, accumulate);
                        };
                        // the steps of the first 32 keys of either half, then the others
                        const bool whole = st0 == 0 && st1 == 8;
                        if (whole) {
                            product(0, j > 0);
                            product(1, true);
                            product(4, true);
                            product(5, true);
                        }
                        ok = wait(sh.p_full[t][1], j);
                        if (!ok) break;
                        tc_fence_after();
                        if (whole) {
                            product(2, true);
                            product(3, true);
                            product(6, true);
                            product(7, true);
                        } else {
                            for (int s = st0; s < st1; s++) product(s, j > 0 || s > st0);
                        }
                        tc_commit(smem_u32(&sh.o_done[t]));
                        if (t == nt - 1) tc_commit(smem_u32(&sh.empty[sv]));
                        if (more) {
                            scores(t, sk);
                            if (t == nt - 1) tc_commit(smem_u32(&sh.empty[sk]));
                        }
                    }
                }
                // every MMA issued so far completes before TMEM is released
                tc_commit(smem_u32(&sh.fin));
                mbar_wait_final(smem_u32(&sh.fin), 0);
            }
        } else if (warp == LOAD_WARP) {
            // ---------------------------------------------------------------- TMA loads
            const int page_shift = 31 - __clz(p.page);
            // what one copy brings: a page, or half of one of 128 tokens where the ring's tiles
            // have 64
            const int shift = WIDE ? page_shift : min(page_shift, 6), per_tile = kTcN >> shift;
            bool bad = false, ok = true;
            uint32_t edges = 0, issued = 0, used = 0, odd = 0;  // raw tiles: barriers in use, and those used an odd number of times
            constexpr int RING = WIDE ? SLOTS : T::RAWS;
            constexpr uint32_t PER_KEYS = WIDE ? 2 : 4;  // ring items of a key tile: K and V, or their halves
            // the pages of a tile that hold a key some row sees, a lane each; looked up one
            // tile ahead
            auto in_sight = [&](int k0) {
                const int token = k0 + (lane << shift);
                return lane < per_tile && token < hi && token + (1 << shift) > lo;
            };
            auto row_of = [&](int k0) {
                const int token = k0 + (lane << shift);
                return in_sight(k0) ? (int)((page_of(p, b, token, page_shift, bad) * p.H + h) << page_shift) +
                                          (token & (p.page - 1))
                                    : 0;
            };
            int row = 0, row_next = n > 0 ? row_of(j0 * kTcN) : 0;
            for (uint32_t it = 0; ok && it < PER_KEYS * n; it++) {
                const int k0 = (j0 + (int)(it / PER_KEYS)) * kTcN, slot = it % RING;
                const bool value = WIDE ? it & 1 : it & 2;
                if (it % PER_KEYS == 0) {
                    row = row_next;
                    if (it + PER_KEYS < PER_KEYS * n) row_next = row_of(k0 + kTcN);
                }
                uint64_t &full = WIDE ? sh.full[slot] : sh.raw_full[value][slot];
                ok = wait(WIDE ? sh.empty[slot] : sh.raw_empty[slot], it / RING + 1);
                ok = !__any_sync(0xffffffffu, !ok);
                if (!ok) break;
                const bool mine = in_sight(k0) && (WIDE || (uint32_t)(lane << shift) / kRawKeys == (it & 1));
                const uint32_t pages = __popc(__ballot_sync(0xffffffffu, mine));
                // a value tile at the edge of what is seen, whose outer rows must be zeroed
                const bool edge = WIDE && value && (((lo - k0) & 15 && lo > k0) || ((hi - k0) & 15 && hi < k0 + kTcN));
                const uint32_t bar = smem_u32(edge ? &sh.edge : &full);
                if (lane == 0) mbar_expect_tx(bar, (pages << shift) * (WIDE ? 2u * kD : (uint32_t)kD));
                __syncwarp();
                if (mine) {
                    const CUtensorMap *map = value ? &tmV : &tmK;
                    if constexpr (WIDE) {
                        const uint32_t dst = smem_u32(sKV) + slot * kSlot + ((uint32_t)lane << shift) * 128;
                        tma_load_2d(dst, map, 0, row, bar);
                        tma_load_2d(dst + kHalf, map, 64, row, bar);
                    } else {
                        tma_load_2d(smem_u32(sRaw) + slot * kRaw + (((uint32_t)lane << shift) & (kRawKeys - 1)) * kD, map, 0, row, bar);
                    }
                }
                issued = it + 1;
                used |= 1u << (3 * value + slot % 3);
                odd ^= 1u << (3 * value + slot % 3);
                if (edge) {
                    // rows of the outer 16-key steps that no row of the CTA sees: zeros
                    mbar_wait_final(bar, edges++ & 1u);
                    const int v0 = max(lo - k0, 0), v1 = min(hi - k0, kTcN);
                    for (int x = lane; x < 2 * 16 * 16; x += 32) {
                        const int side = x >> 8, r = side ? (v1 & ~15) + ((x >> 4) & 15) : (v0 & ~15) + ((x >> 4) & 15);
                        const int c = x & 15;
                        if (side ? (r >= v1 && (v1 & 15)) : r < v0)
                            *reinterpret_cast<uint4 *>(sKV + slot * kSlot + (c >> 3) * kHalf + r * 128 + (c & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&full));
                }
            }
            if (bad) or_status(p.status, QVG_DEV_BAD_INDEX);
            // every copy this CTA started lands before the CTA ends (edge tiles were waited for;
            // their slots' phases were completed by hand)
            if constexpr (WIDE) {
                const uint32_t from = issued > (uint32_t)RING ? issued - RING : 0u;
                for (uint32_t it = from; it < issued; it++) mbar_wait_final(smem_u32(&sh.full[it % RING]), (it / RING) & 1u);
            } else {
                for (int k = 0; k < 6; k++)
                    if (used >> k & 1u) mbar_wait_final(smem_u32(&sh.raw_full[k / 3][k % 3]), ~(odd >> k) & 1u);
            }
        } else if (!WIDE && warp >= WIDEN_WARP) {
            // ---------------------------------------------------------------- 8-bit codes widened
            const bool value = warp >= WIDEN_WARP + 4;  // the first four warps: keys, the others: values
            const int shift = 31 - __clz(p.page), x = (threadIdx.x - 32 * WIDEN_WARP) & 127, id = 1 + value;
            const float *scales = value ? p.vs : p.ks;
            float *wmax = sh.wmax[value];
            int e = -126;
            bool ok = true, bad = false;
            // scales of a tile's keys, one a thread, read one tile ahead; outside what is seen
            // they are 0
            float sc = 0.f;
            auto load_scale = [&](int key) {
                sc = 0.f;
                if (key >= lo && key < hi)
                    sc = __ldg(scales + ((page_of(p, b, key, shift, bad) * p.H + h) << shift) + (key & (p.page - 1)));
            };
            if (n > 0) load_scale(j0 * kTcN + x);
            // 16 codes (chunk c of a row) a thread, rows 16 apart: eight lanes that are served
            // together have eight rows of one chunk, which the swizzle of the raw tile and that
            // of the widened one both spread over all banks
            const int c = (x >> 3) & 7, r8 = x & 7, rb = r8 + ((x >> 6) << 3);
            const unsigned char *src0 = sRaw + rb * kD + ((c ^ r8) << 4);
            unsigned char *dst0 = sKV + (c >> 2) * kHalf + rb * 128;
            const int d0 = ((2 * (c & 3)) ^ r8) << 4, d1 = ((2 * (c & 3) + 1) ^ r8) << 4;
            uint32_t phases = 0;  // of this operand's barriers of the raw tiles, a bit each
            for (int j = 0; j < n; j++) {
                const int it = 2 * j + value, k0 = (j0 + j) * kTcN, slot = it % SLOTS, buf = j & 1;
                // a value scale that is not finite: 0 here, and a bit that makes the outputs of the
                // rows NaN that see the key (and no others)
                const uint32_t odd = __ballot_sync(0xffffffffu, !is_finite(sc));
                float m = is_finite(sc) ? fabsf(sc) : 0.f;
                if (value) sc = is_finite(sc) ? sc : 0.f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                ok = ok && wait(sh.sc_empty[buf], (j >> 1) + 1);
                if (lane == 0) wmax[warp & 3] = m;
                __syncwarp();  // (lanes may come from a wait one by one; a barrier wants the whole warp)
                ok = meet<128>(id, ok);
                if (!ok) break;  // the four warps leave together
                m = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
                const int ee = min(max((int)(__float_as_uint(m) >> 23) - 127, -100), 121);
                if (value) {
                    // the reference moves only when a scale passes it by 2^3: codes of at most
                    // 448 times 2^3 * 2^kValueShift stay below fp16's largest, 65504, and so do
                    // weights of at most 2^kLazy
                    if (j == 0 || ee > e + 2) e = ee;
                    const float f = sc * __uint_as_float((uint32_t)(127 + kValueShift - e) << 23);
                    if constexpr (FOLD)
                        sh.vf[buf][x] = scale_pair(f);
                    else
                        sh.vs[buf][x] = f;
                    if (lane == 0) sh.vnan[buf][warp & 3] = odd;
                    if (x == 0) sh.vexp[buf] = e;
                } else if (FOLD) {
                    sh.kf[buf][x] = scale_pair(sc * __uint_as_float((uint32_t)(127 + kKeyShift - ee) << 23));
                    if (x == 0) sh.kexp[buf] = ee;
                } else {
                    sh.ks[buf][x] = sc * fabsf(p.scale_log2);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.sc_full[buf]));
                if (j + 1 < n) load_scale(k0 + kTcN + x);
                int raw = 2 * it % T::RAWS;
                ok = wait(sh.raw_full[value][raw], phases >> raw) && wait(sh.empty[slot], it / SLOTS + 1);
                __syncwarp();
                ok = meet<128>(id, ok);
                if (!ok) break;  // (otherwise all scales are there, and wmax is free again)
                const bool whole = k0 >= lo && k0 + kTcN <= hi;
                const uint2 *factors = (value ? sh.vf[buf] : sh.kf[buf]) + rb;
                unsigned char *dst = dst0 + slot * kSlot;
#pragma unroll
                for (int part = 0; part < 2; part++) {
                    if (part) {
                        raw = raw == T::RAWS - 1 ? 0 : raw + 1;
                        ok = wait(sh.raw_full[value][raw], phases >> raw);  // (who gives up here meets the others at the next tile)
                    }
                    phases ^= 1u << raw;
                    const unsigned char *src = src0 + raw * kRaw;
#pragma unroll
                    for (int v = 0; v < 4; v++) {
                        const int u = 4 * part + v;
                        uint4 w = *reinterpret_cast<const uint4 *>(src + v * 16 * kD);
                        if (!whole) {  // what no row sees may hold anything
                            const int key = k0 + rb + u * 16;
                            if (key < lo || key >= hi) w = make_uint4(0u, 0u, 0u, 0u);
                        }
                        const uint2 y0 = codes_to_f16<FMT == PF_E4M3>(w.x), y1 = codes_to_f16<FMT == PF_E4M3>(w.y),
                                    y2 = codes_to_f16<FMT == PF_E4M3>(w.z), y3 = codes_to_f16<FMT == PF_E4M3>(w.w);
                        uint4 a0 = make_uint4(y0.x, y0.y, y1.x, y1.y), a1 = make_uint4(y2.x, y2.y, y3.x, y3.y);
                        if constexpr (FOLD) {
                            const uint2 f = factors[u * 16];
                            a0 = make_uint4(scaled(a0.x, f), scaled(a0.y, f), scaled(a0.z, f), scaled(a0.w, f));
                            a1 = make_uint4(scaled(a1.x, f), scaled(a1.y, f), scaled(a1.z, f), scaled(a1.w, f));
                        }
                        *reinterpret_cast<uint4 *>(dst + u * 2048 + d0) = a0;
                        *reinterpret_cast<uint4 *>(dst + u * 2048 + d1) = a1;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.raw_empty[raw]));
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.full[slot]));
            }
            if (bad) or_status(p.status, QVG_DEV_BAD_INDEX);
            // The references are of what any row sees.  Should one lie too far above what a row sees
            // itself, the row is done again; for that, how large the scales are that only some rows
            // see (the softmax is still busy with the last tile), and 256 that all of them see.
            if (n > 0 && redo_possible(p)) {
                const KeySpans sp = key_spans(p, sq, r0, min(rows, r0 + 2 * kTcM), max(lo, j0 * kTcN), min(hi, (j0 + n) * kTcN));
                auto largest_of = [&](int from, int to, uint32_t *most) {
                    float m = 0.f;
#pragma unroll 1
                    for (int key = from + x; key < to; key += 128) {
                        const float s = __ldg(scales + ((page_of(p, b, key, shift, bad) * p.H + h) << shift) + (key & (p.page - 1)));
                        m = fmaxf(m, is_finite(s) ? fabsf(s) : 0.f);
                    }
                    __syncwarp();
                    const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
                    if (lane == 0 && w) atomicMax(most, w);
                };
                if ((value || FOLD) && (sp.a0 < sp.a1 || sp.z0 < sp.z1)) {
                    largest_of(sp.a0, sp.a1, &sh.some[value]);
                    largest_of(sp.z0, sp.z1, &sh.some[value]);
                    largest_of(max(sp.a1, sp.z0 - 256), sp.z0, &sh.all[value]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.sizes));
            }
        }
    } else {
        // -------------------------------------------------------------------- softmax
        regs_inc<T::REGS_SOFTMAX>();
        // Q: both row tiles, swizzled; rows past the end are zeros.  The sign of a negative scale
        // goes into Q, so that the maximum of the scores is the maximum of what is exponentiated.
        {
            const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
            constexpr int CHUNKS = 2 * kTcM * 16, EACH = CHUNKS / 512;
            uint4 w[EACH];  // every read in flight before the first is used; whole warps, 16 lanes a row
#pragma unroll
            for (int u = 0; u < EACH; u++) {
                const int x = threadIdx.x + u * 512, r = r0 + (x >> 4), i = token_of(p, r);
                w[u] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows)
                    w[u] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.Q) + (sq.q0 + i) * p.qt +
                                                                 (int64_t)(h * p.G + r - i * p.G) * p.qh) + (x & 15));
            }
#pragma unroll
            for (int u = 0; u < EACH; u++) {
                const int x = threadIdx.x + u * 512, row = x >> 4, c = x & 15;
                w[u].x ^= flip; w[u].y ^= flip; w[u].z ^= flip; w[u].w ^= flip;
                if constexpr (!WIDE) {
                    float mul = 1.f;
                    if constexpr (QB) w[u] = normalised_f16(w[u], mul, 16);
                    if (c == 0) sh.qmul[row] = mul;
                }
                const uint32_t at = (row >> 7) * kSlot + (c >> 3) * kHalf + (row & 127) * 128 + (((c & 7) ^ (row & 7)) << 4);
                *reinterpret_cast<uint4 *>(sQ + at) = w[u];
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.q_full));
            // 8 bits: the rows' powers of two are read across warps.  No key in sight: the output's
            // rows go where Q lies, and no product's end says that every warp is through with it.
            if (!WIDE || n == 0) meet<512>(11, true);
        }
        const int t = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
        const int row = quarter * 32 + lane, r = r0 + t * kTcM + row;
        const int id = 3 + t * 4 + quarter;  // named barrier of the two warps of these rows
        if (t < nt) {
            const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
            const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + 256 + t * 128 + half * 64;
            // the tiles that every row of this warp sees whole: [open, shut)
            int open, shut;
            {
                const int a = token_of(p, min(r - lane, rows - 1)), z = token_of(p, min(r - lane + 31, rows - 1));
                open = (seen_lo(p, sq, z) + kTcN - 1) / kTcN - j0;
                shut = seen_hi(p, sq, a) / kTcN - j0;
            }
            const float row_mult = WIDE ? fabsf(p.scale_log2) : sh.qmul[t * kTcM + row] * (FOLD ? fabsf(p.scale_log2) : 1.f);
            float m = -INFINITY, l = 0.f;
            int e = 0;
            // (a wait that gives up raises the abort flag: a warp skips its work from then on, but
            // keeps meeting the other at every barrier)
            bool ok = true;
            for (int j = 0; j < n; j++) {
                const int buf = j & 1;
                ok = ok && wait(sh.s_full[t], j) && (WIDE || wait(sh.sc_full[buf], j >> 1));
                ok = !__any_sync(0xffffffffu, !ok);
                const bool masked = j < open || j >= shut;
                // 32 of the thread's 64 scores, from column hc of its half on: scaled by their
                // keys where that was not done before, -infinity where hidden
                auto finish = [&](int hc, float s[32]) {
                    if constexpr (!WIDE && !FOLD) {
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(&sh.ks[buf][half * 64 + hc + c]);
                            const float2 x = __fmul2_rn(make_float2(s[c], s[c + 1]), make_float2(f.x, f.y));
                            const float2 y = __fmul2_rn(make_float2(s[c + 2], s[c + 3]), make_float2(f.z, f.w));
                            s[c] = x.x; s[c + 1] = x.y; s[c + 2] = y.x; s[c + 3] = y.y;
                        }
                    }
                    if (masked) {
                        const int k0 = (j0 + j) * kTcN + half * 64 + hc, i = token_of(p, min(r, rows - 1));
                        const int a = seen_lo(p, sq, i) - k0, z = seen_hi(p, sq, i) - k0;
#pragma unroll
                        for (int c = 0; c < 32; c++) s[c] = c >= a && c < z ? s[c] : -INFINITY;
                    }
                };
                auto largest = [](const float s[32]) {
                    float m0 = fmax3(s[0], s[1], s[2]), m1 = fmax3(s[3], s[4], s[5]);
#pragma unroll
                    for (int c = 6; c < 30; c += 4) {
                        m0 = fmax3(m0, s[c], s[c + 1]);
                        m1 = fmax3(m1, s[c + 2], s[c + 3]);
                    }
                    return fmaxf(fmax3(m0, s[30], s[31]), m1);
                };
                // 16 bits: the scores stay in registers.  8 bits, with more warps and fewer
                // registers each, many would spill (some values do as it is, 20 to 76 bytes a thread
                // in all forms): they are read twice, for their maximum and for the weights (2.03 ->
                // 1.94 ms; in 16 bits it costs 643 -> 675 us).
                constexpr bool TWICE = !WIDE;
                float s[TWICE ? 32 : 64], mx = -INFINITY, mult = row_mult;
                if (ok) {
                    tc_fence_after();
                    // (kept above 0, so that -infinity times it stays -infinity)
                    if constexpr (FOLD) mult = fmaxf(mult * __uint_as_float((uint32_t)(127 + sh.kexp[buf] - kKeyShift) << 23), 1.2e-38f);
                    if constexpr (TWICE) {
                        tc_ld32(s_at + half * 64, s);
                        finish(0, s);
                        mx = largest(s);
                        tc_ld32(s_at + half * 64 + 32, s);
                        finish(32, s);
                        mx = fmaxf(mx, largest(s)) * mult;
                        tc_ld32_start(s_at + half * 64, s);  // arrives during the vote
                    } else {
                        tc_ld32(s_at + half * 64, s);
                        tc_ld32(s_at + half * 64 + 32, s + 32);
                        finish(0, s);
                        finish(32, s + 32);
                        mx = fmaxf(largest(s), largest(s + 32)) * mult;
                    }
                    if constexpr (!WIDE) {
                        const uint4 odd = *reinterpret_cast<const uint4 *>(sh.vnan[buf]);
                        if (odd.x | odd.y | odd.z | odd.w) {
                            const int k0 = (j0 + j) * kTcN + half * 64, i = token_of(p, min(r, rows - 1));
                            const uint64_t bits = half ? odd.z | (uint64_t)odd.w << 32 : odd.x | (uint64_t)odd.y << 32;
                            for (int c = 0; c < 64; c++)
                                if (bits >> c & 1 && k0 + c >= seen_lo(p, sq, i) && k0 + c < seen_hi(p, sq, i)) atomicOr(&sh.bad[t][quarter], 1u << lane);
                        }
                    }
                }
                // The base moves for a row when its scores pass it by 2^8 (the first tile sets
                // it), for all rows of the two warps that share them together, or when the
                // reference of 8-bit values moved.  Nothing else needs the other thread.
                const bool raise = mx > m + kLazy;  // -inf + 8: any score raises it
                int e_new = e;
                if constexpr (!WIDE) e_new = ok ? sh.vexp[buf] : e;
                if (!meet<64>(id, ok && !raise && j > 0 && e_new == e)) {
                    if (TWICE && ok) tc_ld32_wait(s);  // nothing below may move registers that are still to be written
                    // the larger of the two threads' maxima
                    sh.xmax[t][half][row] = mx;
                    meet<64>(id, true);
                    mx = fmaxf(mx, sh.xmax[t][half ^ 1][row]);
                    meet<64>(id, true);
                    const bool up = mx > m + kLazy;
                    const float m_new = up || j == 0 ? mx : m;
                    float f = up ? fast_exp2(m - exp_base(m_new)) : 1.f;
                    l *= f;
                    m = m_new;
                    if constexpr (!WIDE) f = ldexpf(f, e - e_new);
                    if (j > 0) {
                        ok = ok && wait(sh.o_done[t], j - 1);
                        ok = !__any_sync(0xffffffffu, !ok);
                        tc_fence_after();
                        rescale64(o_at, f);
                        // weights of one thread start a product into all of the row's O: both
                        // halves of O are rescaled before either goes on
                        tc_fence_before();
                        meet<64>(id, true);
                    }
                }
                if (!ok) continue;
                e = e_new;
                const float base = exp_base(m);
                const float2 nb = make_float2(-base, -base), sc2 = make_float2(mult, mult);
                float2 la = make_float2(0.f, 0.f), lb = la;
#pragma unroll
                for (int hc = 0; hc < 64; hc += 32) {
                    if constexpr (TWICE) {
                        if (hc) tc_ld32_start(s_at + half * 64 + hc, s);
                        tc_ld32_wait(s);
                        finish(hc, s);
                    }
                    const float *y = TWICE ? s : s + hc;
                    uint32_t w[16];
                    float4 vs4 = make_float4(1.f, 1.f, 1.f, 1.f);
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        float2 x = __ffma2_rn(make_float2(y[c], y[c + 1]), sc2, nb);
                        x.x = fast_exp2(x.x);
                        x.y = fast_exp2(x.y);
                        if (c & 2) lb = __fadd2_rn(lb, x); else la = __fadd2_rn(la, x);
                        if constexpr (!WIDE && !FOLD) {
                            if (!(c & 2)) vs4 = *reinterpret_cast<const float4 *>(&sh.vs[buf][half * 64 + hc + c]);
                            x = __fmul2_rn(x, c & 2 ? make_float2(vs4.z, vs4.w) : make_float2(vs4.x, vs4.y));
                        }
                        w[c >> 1] = BF ? pack_bf16(x.x, x.y) : pack_f16(x.x, x.y);
                    }
                    // weights over scores that were read, so nobody else's: the product starts
                    // with the first 32 keys of either half
                    tc_st16(s_at + half * 64 + (hc >> 1), w);
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_if(smem_u32(&sh.p_full[t][hc >> 5]), lane == 0);
                }
                const float2 ls = __fadd2_rn(la, lb);
                l += ls.x + ls.y;
                if constexpr (!WIDE) {
                    mbar_arrive_if(smem_u32(&sh.sc_empty[buf]), lane == 0);
                }
            }
            if (n > 0) ok = ok && wait(sh.o_done[t], n - 1) && (WIDE || !redo_possible(p) || wait(sh.sizes, 0));
            __syncwarp();
            // the row's weight sum
            float *xl = sh.xmax[t][0];
            meet<64>(id, true);
            xl[half * kTcM + row] = l;
            ok = meet<64>(id, ok);
            l += xl[(half ^ 1) * kTcM + row];
            tc_fence_after();
            if (ok) {
                const int i = token_of(p, min(r, rows - 1)), hq = h * p.G + min(r, rows - 1) - i * p.G;
                const bool live = r < rows, whole = S == 1;
                // rows to be done again: for their scores' size, or (8 bits) what they see is too small
                // for a reference
                bool again = is_finite(m) && fabsf(m) > kHugeScore;
                auto check_sizes = [&] {
                    const uint32_t v_some = sh.some[1], v_all = sh.all[1], k_some = sh.some[0], k_all = sh.all[0];
                    constexpr int VALUE_FAR = FOLD ? kFoldedFar : kValueFar;
                    if (too_far(v_some, __uint_as_float(v_all), VALUE_FAR) || too_far(k_some, __uint_as_float(k_all), kKeyFar)) {
                        const KeySpans sp = key_spans(p, sq, r0, min(rows, r0 + 2 * kTcM), max(lo, j0 * kTcN), min(hi, (j0 + n) * kTcN));
                        again |= sees_too_little(p, p.vs, b, h, sp, r0, i, v_some, v_all, VALUE_FAR);
                        again |= sees_too_little(p, p.ks, b, h, sp, r0, i, k_some, k_all, kKeyFar);
                    }
                };
                // (behind the output, the compiler spills less of the loop over e4m3 pages, 918 -> 904 us
                // for 4680 x 32760 x 12 heads, and more over int8, 957 -> 1000)
                if constexpr (!WIDE && FMT != PF_E4M3) check_sizes();
                float inv = 1.f;
                if (whole) inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
                if constexpr (!WIDE) inv = sh.bad[t][quarter] >> lane & 1u ? NAN : ldexpf(inv, e - kValueShift);
                const int64_t tok = sq.q0 + i;
                const int64_t part = (tail * S + split) * p.unit + t * kTcM + row;
                // The rows go out through shared memory, in the place of this tile's Q, which
                // every product has read: a thread leaves 128 bytes of its row there at a time
                // (64 channels in 16 bits, 32 in fp32; swizzled), and eight lanes write a row's
                // 128 bytes out together.  (Each thread writing its own row, 8 bytes at a time
                // 32 rows apart, took 6 us of a CTA's end.)
                const bool narrow = whole && p.out_dtype != DT_F32;
                const int64_t elem = narrow ? 2 : 4, at = (whole ? tok * p.ot + hq * p.oh : part * kD) * elem;
                unsigned char *dst = static_cast<unsigned char *>(whole ? p.O : p.part);
                unsigned char *stage = sQ + t * kSlot + half * 128;  // + row * 256
                bool odd = false;
                auto leave = [&](int c, uint4 v) { *reinterpret_cast<uint4 *>(stage + row * 256 + ((c ^ (row & 7)) << 4)) = v; };
                auto write_out = [&](int first_channel) {
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 8; u++) {
                        const int src = u * 4 + (lane >> 3), c = lane & 7, other = quarter * 32 + src;
                        const int64_t to = __shfl_sync(0xffffffffu, at, src) + first_channel * elem + c * 16;
                        const uint4 v = *reinterpret_cast<const uint4 *>(stage + other * 256 + ((c ^ (other & 7)) << 4));
                        if (__shfl_sync(0xffffffffu, (int)live, src)) *reinterpret_cast<uint4 *>(dst + to) = v;
                    }
                    __syncwarp();
                };
#pragma unroll
                for (int hc = 0; hc < 64; hc += 32) {
                    float o[32];
                    __syncwarp();
                    if (n > 0) {
                        tc_ld32(o_at + hc, o);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k++) o[k] = 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < 32; k++) {
                        o[k] *= inv;
                        if constexpr (FMT != PF_INT8) odd |= !is_finite(o[k]);
                    }
                    if (narrow) {
                        auto pk = [&](int k) {
                            return p.out_dtype == DT_BF16 ? pack_bf16(o[k], o[k + 1]) : pack_f16(o[k], o[k + 1]);
                        };
#pragma unroll
                        for (int k = 0; k < 32; k += 8) leave((hc + k) >> 3, make_uint4(pk(k), pk(k + 2), pk(k + 4), pk(k + 6)));
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            leave(k >> 2, make_uint4(__float_as_uint(o[k]), __float_as_uint(o[k + 1]), __float_as_uint(o[k + 2]),
                                                     __float_as_uint(o[k + 3])));
                        write_out(half * 64 + hc);
                    }
                }
                if (narrow) write_out(half * 64);
                if constexpr (FMT == PF_E4M3) check_sizes();
                if (!whole) {
                    if (live && half == 0) *reinterpret_cast<float2 *>(p.ml + 2 * part) = make_float2(m, again ? kRedo : l);
                } else {
                    if (live && half == 0 && p.lse) p.lse[tok * p.HQ + hq] = row_lse(m, l);
                    if constexpr (FMT != PF_INT8) {
                        // (with 8 bits, lo and hi kept until here would cost registers in the loop)
                        if (redo_possible(p) && __any_sync(0xffffffffu, odd && live))
                            again |= odd & (WIDE ? spoilt(p, b, h, i, lo, hi) : spoilt_in(p, b, h, i, r0));
                    }
                    // both halves written, then each of the two warps takes its share of the rows
                    // that are to be done again
                    const uint32_t mine = __ballot_sync(0xffffffffu, live && again);
                    if (lane == 0) sh.odd[t][quarter][half] = mine;
                    __threadfence_block();
                    meet<64>(id, true);
                    uint32_t todo = mine | sh.odd[t][quarter][half ^ 1];
                    todo &= half ? 0xAAAAAAAAu : 0x55555555u;
                    while (todo) {
                        const int src = __ffs(todo) - 1;
                        todo &= todo - 1;
                        const int ri = __shfl_sync(0xffffffffu, i, src), rh = __shfl_sync(0xffffffffu, hq, src);
                        float ro[4], rm, rl;
                        redo_row(p, b, ri, rh, ro, rm, rl);
                        const float f = rl == 0.f ? 0.f : __fdiv_rn(1.f, rl);
#pragma unroll
                        for (int c = 0; c < 4; c++) ro[c] *= f;
                        store_out4(p, (sq.q0 + ri) * p.ot + rh * p.oh + 4 * lane, ro);
                        if (p.lse && lane == 0) p.lse[(sq.q0 + ri) * p.HQ + rh] = row_lse(rm, rl);
                    }
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) or_status(p.status, QVG_DEV_TIMEOUT);
    if (warp == MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

namespace {
template <bool QB, int FMT, bool FOLD>
cudaError_t launch_tc(const PAttnPlan &p, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st) {
    using T = TcShape<FMT>;
    constexpr size_t smem = tc_smem<FMT>();
    const auto kernel = k_page_attn_tc<QB, FMT, FOLD>;
    cudaError_t e = allow_smem<k_page_attn_tc<QB, FMT, FOLD>>(smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = p.whole + (p.items - p.whole) * p.S;
    return launch_kernel(kernel, dim3((unsigned)grid), dim3(T::THREADS), smem, st, mk, mv, p);
}
}  // namespace

cudaError_t launch_page_attention_tc(const PAttnPlan &p, cudaStream_t st) {
    CUtensorMap maps[2];
    const bool wide = p.fmt == PF_F16 || p.fmt == PF_BF16;
    const int box = wide ? p.page : std::min(p.page, kRawKeys);
    if (!page_map(p, p.k, box, &maps[0]) || !page_map(p, p.v, box, &maps[1])) return cudaErrorInvalidValue;
    const bool fold = !p.lse && p.out_dtype == DT_BF16;
    auto go = [&](auto qb) {
        constexpr bool QB = decltype(qb)::value;
        if (p.fmt == PF_E4M3)
            return fold ? launch_tc<QB, PF_E4M3, true>(p, maps[0], maps[1], st) : launch_tc<QB, PF_E4M3, false>(p, maps[0], maps[1], st);
        if (p.fmt == PF_INT8)
            return fold ? launch_tc<QB, PF_INT8, true>(p, maps[0], maps[1], st) : launch_tc<QB, PF_INT8, false>(p, maps[0], maps[1], st);
        return launch_tc<QB, QB ? PF_BF16 : PF_F16, false>(p, maps[0], maps[1], st);
    };
    return p.q_dtype == DT_BF16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace qvg
