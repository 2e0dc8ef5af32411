// The pages of sequences: copied, taken for new tokens, shared by forks, given back, and packed
// into another pool.  refs[p] counts the table entries that name page p; 0 is free.
//
// Data movement (copies, the part-filled pages of forks, compaction) is bound by memory: pages are
// whole arrays of 16-byte pieces, read and written once.  The bookkeeping is bound by latency: one
// thread-block cluster finds the lowest free (or live) pages by counting, in tiles of 16 pages a
// thread, so that what is taken does not depend on the order in which threads run, and a call is one
// launch, or two where pages are copied.
#include "internal.cuh"
#include "tcgen.cuh"

namespace qvg {

namespace {
constexpr int kCopyThreads = 256;
constexpr int kCopyEach = 4;                         // 16-byte pieces of a thread, all in flight
constexpr int kCopyPieces = kCopyThreads * kCopyEach;
constexpr int kBookThreads = 1024;
constexpr int kTilePages = kBookThreads * 16;        // pages that a CTA counts at a time
constexpr int kBookCluster = 8;
constexpr int kBookRows = kBookSharedRows;
constexpr int kBookCows = 256;
constexpr int kBookFew = 1024;                       // pages taken that are handed over in shared memory

__device__ __forceinline__ bool in_pool(int page, int64_t n_pages) { return (unsigned)page < (uint64_t)n_pages; }
__device__ __forceinline__ int pages_for(int64_t tokens, int shift) { return (int)((tokens + (1 << shift) - 1) >> shift); }

// Piece x of a page: which array, and where in the page's part of it.  Rows [0, rows) are copied.
__device__ __forceinline__ void copy_piece(const PoolCopy &c, int64_t src, int64_t dst, int64_t x, int rows, uint4 *held, bool store) {
    int a = 0;
#pragma unroll
    for (int k = 1; k < 6; k++) a += x >= c.from[k];
    const int64_t at = x - c.from[a], bytes = c.bytes[a];
    const int row = (int)((at * 16) >> c.row_shift[a]) & (c.page - 1);
    if (row >= rows) return;
    if (!store) {
        *held = __ldg(reinterpret_cast<const uint4 *>(c.src[a] + src * bytes) + at);
        return;
    }
    uint8_t *to = c.dst[a] + dst * bytes + at * 16;
    const int units = (rows - row) << c.row_shift[a];  // bytes of the piece's rows that are copied
    if (units >= 16) {
        *reinterpret_cast<uint4 *>(to) = *held;
    } else {  // scales of 4 bytes, group scales of 8
        const uint32_t w[4] = {held->x, held->y, held->z, held->w};
#pragma unroll
        for (int k = 0; k < 3; k++)
            if (4 * k < units) reinterpret_cast<uint32_t *>(to)[k] = w[k];
    }
}
__device__ __forceinline__ void copy_block(const PoolCopy &c, int64_t src, int64_t dst, int64_t block, int rows) {
    uint4 held[kCopyEach];
    const int64_t x0 = block * kCopyPieces + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kCopyEach; k++)
        if (x0 + k * kCopyThreads < c.from[6]) copy_piece(c, src, dst, x0 + k * kCopyThreads, rows, &held[k], false);
#pragma unroll
    for (int k = 0; k < kCopyEach; k++)
        if (x0 + k * kCopyThreads < c.from[6]) copy_piece(c, src, dst, x0 + k * kCopyThreads, rows, &held[k], true);
}

// Sums over the threads before this one, and over all, of a CTA of 1024: N numbers at a time, none
// negative, cut at the largest (what comes to that much is too much for any call).
constexpr uint32_t kMost = 0x7FFFFFFFu;
__device__ __forceinline__ uint32_t add_cut(uint32_t a, uint32_t b) { return min(a + b, kMost); }
template <int N>
__device__ __forceinline__ void block_scan(uint32_t (&v)[N], uint32_t (*s_warp)[32], uint32_t (&all)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t upto[N], before[N];
#pragma unroll
    for (int k = 0; k < N; k++) upto[k] = v[k];
#pragma unroll
    for (int x = 1; x < 32; x <<= 1)
#pragma unroll
        for (int k = 0; k < N; k++) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto[k], x);
            if (lane >= x) upto[k] = add_cut(upto[k], y);
        }
#pragma unroll
    for (int k = 0; k < N; k++) {
        before[k] = __shfl_up_sync(0xffffffffu, upto[k], 1);
        if (lane == 0) before[k] = 0;
    }
    __syncthreads();  // (s_warp may still be read from the scan before)
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < N; k++) s_warp[k][warp] = upto[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; k++) {
        uint32_t w = s_warp[k][lane];
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, w, x);
            if (lane >= x) w = add_cut(w, y);
        }
        all[k] = __shfl_sync(0xffffffffu, w, 31);
        const uint32_t warps = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
        v[k] = add_cut(before[k], warp ? warps : 0u);
    }
}
__device__ __forceinline__ void book_meet(int ctas) {
    if (ctas > 1) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
}

// Counts of the CTAs before this one, and of all, from their shared memory; they meet once more before
// any of them leaves.
__device__ __forceinline__ void book_counts(uint32_t *s_count, int rank, int ctas, uint32_t &before, uint32_t &all) {
    before = 0;
    all = *s_count;
    if (ctas == 1) return;
    all = 0;
    for (int c = 0; c < ctas; c++) {
        uint32_t at, n;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(s_count)), "r"(c));
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(n) : "r"(at));
        if (c < rank) before += n;
        all += n;
    }
}

// Bits of this thread's 16 pages from p0 on: free ones, or those in use.
__device__ __forceinline__ uint32_t page_bits(const int32_t *refs, int64_t p0, int64_t end, bool in_use) {
    uint32_t bits = 0;
    if (p0 + 16 <= end) {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int4 r = *reinterpret_cast<const int4 *>(refs + p0 + 4 * k);
            bits |= ((uint32_t)(r.x > 0) | (uint32_t)(r.y > 0) << 1 | (uint32_t)(r.z > 0) << 2 | (uint32_t)(r.w > 0) << 3) << (4 * k);
        }
        return in_use ? bits : ~bits & 0xFFFFu;
    }
    for (int k = 0; k < 16; k++)
        if (p0 + k < end && (refs[p0 + k] > 0) == in_use) bits |= 1u << k;
    return bits;
}
// This CTA's pages: whole tiles, as many for each.
__device__ __forceinline__ void book_span(int64_t n_pages, int rank, int ctas, int64_t &from, int64_t &to) {
    const int64_t tiles = (n_pages + kTilePages - 1) / kTilePages, per = (tiles + ctas - 1) / ctas;
    from = min(rank * per * kTilePages, n_pages);
    to = min(from + per * kTilePages, n_pages);
}
// Pages of this CTA, in use or free.  The first tile is looked at once, at the start, and kept.
struct BookPages {
    const int32_t *refs;
    int64_t n_pages, from, to;
    bool in_use;
    uint32_t bits, at;  // the first tile's, and this thread's place in it
    uint32_t tile, count;  // pages found in the first tile, and in all
    __device__ __forceinline__ BookPages(const int32_t *r, int64_t n, int rank, int ctas, bool used) : refs(r), n_pages(n), in_use(used) {
        book_span(n, rank, ctas, from, to);
        const int64_t p0 = from + threadIdx.x * 16;
        bits = p0 < to ? page_bits(refs, p0, n_pages, in_use) : 0u;
    }
    // `scanned`: the first tile's scan, if it was made with others
    __device__ __forceinline__ void count_all(uint32_t before, uint32_t all, uint32_t (*s_warp)[32]) {
        at = before;
        tile = count = all;
        if (to - from <= kTilePages) return;
        uint32_t n[1] = {0}, rest[1];
        for (int64_t p = from + kTilePages + threadIdx.x * 16; p < to; p += kTilePages) n[0] += __popc(page_bits(refs, p, n_pages, in_use));
        block_scan(n, s_warp, rest);
        count += rest[0];
    }
    // Calls take(place, page) for each page, place counting from `first`, until `limit`.
    template <typename F>
    __device__ __forceinline__ void each(uint32_t first, uint32_t limit, uint32_t (*s_warp)[32], F &&take) {
        auto go = [&](uint32_t b, uint32_t place, int64_t p0) {
            while (b && place < limit) {
                const int k = __ffs(b) - 1;
                b &= b - 1;
                take((int)place++, (int)(p0 + k));
            }
        };
        go(bits, first + at, from + threadIdx.x * 16);
        first += tile;
        for (int64_t t = from + kTilePages; t < to && first < limit; t += kTilePages) {
            const int64_t p0 = t + threadIdx.x * 16;
            const uint32_t b = p0 < n_pages ? page_bits(refs, p0, n_pages, in_use) : 0u;
            uint32_t n[1] = {(uint32_t)__popc(b)}, all[1];
            block_scan(n, s_warp, all);
            go(b, first + n[0], p0);
            first += all[0];
        }
    }
};

// Last row whose first place is at most x, of n > 0 rows in order.
template <typename F>
__device__ __forceinline__ int row_of_place(F &&first, int n, int64_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first(mid) <= x) lo = mid; else hi = mid;
    }
    return lo;
}
}  // namespace

// ------------------------------------------------------------------------------------ copies

__global__ void __launch_bounds__(kCopyThreads) k_page_copy(const __grid_constant__ PCopyPlan p) {
    pdl_begin();
    const int64_t i = blockIdx.x / p.per;
    const int src = __ldg(p.src + i), dst = __ldg(p.dst + i);
    int rows = p.rows ? __ldg(p.rows + i) : p.pool.page;
    if (src < 0 || dst < 0) return;
    if (!in_pool(src, p.src_pages) || !in_pool(dst, p.dst_pages) || rows < 0 || rows > p.pool.page) {
        if (threadIdx.x == 0 && blockIdx.x == i * p.per) or_status(p.status, QVG_DEV_BAD_INDEX);
        if (!in_pool(src, p.src_pages) || !in_pool(dst, p.dst_pages)) return;
        rows = min(max(rows, 0), p.pool.page);
    }
    copy_block(p.pool, src, dst, blockIdx.x - i * p.per, rows);
}

// ------------------------------------------------------------------------------------ pages taken

// What a sequence wants of the free pages.
struct TakeRow {
    int first, need;   // its places among the pages taken
    int len, count;    // tokens before, new tokens
    int entries;       // table entries that stay before the new ones
    int src;           // page to be copied, -1: none
    int last;          // page of the last of those entries, where it is part filled
    int token;         // first of its tokens among all
    int ok;
};

__device__ __forceinline__ bool in_use(const PTakePlan &p, int page) { return in_pool(page, p.n_pages) && p.refs[page] > 0; }

// One cluster.  Sequence b wants need pages: for a fork, one if its parent's last page is part
// filled; for new tokens, what they fill, and one more in place of a part-filled last page that others
// share.  The wants in order of sequence are places 0, 1, ... of the free pages in ascending order;
// from the first sequence that they do not suffice for, none that wants any is served.  Every CTA
// works out all wants (so that only the counts of free pages have to be exchanged), in shared memory
// where there is room.
template <bool FORK>
__global__ void __launch_bounds__(kBookThreads, 1) k_page_take(const __grid_constant__ PTakePlan p) {
    pdl_begin();
    __shared__ TakeRow s_rows[kBookRows];
    __shared__ uint32_t s_warp[3][32], s_count;
    __shared__ int s_cow, s_list[kBookFew], s_cows[kBookCows];  // shared last pages: how many, whose
    const int ctas = gridDim.x, rank = blockIdx.x, tid = threadIdx.x;
    const int shift = 31 - __clz(p.page);
    const int64_t cap = (int64_t)p.max_pages << shift;
    TakeRow *rows = p.B <= kBookRows ? s_rows : static_cast<TakeRow *>(p.rows);
    uint32_t *status = rank == 0 ? p.status : nullptr;
    BookPages pages(p.refs, p.n_pages, rank, ctas, false);
    if (tid == 0) s_cow = 0;
    uint32_t places = 0, tokens = 0;
    // Few pages and tokens for each sequence, all in one CTA: each thread sees to one sequence, with
    // the pages by place in shared memory.  (Else a thread has a page, or a token, and looks its sequence
    // up.)
    bool few = FORK || p.total <= kBookThreads * 16;
    for (int b0 = 0; b0 < p.B; b0 += kBookThreads) {
        const int b = b0 + tid;
        TakeRow r = {};
        r.src = -1;
        uint32_t n = 0;
        if (b < p.B) {
            int64_t len = p.lens[b];
            if constexpr (FORK) {
                const int parent = p.wants[b];
                if (parent >= 0) {
                    bool ok = parent < p.B && len == 0 && p.wants[parent] < 0;
                    if (ok) {
                        len = p.lens[parent];
                        ok = len >= 0 && len <= cap;
                    }
                    if (ok) {
                        r.entries = (int)(len >> shift);
                        r.len = (int)len;
                        r.ok = 1;
                        if (len & (p.page - 1)) {
                            r.need = 1;
                            r.src = p.table[(int64_t)parent * p.max_pages + r.entries];
                            ok = in_use(p, r.src);
                        }
                    }
                    if (!ok) {
                        r = {};
                        r.src = -1;
                        or_status(status, QVG_DEV_BAD_INDEX);
                    }
                }
            } else {
                const int wanted = p.wants[b];
                if (wanted < 0) or_status(status, QVG_DEV_BAD_INDEX);
                n = (uint32_t)max(wanted, 0);
                r.count = (int)n;
                if (n > 0) {
                    if (len < 0 || len > cap) {
                        or_status(status, QVG_DEV_BAD_INDEX);
                    } else if (len + n > cap) {
                        or_status(status, QVG_DEV_NO_PAGES);
                    } else {
                        const int have = pages_for(len, shift);
                        r.len = (int)len;
                        r.entries = have;
                        r.need = pages_for(len + n, shift) - have;
                        r.ok = 1;
                        if (len & (p.page - 1)) {
                            const int last = r.last = p.table[(int64_t)b * p.max_pages + have - 1];
                            if (!in_use(p, last)) {
                                r.ok = r.need = 0;
                                or_status(status, QVG_DEV_BAD_INDEX);
                            } else if (p.refs[last] > 1) {
                                r.src = last;
                                r.need++;
                                r.entries--;
                            }
                        }
                    }
                }
            }
        }
        // one scan for the tokens, the wants and, the first time, the free pages.  (A sequence whose tokens
        // pass the total wants no page, which only a scan of the tokens can tell: then the wants are
        // scanned again.)
        const uint32_t wanted = r.need;
        uint32_t v[3] = {n, wanted, b0 == 0 ? (uint32_t)__popc(pages.bits) : 0u}, all[3];
        block_scan(v, s_warp, all);
        if (b0 == 0) pages.count_all(v[2], all[2], s_warp);
        if constexpr (!FORK) {
            r.token = (int)add_cut(tokens, v[0]);
            const bool over = r.ok && (int64_t)r.token + n > p.total;
            tokens = add_cut(tokens, all[0]);
            if (over) {
                r.ok = r.need = 0;
                or_status(status, QVG_DEV_BAD_INDEX);
            }
            few &= !__syncthreads_or(n > 16);
            if (__syncthreads_or(over)) {
                uint32_t w[1] = {(uint32_t)r.need}, sum[1];
                block_scan(w, s_warp, sum);
                v[1] = w[0];
                all[1] = sum[0];
            }
            if (r.ok && r.src >= 0) {
                const int k = atomicAdd(&s_cow, 1);
                if (k < kBookCows) s_cows[k] = b;
            }
        }
        r.first = (int)add_cut(places, v[1]);
        places = add_cut(places, all[1]);
        if (b < p.B) rows[b] = r;
    }
    if (tid == 0) s_count = pages.count;
    book_meet(ctas);
    uint32_t before, free_pages;
    book_counts(&s_count, rank, ctas, before, free_pages);
    // a sequence that wants nothing is served; others, if all up to it are
    auto served = [&](const TakeRow &r) { return r.ok && (r.need == 0 || (uint32_t)r.first + (uint32_t)r.need <= free_pages); };
    uint32_t take = places;
    if (take > free_pages) {
        take = 0;
        for (int b = tid; b < p.B; b += kBookThreads) {
            const uint32_t end = (uint32_t)rows[b].first + (uint32_t)rows[b].need;
            if (end <= free_pages) take = max(take, end);
        }
        __syncthreads();
        take = __reduce_max_sync(0xffffffffu, take);
        if ((tid & 31) == 0) s_warp[0][tid >> 5] = take;
        __syncthreads();
        take = __reduce_max_sync(0xffffffffu, s_warp[0][tid & 31]);
    }
    few &= ctas == 1 && p.B <= kBookRows && take <= kBookFew;
    pages.each(before, take, s_warp, [&](int place, int page) {
        p.refs[page] = 1;  // (this thread alone looks at this count)
        if (few) {
            s_list[place] = page;
            return;
        }
        const int b = row_of_place([&](int k) { return rows[k].first; }, p.B, place);
        p.table[(int64_t)b * p.max_pages + rows[b].entries + place - rows[b].first] = page;
        if constexpr (FORK) p.copies[p.B + b] = page;
    });
    if (few || !FORK || ctas > 1) book_meet(ctas);  // the table is complete; nobody leaves while its count is read
    const int grid = ctas * kBookThreads, me = rank * kBookThreads + tid;
    for (int b = me; b < p.B; b += grid) {
        const TakeRow r = rows[b];
        const bool ok = served(r), copied = ok && r.src >= 0 && r.need > 0;
        if (r.ok && !ok) or_status(p.status, QVG_DEV_NO_PAGES);
        if (few && ok) {
            for (int j = 0; j < r.need; j++) p.table[(int64_t)b * p.max_pages + r.entries + j] = s_list[r.first + j];
            if (FORK && copied) p.copies[p.B + b] = s_list[r.first];
        }
        if constexpr (FORK) {
            // (the entries that are shared, and the copies, are left to the next kernel)
            p.copies[b] = copied ? r.src : -1;
            if (!copied) p.copies[p.B + b] = -1;
            p.copies[2 * p.B + b] = copied ? r.len & (p.page - 1) : 0;
            p.copies[3 * p.B + b] = ok ? r.entries : -1;
            if (ok) p.lens[b] = r.len;
            if (ok && p.starts) p.starts[b] = p.starts[p.wants[b]];
        } else {
            if (ok && r.count > 0) p.lens[b] = r.len + r.count;
            if (copied) atomicSub(p.refs + r.src, 1);
            if (p.copies) {
                p.copies[b] = copied ? r.src : -1;
                p.copies[p.B + b] = copied ? p.table[(int64_t)b * p.max_pages + r.entries] : -1;
                p.copies[2 * p.B + b] = copied ? r.len & (p.page - 1) : 0;
            }
            if (few) {
                const int64_t start = ok && r.count > 0 && p.starts ? p.starts[b] : 0;
                for (int k = 0; k < r.count && r.token + k < p.total; k++) {
                    int64_t slot = -1, pos = -1;
                    if (ok) {
                        pos = r.len + k;
                        const int entry = (int)(pos >> shift), page = entry < r.entries ? r.last : s_list[r.first + entry - r.entries];
                        slot = ((int64_t)page << shift) + (pos & (p.page - 1));
                        pos += start;
                    }
                    p.slots[r.token + k] = slot;
                    p.positions[r.token + k] = pos;
                }
            }
        }
    }
    if constexpr (!FORK) {
        for (int64_t x = few ? (int64_t)tokens + me : me; x < p.total; x += grid) {  // (few: what no sequence has)
            int64_t slot = -1, pos = -1;
            if (x < tokens) {
                const int b = row_of_place([&](int k) { return rows[k].token; }, p.B, x);
                const TakeRow r = rows[b];
                if (served(r)) {
                    pos = r.len + (x - r.token);
                    const int64_t page = p.table[(int64_t)b * p.max_pages + (pos >> shift)];
                    slot = (page << shift) + (pos & (p.page - 1));
                    if (p.starts) pos += p.starts[b];
                }
            }
            p.slots[x] = slot;
            p.positions[x] = pos;
        }
        // shared last pages, which nobody else of this call writes: seldom any
        if (s_cow > 0) {
            if (few) __syncthreads();  // (the table has its copies)
            const bool listed = s_cow <= kBookCows;  // (in any order: nothing depends on it)
            for (int c = 0; c < (listed ? s_cow : p.B); c++) {
                const int b = listed ? s_cows[c] : c;
                const TakeRow r = rows[b];
                if (r.src < 0 || !served(r)) continue;
                const int dst = p.table[(int64_t)b * p.max_pages + r.entries];
                for (int64_t x = me; x < p.pool.from[6]; x += grid) {
                    uint4 v;
                    copy_piece(p.pool, r.src, dst, x, r.len & (p.page - 1), &v, false);
                    copy_piece(p.pool, r.src, dst, x, r.len & (p.page - 1), &v, true);
                }
            }
        }
    }
}

// The rest of a fork, `split` blocks a sequence: its shared entries, and its part-filled page's rows.
__global__ void __launch_bounds__(kCopyThreads) k_page_fork(const __grid_constant__ PTakePlan p, int split, int per) {
    pdl_begin();
    const int b = blockIdx.x / split, part = blockIdx.x - b * split;
    const int n = p.copies[3 * p.B + b];
    if (n < 0) return;
    const int src = p.copies[b], dst = p.copies[p.B + b], rows = p.copies[2 * p.B + b];
    const int32_t *from = p.table + (int64_t)p.wants[b] * p.max_pages;
    for (int j = part * kCopyThreads + threadIdx.x; j < n; j += split * kCopyThreads) {
        const int page = from[j];
        p.table[(int64_t)b * p.max_pages + j] = page;
        if (in_pool(page, p.n_pages))
            atomicAdd(p.refs + page, 1);
        else
            or_status(p.status, QVG_DEV_BAD_INDEX);
    }
    if (src >= 0)
        for (int x = part; x < per; x += split) copy_block(p.pool, src, dst, x, rows);
}

// ------------------------------------------------------------------------------------ pages given back

__global__ void __launch_bounds__(256) k_page_free(const __grid_constant__ PFreePlan p) {
    pdl_begin();
    const int shift = 31 - __clz(p.page), tid = threadIdx.x;
    const int64_t cap = (int64_t)p.max_pages << shift;
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const int64_t first = p.first ? p.first[b] : 0, last = p.last ? p.last[b] : 0, given = p.lens[b];
        const int64_t len = min(max(given, (int64_t)0), cap);
        if (tid == 0 && (first < 0 || last < 0 || len != given)) or_status(p.status, QVG_DEV_BAD_INDEX);
        if (first <= 0 && last <= 0) {
            if (tid == 0 && len != given) p.lens[b] = (int)len;
            continue;
        }
        // tokens [a, z) stay, a at the start of a page
        const int64_t z = len - min(max(last, (int64_t)0), len);
        const int64_t a = max(first, (int64_t)0) >= z ? z : (max(first, (int64_t)0) >> shift) << shift;
        const int have = pages_for(len, shift);
        const int e0 = a == z ? have : (int)(a >> shift), e1 = a == z ? have : pages_for(z, shift);  // entries that stay
        int32_t *row = p.table + (int64_t)b * p.max_pages;
        for (int j = tid; j < have; j += 256) {
            if (j >= e0 && j < e1) continue;
            const int page = row[j];
            bool ok = in_pool(page, p.n_pages);
            if (ok && atomicSub(p.refs + page, 1) <= 0) {  // it was free
                atomicAdd(p.refs + page, 1);
                ok = false;
            }
            if (!ok) or_status(p.status, QVG_DEV_BAD_INDEX);
        }
        __syncthreads();
        // entries move up, chunk by chunk: a chunk is read before any of it is written, and what is
        // read lies behind what was written before
        for (int j0 = e0 ? 0 : e1; j0 < have; j0 += 256) {
            const int j = j0 + tid;
            const int page = j + e0 < e1 ? row[j + e0] : -1;
            __syncthreads();
            if (j < have) row[j] = page;
        }
        if (tid == 0) {
            p.lens[b] = (int)(z - a);
            if (p.starts) p.starts[b] = z == 0 && last > 0 ? 0 : p.starts[b] + a;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------ compaction

__global__ void __launch_bounds__(kBookThreads, 1) k_page_rank(const __grid_constant__ PCompactPlan p) {
    pdl_begin();
    __shared__ uint32_t s_warp[1][32], s_count;
    const int ctas = gridDim.x, rank = blockIdx.x, tid = threadIdx.x;
    BookPages pages(p.refs, p.n_pages, rank, ctas, true);
    uint32_t v[1] = {(uint32_t)__popc(pages.bits)}, all[1];
    block_scan(v, s_warp, all);
    pages.count_all(v[0], all[0], s_warp);
    if (tid == 0) s_count = pages.count;
    book_meet(ctas);
    uint32_t before, live;
    book_counts(&s_count, rank, ctas, before, live);
    pages.each(before, kMost, s_warp, [&](int place, int page) {
        p.place[page] = place;
        if (place < p.out_pages) {
            p.old[place] = page;
            p.out_refs[place] = p.refs[page];
        }
    });
    for (int64_t x = (int64_t)rank * kBookThreads + tid; x < p.out_pages; x += ctas * kBookThreads)
        if (x >= live) p.out_refs[x] = 0;
    if (rank == 0 && tid == 0) {
        *p.live = live;
        if (live > p.out_pages) or_status(p.status, QVG_DEV_NO_PAGES);
    }
    if (ctas > 1) book_meet(ctas);
}

// Blocks [0, copy_blocks) copy live pages, the others renumber the table.
__global__ void __launch_bounds__(kCopyThreads) k_page_compact(const __grid_constant__ PCompactPlan p, int copy_blocks, int per) {
    pdl_begin();
    if (blockIdx.x < copy_blocks) {
        const int64_t items = min((int64_t)*p.live, p.out_pages) * per;
        for (int64_t x = blockIdx.x; x < items; x += copy_blocks) {
            const int64_t to = x / per;
            copy_block(p.pool, p.old[to], to, x - to * per, p.pool.page);
        }
        return;
    }
    const int shift = 31 - __clz(p.pool.page);
    const int64_t cap = (int64_t)p.max_pages << shift;
    for (int b = blockIdx.x - copy_blocks; b < p.B; b += gridDim.x - copy_blocks) {
        const int64_t len = p.lens[b];
        if (threadIdx.x == 0 && (len < 0 || len > cap)) or_status(p.status, QVG_DEV_BAD_INDEX);
        const int have = pages_for(min(max(len, (int64_t)0), cap), shift);
        for (int j = threadIdx.x; j < p.max_pages; j += kCopyThreads) {
            int to = -1;
            if (j < have) {
                const int page = p.table[(int64_t)b * p.max_pages + j];
                if (in_pool(page, p.n_pages) && p.refs[page] > 0) {
                    to = p.place[page];
                    if (to >= p.out_pages) to = -1;  // (no room: reported)
                } else {
                    or_status(p.status, QVG_DEV_BAD_INDEX);
                }
            }
            p.out_table[(int64_t)b * p.max_pages + j] = to;
        }
    }
}

// ------------------------------------------------------------------------------------ launches

namespace {
// CTAs of the bookkeeping's cluster: one for small pools and few tokens, where a barrier among CTAs
// costs more than it saves.
int book_ctas(int64_t n_pages, int64_t tokens) {
    int ctas = 1;
    while (ctas < kBookCluster && (n_pages > (int64_t)ctas * kTilePages || tokens > (int64_t)ctas * kBookThreads * 4)) ctas *= 2;
    return ctas;
}
// Blocks of a copy whose size only the device knows: so many that a block has one or a few 16 KB pieces
// (24500 INT4 pages of 8 x 32 tokens, a third shared: 170 us; eight blocks an SM in a loop 202).
int copy_grid(int64_t items) { return (int)std::min<int64_t>(std::max<int64_t>(items, 1), 152 * 256); }
}  // namespace

size_t take_bytes(int64_t sequences) { return sequences <= kBookRows ? 0 : (size_t)sequences * sizeof(TakeRow); }

int64_t copy_blocks_per_page(const PoolCopy &c) { return (c.from[6] + kCopyPieces - 1) / kCopyPieces; }

cudaError_t launch_page_copy(const PCopyPlan &p, cudaStream_t st) {
    return launch_kernel(k_page_copy, dim3((unsigned)(p.n * p.per)), dim3(kCopyThreads), 0, st, p);
}

cudaError_t launch_page_append(const PTakePlan &p, cudaStream_t st) {
    const int ctas = book_ctas(p.n_pages, p.total);
    return launch_kernel_cluster(k_page_take<false>, dim3(ctas), dim3(kBookThreads), 0, ctas, st, p);
}

cudaError_t launch_page_fork(const PTakePlan &p, cudaStream_t st) {
    const int ctas = book_ctas(p.n_pages, 0);
    cudaError_t e = launch_kernel_cluster(k_page_take<true>, dim3(ctas), dim3(kBookThreads), 0, ctas, st, p);
    if (e != cudaSuccess) return e;
    const int per = (int)copy_blocks_per_page(p.pool), split = std::min(per, std::max(1, 152 * 8 / p.B));
    return launch_kernel(k_page_fork, dim3((unsigned)(p.B * split)), dim3(kCopyThreads), 0, st, p, split, per);
}

cudaError_t launch_page_free(const PFreePlan &p, cudaStream_t st) {
    return launch_kernel(k_page_free, dim3((unsigned)std::min(p.B, 152 * 8)), dim3(256), 0, st, p);
}

cudaError_t launch_page_compact(const PCompactPlan &p, cudaStream_t st) {
    const int ctas = book_ctas(p.n_pages, 0);
    cudaError_t e = launch_kernel_cluster(k_page_rank, dim3(ctas), dim3(kBookThreads), 0, ctas, st, p);
    if (e != cudaSuccess) return e;
    const int per = (int)copy_blocks_per_page(p.pool), copies = copy_grid(p.out_pages * per), rows = std::min(p.B, 152 * 4);
    return launch_kernel(k_page_compact, dim3((unsigned)(copies + rows)), dim3(kCopyThreads), 0, st, p, copies, per);
}

}  // namespace qvg
