// Rotary positions: pair (x, y) of a row becomes m (x cos a - y sin a, x sin a + y cos a) with
// a = 2 pi * position * frequency; the gradient is the same with the angle negated.
//
// Bound by memory: each row is read and written once (512 bytes a row in 16 bits against
// about 20 warp instructions).  Sixteen lanes hold a row (rows.cuh) and take up to eight heads
// of one token, so the sines and cosines, four pairs a lane, are computed once for all of them.
// 65536 tokens of 32 heads in bf16: 153 us (7.0 TB/s); 4680 of 12: 6 us.  The first rows are
// asked for before the positions (after them: 163 us).
#include "rows.cuh"

namespace qvg {

namespace {
constexpr int kRopeHeads = 8;  // heads of one token that a half-warp turns
constexpr int kRopeRows = 4;   // of which this many are in flight at once
}  // namespace

template <int DT, bool INTER>
__global__ void __launch_bounds__(256) k_rope(RopePlan p) {
    pdl_begin();
    const int l = threadIdx.x & 15;
    const int groups = (p.heads + kRopeHeads - 1) / kRopeHeads;
    const int64_t unit = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int64_t token = unit / groups;
    if (token >= p.n) return;
    const int h0 = (int)(unit - token * groups) * kRopeHeads, h1 = min(p.heads, h0 + kRopeHeads);
    const Pieces at = pieces_of(l, p.r);
    Raw8<DT> raw[kRopeRows];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < kRopeRows; u++)
            if (h + u < h1) raw[u] = load_raw8<DT, !INTER>(p.X, token * p.xt + (h + u) * p.xh, at);
    };
    load(h0);  // the first rows arrive beside the positions
    Turn t;
    if (at.turned) t = turn_of(p.r, token, l, p.backward ? -1.f : 1.f);
    for (int h = h0; h < h1; h += kRopeRows) {
        if (h > h0) load(h);
#pragma unroll
        for (int u = 0; u < kRopeRows; u++) {
            if (h + u < h1) {
                float v[8];
                unpack4(raw[u].a, v);
                unpack4(raw[u].b, v + 4);
                if (at.turned) apply_turn<INTER>(v, v + 4, t);
                store8<DT, !INTER>(p.Y, token * p.yt + (h + u) * p.yh, at, v);
            }
        }
    }
}

cudaError_t launch_rope(const RopePlan &p, cudaStream_t st) {
    const int64_t units = p.n * ((p.heads + kRopeHeads - 1) / kRopeHeads);
    const dim3 grid((unsigned)((units + 15) / 16));
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(256), 0, st, p); };
    if (p.r.interleaved)
        return p.dtype == DT_F32 ? go(k_rope<DT_F32, true>)
               : p.dtype == DT_BF16 ? go(k_rope<DT_BF16, true>) : go(k_rope<DT_F16, true>);
    return p.dtype == DT_F32 ? go(k_rope<DT_F32, false>)
           : p.dtype == DT_BF16 ? go(k_rope<DT_BF16, false>) : go(k_rope<DT_F16, false>);
}

}  // namespace qvg
