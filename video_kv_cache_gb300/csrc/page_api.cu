// C ABI of the paged cache: argument checks and plans of qvg_rope, qvg_page_write,
// qvg_page_read and qvg_page_attention.  Declarations and their contracts are in
// include/qvg.h.
#include <cmath>
#include <limits>

#include "internal.cuh"
#include "qvg.h"

namespace qvg {
namespace {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t elem(int dtype) { return dtype == DT_F32 ? 4 : 2; }
inline bool is_dtype(int dtype) { return dtype >= QVG_F16 && dtype <= QVG_F32; }

// A row stride of an input (may be 0) or an output (at least a row where it is used).
inline bool stride_ok(int64_t stride, int64_t rows, int dtype, bool output) {
    if (stride < 0 || stride > (int64_t(1) << 40) || stride * elem(dtype) % 16 != 0) return false;
    return !output || rows <= 1 || stride >= kD;
}

qvg_status check_rotary(const qvg_rotary *r, int64_t n_tokens) {
    if (r->rot_dim < 8 || r->rot_dim > kD || r->rot_dim % 8 != 0) return QVG_ERR_UNSUPPORTED;
    if (r->interleaved != 0 && r->interleaved != 1) return QVG_ERR_UNSUPPORTED;
    if (r->n_axes < 1 || r->n_axes > 4) return QVG_ERR_UNSUPPORTED;
    int64_t pairs = 0;
    for (int a = 0; a < r->n_axes; a++) {
        if (r->sections[a] < 0) return QVG_ERR_INVALID_ARG;
        pairs += r->sections[a];
    }
    if (pairs != r->rot_dim / 2 || !std::isfinite(r->mscale)) return QVG_ERR_INVALID_ARG;
    if (r->n_axes > 1 && r->pos_stride < n_tokens) return QVG_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!r->positions || !r->freqs)) return QVG_ERR_INVALID_ARG;
    if (!aligned(r->positions, 8) || !aligned(r->freqs, 16)) return QVG_ERR_INVALID_ARG;
    return QVG_OK;
}

Rotary make_rotary(const qvg_rotary *r) {
    Rotary o{};
    if (!r) return o;
    o.rot = r->rot_dim;
    o.interleaved = r->interleaved;
    int end = 0;
    for (int a = 0; a < 3; a++) {
        end += a < r->n_axes ? r->sections[a] : 0;
        o.end[a] = a + 1 < r->n_axes ? end : kD;  // the last axis has no end
    }
    o.mscale = r->mscale;
    o.pos_stride = r->pos_stride;
    o.pos = r->positions;
    o.freqs = r->freqs;
    return o;
}

bool wide_format(int format) { return format == QVG_PAGE_F16 || format == QVG_PAGE_BF16; }

qvg_status check_pool(int32_t n_heads, int32_t d, int32_t page_tokens, int32_t format, int64_t n_pages) {
    if (n_heads < 1 || n_pages < 1) return QVG_ERR_INVALID_ARG;
    if (d != kD || n_heads > 32767) return QVG_ERR_UNSUPPORTED;
    if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64 && page_tokens != 128)
        return QVG_ERR_UNSUPPORTED;
    if (format < QVG_PAGE_F16 || format > QVG_PAGE_INT8) return QVG_ERR_UNSUPPORTED;
    if (n_pages >= (int64_t(1) << 31) || n_pages * n_heads * page_tokens >= (int64_t(1) << 31))
        return QVG_ERR_UNSUPPORTED;
    return QVG_OK;
}

qvg_status check_pages(const qvg_pages *g, int32_t format) {
    if (!g || !g->k || !g->v || !aligned(g->k, 16) || !aligned(g->v, 16)) return QVG_ERR_INVALID_ARG;
    if (!wide_format(format) &&
        (!g->k_scale || !g->v_scale || !aligned(g->k_scale, 16) || !aligned(g->v_scale, 16)))
        return QVG_ERR_INVALID_ARG;
    return QVG_OK;
}

qvg_status check_attention(const qvg_page_attention_params *p) {
    if (!p) return QVG_ERR_INVALID_ARG;
    if (p->n_seqs < 1 || p->n_q_heads < 1 || p->max_pages < 1 || p->total_q < 0 || p->max_q < 0 ||
        p->max_kv < 0 || p->window < 0)
        return QVG_ERR_INVALID_ARG;
    qvg_status rc = check_pool(p->n_heads, p->d, p->page_tokens, p->format, p->n_pages);
    if (rc != QVG_OK) return rc;
    if (p->n_seqs > 65535) return QVG_ERR_UNSUPPORTED;
    if (p->n_q_heads % p->n_heads != 0) return QVG_ERR_INVALID_ARG;
    if (p->n_q_heads / p->n_heads > 128) return QVG_ERR_UNSUPPORTED;
    if (p->q_dtype != QVG_F16 && p->q_dtype != QVG_BF16) return QVG_ERR_UNSUPPORTED;
    if (wide_format(p->format) && (p->format == QVG_PAGE_BF16) != (p->q_dtype == QVG_BF16))
        return QVG_ERR_UNSUPPORTED;
    if (!is_dtype(p->out_dtype)) return QVG_ERR_UNSUPPORTED;
    if (p->causal != 0 && p->causal != 1) return QVG_ERR_UNSUPPORTED;
    if (p->total_q > 0 && p->max_q < 1) return QVG_ERR_INVALID_ARG;
    // rows and the grids that cover them are counted in 32 bits
    if (p->total_q * (int64_t)p->n_q_heads >= (int64_t(1) << 31) ||
        p->max_q * (p->n_q_heads / p->n_heads) >= (int64_t(1) << 26) || p->max_q >= (int64_t(1) << 26))
        return QVG_ERR_UNSUPPORTED;
    if (((p->max_q * (p->n_q_heads / p->n_heads) + 255) / 256) * p->n_heads * (int64_t)p->n_seqs >= (int64_t(1) << 30))
        return QVG_ERR_UNSUPPORTED;
    if (!std::isfinite(p->scale)) return QVG_ERR_INVALID_ARG;
    if (!stride_ok(p->q_token_stride, 0, p->q_dtype, false) || !stride_ok(p->q_head_stride, 0, p->q_dtype, false) ||
        !stride_ok(p->o_token_stride, p->total_q, p->out_dtype, true) ||
        !stride_ok(p->o_head_stride, p->n_q_heads, p->out_dtype, true))
        return QVG_ERR_INVALID_ARG;
    return QVG_OK;
}

PAttnPlan attention_plan(const qvg_page_attention_params *prm) {
    PAttnPlan p{};
    p.B = prm->n_seqs;
    p.HQ = prm->n_q_heads;
    p.H = prm->n_heads;
    p.G = p.HQ / p.H;
    p.g_inv = (uint64_t(1) << 34) / (uint64_t)p.G + 1;
    p.page = prm->page_tokens;
    p.max_pages = prm->max_pages;
    p.fmt = prm->format;
    p.q_dtype = prm->q_dtype;
    p.out_dtype = prm->out_dtype;
    p.causal = prm->causal;
    p.n_pages = prm->n_pages;
    p.window = prm->window;
    p.total_q = prm->total_q;
    p.max_q = std::min(prm->max_q, prm->total_q);
    p.max_kv = std::min(prm->max_kv, (int64_t)prm->max_pages * prm->page_tokens);
    // (a scale of zero keeps a trace, so that -infinity times it stays -infinity)
    p.scale_log2 = prm->scale * 1.4426950408889634f;
    if (std::fabs(p.scale_log2) < std::numeric_limits<float>::min()) p.scale_log2 = std::numeric_limits<float>::min();
    p.qt = prm->q_token_stride;
    p.qh = prm->q_head_stride;
    p.ot = prm->o_token_stride;
    p.oh = prm->o_head_stride;
    if (prm->total_q) page_attention_cut(p);
    return p;
}

// Workspace: the splits' partial rows, then their (maximum, sum) pairs, then the heads' spans.
size_t attention_part_bytes(const PAttnPlan &p) { return (size_t)page_attention_part_rows(p) * kD * sizeof(float); }
size_t attention_bytes(const PAttnPlan &p) {
    return (size_t)page_attention_part_rows(p) * (kD + 2) * sizeof(float) + (p.stream ? (size_t)p.B * p.H * sizeof(int2) : 0);
}

// Checks that come after the arguments': the injected failure, the device.
qvg_status ready() {
    if (fault_inject_launch()) return QVG_ERR_CUDA;
    int num_sms = 0;
    return device_info(&num_sms);
}

qvg_status launched(cudaError_t e) {
    if (e == cudaSuccess) return QVG_OK;
    (void)cudaGetLastError();
    return QVG_ERR_CUDA;
}

}  // namespace
}  // namespace qvg

using namespace qvg;

extern "C" {

qvg_status qvg_rope(const qvg_rope_params *prm, const qvg_rotary *rotary, const void *X, void *Y,
                    void *stream) {
    if (!prm || !rotary) return QVG_ERR_INVALID_ARG;
    if (prm->n_tokens < 0 || prm->n_heads < 1) return QVG_ERR_INVALID_ARG;
    if (prm->d != kD || !is_dtype(prm->dtype)) return QVG_ERR_UNSUPPORTED;
    if (prm->backward != 0 && prm->backward != 1) return QVG_ERR_UNSUPPORTED;
    if (prm->n_tokens * (int64_t)prm->n_heads >= (int64_t(1) << 34) || prm->n_tokens >= (int64_t(1) << 34))
        return QVG_ERR_UNSUPPORTED;
    qvg_status rc = check_rotary(rotary, prm->n_tokens);
    if (rc != QVG_OK) return rc;
    if (!stride_ok(prm->x_token_stride, prm->n_tokens, prm->dtype, false) ||
        !stride_ok(prm->x_head_stride, prm->n_heads, prm->dtype, false) ||
        !stride_ok(prm->y_token_stride, prm->n_tokens, prm->dtype, true) ||
        !stride_ok(prm->y_head_stride, prm->n_heads, prm->dtype, true))
        return QVG_ERR_INVALID_ARG;
    if (prm->n_tokens == 0) return QVG_OK;
    if (!X || !Y || !aligned(X, 16) || !aligned(Y, 16)) return QVG_ERR_INVALID_ARG;
    if ((rc = ready()) != QVG_OK) return rc;
    RopePlan p{};
    p.n = prm->n_tokens;
    p.heads = prm->n_heads;
    p.dtype = prm->dtype;
    p.backward = prm->backward;
    p.xt = prm->x_token_stride;
    p.xh = prm->x_head_stride;
    p.yt = prm->y_token_stride;
    p.yh = prm->y_head_stride;
    p.r = make_rotary(rotary);
    p.X = X;
    p.Y = Y;
    return launched(launch_rope(p, static_cast<cudaStream_t>(stream)));
}

qvg_status qvg_page_write(const qvg_page_write_params *prm, const void *K, const void *V,
                          const int64_t *slots, const qvg_rotary *rotary, const qvg_pages *pages,
                          uint32_t *dev_status, void *stream) {
    if (!prm || prm->n_tokens < 0) return QVG_ERR_INVALID_ARG;
    qvg_status rc = check_pool(prm->n_heads, prm->d, prm->page_tokens, prm->format, prm->n_pages);
    if (rc != QVG_OK) return rc;
    if (!is_dtype(prm->in_dtype)) return QVG_ERR_UNSUPPORTED;
    if (prm->n_tokens * (int64_t)prm->n_heads >= (int64_t(1) << 34) || prm->n_tokens >= (int64_t(1) << 34))
        return QVG_ERR_UNSUPPORTED;
    if (rotary && (rc = check_rotary(rotary, prm->n_tokens)) != QVG_OK) return rc;
    if (!stride_ok(prm->k_token_stride, 0, prm->in_dtype, false) || !stride_ok(prm->k_head_stride, 0, prm->in_dtype, false) ||
        !stride_ok(prm->v_token_stride, 0, prm->in_dtype, false) || !stride_ok(prm->v_head_stride, 0, prm->in_dtype, false))
        return QVG_ERR_INVALID_ARG;
    if ((rc = check_pages(pages, prm->format)) != QVG_OK) return rc;
    if (prm->n_tokens == 0) return QVG_OK;
    if (!K || !V || !slots || !aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 8)) return QVG_ERR_INVALID_ARG;
    if ((rc = ready()) != QVG_OK) return rc;
    PWritePlan p{};
    p.n = prm->n_tokens;
    p.heads = prm->n_heads;
    p.page = prm->page_tokens;
    p.fmt = prm->format;
    p.dtype = prm->in_dtype;
    p.n_pages = prm->n_pages;
    p.kt = prm->k_token_stride;
    p.kh = prm->k_head_stride;
    p.vt = prm->v_token_stride;
    p.vh = prm->v_head_stride;
    p.r = make_rotary(rotary);
    p.K = K;
    p.V = V;
    p.slots = slots;
    p.k = pages->k;
    p.v = pages->v;
    p.ks = pages->k_scale;
    p.vs = pages->v_scale;
    p.status = dev_status;
    return launched(launch_page_write(p, static_cast<cudaStream_t>(stream)));
}

qvg_status qvg_page_read(const qvg_page_read_params *prm, const qvg_pages *pages,
                         const int32_t *page_table, const int32_t *seq_lens, void *X,
                         uint32_t *dev_status, void *stream) {
    if (!prm) return QVG_ERR_INVALID_ARG;
    if (prm->n_seqs < 1 || prm->max_pages < 1 || prm->first < 0 || prm->count < 0) return QVG_ERR_INVALID_ARG;
    qvg_status rc = check_pool(prm->n_heads, prm->d, prm->page_tokens, prm->format, prm->n_pages);
    if (rc != QVG_OK) return rc;
    if (!is_dtype(prm->out_dtype) || prm->n_seqs > 65535) return QVG_ERR_UNSUPPORTED;
    if (prm->first >= (int64_t(1) << 31) || prm->count >= (int64_t(1) << 31)) return QVG_ERR_UNSUPPORTED;
    if (!stride_ok(prm->x_seq_stride, prm->n_seqs, prm->out_dtype, false) ||
        !stride_ok(prm->x_tensor_stride, 2, prm->out_dtype, false) ||
        prm->x_tensor_stride < prm->count * kD || (prm->n_seqs > 1 && prm->x_seq_stride < prm->count * kD))
        return QVG_ERR_INVALID_ARG;
    if ((rc = check_pages(pages, prm->format)) != QVG_OK) return rc;
    if (prm->count == 0) return QVG_OK;
    if (!page_table || !seq_lens || !X || !aligned(X, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4))
        return QVG_ERR_INVALID_ARG;
    if ((rc = ready()) != QVG_OK) return rc;
    PReadPlan p{};
    p.B = prm->n_seqs;
    p.heads = prm->n_heads;
    p.page = prm->page_tokens;
    p.fmt = prm->format;
    p.dtype = prm->out_dtype;
    p.max_pages = prm->max_pages;
    p.n_pages = prm->n_pages;
    p.first = prm->first;
    p.count = prm->count;
    p.xs = prm->x_seq_stride;
    p.xt = prm->x_tensor_stride;
    p.k = pages->k;
    p.v = pages->v;
    p.ks = pages->k_scale;
    p.vs = pages->v_scale;
    p.table = page_table;
    p.lens = seq_lens;
    p.X = X;
    p.status = dev_status;
    return launched(launch_page_read(p, static_cast<cudaStream_t>(stream)));
}

size_t qvg_page_attention_workspace_bytes(const qvg_page_attention_params *prm) {
    if (check_attention(prm) != QVG_OK || prm->total_q == 0) return 0;
    return attention_bytes(attention_plan(prm));
}

qvg_status qvg_page_attention(const qvg_page_attention_params *prm, const void *Q,
                              const qvg_pages *pages, const int32_t *page_table,
                              const int32_t *seq_lens, const int32_t *cu_q, void *O, float *lse,
                              void *workspace, size_t workspace_bytes, uint32_t *dev_status,
                              void *stream) {
    qvg_status rc = check_attention(prm);
    if (rc != QVG_OK) return rc;
    if ((rc = check_pages(pages, prm->format)) != QVG_OK) return rc;
    if (!cu_q && prm->total_q != prm->max_q * prm->n_seqs) return QVG_ERR_INVALID_ARG;
    if (prm->total_q == 0) return QVG_OK;
    if (!Q || !O || !page_table || !seq_lens || !aligned(Q, 16) || !aligned(O, 16) || !aligned(lse, 4) ||
        !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4))
        return QVG_ERR_INVALID_ARG;
    PAttnPlan p = attention_plan(prm);
    const size_t need = attention_bytes(p);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return QVG_ERR_WORKSPACE;
    if ((rc = ready()) != QVG_OK) return rc;
    p.Q = Q;
    p.k = pages->k;
    p.v = pages->v;
    p.ks = pages->k_scale;
    p.vs = pages->v_scale;
    p.table = page_table;
    p.lens = seq_lens;
    p.cu = cu_q;
    p.O = O;
    p.lse = lse;
    p.part = static_cast<float *>(workspace);
    p.ml = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + attention_part_bytes(p));
    p.spans = reinterpret_cast<int2 *>(p.ml + 2 * page_attention_part_rows(p));
    p.status = dev_status;
    return launched(launch_page_attention(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
