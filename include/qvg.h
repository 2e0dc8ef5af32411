/*
 * qvg.h -- C ABI of libqvg, a GB300 (sm_103a) implementation of the KV-cache compression
 * path of Quant VideoGen (arXiv 2602.02958).
 *
 * The method, as the pages state it:
 *   - Semantic-Aware Smoothing ("Quant VideoGen" notes page, section Semantic-Aware
 *     Smoothing; review page "Quant VideoGen: 基于2-Bit KV缓存量化的自回归长视频生成",
 *     pipeline paragraph, steps (a)-(c)): the N tokens of a per-head tensor X in R^{N x d}
 *     are clustered by k-means along the token axis into C groups, and each token has its
 *     group's centroid (the group mean) subtracted.
 *   - Progressive Residual Quantization (notes page, section Progressive Residual
 *     Quantization; review page, pipeline paragraph): with R^(0) = X, stage t = 1..T
 *     re-applies the smoothing to R^(t-1), producing R^(t), centroids C^(t) and
 *     assignments pi^(t); only R^(T) is quantized.
 *   - Q(R^(T)) is symmetric group integer quantization, INT2 or INT4, with one scale per
 *     group stored as FP8 E4M3 (notes page, section Algorithm-System Co-design; explainer
 *     "Quant VideoGen: Auto-Regressive Long Video Generation via 2-Bit KV-Cache
 *     Quantization", section Step-by-step).
 *   - Reconstruction dequantizes and adds the stages' assigned centroids back from stage T
 *     down to stage 1, fused in one pass (notes page, sections Progressive Residual
 *     Quantization and Algorithm-System Co-design).
 *   - Streaming: the previous chunk's centroids initialise the next chunk's k-means
 *     (notes page, section Algorithm-System Co-design).
 *
 * Conventions for every call:
 *   - All data pointers are DEVICE pointers into memory the caller owns and keeps alive
 *     until the work on `stream` has finished.  The library allocates no device memory and
 *     keeps no mutable global state; scratch space is the caller's `workspace`.  The one
 *     exception is qvg_quantize_static, whose scratch is a fixed area inside the library.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream).  Work
 *     is enqueued asynchronously; a call returns once it is enqueued.  qvg_quantize,
 *     qvg_reassign and qvg_dequantize enqueue only kernels and memsets on `stream`, so a
 *     caller may capture them in a CUDA graph and replay it with the same buffers.
 *   - The kernels are launched with programmatic dependent launch: each one may become
 *     resident before the previous kernel on `stream` has finished, and waits for it
 *     (griddepcontrol.wait) before touching memory, so the order of memory effects is plain
 *     stream order.  Each also lets its dependents launch early.  A kernel the caller
 *     launches next with programmatic serialisation allowed must itself wait
 *     (griddepcontrol.wait) before reading the results; one launched without it needs
 *     nothing.
 *   - Argument errors are detected on the host before anything is enqueued and returned as
 *     QVG_ERR_INVALID_ARG / QVG_ERR_UNSUPPORTED / QVG_ERR_WORKSPACE.  A CUDA error reported
 *     while enqueuing returns QVG_ERR_CUDA; work already enqueued may have run.
 *   - Conditions only the device can see are OR-ed into *dev_status (a device uint32, may
 *     be NULL) as QVG_DEV_* bits; read it after synchronising the stream.  No call aborts
 *     the process or traps the device.
 *   - Pointers must be 16-byte aligned.
 *   - Fault injection, for testing a caller's error handling without faulting a GPU (read
 *     from the environment at every call): QVG_FAULT_INJECT=launch makes every call that
 *     would enqueue device work return QVG_ERR_CUDA after its argument checks, with nothing
 *     enqueued; =alloc does the same for qvg_quantize_static alone (its scratch lookup);
 *     =timeout runs qvg_quantize's tensor-core assignments with their centroid operand
 *     withheld and a 1 ms wait limit (as qvg_selftest_assign_timeout does), so the call
 *     returns QVG_OK, the device status gets QVG_DEV_TIMEOUT and the results are
 *     unspecified; =assign makes qvg_quantize's first tensor-core assignment launch fail
 *     after the kernels before it were enqueued, so the call returns QVG_ERR_CUDA from the
 *     middle of its sequence (nothing after the failed launch is enqueued; the outputs are
 *     unspecified).  Unset, or any other value: no effect.
 *
 * Supported shapes: d = 128; group in {16, 32, 64}; bits in {2, 4}; 1 <= C <= 256 and
 * C <= N when T > 0; 0 <= T <= 8; iters >= 1; N >= 1.
 */
#ifndef QVG_H
#define QVG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QVG_OK = 0,
    QVG_ERR_INVALID_ARG = 1, /* NULL / misaligned pointer, negative or inconsistent size */
    QVG_ERR_UNSUPPORTED = 2, /* a value outside the supported shapes listed above */
    QVG_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than qvg_quantize_workspace_bytes */
    QVG_ERR_CUDA = 4,        /* a CUDA runtime call failed while enqueuing (no device, launch) */
    QVG_ERR_DEVICE = 5,      /* the current device is not an sm_103 (GB300-class) GPU */
    QVG_ERR_SCRATCH_LIMIT = 6 /* qvg_quantize_static: the problem needs more scratch than
                                 QVG_STATIC_SCRATCH_BYTES */
} qvg_status;

/* Bits OR-ed into *dev_status by the device. */
#define QVG_DEV_NONFINITE 0x1u /* X held a NaN or an infinity */
#define QVG_DEV_TIMEOUT 0x2u   /* a pipeline wait in a tensor-core kernel gave up */
#define QVG_DEV_BAD_INDEX 0x4u /* a stored cluster index was >= C (it was clamped to C-1), or a
                                  slot, page or length out of range */
#define QVG_DEV_NO_PAGES 0x8u  /* a sequence did not get the pages that it asked for */

typedef enum { QVG_F16 = 0, QVG_BF16 = 1, QVG_F32 = 2 } qvg_dtype;

/* Parameters of one qvg_quantize call: n_tensors independent tensors of N tokens each. */
/* Integer grid of the codes.
 *   QVG_QSCHEME_SYMMETRIC: q in [-qmax, qmax], qmax = 2^(bits-1) - 1 (INT2 is ternary);
 *     s = max|r| / qmax; q = r / s_q rounded half to even and clamped; u = q + 2^(bits-1);
 *     x = s_q * (u - 2^(bits-1)).
 *   QVG_QSCHEME_MIDRISE: the 2^bits levels sit at half-integers (4 levels at INT2, the
 *     reading of one critique page of the method); s = max|r| / (2^(bits-1) - 1/2);
 *     u = floor(r / s_q) + 2^(bits-1) clamped to [0, 2^bits - 1] (a value exactly between
 *     two levels takes the upper one); x = s_q * (u - 2^(bits-1) + 1/2).
 * Either way s_q = E4M3(s) and s_q = 0 stores every code as 2^(bits-1). */
typedef enum { QVG_QSCHEME_SYMMETRIC = 0, QVG_QSCHEME_MIDRISE = 1 } qvg_qscheme;

/* Value format of the stored centroids.  The tables stay float arrays; with a 16-bit format
 * every stored value is exactly representable in it, so a consumer may narrow the tables
 * without loss, and residuals, codes and reconstruction all use those rounded values.
 *   QVG_CENTROIDS_F32:  the fp32 mean (the default).
 *   QVG_CENTROIDS_F16:  IEEE binary16; QVG_CENTROIDS_BF16: bfloat16.  The cluster mean, a
 *     cold-start row and a warm-start value are each rounded once to nearest even in the
 *     format.  The mean is carried to about twice fp32's precision, so it rounds as the
 *     exact mean of the stage's inputs does (from the second stage on, the exact residuals
 *     against the stored earlier centroids), save within about 2^-38 of the members' size
 *     of a tie.
 * Quant VideoGen explainer page, compression and metadata overhead: the ratios it prints
 * count centroids in a 16-bit format. */
typedef enum { QVG_CENTROIDS_F32 = 0, QVG_CENTROIDS_F16 = 1, QVG_CENTROIDS_BF16 = 2 }
    qvg_centroid_format;

typedef struct {
    int32_t n_tensors;      /* H >= 1: independent (layer, head, K/V) tensors in this call */
    int32_t d;              /* channels per token; must be 128 */
    int64_t N;              /* tokens per tensor in this call */
    int32_t C;              /* clusters per stage */
    int32_t T;              /* smoothing stages (0 = plain group quantization) */
    int32_t bits;           /* 2 or 4 */
    int32_t group;          /* channels per scale group: 16, 32 or 64 */
    int32_t iters;          /* Lloyd rounds (assign + mean update) per stage */
    int32_t in_dtype;       /* qvg_dtype of X */
    uint64_t seed;          /* cold-start seed */
    int64_t tensor_id_base; /* tensor h of this call uses id tensor_id_base + h for seeding */
    int64_t x_stride;       /* elements between consecutive tensors of X (0 = N*d) */
    int64_t token_offset;   /* first token slot written in codes / scales / pi */
    int64_t token_capacity; /* token slots per tensor in codes / scales / pi (0 = N) */
    int32_t table_index;    /* centroid-table slot written by this call */
    int32_t n_tables;       /* centroid-table slots per tensor (0 = 1) */
    int64_t warm_stride;    /* floats between consecutive tensors of warm_centroids
                               (0 = T*C*d) */
    int32_t qscheme;        /* qvg_qscheme of the codes (zero-initialised = symmetric) */
    int32_t centroid_format; /* qvg_centroid_format of the stored centroids (0 = fp32) */
} qvg_quant_params;

/* The compressed cache.  Layouts (all row-major, caller-owned device memory):
 *   codes     uint8 [H][token_capacity][d*bits/8]  channel k of a token sits at bits
 *             (k*bits) mod 8 of byte (k*bits)/8 of its row; stored code u = q + 2^(bits-1)
 *   scales    uint8 [H][token_capacity][d/group]   FP8 E4M3 bit patterns
 *   pi        uint8 [H][T][token_capacity]         cluster index per stage and token
 *   centroids float [H][n_tables][T][C][d]         one table per chunk of tokens
 * For T = 0, pi and centroids are not touched and may be NULL. */
typedef struct {
    uint8_t *codes;
    uint8_t *scales;
    uint8_t *pi;
    float *centroids;
} qvg_buffers;

/* Bytes of device scratch qvg_quantize needs for these parameters (0 if they are invalid).
 * Depends only on n_tensors, N, C, T. */
size_t qvg_quantize_workspace_bytes(const qvg_quant_params *params);

/* Compress X: T smoothing stages of `iters` Lloyd rounds each, then group quantization of
 * the last residual.  Writes codes/scales for tokens [token_offset, token_offset + N),
 * pi^(1..T) for the same slots, and C^(1..T) into table slot table_index.
 *   X               [H][N][d] of in_dtype, tensor h at X + h*x_stride elements
 *   warm_centroids  NULL for a cold start (seeded distinct rows of R^(t-1) as the initial
 *                   centroids of stage t), or fp32 [H][T][C][d] (tensor stride warm_stride)
 *                   used as stage t's initial centroids -- the streaming warm start.  It
 *                   may point into out->centroids (another table slot than table_index).
 *   workspace       >= qvg_quantize_workspace_bytes(params) bytes, 256-byte aligned; its
 *                   contents on entry do not matter.  Once the call's work has finished,
 *                   its first two uint32 words count, over all stages and Lloyd rounds, the
 *                   token rows whose nearest centroid the tensor-core scores could not
 *                   settle and the candidate clusters re-scored exactly for them.
 * Calls that share a workspace must be ordered on one stream. */
qvg_status qvg_quantize(const qvg_quant_params *params, const void *X,
                        const float *warm_centroids, const qvg_buffers *out, void *workspace,
                        size_t workspace_bytes, uint32_t *dev_status, void *stream);

/* Size of the fixed scratch area behind qvg_quantize_static: 64 MiB per device.  The area is
 * part of libqvg's device code, so it is reserved on every device (in every CUDA context)
 * where that code is loaded -- whichever entry points the process calls, qvg_quantize,
 * qvg_dequantize and qvg_attention included.  A caller sizing a KV pool to the last
 * megabyte should count it. */
#define QVG_STATIC_SCRATCH_BYTES ((size_t)64 << 20)

/* qvg_quantize without a workspace argument, for callers that cannot allocate.
 *
 * The paper has no counterpart to this call: it is a convenience of this library.  It
 * runs the same kernels as qvg_quantize and gives the same results, but takes its scratch
 * from one area of QVG_STATIC_SCRATCH_BYTES compiled into the library (a separate copy on
 * each device) instead of from the caller, and allocates nothing itself: no cudaMalloc or
 * cudaFree, no allocating library, no host heap.
 *
 * Who needs it: a caller that may not or cannot allocate device memory at the moment it
 * compresses -- a server that has handed all free memory to its KV pool or to a caching
 * allocator, a latency-bound loop in which cudaMalloc / cudaFree (which can synchronise
 * the device) would stall the other streams, or a plain C host with no allocator of its
 * own.
 *
 * Limit: qvg_quantize_workspace_bytes(params) must not exceed QVG_STATIC_SCRATCH_BYTES;
 * otherwise the call returns QVG_ERR_SCRATCH_LIMIT before touching the device.  The
 * scratch is about 450 bytes per token row plus about 630 KB per tensor, whatever T: one
 * tensor of up to about 148 000 tokens fits, 24 tensors of up to about 4 800 each (116 000
 * rows), 100 tensors of up to about 250 each.
 *
 * First call in a context: the area's device address belongs to the CUDA context whose
 * copy of the library's device code holds it, so the first call made while a given context
 * is current (a device's primary context, or one the caller created and made current) looks
 * it up once (cudaGetSymbolAddress, which can load the library's device code in that
 * context); if that fails the call returns QVG_ERR_CUDA.  Make this first call before any
 * stream capture begins in that context.  Later calls in the same context reuse the
 * address.  After cudaDeviceReset, or once a context is destroyed, the address kept for it
 * is stale: do not call this function again in that process.
 *
 * Contents on entry do not matter: everything the path needs to start at zero is cleared
 * by the call itself, on `stream`, before it is used.
 *
 * Races: all calls on one device share the one area.  Two calls whose device work can
 * overlap -- on different streams with no event ordering them, e.g. from different host
 * threads -- overwrite each other's scratch and both results are wrong.  Issue them on
 * one stream, or order them with events.
 *
 * Arguments other than the workspace, layouts and the other errors are those of
 * qvg_quantize. */
qvg_status qvg_quantize_static(const qvg_quant_params *params, const void *X,
                               const float *warm_centroids, const qvg_buffers *out,
                               uint32_t *dev_status, void *stream);

/* Assign every token's stage-T residual R^(T-1) to its nearest centroid of C^(T) as stored
 * in out->centroids (table slot table_index), writing pi^(T).  This is one assignment step
 * of the Lloyd iteration (notes page, section Semantic-Aware Smoothing, step 1), run on the
 * state a preceding qvg_quantize call with the same params, X, out and workspace left
 * behind: the residual planes of stage T stay in the workspace.  It lets the tensor-core
 * assignment be timed and checked on its own.  Requires T >= 1.  The codes and scales
 * are not updated. */
qvg_status qvg_reassign(const qvg_quant_params *params, const void *X, const qvg_buffers *out,
                        void *workspace, size_t workspace_bytes, uint32_t *dev_status,
                        void *stream);

/* The steps of qvg_reassign, for timing them one at a time: */
#define QVG_STEP_PLANES 1 /* the centroids' GEMM operands (fp16 plane, offsets, norms) */
#define QVG_STEP_GEMM 2   /* the tensor-core GEMM with its fused argmax epilogue: pi^(T)
                             for every row with one candidate, the lowest candidate and a
                             re-scoring request for the others */
#define QVG_STEP_REFINE 4 /* the exact re-scoring of the requested rows */
/* qvg_reassign with only the steps in the `steps` mask.  Each step reads what the earlier
 * ones wrote in the workspace: run them in order, on one stream (the GEMM after the planes
 * of the same centroids, the re-scoring after the GEMM).  A re-scoring step whose queue no
 * GEMM step wrote (a fresh workspace) reads no request outside the queue's capacity: it
 * skips what is out of range and ORs QVG_DEV_BAD_INDEX into *dev_status.
 * QVG_ERR_INVALID_ARG for other bits; otherwise as qvg_reassign. */
qvg_status qvg_reassign_steps(const qvg_quant_params *params, const void *X,
                              const qvg_buffers *out, void *workspace, size_t workspace_bytes,
                              int32_t steps, uint32_t *dev_status, void *stream);

/* Self-test of the assignment kernel's failure handling; no step of the method.  It runs the
 * tensor-core assignment of qvg_reassign once with the load of the centroid operand withheld
 * and a wait limit of one millisecond (2 s in normal calls), so that the kernel's first wait
 * on that operand never completes: the wait gives up, the kernel ORs QVG_DEV_TIMEOUT into
 * *dev_status, waits for the copies it did issue, frees its tensor memory and returns.  The
 * device stays usable, and later calls run normally.  Arguments as for qvg_reassign; pi^(T)
 * is left unspecified.  The device is never faulted or trapped. */
qvg_status qvg_selftest_assign_timeout(const qvg_quant_params *params, const void *X,
                                       const qvg_buffers *out, void *workspace,
                                       size_t workspace_bytes, uint32_t *dev_status,
                                       void *stream);

/* Parameters of one qvg_dequantize call. */
typedef struct {
    int32_t n_tensors;      /* H */
    int32_t d;              /* 128 */
    int64_t N;              /* tokens to reconstruct per tensor, slots [0, N) */
    int32_t C, T, bits, group;
    int32_t out_dtype;      /* qvg_dtype of X_hat */
    int64_t chunk_len;      /* tokens per centroid table: slot i uses table i / chunk_len
                               (0 = N, one table) */
    int64_t token_capacity; /* token slots per tensor in codes / scales / pi (0 = N) */
    int32_t n_tables;       /* centroid-table slots per tensor (0 = 1) */
    int64_t out_stride;     /* elements between consecutive tensors of X_hat (0 = N*d) */
    int32_t qscheme;        /* qvg_qscheme the codes were written with */
} qvg_dequant_params;

/* Reconstruct X_hat[h][i] = x(u) + C^(T)[pi^(T)_i] + ... + C^(1)[pi^(1)_i], x(u) the level
 * of the code's scheme, added in that order (stage T first) in fp32 registers, rounded
 * once to out_dtype. */
qvg_status qvg_dequantize(const qvg_dequant_params *params, const qvg_buffers *in,
                          void *X_hat, uint32_t *dev_status, void *stream);

/* Parameters of one qvg_attention call. */
typedef struct {
    int32_t n_heads;        /* H: 1 .. 65535 */
    int32_t d;              /* 128 */
    int32_t M;              /* queries per head: 1 .. 16 */
    int64_t N;              /* keys per head: cache slots [0, N) */
    int32_t C, T, bits, group, qscheme;  /* of both caches, as they were quantized */
    int64_t chunk_len;      /* tokens per centroid table (0 = N), as in qvg_dequant_params */
    int64_t token_capacity; /* token slots per tensor of both caches (0 = N) */
    int32_t n_tables;       /* centroid-table slots per tensor (0 = 1) */
    int32_t q_dtype;        /* qvg_dtype of Q */
    int32_t out_dtype;      /* qvg_dtype of O */
    float scale;            /* multiplies q.k before the softmax, e.g. 1/sqrt(d); finite */
    int64_t k_first;        /* head h reads key tensor k_first + h * tensor_step of k_cache */
    int64_t v_first;        /* and value tensor v_first + h * tensor_step of v_cache */
    int64_t tensor_step;    /* >= 0; keys and values interleaved in one cache: pass it as
                               both caches with k_first 0, v_first 1, tensor_step 2 */
} qvg_attention_params;

/* Workspace bytes qvg_attention needs for these parameters (0 if they are invalid). */
size_t qvg_attention_workspace_bytes(const qvg_attention_params *params);

/* Softmax attention read straight from the compressed cache.  For head h and query m:
 *   O[h][m] = sum_j p_j v_j,  p = softmax over j < N of (scale * Q[h][m] . k_j),
 * where k_j and v_j are token j of the head's key and value tensors rebuilt exactly as
 * qvg_dequantize writes them in fp32.  The rebuilt rows stay in registers and shared
 * memory; nothing of size N x d is written (the notes page's fused reconstruction,
 * section Algorithm-System Co-design, feeding attention on the fly).
 * Layouts: Q [H][M][d] of q_dtype, O [H][M][d] of out_dtype, both contiguous and 16-byte
 * aligned; the caches as qvg_buffers describes.  Scores, softmax and sums are fp32, the
 * output rounded once to out_dtype.  Tensor indices are not checked against the caches'
 * sizes: the caller guarantees them.  A cluster index >= C is clamped and reported as
 * QVG_DEV_BAD_INDEX. */
qvg_status qvg_attention(const qvg_attention_params *params, const void *Q,
                         const qvg_buffers *k_cache, const qvg_buffers *v_cache, void *O,
                         void *workspace, size_t workspace_bytes, uint32_t *dev_status,
                         void *stream);

/* ------------------------------------------------------------------------------------
 * A paged cache of recent tokens.
 *
 * qvg_quantize compresses whole chunks of tokens.  The tokens of the chunk that is still
 * growing, and any that are to stay uncompressed, live in pages: qvg_rope turns queries (and
 * gradients) by their positions, qvg_page_write stores new keys (turned on the way if asked)
 * and values in 16 or 8 bits, qvg_page_attention lets the new tokens attend to the pages,
 * qvg_page_read gives rows back in the layout qvg_quantize takes.
 *
 * A page holds page_tokens consecutive tokens of one sequence, all heads.  Arrays
 * (row-major, caller-owned device memory, 16-byte aligned):
 *   k, v              [n_pages][n_heads][page_tokens][128] of the page format
 *   k_scale, v_scale  float [n_pages][n_heads][page_tokens], 8-bit and 4-bit formats only
 *   k_group, v_group  4-bit formats only, see there
 * A slot is page * page_tokens + row.  Token t of sequence b is row t % page_tokens of page
 * page_table[b][t / page_tokens]; page_table is int32 [n_seqs][max_pages], and entries that
 * no token below the sequence's length falls in are never read.
 * page_tokens: 16, 32, 64 or 128.
 * ------------------------------------------------------------------------------------ */

/* Page formats.  The 16-bit ones hold the value rounded to nearest even.  The 8-bit ones hold
 * codes and one scale per (token, head, key or value): with a = max_k |x_k| over the row,
 *   E4M3: s = a / 448, code = E4M3(x * (448 / a)), to nearest even;
 *   INT8: s = a / 127, code = rint(x * (127 / a)),
 * in fp32, and the stored value is s * code.  A row with a < 2^-100 is stored as zeros
 * (s = 0); a row that holds a NaN or an infinity gets s = NaN, so that it reads as NaN, and
 * QVG_DEV_NONFINITE is reported. */
typedef enum {
    QVG_PAGE_F16 = 0,
    QVG_PAGE_BF16 = 1,
    QVG_PAGE_E4M3 = 2,
    QVG_PAGE_INT8 = 3,
    QVG_PAGE_E2M1 = 8, /* 4 to 7 are refused */
    QVG_PAGE_INT4 = 9
} qvg_page_format;

/* The 4-bit formats hold codes of 4 bits (E2M1: sign, two bits of exponent, one of mantissa,
 * largest code 6; INT4: two's complement, largest 7), a scale for each group of 16 channels
 * and one for the row.  With a as above, a_g = max_k |x_k| over a group and TOP the largest code:
 *   s = a / (64 TOP) in fp32,  t_g = E4M3(64 a_g / a), at most 64,
 *   code = x * 64 TOP / (a t_g) rounded to the format, to nearest even, at most TOP,
 * and the stored value is s * t_g * code.  From 16-bit rows that are not turned the codes and group
 * scales are exactly these: values halfway between two codes go to the even one.  From fp32 rows and
 * turned keys the quotients are worked out in fp32, within 2^-21 of them, so that a value that near to a
 * halfway one may go to either code (and a group's scale likewise).  Rows of zeros, tiny rows and rows
 * that are not finite as in 8 bits.
 *   k, v              two codes a byte, channel 2i in the low four bits: [..][64] bytes
 *   k_group, v_group  E4M3 [n_pages][n_heads][page_tokens][8], group g channels 16g .. 16g + 15
 * Group scales that a caller writes itself may be any E4M3 number up to 64 in magnitude, or NaN; larger
 * ones, and codes of -8, which qvg_page_write does not store, leave the attention over rows that see them
 * unspecified (qvg_page_read gives what they stand for). */
typedef struct {
    void *k;
    void *v;
    float *k_scale; /* NULL for the 16-bit formats */
    float *v_scale;
    uint8_t *k_group; /* read for the 4-bit formats only */
    uint8_t *v_group;
} qvg_pages;

/* Rotary positions.  Pair p of a row, 0 <= p < rot_dim / 2, is turned by the angle
 * 2 pi * positions[axis(p)][token] * freqs[p] / 2^64 and multiplied by mscale; channels from
 * rot_dim on stay as they are.  Pair p is channels (2p, 2p + 1) when interleaved, else
 * (p, p + rot_dim / 2).  Axis a owns the next sections[a] pairs.
 * freqs[p] is the pair's turns per position as a 64-bit fraction, round(f * 2^64) mod 2^64:
 * the product with an integer position wraps exactly, so far positions lose nothing. */
typedef struct {
    int32_t rot_dim;     /* a multiple of 8, 8 .. 128 */
    int32_t interleaved; /* 0 or 1 */
    int32_t n_axes;      /* 1 .. 4 */
    int32_t sections[4]; /* pairs of each axis; they add up to rot_dim / 2 */
    float mscale;        /* finite */
    int64_t pos_stride;  /* elements between the axes' rows of positions */
    const int64_t *positions; /* [n_axes][n_tokens], 8-byte aligned */
    const uint64_t *freqs;    /* [rot_dim / 2] */
} qvg_rotary;

/* Strides in elements; a row's 128 channels are contiguous, and row starts are 16-byte
 * aligned.  An input stride may be 0 (one row for every head, say). */
typedef struct {
    int64_t n_tokens; /* >= 0; 0 enqueues nothing */
    int32_t n_heads;
    int32_t d;        /* 128 */
    int32_t dtype;    /* qvg_dtype of X and Y */
    int32_t backward; /* 0: Y = R X.  1: Y = R^T X, the gradient of X given that of Y (the
                         angles negated, mscale kept) */
    int64_t x_token_stride, x_head_stride;
    int64_t y_token_stride, y_head_stride;
} qvg_rope_params;

/* Turn X [n_tokens][n_heads][128] into Y.  In place when Y is X with the same strides;
 * otherwise the two may not overlap.  fp32 arithmetic, one rounding to dtype. */
qvg_status qvg_rope(const qvg_rope_params *params, const qvg_rotary *rotary, const void *X,
                    void *Y, void *stream);

typedef struct {
    int64_t n_tokens;    /* >= 0; 0 enqueues nothing */
    int32_t n_heads;     /* key/value heads */
    int32_t d;           /* 128 */
    int32_t page_tokens;
    int32_t format;      /* qvg_page_format */
    int64_t n_pages;     /* n_pages * n_heads * page_tokens < 2^31 */
    int32_t in_dtype;    /* qvg_dtype of K and V */
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
} qvg_page_write_params;

/* Store K and V [n_tokens][n_heads][128] at slots[token] (int64, 8-byte aligned, one slot at
 * most once).  A negative slot skips its token; one past the pool is skipped and reported as
 * QVG_DEV_BAD_INDEX.  rotary: NULL, or the turn that keys (not values) get in fp32 before
 * they are rounded. */
qvg_status qvg_page_write(const qvg_page_write_params *params, const void *K, const void *V,
                          const int64_t *slots, const qvg_rotary *rotary, const qvg_pages *pages,
                          uint32_t *dev_status, void *stream);

typedef struct {
    int32_t n_seqs;
    int32_t n_heads;
    int32_t d;           /* 128 */
    int32_t page_tokens;
    int32_t format;
    int32_t out_dtype;   /* qvg_dtype of X */
    int64_t n_pages;
    int32_t max_pages;   /* entries of a page-table row */
    int64_t first;       /* tokens [first, first + count) of every sequence are read */
    int64_t count;       /* >= 0; 0 enqueues nothing */
    int64_t x_seq_stride, x_tensor_stride; /* elements of X between sequences / tensors */
} qvg_page_read_params;

/* Give tokens back as X [n_seqs][2 * n_heads][count][128]: head h's keys in tensor 2h, its
 * values in tensor 2h + 1 (one sequence is then an X of qvg_quantize).  Rows at and past a
 * sequence's length (seq_lens int32 [n_seqs]) are zeros.  A page-table entry outside the pool
 * gives zeros and QVG_DEV_BAD_INDEX; a length past the table is cut to it and reported so. */
qvg_status qvg_page_read(const qvg_page_read_params *params, const qvg_pages *pages,
                         const int32_t *page_table, const int32_t *seq_lens, void *X,
                         uint32_t *dev_status, void *stream);

typedef struct {
    int32_t n_seqs;
    int32_t n_q_heads;   /* a multiple of n_heads: query heads h * g .. h * g + g - 1, with
                            g = n_q_heads / n_heads <= 128, share key/value head h */
    int32_t n_heads;
    int32_t d;           /* 128 */
    int32_t page_tokens;
    int32_t format;      /* QVG_PAGE_F16 with fp16 queries, QVG_PAGE_BF16 with bf16 queries,
                            or an 8-bit or 4-bit format */
    int32_t q_dtype;     /* QVG_F16 or QVG_BF16 */
    int32_t out_dtype;   /* qvg_dtype of O */
    int64_t n_pages;
    int32_t max_pages;   /* entries of a page-table row */
    int32_t causal;      /* 1: a query sees keys up to its own position; 0: every key */
    int64_t window;      /* > 0: only the last `window` positions up to the query's own (and,
                            unless causal, all after it); 0: no limit */
    int64_t total_q;     /* query tokens of all sequences; 0 enqueues nothing */
    int64_t max_q;       /* no sequence has more query tokens */
    int64_t max_kv;      /* about the longest sequence: sizes the split of the work only */
    float scale;         /* multiplies q.k before the softmax; finite */
    int64_t q_token_stride, q_head_stride;
    int64_t o_token_stride, o_head_stride;
} qvg_page_attention_params;

/* Workspace bytes qvg_page_attention needs (0 if the parameters are invalid, or none is). */
size_t qvg_page_attention_workspace_bytes(const qvg_page_attention_params *params);

/* Softmax attention of new tokens over the pages.  Sequence b has seq_lens[b] cached tokens,
 * the last q_len of which are its queries' own: query i sits at position
 * seq_lens[b] - q_len + i.  cu_q (int32 [n_seqs + 1], NULL: max_q queries each) holds where
 * each sequence's queries start among the rows of Q [total_q][n_q_heads][128].
 *   O_i = sum_j p_j v_j,  p = softmax over the keys j that i sees of scale * (q_i . k_j)
 *   lse_i = log sum_j exp(scale * (q_i . k_j))    (lse: float [total_q][n_q_heads] or NULL)
 * A query that sees no key gets O = 0 and lse = -infinity.  What a query does not see cannot
 * change its row, NaN, infinities, E4M3 codes and group scales that are NaN included, nor may a scale that it
 * does not see cost it more than the roundings below.  Values that are not finite leave lse as
 * the scores give it.
 * Scores, softmax and sums are fp32.  The weights p enter the product with the values in
 * 16 bits, relative to a running maximum: in q_dtype, or for the 8-bit and 4-bit formats in fp16, after
 * the value's scale is multiplied in (a relative 2^-11 each, or 2^-25 of the largest value that
 * the query sees); O is rounded once to out_dtype.  Over 8-bit pages, with more than 16 query
 * rows (tokens x grouped heads) a key/value head, a bf16 output and no lse, keys and values are
 * multiplied by their scales and rounded to fp16 instead (a relative 2^-11 each, or 2^-30 and
 * 2^-25 of the largest key and value that the query sees).  4-bit pages are like 8-bit ones in all of
 * this, with a group's scale times a code, which is exact, in the place of the code; where scales are
 * multiplied in, the product of the row's and the group's is rounded to fp16 too (2^-10 in all).
 * Out-of-range page-table entries (read as page 0), lengths past the table (cut), and cu_q
 * out of order, past total_q or with more than max_q queries (cut; the rows left out are
 * not written) are reported as QVG_DEV_BAD_INDEX; a wait in a kernel's pipeline that gives
 * up is reported as QVG_DEV_TIMEOUT, the rows concerned unspecified. */
qvg_status qvg_page_attention(const qvg_page_attention_params *params, const void *Q,
                              const qvg_pages *pages, const int32_t *page_table,
                              const int32_t *seq_lens, const int32_t *cu_q, void *O, float *lse,
                              void *workspace, size_t workspace_bytes, uint32_t *dev_status,
                              void *stream);

/* ------------------------------------------------------------------------------------
 * Pages of sequences.  refs (int32 [n_pages]) counts, for each page, the entries of the page table
 * that name it; 0 is free.  A sequence of n tokens holds the first ceil(n / page_tokens) entries of its
 * row; what the others hold is not read.  qvg_page_append gives sequences the pages of new tokens,
 * qvg_page_fork lets one begin as a copy of another, sharing its whole pages, qvg_page_free gives
 * pages back, qvg_page_compact moves what is live into another pool, qvg_page_copy copies single pages.
 * They change refs, page_table and seq_lens on the device, in stream order, and need no word from the
 * host about what is free.  Pages are always taken in ascending order, for sequences in order, so that
 * the outcome is the same in every run.
 *
 * Several layers with a cache each and one page table: qvg_page_append and qvg_page_fork copy pages of
 * the one cache that they are given and leave what they copied in `copies`, with whose first three
 * rows qvg_page_copy does the same in another layer's cache; qvg_page_compact moves the same pages for every cache.
 * ------------------------------------------------------------------------------------ */
typedef struct {
    int32_t n_seqs;      /* rows of the page table: 1 .. 65535 */
    int32_t n_heads;
    int32_t d;           /* 128 */
    int32_t page_tokens;
    int32_t format;
    int32_t max_pages;   /* entries of a page-table row, at most 2^27 / page_tokens */
    int64_t n_pages;
    int64_t total;       /* qvg_page_append: entries of slots and positions, < 2^31 */
    int64_t out_pages;   /* qvg_page_compact: pages of the other pool */
    int64_t *starts;     /* device int64 [n_seqs], or NULL (0 for every sequence): the position of the
                            token that is each sequence's first now.  qvg_page_free moves it on,
                            qvg_page_fork copies it, qvg_page_append counts from it */
} qvg_page_table_params;

/* Workspace bytes that qvg_page_append and qvg_page_fork need (out_pages 0), or qvg_page_compact does;
 * 0 if none is needed, or the parameters are invalid.  The first two need none for up to
 * QVG_FEW_SEQS sequences. */
#define QVG_FEW_SEQS 1024
size_t qvg_page_table_workspace_bytes(const qvg_page_table_params *params);

/* Page src[i]'s rows [0, rows[i]) (all with rows NULL), of every head, keys and values, with their
 * scales, to page dst[i] of `to`, a pool of the same heads, page_tokens and format, which may be
 * `pages` itself; the rows behind stay as they were.  src, dst, rows: int32 [n].  A negative src or dst
 * skips its copy; one past its pool skips it, and rows out of range are cut, with QVG_DEV_BAD_INDEX.  No
 * page may be a destination twice, nor in one pool both a destination and a source. */
qvg_status qvg_page_copy(const qvg_page_table_params *params, int64_t n, const qvg_pages *pages,
                         const int32_t *src, const int32_t *dst, const int32_t *rows,
                         const qvg_pages *to, int64_t to_pages, uint32_t *dev_status, void *stream);

/* Sequence b grows by counts[b] tokens (int32 [n_seqs], 0: none): seq_lens and the page table are
 * brought up to date, and slots and positions (int64 [total]) of the new tokens are written, sequence
 * after sequence, as qvg_page_write and qvg_rope take them; entries behind the last token are -1.
 * A token's position is its place in the sequence plus starts[b].  Without starts it is the place alone,
 * which is no position to turn by once qvg_page_free has dropped first tokens: what is kept was turned by
 * positions that lie as many tokens further on.
 * A last page that is part filled and that other entries name too (refs > 1) is first replaced by a copy
 * of its rows in use; copies (int32 [3][n_seqs], or NULL) gets source, destination and rows of it, -1, -1, 0
 * where there is none.
 * A sequence whose pages, with those of the sequences before it, are more than the free ones, or
 * that would pass its row of the table, stays as it is, with QVG_DEV_NO_PAGES and -1 for its tokens (a
 * sequence that needs no page grows all the same); so does one that counts or lengths out of range, more
 * tokens than total, or a part-filled last page that is out of the pool or free keep from it, with
 * QVG_DEV_BAD_INDEX. */
qvg_status qvg_page_append(const qvg_page_table_params *params, const qvg_pages *pages, int32_t *refs,
                           int32_t *page_table, int32_t *seq_lens, const int32_t *counts,
                           int64_t *slots, int64_t *positions, int32_t *copies, void *workspace,
                           size_t workspace_bytes, uint32_t *dev_status, void *stream);

/* Sequence b, which has to be empty, becomes a fork of sequence parents[b] (int32 [n_seqs], negative:
 * none): the parent's whole pages are shared, its last one, if part filled, is copied as far as it
 * is filled, starts[b] becomes the parent's.  copies (int32 [4][n_seqs]) gets source, destination and rows of that copy, -1, -1, 0 where
 * there is none, and the whole pages shared, -1 where there is no fork.  A parent may have many forks in a call but be none itself.
 * Sequences that are not empty, and parents that are not valid or whose part-filled last page is out
 * of the pool or free, are left out with QVG_DEV_BAD_INDEX (whole pages out of the pool are shared as the
 * entries that they are, with QVG_DEV_BAD_INDEX), those for which free pages do not suffice (as above) with QVG_DEV_NO_PAGES. */
qvg_status qvg_page_fork(const qvg_page_table_params *params, const qvg_pages *pages, int32_t *refs,
                         int32_t *page_table, int32_t *seq_lens, const int32_t *parents,
                         int32_t *copies, void *workspace, size_t workspace_bytes,
                         uint32_t *dev_status, void *stream);

/* Sequence b gives up its first drop_first[b] tokens, as far as they fill whole pages, and its last
 * drop_last[b] (int32 [n_seqs] each, one of them may be NULL; anything past the length means all of it).  The
 * entries that stay move to the front of the row, the ones behind them become -1, and the length
 * is what is left.  Pages that no entry names any more are free.  starts[b] grows by the first tokens
 * given up (one whose tokens were all first ones goes on where it was); it becomes 0 for a sequence
 * that drop_last leaves without tokens, which has ended.  Negative counts are 0, entries out of the
 * pool or of free pages are dropped, lengths past the table cut (of sequences that give up nothing
 * too), with QVG_DEV_BAD_INDEX. */
qvg_status qvg_page_free(const qvg_page_table_params *params, int32_t *refs, int32_t *page_table,
                         int32_t *seq_lens, const int32_t *drop_first, const int32_t *drop_last,
                         uint32_t *dev_status, void *stream);

/* Pages in use (refs > 0), in ascending order, become pages 0, 1, ... of `to`, another pool of
 * params->out_pages pages; out_table ([n_seqs][max_pages], -1 behind each sequence's entries) and out_refs
 * ([out_pages]) are the page table and the counts for it, *live the number of pages in use.  The first
 * pool, page_table and refs stay as they are, so nothing that is written may share memory with them
 * (arrays of the pools, the tables and the counts that do are refused).  What out_pages has no room
 * for is left out, its entries -1, with QVG_DEV_NO_PAGES; entries out of the pool or of free pages
 * become -1 with QVG_DEV_BAD_INDEX. */
qvg_status qvg_page_compact(const qvg_page_table_params *params, const qvg_pages *pages,
                            const int32_t *refs, const int32_t *page_table, const int32_t *seq_lens,
                            const qvg_pages *to, int32_t *out_table, int32_t *out_refs, int32_t *live,
                            void *workspace, size_t workspace_bytes, uint32_t *dev_status,
                            void *stream);

/* Static description of a status code. */
const char *qvg_status_string(qvg_status status);

/* Library version, (major << 16) | minor.
 *   1.0  quantize, reassign, dequantize, the static-scratch quantize.
 *   1.1  qvg_quant_params.qscheme and .centroid_format, qvg_dequant_params.qscheme (both
 *        structs grew: rebuild callers), qvg_attention.  The paged cache (qvg_rope,
 *        qvg_page_*) came later without a change to what 1.1 had, and later still its 4-bit
 *        formats (qvg_pages grew by two pointers that the others do not read) and the calls on
 *        the pages of sequences (whose qvg_page_table_params then grew by starts: rebuild callers). */
uint32_t qvg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QVG_H */
