/*
 * qvg.h -- C ABI of libqvg: 2-bit / 4-bit compression of an autoregressive
 * video model's KV cache (Quant VideoGen, "QVG" / "QVG-Pro") with the QuantWM
 * extensions (QSAC, PSAC), and attention that reads the compressed cache
 * directly.  One GPU (NVIDIA GB300, sm_103a).
 *
 * Sources cited below by page title and section:
 *   [QVG]  Quant VideoGen: Auto-Regressive Long Video Generation via 2-Bit
 *          KV-Cache Quantization (papernotes.org notes, ICML 2026).
 *   [P1]   The 2-bit quantisation trap in video generation (cloud.baidu.com).
 *   [QWM]  QuantWM write-up (loncent.com): QSAC and PSAC.
 *   [P2]   Temporally stable 2-bit KV-cache compression for video world models, in practice (hmyw.cn): section 3.3 (temporal anchors), section 3.4
 *          (outlier separation).
 *
 * Conventions for every call:
 *   - Buffers are device pointers owned by the caller unless stated; the
 *     library never allocates device memory and never frees caller memory.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *     default stream).  Only qvg_get_status synchronises.
 *   - Every call returns a qvg_status.  Argument errors are found on the
 *     host before anything is launched and leave all buffers untouched.
 *     A failed launch returns QVG_ERR_CUDA.  Errors found on the device
 *     (an exceeded wait bound; in the token-wise operators also values in
 *     device arrays that are out of range: slots, pages, lengths, parents)
 *     are latched in a per-device status word and reported by
 *     qvg_get_status(stream).
 *   - bf16 / fp16 values travel as their 16-bit patterns (uint16_t).
 *   - Layouts are row-major; "[a][b][c]" lists dimensions outermost first.
 *   - Thread safety: calls on different streams, from any host threads, may
 *     run concurrently as long as they do not write the same buffers.  Each
 *     call works on the device current on its host thread.  Library state:
 *     the per-device error word, the no-alloc scratch
 *     (qvg_compress_chunk_noalloc), and per-device launch set-up tables
 *     (each kernel's shared-memory limit, the SM count, the error word's
 *     address), each entry made once per device by the first call that
 *     needs it and published atomically, so first calls may race and one
 *     process may drive several devices.  Per host thread: the last CUDA
 *     error (qvg_last_cuda_error) and the wait settings of
 *     qvg_debug_set_wait.
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
    QVG_ERR_INVALID_ARG = 1, /* a pointer, size or layout argument is wrong   */
    QVG_ERR_UNSUPPORTED = 2, /* valid, but outside what the kernels implement  */
    QVG_ERR_CUDA = 3,        /* a CUDA launch or runtime call failed           */
    QVG_ERR_TIMEOUT = 4,     /* a device-side wait exceeded its bound          */
    QVG_ERR_WORKSPACE = 5,   /* workspace missing or smaller than required     */
    QVG_ERR_CAPACITY = 6     /* the cache has no room for another chunk        */
} qvg_status;

/* qvg_params.flags */
#define QVG_QSAC 1            /* weight the clustering distance by qsac_w        */
#define QVG_PSAC 2            /* store the rank-8 key-error projection            */
#define QVG_GIVEN_CENTROIDS 4 /* start k-means from centroids the caller wrote   */
                              /* into this chunk's centroid slot                 */
#define QVG_OUTLIER 8         /* outlier split in the residual quantiser: per    */
                              /* group, a value above the group's P99 is kept   */
                              /* in fp16 (G <= 64; see outl_val below)           */
#define QVG_KEEP_MEANS 16     /* qvg_compress_chunk leaves each stage's fp32     */
                              /* centroid means in the workspace (see there)     */

#define QVG_TILE 128      /* chunks start at multiples of this many token slots */
#define QVG_PSAC_RANK 8   /* PSAC subspace rank ([QWM] PSAC: top-8 directions)  */
#define QVG_MAX_CLUSTERS 256
#define QVG_CACHE_NBUF 14

/* Output element types of qvg_decompress / qvg_attention. */
#define QVG_OUT_F32 0
#define QVG_OUT_BF16 1

/*
 * Method parameters ([QVG] "training strategy": the hyperparameters are the
 * cluster count C, the residual stage count L and the bit width b; the group
 * size G is that of the per-group quantiser, [P1] section 2 and [QVG]
 * "core tension").
 *   C          clusters per (chunk, head, stage), 0..256; 0 = plain per-group
 *              quantisation without centroid (the RTN baseline of [QVG]
 *              "main results").  C > N clusters a chunk of N tokens with N.
 *   L          progressive residual stages, >= 1 ([QVG] "Progressive
 *              Residual Quantization").  L = 1 is QVG, L > 1 QVG-Pro.
 *   bits       2 or 4.
 *   group      G: channels per quantisation group; head_dim % G == 0,
 *              G >= head_dim / 32.
 *   iters      Lloyd iterations (assign + update) before the final assign.
 *   scale_mode 0: S = max|r| / (2^{b-1} - 1)  ([QVG] "core tension");
 *              1: S = max|r| / 2, codes in [-2, 1]  ([P1] section 2; bits = 2).
 *   flags      QVG_QSAC | QVG_PSAC | QVG_GIVEN_CENTROIDS | QVG_OUTLIER |
 *              QVG_KEEP_MEANS.
 *   anchor_every  temporal anchors ([P2] section 3.3: the first frames of
 *              each window are kept at high precision so that errors do not
 *              pile up from window to window): 0 = none; k > 0 = chunk c of
 *              a cache (0-based) with c % k == 0 is stored as its bf16 K/V
 *              in the cache's anchor arena instead of being compressed.
 *   seed       k-means initialisation seed.
 * A cache must always be used with the C, L, bits and group it was sized for.
 */
typedef struct {
    int32_t C;
    int32_t L;
    int32_t bits;
    int32_t group;
    int32_t iters;
    int32_t scale_mode;
    int32_t flags;
    int32_t anchor_every;
    uint64_t seed;
} qvg_params;

/*
 * One compressed tensor (K or V) of one layer: an arena of token slots that
 * grows chunk by chunk ([QVG] "overall framework": the cache is processed
 * chunk by chunk; [P1] section 1: the cache grows linearly with frames).
 * Every buffer is caller-allocated device memory of the size that
 * qvg_cache_bytes reports, 16-byte aligned (the kernels read it with vector
 * loads; a misaligned buffer is refused with QVG_ERR_INVALID_ARG before any
 * launch).  Chunks start at slot multiples of QVG_TILE; the
 * slots between a chunk's end and the next multiple are padding.
 *   codes      uint8 [L][H][capacity][d*bits/8]  packed offset-binary codes:
 *              element j of a row at bits (j*bits)%8 of byte (j*bits)/8,
 *              value q + 2^{bits-1} ([QVG] "algorithm-system co-design":
 *              packed INT representation).
 *   scales     fp16  [L][H][capacity][d/G]       per-group scales.
 *   ids        uint8 [L][H][capacity]            cluster of each token.
 *   cent       bf16  [L][H][max_chunks][C][d]    centroids ([QVG] "overall
 *              framework": centroids kept in BF16).
 *   chunk_start int32 [max_chunks]  first slot of each chunk.
 *   chunk_len   int32 [max_chunks]  tokens in each chunk.
 *   tile_chunk  int32 [capacity/QVG_TILE] chunk owning each slot tile.
 *   psac_p     int8  [H][capacity][8]  PSAC projection codes (K only, or NULL).
 *   psac_s     fp16  [H][capacity]     PSAC per-token scales (or NULL).
 *   psac_basis fp32  [max_chunks][H][d][8] basis each chunk was encoded with
 *              (or NULL).
 *   outl_val   fp16  [L][H][capacity][d/G]  outlier split ([P2] section 3.4,
 *              "outlier separation"; with QVG_OUTLIER, else NULL): per group
 *              of a stage's residual, the value above the group's 99th
 *              percentile of |r| (linear interpolation; for G <= 100 at most
 *              the largest), fp16, saturated at 65504.  The group's scale and
 *              codes come from the other values; the outlier's code is 0 and
 *              it is rebuilt as outl_val + centroid.
 *   outl_idx   uint8 [L][H][capacity][d/G]  its channel within the group,
 *              0xFF when no value lies above the percentile (0 in outl_val).
 *   anchor     bf16  [A][H][d]  anchor chunks' K or V as given (with
 *              anchor_every > 0, else NULL).  Anchor chunk c starts at row
 *              (c / anchor_every) * S, S = capacity / max_chunks rounded up
 *              to QVG_TILE, and A = ceil(max_chunks / anchor_every) * S; an
 *              anchor chunk longer than S is refused (QVG_ERR_CAPACITY).  Its
 *              token slots in the other buffers are reserved but unused.
 *   chunk_anchor int32 [max_chunks]  first anchor row of each chunk, -1 for
 *              a compressed chunk (with anchor_every > 0, else NULL).
 * n_chunks and n_tokens are host-side counters that qvg_compress_chunk
 * advances; set both to 0 for an empty cache.  A cache can be saved and
 * restored by copying its buffers and these two counters.
 */
typedef struct {
    int32_t H;
    int32_t d;
    int32_t capacity_tokens; /* multiple of QVG_TILE */
    int32_t max_chunks;
    int32_t n_chunks;
    int32_t n_tokens;        /* first free slot (a multiple of QVG_TILE) */
    uint8_t *codes;
    uint16_t *scales;
    uint8_t *ids;
    uint16_t *cent;
    int32_t *chunk_start;
    int32_t *chunk_len;
    int32_t *tile_chunk;
    int8_t *psac_p;
    uint16_t *psac_s;
    float *psac_basis;
    uint16_t *outl_val;
    uint8_t *outl_idx;
    uint16_t *anchor;
    int32_t *chunk_anchor;
} qvg_cache;

/* Text for a status code (static storage; never NULL). */
const char *qvg_status_string(qvg_status s);

/*
 * Bytes of each cache buffer, in the order codes, scales, ids, cent,
 * chunk_start, chunk_len, tile_chunk, psac_p, psac_s, psac_basis, outl_val,
 * outl_idx, anchor, chunk_anchor (out_sizes has QVG_CACHE_NBUF entries).
 * The PSAC entries are 0 unless p->flags has QVG_PSAC, the outlier entries
 * 0 unless QVG_OUTLIER, the anchor entries 0 unless p->anchor_every > 0.  capacity_tokens must be a positive multiple of
 * QVG_TILE.  The total is the compressed footprint; [P1] section 1 gives
 * the uncompressed one, 2 (K and V) x layers x heads x head_dim x tokens x
 * bytes per element.
 */
qvg_status qvg_cache_bytes(const qvg_params *p, int32_t H, int32_t d,
                           int32_t capacity_tokens, int32_t max_chunks,
                           size_t out_sizes[QVG_CACHE_NBUF]);

/* Operations for qvg_workspace_size. */
#define QVG_OP_COMPRESS 0
#define QVG_OP_ATTENTION 1
#define QVG_OP_PSAC_BASIS 2

/*
 * Scratch bytes an operation needs for a chunk of n tokens (compress) or n
 * queries (attention), H KV heads, head_dim d and Hq query heads.  The
 * caller allocates it (256-byte aligned) and passes it to the call; its
 * contents need no initialisation and are dead after the call completes.
 * For attention it is 0 when n queries already fill the GPU (the cache is
 * then not split) and otherwise enough for the largest split the current
 * device's SM count can call for.
 */
qvg_status qvg_workspace_size(const qvg_params *p, int32_t op, int32_t n,
                              int32_t H, int32_t d, int32_t Hq, size_t *bytes);

/*
 * Compress one chunk of N new tokens and append it to `cache`
 * ([QVG] "overall framework", "Semantic-Aware Smoothing", "Progressive
 * Residual Quantization"; [QWM] QSAC and PSAC).  For each KV head and each
 * stage l = 1..L:
 *   k-means over the chunk's tokens: seeded init, p->iters Lloyd iterations,
 *   one final assignment (distance sum_j w_j (x_j - c_j)^2, w = qsac_w with
 *   QVG_QSAC, else 1; ties to the lowest cluster);
 *   residual r = X_l - C_id; per-group quantisation of r with fp16 scales
 *   (with QVG_OUTLIER, first splitting off each group's value above its
 *   P99 into the fp16 side list, [P2] section 3.4);
 *   X_{l+1} = X_l - (S q + C_id).
 * With QVG_PSAC, the remaining key error E = X_{L+1} is projected on the
 * rank-8 basis and stored as INT8 per token with one fp16 scale.
 * With p->anchor_every = k > 0, chunk n_chunks is an anchor when
 * n_chunks % k == 0 ([P2] section 3.3): its bf16 K or V is copied into the
 * anchor arena as given, and nothing else is computed for it.
 *   x_bf16     bf16 [N][H][d] device, the chunk's K or V (token-major),
 *              16-byte aligned.
 *   N          1 .. 65535 tokens.
 *   qsac_w     fp32 [H][d] device per-channel weights (required with QVG_QSAC,
 *              else ignored); positive and finite.
 *   psac_basis fp32 [H][d][8] device, 16-byte aligned (required with
 *              QVG_PSAC, else ignored); copied into the cache's per-chunk
 *              basis slot.
 *   cache      appended in place: the chunk occupies slots
 *              [n_tokens, n_tokens + N); n_chunks += 1 and n_tokens advances to
 *              the next multiple of QVG_TILE.  With QVG_GIVEN_CENTROIDS the
 *              caller has written all L stages' starting centroids into the
 *              new chunk's centroid slot (index n_chunks).
 *   workspace  device scratch of at least qvg_workspace_size(QVG_OP_COMPRESS).
 *              With QVG_KEEP_MEANS (and C > 0, iters >= 1) its first
 *              L*H*C*d*4 bytes hold, after the call, fp32 [L][H][C][d]: each
 *              stage's centroids of its last Lloyd update before the bf16
 *              rounding (the member mean in fp32; an empty cluster's kept
 *              centroid), for checking the update against a reference.
 * Returns QVG_ERR_CAPACITY when the chunk does not fit, in the slots or (an
 * anchor chunk) in its anchor rows; nothing is written then.
 */
qvg_status qvg_compress_chunk(const qvg_params *p, const void *x_bf16,
                              int32_t N, const float *qsac_w,
                              const float *psac_basis, qvg_cache *cache,
                              void *workspace, size_t ws_bytes, void *stream);

/*
 * Size of the fixed device scratch behind qvg_compress_chunk_noalloc: 32 MiB,
 * reserved on every device that loads the library, until the process exits.
 */
#define QVG_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * qvg_compress_chunk without a caller workspace (the pages have no
 * counterpart: this serves callers that cannot allocate device memory, such
 * as code inside a framework whose memory pool owns the whole device and
 * forbids further cudaMalloc calls, or code that must not risk the
 * device-wide synchronisation of cudaMalloc / cudaFree).  Same arguments,
 * results and errors as qvg_compress_chunk, which it calls; the workspace is
 * a fixed scratch array of QVG_NOALLOC_SCRATCH_BYTES inside the library.
 *   - Checks its arguments and the cache's capacity first, in the order
 *     and with the codes of qvg_compress_chunk; then returns
 *     QVG_ERR_WORKSPACE, before anything is launched, when
 *     qvg_workspace_size(QVG_OP_COMPRESS) for this call exceeds the scratch
 *     (for example L > 1 or PSAC on large chunks: use qvg_compress_chunk).
 *   - The first call on a device, made with that device current, looks up
 *     the scratch's device address (cudaGetSymbolAddress); make that first
 *     call before any stream capture.  It allocates nothing, ever.
 *   - Every call on a device shares the one scratch array, which keeps the
 *     last call's contents; nothing in it needs to start at zero.  Calls
 *     whose work overlaps on the GPU (different streams, or different host
 *     threads without ordering) race on the scratch: order them.
 */
qvg_status qvg_compress_chunk_noalloc(const qvg_params *p, const void *x_bf16,
                                      int32_t N, const float *qsac_w,
                                      const float *psac_basis, qvg_cache *cache,
                                      void *stream);

/*
 * Rebuild ntok token slots starting at slot tok0 ([QVG] "overall
 * framework": X_hat = S_X * X_INT + C_i, summed over stages per
 * "Progressive Residual Quantization"; with PSAC data present, plus the
 * correction P_hat U^T of [QWM] PSAC).  Stages are summed in fp32 in stage
 * order.  With QVG_OUTLIER, a value split off from its group is rebuilt as
 * its fp16 copy plus the centroid ([P2] section 3.4); an anchor chunk's
 * slots give its stored bf16 K/V ([P2] section 3.3).
 *   out      [ntok][H][d] fp32 or bf16 (out_dtype), 4-byte aligned (16-byte
 *            for fp32 and 8-byte for bf16 take vector stores); the caller's
 *            device buffer.  Padding slots give 0.
 * Errors: QVG_ERR_INVALID_ARG for tok0 < 0, ntok < 0, tok0 + ntok past
 * n_tokens or a misaligned out; ntok = 0 does nothing.
 */
qvg_status qvg_decompress(const qvg_params *p, const qvg_cache *cache,
                          int32_t tok0, int32_t ntok, void *out,
                          int32_t out_dtype, void *stream);

/*
 * Attention of Nq query tokens over every token in the compressed K and V
 * caches, reading codes, scales, ids and centroids directly and never
 * writing a reconstructed K or V to memory ([QVG] "algorithm-system
 * co-design": dequantisation fused with attention):
 *   O = softmax(scale * Q K_hat^T) V_hat, K_hat including the PSAC
 *   correction when the K cache holds PSAC data.
 *   q_bf16   bf16 [Nq][Hq][d], 16-byte aligned; query head hq reads KV head
 *            hq / (Hq / H).
 *   scale    softmax scale; <= 0 selects 1/sqrt(d).
 *   out      [Nq][Hq][d] fp32 or bf16, 16-byte aligned.
 *   lse      fp32 [Hq][Nq] natural-log log-sum-exp of the scaled logits, or NULL.
 *   top1     int32 [Hq][Nq] slot of the largest logit (lowest on ties), or NULL.
 *   workspace, ws_bytes  optional device scratch (256-byte aligned).  When
 *            ceil(Nq / 256) * Hq work units cannot occupy every SM (a few
 *            queries, as in decoding), a workspace of at least
 *            qvg_workspace_size(QVG_OP_ATTENTION, Nq, H, d, Hq) lets the call
 *            split the cache over more CTAs: each split writes its
 *            normalised fp32 output, log-sum-exp and best logit there, and a
 *            second kernel merges them (weights e^{lse_split - max}).  With no
 *            workspace, or a smaller one, the call runs unsplit; the results
 *            agree within fp32 rounding of the merge.
 * No mask: every cached token precedes the queries.  k and v must hold the
 * same chunks.  Errors: QVG_ERR_INVALID_ARG for a misaligned q_bf16 or out
 * (Nq > 0), QVG_ERR_WORKSPACE for a misaligned workspace.
 */
qvg_status qvg_attention(const qvg_params *p, const void *q_bf16, int32_t Nq,
                         int32_t Hq, const qvg_cache *k, const qvg_cache *v,
                         float scale, void *out, int32_t out_dtype, float *lse,
                         int32_t *top1, void *workspace, size_t ws_bytes,
                         void *stream);

/*
 * Attention of one autoregressive step: the Nq queries of the chunk being
 * generated attend to every token of the compressed cache (the earlier
 * chunks) and to the chunk's own n_cur tokens, whose K/V are still raw bf16
 * ([QVG] research background: chunk-by-chunk generation in which each chunk
 * attends to the cached K/V of the chunks before it; within a chunk there is
 * no mask).  The keys are the concatenation [K_hat ; K_cur] and the values
 * [V_hat ; V_cur], in one softmax:
 *   O = softmax(scale * Q [K_hat ; K_cur]^T) [V_hat ; V_cur].
 *   k_cur_bf16, v_cur_bf16  bf16 [n_cur][H][d], 16-byte aligned (the layout
 *            qvg_compress_chunk takes, so the same buffers are compressed
 *            into the cache after the step); read only, owned by the caller.
 *   n_cur    >= 0; 0 gives qvg_attention.  The cache may be empty (first
 *            chunk) when n_cur > 0.
 *   top1     current-chunk token j is reported as slot k->n_tokens + j, the
 *            slot it takes once the chunk is compressed into this cache.
 * The other arguments, the workspace rule and the outputs are those of
 * qvg_attention.  The raw rows are rounded to fp16 for the tensor core like
 * the reconstructed ones (exact inside fp16's normal range).
 * Errors: QVG_ERR_INVALID_ARG for n_cur < 0, a missing or misaligned raw
 * buffer, or no keys at all.
 */
qvg_status qvg_attention_ar(const qvg_params *p, const void *q_bf16, int32_t Nq,
                            int32_t Hq, const qvg_cache *k, const qvg_cache *v,
                            const void *k_cur_bf16, const void *v_cur_bf16,
                            int32_t n_cur, float scale, void *out,
                            int32_t out_dtype, float *lse, int32_t *top1,
                            void *workspace, size_t ws_bytes, void *stream);

/*
 * History-query statistics ([QWM] QSAC: per-channel activity of history
 * queries; PSAC: their second-moment matrix).  For KV head h, the query
 * heads hq with hq / (Hq/H) == h are pooled:
 *   M[h] (+)= sum over the n tokens and those heads of q q^T   fp32 [H][d][d]
 *   count (+)= n * Hq / H                                      int64 [1]
 *   w[h][j] = M[h][j][j] / count  (mean q_j^2, the QSAC weight) fp32 [H][d]
 * accumulate = 0 overwrites M and count, 1 adds to them.
 */
qvg_status quantwm_query_stats(const void *q_hist_bf16, int32_t n, int32_t Hq,
                               int32_t H, int32_t d, int32_t accumulate,
                               float *M, float *w, int64_t *count,
                               void *stream);

/*
 * PSAC basis ([QWM] PSAC: eigendecomposition of the history-query second
 * moment, top-8 eigenvectors as the principal subspace).  Jacobi
 * eigendecomposition of M[h] / count per head; outputs sorted by eigenvalue,
 * descending, each vector's largest-magnitude component made positive:
 *   U        fp32 [H][d][rank]  column k = k-th eigenvector
 *   eigvals  fp32 [H][rank]     eigenvalues of M / count
 *   energy_frac fp32 [H]        sum of the top-rank eigenvalues / trace
 * rank must be QVG_PSAC_RANK; d is 64 or 128.
 */
qvg_status quantwm_psac_basis(const float *M, const int64_t *count, int32_t H,
                              int32_t d, int32_t rank, float *U,
                              float *eigvals, float *energy_frac,
                              void *stream);

/*
 * Name of the CUDA error behind the latest QVG_ERR_CUDA returned to the
 * calling host thread ("cudaSuccess" if none); static storage.
 */
const char *qvg_last_cuda_error(void);

/*
 * Synchronise with `stream` (NULL: with the whole current device), then
 * return and clear the current device's latched device-side error (QVG_OK
 * if none).  The word is per device, so an error raised by work on another
 * stream that has completed is reported too; work still running elsewhere
 * may latch one after the read.  Returns QVG_ERR_CUDA when the
 * synchronisation reports a CUDA error.
 */
qvg_status qvg_get_status(void *stream);

/*
 * Device-side waits, a test hook for the failure path (the pages have no
 * counterpart).  Every wait of a kernel on a barrier (the k-means
 * assignment's tile and MMA hand-offs, the attention pipelines') is bounded;
 * when the bound runs out the kernel stops its work, waits at the default
 * bound for the tensor-core work it has issued, frees its tensor memory,
 * latches QVG_ERR_TIMEOUT in the device word and returns, leaving the
 * context usable.  This call sets, for the kernels that the calling host
 * thread launches afterwards:
 *   limit_ns  the bound of those waits in nanoseconds; 0 restores the
 *             default of 2 s.
 *   inject    1: each such kernel additionally waits once on a barrier that
 *             nothing completes, with tensor-core work in flight, so that
 *             the bound runs out (qvg_get_status then reports
 *             QVG_ERR_TIMEOUT and the call's outputs are undefined);
 *             0: no such wait.
 * Errors: QVG_ERR_INVALID_ARG for inject other than 0 or 1.
 */
qvg_status qvg_debug_set_wait(uint64_t limit_ns, int32_t inject);

/* ======================================================================
 * Token-wise operators: rotary positions, a paged cache that is written one
 * token at a time, and attention of a few new tokens over it.
 *
 * A chunk is compressed (above) once it is complete.  The tokens of the
 * chunk being generated, and any history whose tokens arrive one by one or
 * as a drafted tree, live in a paged cache instead: fp8 or fp4 codes with
 * power-of-two scales, which need nothing but the token's own row.  The
 * pages have no counterpart for this part; its formulas stand here.
 * ====================================================================== */

/* qvg_rope_plan.layout */
#define QVG_ROPE_HALF 0        /* pair i = channels i and i + dims / 2           */
#define QVG_ROPE_INTERLEAVED 1 /* pair i = channels 2 i and 2 i + 1              */
/* `scaling` of qvg_rope_plan_init, for contexts longer than the trained one. */
#define QVG_ROPE_PLAIN 0
#define QVG_ROPE_LINEAR 1 /* positions divided by `factor`                       */
#define QVG_ROPE_NTK 2    /* base * factor^(n / (n - 2)), n = the axis' channels */
#define QVG_ROPE_PARTS 3  /* fast pairs kept, slow pairs divided (see below)     */

#define QVG_ROPE_MAX_PAIRS 64
#define QVG_ROPE_MAX_AXES 4

/*
 * Rotary positions of one model: a host structure that qvg_rope_plan_init
 * fills and every call takes by pointer (its contents travel with the
 * launch; nothing is allocated, and the structure may be copied, saved, or
 * changed after the call).
 *   step   what one position adds to pair i's angle, in units of 2^-64 turns.
 *          A position times a step, modulo 2^64, is the angle's fraction of
 *          a turn to 2^-64 with no rounding, at any int32 position.
 *   axis   the position axis that pair i follows.
 */
typedef struct {
    int32_t dims;  /* rotated channels: the first `dims` of each head */
    int32_t axes;  /* positions per token                             */
    int32_t layout;
    float mscale;  /* factor on the rotated channels                  */
    uint64_t step[QVG_ROPE_MAX_PAIRS];
    uint8_t axis[QVG_ROPE_MAX_PAIRS];
} qvg_rope_plan;

/*
 * Fill a plan.  Axis a owns axis_dims[a] channels, i.e. axis_dims[a] / 2
 * consecutive pairs; the axes follow one another, and dims is their sum (one
 * axis: text; frame, row and column: video).  Pair i of an axis with n
 * channels turns by f_i = base^(-2 i / n) radians per position, and
 *   QVG_ROPE_LINEAR: f_i / factor;
 *   QVG_ROPE_NTK:    f_i with base * factor^(n / (n - 2)) (n = 2: base);
 *   QVG_ROPE_PARTS:  f_i (k + (1 - k) / factor), with r = original f_i / 2 pi
 *                    the turns of the pair over the trained context of
 *                    `original` positions and k = (r - slow) / (fast - slow)
 *                    clamped to [0, 1];
 * scaled_axes: bit a set = axis a is scaled (others stay plain).
 * Errors: QVG_ERR_INVALID_ARG for axes outside 1 .. QVG_ROPE_MAX_AXES, an
 * odd, zero or negative axis_dims, more than QVG_ROPE_MAX_PAIRS pairs, an
 * unknown layout or scaling, a base or factor that is not finite or below 1,
 * a non-finite mscale; with QVG_ROPE_PARTS original <= 0 or fast <= slow.
 */
qvg_status qvg_rope_plan_init(qvg_rope_plan *plan, int32_t axes, const int32_t *axis_dims, int32_t layout,
                              double base, int32_t scaling, double factor, double original, double fast,
                              double slow, uint32_t scaled_axes, float mscale);

/*
 * Rotate n tokens' heads: pair (a, b) at angle t becomes
 *   mscale (a cos t - b sin t, b cos t + a sin t);
 * channels from `dims` on are copied.  In fp32, rounded once to the type.
 *   x          [n][H][d] of `dtype` (QVG_OUT_F32 or QVG_OUT_BF16), d = 64 or
 *              128; token t starts at element t * x_stride (>= H d).
 *   positions  int32 [n][axes] device.
 *   transpose  1: the angles' signs turned -- the gradient of this call with
 *              respect to x (and, where mscale is 1, its inverse).
 *   out        as x, with out_stride.  out may be x itself when the strides
 *              are equal; otherwise they must not overlap.
 * Errors: QVG_ERR_INVALID_ARG for a bad plan (dims over d, an axis out of
 * range), n < 0, H < 1, a stride below H d, an unknown dtype, x, out or
 * positions missing or not aligned to their elements; QVG_ERR_UNSUPPORTED
 * for another d.  n = 0 does nothing.
 */
qvg_status qvg_rope(const qvg_rope_plan *plan, const void *x, int32_t dtype, int32_t n, int32_t H, int32_t d,
                    int64_t x_stride, const int32_t *positions, int32_t transpose, void *out, int64_t out_stride,
                    void *stream);

/*
 * A paged token cache (K and V of one layer): num_pages pages of page_size
 * token slots; slot s is token s % page_size of page s / page_size.  Which
 * page holds what is the caller's business (a block table, below).
 *   bits 8: codes are fp8 numbers (e4m3: 4 exponent bits, 3 mantissa bits,
 *           largest 448), one scale per token and head;
 *   bits 4: codes are fp4 numbers (e2m1: 0 0.5 1 1.5 2 3 4 6 and their
 *           negatives), channel 2 i in the low half of byte i, one scale per
 *           token, head and 32 consecutive channels.
 *   k_codes, v_codes    uint8 [num_pages][H][page_size][d * bits / 8]
 *   k_scales, v_scales  uint8 [num_pages][H][page_size][G], G = 1 (8 bits) or
 *                       d / 32: a scale of 2^(byte - 127), the smallest with
 *                       which no value of the group exceeds the largest code
 *                       (at least byte 1); 255 marks a row (token and head)
 *                       that held an infinity or a NaN: its codes are 0, its
 *                       scales all 255, and its values read as NaN.
 * A power-of-two scale makes each step exact but the rounding to the code
 * (nearest, ties to even): a value is off by at most 2^-4 of itself (8 bits)
 * or a quarter of it (4 bits), or half the smallest step, and reading it back
 * into bf16 adds nothing.  (A value within the last step below 2^128 takes the
 * code below it, so that every finite value stays finite.)
 * All four buffers are caller-allocated, 16-byte aligned device memory of the
 * size that qvg_paged_bytes reports, and share no byte.  H >= 1, d = 64 or
 * 128, page_size 16, 32, 64, 128 or 256.
 */
typedef struct {
    int32_t H;
    int32_t d;
    int32_t page_size;
    int32_t num_pages;
    int32_t bits;
    uint8_t *k_codes;
    uint8_t *k_scales;
    uint8_t *v_codes;
    uint8_t *v_scales;
} qvg_paged;

/* Bytes of a codes buffer and of a scales buffer (K's and V's are alike). */
qvg_status qvg_paged_bytes(int32_t H, int32_t d, int32_t page_size, int32_t num_pages, int32_t bits,
                           size_t *codes, size_t *scales);

/*
 * Quantise n tokens into their slots.
 *   k, v       bf16 [n][H][d], 16-byte aligned; token t starts at element
 *              t * k_stride (t * v_stride), a multiple of 8 and >= H d.
 *   slots      int64 [n] device.  A negative slot skips its token; the
 *              others must differ from one another (a slot given twice ends
 *              up with parts of both tokens).
 *   plan       NULL, or rotary positions that K gets on the way: the rotated
 *              row is rounded to bf16 and then quantised, as if qvg_rope had
 *              written it.  positions int32 [n][axes] device.
 * A slot at or beyond num_pages * page_size is skipped and latches
 * QVG_ERR_INVALID_ARG in the device's status word (qvg_get_status).
 * Nothing but the tokens' slots is written.
 * Errors: QVG_ERR_INVALID_ARG for a bad cache or plan, n < 0, missing or
 * misaligned pointers, bad strides; QVG_ERR_UNSUPPORTED for another d.
 */
qvg_status qvg_paged_append(const qvg_paged *cache, const void *k_bf16, const void *v_bf16, int32_t n,
                            int64_t k_stride, int64_t v_stride, const int64_t *slots, const qvg_rope_plan *plan,
                            const int32_t *positions, void *stream);

/*
 * Read n slots back: k_out, v_out [n][H][d] fp32 or bf16 (out_dtype), 16-byte
 * aligned; either may be NULL.  Exact in both types.  A negative slot gives
 * zeros; a slot beyond the cache gives zeros and latches QVG_ERR_INVALID_ARG.
 */
qvg_status qvg_paged_read(const qvg_paged *cache, const int64_t *slots, int32_t n, void *k_out, void *v_out,
                          int32_t out_dtype, void *stream);

/* mask_mode of qvg_paged_attention */
#define QVG_MASK_NONE 0   /* every token of the sequence                          */
#define QVG_MASK_CAUSAL 1 /* new token t sees the history and new tokens 0 .. t   */
#define QVG_MASK_TREE 2   /* the history and the new tokens its mask row names    */

/*
 * Mask rows of drafted trees: row t of a sequence has the bits of t itself
 * and of all its ancestors.
 *   parents  int32 [total_q] device: the parent's number within the
 *            sequence's new tokens, which is below the token's own, or -1
 *            (the token follows the history).  Another value latches
 *            QVG_ERR_INVALID_ARG and counts as -1.
 *   cu_q     int32 [B + 1] device: sequence b's new tokens are rows
 *            cu_q[b] .. cu_q[b + 1] - 1; NULL: max_q rows each.  A sequence
 *            of more than max_q, or with rows outside total_q, latches
 *            QVG_ERR_INVALID_ARG; rows past its max_q, or all of its rows,
 *            are left as they were.
 *   total_q  rows of parents and mask.
 *   mask     uint32 [total_q][words] device, words >= ceil(max_q / 32);
 *            bit j % 32 of word j / 32 is new token j.  Every word of the
 *            rows cu_q[0] .. cu_q[B] - 1 is written.
 * Errors: QVG_ERR_INVALID_ARG for B < 0, max_q < 0, total_q < 0 or (without
 * cu_q) below B * max_q, too few words, missing or misaligned pointers;
 * QVG_ERR_UNSUPPORTED for max_q > 8192.
 */
qvg_status qvg_tree_mask(const int32_t *parents, const int32_t *cu_q, int32_t B, int32_t max_q, int32_t total_q,
                         int32_t words, uint32_t *mask, void *stream);

/*
 * Scratch bytes of qvg_paged_attention on the current device (256-byte
 * aligned; no initialisation needed, dead after the call).
 */
qvg_status qvg_paged_workspace_size(int32_t H, int32_t d, int32_t Hq, int32_t B, int32_t max_q, size_t *bytes);

/*
 * Attention of B sequences' new tokens over their pages: one token each
 * (decoding), a drafted tree, or the tokens of a chunk.  The new tokens' K
 * and V have been appended: they are the last tokens of the sequence.  With
 * L = kv_len[b] tokens and T new ones, key j < L - T is history and key
 * L - T + i is new token i (T > L: the first T - L have none); new token t
 * sees what mask_mode says, and
 *   O = softmax(scale * Q K^T) V   over the keys it sees.
 *   q          bf16 [total_q][Hq][d], 16-byte aligned; token t starts at
 *              element t * q_stride (a multiple of 8, >= Hq d).  Query head
 *              hq reads KV head hq / (Hq / H).
 *   cu_q       int32 [B + 1] device, ascending from 0: first row of each
 *              sequence's new tokens; NULL: max_q rows each.  Rows from
 *              cu_q[B] on are neither read nor written.
 *   max_q      at least the largest T.  A longer sequence latches
 *              QVG_ERR_INVALID_ARG: its tokens beyond max_q are left out, and
 *              what the others get is undefined.
 *   table      int32 [B][table_stride] device: page of tokens
 *              p * page_size .. of sequence b.  Entries past the sequence's
 *              last page are not read.
 *   kv_len     int32 [B] device, the new tokens included; 0: no keys.  A
 *              sequence longer than its table row or than 2^31 - 4096, one
 *              with more than 2^32 tiles (128 keys each, for every KV head and
 *              block of query rows), and a page outside the cache, latch
 *              QVG_ERR_INVALID_ARG and make the sequence's output undefined.
 *   mask       QVG_MASK_TREE: uint32 [total_q][mask_words] (qvg_tree_mask, or
 *              any bits); mask_words >= ceil(max_q / 32).
 *   scale      as in qvg_attention.
 *   out        [total_q][Hq][d] fp32 or bf16, 16-byte aligned; a row that
 *              sees no key is 0.
 *   lse        fp32 [Hq][total_q] natural-log log-sum-exp of the scaled
 *              logits (-inf for a row that sees no key), or NULL.
 *   total_q    rows of q, out and lse.
 *   workspace  at least qvg_paged_workspace_size(H, d, Hq, B, max_q) bytes.
 * Keys that a token does not see, and slots past kv_len, have no influence
 * on it, whatever they hold.  Q enters the product as the sum of two fp8
 * numbers, K and V as their codes, the weights times V's scale as the sum of
 * three fp8 numbers or as fp16; all sums are fp32.
 *   max_q * Hq / H <= 64 (32 with 4 bits): a channel of q is exact down to
 *     2^-13 of its row's largest and off by at most 2^-21 of the largest
 *     below; a weight is off by at most 2^-9 + 2^-11 of itself or 2^-25 of the
 *     largest.
 *   more rows: 2^-9 and 2^-17; 2^-11.
 *   Where V is so small that it matters, an output over n keys is off by at
 *   most n 2^-106 more (the weights' range ends), and from 2^23 keys on lse
 *   may be infinite.
 *   Where V passes 2^111, a weight below 2^-8 of the largest may count as 0.
 *   4 bits: K groups (with few rows V's too) whose scale is below 2^-14 of
 *     their row's largest count as 0 (with many rows V's below 2^-24).
 * A row of q with an infinity or a NaN, and one that sees a K or V row marked
 * with scale 255, gives NaN (with many rows its lse is NaN too where only V is
 * marked).  The results do not depend on what else the GPU runs: the split of
 * the work follows from the sizes and the number of SMs alone.
 * All sizes on the device are read when the kernels run: a captured call can
 * be replayed with other lengths, tables and masks.
 */
qvg_status qvg_paged_attention(const qvg_paged *cache, const void *q_bf16, int64_t q_stride, int32_t total_q,
                               int32_t Hq, int32_t B, int32_t max_q, const int32_t *cu_q, const int32_t *table,
                               int32_t table_stride, const int32_t *kv_len, int32_t mask_mode,
                               const uint32_t *mask, int32_t mask_words, float scale, void *out,
                               int32_t out_dtype, float *lse, void *workspace, size_t ws_bytes, void *stream);

/* ======================================================================
 * The latent cache: for models that keep one latent vector a token, from
 * which every head's key and value are projected, and one key part that
 * carries the rotary position and is shared by the heads.
 * ====================================================================== */

/*
 * A paged cache of latents (one layer), slots and pages as in qvg_paged:
 *   c    bf16 [num_pages][page_size][dc]   the latent;
 *   kr   bf16 [num_pages][page_size][dr]   the shared key part, rotated.
 * A token that held an infinity or a NaN is all NaN, both parts.
 * dc = 64, 128, 192 or 256; dr a multiple of 8 up to 128 (0: none, kr NULL);
 * page_size 16, 32, 64, 128 or 256.  Both buffers are caller-allocated,
 * 16-byte aligned device memory of the size that qvg_latent_bytes reports, and
 * share no byte.
 */
typedef struct {
    int32_t dc;
    int32_t dr;
    int32_t page_size;
    int32_t num_pages;
    void *c;
    void *kr;
} qvg_latent;

/* Bytes of the two buffers. */
qvg_status qvg_latent_bytes(int32_t dc, int32_t dr, int32_t page_size, int32_t num_pages, size_t *c, size_t *kr);

/*
 * Write n tokens into their slots.
 *   c, k_rope  bf16 [n][dc] and [n][dr], 16-byte aligned; token t starts at
 *              element t * c_stride (t * kr_stride), a multiple of 8 and
 *              >= dc (dr).  (Both may be parts of one wider row.)
 *   slots      int64 [n] device, as in qvg_paged_append.
 *   plan       NULL, or rotary positions that k_rope gets on the way (its
 *              first plan->dims channels), in fp32 and rounded once, as
 *              qvg_rope does.  positions int32 [n][axes] device.
 * A slot at or beyond the cache's end is skipped and latches
 * QVG_ERR_INVALID_ARG.  Nothing but the tokens' slots is written.
 * Errors: QVG_ERR_INVALID_ARG for a bad cache or plan, n < 0, missing or
 * misaligned pointers, bad strides; QVG_ERR_UNSUPPORTED for another dc, and
 * for n above 2^30.
 */
qvg_status qvg_latent_append(const qvg_latent *cache, const void *c_bf16, const void *k_rope_bf16, int32_t n,
                             int64_t c_stride, int64_t kr_stride, const int64_t *slots, const qvg_rope_plan *plan,
                             const int32_t *positions, void *stream);

/*
 * Read n slots back: c_out bf16 [n][dc], kr_out bf16 [n][dr], 16-byte aligned;
 * either may be NULL.  A negative slot gives zeros; a slot beyond the cache
 * gives zeros and latches QVG_ERR_INVALID_ARG.
 */
qvg_status qvg_latent_read(const qvg_latent *cache, const int64_t *slots, int32_t n, void *c_out, void *kr_out,
                           void *stream);

/*
 * bf16 values [tokens][heads][channels] whose channels are contiguous: token t
 * of head h starts at element t * token_stride + h * head_stride.  data is
 * 16-byte aligned; the strides are multiples of 8 and at least the channels
 * (a stride that is never taken, of one token or one head, may be anything).
 */
typedef struct {
    const void *data;
    int64_t token_stride;
    int64_t head_stride;
} qvg_view;

/*
 * Scratch bytes of qvg_latent_attention on the current device (256-byte
 * aligned; no initialisation needed, dead after the call).
 */
qvg_status qvg_latent_workspace_size(int32_t dc, int32_t dr, size_t *bytes);

/*
 * Attention of B sequences' new tokens over a latent cache, in the absorbed
 * form: the heads' key projections have been multiplied into the queries, and
 * the value projections come after the call, so all Hq heads read the same
 * latents.  Row (t, h) against token j:
 *   S_j = scale * (q[t][h] . c_j + q_rope[t][h] . kr_j),   O[t][h] = softmax(S) c.
 *   q       [total_q][Hq][dc];  q_rope [total_q][Hq][dr] (NULL where dr = 0).
 *   scale   > 0 (it follows from the channels before the absorption).
 *   out     [total_q][Hq][dc] fp32 or bf16, 16-byte aligned.
 *   total_q, B, max_q, cu_q, table, table_stride, kv_len, mask_mode, mask,
 *   mask_words, lse: as in qvg_paged_attention, here with one KV head.
 *   workspace  at least qvg_latent_workspace_size(dc, dr) bytes.
 * Products are of bf16 numbers with fp32 sums; a weight enters the second one
 * rounded to bf16, i.e. off by at most 2^-8 of itself (lse takes it in fp32).
 * Keys that a token does not see, and slots past kv_len, have no influence
 * on it, whatever they hold.  A row of q with an infinity or a NaN, one that
 * sees a token that is NaN, and one whose every logit falls below fp32's range
 * gives NaN, where it sees a key.  The results do not depend on what
 * else the GPU runs.  All sizes on the device are read when the kernels run: a
 * captured call can be replayed with other lengths, tables and masks.
 * QVG_ERR_INVALID_ARG for sizes, modes, a scale or strides outside the above,
 * and missing or misaligned pointers; QVG_ERR_UNSUPPORTED for another dc,
 * B above 2^20, max_q * Hq above 2^31 - 129, or num_pages * page_size above
 * 2^31 - 1;
 * QVG_ERR_WORKSPACE for a workspace missing, too small or misaligned.  A
 * batch whose blocks of 128 rows, each counted as its sequence's tiles of 64
 * keys and 5 more, make 2^32 - 1 or more is left out altogether and latches
 * QVG_ERR_INVALID_ARG.
 */
qvg_status qvg_latent_attention(const qvg_latent *cache, const qvg_view *q, const qvg_view *q_rope, int32_t total_q,
                                int32_t Hq, int32_t B, int32_t max_q, const int32_t *cu_q, const int32_t *table,
                                int32_t table_stride, const int32_t *kv_len, int32_t mask_mode, const uint32_t *mask,
                                int32_t mask_words, float scale, void *out, int32_t out_dtype, float *lse,
                                void *workspace, size_t ws_bytes, void *stream);

/*
 * Attention of prompts in the expanded form: keys and values projected per
 * head, the rotated key part still one for all heads.  For B sequences, with T
 * new tokens (rows of q) that are the last of L keys,
 *   S[t][h][j] = scale * (q[t][h] . k[j][h] + q_rope[t][h] . k_rope[j]),
 *   O[t][h] = softmax(S) v[:][h].
 *   q, k       [total_q][H][dn], [total_k][H][dn];  dn = 64 or 128.
 *   q_rope, k_rope  [total_q][H][dr], [total_k][dr] (head_stride not used); dr
 *              a multiple of 8 up to 64; 0: none, both NULL.
 *   v          [total_k][H][dv];  dv = 64 or 128.
 *   cu_q, cu_k int32 [B + 1] device, ascending from 0: first rows of each
 *              sequence's new tokens and keys; NULL: max_q, max_k rows each.
 *              A sequence with more than max_q new tokens, or rows outside
 *              total_q or total_k, latches QVG_ERR_INVALID_ARG: its tokens
 *              beyond max_q are left out, rows outside are not touched.
 *   max_k      used where cu_k is NULL.
 *   mask_mode  QVG_MASK_NONE, or QVG_MASK_CAUSAL: new token t sees the keys
 *              0 .. L - T + t.
 *   scale      <= 0: 1 / sqrt(dn + dr).
 *   out        [total_q][H][dv] fp32 or bf16, 16-byte aligned; a row that
 *              sees no key is 0.  Rows from cu_q[B] on are left as they were.
 *   lse        fp32 [H][total_q] or NULL, as in qvg_paged_attention.
 * Rounding, NaN and unseen keys as in qvg_latent_attention (a row that sees a
 * value with an infinity or a NaN may be NaN in all its channels).
 * QVG_ERR_INVALID_ARG as there; QVG_ERR_UNSUPPORTED for another dn or dv, dr
 * above 64, B above 2^20, max_q above 2^31 - 257, total_k above 2^31 - 65, or
 * more than 2^31 - 1 blocks of 256 rows.
 */
qvg_status qvg_expanded_attention(const qvg_view *q, const qvg_view *q_rope, const qvg_view *k, const qvg_view *k_rope,
                                  const qvg_view *v, int32_t total_q, int32_t total_k, int32_t H, int32_t dn, int32_t dr,
                                  int32_t dv, int32_t B, int32_t max_q, int32_t max_k, const int32_t *cu_q,
                                  const int32_t *cu_k, int32_t mask_mode, float scale, void *out, int32_t out_dtype,
                                  float *lse, void *stream);

/* ======================================================================
 * Pages: which sequence holds which page of the paged caches, and moving what
 * is in them.  One block table serves every layer's cache.
 * ====================================================================== */

/*
 * The pages of a pool: refs int32 [num_pages] device, how many sequences hold
 * each page (0: free).  It starts as zeros and is all the state there is.
 */
typedef struct {
    int32_t num_pages;
    int32_t *refs;
} qvg_page_pool;

/*
 * A batch of sequences, device arrays that the calls read and change:
 *   table   int32 [B][table_stride]  pages of sequence b in order; entries past
 *           its last page mean nothing;
 *   kv_len  int32 [B]                its tokens.
 * Sequence b holds the first ceil(kv_len[b] / page_size) pages of its row.
 * page_size 16, 32, 64, 128 or 256.
 */
typedef struct {
    int32_t B;
    int32_t page_size;
    int32_t table_stride;
    int32_t *table;
    int32_t *kv_len;
} qvg_sequences;

/*
 * Make children[i] a copy of sequence parents[i] that shares its pages (int32
 * [n] device): the row's entries and the length are copied, and each page is
 * held once more.  A child must be empty (kv_len 0), be named once, and not
 * be a parent in the same call.  A pair that breaks this, names a sequence
 * outside the batch, or a parent with more pages than its row, is left out and
 * latches QVG_ERR_INVALID_ARG; so does a page outside the pool, whose entry is
 * copied all the same.  QVG_ERR_UNSUPPORTED for n above 2^20.
 */
qvg_status qvg_pages_fork(const qvg_page_pool *pool, const qvg_sequences *seqs, const int32_t *parents,
                          const int32_t *children, int32_t n, void *stream);

/*
 * Cut sequences ids[i] (int32 [n] device) to their first keep[i] tokens (keep
 * NULL: 0, the whole sequence is freed): pages past those are held once less,
 * and free where nobody holds them.  A sequence outside the batch, one named
 * twice, and a keep outside 0 .. kv_len is left as it was and latches
 * QVG_ERR_INVALID_ARG; a page outside the pool or held by nobody latches it and
 * is passed over.  QVG_ERR_UNSUPPORTED for n above 2^20.
 */
qvg_status qvg_pages_release(const qvg_page_pool *pool, const qvg_sequences *seqs, const int32_t *ids,
                             const int32_t *keep, int32_t n, void *stream);

/* Scratch bytes of qvg_pages_reserve (16-byte aligned; dead after the call). */
qvg_status qvg_pages_workspace_size(int32_t num_pages, int32_t B, size_t *bytes);

/*
 * Make room for new tokens at the sequences' ends and say where they go.
 *   cu_new   int32 [B + 1] device, ascending from 0: sequence b gets
 *            cu_new[b + 1] - cu_new[b] tokens (0 is allowed); NULL: n_new each.
 *   slots    int64 [total] device: slot of each new token, sequence by sequence
 *            (for the append calls).  total = cu_new[B] or B * n_new.
 *   copies   int32 [B][2] device: (page, new page) where a sequence's last page
 *            was partly filled and shared and so is replaced by a copy of its
 *            own (to be filled by qvg_pages_copy in every layer's cache, before
 *            the append); (-1, -1) elsewhere.
 * Of k sequences that write to one shared page, in their order, each takes a
 * copy while another holder is left; the last holder keeps the page.  New pages
 * are the lowest free ones, in the order in which the sequences need them (a
 * copy first); a page that becomes free in the call is not given out by it.
 * kv_len grows by the new tokens.
 * If the free pages or a table row do not suffice, nothing changes but slots
 * and copies, which are -1 throughout, and QVG_ERR_CAPACITY is latched; if
 * cu_new does not ascend from 0 to total, kv_len is negative or a
 * shared page lies outside the pool, the same with QVG_ERR_INVALID_ARG.
 *   workspace  at least qvg_pages_workspace_size(num_pages, B) bytes.
 * QVG_ERR_UNSUPPORTED for B, total or num_pages above 2^31 - 2049.
 */
qvg_status qvg_pages_reserve(const qvg_page_pool *pool, const qvg_sequences *seqs, const int32_t *cu_new, int32_t n_new,
                             int32_t total, int64_t *slots, int32_t *copies, void *workspace, size_t ws_bytes,
                             void *stream);

/*
 * What the next two calls move: the buffers of a cache as rows.  Buffer i is
 * [num_pages][heads[i]][page_size][row_bytes[i]] bytes at base[i], below 2^63.
 */
typedef struct {
    int32_t page_size;
    int32_t num_pages;
    int32_t n;
    void *base[4];
    int32_t heads[4];
    int32_t row_bytes[4];
} qvg_page_rows;

qvg_status qvg_paged_rows(const qvg_paged *cache, qvg_page_rows *rows);
qvg_status qvg_latent_rows(const qvg_latent *cache, qvg_page_rows *rows);

/*
 * Copy whole pages: copies int32 [n][2] device, (from, to); a pair with a
 * negative page is passed over, one with a page beyond the cache latches
 * QVG_ERR_INVALID_ARG and is passed over.  The copies run at the same time: no
 * page may be written twice, or be both read and written.
 * QVG_ERR_UNSUPPORTED for n above 2^31 - 65536.
 */
qvg_status qvg_pages_copy(const qvg_page_rows *rows, const int32_t *copies, int32_t n, void *stream);

/*
 * Move the tokens that are kept together, in place: token first[b] + i of
 * sequence b becomes what token keep[b][i] was, for i < n_keep[b].
 *   first, n_keep  int32 [B] device;  keep int32 [B][keep_stride] device,
 *           ascending, and not below first[b] (accepted tokens of a drafted
 *           tree, or what is left of a history).
 * Tokens past those keep what they held (qvg_pages_release cuts them off).
 * Pages that are written must not be shared with another sequence.
 *   table, table_stride, B  as in qvg_paged_attention.
 * n_keep outside 0 .. keep_stride, a negative first, a keep that does not
 * ascend or is beyond the row, and a page outside the cache latch
 * QVG_ERR_INVALID_ARG; that sequence is left as it was.  (Where keep_stride is
 * 0 nothing is looked at.)  QVG_ERR_UNSUPPORTED for B above 65535 or keep_stride above 2^31 - 2049.
 */
qvg_status qvg_paged_compact(const qvg_page_rows *rows, const int32_t *table, int32_t table_stride, int32_t B,
                             const int32_t *first, const int32_t *keep, int32_t keep_stride, const int32_t *n_keep,
                             void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QVG_H */
