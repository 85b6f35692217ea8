// latent_attention.cu -- attention over a latent cache (absorbed form) and of
// prompts (expanded form): launch, the join of units that several CTAs shared,
// and the entry points.  The kernels are in latent_attention.cuh and
// expanded_attention.cuh.
#include <cmath>

#include "expanded_attention.cuh"
#include "latent_attention.cuh"

namespace qvg {
namespace {

// Units that several CTAs shared: with references m_z, sums l_z and O_z of the
// P parts, m = max m_z, l = sum l_z 2^(m_z - m), O likewise.  The unit that
// begins in CTA i has its part in slot 1 of CTA i and in slot 0 of the CTAs after
// it, up to `last`.  Each of them takes part in the join: block x, as the CTA of rank x - i, has rows
// rank, rank + P, ..; blockIdx.y: a half of the channels.  Few parts: a warp
// a row, part by part; many: the block's warps share a row's parts and add up
// in their order, so the result is the same each time.  (One warp per row and
// part after part, 152 parts of 16 rows took 48 us.)
constexpr int kJoinWarps = 8, kFewParts = 8;

template <int DC>
__device__ __forceinline__ void join(const la::Args &a, const int4 u, int rank, float (*s_acc)[DC / 2], float *s_l) {
    constexpr int E = DC / 64;  // a lane's channels: lane, lane + 32, .. of the half
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const pa::Seq s = pa::seq_of<la::kRows, la::kKeys>(a, u.x, false);
    const int first = u.z, last = min(u.w, static_cast<int>(gridDim.x) - 1), parts = last - first + 1;
    const bool few = parts <= kFewParts;
    const long long row0 = static_cast<long long>(u.y) * la::kRows;
    const int rows = static_cast<int>(max(0ll, min(static_cast<long long>(la::kRows), static_cast<long long>(s.nq) * a.grp - row0)));
    const int step = few ? kJoinWarps : 1;
    for (int n0 = rank; n0 < rows; n0 += parts * step) {  // (the block's warps go through this together)
        const int n = few ? n0 + parts * warp : n0;
        auto at = [&](int z) { return static_cast<size_t>(2 * z + (z == first ? 1 : 0)) * la::kRows + n; };
        float acc[E], l = 0.0f, m = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        if (n < rows) {
            for (int z = first + lane; z <= last; z += 32)
                if (a.pl[at(z)] != 0.0f) m = fmaxf(m, a.pm[at(z)]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
#pragma unroll 8
            for (int z = first + (few ? 0 : warp); z <= last; z += few ? 1 : kJoinWarps) {
                const float lz = a.pl[at(z)], w = lz == 0.0f ? 0.0f : exp2f(a.pm[at(z)] - m);
                const float *o = a.po + at(z) * DC + blockIdx.y * (DC / 2) + lane;
                l = fmaf(lz, w, l);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float x = o[32 * e];
                    acc[e] = w == 0.0f ? acc[e] : fmaf(w, x, acc[e]);
                }
            }
        }
        if (!few) {
#pragma unroll
            for (int e = 0; e < E; ++e) s_acc[warp][lane + 32 * e] = acc[e];
            if (lane == 0) s_l[warp] = l;
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int w = 1; w < kJoinWarps; ++w) {
                    l += s_l[w];
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += s_acc[w][lane + 32 * e];
                }
            }
            __syncthreads();
        }
        if (n >= rows || (!few && warp > 0)) continue;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const long long gi = row0 + n;
        const int tq = static_cast<int>(gi / a.grp), h = static_cast<int>(gi - static_cast<long long>(tq) * a.grp);
        const long long out = (static_cast<long long>(s.q0 + tq) * a.Hq + h) * DC + blockIdx.y * (DC / 2) + lane;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (a.out32)
                a.out32[out + 32 * e] = acc[e] * inv;
            else
                a.out16[out + 32 * e] = f32_to_bf16(acc[e] * inv);
        }
        if (lane == 0 && blockIdx.y == 0 && a.lse)
            a.lse[static_cast<long long>(h) * a.total_q + s.q0 + tq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
}

template <int DC>
__global__ void __launch_bounds__(kJoinWarps * 32) k_latent_merge(const __grid_constant__ la::Args a) {
    __shared__ float s_acc[kJoinWarps][DC / 2], s_l[kJoinWarps];
    pdl_wait();
    const int x = blockIdx.x;
    const int4 head = a.desc[2 * x], cut = a.desc[2 * x + 1];
    if (head.x >= 0) join<DC>(a, head, x - head.z, s_acc, s_l);
    if (cut.x >= 0) join<DC>(a, cut, 0, s_acc, s_l);
}

struct Workspace {
    size_t pm, pl, desc, bytes;  // offsets (the partial sums of O are first)
};
Workspace carve(int ctas, int dc) {
    auto al = [](size_t b) { return (b + 255) & ~static_cast<size_t>(255); };
    const size_t rows = static_cast<size_t>(ctas) * 2 * la::kRows;
    Workspace w{};
    w.pm = al(rows * dc * 4);
    w.pl = w.pm + al(rows * 4);
    w.desc = w.pl + al(rows * 4);
    w.bytes = w.desc + al(static_cast<size_t>(ctas) * 2 * sizeof(int4));
    return w;
}

// bf16 values [rows][heads][channels], channels by chunks of 64: dimensions
// (channel of a chunk, row, chunk, head); a box is `box` rows of one head's
// `chunks` chunks, laid out chunk after chunk and swizzled as the tensor core
// reads them.
bool chunk_map(CUtensorMap *m, const void *data, int channels, int heads, int64_t rows, int64_t head_stride, int64_t row_stride, int box, int chunks) {
    const auto fn = tensor_map_encoder();
    if (!fn) return false;
    if (rows == 1) row_stride = 64;  // (never taken)
    if (heads == 1) head_stride = 64;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(channels / 64), static_cast<cuuint64_t>(heads)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(2 * row_stride), 128, static_cast<cuuint64_t>(2 * head_stride)};
    const cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(chunks), 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, heads > 0 ? 4 : 3, const_cast<void *>(data), dims, strides, boxes, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The rotated part, bf16 [rows][channels]; a box is 64 channels of `box` rows,
// channels beyond the last are filled with 0.
bool rotated_map(CUtensorMap *m, const void *data, int channels, int64_t rows, int64_t row_stride, int box) {
    const auto fn = tensor_map_encoder();
    if (!fn) return false;
    if (rows == 1) row_stride = 64;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(channels), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(2 * row_stride)};
    const cuuint32_t boxes[2] = {64, static_cast<cuuint32_t>(box)};
    const cuuint32_t es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(data), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

qvg_status launch_latent(const CUtensorMap (&map)[2], la::Args &a, int ctas, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const qvg_status s = smem_limit_once(done, reinterpret_cast<const void *>(la::k_latent_attention), la::kSmem);
    if (s != QVG_OK) return s;
    // the stages: what Q's rotated part leaves of the shared memory
    a.sb = std::min(la::kMostStages, (la::kSmem - 1024 - a.na * la::kQChunk) / ((a.na + a.nb) * la::kChunk));
    la::k_latent_attention<<<ctas, la::kLatentWarps * 32, la::kSmem, st>>>(map[0], map[1], a);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

qvg_status launch_expanded(const CUtensorMap (&map)[3], la::Args &a, int grid, int blocks, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const qvg_status s = smem_limit_once(done, reinterpret_cast<const void *>(la::k_expanded_attention), la::kSmem);
    if (s != QVG_OK) return s;
    // two tiles of K at least, then as many half tiles of V as there is room for
    const int room = la::kSmem - 1024 - 2 * a.na * la::kQChunk, A = a.na * la::kKChunk, B = a.nb * la::kChunk;
    a.sb = std::min(la::kMostStages, (room - 2 * A) / B);
    a.sa = std::min(la::kMostStages, (room - a.sb * B) / A);
    la::k_expanded_attention<<<grid, la::kPromptWarps * 32, la::kSmem, st>>>(map[0], map[1], map[2], a, blocks);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

template <int DC>
qvg_status launch_merge(const la::Args &a, int ctas, cudaStream_t st) {
    const cudaError_t e = launch_pdl(k_latent_merge<DC>, dim3(ctas, 2), dim3(kJoinWarps * 32), 0, st, a);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        note_cuda_error(e);
        return QVG_ERR_CUDA;
    }
    return QVG_OK;
}

bool misaligned(const void *p, uintptr_t to) { return !p || reinterpret_cast<uintptr_t>(p) % to != 0; }

// A view's data and strides (channels: of a head; heads and tokens: how many the call takes).
bool view_ok(const qvg_view *v, int channels, int64_t tokens, int heads) {
    if (!v || misaligned(v->data, 16)) return false;
    if (tokens > 1 && (v->token_stride < channels || v->token_stride % 8 != 0)) return false;
    return heads <= 1 || (v->head_stride >= channels && v->head_stride % 8 == 0);
}

}  // namespace
}  // namespace qvg

using namespace qvg;

extern "C" {

qvg_status qvg_latent_workspace_size(int32_t dc, int32_t dr, size_t *bytes) {
    if (!bytes) return QVG_ERR_INVALID_ARG;
    const qvg_latent l{dc, dr, 16, 1, nullptr, nullptr};
    const qvg_status s = check_latent(&l, true);
    if (s != QVG_OK) return s;
    *bytes = carve(sm_count_current(), dc).bytes;
    return QVG_OK;
}

qvg_status qvg_latent_attention(const qvg_latent *cache, const qvg_view *q, const qvg_view *q_rope, int32_t total_q,
                                int32_t Hq, int32_t B, int32_t max_q, const int32_t *cu_q, const int32_t *table,
                                int32_t table_stride, const int32_t *kv_len, int32_t mask_mode, const uint32_t *mask,
                                int32_t mask_words, float scale, void *out, int32_t out_dtype, float *lse,
                                void *workspace, size_t ws_bytes, void *stream) {
    qvg_status s = check_latent(cache, false);
    if (s != QVG_OK) return s;
    const int dc = cache->dc, dr = cache->dr;
    if (Hq < 1 || B < 0 || max_q < 0 || total_q < 0 || table_stride < 1) return QVG_ERR_INVALID_ARG;
    if (mask_mode != QVG_MASK_NONE && mask_mode != QVG_MASK_CAUSAL && mask_mode != QVG_MASK_TREE) return QVG_ERR_INVALID_ARG;
    if (out_dtype != QVG_OUT_F32 && out_dtype != QVG_OUT_BF16) return QVG_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || scale <= 0.0f) return QVG_ERR_INVALID_ARG;
    if (!cu_q && static_cast<int64_t>(B) * max_q > total_q) return QVG_ERR_INVALID_ARG;
    if (B == 0 || max_q == 0 || total_q == 0) return QVG_OK;
    if (!view_ok(q, dc, total_q, Hq) || (dr > 0 && !view_ok(q_rope, dr, total_q, Hq))) return QVG_ERR_INVALID_ARG;
    if (misaligned(out, 16) || misaligned(table, 4) || misaligned(kv_len, 4) || (cu_q && misaligned(cu_q, 4)) ||
        (lse && misaligned(lse, 4)))
        return QVG_ERR_INVALID_ARG;
    if (mask_mode == QVG_MASK_TREE && (misaligned(mask, 4) || mask_words < ceil_div(max_q, 32))) return QVG_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_q) * Hq > INT32_MAX - la::kRows ||
        static_cast<int64_t>(cache->num_pages) * cache->page_size > INT32_MAX)
        return QVG_ERR_UNSUPPORTED;
    const int ctas = sm_count_current();
    const Workspace w = carve(ctas, dc);
    if (!workspace || ws_bytes < w.bytes || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return QVG_ERR_WORKSPACE;
    const int64_t slots = static_cast<int64_t>(cache->num_pages) * cache->page_size;
    const int box = std::min(cache->page_size, la::kKeys);
    CUtensorMap map[2] = {};
    // (a page that holds a whole tile is copied in one go, a smaller one chunk by chunk)
    if (!chunk_map(&map[0], cache->c, dc, 0, slots, 0, dc, box, box == la::kKeys ? dc / 64 : 1) ||
        (dr > 0 && !rotated_map(&map[1], cache->kr, dr, slots, dr, box)))
        return QVG_ERR_CUDA;
    la::Args a{};
    a.q = static_cast<const uint16_t *>(q->data);
    a.q_stride = q->token_stride;
    a.q_h = q->head_stride;
    if (dr > 0) {
        a.qr = static_cast<const uint16_t *>(q_rope->data);
        a.qr_t = q_rope->token_stride;
        a.qr_h = q_rope->head_stride;
    }
    a.total_q = total_q;
    a.Hq = a.grp = Hq;
    a.H = 1;
    a.dk = a.dv = dc;
    a.dr = dr;
    a.na = ceil_div(dr, 64);
    a.nb = dc / 64;
    a.B = B;
    a.max_q = max_q;
    a.cu_q = cu_q;
    a.table = table;
    a.kv_len = kv_len;
    a.table_stride = table_stride;
    a.page_log2 = __builtin_ctz(static_cast<unsigned>(cache->page_size));
    a.num_pages = cache->num_pages;
    a.mode = mask_mode;
    a.mask = mask;
    a.words = mask_words;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out32 = out_dtype == QVG_OUT_F32 ? static_cast<float *>(out) : nullptr;
    a.out16 = out_dtype == QVG_OUT_BF16 ? static_cast<uint16_t *>(out) : nullptr;
    a.lse = lse;
    char *base = static_cast<char *>(workspace);
    a.po = reinterpret_cast<float *>(base);
    a.pm = reinterpret_cast<float *>(base + w.pm);
    a.pl = reinterpret_cast<float *>(base + w.pl);
    a.desc = reinterpret_cast<int4 *>(base + w.desc);
    a.err = device_error_word();
    a.wait_ns = wait_limit_ns();
    a.inject = wait_inject();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    s = launch_latent(map, a, ctas, st);
    if (s != QVG_OK) return s;
    switch (dc) {
        case 64: return launch_merge<64>(a, ctas, st);
        case 128: return launch_merge<128>(a, ctas, st);
        case 192: return launch_merge<192>(a, ctas, st);
        default: return launch_merge<256>(a, ctas, st);
    }
}

qvg_status qvg_expanded_attention(const qvg_view *q, const qvg_view *q_rope, const qvg_view *k, const qvg_view *k_rope,
                                  const qvg_view *v, int32_t total_q, int32_t total_k, int32_t H, int32_t dn, int32_t dr,
                                  int32_t dv, int32_t B, int32_t max_q, int32_t max_k, const int32_t *cu_q,
                                  const int32_t *cu_k, int32_t mask_mode, float scale, void *out, int32_t out_dtype,
                                  float *lse, void *stream) {
    if (H < 1 || B < 0 || max_q < 0 || max_k < 0 || total_q < 0 || total_k < 0 || dr < 0 || dr % 8 != 0) return QVG_ERR_INVALID_ARG;
    if ((dn != 64 && dn != 128) || (dv != 64 && dv != 128) || dr > 64) return QVG_ERR_UNSUPPORTED;
    if (mask_mode != QVG_MASK_NONE && mask_mode != QVG_MASK_CAUSAL) return QVG_ERR_INVALID_ARG;
    if (out_dtype != QVG_OUT_F32 && out_dtype != QVG_OUT_BF16) return QVG_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return QVG_ERR_INVALID_ARG;
    if (!cu_q && static_cast<int64_t>(B) * max_q > total_q) return QVG_ERR_INVALID_ARG;
    if (!cu_k && static_cast<int64_t>(B) * max_k > total_k) return QVG_ERR_INVALID_ARG;
    if (B == 0 || max_q == 0 || total_q == 0) return QVG_OK;
    if (!view_ok(q, dn, total_q, H) || (dr > 0 && !view_ok(q_rope, dr, total_q, H))) return QVG_ERR_INVALID_ARG;
    if (total_k > 0 && (!view_ok(k, dn, total_k, H) || !view_ok(v, dv, total_k, H) || (dr > 0 && !view_ok(k_rope, dr, total_k, 1))))
        return QVG_ERR_INVALID_ARG;
    if (misaligned(out, 16) || (cu_q && misaligned(cu_q, 4)) || (cu_k && misaligned(cu_k, 4)) || (lse && misaligned(lse, 4)))
        return QVG_ERR_INVALID_ARG;
    const int64_t blocks = ceil_div(max_q, 256), grid = blocks * B * H;
    if (max_q > INT32_MAX - 256 || static_cast<int64_t>(B) * H > INT32_MAX || grid > INT32_MAX) return QVG_ERR_UNSUPPORTED;
    CUtensorMap map[3] = {};
    if (total_k > 0 && (!chunk_map(&map[0], k->data, dn, H, total_k, k->head_stride, k->token_stride, la::kPromptKeys, dn / 64) ||
                        (dr > 0 && !rotated_map(&map[1], k_rope->data, dr, total_k, k_rope->token_stride, la::kPromptKeys)) ||
                        !chunk_map(&map[2], v->data, dv, H, total_k, v->head_stride, v->token_stride, la::kKeys, dv / 64)))
        return QVG_ERR_CUDA;
    la::Args a{};
    a.q = static_cast<const uint16_t *>(q->data);
    a.q_stride = q->token_stride;
    a.q_h = q->head_stride;
    if (dr > 0) {
        a.qr = static_cast<const uint16_t *>(q_rope->data);
        a.qr_t = q_rope->token_stride;
        a.qr_h = q_rope->head_stride;
    }
    a.total_q = total_q;
    a.total_k = total_k;
    a.Hq = a.H = H;
    a.grp = 1;
    a.dk = dn;
    a.dv = dv;
    a.dr = dr;
    a.na = dn / 64 + (dr > 0 ? 1 : 0);
    a.nb = dv / 64;
    a.B = B;
    a.max_q = max_q;
    a.max_k = max_k;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.mode = mask_mode;
    a.scale_log2 = (scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(dn + dr))) * 1.4426950408889634f;
    a.out32 = out_dtype == QVG_OUT_F32 ? static_cast<float *>(out) : nullptr;
    a.out16 = out_dtype == QVG_OUT_BF16 ? static_cast<uint16_t *>(out) : nullptr;
    a.lse = lse;
    a.err = device_error_word();
    a.wait_ns = wait_limit_ns();
    a.inject = wait_inject();
    return launch_expanded(map, a, static_cast<int>(grid), static_cast<int>(blocks), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
