// latent_attention.cu -- attention over a latent cache (absorbed form) and of
// prompts (expanded form): launch, the join of units that several CTAs shared,
// and the entry points.  The kernel is in latent_attention.cuh.
#include <cmath>

#include "latent_attention.cuh"

namespace qvg {
namespace {

// The unit that begins in CTA i and goes on to CTA `last` left one partial
// sum per CTA: slot 1 of CTA i, slot 0 of the others.  With references m_z,
// sums l_z and O_z: m = max m_z, l = sum l_z 2^(m_z - m), O likewise.  One
// warp per query row; lane z weighs part z, then the lanes share the channels
// and go through the parts in CTA order, so the result is the same each time.
template <int DC>
__global__ void __launch_bounds__(256) k_latent_merge(const __grid_constant__ la::Args a) {
    constexpr int E = DC / 32, V = E % 4 == 0 ? 4 : 2, NV = E / V;  // a lane's channels: NV runs of V, 32 V apart
    pdl_wait();
    const int4 u = a.desc[blockIdx.x];
    if (u.x < 0) return;
    const int n = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const pa::Seq s = pa::seq_of<la::kRows, la::kKeys>(a, u.x, false);
    const long long gi = static_cast<long long>(u.z) * la::kRows + n;
    const int tq = static_cast<int>(gi / a.grp), h = static_cast<int>(gi - static_cast<long long>(tq) * a.grp);
    if (tq >= s.nq) return;
    const int first = blockIdx.x, last = min(u.w, static_cast<int>(gridDim.x) - 1);
    auto at = [&](int z) { return static_cast<size_t>(2 * z + (z == first ? 1 : 0)) * la::kRows + n; };
    float m = -INFINITY;
    for (int z = first + lane; z <= last; z += 32)
        if (a.pl[at(z)] != 0.0f) m = fmaxf(m, a.pm[at(z)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float acc[E], l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    for (int z0 = first; z0 <= last; z0 += 32) {
        const int z = z0 + lane;
        float lz = z <= last ? a.pl[at(z)] : 0.0f;
        const float w = lz == 0.0f ? 0.0f : exp2f(a.pm[at(z)] - m);
        lz *= w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lz += __shfl_xor_sync(0xFFFFFFFFu, lz, o);
        l += lz;
        const int parts = min(32, last - z0 + 1);
#pragma unroll 8
        for (int k = 0; k < parts; ++k) {
            const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
            const float *o = a.po + at(z0 + k) * DC + lane * V;
            if (wk != 0.0f) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        const float2 x = *reinterpret_cast<const float2 *>(o + i * 32 * V + e);
                        acc[i * V + e] = fmaf(wk, x.x, acc[i * V + e]);
                        acc[i * V + e + 1] = fmaf(wk, x.y, acc[i * V + e + 1]);
                    }
            }
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const long long row = static_cast<long long>(s.q0 + tq) * a.Hq + h;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const long long c = row * DC + i * 32 * V + lane * V + e;
            const float x = acc[i * V + e] * inv, y = acc[i * V + e + 1] * inv;
            if (a.out32)
                *reinterpret_cast<float2 *>(a.out32 + c) = make_float2(x, y);
            else
                *reinterpret_cast<uint32_t *>(a.out16 + c) = la::bf16x2(x, y);
        }
    if (lane == 0 && a.lse)
        a.lse[static_cast<long long>(h) * a.total_q + s.q0 + tq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
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
    w.bytes = w.desc + al(static_cast<size_t>(ctas) * sizeof(int4));
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

// The rings' stages: what Q leaves of the shared memory.
void stages(la::Args &a, bool latent) {
    const int room = la::kSmem - 1024 - (latent ? 1 : 2) * a.na * la::kQChunk, A = a.na * la::kChunk, B = a.nb * la::kChunk;
    a.sb = std::min(la::kMostStages, room / (A + B));
    a.sa = latent ? 0 : std::min(la::kMostStages, (room - a.sb * B) / A);
}

template <bool LATENT>
qvg_status launch(const CUtensorMap (&map)[3], const la::Args &a, int grid, int blocks, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const qvg_status s = smem_limit_once(done, reinterpret_cast<const void *>(la::k_latent_attention<LATENT>), la::kSmem);
    if (s != QVG_OK) return s;
    la::k_latent_attention<LATENT><<<grid, LATENT ? 384 : 512, la::kSmem, st>>>(map[0], map[1], map[2], a, blocks);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

template <int DC>
qvg_status launch_merge(const la::Args &a, int ctas, cudaStream_t st) {
    const cudaError_t e = launch_pdl(k_latent_merge<DC>, dim3(ctas, la::kRows / 8), dim3(256), 0, st, a);
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
    CUtensorMap map[3] = {};
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
    stages(a, true);
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
    s = launch<true>(map, a, ctas, 0, st);
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
    if (total_k > 0 && (!chunk_map(&map[0], k->data, dn, H, total_k, k->head_stride, k->token_stride, la::kKeys, dn / 64) ||
                        (dr > 0 && !rotated_map(&map[1], k_rope->data, dr, total_k, k_rope->token_stride, la::kKeys)) ||
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
    stages(a, false);
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
    return launch<false>(map, a, static_cast<int>(grid), static_cast<int>(blocks), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
