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
// it.  A task is 8 rows and some channels of a unit; the unit's CTAs share its
// tasks, as the blocks x of their numbers.  What bounds it is latency: the unit's
// description, then everything else, the parts (those that registers hold) along with
// their references and sums.
//   few parts: a warp a task (64 channels), parts one after another;
//   many: a block a task (16 channels), each warp every eighth part, whose sums
//   are added in the warps' order.
// Either way the result is the same each time.  152 parts of 16 rows add 8 us to the call.
// Few: eight, what a warp's lanes hold of references and sums (all joins the other way: 74 -> 91 us for the
// decode batch, 73 -> 154 for the trees).  kAhead: parts asked for along with the weights; four or ten, 59 us for
// one long token either way.
constexpr int kJoinWarps = 8, kJoinY = 2, kFewParts = 8, kMostParts = 512, kAhead = 10;

struct JoinRoom {
    float w[kMostParts][8], l[kMostParts][8], red[2][kJoinWarps][8];
    float4 acc[kJoinWarps][32];
};

__device__ __forceinline__ void add_weighed(float4 &a, float e, const float4 &x) {
    if (e != 0.0f) a = make_float4(fmaf(e, x.x, a.x), fmaf(e, x.y, a.y), fmaf(e, x.z, a.z), fmaf(e, x.w, a.w));
}

// What a joined row's sums are multiplied with: 0 without keys, NaN where there are keys and no weight (la::Row::lost).
__device__ __forceinline__ float joined_inverse(float m, float l) { return l != 0.0f ? 1.0f / l : m > -INFINITY ? __uint_as_float(0x7FFFFFFFu) : 0.0f; }

// Four channels of a joined row.
template <int DC>
__device__ __forceinline__ void put(const la::Args &a, const la::Shared &u, int n, int c, const float4 &acc, float inv) {
    const int gi = u.row0 + n, tq = gi / a.grp, h = gi - tq * a.grp;
    const long long out = (static_cast<long long>(u.q0 + tq) * a.Hq + h) * DC + c;
    const float4 x = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (a.out32)
        *reinterpret_cast<float4 *>(a.out32 + out) = x;
    else
        *reinterpret_cast<uint2 *>(a.out16 + out) = make_uint2(la::bf16x2(x.x, x.y), la::bf16x2(x.z, x.w));
}
__device__ __forceinline__ void put_lse(const la::Args &a, const la::Shared &u, int n, float m, float l) {
    const int gi = u.row0 + n, tq = gi / a.grp, h = gi - tq * a.grp;
    a.lse[static_cast<long long>(h) * a.total_q + u.q0 + tq] = l != 0.0f ? (m + log2f(l)) * 0.69314718055994531f : joined_inverse(m, l) == 0.0f ? -INFINITY : __uint_as_float(0x7FFFFFFFu);
}

template <int DC>
__device__ __forceinline__ void join(const la::Args &a, const la::Shared &u, int rank, int y, JoinRoom &s) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r8 = lane & 7, cg = lane >> 3;
    const int parts = min(u.last, static_cast<int>(gridDim.x) - 1) - u.first + 1, octets = (u.rows + 7) / 8;
    auto slot = [&](int z) { return static_cast<size_t>(2 * (u.first + z) + (z == 0 ? 1 : 0)); };
    if (parts <= kFewParts) {
        for (int task = rank + parts * (y * kJoinWarps + warp); task < octets * (DC / 64); task += parts * (kJoinY * kJoinWarps)) {
            const int slice = task % (DC / 64), n = task / (DC / 64) * 8 + r8;
            const float *src = a.po + (static_cast<size_t>(slice * 16 + cg) * la::kRows + n) * 4;
            auto part = [&](int z, int i) { return *reinterpret_cast<const float4 *>(src + slot(z) * (la::kRows * DC) + i * (16 * la::kRows)); };
            float4 x[2][4];
#pragma unroll
            for (int z = 0; z < 2; ++z)  // (a shared unit has two parts at least)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[z][i] = part(z, i);
            float pm[2], w[2], m = -INFINITY, l = 0.0f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int z = 4 * k + cg;
                pm[k] = z < parts ? a.pm[slot(z) * la::kRows + n] : -INFINITY;
                w[k] = z < parts ? a.pl[slot(z) * la::kRows + n] : 0.0f;
                m = fmaxf(m, pm[k]);
            }
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float e = w[k] == 0.0f ? 0.0f : exp2f(pm[k] - m);
                l = fmaf(w[k], e, l);
                w[k] = e;
            }
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
            float4 acc[4] = {};
            for (int z0 = 0; z0 < parts; z0 += 2) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float e = __shfl_sync(0xFFFFFFFFu, z0 < 4 ? w[0] : w[1], ((z0 + k) & 3) * 8 + r8);  // (0 past the last part)
#pragma unroll
                    for (int i = 0; i < 4; ++i) add_weighed(acc[i], e, x[k][i]);
                    if (z0 + 2 + k < parts) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[k][i] = part(z0 + 2 + k, i);
                    }
                }
            }
            if (n >= u.rows) continue;
            const float inv = joined_inverse(m, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) put<DC>(a, u, n, slice * 64 + 16 * i + 4 * cg, acc[i], inv);
            if (cg == 0 && slice == 0 && a.lse) put_lse(a, u, n, m, l);
        }
        return;
    }
    for (int task = rank + parts * y; task < octets * (DC / 16); task += parts * kJoinY) {
        const int slice = task % (DC / 16), n = task / (DC / 16) * 8 + r8, z0 = tid >> 3;
        const float *src = a.po + (static_cast<size_t>(slice * 4 + cg) * la::kRows + n) * 4;
        float m = -INFINITY, l = 0.0f;
        float4 x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (warp + k * kJoinWarps < parts) x[k] = *reinterpret_cast<const float4 *>(src + slot(warp + k * kJoinWarps) * (la::kRows * DC));
        __syncthreads();  // (the last task's room has been read)
        // thread (row r8, parts z0 + 32 k)
#pragma unroll 5
        for (int z = z0; z < parts; z += 32) {
            const float y = a.pm[slot(z) * la::kRows + n];
            s.w[z][r8] = y;
            s.l[z][r8] = a.pl[slot(z) * la::kRows + n];
            m = fmaxf(m, y);
        }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
        if (lane < 8) s.red[0][warp][r8] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) m = fmaxf(m, s.red[0][k][r8]);
        for (int z = z0; z < parts; z += 32) {
            const float lz = s.l[z][r8], e = lz == 0.0f ? 0.0f : exp2f(s.w[z][r8] - m);
            l = fmaf(lz, e, l);
            s.w[z][r8] = e;
        }
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
        if (lane < 8) s.red[1][warp][r8] = l;
        __syncthreads();
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) l += s.red[1][k][r8];
        float4 acc = {};
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (warp + k * kJoinWarps < parts) add_weighed(acc, s.w[warp + k * kJoinWarps][r8], x[k]);
#pragma unroll 4
        for (int z = warp + kAhead * kJoinWarps; z < parts; z += kJoinWarps)
            add_weighed(acc, s.w[z][r8], *reinterpret_cast<const float4 *>(src + slot(z) * (la::kRows * DC)));
        s.acc[warp][lane] = acc;
        __syncthreads();
        if (warp > 0) continue;
#pragma unroll
        for (int k = 1; k < kJoinWarps; ++k) add_weighed(acc, 1.0f, s.acc[k][lane]);
        if (n >= u.rows) continue;
        put<DC>(a, u, n, slice * 16 + 4 * cg, acc, joined_inverse(m, l));
        if (cg == 0 && slice == 0 && a.lse) put_lse(a, u, n, m, l);
    }
}

// blockIdx.y: which of the CTA's two shared units, and a share of the tasks.
template <int DC>
__global__ void __launch_bounds__(kJoinWarps * 32, 3) k_latent_merge(const __grid_constant__ la::Args a) {
    __shared__ JoinRoom s;
    pdl_wait();
    const int x = blockIdx.x, which = blockIdx.y & 1;
    const la::Shared u = reinterpret_cast<const la::Shared *>(a.desc)[2 * x + which];
    if (u.rows > 0) join<DC>(a, u, which ? 0 : x - u.first, blockIdx.y >> 1, s);
}

// Sequences of a call: every CTA walks over all of them, 32 (prompts: 512) at a time, with 32-bit numbers that step
// past the last one, while the other roles' waits run.
constexpr int kMostSequences = 1 << 20;

// CTAs of the absorbed form: one an SM (and no unit may have more parts than the join has room for).
int cta_count() { return std::min(sm_count_current(), kMostParts); }

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
    w.bytes = w.desc + al(static_cast<size_t>(ctas) * 2 * sizeof(la::Shared));
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

// A rotated part, bf16 [rows][channels] (heads > 0: [rows][heads][channels]); a
// box is 64 channels of `box` rows (of one head), channels beyond the last are
// filled with 0.
bool rotated_map(CUtensorMap *m, const void *data, int channels, int heads, int64_t rows, int64_t head_stride, int64_t row_stride, int box) {
    const auto fn = tensor_map_encoder();
    if (!fn) return false;
    if (rows == 1) row_stride = 64;
    if (heads == 1) head_stride = 64;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(channels), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(heads)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * row_stride), static_cast<cuuint64_t>(2 * head_stride)};
    const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(box), 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, heads > 0 ? 3 : 2, const_cast<void *>(data), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
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

qvg_status launch_expanded(const CUtensorMap (&map)[5], la::Args &a, int grid, int blocks, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const qvg_status s = smem_limit_once(done, reinterpret_cast<const void *>(la::k_expanded_attention), la::kSmem);
    if (s != QVG_OK) return s;
    // two tiles of K at least, then as many half tiles of V as there is room for
    const int room = la::kSmem - 1024 - 2 * a.na * la::kQChunk, A = a.na * la::kKChunk, B = a.nb * la::kChunk;
    a.sb = std::min(la::kMostStages, (room - 2 * A) / B);
    a.sa = std::min(la::kMostStages, (room - a.sb * B) / A);
    la::k_expanded_attention<<<grid, la::kPromptWarps * 32, la::kSmem, st>>>(map[0], map[1], map[2], map[3], map[4], a, blocks);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

template <int DC>
qvg_status launch_merge(const la::Args &a, int ctas, cudaStream_t st) {
    const cudaError_t e = launch_pdl(k_latent_merge<DC>, dim3(ctas, 2 * kJoinY), dim3(kJoinWarps * 32), 0, st, a);
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
    *bytes = carve(cta_count(), dc).bytes;
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
    if (B > kMostSequences || static_cast<int64_t>(max_q) * Hq > INT32_MAX - la::kRows ||
        static_cast<int64_t>(cache->num_pages) * cache->page_size > INT32_MAX)
        return QVG_ERR_UNSUPPORTED;
    const int ctas = cta_count();
    const Workspace w = carve(ctas, dc);
    if (!workspace || ws_bytes < w.bytes || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return QVG_ERR_WORKSPACE;
    const int64_t slots = static_cast<int64_t>(cache->num_pages) * cache->page_size;
    const int box = std::min(cache->page_size, la::kKeys);
    CUtensorMap map[2] = {};
    // (a page that holds a whole tile is copied in one go, a smaller one chunk by chunk)
    if (!chunk_map(&map[0], cache->c, dc, 0, slots, 0, dc, box, box == la::kKeys ? dc / 64 : 1) ||
        (dr > 0 && !rotated_map(&map[1], cache->kr, dr, 0, slots, 0, dr, box)))
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
    a.wide_out = reinterpret_cast<uintptr_t>(out) % 32 == 0;
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
    if (B > kMostSequences || max_q > INT32_MAX - la::kPromptRows || total_k > INT32_MAX - la::kKeys) return QVG_ERR_UNSUPPORTED;
    const int blocks = ceil_div(max_q, la::kPromptRows);
    const int64_t grid = la::pair_count(B, blocks, total_q) * H;
    if (grid > INT32_MAX) return QVG_ERR_UNSUPPORTED;
    CUtensorMap map[5] = {};
    if (!chunk_map(&map[0], q->data, dn, H, total_q, q->head_stride, q->token_stride, la::kRows, dn / 64) ||
        (dr > 0 && !rotated_map(&map[1], q_rope->data, dr, H, total_q, q_rope->head_stride, q_rope->token_stride, la::kRows)) ||
        (total_k > 0 && (!chunk_map(&map[2], k->data, dn, H, total_k, k->head_stride, k->token_stride, la::kPromptKeys, dn / 64) ||
                         (dr > 0 && !rotated_map(&map[3], k_rope->data, dr, 0, total_k, 0, k_rope->token_stride, la::kPromptKeys)) ||
                         !chunk_map(&map[4], v->data, dv, H, total_k, v->head_stride, v->token_stride, la::kKeys, dv / 64))))
        return QVG_ERR_CUDA;
    la::Args a{};
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
    a.wide_out = reinterpret_cast<uintptr_t>(out) % 32 == 0;
    a.err = device_error_word();
    a.wait_ns = wait_limit_ns();
    a.inject = wait_inject();
    return launch_expanded(map, a, static_cast<int>(grid), blocks, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
