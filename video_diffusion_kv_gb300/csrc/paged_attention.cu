// paged_attention.cu -- attention over a paged cache: launch, the join of
// units that several CTAs shared, the mask rows of drafted trees, and the
// entry points.  The kernel is in paged_attention.cuh.
#include <cmath>

#include "paged_attention_wide.cuh"

namespace qvg {

namespace {

// The unit that begins in CTA i and goes on to CTA `last` left one partial
// sum per CTA: slot 1 of CTA i, slot 0 of the others.  With references m_z,
// sums l_z and O_z: m = max m_z, l = sum l_z 2^(m_z - m), O likewise.  One
// warp per query row; lane z weighs part z, then the lanes share the channels
// and go through the parts in CTA order (32 at a time, the loads of eight in
// flight), so the result is the same each time.
template <int D, int NB>
__global__ void __launch_bounds__(256) k_paged_merge(const __grid_constant__ pa::Args a) {
    constexpr int E = D / 32;
    pdl_wait();
    const int4 u = a.desc[blockIdx.x];
    if (u.x < 0) return;
    const int n = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const pa::Seq s = pa::seq_of<NB>(a, u.x, false);
    const long long gi = static_cast<long long>(u.z) * NB + n;
    const int tq = static_cast<int>(gi / a.grp), j = static_cast<int>(gi - static_cast<long long>(tq) * a.grp);
    if (tq >= s.nq) return;
    const int first = blockIdx.x, last = min(u.w, static_cast<int>(gridDim.x) - 1);
    auto at = [&](int z) { return static_cast<size_t>(2 * z + (z == first ? 1 : 0)) * NB + n; };
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
        // in two factors: references follow V's scale, and may lie further apart than fp32's range reaches while l_z
        // still counts (up to 2^120 apart the second is 1); 0: no key of this part is seen
        const float e = lz == 0.0f ? -INFINITY : a.pm[at(z)] - m, e1 = fmaxf(e, -120.0f);
        const float w1 = exp2f(e1), w2 = exp2f(e - e1), w = w1 * w2;
        lz = lz * w1 * w2;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lz += __shfl_xor_sync(0xFFFFFFFFu, lz, o);
        l += lz;
        const int parts = min(32, last - z0 + 1);
#pragma unroll 8
        for (int k = 0; k < parts; ++k) {
            const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
            const float *o = a.po + at(z0 + k) * D + lane * E;
            if (wk != 0.0f) {
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(wk, o[e], acc[e]);
            }
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const long long row = static_cast<long long>(s.q0 + tq) * a.Hq + u.y * a.grp + j;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (a.out32)
            a.out32[row * D + lane * E + e] = acc[e] * inv;
        else
            a.out16[row * D + lane * E + e] = f32_to_bf16(acc[e] * inv);
    }
    if (lane == 0 && a.lse)
        a.lse[(row % a.Hq) * a.total_q + row / a.Hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// One block per sequence: parents in shared memory, a thread walks up from
// its token.  A parent is below its child, so a walk has at most T steps and
// meets the row's words in falling order: each is written once it is left.
// What bounds it is the walk (one shared load a step), T of them for a chain.
__global__ void k_tree_mask(const int32_t *__restrict__ parents, const int32_t *__restrict__ cu_q, int max_q, int total_q,
                            int words, uint32_t *__restrict__ mask, int *err) {
    extern __shared__ int32_t s_up[];
    const int b = blockIdx.x;
    const long long q0 = cu_q ? cu_q[b] : static_cast<long long>(b) * max_q;
    const long long all = cu_q ? static_cast<long long>(cu_q[b + 1]) - q0 : max_q;
    const bool good = q0 >= 0 && all >= 0 && q0 + all <= total_q;
    const int n = good ? static_cast<int>(min(all, static_cast<long long>(max_q))) : 0;
    if (threadIdx.x == 0 && (!good || all > max_q)) raise_error(err, QVG_ERR_INVALID_ARG);
    for (int t = threadIdx.x; t < n; t += blockDim.x) {
        int p = parents[q0 + t];
        if (p < -1 || p >= t) {
            raise_error(err, QVG_ERR_INVALID_ARG);
            p = -1;
        }
        s_up[t] = p;
    }
    __syncthreads();
    for (int t = threadIdx.x; t < n; t += blockDim.x) {
        uint32_t *row = mask + (q0 + t) * words;
        int j = t;
        for (int w = words - 1; w >= 0; --w) {
            uint32_t m = 0;
            for (; j >= 32 * w; j = s_up[j]) m |= 1u << (j & 31);
            row[w] = m;
        }
    }
}

constexpr int kMaxTree = 8192;  // new tokens of one sequence whose parents fit 32 KB of shared memory

// Query rows of a unit, from a sequence's rows (max_q new tokens times the
// query heads of a KV head): 16 or 32 (narrow kernel) up to two blocks of
// them, else 256 (wide kernel), whose time hardly depends on them.  4-bit caches
// have no blocks of 32: the narrow kernel's converters need registers too.
// Microseconds for 16 sequences of 2,000 to 12,000 keys (8 KV heads, d = 128):
//            rows     16   32   64   96  128
//   8 bits   16       62   89  148
//            32       74   81  124  171  214
//            256     137  141  147  152  158
//   4 bits   16       87  146  260
//            256     186  191  195  200  203
// At the borders, 64 rows of 8 bits (32 each) and 32 rows of 4 bits (16 each)
// against 256: d = 64: 101 against 125, 100 against 153; 48 sequences: 311 against 382,
// 386 against 516; one sequence of 150,000: 125 against 168, 175 against 220.  Only where a
// call is as short as its launch is the order the other way (40 sequences of 300
// to 2,000, 2 KV heads: 50 against 41, 44 against 41).
int rows_of_block(long long rows, int bits) {
    return rows <= (bits == 8 ? 16 : 32) ? 16 : rows <= 64 && bits == 8 ? 32 : pa::kWideRows;
}

// The narrow kernel has two CTAs an SM, the wide one has one.
int cta_count(int NB) { return (NB == pa::kWideRows ? 1 : 2) * sm_count_current(); }

struct Workspace {
    size_t po, pm, pl, desc, bytes;  // offsets
};
Workspace carve(int ctas, int NB, int d) {
    auto al = [](size_t b) { return (b + 255) & ~static_cast<size_t>(255); };
    const size_t rows = static_cast<size_t>(ctas) * 2 * NB;
    Workspace w{};
    w.pm = al(rows * d * 4);
    w.pl = w.pm + al(rows * 4);
    w.desc = w.pl + al(rows * 4);
    w.bytes = w.desc + al(static_cast<size_t>(ctas) * sizeof(int4));
    return w;
}

// A tensor's 8-bit codes as [pages][H][page][d] bytes; a box is one page's rows
// of a head (at most 128), swizzled as the tensor core reads them.
bool codes_map(CUtensorMap *m, const qvg_paged *c, const uint8_t *codes) {
    const auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t d = static_cast<cuuint64_t>(c->d), pg = static_cast<cuuint64_t>(c->page_size);
    const cuuint64_t dims[4] = {d, pg, static_cast<cuuint64_t>(c->H), static_cast<cuuint64_t>(c->num_pages)};
    const cuuint64_t strides[3] = {d, d * pg, d * pg * static_cast<cuuint64_t>(c->H)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(c->d), static_cast<cuuint32_t>(std::min(c->page_size, 128)), 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(codes), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, c->d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NB>
qvg_status launch_merge(const pa::Args &a, int ctas, cudaStream_t st) {
    const cudaError_t e = launch_pdl(k_paged_merge<D, NB>, dim3(ctas, NB / 8), dim3(256), 0, st, a);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        note_cuda_error(e);
        return QVG_ERR_CUDA;
    }
    return QVG_OK;
}

template <int D, int BITS, int NB>
qvg_status launch(const CUtensorMap (&map)[2], const pa::Args &a, int ctas, cudaStream_t st) {
    using C = pa::Cfg<D, BITS, NB>;
    static std::atomic<uint64_t> done{0};
    const qvg_status s = smem_limit_once(done, reinterpret_cast<const void *>(pa::k_paged_attention<D, BITS, NB>), C::kSmem);
    if (s != QVG_OK) return s;
    pa::k_paged_attention<D, BITS, NB><<<ctas, C::kWarps * 32, C::kSmem, st>>>(map[0], map[1], a);
    QVG_LAUNCH_CHECK();
    return launch_merge<D, NB>(a, ctas, st);
}

template <int D, int BITS>
qvg_status launch_wide(const CUtensorMap (&map)[2], const pa::Args &a, int ctas, cudaStream_t st) {
    using C = pa::Wide<D, BITS>;
    static std::atomic<uint64_t> done{0};
    const void *kernel = reinterpret_cast<const void *>(pa::k_paged_attention_wide<D, BITS>);
    const qvg_status s = smem_limit_once(done, kernel, C::kSmem);
    if (s != QVG_OK) return s;
    // The kernel's register split is made for what it is compiled to have at
    // launch: with fewer, its softmax warps would wait for registers that never
    // come.
    static std::atomic<int> regs{0};
    int n = regs.load(std::memory_order_acquire);
    if (n == 0) {
        cudaFuncAttributes at{};
        const cudaError_t e = cudaFuncGetAttributes(&at, kernel);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            note_cuda_error(e);
            return QVG_ERR_CUDA;
        }
        regs.store(n = at.numRegs, std::memory_order_release);
    }
    if (n != pa::kWideRegs) return QVG_ERR_UNSUPPORTED;
    pa::k_paged_attention_wide<D, BITS><<<ctas, C::kWarps * 32, C::kSmem, st>>>(map[0], a);
    QVG_LAUNCH_CHECK();
    return launch_merge<D, pa::kWideRows>(a, ctas, st);
}

bool misaligned(const void *p, uintptr_t to) { return !p || reinterpret_cast<uintptr_t>(p) % to != 0; }

}  // namespace
}  // namespace qvg

using namespace qvg;

extern "C" {

qvg_status qvg_tree_mask(const int32_t *parents, const int32_t *cu_q, int32_t B, int32_t max_q, int32_t total_q,
                         int32_t words, uint32_t *mask, void *stream) {
    if (B < 0 || max_q < 0 || total_q < 0 || words < ceil_div(max_q, 32)) return QVG_ERR_INVALID_ARG;
    if (!cu_q && static_cast<int64_t>(B) * max_q > total_q) return QVG_ERR_INVALID_ARG;
    if (max_q > kMaxTree) return QVG_ERR_UNSUPPORTED;
    if (B == 0 || max_q == 0) return QVG_OK;
    if (misaligned(parents, 4) || misaligned(mask, 4) || (cu_q && misaligned(cu_q, 4))) return QVG_ERR_INVALID_ARG;
    const int threads = std::min(1024, ceil_div(max_q, 32) * 32);
    k_tree_mask<<<B, threads, static_cast<size_t>(max_q) * sizeof(int32_t), static_cast<cudaStream_t>(stream)>>>(
        parents, cu_q, max_q, total_q, words, mask, device_error_word());
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

qvg_status qvg_paged_workspace_size(int32_t H, int32_t d, int32_t Hq, int32_t B, int32_t max_q, size_t *bytes) {
    if (!bytes || H < 1 || Hq < 1 || Hq % H != 0 || B < 0 || max_q < 0) return QVG_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return QVG_ERR_UNSUPPORTED;
    *bytes = 0;  // (of a cache of either bit width)
    for (int bits = 4; bits <= 8; bits += 4) {
        const int NB = rows_of_block(static_cast<long long>(max_q) * (Hq / H), bits);
        *bytes = std::max(*bytes, carve(cta_count(NB), NB, d).bytes);
    }
    return QVG_OK;
}

qvg_status qvg_paged_attention(const qvg_paged *cache, const void *q_bf16, int64_t q_stride, int32_t total_q,
                               int32_t Hq, int32_t B, int32_t max_q, const int32_t *cu_q, const int32_t *table,
                               int32_t table_stride, const int32_t *kv_len, int32_t mask_mode,
                               const uint32_t *mask, int32_t mask_words, float scale, void *out,
                               int32_t out_dtype, float *lse, void *workspace, size_t ws_bytes, void *stream) {
    qvg_status s = check_paged(cache, false);
    if (s != QVG_OK) return s;
    const int H = cache->H, d = cache->d;
    if (Hq < 1 || Hq % H != 0 || B < 0 || max_q < 0 || total_q < 0 || table_stride < 1) return QVG_ERR_INVALID_ARG;
    if (q_stride < static_cast<int64_t>(Hq) * d || q_stride % 8 != 0) return QVG_ERR_INVALID_ARG;
    if (mask_mode != QVG_MASK_NONE && mask_mode != QVG_MASK_CAUSAL && mask_mode != QVG_MASK_TREE) return QVG_ERR_INVALID_ARG;
    if (out_dtype != QVG_OUT_F32 && out_dtype != QVG_OUT_BF16) return QVG_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return QVG_ERR_INVALID_ARG;
    if (!cu_q && static_cast<int64_t>(B) * max_q > total_q) return QVG_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_q) * (Hq / H) > INT32_MAX - pa::kWideRows) return QVG_ERR_UNSUPPORTED;
    if (B == 0 || max_q == 0 || total_q == 0) return QVG_OK;
    if (misaligned(q_bf16, 16) || misaligned(out, 16) || misaligned(table, 4) || misaligned(kv_len, 4) ||
        (cu_q && misaligned(cu_q, 4)) || (lse && misaligned(lse, 4)))
        return QVG_ERR_INVALID_ARG;
    if (mask_mode == QVG_MASK_TREE && (misaligned(mask, 4) || mask_words < ceil_div(max_q, 32))) return QVG_ERR_INVALID_ARG;
    const int NB = rows_of_block(static_cast<long long>(max_q) * (Hq / H), cache->bits), ctas = cta_count(NB);
    const Workspace w = carve(ctas, NB, d);
    if (!workspace || ws_bytes < w.bytes || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return QVG_ERR_WORKSPACE;
    CUtensorMap map[2] = {};
    if (cache->bits == 8 && (!codes_map(&map[0], cache, cache->k_codes) || !codes_map(&map[1], cache, cache->v_codes)))
        return QVG_ERR_CUDA;
    pa::Args a{};
    a.q = static_cast<const uint16_t *>(q_bf16);
    a.q_stride = q_stride;
    a.total_q = total_q;
    a.Hq = Hq;
    a.H = H;
    a.grp = Hq / H;
    a.B = B;
    a.max_q = max_q;
    a.cu_q = cu_q;
    a.table = table;
    a.kv_len = kv_len;
    a.table_stride = table_stride;
    a.mode = mask_mode;
    a.mask = mask;
    a.words = mask_words;
    a.scale_log2 = (scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(d))) * 1.4426950408889634f;
    a.out32 = out_dtype == QVG_OUT_F32 ? static_cast<float *>(out) : nullptr;
    a.out16 = out_dtype == QVG_OUT_BF16 ? static_cast<uint16_t *>(out) : nullptr;
    a.lse = lse;
    a.kc = cache->k_codes;
    a.ks = cache->k_scales;
    a.vc = cache->v_codes;
    a.vs = cache->v_scales;
    a.page_log2 = __builtin_ctz(static_cast<unsigned>(cache->page_size));
    a.num_pages = cache->num_pages;
    char *base = static_cast<char *>(workspace);
    a.po = reinterpret_cast<float *>(base + w.po);
    a.pm = reinterpret_cast<float *>(base + w.pm);
    a.pl = reinterpret_cast<float *>(base + w.pl);
    a.desc = reinterpret_cast<int4 *>(base + w.desc);
    a.err = device_error_word();
    a.wait_ns = wait_limit_ns();
    a.inject = wait_inject();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (NB == pa::kWideRows) {
        if (cache->bits == 4) return d == 64 ? launch_wide<64, 4>(map, a, ctas, st) : launch_wide<128, 4>(map, a, ctas, st);
        return d == 64 ? launch_wide<64, 8>(map, a, ctas, st) : launch_wide<128, 8>(map, a, ctas, st);
    }
    if (cache->bits == 4) return d == 64 ? launch<64, 4, 16>(map, a, ctas, st) : launch<128, 4, 16>(map, a, ctas, st);
    if (NB == 16) return d == 64 ? launch<64, 8, 16>(map, a, ctas, st) : launch<128, 8, 16>(map, a, ctas, st);
    return d == 64 ? launch<64, 8, 32>(map, a, ctas, st) : launch<128, 8, 32>(map, a, ctas, st);
}

}  // extern "C"
