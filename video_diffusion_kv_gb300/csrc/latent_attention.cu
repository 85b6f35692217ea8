// latent_attention.cu -- attention over a latent cache (absorbed form) and of
// prompts (expanded form): a first form, one warp per query row and head.
#include <cmath>

#include "latent.cuh"

namespace qvg {
namespace {

struct Args {
    const uint16_t *q, *qr, *k, *kr, *v;
    long long q_t, q_h, qr_t, qr_h, k_t, k_h, kr_t, v_t, v_h;
    int total_q, total_k, Hq, dk, dr, dv, B, max_q, max_k;
    const int32_t *cu_q, *cu_k, *table, *kv_len;
    long long table_stride;
    int page_log2, num_pages;
    int mode;
    const uint32_t *mask;
    int words;
    float scale_log2;
    float *out32;
    uint16_t *out16;
    float *lse;
    int *err;
};

// Row t of sequence b: blockIdx.x = (b, t), a warp per head.
__global__ void __launch_bounds__(128) k_rows(Args a) {
    const int lane = threadIdx.x & 31, h = blockIdx.y * 4 + (threadIdx.x >> 5);
    const int b = blockIdx.x / a.max_q, t = blockIdx.x - b * a.max_q;
    int q0 = b * a.max_q, nq = a.max_q, k0 = b * a.max_k, kv = a.max_k;
    bool bad = false;
    if (a.cu_q) {
        q0 = a.cu_q[b];
        nq = a.cu_q[b + 1] - q0;
        bad = nq < 0 || nq > a.max_q || q0 < 0 || q0 > a.total_q - nq;
        if (q0 < 0 || q0 > a.total_q) q0 = nq = 0;
        nq = max(0, min(min(nq, a.max_q), a.total_q - q0));
    }
    if (a.table) {
        kv = a.kv_len[b];
        bad = bad || kv < 0 || kv > a.table_stride << a.page_log2;
        kv = static_cast<int>(max(0ll, min(static_cast<long long>(kv), a.table_stride << a.page_log2)));
    } else if (a.cu_k) {
        k0 = a.cu_k[b];
        kv = a.cu_k[b + 1] - k0;
        bad = bad || kv < 0 || k0 < 0 || k0 > a.total_k - kv;
        if (k0 < 0 || k0 > a.total_k) k0 = kv = 0;
        kv = max(0, min(kv, a.total_k - k0));
    }
    if (bad && t == 0 && h == 0 && lane == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
    if (t >= nq || h >= a.Hq) return;
    float q[8], qr[4], acc[8], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = lane + 32 * i;
        q[i] = c < a.dk ? bf16_to_f32(a.q[(q0 + t) * a.q_t + h * a.q_h + c]) : 0.0f;
        acc[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = lane + 32 * i;
        qr[i] = c < a.dr ? bf16_to_f32(a.qr[(q0 + t) * a.qr_t + h * a.qr_h + c]) : 0.0f;
    }
    const int hist = kv - nq;
    for (int j = 0; j < kv; ++j) {
        if (a.mode == QVG_MASK_CAUSAL && j > hist + t) break;
        if (a.mode == QVG_MASK_TREE && j >= hist) {
            const int i = j - hist;
            if (!((a.mask[static_cast<long long>(q0 + t) * a.words + (i >> 5)] >> (i & 31)) & 1u)) continue;
        }
        long long at = k0 + j;
        if (a.table) {
            const int page = a.table[b * a.table_stride + (j >> a.page_log2)];
            if (page < 0 || page >= a.num_pages) {
                raise_error(a.err, QVG_ERR_INVALID_ARG);
                continue;
            }
            at = (static_cast<long long>(page) << a.page_log2) + (j & ((1 << a.page_log2) - 1));
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < a.dk) s = fmaf(q[i], bf16_to_f32(a.k[at * a.k_t + h * a.k_h + lane + 32 * i]), s);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < a.dr) s = fmaf(qr[i], bf16_to_f32(a.kr[at * a.kr_t + lane + 32 * i]), s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        s *= a.scale_log2;
        const float top = fmaxf(m, s), f = m == -INFINITY ? 0.0f : exp2f(m - top), p = exp2f(s - top);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < a.dv) acc[i] = fmaf(p, bf16_to_f32(a.v[at * a.v_t + h * a.v_h + lane + 32 * i]), acc[i] * f);
        m = top;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const long long row = static_cast<long long>(q0 + t) * a.Hq + h;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = lane + 32 * i;
        if (c >= a.dv) continue;
        if (a.out32)
            a.out32[row * a.dv + c] = acc[i] * inv;
        else
            a.out16[row * a.dv + c] = f32_to_bf16(acc[i] * inv);
    }
    if (lane == 0 && a.lse)
        a.lse[static_cast<long long>(h) * a.total_q + q0 + t] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

bool misaligned(const void *p, uintptr_t to) { return !p || reinterpret_cast<uintptr_t>(p) % to != 0; }

// A view's data and strides (channels: of a head; heads and tokens: how many the call takes).
bool view_ok(const qvg_view *v, int channels, int64_t tokens, int heads) {
    if (!v || misaligned(v->data, 16)) return false;
    if (tokens > 1 && (v->token_stride < channels || v->token_stride % 8 != 0)) return false;
    return heads <= 1 || (v->head_stride >= channels && v->head_stride % 8 == 0);
}

qvg_status launch(const Args &a, cudaStream_t st) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.max_q;
    if (rows > INT32_MAX) return QVG_ERR_UNSUPPORTED;
    k_rows<<<dim3(static_cast<unsigned>(rows), ceil_div(a.Hq, 4)), 128, 0, st>>>(a);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
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
    *bytes = 256;
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
    if (!workspace || ws_bytes < 256 || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return QVG_ERR_WORKSPACE;
    Args a{};
    a.q = static_cast<const uint16_t *>(q->data);
    a.q_t = q->token_stride;
    a.q_h = q->head_stride;
    if (dr > 0) {
        a.qr = static_cast<const uint16_t *>(q_rope->data);
        a.qr_t = q_rope->token_stride;
        a.qr_h = q_rope->head_stride;
    }
    a.k = a.v = static_cast<const uint16_t *>(cache->c);
    a.kr = static_cast<const uint16_t *>(cache->kr);
    a.k_t = a.v_t = dc;
    a.kr_t = dr;
    a.total_q = total_q;
    a.Hq = Hq;
    a.dk = a.dv = dc;
    a.dr = dr;
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
    a.err = device_error_word();
    return launch(a, static_cast<cudaStream_t>(stream));
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
    Args a{};
    a.q = static_cast<const uint16_t *>(q->data);
    a.q_t = q->token_stride;
    a.q_h = q->head_stride;
    if (total_k > 0) {
        a.k = static_cast<const uint16_t *>(k->data);
        a.k_t = k->token_stride;
        a.k_h = k->head_stride;
        a.v = static_cast<const uint16_t *>(v->data);
        a.v_t = v->token_stride;
        a.v_h = v->head_stride;
    }
    if (dr > 0) {
        a.qr = static_cast<const uint16_t *>(q_rope->data);
        a.qr_t = q_rope->token_stride;
        a.qr_h = q_rope->head_stride;
        if (total_k > 0) {
            a.kr = static_cast<const uint16_t *>(k_rope->data);
            a.kr_t = k_rope->token_stride;
        }
    }
    a.total_q = total_q;
    a.total_k = total_k;
    a.Hq = H;
    a.dk = dn;
    a.dv = dv;
    a.dr = dr;
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
    return launch(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
