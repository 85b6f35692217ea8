// bf16_attention.cuh -- pieces shared by the attention kernels with bf16
// operands: over a latent cache (latent_attention.cuh) and of prompts
// (expanded_attention.cuh).
//
//   S [128 rows x keys] = Q K^T   K-major tiles of 64 channels, 128-byte
//                                 swizzle, as the copies write them
//   O [128 rows x dv]  += P V     P in bf16 in tensor memory, over its S
//
// A softmax thread owns a row and takes 64 keys at a time.  A row's reference
// is raised only where a logit passes it by 2^8 (then O is rescaled first,
// after the product in flight).
//
// Keys that some row does not see, and slots past the sequence's end, may hold
// anything, also NaN, and a weight of 0 times NaN is not 0: in the tiles that
// have such keys the helper warps look at V before the products read it, and
// set rows that lie past the end or hold an infinity or a NaN to 0; the latter
// are marked, and the rows of Q that see them become NaN by their logits.
#pragma once

#include "latent.cuh"
#include "paged_attention.cuh"

namespace qvg {
namespace la {

constexpr int kKeys = 64, kRows = 128;       // a tile's keys, a group's rows
constexpr int kChunk = kKeys * 128;          // 64 channels of a tile's keys
constexpr int kQChunk = kRows * 128;         // 64 channels of a group's rows
constexpr int kMostStages = 8, kFix = 8;     // kFix >= kMostStages: the helpers are never further ahead
constexpr int kSmem = 230400;                // dynamic shared memory, 1024 of it for alignment
constexpr float kRaise = 8.0f;               // a reference is raised where a weight would pass 2^8

struct Args : pa::Args {
    const uint16_t *qr;  // (q: the part of the queries before the rotated one)
    long long q_h, qr_t, qr_h;  // (q_stride: q's token stride)
    int dk, dr, dv;      // channels of q; of the rotated part; of v
    int na, nb;          // 64-channel chunks of a tile: read by S alone (the rotated part; expanded form: all of K), and V's
    int sa, sb;          // stages of the rings of both (absorbed form: sb stages of both)
    bool wide_out;       // out is 32-byte aligned
    // expanded form
    const int32_t *cu_k;
    int total_k, max_k;
};

// Position in a ring and the parity of its current use.
struct Ring {
    int i = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            parity ^= 1u;
        }
    }
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void *map, int c0, int c1, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(umma::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *map, int c0, int c1, int c2, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(umma::smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *map, int c0, int c1, int c2, int c3, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(umma::smem_u32(bar))
        : "memory");
}

// The issuing warps stay whole and name the thread that issues by a predicate, so that
// addresses and counts are the same for the warp as the compiler sees it (4680 causal tokens of
// 16 heads: 149 us where `if (lane == 0)` took 213, when this was changed).
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc, bool one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc), "r"(one ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc, bool one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc), "r"(one ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar, bool one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(umma::smem_u32(bar)),
        "r"(one ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Which of the tile's 64 keys the row of new token tq sees, as bits.
__device__ __forceinline__ uint2 seen_keys(const Args &a, int t, int kv, int nq, int q0, int tq) {
    const int k0 = t * kKeys, hist = kv - nq;
    int end = min(kv - k0, kKeys);  // keys of the sequence in this tile
    if (a.mode == QVG_MASK_CAUSAL) end = min(end, hist + tq + 1 - k0);
    const uint32_t *m = a.mask + static_cast<long long>(q0 + tq) * a.words;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int n = end - 32 * i;
        uint32_t x = n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
        const int j = 32 * i + k0 - hist;  // the word's first key among the new tokens (below 0: history)
        if (a.mode == QVG_MASK_TREE && x != 0u && j > -32) {
            if (j < 0) {
                x &= (m[0] << -j) | ((1u << -j) - 1u);
            } else {
                const int k = j >> 5, s = j & 31;
                const uint32_t lo = k < a.words ? m[k] : 0u, hi = k + 1 < a.words ? m[k + 1] : 0u;
                x &= __funnelshift_r(lo, hi, s);
            }
        }
        w[i] = x;
    }
    return make_uint2(w[0], w[1]);
}

// A warp's rows of O, dv channels, times their factors.
__device__ __forceinline__ void rescale_rows(uint32_t t_o, int dv, float f) {
#pragma unroll 1
    for (int c = 0; c < dv; c += 16) {
        uint32_t o[16];
        pa::tmem_ld16(t_o + c, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        umma::tmem_st16(t_o + c, o);
    }
    umma::tmem_st_wait();
}

// A row's softmax so far: its reference (of the logits as S has them) and the
// sum of its weights, in four parts; whether it has seen a key.
struct Row {
    float ref = -INFINITY;
    bool saw = false;
    uint64_t l2[2] = {0, 0};
    __device__ __forceinline__ float sum() const {
        float a, b, c, d;
        pa::up2(l2[0], a, b);
        pa::up2(l2[1], c, d);
        return (a + b) + (c + d);
    }
    // Keys, and every logit -inf, the value of keys that are not seen: an infinity in q (each key turns it to -inf) or
    // sums beyond fp32.  The softmax has no value; without this the row would come out as one without keys.
    __device__ __forceinline__ bool lost() const { return saw && ref == -INFINITY; }
};
// Stands for the reference of a partial sum whose row is lost: weighs nothing beside others, and tells a
// row without weights that has keys from one without.
constexpr float kLost = -3.402823466e38f;

// 64 keys of a warp's rows, in three steps: the logits at t_s, with those that
// the row does not see at -inf; the largest; weights in the logits' place.
using Logits = uint32_t[2][32];

// part: some row does not see all of them (see: which this row does, bad: marked keys).
__device__ __forceinline__ void read_logits(Logits &v, uint32_t t_s, bool part, uint2 see, uint2 bad) {
    umma::tmem_ld32(t_s, v[0]);
    umma::tmem_ld32(t_s + 32, v[1]);
    umma::tmem_ld_wait_regs(v[0]);
    umma::reg_fence32(v[1]);
    if (part) {
        const uint32_t sw[2] = {see.x, see.y}, bw[2] = {see.x & bad.x, see.y & bad.y};
#pragma unroll
        for (int c = 0; c < kKeys; ++c)
            if (!((sw[c / 32] >> (c & 31)) & 1u)) v[c / 32][c % 32] = 0xFF800000u;
        if (bw[0] | bw[1]) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c)
                if ((bw[c / 32] >> (c & 31)) & 1u) v[c / 32][c % 32] = 0x7FFFFFFFu;
        }
    }
}
__device__ __forceinline__ float largest(const Logits &v) {
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < kKeys; c += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top[i] = fmaxf(fmaxf(top[i], __uint_as_float(v[c / 32][c % 32 + 2 * i])), __uint_as_float(v[c / 32][c % 32 + 2 * i + 1]));
    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}
// Raises the reference where the largest logit asks for it; what O has to be multiplied with.
__device__ __forceinline__ float raise_ref(const Args &a, Row &m, float top, bool live) {
    const bool fresh = m.ref == -INFINITY;
    const bool move = live && (fresh ? top > -INFINITY : (top - m.ref) * a.scale_log2 > kRaise);
    const float f = move && !fresh ? pa::ex2((m.ref - top) * a.scale_log2) : 1.0f;
    if (move) m.ref = top;
    return f;
}
__device__ __forceinline__ void write_weights(const Args &a, Row &m, const Logits &v, uint32_t t_s, float f) {
    const float nm = m.ref == -INFINITY ? 0.0f : -m.ref * a.scale_log2;
    const uint64_t sl2 = pa::pk2(a.scale_log2, a.scale_log2), nm2 = pa::pk2(nm, nm), f2 = pa::pk2(f, f);
    m.l2[0] = pa::mul2(m.l2[0], f2);
    m.l2[1] = pa::mul2(m.l2[1], f2);
    uint32_t w[32];
#pragma unroll
    for (int c = 0; c < kKeys; c += 2) {
        float y0, y1;
        pa::up2(pa::fma2(pa::pk2(__uint_as_float(v[c / 32][c % 32]), __uint_as_float(v[c / 32][c % 32 + 1])), sl2, nm2), y0, y1);
        y0 = pa::ex2(y0);
        y1 = pa::ex2(y1);
        m.l2[(c / 2) & 1] = pa::add2(m.l2[(c / 2) & 1], pa::pk2(y0, y1));
        w[c / 2] = bf16x2(y0, y1);
    }
    umma::tmem_st32(t_s, w);
    umma::tmem_st_wait();
}

// 32 bytes, 32-byte aligned.
__device__ __forceinline__ void store32(void *p, const uint32_t (&x)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]),
                 "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// A warp's rows of O: the result (whole), or a partial sum with its reference
// and the sum of its weights.  none: no product has been made.  A partial sum
// lies as [dv / 4][128 rows][4], so that a warp's stores are whole lines
// (as rows, 128 of them took 6 us; so 3).
__device__ __forceinline__ void store_rows(const Args &a, const Row &m, uint32_t t_o, bool none, bool live, bool whole, long long slot, int r,
                                           long long row, int h, int token) {
    const float ref = m.ref * a.scale_log2, l = whole && m.lost() ? __uint_as_float(0x7FFFFFFFu) : m.sum();
    if (live && !whole) {
        a.pm[slot * kRows + r] = m.lost() ? kLost : ref;
        a.pl[slot * kRows + r] = l;
    } else if (live && a.lse) {
        a.lse[static_cast<long long>(h) * a.total_q + token] = l == 0.0f ? -INFINITY : (log2f(l) + ref) * 0.69314718055994531f;
    }
    const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
    float *part = a.po + slot * kRows * a.dv + 4 * r;
    const bool wide = a.wide_out;
#pragma unroll 1
    for (int c = 0; c < a.dv; c += 32) {
        uint32_t o[32];
        if (none) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
        } else {
            umma::tmem_ld32(t_o + c, o);
            umma::tmem_ld_wait_regs(o);
        }
        if (!live) continue;
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4 *>(part + (c / 4 + i) * (4 * kRows)) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else if (a.out16) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = bf16x2(__uint_as_float(o[16 * k + 2 * i]) * inv, __uint_as_float(o[16 * k + 2 * i + 1]) * inv);
                uint16_t *dst = a.out16 + row * a.dv + c + 16 * k;
                if (wide) {
                    store32(dst, y);
                } else {
                    reinterpret_cast<uint4 *>(dst)[0] = make_uint4(y[0], y[1], y[2], y[3]);
                    reinterpret_cast<uint4 *>(dst)[1] = make_uint4(y[4], y[5], y[6], y[7]);
                }
            }
        } else {
            float4 *dst = reinterpret_cast<float4 *>(a.out32 + row * a.dv + c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dst[i] = make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv, __uint_as_float(o[4 * i + 2]) * inv,
                                     __uint_as_float(o[4 * i + 3]) * inv);
        }
    }
}

// A helper warp's look at keys [k0, k0 + 16) of 64 keys of V (nb chunks at `v`),
// two threads a key.  `left`: keys before the sequence's end.  Returns the
// marks, key i at bit i.
__device__ __forceinline__ uint32_t clean16(uint8_t *v, int nb, int k0, int left) {
    const int lane = threadIdx.x & 31, row = k0 + (lane >> 1);
    uint8_t *line = v + row * 128 + (lane & 1) * 64;
    bool bad = false;
    for (int c = 0; c < nb; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 x = *reinterpret_cast<const uint4 *>(line + c * kChunk + 16 * i);
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) bad = bad || (y[e] & 0x7F80u) == 0x7F80u || (y[e] & 0x7F800000u) == 0x7F800000u;
        }
    bad = __shfl_xor_sync(0xFFFFFFFFu, bad, 1) || bad;
    const bool past = row >= left;
    if (past || bad) {
        for (int c = 0; c < nb; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(line + c * kChunk + 16 * i) = make_uint4(0, 0, 0, 0);
    }
    umma::fence_proxy_async_smem();
    uint32_t b = __ballot_sync(0xFFFFFFFFu, bad && !past) & 0x55555555u;  // every other bit, moved together
    b = (b | b >> 1) & 0x33333333u;
    b = (b | b >> 2) & 0x0F0F0F0Fu;
    b = (b | b >> 4) & 0x00FF00FFu;
    return (b | b >> 8) & 0xFFFFu;
}

}  // namespace la
}  // namespace qvg
