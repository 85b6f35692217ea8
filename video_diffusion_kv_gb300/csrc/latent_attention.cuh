// latent_attention.cuh -- attention with bf16 operands on the tensor cores: of
// new tokens over a latent cache (absorbed form), and of prompts (expanded
// form).  One kernel, two instances; launch, join and entry points are in
// latent_attention.cu.
//
//   S [128 rows x 64 keys] = Q K^T   K-major tiles of 64 channels, 128-byte
//                                    swizzle, as the copies write them
//   O [128 rows x dv]     += P V     P in bf16 in tensor memory, over its S
//
// Absorbed (LATENT): a row is a (new token, query head) pair.  All heads read
// the same latents, so a unit of work is 128 rows of one sequence, and a tile's
// latents are loaded once for both products: as K, and read across (MN-major)
// as V.  All units' tiles form one line that is cut into equal parts, one per CTA
// (pa::Line); a unit cut by a border leaves fp32 partial sums that
// k_latent_merge joins.
// Expanded: a unit is 256 rows of one head (two groups of 128), so that a tile
// of K and V serves both; one unit per CTA, the longest first.
//
// Roles: a softmax thread owns a row; one thread issues S, another one PV.  S has two
// buffers of 64 columns a group, so that the next tile's S runs while this
// tile's softmax does.  A row's reference is raised only where a logit passes it
// by 2^8 (then O is rescaled first, after the product in flight).
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
    int sa, sb;          // stages of the rings (absorbed form: one ring, whose stages hold both)
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

// The issuing warps stay whole and name the thread that issues by a predicate:
// addresses and counts are then the same for the warp as the compiler sees it, and
// an instruction takes about 25 clocks to issue, where one under `if (lane == 0)` takes 90.
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

// A warp's rows of O times their factors.
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

// The unit of a CTA of the expanded form, and how many tiles each group needs.
struct Unit {
    int b, h, r, q0, nq, k0, kv, nt[2];
};
__device__ __forceinline__ Unit unit_of(const Args &a, int blocks) {
    Unit u;
    const int bh = a.B * a.H, i = blockIdx.x / bh, j = blockIdx.x - i * bh;
    u.r = blocks - 1 - i;  // causal: the last rows see the most keys
    u.b = j / a.H;
    u.h = j - u.b * a.H;
    bool bad = false;
    u.q0 = u.b * a.max_q;
    u.nq = a.max_q;
    if (a.cu_q) {
        u.q0 = a.cu_q[u.b];
        u.nq = a.cu_q[u.b + 1] - u.q0;
        bad = u.nq < 0 || u.nq > a.max_q || u.q0 < 0 || u.q0 > a.total_q - u.nq;
        if (u.q0 < 0 || u.q0 > a.total_q) u.q0 = u.nq = 0;
        u.nq = max(0, min(min(u.nq, a.max_q), a.total_q - u.q0));
    }
    u.k0 = u.b * a.max_k;
    u.kv = a.max_k;
    if (a.cu_k) {
        u.k0 = a.cu_k[u.b];
        u.kv = a.cu_k[u.b + 1] - u.k0;
        bad = bad || u.kv < 0 || u.k0 < 0 || u.k0 > a.total_k - u.kv;
        if (u.k0 < 0 || u.k0 > a.total_k) u.k0 = u.kv = 0;
        u.kv = max(0, min(u.kv, a.total_k - u.k0));
    }
    if (bad && u.r == 0 && u.h == 0 && threadIdx.x == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int first = u.r * 256 + g * kRows, last = min(u.nq, first + kRows);
        const int end = first >= u.nq ? 0 : a.mode == QVG_MASK_CAUSAL ? min(u.kv, u.kv - u.nq + last) : u.kv;
        u.nt[g] = end <= 0 ? 0 : (end - 1) / kKeys + 1;
    }
    return u;
}

// kmap: LATENT the latents, else k; rmap: the rotated key parts; vmap: v (not LATENT).
template <bool LATENT>
__global__ void __launch_bounds__(LATENT ? 384 : 512, 1)
    k_latent_attention(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap rmap,
                       const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a, int blocks) {
    constexpr int G = LATENT ? 1 : 2, W0 = 4 * G, WARPS = W0 + 8;
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t a_full[kMostStages], a_empty[kMostStages], b_full[kMostStages], b_empty[kMostStages], fixed[kFix];
    __shared__ uint64_t s_full[G][2], p_full[G][2], o_done[G][2], q_full, q_free, drain, never;
    __shared__ uint64_t seg_full[pa::kRing], seg_free[pa::kRing];
    __shared__ pa::Segment s_seg[pa::kRing];
    __shared__ uint4 s_bad[kFix];  // marked keys of a tile: key 16 w + i at bit 2 i of word w
    __shared__ uint32_t tmem_base;
    __shared__ int fail, issued[2];  // tiles whose copies into A and B have been issued

    Unit u{};
    if constexpr (!LATENT) {
        u = unit_of(a, blocks);
        if (u.r * 256 >= u.nq) return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    const int q_group = a.na * kQChunk;  // of a group's Q in shared memory (absorbed form: the rotated part, the rest is in tensor memory)
    uint8_t *base = dyn + ((1024u - (umma::smem_u32(dyn) & 1023u)) & 1023u);
    const uint32_t sm = umma::smem_u32(base);
    // ring A: stages of na chunks, then ring B: of nb; absorbed form: stages of both, ring B's place is within them
    const int a_bytes = (LATENT ? a.na + a.nb : a.na) * kChunk, b_bytes = LATENT ? a_bytes : a.nb * kChunk;
    const uint32_t a0 = sm + G * q_group, b0 = a0 + (LATENT ? a.na * kChunk : a.sa * a_bytes);
    if (tid == 0) {
        fail = 0;
        issued[0] = issued[1] = 0;
        for (int i = 0; i < kMostStages; ++i) {
            umma::mbar_init(&a_full[i], 1);
            umma::mbar_init(&a_empty[i], 1);
            umma::mbar_init(&b_full[i], 1);
            umma::mbar_init(&b_empty[i], 5);  // PV, and the helpers' warps
        }
        for (int i = 0; i < kFix; ++i) umma::mbar_init(&fixed[i], 4);
        for (int g = 0; g < G; ++g)
            for (int i = 0; i < 2; ++i) {
                umma::mbar_init(&s_full[g][i], 1);
                umma::mbar_init(&p_full[g][i], 4);
                umma::mbar_init(&o_done[g][i], 1);
            }
        umma::mbar_init(&q_full, 4);
        umma::mbar_init(&q_free, 1);
        umma::mbar_init(&drain, 2);
        umma::mbar_init(&never, 1);
        for (int i = 0; i < pa::kRing; ++i) {
            umma::mbar_init(&seg_full[i], 1);
            umma::mbar_init(&seg_free[i], WARPS - 1);
        }
        umma::fence_barrier_init();
    }
    if (warp == W0 + 7) {
        umma::tmem_alloc(&tmem_base, 512);
        umma::tmem_relinquish();
    }
    __syncthreads();
    umma::tc_fence_after();
    // O of the groups from 0 (128 columns each; LATENT: 256), S from 256, two buffers a group, LATENT: Q but its rotated part from 384
    const uint32_t tmem = tmem_base;
    volatile int *vfail = &fail;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return pa::wait(bar, parity, vfail, a.wait_ns); };
    auto next_segment = [&](pa::Segment &g, int n) {
        if constexpr (LATENT) {
            const int i = n & (pa::kRing - 1);
            const bool ok = wait(&seg_full[i], (n / pa::kRing) & 1);
            g = s_seg[i];
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&seg_free[i]);
            return __all_sync(0xFFFFFFFFu, ok) && g.t1 > 0;
        } else {
            g.b = u.b;
            g.h = u.h;
            g.r = u.r;
            g.t0 = 0;
            g.t1 = g.nt = max(u.nt[0], u.nt[1]);
            g.q0 = u.q0;
            g.nq = u.nq;
            g.kv = u.kv;
            return n == 0;
        }
    };
    // Tiles of group grp in a segment, and the first key that some row does not see.
    auto tiles_end = [&](const pa::Segment &g, int grp) { return LATENT ? g.t1 : u.nt[grp]; };
    auto clear_of = [&](const pa::Segment &g) {
        const int hist = g.kv - g.nq;
        if (a.mode == QVG_MASK_NONE) return g.kv;
        if (a.mode == QVG_MASK_TREE) return min(g.kv, hist);
        return min(g.kv, hist + 1 + (LATENT ? static_cast<int>(static_cast<long long>(g.r) * kRows / a.grp) : g.r * 256));
    };
    auto partial = [&](int t, int clear) { return (t + 1) * kKeys > clear; };

    if (warp < W0) {
        // ---- softmax: thread = row -----------------------------------------------------------------
        const int grp = warp >> 2, r = tid & 127;
        const uint32_t t_lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_o = tmem + grp * 128 + t_lane, t_s = tmem + 256 + grp * 128 + t_lane;
        const uint64_t sl2 = pa::pk2(a.scale_log2, a.scale_log2);
        pa::Segment g;
        int mine = 0, n_fix = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            const uint32_t gi = static_cast<uint32_t>(g.r) * (G * kRows) + grp * kRows + r;
            const int tq = LATENT ? static_cast<int>(gi / static_cast<uint32_t>(a.grp)) : static_cast<int>(gi);
            const int h = LATENT ? static_cast<int>(gi) - tq * a.grp : g.h;
            const bool live = tq < g.nq, idle = !__any_sync(0xFFFFFFFFu, live);
            const int clear = clear_of(g), end = tiles_end(g, grp);
            float ref = -INFINITY;  // of the logits as S has them
            uint64_t l2[2] = {0, 0};
            for (int t = g.t0; t < end; ++t, ++mine) {
                const int bf = mine & 1;
                const bool part = partial(t, clear);
                ok = wait(&s_full[grp][bf], (mine >> 1) & 1);
                uint4 bad = make_uint4(0, 0, 0, 0);
                if (part) {
                    ok = ok && wait(&fixed[n_fix % kFix], (n_fix / kFix) & 1);
                    bad = s_bad[n_fix % kFix];
                    ++n_fix;
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                umma::tc_fence_after();
                if (!idle) {
                    uint32_t v[2][32];
                    umma::tmem_ld32(t_s + bf * 64, v[0]);
                    umma::tmem_ld32(t_s + bf * 64 + 32, v[1]);
                    umma::tmem_ld_wait_regs(v[0]);
                    umma::reg_fence32(v[1]);
                    if (part) {
                        const uint2 see = seen_keys(a, t, g.kv, g.nq, g.q0, live ? tq : 0);
                        const uint32_t sw[2] = {see.x, see.y}, bw[4] = {bad.x, bad.y, bad.z, bad.w};
#pragma unroll
                        for (int c = 0; c < kKeys; ++c)
                            if (!((sw[c / 32] >> (c & 31)) & 1u)) v[c / 32][c % 32] = 0xFF800000u;
                        if (bad.x | bad.y | bad.z | bad.w) {
#pragma unroll
                            for (int c = 0; c < kKeys; ++c)
                                if ((sw[c / 32] >> (c & 31)) & (bw[c / 16] >> (2 * (c % 16))) & 1u) v[c / 32][c % 32] = 0x7FFFFFFFu;
                        }
                    }
                    float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < kKeys; c += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            top4[i] = fmaxf(fmaxf(top4[i], __uint_as_float(v[c / 32][c % 32 + 2 * i])), __uint_as_float(v[c / 32][c % 32 + 2 * i + 1]));
                    const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                    const bool fresh = ref == -INFINITY;
                    const bool move = live && (fresh ? top > -INFINITY : (top - ref) * a.scale_log2 > kRaise);
                    const float f = move && !fresh ? pa::ex2((ref - top) * a.scale_log2) : 1.0f;
                    if (move) ref = top;
                    if (t != g.t0 && __any_sync(0xFFFFFFFFu, f != 1.0f)) {
                        // the product of the tile before has to be in O
                        ok = wait(&o_done[grp][(mine - 1) & 1], ((mine - 1) >> 1) & 1);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        umma::tc_fence_after();
                        rescale_rows(t_o, a.dv, f);
                    }
                    const float nm = ref == -INFINITY ? 0.0f : -ref * a.scale_log2;
                    const uint64_t nm2 = pa::pk2(nm, nm), f2 = pa::pk2(f, f);
                    l2[0] = pa::mul2(l2[0], f2);
                    l2[1] = pa::mul2(l2[1], f2);
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < kKeys; c += 2) {
                        float y0, y1;
                        pa::up2(pa::fma2(pa::pk2(__uint_as_float(v[c / 32][c % 32]), __uint_as_float(v[c / 32][c % 32 + 1])), sl2, nm2), y0, y1);
                        y0 = pa::ex2(y0);
                        y1 = pa::ex2(y1);
                        l2[(c / 2) & 1] = pa::add2(l2[(c / 2) & 1], pa::pk2(y0, y1));
                        w[c / 2] = bf16x2(y0, y1);
                    }
                    umma::tmem_st32(t_s + bf * 64, w);  // over the logits
                    umma::tmem_st_wait();
                }
                umma::tc_fence_before();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&p_full[grp][bf]);
            }
            if (!ok) break;
            const bool none = end <= g.t0;  // (expanded form: rows that see no key)
            if (!none) {
                ok = wait(&o_done[grp][(mine - 1) & 1], ((mine - 1) >> 1) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                umma::tc_fence_after();
            }
            float x0, x1, x2, x3;
            pa::up2(l2[0], x0, x1);
            pa::up2(l2[1], x2, x3);
            const float l = (x0 + x1) + (x2 + x3);
            const bool whole = !LATENT || g.whole();
            const int slot = cta * 2 + (g.t0 > 0 ? 0 : 1);
            const long long prow = static_cast<long long>(slot) * kRows + r, row = static_cast<long long>(g.q0 + tq) * a.Hq + h;
            const float m = ref * a.scale_log2;
            if (live && !whole) {
                a.pm[prow] = m;
                a.pl[prow] = l;
            } else if (live && a.lse) {
                a.lse[static_cast<long long>(h) * a.total_q + g.q0 + tq] = l == 0.0f ? -INFINITY : (log2f(l) + m) * 0.69314718055994531f;
            }
            const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
            if (!idle) {
#pragma unroll 1
                for (int c = 0; c < a.dv; c += 16) {
                    uint32_t o[16];
                    if (none) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = 0;
                    } else {
                        pa::tmem_ld16(t_o + c, o);
                    }
                    if (!live) continue;
                    if (whole && a.out16) {
                        uint32_t y[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out16 + row * a.dv + c);
                        dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                        dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(whole ? a.out32 + row * a.dv + c : a.po + prow * a.dv + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                                 __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
                    }
                }
            }
            umma::tc_fence_before();
        }
    } else if (warp < W0 + 4) {
        // ---- helpers: Q, and V where some row does not see all of it ---------------------------------
        const int w = tid - W0 * 32;
        pa::Segment g;
        Ring rb;
        int n_fix = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            if (n_seg > 0) ok = wait(&q_free, (n_seg - 1) & 1);
            ++n_seg;
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const int piece = w & 7;
            for (int i = w >> 3; i < G * kRows; i += 16) {
                const uint32_t gi = static_cast<uint32_t>(g.r) * (G * kRows) + i;
                const int tq = LATENT ? static_cast<int>(gi / static_cast<uint32_t>(a.grp)) : static_cast<int>(gi);
                if (tq >= g.nq) break;  // (rows that are left out keep what is there: no other row reads them)
                const int h = LATENT ? static_cast<int>(gi) - tq * a.grp : g.h, row = i & (kRows - 1);
                const uint16_t *q = a.q + (g.q0 + tq) * a.q_stride + h * a.q_h + piece * 8;
                const uint16_t *qr = a.qr + (g.q0 + tq) * a.qr_t + h * a.qr_h + piece * 8;
                uint8_t *dst = base + (i >> 7) * q_group + row * 128 + ((piece ^ (row & 7)) << 4);
                const int plain = LATENT ? 0 : a.dk / 64;  // chunks before the rotated part's
                for (int c = 0; c < a.na; ++c) {
                    const bool in = c < plain || (c - plain) * 64 + piece * 8 < a.dr;
                    umma::cp_async16(dst + c * kQChunk, !in ? a.q : c < plain ? q + c * 64 : qr + (c - plain) * 64, in);
                }
            }
            if constexpr (LATENT) {  // a thread's row into its lane of tensor memory
                const uint32_t gi = static_cast<uint32_t>(g.r) * kRows + w;
                const int tq = static_cast<int>(gi / static_cast<uint32_t>(a.grp)), h = static_cast<int>(gi) - tq * a.grp;
                const bool live = tq < g.nq;
                const uint4 *q = reinterpret_cast<const uint4 *>(a.q + (g.q0 + (live ? tq : 0)) * a.q_stride + (live ? h : 0) * a.q_h);
                const uint32_t t_q = tmem + 384 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
                if (__any_sync(0xFFFFFFFFu, live)) {
                    for (int c = 0; c < a.nb; ++c) {
                        uint32_t x[32];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint4 v = live ? q[c * 8 + e] : make_uint4(0, 0, 0, 0);
                            x[4 * e] = v.x, x[4 * e + 1] = v.y, x[4 * e + 2] = v.z, x[4 * e + 3] = v.w;
                        }
                        umma::tmem_st32(t_q + c * 32, x);
                    }
                    umma::tmem_st_wait();
                }
                umma::tc_fence_before();
            }
            umma::cp_async_wait_all();
            umma::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&q_full);
            const int clear = clear_of(g), row = w >> 1;
            for (int t = g.t0; t < g.t1; ++t, rb.next(a.sb)) {
                ok = wait(&b_full[rb.i], rb.parity);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (partial(t, clear)) {
                    uint8_t *line = base + (b0 - sm) + rb.i * b_bytes + row * 128 + (w & 1) * 64;
                    bool bad = false;
                    for (int c = 0; c < a.nb; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(line + c * kChunk + 16 * i);
                            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) bad = bad || (y[e] & 0x7F80u) == 0x7F80u || (y[e] & 0x7F800000u) == 0x7F800000u;
                        }
                    const uint32_t any = __ballot_sync(0xFFFFFFFFu, bad);
                    const bool past = t * kKeys + row >= g.kv;
                    if (past || (any >> (lane & 30) & 3u)) {
                        for (int c = 0; c < a.nb; ++c)
#pragma unroll
                            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(line + c * kChunk + 16 * i) = make_uint4(0, 0, 0, 0);
                    }
                    const uint32_t marks = __ballot_sync(0xFFFFFFFFu, !past && (lane & 1) == 0 && (any >> lane & 3u));
                    if (lane == 0) reinterpret_cast<uint32_t *>(&s_bad[n_fix % kFix])[warp - W0] = marks;
                    umma::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(&fixed[n_fix % kFix]);
                    ++n_fix;
                }
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&b_empty[rb.i]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == W0 + 4) {
        // ---- loads -------------------------------------------------------------------------------------
        // A tile's latents (k, v) take one copy where a page holds the whole tile, else one for each piece of a page and
        // chunk; the rotated part's chunks one copy each.
        const int pr_log2 = LATENT ? min(a.page_log2, 6) : 6, pr = 1 << pr_log2, pieces = kKeys >> pr_log2;
        const bool one = elected();
        pa::Segment g;
        Ring ra, rb;
        int it = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            // first slot of piece `lane` of tile t (expanded form: first key); -1: no such page
            auto first_of = [&](int t) {
                if (!LATENT) return u.k0 + t * kKeys;
                const long long tok = static_cast<long long>(t) * kKeys + (lane << pr_log2);
                if (lane >= pieces || tok >= g.kv || t >= g.t1) return -1;
                const int page = a.table[g.b * a.table_stride + (tok >> a.page_log2)];
                if (page < 0 || page >= a.num_pages) {
                    raise_error(a.err, QVG_ERR_INVALID_ARG);
                    return -1;
                }
                return (page << a.page_log2) + static_cast<int>(tok & ((1 << a.page_log2) - 1));
            };
            int now = first_of(g.t0);
            for (int t = g.t0; t < g.t1; ++t, ++it) {
                const int then = first_of(t + 1);
                const int there = LATENT ? __popc(__ballot_sync(0xFFFFFFFFu, now >= 0)) : 0;
                if constexpr (LATENT) {
                    if (it >= a.sb) ok = wait(&b_empty[rb.i], rb.parity ^ 1u);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    uint64_t *full = &b_full[rb.i];
                    const uint32_t dst = b0 + rb.i * b_bytes, dst_r = a0 + rb.i * a_bytes;
                    if (one) umma::mbar_arrive_expect_tx(full, there * (a.na + a.nb) * (pr * 128));
                    for (int p = 0; p < pieces; ++p) {
                        const int at = __shfl_sync(0xFFFFFFFFu, now, p);
                        if (at < 0) continue;
                        if (pieces == 1) {
                            if (one) tma_load_3d(dst, &kmap, 0, at, 0, full);
                        } else {
                            for (int c = 0; c < a.nb; ++c)
                                if (one) tma_load_3d(dst + c * kChunk + p * (pr * 128), &kmap, 0, at, c, full);
                        }
                        for (int c = 0; c < a.na; ++c)
                            if (one) tma_load_2d(dst_r + c * kChunk + p * (pr * 128), &rmap, c * 64, at, full);
                    }
                } else {
                    if (it >= a.sa) ok = wait(&a_empty[ra.i], ra.parity ^ 1u);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const uint32_t dst = a0 + ra.i * a_bytes;
                    if (one) {
                        umma::mbar_arrive_expect_tx(&a_full[ra.i], a_bytes);
                        tma_load_4d(dst, &kmap, 0, now, 0, u.h, &a_full[ra.i]);
                        if (a.dr > 0) tma_load_2d(dst + (a.na - 1) * kChunk, &rmap, 0, now, &a_full[ra.i]);
                        issued[0] = it + 1;
                    }
                    __syncwarp();
                    ra.next(a.sa);
                    if (it >= a.sb) ok = wait(&b_empty[rb.i], rb.parity ^ 1u);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (one) {
                        umma::mbar_arrive_expect_tx(&b_full[rb.i], b_bytes);
                        tma_load_4d(b0 + rb.i * b_bytes, &vmap, 0, now, 0, u.h, &b_full[rb.i]);
                    }
                }
                if (one) issued[1] = it + 1;
                rb.next(a.sb);
                now = then;
            }
        }
        __syncwarp();
    } else if (warp == W0 + 5) {
        // ---- S -----------------------------------------------------------------------------------------
        constexpr uint32_t id = umma::idesc_f16(kRows, kKeys, 1);
        const int plain = LATENT ? 0 : a.dk / 64;  // chunks before the rotated part's
        const bool one = elected();
        pa::Segment g;
        Ring ra, rb;
        int mine[G] = {}, n_fix = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            const int clear = clear_of(g);
            ok = wait(&q_full, n_seg & 1);
            ++n_seg;
            for (int t = g.t0; t < g.t1; ++t) {
                if (!LATENT) ok = ok && wait(&a_full[ra.i], ra.parity);
                if (LATENT) {
                    ok = ok && wait(&b_full[rb.i], rb.parity);
                    if (partial(t, clear)) {
                        ok = ok && wait(&fixed[n_fix % kFix], (n_fix / kFix) & 1);
                        ++n_fix;
                    }
                }
#pragma unroll
                for (int grp = 0; grp < G; ++grp) {
                    if (t >= tiles_end(g, grp)) continue;
                    const int bf = mine[grp] & 1;
                    if (mine[grp] >= 2) ok = ok && wait(&o_done[grp][bf], ((mine[grp] >> 1) - 1) & 1);  // the buffer's last weights have been used
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    umma::tc_fence_after();
                    const uint32_t t_s = tmem + 256 + grp * 128 + bf * 64;
                    uint32_t acc = 0;
                    uint64_t dk;
                    if (LATENT) {
                        dk = umma::desc_sw128(b0 + rb.i * b_bytes);
                        for (int c = 0; c < a.nb; ++c, dk += kChunk >> 4)
#pragma unroll
                            for (int s = 0; s < 4; ++s, acc = 1) mma_ts(t_s, tmem + 384 + c * 32 + 8 * s, dk + 2 * s, id, acc, one);
                    }
                    uint64_t dq = umma::desc_sw128(sm + grp * q_group);
                    dk = umma::desc_sw128(a0 + (LATENT ? rb.i : ra.i) * a_bytes);
                    for (int c = 0; c < a.na; ++c, dq += kQChunk >> 4, dk += kChunk >> 4) {
                        const int steps = c < plain ? 4 : min(4, (a.dr - (c - plain) * 64 + 15) / 16);
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            if (s < steps) {
                                mma_ss(t_s, dq + 2 * s, dk + 2 * s, id, acc, one);
                                acc = 1;
                            }
                    }
                    commit(&s_full[grp][bf], one);
                    // test hook: with S in flight, wait for what never comes
                    if (a.inject && mine[grp] == 0) ok = wait(&never, 0);
                    ++mine[grp];
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (LATENT) {
                    rb.next(a.sb);  // (the stage is given back by PV)
                } else {
                    commit(&a_empty[ra.i], one);
                    ra.next(a.sa);
                }
            }
            if (ok) commit(&q_free, one);
        }
        commit(&drain, one);  // all products issued complete before tensor memory goes back
        umma::mbar_wait(&drain, 0, pa::kDrainNs);
    } else if (warp == W0 + 6) {
        // ---- PV ---------------------------------------------------------------------------------------
        const uint32_t id = umma::idesc_f16_bmn(kRows, a.dv, 1);
        const bool one = elected();
        pa::Segment g;
        Ring rb;
        int mine[G] = {}, n_fix = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            const int clear = clear_of(g);
            for (int t = g.t0; t < g.t1; ++t, rb.next(a.sb)) {
                ok = wait(&b_full[rb.i], rb.parity);
                if (partial(t, clear)) {
                    ok = ok && wait(&fixed[n_fix % kFix], (n_fix / kFix) & 1);
                    ++n_fix;
                }
                const uint64_t dv = umma::desc_sw128_mn(b0 + rb.i * b_bytes, kChunk);
#pragma unroll
                for (int grp = 0; grp < G; ++grp) {
                    if (t >= tiles_end(g, grp)) continue;
                    const int bf = mine[grp] & 1;
                    ok = ok && wait(&p_full[grp][bf], (mine[grp] >> 1) & 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    umma::tc_fence_after();
                    const uint32_t t_p = tmem + 256 + grp * 128 + bf * 64, t_o = tmem + grp * 128;
#pragma unroll
                    for (int s = 0; s < kKeys / 16; ++s) mma_ts(t_o, t_p + 8 * s, dv + s * 128, id, !(t == g.t0 && s == 0), one);
                    commit(&o_done[grp][bf], one);
                    ++mine[grp];
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                commit(&b_empty[rb.i], one);
            }
        }
        commit(&drain, one);
        umma::mbar_wait(&drain, 0, pa::kDrainNs);
    } else if constexpr (LATENT) {
        // ---- this CTA's part of the line, unit by unit ---------------------------------------------------
        pa::Line<kRows, kKeys> line(a, reinterpret_cast<long long *>(base));  // (Q's place: no segment is out yet)
        bool ok = true;
        for (int n_seg = 0; ok; ++n_seg) {
            pa::Segment g;
            line.next(a, g);
            const int i = n_seg & (pa::kRing - 1);
            if (n_seg >= pa::kRing) ok = wait(&seg_free[i], ((n_seg / pa::kRing) - 1) & 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane == 0) {
                s_seg[i] = g;
                umma::mbar_arrive(&seg_full[i]);
            }
            if (g.t1 == 0) break;
        }
        if (lane == 0) a.desc[cta] = ok ? line.cut : make_int4(-1, 0, 0, 0);
    }
    __syncwarp();
    umma::tc_fence_before();
    __syncthreads();
    if (tid == 0 && *vfail) {
        raise_error(a.err, QVG_ERR_TIMEOUT);
        // the copies in flight land before the CTA ends
        for (int j = max(0, issued[0] - a.sa); j < issued[0]; ++j)  // (none in the absorbed form)
            umma::mbar_wait(&a_full[j % a.sa], (j / a.sa) & 1, pa::kDrainNs);
        for (int j = max(0, issued[1] - a.sb); j < issued[1]; ++j) umma::mbar_wait(&b_full[j % a.sb], (j / a.sb) & 1, pa::kDrainNs);
    }
    if (warp == W0 + 7) {
        umma::tc_fence_after();
        umma::tmem_dealloc(tmem, 512);
    }
}

}  // namespace la
}  // namespace qvg
