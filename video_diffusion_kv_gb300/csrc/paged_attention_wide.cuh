// paged_attention_wide.cuh -- attention over a paged cache for sequences with
// many query rows (trees, short chunks): the kernel.  The line of tiles, the
// segments and the partial sums are those of paged_attention.cuh; a unit has
// 256 rows here.
//
// With many rows the product is turned the usual way round, rows on the tensor
// core's 128 rows, two groups of them sharing each tile of 128 keys:
//   S [rows x keys] = Q K^T    Q as two e4m3 numbers hi + lo (hi + lo / 16 would
//                              need two accumulators; a channel is exact down
//                              to 2^-9 of the row's largest), K's codes as they
//                              lie in the cache
//   O [rows x d]   += P V      P in fp16 in tensor memory, over S; V's codes as
//                              fp16, made by four converter warps (4 bits: K's
//                              codes become e4m3 on the way as well)
// A softmax thread owns a row, so its maximum and sum need no other thread, and
// there are no three parts and no weights through shared memory; a key's scales
// are read from shared memory.  A row's 128 logits stay in registers from the
// one read of S to the weights, for which the softmax warps take registers from
// the others (with two reads of S and 128 registers: 510 us for the frame
// below, where this takes 367); the largest logit is looked for only where a
// weight overflows (375 us with the search in every tile).
// One group's products run while the other group is at its softmax.
//
// Bound: the chain of a group and tile, about 6000 clocks in the frame below: a
// thread waits for S 2400 (its own weights' products and then S's: eight each,
// which one thread takes 820 and 560 clocks to issue and which end 350 and 260 later),
// for V's operand 240, reads S in 610, masks and makes the weights in 2150; the
// rest is the segments' ends.  880 causal tokens over 21,120 (24 heads, d = 128, 8
// bits; 2.3e11 operations): 367 us, 623 TFLOP/s, 33 % of a large bf16 product's
// rate.  16 trees of 17 to 48 tokens (4 query heads each) over 2,000 to 12,000:
// 199 us; a unit there has 68 to 192 of the 256 rows, and with up to 128 of them
// the second group has nothing to do.
#pragma once

#include "paged_attention.cuh"

namespace qvg {
namespace pa {

constexpr int kWideRows = 256, kWideRegs = 128;  // rows of a unit; registers a thread at launch

template <int D, int BITS>
struct Wide {
    static constexpr int G = BITS == 8 ? 1 : D / 32;
    static constexpr int kRow = D * BITS / 8;
    static constexpr int kRaw = kTile * kRow;              // a tile's codes as loaded
    static constexpr int kScales = 256 * G;
    static constexpr int kK8 = BITS == 4 ? kTile * D : 0;  // K as e4m3 (4 bits), two buffers
    static constexpr int kVf = kTile * D * 2;              // V as fp16, two buffers
    static constexpr int kQ = 2 * 128 * D;                 // a group's Q: hi rows, lo rows
    static constexpr int SK = 3, SV = 2;                   // K's and V's copies in flight
    static constexpr int kSmem = 2 * kK8 + 2 * kVf + 2 * kQ + SK * kRaw + SV * kRaw + SV * kScales + 1024;
    static constexpr int kWarps = 16;  // softmax 0 - 7; converters 8 - 11; loads, S and PV of each group, segments
    static_assert(kSmem <= 224 * 1024, "shared memory");
};

// (This kernel splits its registers unevenly, which the compiler does not
// combine with calls: everything is inlined, the waits too.)
__device__ __forceinline__ bool wait_here(uint64_t *bar, uint32_t parity, volatile int *fail, uint64_t limit_ns) {
    if (umma::mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;
#pragma unroll 1
    for (int i = 0;; ++i) {
        if (try_wait_long(bar, parity)) return true;
        if (i < 4) continue;
        if (i == 4) t0 = umma::globaltimer_ns();
        if (*fail) return false;
        if (umma::globaltimer_ns() - t0 > limit_ns) {
            *fail = 1;
            return false;
        }
    }
}

// Which of the tile's 128 keys the row of new token tq sees, as bits.
__device__ __forceinline__ uint4 seen_keys(const Args &a, int t, int kv, int nq, int q0, int tq) {
    const int k0 = t * kTile, hist = kv - nq;
    int end = min(kv - k0, kTile);  // keys of the sequence in this tile
    if (a.mode == QVG_MASK_CAUSAL) end = min(end, hist + tq + 1 - k0);
    const uint32_t *m = a.mask + static_cast<long long>(q0 + tq) * a.words;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp's rows of O times their factors (the references of some have moved).
template <int D>
__device__ __forceinline__ void rescale_rows(uint32_t t_o, float f) {
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tmem_ld16(t_o + c, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        umma::tmem_st16(t_o + c, o);
    }
    umma::tmem_st_wait();
}

// 2^-d (d >= 0) as two factors, each within fp32's range up to d = 246: the
// references follow V's scale, which may rise by more than 2^126 while the
// sum l, up to 2^120, still counts.  (up to d = 120 the second is 1)
__device__ __forceinline__ float2 fall(float d) {
    const float a = fminf(d, 120.0f);
    return make_float2(ex2(-a), ex2(a - d));
}

// A thread's Q row as two rows of e4m3 numbers; returns its scale.
template <int D>
__device__ __forceinline__ float make_q_row(const uint16_t *q, uint8_t *hi, uint8_t *lo, int r) {
    uint4 v[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) v[i] = q ? reinterpret_cast<const uint4 *>(q)[i] : make_uint4(0, 0, 0, 0);
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
        m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu), __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu)));
    const uint32_t sb = scale_byte<8>(max(m2 & 0xFFFFu, m2 >> 16));
    const float inv = sb == 255u ? 0.0f : scale_inverse(sb);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t h[4], l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float f0 = __uint_as_float(x[k] << 16) * inv, f1 = __uint_as_float(x[k] & 0xFFFF0000u) * inv;
            h[k] = e4m3x2(f0, f1);
            const uint32_t hh = e4m3x2_to_f16x2(h[k]);
            const float2 b2 = __half22float2(*reinterpret_cast<const __half2 *>(&hh));
            l[k] = e4m3x2(f0 - b2.x, f1 - b2.y);
            if (sb == 255u) h[k] = 0x7F7Fu, l[k] = 0;  // an infinity or a NaN: the row is NaN
        }
        const uint32_t off = swizzle8<D>(r * D + i * 8);
        *reinterpret_cast<uint2 *>(hi + off) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
        *reinterpret_cast<uint2 *>(lo + off) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
    }
    return sb == 255u ? 1.0f : scale_of(sb);
}

template <int D, int BITS>
__global__ void __launch_bounds__(Wide<D, BITS>::kWarps * 32, 1)
    k_paged_attention_wide(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ Args a) {
    using C = Wide<D, BITS>;
    constexpr int SK = C::SK, SV = C::SV, NB = kWideRows;
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t k_full[SK], k_empty[SK], v_full[SV], v_empty[SV];  // codes (and scales, with V's) as loaded
    __shared__ uint64_t ko_full[2], ko_done[2], vo_full[2], vo_done[2];    // operands made of them (ko: 4 bits)
    __shared__ uint64_t s_full[2], p_full[2], o_done[2], q_full[2], drain, never;  // one per group
    __shared__ uint64_t seg_full[kRing], seg_free[kRing];
    __shared__ Segment s_seg[kRing];
    __shared__ long long s_chunk[kChunks];
    __shared__ uint32_t tmem_base;
    __shared__ int fail, s_issued[2];  // tiles of K and of V whose copies have been issued
    __shared__ __align__(16) float s_ka[2][kTile], s_sv[2][kTile], s_lsv[2][kTile];  // per key: K's scale, V's, its log
    __shared__ uint2 s_lv[BITS == 4 ? 16 : 1];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    uint8_t *base = dyn + ((1024u - (umma::smem_u32(dyn) & 1023u)) & 1023u);
    const uint32_t sm = umma::smem_u32(base);
    const uint32_t vf0 = sm, k80 = vf0 + 2 * C::kVf, q0 = k80 + 2 * C::kK8, kr0 = q0 + 2 * C::kQ, vr0 = kr0 + SK * C::kRaw,
                   sc0 = vr0 + SV * C::kRaw;
    if (tid == 0) {
        fail = 0;
        s_issued[0] = s_issued[1] = 0;
        for (int i = 0; i < kRing; ++i) {
            umma::mbar_init(&seg_full[i], 1);
            umma::mbar_init(&seg_free[i], C::kWarps - 1);
        }
        for (int i = 0; i < SK; ++i) {
            umma::mbar_init(&k_full[i], 1);
            umma::mbar_init(&k_empty[i], BITS == 8 ? 2 : 4);  // each group's S, or the converters
        }
        for (int i = 0; i < SV; ++i) {
            umma::mbar_init(&v_full[i], 33);
            umma::mbar_init(&v_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(&ko_full[i], 4);
            umma::mbar_init(&ko_done[i], 2);
            umma::mbar_init(&vo_full[i], 4);
            umma::mbar_init(&vo_done[i], 2);
            umma::mbar_init(&s_full[i], 1);
            umma::mbar_init(&p_full[i], 4);
            umma::mbar_init(&o_done[i], 1);
            umma::mbar_init(&q_full[i], 4);
        }
        umma::mbar_init(&drain, 2);
        umma::mbar_init(&never, 1);
        umma::fence_barrier_init();
    }
    if (warp == 15) {
        umma::tmem_alloc(&tmem_base, 512);
        umma::tmem_relinquish();
    }
    if (BITS == 4 && tid < 16) s_lv[tid] = levels_of(tid);
    __syncthreads();
    umma::tc_fence_after();
    const uint32_t tmem = tmem_base;  // S (and P) of the groups at 0 and 128, O at 256 and 384
    volatile int *vfail = &fail;
    auto next_segment = [&](Segment &g, int n) {
        const int i = n & (kRing - 1);
        const bool ok = wait_here(&seg_full[i], (n / kRing) & 1, vfail, a.wait_ns);
        g = s_seg[i];
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&seg_free[i]);
        return __all_sync(0xFFFFFFFFu, ok) && g.t1 > 0;
    };
    // Whether group 1 has rows in this unit.
    auto both = [&](const Segment &g) { return static_cast<long long>(g.nq) * a.grp - static_cast<long long>(g.r) * NB > 128; };

    // Registers: 2 x 128 softmax threads take 200, the other 2 x 128 keep 56; the sum is what the block was launched
    // with (512 x 128, which the launch makes sure of).
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---- softmax: thread = row ---------------------------------------------------------------
        const int grp = warp >> 2, r = tid & 127;
        const uint32_t t_lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + grp * 128 + t_lane, t_o = tmem + 256 + grp * 128 + t_lane;
        uint8_t *q_hi = base + (q0 - sm) + grp * C::kQ;
        Segment g;
        int it = 0, mine = 0, n_own = 0, n_seg = 0;  // tiles; tiles and segments of this group
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            if (grp == 1 && !both(g)) {
                it += g.t1 - g.t0;
                continue;
            }
            // the row; its Q (the last unit's products with the group's Q are done: its S have been seen)
            const uint32_t gi = static_cast<uint32_t>(g.r) * NB + grp * 128 + r;
            const int tq = static_cast<int>(gi / static_cast<uint32_t>(a.grp)), j = static_cast<int>(gi) - tq * a.grp;
            const bool live = tq < g.nq;
            const float qs = make_q_row<D>(
                live ? a.q + (g.q0 + tq) * a.q_stride + static_cast<long long>(g.h * a.grp + j) * D : nullptr, q_hi, q_hi + 128 * D, r);
            umma::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&q_full[grp]);
            ++n_own;
            const int clear = a.mode == QVG_MASK_NONE ? g.kv : min(g.kv, g.kv - g.nq);
            float nm = 0.0f;  // minus the reference
            uint64_t l2[2] = {0, 0};
            for (int t = g.t0; t < g.t1; ++t, ++it, ++mine) {
                const int bf = it & 1;
                const bool first = t == g.t0, part = (t + 1) * kTile > clear;
                ok = wait_here(&s_full[grp], mine & 1, vfail, a.wait_ns);
                // The keys' scales.  (After S: group 1 may have left tiles out, and only once S(t) is there has its
                // buffer's last use but one surely begun, which the parity cannot tell.)
                ok = ok && wait_here(&vo_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                umma::tc_fence_after();
                // the row's logits less qs, in registers: x = S ka
                float x[kTile];
                {
                    uint32_t v[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) umma::tmem_ld32(t_s + 32 * c, v[c]);
                    umma::tmem_ld_wait_regs(v[0]);
                    umma::reg_fence32(v[1]);
                    umma::reg_fence32(v[2]);
                    umma::reg_fence32(v[3]);
#pragma unroll
                    for (int i = 0; i < kTile / 4; ++i) {
                        const float4 ka = *reinterpret_cast<const float4 *>(&s_ka[bf][4 * i]);
                        const uint32_t(&w)[32] = v[i / 8];
                        const int e = 4 * (i % 8);
                        up2(mul2(pk2(__uint_as_float(w[e]), __uint_as_float(w[e + 1])), pk2(ka.x, ka.y)), x[4 * i], x[4 * i + 1]);
                        up2(mul2(pk2(__uint_as_float(w[e + 2]), __uint_as_float(w[e + 3])), pk2(ka.z, ka.w)), x[4 * i + 2], x[4 * i + 3]);
                    }
                }
                if (part) {
                    const uint4 see = seen_keys(a, t, g.kv, g.nq, g.q0, live ? tq : 0);
                    const uint32_t sw[4] = {see.x, see.y, see.z, see.w};
#pragma unroll
                    for (int c = 0; c < kTile; ++c) x[c] = (sw[c / 32] >> (c & 31)) & 1u ? x[c] : -INFINITY;
                }
                const uint64_t qs2 = pk2(qs, qs), l_was[2] = {l2[0], l2[1]};
                const bool fresh = (l2[0] | l2[1]) == 0;
                // The reference is set by the first tile that the row sees a key of, and raised where a weight passes
                // 2^kTop: then the weights are made once more.
                bool look = __any_sync(0xFFFFFFFFu, fresh);
                for (bool again = true; again;) {
                    uint64_t lp[2] = {l_was[0], l_was[1]};
                    if (look) {
                        // the row's largest logit plus log of V's scale
                        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < kTile / 4; ++i) {
                            const float4 ls = *reinterpret_cast<const float4 *>(&s_lsv[bf][4 * i]);
                            float y0, y1, y2, y3;
                            up2(fma2(pk2(x[4 * i], x[4 * i + 1]), qs2, pk2(ls.x, ls.y)), y0, y1);
                            up2(fma2(pk2(x[4 * i + 2], x[4 * i + 3]), qs2, pk2(ls.z, ls.w)), y2, y3);
                            top4[i & 1] = fmaxf(fmaxf(top4[i & 1], y0), y1);
                            top4[2 + (i & 1)] = fmaxf(fmaxf(top4[2 + (i & 1)], y2), y3);
                        }
                        const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                        const bool move = top > -INFINITY && (fresh || top + nm > kTop);
                        const float to = move ? kTarget - top : nm;
                        const float2 f = fall(move && !fresh ? nm - to : 0.0f);
                        nm = to;
#pragma unroll
                        for (int h = 0; h < 2; ++h) lp[h] = mul2(mul2(lp[h], pk2(f.x, f.x)), pk2(f.y, f.y));
                        if (!first && __any_sync(0xFFFFFFFFu, f.x != 1.0f)) rescale_rows<D>(t_o, f.x * f.y);  // (the last product is done: S came after it)
                    }
                    const uint64_t nm2 = pk2(nm, nm);
                    __half2 high = __half2half2(__ushort_as_half(0));  // the largest weights
#pragma unroll
                    for (int c = 0; c < kTile; c += 32) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 sv = *reinterpret_cast<const float4 *>(&s_sv[bf][c + 4 * i]);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int e = 4 * i + 2 * h;
                                float y0, y1, w0, w1;
                                up2(fma2(pk2(x[c + e], x[c + e + 1]), qs2, nm2), y0, y1);
                                const uint64_t p = pk2(ex2(y0), ex2(y1));
                                lp[h] = add2(lp[h], p);
                                up2(mul2(p, h ? pk2(sv.z, sv.w) : pk2(sv.x, sv.y)), w0, w1);
                                w[e / 2] = f16x2(w0, w1);
                                high = __hmax2(high, *reinterpret_cast<const __half2 *>(&w[e / 2]));
                            }
                        }
                        umma::tmem_st16(t_s + c / 2, w);  // over the logits
                    }
                    l2[0] = lp[0];
                    l2[1] = lp[1];
                    const uint32_t hb = *reinterpret_cast<const uint32_t *>(&high);
                    float a0, a1, a2, a3;
                    up2(l2[0], a0, a1);
                    up2(l2[1], a2, a3);
                    // (the sum has no V scale in it: where V's is below 2^kLeastV it could overflow before a weight does)
                    again = !look && __any_sync(0xFFFFFFFFu, max(hb & 0xFFFFu, hb >> 16) >= 0x7800u ||  // 2^kTop
                                                                 fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) > 0x1p120f);
                    if (again) umma::tmem_st_wait();
                    look = true;
                }
                umma::tmem_st_wait();
                umma::tc_fence_before();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&p_full[grp]);
            }
            if (!ok) break;
            ok = wait_here(&o_done[grp], (mine - 1) & 1, vfail, a.wait_ns);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            umma::tc_fence_after();
            float a0, a1, a2, a3;
            up2(l2[0], a0, a1);
            up2(l2[1], a2, a3);
            const float l = (a0 + a1) + (a2 + a3);
            const bool whole = g.whole();
            const int slot = cta * 2 + (g.t0 > 0 ? 0 : 1);
            const long long prow = static_cast<long long>(slot) * NB + grp * 128 + r, row = static_cast<long long>(g.q0 + tq) * a.Hq + g.h * a.grp + j;
            if (live && !whole) {
                a.pm[prow] = -nm;
                a.pl[prow] = l;
            } else if (live && a.lse) {
                a.lse[static_cast<long long>(g.h * a.grp + j) * a.total_q + g.q0 + tq] =
                    l == 0.0f ? -INFINITY : (log2f(l) - nm) * 0.69314718055994531f;
            }
            const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_ld16(t_o + c, o);
                if (!live) continue;
                if (whole && a.out16) {
                    uint32_t b[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                        b[i] = *reinterpret_cast<const uint32_t *>(&y);
                    }
                    uint4 *dst = reinterpret_cast<uint4 *>(a.out16 + row * D + c);
                    dst[0] = make_uint4(b[0], b[1], b[2], b[3]);
                    dst[1] = make_uint4(b[4], b[5], b[6], b[7]);
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(whole ? a.out32 + row * D + c : a.po + prow * D + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dst[i] = make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                             __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
                }
            }
            umma::tc_fence_before();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp < 12) {
        // ---- converters: V's codes into fp16, the scales into floats (4 bits: K's codes into e4m3) ----
        const int w = tid - 256;
        constexpr int GR = D / 32;
        Segment g;
        Ring<SK> rk;
        Ring<SV> rv;
        int it = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            for (int t = g.t0; t < g.t1; ++t, ++it, rk.next(), rv.next()) {
                const int bf = it & 1;
                ok = wait_here(&v_full[rv.i], rv.parity, vfail, a.wait_ns);
                if (BITS == 4) {
                    ok = ok && wait_here(&k_full[rk.i], rk.parity, vfail, a.wait_ns);
                    if (it >= 2) ok = ok && wait_here(&ko_done[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint8_t *sc = base + (sc0 - sm) + rv.i * C::kScales;
                uint8_t *vdst = base + (vf0 - sm) + bf * C::kVf;
                if constexpr (BITS == 4) {
                    const uint8_t *src = base + (kr0 - sm) + rk.i * C::kRaw;
                    uint8_t *dst = base + (k80 - sm) + bf * C::kK8;
#pragma unroll 2
                    for (int i = 0; i < GR; ++i) {
                        const int idx = w + 128 * i, row = idx / GR, gq = idx % GR;
                        const uint4 v = *reinterpret_cast<const uint4 *>(src + idx * 16);
                        const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
                        uint32_t top = 0;
#pragma unroll
                        for (int e = 0; e < GR; ++e) top = max(top, static_cast<uint32_t>(sc[row * GR + e]));
                        const uint2 lv = s_lv[min(top - sc[row * GR + gq], 15u)];
                        uint32_t o[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t mg = vw[e] & 0x77777777u, sg = vw[e] & 0x88888888u;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                uint32_t s;
                                asm("prmt.b32 %0, %1, 0, %2;" : "=r"(s) : "r"(0x80u), "r"(sg >> (16 * k)));
                                o[2 * e + k] = __byte_perm(lv.x, lv.y, mg >> (16 * k)) | ((s << 7) & 0x80808080u);
                            }
                        }
                        *reinterpret_cast<uint4 *>(dst + swizzle8<D>(row * D + gq * 32)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(dst + swizzle8<D>(row * D + gq * 32 + 16)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                    umma::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        umma::mbar_arrive(&ko_full[bf]);
                        umma::mbar_arrive(&k_empty[rk.i]);
                    }
                }
                if (it >= 2) ok = wait_here(&vo_done[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                {
                    uint32_t kb = 0, vb = 0;
#pragma unroll
                    for (int e = 0; e < C::G; ++e) {
                        kb = max(kb, static_cast<uint32_t>(sc[w * C::G + e]));
                        vb = max(vb, static_cast<uint32_t>(sc[128 * C::G + w * C::G + e]));
                    }
                    if (t * kTile + w >= g.kv) kb = vb = 127u;  // (whatever is there)
                    // 4 bits: K's operand is 2^6 times the values over the largest scale
                    s_ka[bf][w] = scale_of(kb) * (BITS == 8 ? a.scale_log2 : a.scale_log2 * 0x1p-6f);
                    s_sv[bf][w] = vb == 255u ? 1.0f : scale_of(vb);
                    if (vb == 255u) s_ka[bf][w] = NAN;  // (its V row is 0: the rows that see it become NaN this way)
                    s_lsv[bf][w] = vb == 255u ? 0.0f : fmaxf(static_cast<float>(static_cast<int>(vb) - 127), kLeastV);
                }
                const uint8_t *src = base + (vr0 - sm) + rv.i * C::kRaw;
                if constexpr (BITS == 8) {
                    constexpr int PPR = D / 16;  // 16-code pieces a row
#pragma unroll 4
                    for (int i = 0; i < PPR; ++i) {
                        const int idx = w + 128 * i, row = idx / PPR, c = idx % PPR;
                        const uint4 v = *reinterpret_cast<const uint4 *>(src + idx * 16);
                        const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
                        uint32_t o[8];
                        // a code that is no number (slots never written) becomes one: weights of 0 stay 0
                        const __half2 floor2 = __half2half2(__ushort_as_half(0xDF00));  // -448
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t h = e4m3x2_to_f16x2(vw[e / 2] >> (16 * (e & 1)));
                            const __half2 m = __hmax2(*reinterpret_cast<const __half2 *>(&h), floor2);
                            o[e] = *reinterpret_cast<const uint32_t *>(&m);
                        }
                        uint8_t *line = vdst + (c >> 2) * (kTile * 128) + row * 128;
                        const int e0 = ((2 * (c & 3)) ^ (row & 7)) << 4, e1 = ((2 * (c & 3) + 1) ^ (row & 7)) << 4;
                        const uint4 x = make_uint4(o[0], o[1], o[2], o[3]), y = make_uint4(o[4], o[5], o[6], o[7]);
                        const bool swap = c >= 4;  // the halves' lanes store in opposite order: no bank twice
                        *reinterpret_cast<uint4 *>(line + (swap ? e1 : e0)) = swap ? y : x;
                        *reinterpret_cast<uint4 *>(line + (swap ? e0 : e1)) = swap ? x : y;
                    }
                } else {
#pragma unroll 2
                    for (int i = 0; i < GR; ++i) {
                        const int idx = w + 128 * i, row = idx / GR, gq = idx % GR;
                        const uint4 v = *reinterpret_cast<const uint4 *>(src + idx * 16);
                        const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
                        const uint8_t *s = sc + 128 * GR + row * GR;
                        uint32_t top = 0;
#pragma unroll
                        for (int e = 0; e < GR; ++e) top = max(top, static_cast<uint32_t>(s[e]));
                        const uint32_t down = top - s[gq];  // fp16 values of the codes times 2^-down (below 2^-24: 0)
                        const __half2 f = __half2half2(down > 24u ? __ushort_as_half(0) : __float2half_rn(__uint_as_float((127u - down) << 23)));
                        uint8_t *line = vdst + (gq >> 1) * (kTile * 128) + row * 128;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t o[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t h = e2m1x2_to_f16x2((vw[e] >> (8 * k)) & 0xFFu);
                                const __half2 m = __hmul2(*reinterpret_cast<const __half2 *>(&h), f);
                                o[k] = *reinterpret_cast<const uint32_t *>(&m);
                            }
                            *reinterpret_cast<uint4 *>(line + (((4 * (gq & 1) + e) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
                umma::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    umma::mbar_arrive(&vo_full[bf]);
                    umma::mbar_arrive(&v_empty[rv.i]);
                }
            }
        }
    } else if (warp == 12) {
        // ---- loads, as in the narrow kernel, V's codes without a swizzle ------------------------------
        const int pr_log2 = min(a.page_log2, 7), pr = 1 << pr_log2;
        Segment g;
        Ring<SK> rk;
        Ring<SV> rv;
        int it = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            const int32_t *row = a.table + g.b * a.table_stride;
            const int pages = (g.kv + (1 << a.page_log2) - 1) >> a.page_log2;
            int have = (g.t0 * kTile) >> a.page_log2 & ~31;
            auto entries = [&](int e) { return e + lane < pages ? row[e + lane] : 0; };
            int now = entries(have), then = entries(have + 32);
            for (int t = g.t0; t < g.t1; ++t, ++it, rk.next(), rv.next()) {
                if ((t * kTile) >> a.page_log2 >= have + 32) {
                    have += 32;
                    now = then;
                    then = entries(have + 32);
                }
                const int tok = t * kTile + (lane << pr_log2);
                const bool there = lane < (kTile >> pr_log2) && tok < g.kv;
                const int page = __shfl_sync(0xFFFFFFFFu, now, (tok >> a.page_log2) & 31);
                const bool good = there && page >= 0 && page < a.num_pages;
                if (there && !good) raise_error(a.err, QVG_ERR_INVALID_ARG);
                const int off = tok & ((1 << a.page_log2) - 1);
                const long long at = good ? ((static_cast<long long>(page) * a.H + g.h) << a.page_log2) + off : -1;  // first row
                const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, good)) * C::kRow * pr;
#pragma unroll
                for (int which = 0; which < 2; ++which) {  // K, V
                    uint64_t *full = which ? &v_full[rv.i] : &k_full[rk.i];
                    const uint32_t dst = (which ? vr0 + rv.i * C::kRaw : kr0 + rk.i * C::kRaw) + lane * pr * C::kRow;
                    if (it >= (which ? SV : SK))
                        ok = ok && wait_here(which ? &v_empty[rv.i] : &k_empty[rk.i], (which ? rv.parity : rk.parity) ^ 1u, vfail, a.wait_ns);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (lane == 0) umma::mbar_arrive_expect_tx(full, bytes);
                    __syncwarp();
                    if (good) {
                        if (BITS == 8 && which == 0)
                            tma_load_4d(dst, &kmap, off, g.h, page, full);
                        else
                            bulk_copy(dst, (which ? a.vc : a.kc) + at * C::kRow, pr * C::kRow, full);
                    }
                    if (lane == 0) s_issued[which] = it + 1;
                    __syncwarp();
                }
                if (!ok) break;
#pragma unroll
                for (int i0 = 0; i0 < 16 * C::G; i0 += 32) {
                    const int i = i0 + lane;
                    const bool v = i >= 8 * C::G;
                    const int c = v ? i - 8 * C::G : i, first = c * (16 / C::G);
                    const long long piece_at = __shfl_sync(0xFFFFFFFFu, at, (first >> pr_log2) & 31);
                    if (i < 16 * C::G && piece_at >= 0)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(sc0 + rv.i * C::kScales + i * 16),
                                     "l"((v ? a.vs : a.ks) + (piece_at + (first & (pr - 1))) * C::G)
                                     : "memory");
                }
                umma::cp_async_arrive_noinc(&v_full[rv.i]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < 15) {
        // ---- a group's products: PV(t) and then S(t + 1), so that S is only written once its weights have been used
        const int grp = warp - 13;
        constexpr uint32_t id_s = idesc_f8(128, 128, 0), id_o = umma::idesc_f16_bmn(128, D, 0);
        const uint64_t dqh = desc_rows8<D>(q0 + grp * C::kQ), dql = desc_rows8<D>(q0 + grp * C::kQ + 128 * D);
        const uint32_t t_s = tmem + grp * 128, t_o = tmem + 256 + grp * 128;
        Segment g;
        Ring<SK> rk;
        int it = 0, mine = 0, n_own = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            if (lane == 0 && grp == 1 && !both(g)) {
                // no rows here: K's and V's buffers are given back as they come
                for (int t = g.t0; ok && t < g.t1; ++t, ++it, rk.next()) {
                    const int bf = it & 1;
                    ok = BITS == 8 ? wait_here(&k_full[rk.i], rk.parity, vfail, a.wait_ns) : wait_here(&ko_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                    ok = ok && wait_here(&vo_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                    if (!ok) break;
                    umma::mbar_arrive(BITS == 8 ? &k_empty[rk.i] : &ko_done[bf]);
                    umma::mbar_arrive(&vo_done[bf]);
                }
            } else if (lane == 0) {
                auto scores = [&](int i, const Ring<SK> &k) {
                    ok = ok && (BITS == 8 ? wait_here(&k_full[k.i], k.parity, vfail, a.wait_ns) : wait_here(&ko_full[i & 1], (i >> 1) & 1, vfail, a.wait_ns));
                    if (!ok) return;
                    umma::tc_fence_after();
                    const uint64_t dk = desc_rows8<D>(BITS == 8 ? kr0 + k.i * C::kRaw : k80 + (i & 1) * C::kK8);
#pragma unroll
                    for (int s = 0; s < D / 32; ++s) mma_f8(t_s, dqh + 2 * s, dk + 2 * s, id_s, s != 0);
#pragma unroll
                    for (int s = 0; s < D / 32; ++s) mma_f8(t_s, dql + 2 * s, dk + 2 * s, id_s, 1);
                    umma::mma_commit(&s_full[grp]);
                    umma::mma_commit(BITS == 8 ? &k_empty[k.i] : &ko_done[i & 1]);
                };
                ok = wait_here(&q_full[grp], n_own & 1, vfail, a.wait_ns);
                scores(it, rk);
                // test hook: with S in flight, wait for what never comes
                if (ok && mine == 0 && a.inject) ok = wait_here(&never, 0, vfail, a.wait_ns);
                for (int t = g.t0; ok && t < g.t1; ++t, ++it, ++mine) {
                    const int bf = it & 1;
                    ok = wait_here(&vo_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                    ok = ok && wait_here(&p_full[grp], mine & 1, vfail, a.wait_ns);
                    if (!ok) break;
                    umma::tc_fence_after();
                    const uint64_t dv = umma::desc_sw128_mn(vf0 + bf * C::kVf, kTile * 128);
#pragma unroll
                    for (int s = 0; s < kTile / 16; ++s) umma::mma_f16_ts(t_o, t_s + 8 * s, dv + s * 128, id_o, !(t == g.t0 && s == 0));
                    umma::mma_commit(&vo_done[bf]);
                    umma::mma_commit(&o_done[grp]);
                    rk.next();
                    if (t + 1 < g.t1) {
                        // (products of two kinds into different accumulators need not run in the order of issue)
                        ok = wait_here(&o_done[grp], mine & 1, vfail, a.wait_ns);
                        scores(it + 1, rk);
                    }
                }
                ++n_own;
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        // all products issued complete before TMEM goes back
        if (lane == 0) {
            umma::mma_commit(&drain);
            umma::mbar_wait(&drain, 0, kDrainNs);
        }
        __syncwarp();
    } else {
        // ---- this CTA's part of the line, unit by unit ------------------------------------------------
        Line<NB> line(a, s_chunk);
        bool ok = true;
        for (int n_seg = 0; ok; ++n_seg) {
            Segment g;
            line.next(a, g);
            const int i = n_seg & (kRing - 1);
            if (n_seg >= kRing) ok = wait_here(&seg_free[i], ((n_seg / kRing) - 1) & 1, vfail, a.wait_ns);
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
    }
    __syncwarp();
    umma::tc_fence_before();
    __syncthreads();
    if (tid == 0 && *vfail) {
        raise_error(a.err, QVG_ERR_TIMEOUT);
        // the copies in flight land before the CTA ends (K's of a tile may be out without V's)
        for (int j = max(0, s_issued[0] - SK); j < s_issued[0]; ++j) umma::mbar_wait(&k_full[j % SK], (j / SK) & 1, kDrainNs);
        for (int j = max(0, s_issued[1] - SV); j < s_issued[1]; ++j) umma::mbar_wait(&v_full[j % SV], (j / SV) & 1, kDrainNs);
    }
    if (warp == 15) {
        umma::tc_fence_after();
        umma::tmem_dealloc(tmem, 512);
    }
}

}  // namespace pa
}  // namespace qvg
