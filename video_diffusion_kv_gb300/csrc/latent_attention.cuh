// latent_attention.cuh -- attention of new tokens over a latent cache (absorbed
// form): the kernel.  Launch, join and entry points: latent_attention.cu.
//
// A query row is a (new token, query head) pair.  All heads read the same
// latents, so a unit of work is 128 rows of one sequence, and a tile's 64 keys
// are loaded once for both products: as K, and read across (MN-major) as V.  All
// units' tiles form one line that is cut into equal parts, one per CTA;
// a unit cut by a border leaves fp32 partial sums that k_latent_merge joins.
//
// Q's latent part is the A operand in tensor memory, where it costs shared
// memory's bandwidth nothing (from there the products take 46 clocks each, from shared
// memory 73) and leaves room for five stages of 256 + 64 channels; the rotated part is
// in shared memory.  S has two buffers of 64 columns, so that the next tile's S runs while
// this tile's softmax does.
//
// Bound: HBM for single tokens (a tile of 40 KB comes in 0.9 us, which is the rate of a
// plain copy), the products for many rows.  One token of 16 heads over
// 449,280 (256 + 64 channels, 288 MB): 60 us, 4.8 TB/s; of it 5 to 7 us until a CTA's
// first tile is there, 2 to 3 for the last tile and its sums, 8 for the join.  48 tokens of 32 heads over 700 to 24,000
// (381 MB): 74 us, 5.1 TB/s.  16 trees of 17 to 48 tokens, 16 heads, pages of 16 (6.8e10
// operations): 74 us, 920 TFLOP/s, 48 % of a large bf16 product's rate.
//
// Tensor memory: O 256 columns, S 2 x 64, Q 128.
// Roles: softmax (4 warps, thread = row), helpers (4: Q, and V in tiles that
// some row does not see all of), loads (4), S, PV, segments.
#pragma once

#include "bf16_attention.cuh"

namespace qvg {
namespace la {

// What a unit costs besides its tiles, in tiles: the line counts it, so that a CTA with
// three short units gets fewer tiles than one inside a long sequence (48 sequences of 700 to
// 24,000: 89 us without, 85 with).
constexpr int kUnitCost = 5;
constexpr int kLoads = 4, kLatentWarps = 4 + 4 + kLoads + 3;

// A unit of which a CTA has a part: the CTAs that share it, its rows (0: there
// is none), the first of them among the sequence's rows, the sequence's first token.
struct __align__(16) Shared {
    int first = 0, last = 0, rows = 0, row0 = 0, q0 = 0, pad[3] = {0, 0, 0};
};

// The sum, or 2^32 - 1 where it does not fit.
__device__ __forceinline__ uint32_t add_up_to(uint32_t x, uint32_t y) { return x + y < x ? UINT32_MAX : x + y; }

// cmap: latents; rmap: rotated key parts.
__global__ void __launch_bounds__(kLatentWarps * 32, 1)
    k_latent_attention(const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap rmap, const __grid_constant__ Args a) {
    constexpr int W0 = 4, WARPS = kLatentWarps;
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t full[kMostStages], empty[kMostStages], fixed[kFix];
    __shared__ uint64_t s_full[2], p_full[2], o_done[2], q_full, q_more, q_free, drain, never;
    __shared__ uint64_t seg_full[pa::kRing], seg_free[pa::kRing];
    __shared__ pa::Segment s_seg[pa::kRing];
    __shared__ uint2 s_bad[kFix];  // marked keys of a tile
    __shared__ uint32_t tmem_base;
    __shared__ int fail, issued[kLoads];  // tiles whose copies each loading warp has issued

    pdl_trigger();  // the join's blocks may take the places of CTAs that are done (they wait for all of them)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    uint8_t *base = dyn + ((1024u - (umma::smem_u32(dyn) & 1023u)) & 1023u);
    const uint32_t sm = umma::smem_u32(base);
    // Q's rotated part, then the stages: the rotated parts' chunks, the latents'
    const int stage = (a.na + a.nb) * kChunk;
    const uint32_t r0 = sm + a.na * kQChunk, c0 = r0 + a.na * kChunk;
    if (tid == 0) {
        fail = 0;
        for (int i = 0; i < kLoads; ++i) issued[i] = 0;
        for (int i = 0; i < kMostStages; ++i) {
            umma::mbar_init(&full[i], kLoads);
            umma::mbar_init(&empty[i], 5);  // PV, and the helpers' warps
        }
        for (int i = 0; i < kFix; ++i) umma::mbar_init(&fixed[i], 4);
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(&s_full[i], 1);
            umma::mbar_init(&p_full[i], 4);
            umma::mbar_init(&o_done[i], 1);
        }
        umma::mbar_init(&q_full, 4);
        umma::mbar_init(&q_more, 4);
        umma::mbar_init(&q_free, 1);
        umma::mbar_init(&drain, 2);
        umma::mbar_init(&never, 1);
        for (int i = 0; i < pa::kRing; ++i) {
            umma::mbar_init(&seg_full[i], 1);
            umma::mbar_init(&seg_free[i], WARPS - 1);
        }
        umma::fence_barrier_init();
    }
    if (warp == W0 + 5 + kLoads) {
        umma::tmem_alloc(&tmem_base, 512);
        umma::tmem_relinquish();
    }
    __syncthreads();
    umma::tc_fence_after();
    const uint32_t tmem = tmem_base, t_s0 = tmem + 256, t_q0 = tmem + 384;
    volatile int *vfail = &fail;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return pa::wait(bar, parity, vfail, a.wait_ns); };
    auto next_segment = [&](pa::Segment &g, int n) {
        const int i = n & (pa::kRing - 1);
        const bool ok = wait(&seg_full[i], (n / pa::kRing) & 1);
        g = s_seg[i];
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&seg_free[i]);
        return __all_sync(0xFFFFFFFFu, ok) && g.t1 > 0;
    };
    // The first key that some row of the unit does not see; whether tile t has such keys.
    auto clear_of = [&](const pa::Segment &g) {
        const int hist = g.kv - g.nq;
        if (a.mode == QVG_MASK_NONE) return g.kv;
        if (a.mode == QVG_MASK_TREE) return min(g.kv, hist);
        return min(g.kv, hist + 1 + static_cast<int>(static_cast<long long>(g.r) * kRows / a.grp));
    };
    // A row of Q into its lane of tensor memory, 128 channels at a time.
    struct Fetch {
        const uint4 *q;
        bool live;
        uint4 x[16];
        __device__ __forceinline__ void ask(int c, int nb) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = live && c * 8 + e < nb * 8 ? q[c * 8 + e] : make_uint4(0, 0, 0, 0);
        }
        __device__ __forceinline__ void put(uint32_t t_q, int c, int nb) const {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t y[32];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[4 * e] = x[8 * k + e].x, y[4 * e + 1] = x[8 * k + e].y, y[4 * e + 2] = x[8 * k + e].z, y[4 * e + 3] = x[8 * k + e].w;
                if (c + k < nb) umma::tmem_st32(t_q + (c + k) * 32, y);
            }
        }
    };
    auto row_of = [&](const pa::Segment &g, int w) {
        const uint32_t gi = static_cast<uint32_t>(g.r) * kRows + w;
        const int t = static_cast<int>(gi / static_cast<uint32_t>(a.grp)), h = static_cast<int>(gi) - t * a.grp;
        Fetch f;
        f.live = t < g.nq;
        f.q = reinterpret_cast<const uint4 *>(a.q + (g.q0 + (f.live ? t : 0)) * a.q_stride + (f.live ? h : 0) * a.q_h);
        return f;
    };
    auto partial = [&](int t, int clear) { return (t + 1) * kKeys > clear; };

    if (warp < W0) {
        // ---- softmax: thread = row -----------------------------------------------------------------
        const uint32_t t_lane = static_cast<uint32_t>(warp * 32) << 16, t_o = tmem + t_lane;
        pa::Segment g;
        int n = 0, n_fix = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            const uint32_t gi = static_cast<uint32_t>(g.r) * kRows + tid;
            const int tq = static_cast<int>(gi / static_cast<uint32_t>(a.grp)), h = static_cast<int>(gi) - tq * a.grp;
            const bool live = tq < g.nq, idle = !__any_sync(0xFFFFFFFFu, live);
            const int clear = clear_of(g);
            if (n_seg == 1) {  // the first unit's channels from 128 on: all at once they arrive a read earlier
                if (a.nb > 2) {
                    Fetch f = row_of(g, tid);
                    f.ask(2, a.nb);
                    f.put(t_q0 + t_lane, 2, a.nb);
                    umma::tmem_st_wait();
                }
                umma::tc_fence_before();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&q_more);
            }
            Row m;
            for (int t = g.t0; t < g.t1; ++t, ++n) {
                const int bf = n & 1;
                const bool part = partial(t, clear);
                ok = wait(&s_full[bf], (n >> 1) & 1);
                uint2 bad = make_uint2(0, 0);
                if (part) {
                    ok = ok && wait(&fixed[n_fix % kFix], (n_fix / kFix) & 1);
                    bad = s_bad[n_fix % kFix];
                    ++n_fix;
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                umma::tc_fence_after();
                if (!idle) {
                    uint2 see = make_uint2(0, 0);
                    if (part) see = seen_keys(a, t, g.kv, g.nq, g.q0, live ? tq : 0);
                    m.saw = m.saw || !part || (see.x | see.y) != 0u;
                    Logits v;
                    read_logits(v, t_s0 + bf * 64 + t_lane, part, see, bad);
                    const float f = raise_ref(a, m, largest(v), live);
                    if (t != g.t0 && __any_sync(0xFFFFFFFFu, f != 1.0f)) {
                        // the product of the tile before has to be in O
                        ok = wait(&o_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        umma::tc_fence_after();
                        rescale_rows(t_o, a.dv, f);
                    }
                    write_weights(a, m, v, t_s0 + bf * 64 + t_lane, f);
                }
                umma::tc_fence_before();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&p_full[bf]);
            }
            if (!ok) break;
            ok = wait(&o_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            umma::tc_fence_after();
            if (!idle)
                store_rows(a, m, t_o, false, live, g.whole(), cta * 2 + (g.t0 > 0 ? 0 : 1), tid, static_cast<long long>(g.q0 + tq) * a.Hq + h, h, g.q0 + tq);
            umma::tc_fence_before();
        }
    } else if (warp < W0 + 4) {
        // ---- helpers: Q, and V where some row does not see all of it ---------------------------------
        const int w = tid - W0 * 32;
        pa::Segment g;
        Ring rg;
        int n_fix = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            // (on their way before the last unit's products are done with its row)
            Fetch f = row_of(g, w);
            const uint32_t t_q = t_q0 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            const int upto = n_seg == 0 ? min(2, a.nb) : a.nb;  // (the first unit's others: the softmax warps)
            f.ask(0, upto);
            if (n_seg > 0) ok = wait(&q_free, (n_seg - 1) & 1);
            ++n_seg;
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            umma::tc_fence_after();  // (the stores into tensor memory come behind the products that have read the last unit's row)
            const int piece = w & 7;
            for (int i = w >> 3; a.na > 0 && i < kRows; i += 16) {
                const uint32_t gi = static_cast<uint32_t>(g.r) * kRows + i;
                const int tq = static_cast<int>(gi / static_cast<uint32_t>(a.grp)), h = static_cast<int>(gi) - tq * a.grp;
                if (tq >= g.nq) break;  // (rows that are left out keep what is there: no other row reads them)
                const uint16_t *qr = a.qr + (g.q0 + tq) * a.qr_t + h * a.qr_h + piece * 8;
                uint8_t *dst = base + i * 128 + ((piece ^ (i & 7)) << 4);
                for (int c = 0; c < a.na; ++c) {
                    const bool in = c * 64 + piece * 8 < a.dr;
                    umma::cp_async16(dst + c * kQChunk, in ? qr + c * 64 : a.q, in);
                }
            }
            for (int c = 0; c < upto; c += 2) {
                if (c > 0) f.ask(c, upto);
                f.put(t_q, c, upto);
            }
            umma::tmem_st_wait();
            umma::tc_fence_before();
            umma::cp_async_wait_all();
            umma::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&q_full);
            const int clear = clear_of(g);
            for (int t = g.t0; t < g.t1; ++t, rg.next(a.sb)) {
                ok = wait(&full[rg.i], rg.parity);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (partial(t, clear)) {
                    const int k0 = 16 * (warp - W0);
                    const uint32_t marks = clean16(base + (c0 - sm) + rg.i * stage, a.nb, k0, g.kv - t * kKeys);
                    __syncwarp();
                    if (lane == 0) {
                        reinterpret_cast<uint16_t *>(&s_bad[n_fix % kFix])[warp - W0] = static_cast<uint16_t>(marks);
                        umma::mbar_arrive(&fixed[n_fix % kFix]);
                    }
                    ++n_fix;
                }
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&empty[rg.i]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < W0 + 4 + kLoads) {
        // ---- loads -------------------------------------------------------------------------------------
        // A tile's latents take one copy where a page holds the whole tile (the first warp; the second one copies the
        // rotated parts), else one for each piece of a page and chunk, a warp each piece: a copy takes its thread about 100
        // clocks, which with 20 copies a tile (pages of 16) bounded the loop, 3100 clocks a tile with one warp, 1900 with two.
        const int me = warp - (W0 + 4), pr_log2 = min(a.page_log2, 6), pr = 1 << pr_log2, pieces = kKeys >> pr_log2;
        const bool one = elected();
        pa::Segment g;
        Ring rg;
        int it = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            // The page of piece `lane` of tile t, read a tile ahead (nothing looks at it before it is wanted); its first slot (-1:
            // no such page).
            auto page_of = [&](int t) {
                const long long tok = static_cast<long long>(t) * kKeys + (lane << pr_log2);
                return lane < pieces && tok < g.kv && t < g.t1 ? a.table[g.b * a.table_stride + (tok >> a.page_log2)] : -2;
            };
            auto first_of = [&](int t, int page) {
                if (page >= 0 && page < a.num_pages) return (page << a.page_log2) + ((t * kKeys + (lane << pr_log2)) & ((1 << a.page_log2) - 1));
                if (lane < pieces && static_cast<long long>(t) * kKeys + (lane << pr_log2) < g.kv) raise_error(a.err, QVG_ERR_INVALID_ARG);
                return -1;
            };
            int page = page_of(g.t0);
            for (int t = g.t0; t < g.t1; ++t, ++it, rg.next(a.sb)) {
                const int now = first_of(t, page);
                page = page_of(t + 1);
                if (it >= a.sb) ok = wait(&empty[rg.i], rg.parity ^ 1u);
                // (The first Q would wait behind all CTAs' first stages: it is there before the third one is asked for. Only
                // inside the first unit: Q of the second one needs this tile there, so the barrier is at its first or second phase.
                // Later it can be past that, and a wait for parity 0 would be one for the third unit's Q.)
                if (it == 2 && n_seg == 1) ok = ok && wait(&q_full, 0);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                uint64_t *bar = &full[rg.i];
                const uint32_t dst = c0 + rg.i * stage, dst_r = r0 + rg.i * stage;
                if (pieces == 1) {
                    const int at = __shfl_sync(0xFFFFFFFFu, now, 0);
                    if (one) umma::mbar_arrive_expect_tx(bar, at < 0 || me > 1 ? 0 : (me ? a.na : a.nb) * kChunk);
                    if (at >= 0) {
                        if (me == 0) {
                            if (one) tma_load_3d(dst, &cmap, 0, at, 0, bar);
                        } else if (me == 1) {
                            for (int c = 0; c < a.na; ++c)
                                if (one) tma_load_2d(dst_r + c * kChunk, &rmap, c * 64, at, bar);
                        }
                    }
                } else {
                    const int at = __shfl_sync(0xFFFFFFFFu, now, me);  // (-1 past the last piece, too)
                    if (one) umma::mbar_arrive_expect_tx(bar, at < 0 ? 0 : (a.na + a.nb) * (pr * 128));
                    if (at >= 0) {
                        for (int c = 0; c < a.nb; ++c)
                            if (one) tma_load_3d(dst + c * kChunk + me * (pr * 128), &cmap, 0, at, c, bar);
                        for (int c = 0; c < a.na; ++c)
                            if (one) tma_load_2d(dst_r + c * kChunk + me * (pr * 128), &rmap, c * 64, at, bar);
                    }
                }
                if (one) issued[me] = it + 1;
                __syncwarp();
            }
        }
        __syncwarp();
    } else if (warp == W0 + 4 + kLoads) {
        // ---- S -----------------------------------------------------------------------------------------
        constexpr uint32_t id = umma::idesc_f16(kRows, kKeys, 1);
        const bool one = elected();
        const uint64_t dq = umma::desc_sw128(sm);
        pa::Segment g;
        Ring rg;
        int n = 0, n_fix = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            const int clear = clear_of(g);
            ok = wait(&q_full, n_seg & 1);
            if (n_seg == 0) ok = ok && wait(&q_more, 0);
            ++n_seg;
            for (int t = g.t0; t < g.t1; ++t, ++n, rg.next(a.sb)) {
                const int bf = n & 1;
                ok = ok && wait(&full[rg.i], rg.parity);
                if (partial(t, clear)) {
                    ok = ok && wait(&fixed[n_fix % kFix], (n_fix / kFix) & 1);
                    ++n_fix;
                }
                if (n >= 2) ok = ok && wait(&o_done[bf], ((n >> 1) - 1) & 1);  // the buffer's last weights have been used
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                umma::tc_fence_after();
                const uint32_t t_s = t_s0 + bf * 64;
                uint32_t acc = 0;
                uint64_t dk = umma::desc_sw128(c0 + rg.i * stage);
                for (int c = 0; c < a.nb; ++c, dk += kChunk >> 4)
#pragma unroll
                    for (int s = 0; s < 4; ++s, acc = 1) mma_ts(t_s, t_q0 + c * 32 + 8 * s, dk + 2 * s, id, acc, one);
                dk = umma::desc_sw128(r0 + rg.i * stage);
                for (int c = 0; c < a.na; ++c, dk += kChunk >> 4) {
                    const int steps = min(4, (a.dr - c * 64 + 15) / 16);
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        if (s < steps) mma_ss(t_s, dq + c * (kQChunk >> 4) + 2 * s, dk + 2 * s, id, 1, one);
                }
                commit(&s_full[bf], one);
                // test hook: with S in flight, wait for what never comes
                if (a.inject && n == 0) ok = wait(&never, 0);
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) commit(&q_free, one);
        }
        commit(&drain, one);  // all products issued complete before tensor memory goes back
        umma::mbar_wait(&drain, 0, pa::kDrainNs);
        __syncwarp();
    } else if (warp == W0 + 5 + kLoads) {
        // ---- PV ---------------------------------------------------------------------------------------
        const uint32_t id = umma::idesc_f16_bmn(kRows, a.dv, 1);
        const bool one = elected();
        pa::Segment g;
        Ring rg;
        int n = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            for (int t = g.t0; t < g.t1; ++t, ++n, rg.next(a.sb)) {
                const int bf = n & 1;
                ok = wait(&full[rg.i], rg.parity);  // (long since: S has read the same stage)
                ok = ok && wait(&p_full[bf], (n >> 1) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                umma::tc_fence_after();
                const uint64_t dv = umma::desc_sw128_mn(c0 + rg.i * stage, kChunk);
#pragma unroll
                for (int s = 0; s < kKeys / 16; ++s) mma_ts(tmem, t_s0 + bf * 64 + 8 * s, dv + s * 128, id, !(t == g.t0 && s == 0), one);
                commit(&o_done[bf], one);
                commit(&empty[rg.i], one);
            }
        }
        commit(&drain, one);
        umma::mbar_wait(&drain, 0, pa::kDrainNs);
        __syncwarp();
    } else {
        // ---- this CTA's part of the line, unit by unit ---------------------------------------------------
        // One pass over the sequences for the line's length, then a walk from the sequence that holds the part's begin; 32
        // sequences at a time, a lane each.  The sums stop at 2^32 - 1: a line that gets there is refused.  (Code that runs once costs its instructions' way from L2, in a chain: this
        // loop in half the instructions gets the first tile going 2 us earlier.)
        Shared shared[2];  // the unit that this CTA goes on with, and the one that begins here and goes on
        bool ok = true, counting = true;
        uint32_t total = 0, first = 0, per = 1, pos = 0, end = 0;
        int n_seg = 0;
        auto publish = [&](const pa::Segment &g) {
            const int i = n_seg & (pa::kRing - 1);
            if (n_seg >= pa::kRing) ok = wait(&seg_free[i], ((n_seg / pa::kRing) - 1) & 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (lane == 0 && ok) {
                s_seg[i] = g;
                umma::mbar_arrive(&seg_full[i]);
            }
            ++n_seg;
        };
        for (int b0 = 0; ok && b0 < a.B;) {
            pa::Seq q{};
            uint32_t w = 0;
            if (b0 + lane < a.B) {
                q = pa::seq_of<kRows, kKeys>(a, b0 + lane, counting && cta == 0);
                const uint64_t units = static_cast<uint64_t>(q.rb) * static_cast<uint32_t>(q.nt + kUnitCost);
                w = static_cast<uint32_t>(min(units, static_cast<uint64_t>(UINT32_MAX)));
            }
            uint32_t x = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x = add_up_to(x, y);
            }
            const uint32_t all = __shfl_sync(0xFFFFFFFFu, x, 31);
            if (counting) {
                total = add_up_to(total, all);
                b0 += 32;
                if (b0 < a.B) continue;
                counting = false;
                if (total == UINT32_MAX) {
                    if (cta == 0 && lane == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
                    break;
                }
                per = max(1u, (total - 1) / gridDim.x + 1);
                pos = static_cast<uint32_t>(min(static_cast<uint64_t>(total), static_cast<uint64_t>(cta) * per));
                end = total - pos > per ? pos + per : total;
                b0 = 0;
                if (a.B > 32) continue;
            }
            while (ok && pos < end && pos - first < all) {
                const int l = __ffs(__ballot_sync(0xFFFFFFFFu, pos - first < x)) - 1;  // (the first sequence that ends behind pos)
                pa::Segment g;
                g.b = b0 + l;
                g.h = 0;
                g.q0 = __shfl_sync(0xFFFFFFFFu, q.q0, l);
                g.nq = __shfl_sync(0xFFFFFFFFu, q.nq, l);
                g.kv = __shfl_sync(0xFFFFFFFFu, q.kv, l);
                g.nt = __shfl_sync(0xFFFFFFFFu, q.nt, l);
                // `begin`: the unit's, behind which its tiles lie from kUnitCost on
                const uint32_t rel = pos - first - (__shfl_sync(0xFFFFFFFFu, x, l) - __shfl_sync(0xFFFFFFFFu, w, l)), length = g.nt + kUnitCost;
                g.r = static_cast<int>(rel / length);
                const uint32_t begin = pos - (rel - g.r * length), upto = min(end, begin + length);
                g.t0 = max(0, static_cast<int>(pos - begin) - kUnitCost);
                g.t1 = max(0, static_cast<int>(upto - begin) - kUnitCost);
                pos = upto;
                if (g.t1 <= g.t0) continue;  // (the part ends before the unit's first tile)
                publish(g);
                if (!g.whole() && (g.t0 == 0 || n_seg == 1)) {
                    Shared &d = shared[g.t0 == 0 ? 1 : 0];
                    d.first = static_cast<int>((begin + kUnitCost) / per);
                    d.last = static_cast<int>((begin + length - 1) / per);
                    d.row0 = g.r * kRows;
                    d.rows = static_cast<int>(min(static_cast<long long>(kRows), static_cast<long long>(g.nq) * a.grp - d.row0));
                    d.q0 = g.q0;
                }
            }
            if (pos >= end) break;
            first += all;
            b0 += 32;
        }
        pa::Segment none{};
        if (ok) publish(none);
        if (lane == 0) {
            if (!ok) shared[0].rows = shared[1].rows = 0;
            Shared *d = reinterpret_cast<Shared *>(a.desc);
            d[2 * cta] = shared[0];
            d[2 * cta + 1] = shared[1];
        }
    }
    __syncwarp();
    umma::tc_fence_before();
    __syncthreads();
    if (tid == 0 && *vfail) {
        raise_error(a.err, QVG_ERR_TIMEOUT);
        // The copies in flight land before the CTA ends (where one loading warp got further, the others' arrivals are made up for).
        int most = 0;
        for (int i = 0; i < kLoads; ++i) most = max(most, issued[i]);
        for (int i = 0; i < kLoads; ++i)
            for (int j = issued[i]; j < most; ++j) umma::mbar_arrive(&full[j % a.sb]);
        for (int j = max(0, most - a.sb); j < most; ++j) umma::mbar_wait(&full[j % a.sb], (j / a.sb) & 1, pa::kDrainNs);
    }
    if (warp == W0 + 5 + kLoads) {
        umma::tc_fence_after();
        umma::tmem_dealloc(tmem, 512);
    }
}

}  // namespace la
}  // namespace qvg
