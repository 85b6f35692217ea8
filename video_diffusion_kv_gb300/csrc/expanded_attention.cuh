// expanded_attention.cuh -- attention of prompts (expanded form): the kernel.
// Launch and entry point: latent_attention.cu.
//
// A unit of work is 256 query rows of one head, two groups of 128 that share
// each tile of K and V; one unit per CTA, the longest first.  S is made for 128
// keys at once, softmax and PV take 64 at a time: the first half's product runs
// while the second half's weights are made.  One group's products run while the other group is
// at its softmax.
//
// Bound: a group's chain, 4780 clocks for 128 keys of 128 + 64 channels (stamped): S 1440, the
// first half's softmax 930, the step to the second 340, its softmax 1110, PV until the next S 960.
//   4680 causal tokens of 16 heads
// (1.1e11 operations): 105 us, 1.07 PFLOP/s, 55 % of a large bf16 product's rate;
// without the mask 184 us, 1.22 PFLOP/s.  12 prompts of 1 to 1100 tokens after 0 to 1700, 8 heads, 64 + 32
// channels: 52 us, the longest unit's 44 tiles.
//   Tried and slower: two threads a row, a half each (157 us where one took 117 then: they meet
// once a tile, and V's tiles come too late with the room that is left), a part of the weights' powers by a
// polynomial beside the special function unit (112 us and more), S of 64 keys with two
// buffers (a product of 64 columns takes 73 clocks, one of 128 about 60).
//
// Tensor memory: O 2 x 128 columns, S 2 x 128.
// Roles: softmax (8 warps, thread = row), helpers (4: V in tiles that some row
// does not see all of), loads of Q and K, of V, and each group's products.
#pragma once

#include "bf16_attention.cuh"

namespace qvg {
namespace la {

constexpr int kPromptRows = 256, kPromptKeys = 128, kPromptWarps = 16;
constexpr int kKChunk = kPromptKeys * 128;  // 64 channels of K's tile

// A unit, and how many tiles of 64 keys each group needs.
struct Unit {
    int b, h, r, q0, nq, k0, kv, nt[2];
};
__device__ __forceinline__ Unit unit_of(const Args &a, int b, int r, int h, bool report) {
    Unit u;
    u.b = b;
    u.r = r;
    u.h = h;
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
    if (bad && report) raise_error(a.err, QVG_ERR_INVALID_ARG);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int first = u.r * kPromptRows + g * kRows, last = min(u.nq, first + kRows);
        const int end = first >= u.nq ? 0 : a.mode == QVG_MASK_CAUSAL ? min(u.kv, u.kv - u.nq + last) : u.kv;
        u.nt[g] = end <= 0 ? 0 : (end - 1) / kKeys + 1;
    }
    return u;
}

// The CTA's (sequence, block of rows); y < 0: none.  All heads of a block follow one another.
// - One sequence: the last rows first, which with a causal mask see the most keys.  (Counted from the
//   blocks that were launched: max_q may be far above the rows that there are.)
// - Up to kSorted possible blocks: ranked by their tiles (each CTA does it for itself: they
//   all get the same order), so that the short ones fill the GPU's end.  (The ragged prompts above, 60 blocks a
//   head: 52 us, 59 in the sequences' order.  The ranking takes a CTA the longer the more blocks there
//   are: 64 prompts of 10 to 1000 tokens, 256 blocks, 142 us, in the sequences' order 124.)
// - More: the blocks that there are, sequence by sequence, found from the lengths.
// `room`: shared memory for kSorted integers.
constexpr int kSorted = 256;
__host__ __device__ inline long long pair_count(int B, int blocks, int total_q) {
    const long long n = static_cast<long long>(B) * blocks, most = total_q / kPromptRows + static_cast<long long>(B);
    return n <= kSorted || n < most ? n : most;
}
__device__ __forceinline__ int2 pick(const Args &a, int blocks, uint32_t *room, int *got) {
    const long long n = static_cast<long long>(a.B) * blocks;
    const int want = blockIdx.x / a.H, i = threadIdx.x;
    if (a.B == 1) return make_int2(0, static_cast<int>(gridDim.x) / a.H - 1 - want);
    if (i == 0) *got = -1;
    if (n <= kSorted) {
        if (i < n) {
            const Unit u = unit_of(a, i % a.B, blocks - 1 - i / a.B, 0, false);
            room[i] = static_cast<uint32_t>(u.r * kPromptRows < u.nq ? min(max(u.nt[0], u.nt[1]) + 1, (1 << 24) - 1) : 0) << 8 | static_cast<uint32_t>(255 - i);
        }
        __syncthreads();
        if (i < n) {
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += room[j] > room[i];
            if (rank == want) *got = i;
        }
        __syncthreads();
        return make_int2(*got % a.B, blocks - 1 - *got / a.B);
    }
    const int lane = i & 31, warp = i >> 5;
    long long before = 0;
    int r = -1;
    for (int b0 = 0; b0 < a.B; b0 += kPromptWarps * 32) {
        const int b = b0 + i;
        int mine = 0;
        if (b < a.B) mine = (unit_of(a, b, 0, 0, blockIdx.x == 0).nq + kPromptRows - 1) / kPromptRows;
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) room[warp] = x;
        __syncthreads();
        int base = 0, all = 0;
        for (int k = 0; k < kPromptWarps; ++k) {
            base += k < warp ? static_cast<int>(room[k]) : 0;
            all += static_cast<int>(room[k]);
        }
        const long long end = before + base + x;
        if (want < end && want >= end - mine) {
            *got = b;
            room[kPromptWarps] = static_cast<uint32_t>(end - 1 - want);
        }
        before += all;
        __syncthreads();
    }
    if (*got >= 0) r = static_cast<int>(room[kPromptWarps]);
    return make_int2(max(*got, 0), r);
}

// qmap, rqmap: q and its rotated part; kmap, rkmap: k and the rotated key parts; vmap: v.
__global__ void __launch_bounds__(kPromptWarps * 32, 1)
    k_expanded_attention(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap rqmap,
                         const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap rkmap,
                         const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a, int blocks) {
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t a_full[kMostStages], a_empty[kMostStages], b_full[kMostStages], b_empty[kMostStages], fixed[kFix];
    __shared__ uint64_t s_full[2], p_full[2][2], o_done[2][2], q_full[2], step, drain, never;
    __shared__ uint2 s_bad[kFix];  // marked keys of a tile of 64
    __shared__ uint32_t tmem_base;
    __shared__ int fail, issued[2];  // tiles of K and of V whose copies have been issued

    __shared__ int picked;
    const int2 br = pick(a, blocks, reinterpret_cast<uint32_t *>(dyn), &picked);
    if (br.y < 0) return;
    const int head = blockIdx.x % a.H;
    const Unit u = unit_of(a, br.x, br.y, head, br.y == 0 && head == 0 && threadIdx.x == 0);
    if (u.r * kPromptRows >= u.nq) return;
    umma::fence_proxy_async_smem();  // (the room for the pick becomes the copies')
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q_group = a.na * kQChunk, a_bytes = a.na * kKChunk, b_bytes = a.nb * kChunk;
    uint8_t *base = dyn + ((1024u - (umma::smem_u32(dyn) & 1023u)) & 1023u);
    const uint32_t sm = umma::smem_u32(base);
    const uint32_t a0 = sm + 2 * q_group, b0 = a0 + a.sa * a_bytes;
    if (tid == 0) {
        fail = 0;
        issued[0] = issued[1] = 0;
        for (int i = 0; i < kMostStages; ++i) {
            umma::mbar_init(&a_full[i], 1);
            umma::mbar_init(&a_empty[i], 2);
            umma::mbar_init(&b_full[i], 1);
            umma::mbar_init(&b_empty[i], 6);  // each group, and the helpers' warps
        }
        for (int i = 0; i < kFix; ++i) umma::mbar_init(&fixed[i], 4);
        for (int g = 0; g < 2; ++g) {
            umma::mbar_init(&s_full[g], 1);
            umma::mbar_init(&q_full[g], 1);
            for (int i = 0; i < 2; ++i) {
                umma::mbar_init(&p_full[g][i], 4);
                umma::mbar_init(&o_done[g][i], 1);
            }
        }
        umma::mbar_init(&step, 1);  // completes once
        umma::mbar_init(&drain, 2);
        umma::mbar_init(&never, 1);
        umma::fence_barrier_init();
    }
    if (warp == 12) {
        umma::tmem_alloc(&tmem_base, 512);
        umma::tmem_relinquish();
    }
    __syncthreads();
    umma::tc_fence_after();
    const uint32_t tmem = tmem_base;  // O of the groups at 0 and 128, S at 256 and 384
    volatile int *vfail = &fail;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return pa::wait(bar, parity, vfail, a.wait_ns); };
    const int most = max(u.nt[0], u.nt[1]), hist = u.kv - u.nq;
    // The first key that some row of the unit does not see; whether tile t (of 64) has such keys.
    const int clear = a.mode == QVG_MASK_CAUSAL ? min(u.kv, hist + 1 + u.r * kPromptRows) : u.kv;
    auto partial = [&](int t) { return (t + 1) * kKeys > clear; };
    bool ok = true;

    if (warp < 8) {
        // ---- softmax: thread = row -----------------------------------------------------------------
        const int grp = warp >> 2;
        const uint32_t t_lane = static_cast<uint32_t>((warp & 3) * 32) << 16, t_o = tmem + grp * 128 + t_lane, t_s = tmem + 256 + grp * 128 + t_lane;
        const int tq = u.r * kPromptRows + tid, end = u.nt[grp];  // (thread tid of the eight warps has row tid)
        const bool live = tq < u.nq, idle = !__any_sync(0xFFFFFFFFu, live);
        int n_fix = 0;
        Row m;
        for (int t = 0; t < end; ++t) {
            const int half = t & 1, d = t >> 1;
            const bool part = partial(t);
            if (half == 0) ok = wait(&s_full[grp], d & 1);
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
                if (part) see = seen_keys(a, t, u.kv, u.nq, u.q0, live ? tq : 0);
                Logits v;
                read_logits(v, t_s + half * 64, part, see, bad);
                const float f = raise_ref(a, m, largest(v), live);
                if (t > 0 && __any_sync(0xFFFFFFFFu, f != 1.0f)) {
                    // the products before have to be in O (S of this tile came after those of the tile before)
                    if (half == 1) ok = wait(&o_done[grp][0], d & 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    umma::tc_fence_after();
                    rescale_rows(t_o, a.dv, f);
                }
                write_weights(a, m, v, t_s + half * 64, f);
            }
            umma::tc_fence_before();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&p_full[grp][half]);
        }
        if (ok && end > 0) ok = wait(&o_done[grp][(end - 1) & 1], ((end - 1) >> 1) & 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok) {
            umma::tc_fence_after();
            m.saw = u.kv > 0 && (a.mode == QVG_MASK_NONE || hist + tq >= 0);
            if (!idle) store_rows(a, m, t_o, end == 0, live, true, 0, 0, static_cast<long long>(u.q0 + tq) * a.Hq + u.h, u.h, u.q0 + tq);
        }
    } else if (warp < 12) {
        // ---- helpers: V where some row does not see all of it ----------------------------------------------
        Ring rb;
        int n_fix = 0;
        for (int t = 0; t < most; ++t, rb.next(a.sb)) {
            ok = wait(&b_full[rb.i], rb.parity);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (partial(t)) {
                const uint32_t marks = clean16(base + (b0 - sm) + rb.i * b_bytes, a.nb, 16 * (warp - 8), u.kv - t * kKeys);
                __syncwarp();
                if (lane == 0) {
                    reinterpret_cast<uint16_t *>(&s_bad[n_fix % kFix])[warp - 8] = static_cast<uint16_t>(marks);
                    umma::mbar_arrive(&fixed[n_fix % kFix]);
                }
                ++n_fix;
            }
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&b_empty[rb.i]);
        }
    } else if (warp == 12) {
        // ---- loads of Q and K: a copy for the channels, one for the rotated part -------------------------
        // (rows of Q past the sequence's are another one's, or 0; their results go nowhere)
        const bool one = elected();
        auto load_q = [&](int grp) {
            const int first = u.r * kPromptRows + grp * kRows;
            if (!one || u.nt[grp] == 0) return;
            umma::mbar_arrive_expect_tx(&q_full[grp], q_group);
            tma_load_4d(sm + grp * q_group, &qmap, 0, u.q0 + first, 0, u.h, &q_full[grp]);
            if (a.dr > 0) tma_load_3d(sm + grp * q_group + (a.na - 1) * kQChunk, &rqmap, 0, u.q0 + first, u.h, &q_full[grp]);
        };
        load_q(0);
        Ring ra;
        for (int d = 0; 2 * d < most; ++d, ra.next(a.sa)) {
            if (d >= a.sa) ok = wait(&a_empty[ra.i], ra.parity ^ 1u);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const uint32_t dst = a0 + ra.i * a_bytes;
            const int at = u.k0 + d * kPromptKeys;
            if (one) {
                umma::mbar_arrive_expect_tx(&a_full[ra.i], a_bytes);
                tma_load_4d(dst, &kmap, 0, at, 0, u.h, &a_full[ra.i]);
                if (a.dr > 0) tma_load_2d(dst + (a.na - 1) * kKChunk, &rkmap, 0, at, &a_full[ra.i]);
                issued[0] = d + 1;
            }
            if (d == 0) load_q(1);
            __syncwarp();
        }
    } else if (warp == 13) {
        // ---- loads of V -----------------------------------------------------------------------------------
        const bool one = elected();
        Ring rb;
        for (int t = 0; t < most; ++t, rb.next(a.sb)) {
            if (t >= a.sb) ok = wait(&b_empty[rb.i], rb.parity ^ 1u);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (one) {
                umma::mbar_arrive_expect_tx(&b_full[rb.i], b_bytes);
                tma_load_4d(b0 + rb.i * b_bytes, &vmap, 0, u.k0 + t * kKeys, 0, u.h, &b_full[rb.i]);
                issued[1] = t + 1;
            }
            __syncwarp();
        }
    } else {
        // ---- a group's products: S of 128 keys once all weights of the tile before have been used, PV of each half ----
        const int grp = warp - 14, mine = u.nt[grp], plain = a.dk / 64;
        constexpr uint32_t id_s = umma::idesc_f16(kRows, kPromptKeys, 1);
        const uint32_t id_o = umma::idesc_f16_bmn(kRows, a.dv, 1), t_s = tmem + 256 + grp * 128, t_o = tmem + grp * 128;
        const bool one = elected();
        const uint64_t dq = umma::desc_sw128(sm + grp * q_group);
        const int steps_r = (a.dr + 15) / 16;
        Ring ra, rb;
        int n_fix = 0;
        if (mine > 0) ok = wait(&q_full[grp], 0);
        // The groups out of step: group 1 begins once group 0 has its first weights.  (That barrier completes again with group
        // 0's next 128 keys, which wait until group 1 has seen it: else its parity might have come round.  With a barrier
        // of its own that the softmax warps arrive at, 104.6 us for the first case where this takes 103.8.)
        if (grp == 1 && u.nt[0] > 0) ok = ok && wait(&p_full[0][0], 0);
        __syncwarp();
        if (grp == 1 && one && ok) umma::mbar_arrive(&step);
        for (int d = 0; 2 * d < most; ++d, ra.next(a.sa)) {
            if (grp == 0 && d == 1) ok = ok && wait(&step, 0);
            ok = ok && wait(&a_full[ra.i], ra.parity);
            if (2 * d < mine) {
                if (d > 0) ok = ok && wait(&o_done[grp][1], (d - 1) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                umma::tc_fence_after();
                const uint64_t dk = umma::desc_sw128(a0 + ra.i * a_bytes);
                for (int c = 0; c < plain; ++c)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        mma_ss(t_s, dq + c * (kQChunk >> 4) + 2 * s, dk + c * (kKChunk >> 4) + 2 * s, id_s, c | s, one);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (s < steps_r) mma_ss(t_s, dq + plain * (kQChunk >> 4) + 2 * s, dk + plain * (kKChunk >> 4) + 2 * s, id_s, 1, one);
                commit(&s_full[grp], one);
                commit(&a_empty[ra.i], one);
                // test hook: with S in flight, wait for what never comes
                if (a.inject && d == 0) ok = wait(&never, 0);
            } else {
                __syncwarp();  // (all lanes have seen the stage)
                if (one && ok) umma::mbar_arrive(&a_empty[ra.i]);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int t = 2 * d + half;
                if (t >= most) break;
                ok = ok && wait(&b_full[rb.i], rb.parity);
                if (partial(t)) {
                    ok = ok && wait(&fixed[n_fix % kFix], (n_fix / kFix) & 1);
                    ++n_fix;
                }
                if (t < mine) ok = ok && wait(&p_full[grp][half], d & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (t < mine) {
                    umma::tc_fence_after();
                    const uint64_t dv = umma::desc_sw128_mn(b0 + rb.i * b_bytes, kChunk);
#pragma unroll
                    for (int s = 0; s < kKeys / 16; ++s) mma_ts(t_o, t_s + half * 64 + 8 * s, dv + s * 128, id_o, t > 0 || s > 0, one);
                    commit(&o_done[grp][half], one);
                    commit(&b_empty[rb.i], one);
                } else if (one) {
                    umma::mbar_arrive(&b_empty[rb.i]);
                }
                __syncwarp();
                rb.next(a.sb);
            }
            if (!ok) break;
        }
        commit(&drain, one);  // all products issued complete before tensor memory goes back
        umma::mbar_wait(&drain, 0, pa::kDrainNs);
    }
    __syncwarp();
    umma::tc_fence_before();
    __syncthreads();
    if (tid == 0 && *vfail) {
        raise_error(a.err, QVG_ERR_TIMEOUT);
        // the copies in flight land before the CTA ends (Q's are issued with K's first)
        for (int g = 0; g < 2; ++g)
            if (u.nt[g] > 0) umma::mbar_wait(&q_full[g], 0, pa::kDrainNs);
        for (int j = max(0, issued[0] - a.sa); j < issued[0]; ++j) umma::mbar_wait(&a_full[j % a.sa], (j / a.sa) & 1, pa::kDrainNs);
        for (int j = max(0, issued[1] - a.sb); j < issued[1]; ++j) umma::mbar_wait(&b_full[j % a.sb], (j / a.sb) & 1, pa::kDrainNs);
    }
    if (warp == 12) {
        umma::tc_fence_after();
        umma::tmem_dealloc(tmem, 512);
    }
}

}  // namespace la
}  // namespace qvg
