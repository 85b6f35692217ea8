// paged_attention.cuh -- attention of a few new tokens (one, a drafted tree, a
// short chunk) over a paged fp8 / fp4 cache: the kernel.  Launch, merge and
// entry points: paged_attention.cu.
//
// One unit of work is (sequence b, KV head h, block r of NB query rows); a
// query row is a (new token, query head of the group) pair, so the group's
// heads share each key and value that is read.  A unit walks its sequence in
// tiles of 128 keys.  All units' tiles form one line, which is cut into equal
// parts, one per CTA (one CTA per SM): ragged batches and single long
// sequences fill the GPU alike.  A unit cut by a border leaves fp32 partial
// sums that k_paged_merge joins.
//
// The product runs transposed, keys on the tensor core's 128 rows:
//   S^T [keys x rows] = K Q^T        K's fp8 codes as they lie in the cache
//   O^T [d x rows]   += V^T P^T      V's codes as fp16, P in fp16
// so its cost follows the number of query rows (N), not a padded 128.
//   - K needs no conversion: its codes are the A operand, and Q is the sum of
//     two fp8 numbers hi + lo (a bf16 number has 8 significant bits, an e4m3
//     number 4: exact while the channel is within 2^-10 of the row's largest),
//     two products into one accumulator.
//   - A key's scale is one number per row of S^T, i.e. per softmax thread.
//   - V's scale goes into the weight: w = p sv.  V's codes become fp16 in
//     shared memory (exact); w is rounded to fp16 (2^-11).
// Softmax: a thread owns one key and NC columns.  The weights of a column are
// taken relative to a reference that is set from the unit's first tile (its
// largest w becomes 2^kTarget) and raised when a w would pass 2^kTop, so the
// sums l and O are rescaled rarely, and a tile needs one vote, no maximum
// across threads.  A w 2^-29 below the reference's largest still counts in
// fp16 (subnormals); l takes p in fp32.
#pragma once

#include <cuda.h>

#include "paged.cuh"
#include "umma.cuh"

namespace qvg {
namespace pa {

constexpr int kTile = 128;
constexpr float kTarget = 4.0f, kTop = 15.0f;
constexpr uint64_t kDrainNs = 2000000000ull;

struct Args {
    const uint16_t *q;
    long long q_stride;
    int total_q, Hq, H, grp, B, max_q;
    const int32_t *cu_q, *table, *kv_len;
    long long table_stride;
    int mode;
    const uint32_t *mask;
    int words;
    float scale_log2;
    float *out32;
    uint16_t *out16;
    float *lse;
    const uint8_t *kc, *ks, *vc, *vs;
    int page_log2, num_pages;
    // workspace: partial sums of cut units, two slots per CTA (0: a unit that
    // began in an earlier CTA, 1: one that goes on in the next), and the
    // description of the unit that begins in this CTA and is cut
    float *po, *pm, *pl;
    int4 *desc;
    int *err;
    uint64_t wait_ns;
    int inject;
};

// ---- the line of tiles ----------------------------------------------------------

// Sequence b as the kernels see it, clamped to what the call promised.
struct Seq {
    int q0, nq, kv, nt, rb;
    __device__ __forceinline__ long long tiles(int H) const { return static_cast<long long>(H) * rb * nt; }
};

template <int NB>
__device__ __forceinline__ Seq seq_of(const Args &a, int b, bool report) {
    Seq s;
    int q0 = b * a.max_q, nq = a.max_q;
    bool bad = false;
    if (a.cu_q) {
        q0 = a.cu_q[b];
        nq = a.cu_q[b + 1] - q0;
        bad = nq < 0 || nq > a.max_q || q0 < 0 || q0 > a.total_q - nq;
        if (q0 < 0 || q0 > a.total_q) q0 = nq = 0;
        nq = max(0, min(min(nq, a.max_q), a.total_q - q0));
    }
    const long long most = a.table_stride << a.page_log2;
    int kv = a.kv_len[b];
    bad = bad || kv < 0 || kv > most;
    kv = static_cast<int>(max(0ll, min(static_cast<long long>(kv), most)));
    if (report && bad) raise_error(a.err, QVG_ERR_INVALID_ARG);
    s.q0 = q0;
    s.nq = nq;
    s.kv = kv;
    s.nt = max(1, static_cast<int>((static_cast<long long>(kv) + kTile - 1) / kTile));
    s.rb = static_cast<int>((static_cast<long long>(nq) * a.grp + NB - 1) / NB);
    return s;
}

// A stretch of one unit's tiles inside a CTA's part.
struct Segment {
    int b, h, r, t0, t1;
    Seq s;
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == s.nt; }
};

template <int NB>
struct Walk {
    long long pos, end, first;  // first: the position where sequence b begins
    int b;
    Seq s;

    __device__ __forceinline__ Walk(const Args &a, long long pos_, long long end_, int b_, long long first_)
        : pos(pos_), end(end_), first(first_), b(b_), s(seq_of<NB>(a, b_, false)) {}

    __device__ __forceinline__ bool next(const Args &a, Segment &g) {
        if (pos >= end) return false;
        while (pos >= first + s.tiles(a.H)) {
            first += s.tiles(a.H);
            s = seq_of<NB>(a, ++b, false);
        }
        const long long rel = pos - first;
        const long long u = rel / s.nt;
        g.b = b;
        g.s = s;
        g.h = static_cast<int>(u / s.rb);
        g.r = static_cast<int>(u % s.rb);
        g.t0 = static_cast<int>(rel - u * s.nt);
        g.t1 = static_cast<int>(min(static_cast<long long>(s.nt), g.t0 + (end - pos)));
        pos += g.t1 - g.t0;
        return true;
    }
};

// ---- small pieces ---------------------------------------------------------------

__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void up2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// 2^x, relative error about 2^-22; -inf gives 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Barrier over the 128 threads of softmax warpgroup `wg`; true if any of them
// brought true.
__device__ __forceinline__ bool wg_any(int wg, bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\t"
        "setp.ne.u32 a, %1, 0;\n\t"
        "barrier.cta.red.or.pred b, %2, 128, a;\n\t"
        "selp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r)
        : "r"(p ? 1u : 0u), "r"(wg + 1)
        : "memory");
    return r != 0;
}

// Bounded wait that also ends when another role has failed.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *fail, uint64_t limit_ns) {
    for (int i = 0; i < 32; ++i)
        if (umma::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = umma::globaltimer_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (umma::mbar_try_wait(bar, parity)) return true;
        if (*fail) return false;
        if (umma::globaltimer_ns() - t0 > limit_ns) {
            *fail = 1;
            return false;
        }
    }
}

// Contiguous global -> shared copy (16-byte aligned, a multiple of 16 bytes),
// counted on *bar in bytes.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(umma::smem_u32(bar))
                 : "memory");
}
// Tiled 4-D load at coordinates (0, c1, c2, c3).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *map, int c1, int c2, int c3, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(umma::smem_u32(bar))
        : "memory");
}

// Operand of one row of D bytes per key (or query row), K-major, swizzled:
// 128-byte rows with the 128-byte swizzle, 64-byte rows with the 64-byte one
// (16-byte piece c of row i at c ^ (i / 2 % 4)); eight rows are one atom.
template <int D>
__device__ __forceinline__ uint64_t desc_rows8(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((8 * D) >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(D == 128 ? 2u : 4u) << 61;
    return d;
}
template <int D>
__device__ __forceinline__ uint32_t swizzle8(uint32_t off) {
    return D == 128 ? off ^ ((off >> 3) & 0x70u) : off ^ ((off >> 3) & 0x30u);
}
// kind::f8f6f4 with A and B e4m3, both K-major; D fp32.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Lane i receives 16 consecutive columns of TMEM lane (base + i).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Sum or maximum over the warp's lanes of each of W columns held by every
// lane; lane i ends up with column i % W's.  W = 16 or 32.
template <int W, bool MAX>
__device__ __forceinline__ float across_lanes(float (&v)[W]) {
    const int lane = threadIdx.x & 31;
    if constexpr (W == 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float o = __shfl_xor_sync(0xFFFFFFFFu, v[i], 16);
            v[i] = MAX ? fmaxf(v[i], o) : v[i] + o;
        }
    }
#pragma unroll
    for (int s = W / 2; s > 0; s >>= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < s; ++i) {
            const float give = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
            const float o = __shfl_xor_sync(0xFFFFFFFFu, give, s);
            v[i] = MAX ? fmaxf(keep, o) : keep + o;
        }
    }
    return v[0];
}

// ---- shared memory ---------------------------------------------------------------

template <int D, int BITS, int NB>
struct Cfg {
    static constexpr int NSW = NB >= 64 ? 2 : 1;  // softmax warpgroups
    static constexpr int NC = NB / NSW;           // columns of a softmax thread
    static constexpr int G = BITS == 8 ? 1 : D / 32;
    static constexpr int kRow = D * BITS / 8;         // bytes of a row of codes
    static constexpr int kRaw = kTile * kRow;         // a tile's codes (K or V)
    static constexpr int kStage = 2 * kRaw + 1024;    // K, V, their scales
    static constexpr int kK8 = BITS == 4 ? kTile * D : 0;  // K as e4m3 (4 bits), two buffers
    static constexpr int kVf = kTile * D * 2;         // V as fp16, two buffers
    static constexpr int kP = 16384 * ((NB + 63) / 64);  // weights, two buffers
    static constexpr int kQ = NB * D;                 // Q hi; lo follows
    static constexpr int kFixed = 2 * kK8 + 2 * kVf + 2 * kP + 2 * kQ;
    static constexpr int kMaxStages = (225 * 1024 - 4096 - kFixed) / kStage;
    static constexpr int kStages = kMaxStages > 6 ? 6 : kMaxStages;
    static constexpr int kSmem = kFixed + kStages * kStage + 1024;
    static constexpr int kWarps = 8 + 4 * NSW;
    static constexpr int kTmem = NB == 16 ? 64 : NB == 32 ? 128 : 256;
    static_assert(kStages >= 2, "shared memory");
};

// e2m1 magnitudes times 2^(6 - k) as e4m3 bytes, for a group whose scale is
// 2^-k of the row's largest (k <= 14; beyond, the values are under 2^-9 and
// count as 0), eight bytes a row: the K operand of a 4-bit cache.
__device__ __forceinline__ uint2 k_levels(int k) {
    // magnitude 2^e m: byte (e + 7) << 3 | mantissa, subnormal below 2^-6
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        const float lv = i < 2 ? 0.5f : i < 4 ? 0.5f * i : i < 6 ? 1.0f * (i - 2) : 2.0f * (i - 4);
        const float x = k <= 14 ? lv * __uint_as_float(static_cast<uint32_t>(127 + 6 - k) << 23) : 0.0f;
        w[i >> 2] |= (e4m3x2(x, 0.0f) & 0xFFu) << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}

template <int D, int BITS, int NB>
__global__ void __launch_bounds__(Cfg<D, BITS, NB>::kWarps * 32, 1)
    k_paged_attention(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ Args a) {
    using C = Cfg<D, BITS, NB>;
    constexpr int S = C::kStages, NSW = C::NSW, NC = C::NC;
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t full[S], empty[S], s_full[2], s_free[2], p_full[2], v_full[2], k_full[2], k_done[2], pv_done[2],
        q_full, drain, never;
    __shared__ uint32_t tmem_base;
    __shared__ int fail, s_issued;
    __shared__ __align__(16) float2 s_qs[NB / 2], s_nm[NB / 2];  // per column: Q's scale, minus the reference
    __shared__ float s_red[4][NB], s_dl[NB];
    __shared__ int s_tok[NB];       // new token of each row
    __shared__ long long s_row[NB];  // out row, or -1
    __shared__ long long s_scan[C::kWarps], s_at[4];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;

    // ---- this CTA's part of the line ------------------------------------------------
    long long total = 0;
    {
        long long mine = 0;
        for (int b = tid; b < a.B; b += C::kWarps * 32) mine += seq_of<NB>(a, b, cta == 0).tiles(a.H);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
        if (lane == 0) s_scan[warp] = mine;
        if (tid == 0) fail = 0;
        __syncthreads();
        for (int w = 0; w < C::kWarps; ++w) total += s_scan[w];
        __syncthreads();
    }
    const long long per = max(1ll, (total + gridDim.x - 1) / gridDim.x);
    const long long pos0 = min(total, cta * per), pos1 = min(total, pos0 + per);
    if (tid == 0) a.desc[cta] = make_int4(-1, 0, 0, 0);
    if (pos0 >= pos1) return;
    {
        long long before = 0;  // tiles of the sequences before this round's
        for (int b0 = 0; b0 < a.B; b0 += C::kWarps * 32) {
            const int b = b0 + tid;
            const long long w = b < a.B ? seq_of<NB>(a, b, false).tiles(a.H) : 0;
            long long x = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) s_scan[warp] = x;
            __syncthreads();
            long long f = before + x - w;
            for (int v = 0; v < C::kWarps; ++v) {
                if (v < warp) f += s_scan[v];
                before += s_scan[v];
            }
            if (w > 0 && pos0 >= f && pos0 < f + w) s_at[0] = b, s_at[1] = f;
            if (w > 0 && pos1 - 1 >= f && pos1 - 1 < f + w) s_at[2] = b, s_at[3] = f;
            __syncthreads();
        }
    }
    const int b_at = static_cast<int>(s_at[0]);
    const long long f_at = s_at[1];
    if (tid == 0) {
        // the unit at the part's end: if it begins here and goes on, the CTAs that share it
        const int b = static_cast<int>(s_at[2]);
        const Seq s = seq_of<NB>(a, b, false);
        const long long u = (pos1 - 1 - s_at[3]) / s.nt;
        const long long u0 = s_at[3] + u * s.nt, u1 = u0 + s.nt;
        if (u0 >= pos0 && u1 > pos1)
            a.desc[cta] = make_int4(b, static_cast<int>(u / s.rb), static_cast<int>(u % s.rb), static_cast<int>((u1 - 1) / per));
    }

    uint8_t *base = dyn + ((1024u - (umma::smem_u32(dyn) & 1023u)) & 1023u);
    const uint32_t sm = umma::smem_u32(base);
    const uint32_t vf0 = sm, p0 = vf0 + 2 * C::kVf, k80 = p0 + 2 * C::kP, qh = k80 + 2 * C::kK8, ql = qh + C::kQ,
                   st0 = ql + C::kQ;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            umma::mbar_init(&full[i], 1);
            umma::mbar_init(&empty[i], (BITS == 8 ? 1 : 0) + 4 + 4 * NSW);  // S done, V read, scales read
        }
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(&s_full[i], 1);
            umma::mbar_init(&s_free[i], 4 * NSW);
            umma::mbar_init(&p_full[i], 4 * NSW);
            umma::mbar_init(&v_full[i], 4);
            umma::mbar_init(&k_full[i], 4);
            umma::mbar_init(&k_done[i], 1);
            umma::mbar_init(&pv_done[i], 1);
        }
        umma::mbar_init(&q_full, 4 * NSW);
        umma::mbar_init(&drain, 1);
        umma::mbar_init(&never, 1);
        umma::fence_barrier_init();
    }
    if (warp == 2) {
        umma::tmem_alloc(&tmem_base, C::kTmem);
        umma::tmem_relinquish();
    }
    __syncthreads();
    umma::tc_fence_after();
    const uint32_t tmem = tmem_base;
    const uint32_t t_o = tmem + 2 * NB;
    volatile int *vfail = &fail;
    const int n_tiles = static_cast<int>(pos1 - pos0);

    if (warp == 0) {
        // ---- loads: lane i fetches the tile's i-th piece (a page, or 128 tokens of one) ----
        const int pr_log2 = min(a.page_log2, 7), pr = 1 << pr_log2;
        const int pieces = kTile >> pr_log2;
        Walk<NB> walk(a, pos0, pos1, b_at, f_at);
        Segment g;
        int it = 0;
        bool ok = true;
        while (ok && walk.next(a, g)) {
            const int32_t *row = a.table + g.b * a.table_stride;
            for (int t = g.t0; t < g.t1; ++t, ++it) {
                const int tok = t * kTile + (lane << pr_log2);
                const bool there = lane < pieces && tok < g.s.kv;
                const int page = there ? row[tok >> a.page_log2] : 0;
                const bool good = there && page >= 0 && page < a.num_pages;
                if (there && !good) raise_error(a.err, QVG_ERR_INVALID_ARG);
                const int st = it % S;
                if (it >= S) ok = wait(&empty[st], ((it / S) - 1) & 1, vfail, a.wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, good));
                if (lane == 0) umma::mbar_arrive_expect_tx(&full[st], n * 2u * (C::kRow + C::G) * pr);
                __syncwarp();
                if (good) {
                    const uint32_t dst = st0 + st * C::kStage;
                    const int off = tok & ((1 << a.page_log2) - 1);
                    const size_t at = ((static_cast<size_t>(page) * a.H + g.h) << a.page_log2) + off;  // first row
                    if constexpr (BITS == 8)
                        tma_load_4d(dst + lane * pr * C::kRow, &kmap, off, g.h, page, &full[st]);
                    else
                        bulk_copy(dst + lane * pr * C::kRow, a.kc + at * C::kRow, pr * C::kRow, &full[st]);
                    bulk_copy(dst + C::kRaw + lane * pr * C::kRow, a.vc + at * C::kRow, pr * C::kRow, &full[st]);
                    bulk_copy(dst + 2 * C::kRaw + lane * pr * C::G, a.ks + at * C::G, pr * C::G, &full[st]);
                    bulk_copy(dst + 2 * C::kRaw + 512 + lane * pr * C::G, a.vs + at * C::G, pr * C::G, &full[st]);
                }
                __syncwarp();
            }
        }
        if (lane == 0) s_issued = it;
    } else if (warp == 1) {
        // ---- products ------------------------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_e4m3(128, NB), id_o = umma::idesc_f16(128, NB, 0) | (1u << 15) | (1u << 16);
            const uint64_t dqh = desc_rows8<D>(qh), dql = desc_rows8<D>(ql);
            bool ok = true;
            auto issue_s = [&](int it) {
                const int st = it % S, bf = it & 1;
                ok = ok && wait(&full[st], (it / S) & 1, vfail, a.wait_ns);
                if (BITS == 4) ok = ok && wait(&k_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                if (it >= 2) ok = ok && wait(&s_free[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
                if (!ok) return;
                umma::tc_fence_after();
                const uint64_t dk = desc_rows8<D>(BITS == 8 ? st0 + st * C::kStage : k80 + bf * C::kK8);
#pragma unroll
                for (int s = 0; s < D / 32; ++s) mma_f8(tmem + bf * NB, dk + 2 * s, dqh + 2 * s, id_s, s != 0);
#pragma unroll
                for (int s = 0; s < D / 32; ++s) mma_f8(tmem + bf * NB, dk + 2 * s, dql + 2 * s, id_s, 1);
                umma::mma_commit(&s_full[bf]);
                umma::mma_commit(BITS == 8 ? &empty[st] : &k_done[bf]);
            };
            auto issue_pv = [&](int it, bool fresh) {
                const int bf = it & 1;
                ok = ok && wait(&p_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                ok = ok && wait(&v_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                if (!ok) return;
                umma::tc_fence_after();
                // d = 64: the accumulator's upper 64 rows repeat the lower ones and are not read
                const uint64_t dv = umma::desc_sw128_mn(vf0 + bf * C::kVf, D == 128 ? kTile * 128 : 0);
                const uint64_t dp = umma::desc_sw128_mn(p0 + bf * C::kP, kTile * 128);
#pragma unroll
                for (int s = 0; s < kTile / 16; ++s)
                    umma::mma_f16(t_o, dv + s * 128, dp + s * 128, id_o, !(fresh && s == 0));
                umma::mma_commit(&pv_done[bf]);
            };
            Walk<NB> walk(a, pos0, pos1, b_at, f_at);
            Segment g;
            int it = 0, n_seg = 0;
            bool fresh = false;  // tile it - 1 opened its segment
            while (ok && walk.next(a, g)) {
                for (int t = g.t0; ok && t < g.t1; ++t, ++it) {
                    if (t == g.t0) {
                        if (it > 0) issue_pv(it - 1, fresh);
                        ok = ok && wait(&q_full, n_seg & 1, vfail, a.wait_ns);
                        ++n_seg;
                    }
                    issue_s(it);
                    // test hook: with S in flight, wait for what never comes
                    if (ok && it == 0 && a.inject) ok = wait(&never, 0, vfail, a.wait_ns);
                    if (t > g.t0) issue_pv(it - 1, fresh);
                    fresh = t == g.t0;
                }
            }
            if (ok && it > 0) issue_pv(it - 1, fresh);
            // all products issued complete before TMEM goes back
            umma::mma_commit(&drain);
            umma::mbar_wait(&drain, 0, kDrainNs);
        }
    } else if (warp >= 4 && warp < 8) {
        // ---- V (and 4-bit K) into operands ------------------------------------------------
        const int w = tid - 128;
        for (int it = 0; it < n_tiles; ++it) {
            const int st = it % S, bf = it & 1;
            const uint8_t *src = base + (st0 - sm) + st * C::kStage;
            uint8_t *vdst = base + (vf0 - sm) + bf * C::kVf;
            bool ok = wait(&full[st], (it / S) & 1, vfail, a.wait_ns);
            if (it >= 2) {
                if (BITS == 4) ok = ok && wait(&k_done[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
            }
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if constexpr (BITS == 8) {
                if (it >= 2) ok = wait(&pv_done[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                constexpr int PPR = D / 16;  // 16-code pieces a row
#pragma unroll
                for (int i = 0; i < kTile * PPR / 128; ++i) {
                    const int idx = w + 128 * i, row = idx / PPR, c = idx % PPR;
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + C::kRaw + idx * 16);
                    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
                    uint32_t o[8];
                    // a code that is no number (slots never written) becomes one: weights of 0 stay 0
                    const __half2 floor2 = __half2half2(__ushort_as_half(0xDF00));  // -448
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t h = e4m3x2_to_f16x2(vw[j / 2] >> (16 * (j & 1)));
                        const __half2 m = __hmax2(*reinterpret_cast<const __half2 *>(&h), floor2);
                        o[j] = *reinterpret_cast<const uint32_t *>(&m);
                    }
                    // channels 16 c .. of the row: 64-channel half, then 16-byte pieces 2 (c % 4), + 1
                    uint8_t *line = vdst + (c >> 2) * (kTile * 128) + row * 128;
                    const int e0 = ((2 * (c & 3)) ^ (row & 7)) << 4, e1 = ((2 * (c & 3) + 1) ^ (row & 7)) << 4;
                    const uint4 x = make_uint4(o[0], o[1], o[2], o[3]), y = make_uint4(o[4], o[5], o[6], o[7]);
                    // the halves' lanes store their pieces in opposite order: no bank twice
                    const bool swap = c >= 4;
                    *reinterpret_cast<uint4 *>(line + (swap ? e1 : e0)) = swap ? y : x;
                    *reinterpret_cast<uint4 *>(line + (swap ? e0 : e1)) = swap ? x : y;
                }
            } else {
                // one (row, 32-channel group) per step; the group's scale relative to the row's largest
                constexpr int GR = D / 32;
#pragma unroll 1
                for (int which = 0; which < 2; ++which) {
                    if (which == 1) {
                        if (it >= 2) ok = wait(&pv_done[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
                        if (!__all_sync(0xFFFFFFFFu, ok)) break;
                    }
#pragma unroll 2
                    for (int i = 0; i < GR; ++i) {
                        const int idx = w + 128 * i, row = idx / GR, gq = idx % GR;
                        const uint4 v = *reinterpret_cast<const uint4 *>(src + which * C::kRaw + idx * 16);
                        const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
                        const uint8_t *sc = src + 2 * C::kRaw + which * 512 + row * GR;
                        uint32_t top = 0;
#pragma unroll
                        for (int j = 0; j < GR; ++j) top = max(top, static_cast<uint32_t>(sc[j]));
                        const int down = static_cast<int>(top) - sc[gq];
                        if (which == 0) {
                            const uint2 lv = k_levels(down);
                            uint32_t o[8];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t mg = vw[j] & 0x77777777u, sg = vw[j] & 0x88888888u;
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const uint32_t m = __byte_perm(lv.x, lv.y, mg >> (16 * k));
                                    // 0xFF where the sign is set, 0x80 elsewhere: its low bit is the sign
                                    uint32_t s;
                                    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(s) : "r"(0x80u), "r"(sg >> (16 * k)));
                                    o[2 * j + k] = m | ((s << 7) & 0x80808080u);
                                }
                            }
                            uint8_t *kd = base + (k80 - sm) + bf * C::kK8;
                            *reinterpret_cast<uint4 *>(kd + swizzle8<D>(row * D + gq * 32)) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4 *>(kd + swizzle8<D>(row * D + gq * 32 + 16)) = make_uint4(o[4], o[5], o[6], o[7]);
                        } else {
                            // fp16 values of the codes times 2^-down (below 2^-24: 0)
                            const __half2 f = __half2half2(down > 24 ? __ushort_as_half(0) : __float2half_rn(__uint_as_float((127u - down) << 23)));
                            uint8_t *line = vdst + (gq >> 1) * (kTile * 128) + row * 128;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t o[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const uint32_t h = e2m1x2_to_f16x2((vw[j] >> (8 * k)) & 0xFFu);
                                    const __half2 m = __hmul2(*reinterpret_cast<const __half2 *>(&h), f);
                                    o[k] = *reinterpret_cast<const uint32_t *>(&m);
                                }
                                *reinterpret_cast<uint4 *>(line + (((4 * (gq & 1) + j) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                            }
                        }
                    }
                    if (which == 0) {
                        umma::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) umma::mbar_arrive(&k_full[bf]);
                    }
                }
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
            }
            umma::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                umma::mbar_arrive(&v_full[bf]);
                umma::mbar_arrive(&empty[st]);
            }
        }
    } else if (warp >= 8) {
        // ---- softmax: thread = key (S^T's row), columns [c0, c0 + NC) --------------------------
        const int wg = (warp - 8) >> 2, quad = warp & 3, r = quad * 32 + lane, c0 = wg * NC;
        const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
        Walk<NB> walk(a, pos0, pos1, b_at, f_at);
        Segment g;
        int it = 0;
        bool dead = false;
        while (!dead && walk.next(a, g)) {
            // Q rows of this warpgroup's columns: two fp8 numbers a channel
            {
                constexpr int LR = D / 8, RP = 128 / LR;  // lanes a row, rows a pass
#pragma unroll 1
                for (int n = c0 + r / LR; n < c0 + NC; n += RP) {
                    const long long gi = static_cast<long long>(g.r) * NB + n;
                    const int tq = static_cast<int>(gi / a.grp), j = static_cast<int>(gi - static_cast<long long>(tq) * a.grp);
                    const bool live = tq < g.s.nq;
                    const int ch = (r % LR) * 8;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (live)
                        v = *reinterpret_cast<const uint4 *>(a.q + (g.s.q0 + tq) * a.q_stride +
                                                             static_cast<long long>(g.h * a.grp + j) * D + ch);
                    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                    uint32_t m2 = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) m2 = __vmaxu2(m2, x[i] & 0x7FFF7FFFu);
                    uint32_t amax = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
                    for (int o = 1; o < LR; o <<= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
                    const uint32_t sb = scale_byte<8>(amax);
                    const float inv = sb == 255u ? 0.0f : scale_inverse(sb);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float f0 = __uint_as_float(x[i] << 16) * inv, f1 = __uint_as_float(x[i] & 0xFFFF0000u) * inv;
                        hi[i] = e4m3x2(f0, f1);
                        const uint32_t hh = e4m3x2_to_f16x2(hi[i]);
                        const float2 b2 = __half22float2(*reinterpret_cast<const __half2 *>(&hh));
                        lo[i] = e4m3x2(f0 - b2.x, f1 - b2.y);
                        if (sb == 255u) hi[i] = 0x7F7Fu, lo[i] = 0;  // an infinity or a NaN: the row is NaN
                    }
                    const uint32_t off = swizzle8<D>(n * D + ch);
                    *reinterpret_cast<uint2 *>(base + (qh - sm) + off) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                    *reinterpret_cast<uint2 *>(base + (ql - sm) + off) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                    if (r % LR == 0) {
                        reinterpret_cast<float *>(s_qs)[n] = sb == 255u ? 1.0f : scale_of(sb);
                        reinterpret_cast<float *>(s_nm)[n] = 0.0f;
                        s_tok[n] = live ? tq : 0;
                        s_row[n] = live ? static_cast<long long>(g.s.q0 + tq) * a.Hq + g.h * a.grp + j : -1;
                    }
                }
            }
            umma::fence_proxy_async_smem();
            wg_any(wg, false);
            if (lane == 0) umma::mbar_arrive(&q_full);

            uint64_t l2[NC / 2];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) l2[i] = 0;
            const int hist = g.s.kv - g.s.nq;  // keys before the new tokens
            const int clear = a.mode == QVG_MASK_NONE ? g.s.kv : min(g.s.kv, hist);
            for (int t = g.t0; t < g.t1; ++t, ++it) {
                const int st = it % S, bf = it & 1;
                const bool first = t == g.t0;
                bool ok = wait(&s_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                if (it >= 2) ok = ok && wait(&pv_done[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
                // (the scales landed with the tile whose S is here, but through the async proxy: wait on their own barrier)
                ok = ok && wait(&full[st], (it / S) & 1, vfail, a.wait_ns);
                umma::tc_fence_after();
                const uint8_t *sc = base + (st0 - sm) + st * C::kStage + 2 * C::kRaw;
                uint32_t kb = 0, vb = 0;
                if constexpr (BITS == 8) {
                    kb = sc[r];
                    vb = sc[512 + r];
                } else {
#pragma unroll
                    for (int j = 0; j < C::G; ++j) {
                        kb = max(kb, static_cast<uint32_t>(sc[r * C::G + j]));
                        vb = max(vb, static_cast<uint32_t>(sc[512 + r * C::G + j]));
                    }
                }
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&empty[st]);
                // 4 bits: K's operand is 2^6 times the values over the largest scale
                const float ka = scale_of(kb) * (BITS == 8 ? a.scale_log2 : a.scale_log2 * 0x1p-6f);
                const float sv = scale_of(vb), lsv = static_cast<float>(static_cast<int>(vb) - 127);
                const int key = t * kTile + r;
                const bool part = (t + 1) * kTile > clear;
                const uint64_t ka2 = pk2(ka, ka);
                float y[NC];
                // logits (base 2) less the reference; -inf where the row does not see the key
                auto logits = [&]() {
#pragma unroll
                    for (int c = 0; c < NC; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(tmem + t_lane + bf * NB + c0 + c, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 qs = s_qs[(c0 + c) / 2 + i], nm = s_nm[(c0 + c) / 2 + i];
                            const uint64_t x = mul2(pk2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), ka2);
                            up2(fma2(x, pk2(qs.x, qs.y), pk2(nm.x, nm.y)), y[c + 2 * i], y[c + 2 * i + 1]);
                        }
                    }
                    if (part) {
                        const int j = key - hist;
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            const int tq = s_tok[c0 + c];
                            bool see = key < g.s.kv;
                            if (see && j >= 0) {
                                if (a.mode == QVG_MASK_CAUSAL) see = j <= tq;
                                if (a.mode == QVG_MASK_TREE)
                                    see = (a.mask[static_cast<long long>(g.s.q0 + tq) * a.words + (j >> 5)] >> (j & 31)) & 1u;
                            }
                            if (!see) y[c] = -INFINITY;
                        }
                    }
                };
                logits();
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < NC; ++c) top = fmaxf(top, y[c]);
                if (wg_any(wg, first || !ok || top + lsv > kTop)) {
                    // set or raise references: the column maxima of w over the tile
                    float v[NC];
                    const float lw = fmaxf(lsv, -64.0f);
#pragma unroll
                    for (int c = 0; c < NC; ++c) v[c] = y[c] + lw;
                    const float m = across_lanes<NC, true>(v);
                    if (lane < NC) s_red[quad][c0 + lane] = m;
                    if (!first) ok = ok && wait(&pv_done[bf ^ 1], ((it - 1) >> 1) & 1, vfail, a.wait_ns);
                    dead = wg_any(wg, !ok);
                    if (dead) break;
                    umma::tc_fence_after();
                    if (r < NC) {
                        const int n = c0 + r;
                        const float mx = fmaxf(fmaxf(s_red[0][n], s_red[1][n]), fmaxf(s_red[2][n], s_red[3][n]));
                        const bool move = first ? mx > -INFINITY : mx > kTop;
                        const float d = move ? mx - kTarget : 0.0f;
                        reinterpret_cast<float *>(s_nm)[n] -= d;
                        s_dl[n] = ex2(-d);
                    }
                    wg_any(wg, false);
                    if (!first) {
#pragma unroll
                        for (int c = 0; c < NC; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(t_o + t_lane + c0 + c, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * s_dl[c0 + c + i]);
                            umma::tmem_st16(t_o + t_lane + c0 + c, o);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                l2[c / 2 + i] = mul2(l2[c / 2 + i], pk2(s_dl[c0 + c + 2 * i], s_dl[c0 + c + 2 * i + 1]));
                        }
                        umma::tmem_st_wait();
                    }
                    logits();
                }
                umma::tc_fence_before();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&s_free[bf]);
                uint8_t *prow = base + (p0 - sm) + bf * C::kP + r * 128;
#pragma unroll
                for (int c = 0; c < NC; c += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float pa = ex2(y[c + 2 * i]), pb = ex2(y[c + 2 * i + 1]);
                        l2[c / 2 + i] = add2(l2[c / 2 + i], pk2(pa, pb));
                        float wa = pa * sv, wb = pb * sv;
                        if (part) {  // an unseen key has weight 0 whatever its scale is
                            wa = y[c + 2 * i] == -INFINITY ? 0.0f : wa;
                            wb = y[c + 2 * i + 1] == -INFINITY ? 0.0f : wb;
                        }
                        w[i] = f16x2(wa, wb);
                    }
                    const int n = c0 + c;
                    *reinterpret_cast<uint4 *>(prow + (n >> 6) * (kTile * 128) + ((((n >> 3) & 7) ^ (r & 7)) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
                umma::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&p_full[bf]);
            }
            if (dead) break;
            // ---- the segment's sums ---------------------------------------------------------
            const int last = it - 1;
            const bool ok = wait(&pv_done[last & 1], (last >> 1) & 1, vfail, a.wait_ns);
            {
                float v[NC];
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) up2(l2[i], v[2 * i], v[2 * i + 1]);
                const float s = across_lanes<NC, false>(v);
                if (lane < NC) s_red[quad][c0 + lane] = s;
            }
            dead = wg_any(wg, !ok);
            if (dead) break;
            umma::tc_fence_after();
            const int slot = cta * 2 + (g.t0 > 0 ? 0 : 1);
            if (r < NC) {
                const int n = c0 + r;
                const float l = (s_red[0][n] + s_red[1][n]) + (s_red[2][n] + s_red[3][n]);
                const float m = -reinterpret_cast<float *>(s_nm)[n];
                if (g.whole()) {
                    s_dl[n] = l == 0.0f ? 0.0f : 1.0f / l;
                    const long long row = s_row[n];
                    if (a.lse && row >= 0)
                        a.lse[(row % a.Hq) * a.total_q + row / a.Hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                } else {
                    a.pm[static_cast<long long>(slot) * NB + n] = m;
                    a.pl[static_cast<long long>(slot) * NB + n] = l;
                }
            }
            wg_any(wg, false);
#pragma unroll 1
            for (int c = 0; c < NC; c += 16) {
                uint32_t o[16];
                tmem_ld16(t_o + t_lane + c0 + c, o);
                if (r < D) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int n = c0 + c + i;
                        const long long row = s_row[n];
                        if (row < 0) continue;
                        if (!g.whole())
                            a.po[(static_cast<long long>(slot) * NB + n) * D + r] = __uint_as_float(o[i]);
                        else if (a.out32)
                            a.out32[row * D + r] = __uint_as_float(o[i]) * s_dl[n];
                        else
                            a.out16[row * D + r] = f32_to_bf16(__uint_as_float(o[i]) * s_dl[n]);
                    }
                }
            }
            umma::tc_fence_before();
            wg_any(wg, false);  // s_row, s_dl and s_red have been read
        }
    }
    __syncwarp();
    umma::tc_fence_before();
    __syncthreads();
    if (tid == 0 && *vfail) {
        raise_error(a.err, QVG_ERR_TIMEOUT);
        // the copies in flight land before the CTA ends
        for (int j = max(0, s_issued - S); j < s_issued; ++j) umma::mbar_wait(&full[j % S], (j / S) & 1, kDrainNs);
    }
    if (warp == 2) {
        umma::tc_fence_after();
        umma::tmem_dealloc(tmem, C::kTmem);
    }
}

}  // namespace pa
}  // namespace qvg
