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
// The product runs transposed, keys on the tensor core's 128 rows, and takes
// the cache's fp8 codes as they lie there (4-bit codes become fp8 first):
//   S^T [keys x rows] = K Q^T        A = K's codes
//   O^T [d x rows]   += V^T P^T      A = V's codes, read across (MN-major)
// so its cost follows the number of query rows (N), not a padded 128, and K
// and V are touched once by the copy and once by the tensor core.  The other
// operand is made of several fp8 numbers side by side along N, each with its
// own accumulator columns; a product with N <= 64 takes the tensor core the
// same 45 clocks whatever N is, so the extra columns are free there:
//   - Q as two: hi + lo / 16 in e4m3 (4 significant bits each, a bf16 number
//     has 8: exact while the channel is within 2^-14 of the row's largest);
//   - P as three: h1 + h2 / 8 + h3 / 64 in e5m2, the first two cut off an
//     fp16 number's upper byte (e5m2 is just that), the last rounded: at most
//     2^-9 of the weight off, and fp16's range, which e4m3 lacks.
// A key's scale is one number per row of S^T, i.e. per softmax thread; V's
// scale goes into the weight: w = p sv.
// Softmax: a thread owns one key and NC columns.  The weights of a column are
// taken relative to a reference that is set from the first tile (its largest
// w becomes 2^kTarget) and raised when a w would pass 2^kTop, so the sums l
// and O are rescaled rarely, and a tile needs one vote, no maximum across
// threads.  A w of 2^-26 of the reference's largest still counts; l takes p in
// fp32.
// Up to 32 query rows, two softmax warpgroups take the tiles in turn, each
// with its own reference and sums (two streams, joined at the unit's end);
// with 64 rows they share every tile, 32 columns each.
#pragma once

#include <cuda.h>

#include "paged.cuh"
#include "umma.cuh"

namespace qvg {
namespace pa {

constexpr int kTile = 128;
constexpr float kTarget = 4.0f, kTop = 14.0f;  // a w up to 2^14: its remainders times 8 stay in fp16
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

// Barrier `id` over `count` threads; true if any of them brought true.
__device__ __forceinline__ bool any_of(int id, int count, bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\t"
        "setp.ne.u32 a, %1, 0;\n\t"
        "barrier.cta.red.or.pred b, %2, %3, a;\n\t"
        "selp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r)
        : "r"(p ? 1u : 0u), "r"(id), "r"(count)
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

// Tiles of one row of D bytes per key (or query row), swizzled in 16-byte
// pieces: 128-byte rows with the 128-byte swizzle (piece c of row i at
// c ^ (i % 8)), 64-byte rows with the 64-byte one (c ^ (i / 2 % 4)).  Eight
// rows are one atom.  The same bytes serve as a K-major operand (the product
// runs along the row) and as an MN-major one (it runs down the rows; lbo: from
// one D-wide block to the next).
template <int D>
__device__ __forceinline__ uint64_t desc_rows8(uint32_t addr, uint32_t lbo = 0) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>((8 * D) >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(D == 128 ? 2u : 4u) << 61;
    return d;
}
template <int D>
__device__ __forceinline__ uint32_t swizzle8(uint32_t off) {
    return D == 128 ? off ^ ((off >> 3) & 0x70u) : off ^ ((off >> 3) & 0x30u);
}
// kind::f8f6f4, A e4m3, B e4m3 (b = 0) or e5m2 (b = 1), D fp32, K-major.
__host__ __device__ constexpr uint32_t idesc_f8(uint32_t M, uint32_t N, uint32_t b) {
    return (1u << 4) | (b << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Lane i receives 16 consecutive columns of TMEM lane (base + i), from each
// of two places.
__device__ __forceinline__ void tmem_ld16x2(uint32_t t0, uint32_t t1, uint32_t (&r)[16], uint32_t (&q)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(q[0]),
          "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]), "=r"(q[9]),
          "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15])
        : "r"(t0), "r"(t1)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
}
// Eight columns from each of three places `step` columns apart (the three
// parts of O).
__device__ __forceinline__ void tmem_ld8x3(uint32_t t, uint32_t step, uint32_t (&a)[8], uint32_t (&b)[8], uint32_t (&c)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%24];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%25];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%26];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(b[0]),
          "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(c[0]), "=r"(c[1]),
          "=r"(c[2]), "=r"(c[3]), "=r"(c[4]), "=r"(c[5]), "=r"(c[6]), "=r"(c[7])
        : "r"(t), "r"(t + step), "r"(t + 2 * step)
        : "memory");
}

// Four weights (two fp16 pairs) -> their three e5m2 parts, four bytes each.
__device__ __forceinline__ void three_parts(uint32_t a, uint32_t b, uint32_t &h1, uint32_t &h2, uint32_t &h3) {
    const __half2 eight = __half2half2(__ushort_as_half(0x4800));  // 8
    auto rest = [&](uint32_t x) {  // 8 (x - its upper byte): exact
        const uint32_t cut = x & 0xFF00FF00u;
        const __half2 d = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&cut)), eight);
        return *reinterpret_cast<const uint32_t *>(&d);
    };
    h1 = __byte_perm(a, b, 0x7531);
    a = rest(a);
    b = rest(b);
    h2 = __byte_perm(a, b, 0x7531);
    a = rest(a);
    b = rest(b);
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(lo) : "r"(a));
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(hi) : "r"(b));
    h3 = static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
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
    static constexpr int NSTR = NB <= 32 ? 2 : 1;   // streams (see above)
    static constexpr int NC = NSTR == 2 ? NB : NB / 2;  // columns of a softmax thread
    static constexpr int kParty = NSTR == 2 ? 4 : 8;    // softmax warps on one tile
    static constexpr int G = BITS == 8 ? 1 : D / 32;
    static constexpr int kRow = D * BITS / 8;         // bytes of a row of codes
    static constexpr int kRaw = kTile * kRow;         // a tile's codes (K or V)
    static constexpr int kStage = 2 * kRaw + 1024;    // K, V, their scales
    static constexpr int kOp = BITS == 4 ? kTile * D : 0;  // K or V as e4m3 (4 bits), two buffers each
    static constexpr int kP = 16384 * ((3 * NB + 127) / 128);  // weights, two buffers
    static constexpr int kQ = 2 * NB * D;             // Q: hi rows, lo rows
    static constexpr int kFixed = 4 * kOp + 2 * kP + kQ;
    static constexpr int kMaxStages = (225 * 1024 - 6144 - kFixed) / kStage;
    static constexpr int kStages = kMaxStages > 8 ? 8 : kMaxStages;
    static constexpr int kSmem = kFixed + kStages * kStage + 1024;
    static constexpr int kConv = BITS == 4 ? 4 : 0;   // converter warps
    static constexpr int kWarps = 12 + kConv;         // loads, S, PV, TMEM; softmax 4 - 11; converters
    static constexpr int kTmemUsed = 2 * 2 * NB + NSTR * 3 * NB;
    static constexpr int kTmem = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
    static_assert(kStages >= 3, "shared memory");
};

// e2m1 magnitudes times 2^(6 - k) as e4m3 bytes, for a group whose scale is
// 2^-k of the row's largest (k <= 14; beyond, the values are under 2^-9 and
// count as 0), eight bytes: the operands of a 4-bit cache.
__device__ __forceinline__ uint2 levels_of(int k) {
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
    k_paged_attention(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ Args a) {
    using C = Cfg<D, BITS, NB>;
    constexpr int S = C::kStages, NSTR = C::NSTR, NC = C::NC;
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t full[S], empty[S], s_full[2], s_free[2], p_full[2], v_full[2], k_full[2], k_done[2], pv_done[2],
        q_full, drain, never;
    __shared__ uint32_t tmem_base;
    __shared__ int fail, s_issued;
    __shared__ __align__(16) float s_qs[NB], s_nm[NSTR][NB];  // per column: Q's scale, minus the reference
    __shared__ __align__(16) float s_red[2][4][NB], s_dl[2][NB], s_l[NSTR][NB], s_wt[NSTR][NB];
    __shared__ int s_tok[NB];        // new token of each row
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
    const uint32_t p0 = sm, k80 = p0 + 2 * C::kP, v80 = k80 + 2 * C::kOp, q0 = v80 + 2 * C::kOp, st0 = q0 + C::kQ;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            umma::mbar_init(&full[i], 1);
            umma::mbar_init(&empty[i], (BITS == 8 ? 2 : 4) + C::kParty);  // products (or converters) done, scales read
        }
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(&s_full[i], 1);
            umma::mbar_init(&s_free[i], C::kParty);
            umma::mbar_init(&p_full[i], C::kParty);
            umma::mbar_init(&v_full[i], 4);
            umma::mbar_init(&k_full[i], 4);
            umma::mbar_init(&k_done[i], 1);
            umma::mbar_init(&pv_done[i], 1);
        }
        umma::mbar_init(&q_full, 8);
        umma::mbar_init(&drain, 2);
        umma::mbar_init(&never, 1);
        umma::fence_barrier_init();
    }
    if (warp == 3) {
        umma::tmem_alloc(&tmem_base, C::kTmem);
        umma::tmem_relinquish();
    }
    __syncthreads();
    umma::tc_fence_after();
    const uint32_t tmem = tmem_base;
    const uint32_t t_o = tmem + 4 * NB;  // S: two buffers of 2 NB columns; O: 3 NB per stream
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
                    if constexpr (BITS == 8) {
                        tma_load_4d(dst + lane * pr * C::kRow, &kmap, off, g.h, page, &full[st]);
                        tma_load_4d(dst + C::kRaw + lane * pr * C::kRow, &vmap, off, g.h, page, &full[st]);
                    } else {
                        bulk_copy(dst + lane * pr * C::kRow, a.kc + at * C::kRow, pr * C::kRow, &full[st]);
                        bulk_copy(dst + C::kRaw + lane * pr * C::kRow, a.vc + at * C::kRow, pr * C::kRow, &full[st]);
                    }
                    bulk_copy(dst + 2 * C::kRaw + lane * pr * C::G, a.ks + at * C::G, pr * C::G, &full[st]);
                    bulk_copy(dst + 2 * C::kRaw + 512 + lane * pr * C::G, a.vs + at * C::G, pr * C::G, &full[st]);
                }
                __syncwarp();
            }
        }
        if (lane == 0) s_issued = it;
    } else if (warp == 1) {
        // ---- S = K Q^T -------------------------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t id = idesc_f8(128, 2 * NB, 0);
            const uint64_t dq = desc_rows8<D>(q0);
            Walk<NB> walk(a, pos0, pos1, b_at, f_at);
            Segment g;
            int it = 0, n_seg = 0;
            bool ok = true;
            while (ok && walk.next(a, g)) {
                ok = wait(&q_full, n_seg & 1, vfail, a.wait_ns);
                ++n_seg;
                for (int t = g.t0; ok && t < g.t1; ++t, ++it) {
                    const int st = it % S, bf = it & 1;
                    ok = BITS == 8 ? wait(&full[st], (it / S) & 1, vfail, a.wait_ns)
                                   : wait(&k_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                    if (it >= 2) ok = ok && wait(&s_free[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
                    if (!ok) break;
                    umma::tc_fence_after();
                    const uint64_t dk = desc_rows8<D>(BITS == 8 ? st0 + st * C::kStage : k80 + bf * C::kOp);
#pragma unroll
                    for (int s = 0; s < D / 32; ++s) mma_f8(tmem + bf * 2 * NB, dk + 2 * s, dq + 2 * s, id, s != 0);
                    umma::mma_commit(&s_full[bf]);
                    umma::mma_commit(BITS == 8 ? &empty[st] : &k_done[bf]);
                    // test hook: with S in flight, wait for what never comes
                    if (it == 0 && a.inject) ok = wait(&never, 0, vfail, a.wait_ns);
                }
            }
            umma::mma_commit(&drain);
        }
    } else if (warp == 2) {
        // ---- O += V^T P^T (its own warp: starting a batch of products takes longer than the batch) ----
        if (lane == 0) {
            constexpr uint32_t id = idesc_f8(128, 3 * NB, 1) | (1u << 15) | (1u << 16);  // both MN-major
            Walk<NB> walk(a, pos0, pos1, b_at, f_at);
            Segment g;
            int it = 0;
            bool ok = true;
            while (ok && walk.next(a, g)) {
                for (int t = g.t0; ok && t < g.t1; ++t, ++it) {
                    const int st = it % S, bf = it & 1;
                    // (4 bits: the stage itself may be in its next use by now)
                    ok = BITS == 8 ? wait(&full[st], (it / S) & 1, vfail, a.wait_ns)
                                   : wait(&v_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                    ok = ok && wait(&p_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                    if (!ok) break;
                    umma::tc_fence_after();
                    // d = 64: the accumulator's upper 64 rows repeat the lower ones and are not read
                    const uint64_t dv = desc_rows8<D>(BITS == 8 ? st0 + st * C::kStage + C::kRaw : v80 + bf * C::kOp);
                    const uint64_t dp = desc_rows8<128>(p0 + bf * C::kP, kTile * 128);
                    const bool fresh = t - g.t0 < NSTR;  // the stream's first tile of the unit
#pragma unroll
                    for (int s = 0; s < kTile / 32; ++s)
                        mma_f8(t_o + (NSTR == 2 ? bf * 3 * NB : 0), dv + s * (32 * D / 16), dp + s * 256, id, !(fresh && s == 0));
                    umma::mma_commit(&pv_done[bf]);
                    if (BITS == 8) umma::mma_commit(&empty[st]);
                }
            }
            // all products issued, S's too, complete before TMEM goes back
            umma::mma_commit(&drain);
            umma::mbar_wait(&drain, 0, kDrainNs);
        }
    } else if (warp >= 12) {
        // ---- 4-bit codes into e4m3 operands: one (row, 32-channel group) a step, its scale relative to the row's largest
        const int w = tid - 384;
        constexpr int GR = D / 32;
        for (int it = 0; it < n_tiles; ++it) {
            const int st = it % S, bf = it & 1;
            const uint8_t *src = base + (st0 - sm) + st * C::kStage;
            bool ok = wait(&full[st], (it / S) & 1, vfail, a.wait_ns);
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                if (it >= 2) ok = ok && wait(which ? &pv_done[bf] : &k_done[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                uint8_t *dst = base + ((which ? v80 : k80) - sm) + bf * C::kOp;
#pragma unroll 2
                for (int i = 0; i < GR; ++i) {
                    const int idx = w + 128 * i, row = idx / GR, gq = idx % GR;
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + which * C::kRaw + idx * 16);
                    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
                    const uint8_t *sc = src + 2 * C::kRaw + which * 512 + row * GR;
                    uint32_t top = 0;
#pragma unroll
                    for (int j = 0; j < GR; ++j) top = max(top, static_cast<uint32_t>(sc[j]));
                    const uint2 lv = levels_of(static_cast<int>(top) - sc[gq]);
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
                    *reinterpret_cast<uint4 *>(dst + swizzle8<D>(row * D + gq * 32)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(dst + swizzle8<D>(row * D + gq * 32 + 16)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
                umma::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(which ? &v_full[bf] : &k_full[bf]);
            }
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if (lane == 0) umma::mbar_arrive(&empty[st]);
        }
    } else if (warp >= 4) {
        // ---- softmax: thread = key (S^T's row), columns [c0, c0 + NC) --------------------------
        const int wg = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane, c0 = NSTR == 2 ? 0 : wg * NC;
        const int own = NSTR == 2 ? wg : 0;  // the stream
        const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t t_own = t_o + t_lane + own * 3 * NB;
        Walk<NB> walk(a, pos0, pos1, b_at, f_at);
        Segment g;
        int it = 0;
        bool dead = false;
        while (!dead && walk.next(a, g)) {
            // Q rows: two fp8 numbers a channel
            {
                constexpr int LR = D / 8, RP = 256 / LR;  // lanes a row, rows a pass
                const int me = wg * 128 + r;
#pragma unroll 1
                for (int n = me / LR; n < NB; n += RP) {
                    const long long gi = static_cast<long long>(g.r) * NB + n;
                    const int tq = static_cast<int>(gi / a.grp), j = static_cast<int>(gi - static_cast<long long>(tq) * a.grp);
                    const bool live = tq < g.s.nq;
                    const int ch = (me % LR) * 8;
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
                        lo[i] = e4m3x2((f0 - b2.x) * 16.0f, (f1 - b2.y) * 16.0f);
                        if (sb == 255u) hi[i] = 0x7F7Fu, lo[i] = 0;  // an infinity or a NaN: the row is NaN
                    }
                    const uint32_t oh = swizzle8<D>(n * D + ch), ol = swizzle8<D>((NB + n) * D + ch);
                    *reinterpret_cast<uint2 *>(base + (q0 - sm) + oh) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                    *reinterpret_cast<uint2 *>(base + (q0 - sm) + ol) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                    if (me % LR == 0) {
                        s_qs[n] = sb == 255u ? 1.0f : scale_of(sb);
#pragma unroll
                        for (int z = 0; z < NSTR; ++z) s_nm[z][n] = 0.0f;
                        s_tok[n] = live ? tq : 0;
                        s_row[n] = live ? static_cast<long long>(g.s.q0 + tq) * a.Hq + g.h * a.grp + j : -1;
                    }
                }
            }
            umma::fence_proxy_async_smem();
            any_of(3, 256, false);
            if (lane == 0) umma::mbar_arrive(&q_full);

            uint64_t l2[NC / 2];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) l2[i] = 0;
            const int hist = g.s.kv - g.s.nq;  // keys before the new tokens
            const int clear = a.mode == QVG_MASK_NONE ? g.s.kv : min(g.s.kv, hist);
            int last = -1;  // this warpgroup's latest tile of the segment
            for (int t = g.t0; t < g.t1; ++t, ++it) {
                const int st = it % S, bf = it & 1;
                if (NSTR == 2 && bf != wg) continue;
                const bool first = last < 0;
                bool ok = wait(&s_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                if (it >= 2) ok = ok && wait(&pv_done[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
                ok = ok && wait(&full[st], (it / S) & 1, vfail, a.wait_ns);  // (the scales: written by the async proxy)
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
                // 4 bits: the operands are 2^6 times the values over the largest scale
                const float ka = scale_of(kb) * (BITS == 8 ? a.scale_log2 : a.scale_log2 * 0x1p-6f);
                const float sv = scale_of(vb) * (BITS == 8 ? 1.0f : 0x1p-6f);
                const float lsv = static_cast<float>(static_cast<int>(vb) - (BITS == 8 ? 127 : 133));
                const int key = t * kTile + r;
                const bool part = (t + 1) * kTile > clear;
                const uint64_t ka2 = pk2(ka, ka), lo2 = pk2(0.0625f, 0.0625f);
                float y[NC];
                // logits (base 2) less the reference; -inf where the row does not see the key
                auto logits = [&]() {
#pragma unroll
                    for (int c = 0; c < NC; c += 16) {
                        uint32_t v[16], u[16];
                        tmem_ld16x2(tmem + t_lane + bf * 2 * NB + c0 + c, tmem + t_lane + bf * 2 * NB + NB + c0 + c, v, u);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 qs = *reinterpret_cast<const float4 *>(&s_qs[c0 + c + 4 * i]);
                            const float4 nm = *reinterpret_cast<const float4 *>(&s_nm[own][c0 + c + 4 * i]);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int k = 4 * i + 2 * h;
                                const uint64_t x = mul2(fma2(pk2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])), lo2,
                                                             pk2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]))),
                                                        ka2);
                                up2(fma2(x, h ? pk2(qs.z, qs.w) : pk2(qs.x, qs.y), h ? pk2(nm.z, nm.w) : pk2(nm.x, nm.y)),
                                    y[c + k], y[c + k + 1]);
                            }
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
                if (any_of(wg + 1, 128, first || !ok || top + lsv > kTop)) {
                    // set or raise references: the column maxima of w over the tile
                    float v[NC];
                    const float lw = fmaxf(lsv, -64.0f);
#pragma unroll
                    for (int c = 0; c < NC; ++c) v[c] = y[c] + lw;
                    const float m = across_lanes<NC, true>(v);
                    if (lane < NC) s_red[wg][quad][c0 + lane] = m;
                    // (two streams: the last product into these sums is the one whose weights were here before)
                    if (!first && NSTR == 1) ok = ok && wait(&pv_done[bf ^ 1], ((it - 1) >> 1) & 1, vfail, a.wait_ns);
                    dead = any_of(wg + 1, 128, !ok);
                    if (dead) break;
                    umma::tc_fence_after();
                    if (r < NC) {
                        const int n = c0 + r;
                        const float mx = fmaxf(fmaxf(s_red[wg][0][n], s_red[wg][1][n]), fmaxf(s_red[wg][2][n], s_red[wg][3][n]));
                        const bool move = first ? mx > -INFINITY : mx > kTop;
                        const float d = move ? mx - kTarget : 0.0f;
                        s_nm[own][n] -= d;
                        s_dl[wg][n] = ex2(-d);
                    }
                    any_of(wg + 1, 128, false);
                    if (!first) {
#pragma unroll 1
                        for (int z = 0; z < 3; ++z)
#pragma unroll 1
                            for (int c = 0; c < NC; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(t_own + z * NB + c0 + c, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * s_dl[wg][c0 + c + i]);
                                umma::tmem_st16(t_own + z * NB + c0 + c, o);
                            }
                        umma::tmem_st_wait();
#pragma unroll
                        for (int i = 0; i < NC / 2; ++i)
                            l2[i] = mul2(l2[i], pk2(s_dl[wg][c0 + 2 * i], s_dl[wg][c0 + 2 * i + 1]));
                    }
                    logits();
                }
                last = it;
                umma::tc_fence_before();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&s_free[bf]);
                // 8 bits: V's rows meet weights of 0 where a row does not see them, but 0 times a code that is no
                // number would be one more NaN: slots past the end become 0, and so does such a code in the rows of
                // the new tokens, which are the ones that a mask can hide (a slot that was never written)
                if (BITS == 8 && part && (NSTR == 2 || wg == 0) && key >= hist) {
                    uint4 *vr = reinterpret_cast<uint4 *>(base + (st0 - sm) + st * C::kStage + C::kRaw + r * D);
#pragma unroll 1
                    for (int i = 0; i < D / 16; ++i) {
                        uint4 v = vr[i];
                        uint32_t *w = &v.x;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t no = ((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // bytes 0x7F, 0xFF
                            w[j] = key < g.s.kv ? w[j] & ~((no >> 7) * 0xFFu) : 0u;
                        }
                        vr[i] = v;
                    }
                }
                uint8_t *prow = base + (p0 - sm) + bf * C::kP + r * 128;
#pragma unroll
                for (int c = 0; c < NC; c += 16) {
                    uint32_t h[3][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int e = c + 4 * k + 2 * i;
                            const float pa = ex2(y[e]), pb = ex2(y[e + 1]);
                            l2[e / 2] = add2(l2[e / 2], pk2(pa, pb));
                            float wa = pa * sv, wb = pb * sv;
                            if (part) {  // an unseen key has weight 0 whatever its scale is
                                wa = y[e] == -INFINITY ? 0.0f : wa;
                                wb = y[e + 1] == -INFINITY ? 0.0f : wb;
                            }
                            w[i] = f16x2(wa, wb);
                        }
                        three_parts(w[0], w[1], h[0][k], h[1][k], h[2][k]);
                    }
#pragma unroll
                    for (int z = 0; z < 3; ++z) {
                        const int n = z * NB + c0 + c;
                        *reinterpret_cast<uint4 *>(prow + (n >> 7) * (kTile * 128) + ((((n >> 4) & 7) ^ (r & 7)) << 4)) =
                            make_uint4(h[z][0], h[z][1], h[z][2], h[z][3]);
                    }
                }
                umma::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&p_full[bf]);
            }
            // ---- the segment's sums (both warpgroups come here, also after a failure) ------------
            bool ok = !dead;
            if (ok && last >= 0) ok = wait(&pv_done[last & 1], (last >> 1) & 1, vfail, a.wait_ns);
            {
                float v[NC];
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) up2(l2[i], v[2 * i], v[2 * i + 1]);
                const float s = across_lanes<NC, false>(v);
                if (lane < NC) s_red[wg][quad][c0 + lane] = s;
            }
            dead = any_of(3, 256, !ok);
            if (dead) break;
            umma::tc_fence_after();
            const int slot = cta * 2 + (g.t0 > 0 ? 0 : 1);
            const bool whole = g.whole();
            if (wg == 0 && r < NB) {
                float l[NSTR], m = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int z = 0; z < NSTR; ++z) {
                    const int w = NSTR == 2 ? z : (r >= NC ? 1 : 0);
                    l[z] = (s_red[w][0][r] + s_red[w][1][r]) + (s_red[w][2][r] + s_red[w][3][r]);
                    if (l[z] != 0.0f) m = fmaxf(m, -s_nm[z][r]);
                }
                float wt[NSTR];
#pragma unroll
                for (int z = 0; z < NSTR; ++z) {
                    wt[z] = l[z] != 0.0f ? (NSTR == 2 ? ex2(-s_nm[z][r] - m) : 1.0f) : 0.0f;
                    if (wt[z] != 0.0f) sum = fmaf(l[z], wt[z], sum);
                }
                const float inv = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                for (int z = 0; z < NSTR; ++z) s_wt[z][r] = wt[z] * inv;
                const long long row = s_row[r];
                if (!whole) {
                    a.pm[static_cast<long long>(slot) * NB + r] = m;
                    a.pl[static_cast<long long>(slot) * NB + r] = sum;
                } else if (a.lse && row >= 0) {
                    a.lse[(row % a.Hq) * a.total_q + row / a.Hq] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
                }
            }
            any_of(3, 256, false);
#pragma unroll 1
            for (int c = wg * (NB / 2); c < (wg + 1) * (NB / 2); c += 8) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = 0.0f;
#pragma unroll
                for (int z = 0; z < NSTR; ++z) {
                    uint32_t x[3][8];
                    tmem_ld8x3(t_o + t_lane + z * 3 * NB + c, NB, x[0], x[1], x[2]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float w = s_wt[z][c + i];
                        const float f = fmaf(__uint_as_float(x[2][i]), 0x1p-6f, fmaf(__uint_as_float(x[1][i]), 0x1p-3f, __uint_as_float(x[0][i])));
                        if (w != 0.0f) o[i] = fmaf(f, w, o[i]);  // (a stream without a tile holds anything)
                    }
                }
                if (r < D) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int n = c + i;
                        const long long row = s_row[n];
                        if (row < 0) continue;
                        if (!whole)
                            a.po[(static_cast<long long>(slot) * NB + n) * D + r] = o[i];
                        else if (a.out32)
                            a.out32[row * D + r] = o[i];
                        else
                            a.out16[row * D + r] = f32_to_bf16(o[i]);
                    }
                }
            }
            umma::tc_fence_before();
            any_of(3, 256, false);  // everything of this segment has been read
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
    if (warp == 3) {
        umma::tc_fence_after();
        umma::tmem_dealloc(tmem, C::kTmem);
    }
}

}  // namespace pa
}  // namespace qvg
