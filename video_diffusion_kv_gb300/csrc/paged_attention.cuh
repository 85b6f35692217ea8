// paged_attention.cuh -- attention of a few new tokens (one, a drafted tree, a
// short chunk) over a paged fp8 / fp4 cache: the kernel.  Launch, merge and
// entry points: paged_attention.cu.
//
// One unit of work is (sequence b, KV head h, block r of NB query rows); a
// query row is a (new token, query head of the group) pair, so the group's
// heads share each key and value that is read.  A unit walks its sequence in
// tiles of 128 keys.  All units' tiles form one line, which is cut into equal
// parts, one per CTA: ragged batches and single long sequences fill the GPU
// alike.  A unit cut by a border leaves fp32 partial sums that k_paged_merge
// joins.
//
// Two CTAs share an SM (8 warps, half of the shared and tensor memory each), so
// that one's latencies -- a tile is a chain of S, softmax and PV, a unit begins
// and ends with its own -- pass while the other works.  (One CTA with two
// softmax groups: 305 us for the batch below, where two CTAs took 265.)
//
// The product runs transposed, keys on the tensor core's 128 rows, and takes
// the cache's fp8 codes as they lie there (4-bit codes become fp8 first):
//   S^T [keys x rows] = K Q^T        A = K's codes
//   O^T [d x rows]   += V^T P^T      A = V's codes, read across (MN-major)
// so its cost follows the number of query rows (N), not a padded 128, and K
// and V are touched once by the copy and once by the tensor core.  The other
// operand is made of several fp8 numbers side by side along N, each with its
// own accumulator columns; a product with N <= 64 takes the tensor core the
// same 45 to 48 clocks whatever N is, so the extra columns are free there:
//   - Q as two: hi + lo / 16 in e4m3 (4 significant bits each, a bf16 number
//     has 8: exact down to 2^-13 of the row's largest);
//   - P as three: h1 + h2 + h3 in e5m2, which is the upper byte of an fp16
//     number: the first two cut off, the last rounded: at most 2^-9 of the
//     weight off (and 2^-11 by fp16), and nearly fp16's range, which e4m3 lacks.
// A key's scale is one number per row of S^T, i.e. per softmax thread; V's
// scale goes into the weight: w = p sv.
// Softmax: a thread owns one key and 16 or 32 columns.  The weights of a column
// are taken relative to a reference that is set from the first tile (its
// largest w becomes 2^kTarget) and raised when a w would pass 2^kTop, so the
// sums l and O are rescaled rarely, and a tile needs one vote, no maximum
// across threads.  A w of 2^-25 of the reference's largest still counts; l
// takes p in fp32.  The loop's code is kept small (one instance of each part):
// with copies for the rare cases it outgrew the instruction cache and took
// 1.5 times as long.
//
// Bound: HBM for single tokens.  One token over 449,280 (8 KV heads, d = 128,
// 4 query heads each, 8 bits; 0.93 GB): 158 us, 5.85 TB/s, 86 % of a plain copy's
// rate.  48 tokens over 700 to 24,000 each (8 query heads a KV head, pages of
// 16): 231 us, 5.3 TB/s; pages of 16 mean 8 copies a tile for each of K and V,
// and every sequence's ends leave a part tile.
// 4 bits are bound by the conversion into fp8 (four warps, about 500
// instructions a thread and tile): 24 trees of 5 to 13 tokens over 4,000 to
// 16,000, 16 KV heads: 269 us, 1.95 TB/s.
#pragma once

#include <cuda.h>

#include "paged.cuh"
#include "umma.cuh"

namespace qvg {
namespace pa {

constexpr int kTile = 128;
constexpr float kTarget = 8.0f, kTop = 15.0f;
// V's scale enters the reference, so that w = p sv spans its type's range; from 2^kLeastV down only p does, whose sums
// (up to 2^(kTop - kLeastV) a key) stay in fp32.
constexpr float kLeastV = -90.0f;
constexpr long long kMostKeys = (1ll << 31) - 4096;  // of a sequence: key numbers and what a tile adds to them stay in 32 bits
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
    const long long most = min(a.table_stride << a.page_log2, kMostKeys);
    int kv = a.kv_len[b];
    bad = bad || kv < 0 || kv > most;
    kv = static_cast<int>(max(0ll, min(static_cast<long long>(kv), most)));
    s.q0 = q0;
    s.nq = nq;
    s.kv = kv;
    s.nt = max(1, static_cast<int>((static_cast<long long>(kv) + kTile - 1) / kTile));
    s.rb = static_cast<int>((static_cast<long long>(nq) * a.grp + NB - 1) / NB);
    bad = bad || s.tiles(a.H) > 0xFFFFFFFFll;
    if (report && bad) raise_error(a.err, QVG_ERR_INVALID_ARG);
    return s;
}

// A stretch [t0, t1) of one unit's tiles inside a CTA's part.  One warp of the
// CTA makes them and hands them to the others through a ring in shared memory
// (each role working them out for itself cost code that the instruction cache
// then missed, 75 clocks an instruction the first time).
struct __align__(16) Segment {
    int b, h, r, t0, t1;  // t1 = 0: no more
    int q0, nq, kv, nt;
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == nt; }
};
constexpr int kRing = 8;  // segments ahead; a copy can run that far ahead in one-tile units
constexpr int kChunks = 256;

// The CTA's part of the line, made by one whole warp.  (Its walks end with the
// batch even if the lengths change meanwhile.)
template <int NB>
struct Line {
    long long pos, end, first, per;  // first: where sequence b begins
    int b;
    int4 cut;  // the unit that begins here and goes on, and the last of the CTAs that share it
    Seq s;

    // chunk [kChunks]: room in shared memory
    __device__ __forceinline__ Line(const Args &a, long long *chunk) {
        const int lane = threadIdx.x & 31, cta = blockIdx.x;
        // tiles of all sequences, by chunks of `span` sequences
        const int span = ((a.B + kChunks - 1) / kChunks + 31) & ~31;
        long long total = 0;
        for (int k = 0, b0 = 0; b0 < a.B; ++k, b0 += span) {
            long long mine = 0;
            for (int i = b0 + lane; i < min(a.B, b0 + span); i += 32) mine += seq_of<NB>(a, i, cta == 0).tiles(a.H);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
            if (lane == 0) chunk[k] = mine;
            total += mine;
        }
        __syncwarp();
        per = max(1ll, (total + gridDim.x - 1) / gridDim.x);
        pos = min(total, cta * per);
        end = min(total, pos + per);
        first = 0;
        b = 0;
        if (pos < end) {  // the sequence that holds `pos`: its chunk, then by a scan over 32 at a time
            int k = 0;
            while (pos >= first + chunk[k]) first += chunk[k++];
            for (b = k * span; b < a.B; b += 32) {
                const long long w = b + lane < a.B ? seq_of<NB>(a, b + lane, false).tiles(a.H) : 0;
                long long x = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                    if (lane >= o) x += y;
                }
                const uint32_t hit = __ballot_sync(0xFFFFFFFFu, pos < first + x);
                const int l = hit ? __ffs(hit) - 1 : 31;
                const long long upto = __shfl_sync(0xFFFFFFFFu, x, l), own = __shfl_sync(0xFFFFFFFFu, w, l);
                first += hit ? upto - own : upto;
                if (hit) {
                    b += l;
                    break;
                }
            }
        }
        cut = make_int4(-1, 0, 0, 0);
        if (b >= a.B) pos = end;
        s = seq_of<NB>(a, min(b, a.B - 1), false);
    }

    // t1 = 0: no more.
    __device__ __forceinline__ void next(const Args &a, Segment &g) {
        g.t1 = 0;
        if (pos >= end) return;
        while (b < a.B && pos >= first + s.tiles(a.H)) {
            first += s.tiles(a.H);
            s = seq_of<NB>(a, min(++b, a.B - 1), false);
        }
        if (b >= a.B) return;
        const uint32_t rel = static_cast<uint32_t>(pos - first), u = rel / static_cast<uint32_t>(s.nt);
        g.b = b;
        g.h = static_cast<int>(u / static_cast<uint32_t>(s.rb));
        g.r = static_cast<int>(u % static_cast<uint32_t>(s.rb));
        g.t0 = static_cast<int>(rel - u * s.nt);
        g.t1 = static_cast<int>(min(static_cast<long long>(s.nt), g.t0 + (end - pos)));
        g.q0 = s.q0;
        g.nq = s.nq;
        g.kv = s.kv;
        g.nt = s.nt;
        if (g.t0 == 0 && g.t1 < s.nt) cut = make_int4(b, g.h, g.r, static_cast<int>((pos + s.nt - 1) / per));
        pos += g.t1 - g.t0;
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

// Bounded wait that also ends when another role has failed.  (Out of line but
// for the first try: a tile's loop has many waits, and its code has to stay
// small.)
__device__ __forceinline__ bool try_wait_long(uint64_t *bar, uint32_t parity) {  // suspended for up to 20 us
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(umma::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *fail, uint64_t limit_ns) {
    for (int i = 0; i < 4; ++i)
        if (try_wait_long(bar, parity)) return true;
    const uint64_t t0 = umma::globaltimer_ns();
    for (;;) {
        if (try_wait_long(bar, parity)) return true;
        if (*fail) return false;
        if (umma::globaltimer_ns() - t0 > limit_ns) {
            *fail = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *fail, uint64_t limit_ns) {
    return umma::mbar_try_wait(bar, parity) || wait_on(bar, parity, fail, limit_ns);
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

// Lane i receives 16 consecutive columns of TMEM lane (base + i) from t and
// from t + step.
__device__ __forceinline__ void tmem_ld_pair(uint32_t t, uint32_t step, uint32_t (&r)[16], uint32_t (&q)[16]) {
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
        : "r"(t), "r"(t + step)
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

// Four weights (two fp16 pairs, not negative) -> their three e5m2 parts, four
// bytes each.  x less its upper byte is exact; adding half a step to the bits
// of the last rest rounds its upper byte.
__device__ __forceinline__ void three_parts(uint32_t a, uint32_t b, uint32_t &h1, uint32_t &h2, uint32_t &h3) {
    auto rest = [](uint32_t x) {
        const uint32_t cut = x & 0xFF00FF00u;
        const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&cut));
        return *reinterpret_cast<const uint32_t *>(&d);
    };
    h1 = __byte_perm(a, b, 0x7531);
    a = rest(a);
    b = rest(b);
    h2 = __byte_perm(a, b, 0x7531);
    a = rest(a) + 0x00800080u;
    b = rest(b) + 0x00800080u;
    h3 = __byte_perm(a, b, 0x7531);
}

// Position in a ring of N buffers and the parity of its current use.
template <int N>
struct Ring {
    int i = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            parity ^= 1u;
        }
    }
};

// Sum or maximum of each of NC columns over the warpgroup's 128 rows, in part:
// scratch [128][NC] has been filled; thread r takes column r % NC of every
// (128 / NC)-th row from r / NC on, into red[r / NC][r % NC].
template <int NC, bool MAX>
__device__ __forceinline__ void reduce_columns(const float *scratch, float (*red)[NC], int r) {
    float x = MAX ? -INFINITY : 0.0f;
#pragma unroll 4
    for (int i = r / NC; i < 128; i += 128 / NC) {
        const float v = scratch[i * NC + r % NC];
        x = MAX ? fmaxf(x, v) : x + v;
    }
    red[r / NC][r % NC] = x;
}

// ---- shared memory ---------------------------------------------------------------

template <int D, int BITS, int NB>
struct Cfg {
    static constexpr int NC = NB;              // columns of a softmax thread
    static constexpr int G = BITS == 8 ? 1 : D / 32;
    static constexpr int kRow = D * BITS / 8;  // bytes of a row of codes
    static constexpr int kRaw = kTile * kRow;  // a tile's codes (K or V)
    static constexpr int kScales = 256 * G;    // and K's and V's scales
    static constexpr int kOp = BITS == 4 ? kTile * D : 0;  // K or V as e4m3 (4 bits)
    static constexpr int kP = 16384;           // weights: 128 rows of 3 NB (at most 128) bytes
    static constexpr int kQ = 2 * NB * D;      // Q: hi rows, lo rows
    static constexpr int kFixed = 2 * kOp + kP + kQ;
    // K's and V's copies in flight: a K buffer is free once S is there, a V buffer once O has it
    static constexpr int kRoom = 106 * 1024 - kFixed;
    static constexpr int kSlots = kRoom / (kRaw + kScales / 2);
    static constexpr int kSK = kSlots / 2 > 4 ? 4 : kSlots / 2, kSV = kSlots - kSK > 5 ? 5 : kSlots - kSK;
    static constexpr int kSmem = kFixed + (kSK + kSV) * kRaw + kSV * kScales + 1024;
    static constexpr int kConv = BITS == 4 ? 4 : 0;  // converter warps, half for K and half for V
    static constexpr int kWarps = 8 + kConv;   // loads, S, PV, segments and Q; softmax 4 - 7; converters
    static constexpr int kTmemUsed = 2 * 2 * NB + 3 * NB;
    static constexpr int kTmem = kTmemUsed <= 128 ? 128 : 256;
    static_assert(kSK >= 2 && kSV >= 2, "shared memory");
};

// e2m1 magnitudes times 2^(6 - k) as e4m3 bytes, for a group whose scale is
// 2^-k of the row's largest (k <= 14; beyond, the values are under 2^-9 and
// count as 0), eight bytes: the operands of a 4-bit cache.
__device__ __forceinline__ uint2 levels_of(int k) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        const float lv = i < 2 ? 0.5f : i < 4 ? 0.5f * i : i < 6 ? 1.0f * (i - 2) : 2.0f * (i - 4);
        const float x = k <= 14 ? lv * __uint_as_float(static_cast<uint32_t>(127 + 6 - k) << 23) : 0.0f;
        w[i >> 2] |= (e4m3x2(x, 0.0f) & 0xFFu) << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}

// ---- what a softmax warp does rarely, out of its loop's code -----------------------

// Logits of 16 columns, base 2, less the reference.
__device__ __forceinline__ void logits16(uint32_t t_hi, uint32_t t_lo, const float *qs, const float *nm, float ka, float (&y)[16]) {
    uint32_t v[16], u[16];
    tmem_ld16(t_hi, v);
    tmem_ld16(t_lo, u);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        y[i] = fmaf(fmaf(__uint_as_float(u[i]), 0.0625f, __uint_as_float(v[i])) * ka, qs[i], nm[i]);
}

// The rows (columns of S) that do not see this thread's key, as bits.
//   row0: the first column's row; tok: the rows' new tokens; mw: room for the
// tile's mask words; j: the key's number among the new tokens; w0: the first
// mask word that the tile needs.
template <int NC>
__device__ __noinline__ uint32_t hidden_rows(const Args &a, int row0, const int *tok, uint32_t (*mw)[5], int r, int q0, bool past, int j,
                                             int w0) {
    if (a.mode == QVG_MASK_TREE) {
        for (int i = r; i < NC * 5; i += 128) {
            const int c = i / 5, k = w0 + i % 5;
            mw[c][i % 5] = k < a.words ? a.mask[static_cast<long long>(q0 + tok[c]) * a.words + k] : 0u;
        }
        any_of(1, 128, false);
    }
    if (past) return 0xFFFFFFFFu;
    if (j < 0 || a.mode == QVG_MASK_NONE) return 0u;
    if (a.mode == QVG_MASK_CAUSAL) {  // row i is token i / grp: it sees token j from row j grp on
        const long long n = static_cast<long long>(j) * a.grp - row0;
        return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
    }
    uint32_t hidden = 0;
#pragma unroll 4
    for (int c = 0; c < NC; ++c) hidden |= (~(mw[c][(j >> 5) - w0] >> (j & 31)) & 1u) << c;
    return hidden;
}

// V's rows meet weights of 0 where a row does not see them, but 0 times a code
// that is no number would be one more NaN: slots past the end become 0, and so
// does such a code in the rows of the new tokens, which are the ones that a
// mask can hide (a slot that was never written).
// Thread r of 128 takes every 128th 16 bytes from row `from` on; rows from
// `past` on are past the end.
template <int D>
__device__ __noinline__ void clean_values(uint8_t *v, int from, int past, int r) {
#pragma unroll 1
    for (int i = from * (D / 16) + r; i < kTile * (D / 16); i += 128) {
        uint4 x = reinterpret_cast<uint4 *>(v)[i];
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t no = ((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // bytes 0x7F, 0xFF
            w[j] = i >= past * (D / 16) ? 0u : w[j] & ~((no >> 7) * 0xFFu);
        }
        reinterpret_cast<uint4 *>(v)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Set (first) or raise the references of this warpgroup's columns after the
// tile's logits: from the columns' largest w over the tile.  O's sums follow;
// dl gets the factors for l.  A reference follows V's scale and may rise by
// more than 2^126, which is no factor, while l, up to 2^120, still counts: a
// rise of most .. 2 most is left at `most`, to be done again.  (A larger one
// leaves nothing of l.)  0: some thread has given up; 1: done; 2: once more.
template <int NC, int NB>
__device__ __noinline__ int set_references(uint32_t t_s, uint32_t t_own, const float *qs, float *nm, float *scratch, float (*red)[NC],
                                            float *dl, int r, float ka, float lsv, const uint32_t hidden, bool first, bool ok, float most) {
    const float lw = fmaxf(lsv, kLeastV);
#pragma unroll 1
    for (int c = 0; c < NC; c += 16) {
        float y[16];
        logits16(t_s + c, t_s + NB + c, qs + c, nm + c, ka, y);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = (hidden >> (c + i)) & 1u ? -INFINITY : y[i] + lw;
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4 *>(scratch + r * NC + c + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
    }
    if (any_of(1, 128, !ok)) return 0;
    bool more = false;
    reduce_columns<NC, true>(scratch, red, r);
    any_of(1, 128, false);
    umma::tc_fence_after();
    if (r < NC) {
        float mx = -INFINITY;
        for (int i = 0; i < 128 / NC; ++i) mx = fmaxf(mx, red[i][r]);
        const bool move = first ? mx > -INFINITY : mx > kTop;
        float d = move ? mx - kTarget : 0.0f;
        more = !first && d > most && d <= 2.0f * most;
        d = more ? most : d;
        nm[r] -= d;
        dl[r] = first ? 1.0f : ex2(-d);  // (a first reference may lie far below 0, and l is 0 yet)
    }
    more = any_of(1, 128, more);
    if (!first) {
#pragma unroll 1
        for (int z = 0; z < 3 * (NC / 16); ++z) {
            const int c = (z / 3) * 16;
            uint32_t o[16];
            tmem_ld16(t_own + (z % 3) * NB + c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * dl[c + i]);
            umma::tmem_st16(t_own + (z % 3) * NB + c, o);
        }
        umma::tmem_st_wait();
    }
    return more ? 2 : 1;
}

// A unit's Q rows as pairs of fp8 numbers into dst, with their scales, tokens
// and out rows; by one warp.
template <int D, int NB>
__device__ __noinline__ void make_q(const Args &a, const Segment &g, uint8_t *dst, float *qs, int *tok, long long *rows) {
    constexpr int LR = D / 8, step = 32 / LR;  // lanes a row, rows a pass
    const int lane = threadIdx.x & 31, ch = (lane % LR) * 8;
    auto fetch = [&](int n, int &tq, int &j) {
        const uint32_t gi = static_cast<uint32_t>(g.r) * NB + n;  // (the call has made sure that it fits)
        tq = static_cast<int>(gi / static_cast<uint32_t>(a.grp));
        j = static_cast<int>(gi) - tq * a.grp;
        if (n >= NB || tq >= g.nq) return make_uint4(0, 0, 0, 0);
        return *reinterpret_cast<const uint4 *>(a.q + (g.q0 + tq) * a.q_stride + static_cast<long long>(g.h * a.grp + j) * D + ch);
    };
    int n = lane / LR, tq, j, tq1, j1, tq2, j2;
    uint4 v = fetch(n, tq, j), v1 = fetch(n + step, tq1, j1), v2;
#pragma unroll 1
    for (; n < NB; n += step, v = v1, tq = tq1, j = j1, v1 = v2, tq1 = tq2, j1 = j2) {
        v2 = fetch(n + 2 * step, tq2, j2);  // two passes ahead
        const bool live = tq < g.nq;
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
        *reinterpret_cast<uint2 *>(dst + oh) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2 *>(dst + ol) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        if (lane % LR == 0) {
            qs[n] = sb == 255u ? 1.0f : scale_of(sb);
            tok[n] = live ? tq : 0;
            rows[n] = live ? static_cast<long long>(g.q0 + tq) * a.Hq + g.h * a.grp + j : -1;
        }
    }
    umma::fence_proxy_async_smem();
    __syncwarp();
}

template <int D, int BITS, int NB>
__global__ void __launch_bounds__(Cfg<D, BITS, NB>::kWarps * 32, 2)
    k_paged_attention(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ Args a) {
    using C = Cfg<D, BITS, NB>;
    constexpr int SK = C::kSK, SV = C::kSV, NC = C::NC;
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t k_full[SK], k_empty[SK], v_full[SV], v_empty[SV];  // codes (and scales, with V's) as loaded
    __shared__ uint64_t ko_full, ko_done, vo_full;                         // 4 bits: operands made of them
    __shared__ uint64_t s_full[2], s_free[2], p_full, pv_done, q_full[2], q_free, m_free[2], drain, never;
    __shared__ uint64_t seg_full[kRing], seg_free[kRing];
    __shared__ Segment s_seg[kRing];
    __shared__ long long s_chunk[kChunks];
    __shared__ uint32_t tmem_base;
    __shared__ int fail, s_issued[2];  // tiles of K and of V whose copies have been issued
    __shared__ __align__(16) float s_qs[2][NB], s_nm[NB];  // per column: Q's scale, minus the reference
    __shared__ __align__(16) float s_red[128 / NC][NC], s_dl[NC];
    __shared__ int s_tok[2][NB];        // new token of each row
    __shared__ long long s_row[2][NB];  // out row, or -1
    __shared__ uint32_t s_mw[NC][5];    // the mask words of a tile's new tokens
    __shared__ uint2 s_lv[BITS == 4 ? 16 : 1];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    uint8_t *base = dyn + ((1024u - (umma::smem_u32(dyn) & 1023u)) & 1023u);
    const uint32_t sm = umma::smem_u32(base);
    const uint32_t p0 = sm, k80 = p0 + C::kP, v80 = k80 + C::kOp, q0 = v80 + C::kOp, kr0 = q0 + C::kQ, vr0 = kr0 + SK * C::kRaw,
                   sc0 = vr0 + SV * C::kRaw;
    if (tid == 0) {
        fail = 0;
        s_issued[0] = s_issued[1] = 0;
        for (int i = 0; i < kRing; ++i) {
            umma::mbar_init(&seg_full[i], 1);
            umma::mbar_init(&seg_free[i], C::kWarps - 1);  // every other warp
        }
        for (int i = 0; i < SK; ++i) {
            umma::mbar_init(&k_full[i], 1);
            umma::mbar_init(&k_empty[i], BITS == 8 ? 1 : C::kConv / 2);  // S done, or the converters
        }
        for (int i = 0; i < SV; ++i) {
            umma::mbar_init(&v_full[i], 33);  // the codes; each lane's part of the scales
            umma::mbar_init(&v_empty[i], (BITS == 8 ? 1 : C::kConv) + 4);  // O done, or the converters; softmax warps
        }
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(&s_full[i], 1);
            umma::mbar_init(&s_free[i], 4);
            umma::mbar_init(&m_free[i], 4);
            umma::mbar_init(&q_full[i], 1);
        }
        umma::mbar_init(&ko_full, BITS == 8 ? 1 : C::kConv / 2);
        umma::mbar_init(&ko_done, 1);
        umma::mbar_init(&vo_full, BITS == 8 ? 1 : C::kConv / 2);
        umma::mbar_init(&p_full, 4);
        umma::mbar_init(&pv_done, 1);
        umma::mbar_init(&q_free, 1);
        umma::mbar_init(&drain, 2);
        umma::mbar_init(&never, 1);
        umma::fence_barrier_init();
    }
    if (warp == 2) {
        umma::tmem_alloc(&tmem_base, C::kTmem);
        umma::tmem_relinquish();
    }
    if (tid < NB) s_nm[tid] = 0.0f;
    if (BITS == 4 && tid < 16) s_lv[tid] = levels_of(tid);
    __syncthreads();
    umma::tc_fence_after();
    const uint32_t tmem = tmem_base;
    const uint32_t t_o = tmem + 4 * NB;  // S: two buffers of 2 NB columns; O: 3 NB
    volatile int *vfail = &fail;
    // The next segment for this warp (n of them so far); false: no more, or gave up.
    auto next_segment = [&](Segment &g, int n) {
        const int i = n & (kRing - 1);
        const bool ok = wait(&seg_full[i], (n / kRing) & 1, vfail, a.wait_ns);
        g = s_seg[i];
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&seg_free[i]);
        return __all_sync(0xFFFFFFFFu, ok) && g.t1 > 0;
    };

    if (warp >= 4 && warp < 8) {
        // ---- softmax: thread = key (S^T's row), all columns -------------------------------------
        const int quad = warp & 3, r = quad * 32 + lane;
        const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
        uint8_t *p_base = base + (p0 - sm), *prow = p_base + r * 128;
        Segment g;
        Ring<SV> rv;
        int it = 0, n_seg = 0;
        bool dead = false;
        while (!dead) {
            // The four warps vote: the segment may be handed out while a wait runs out, after some have given up, and
            // the barriers below have no bound.  Nor does any of them go on without the unit's rows (s_tok leads into
            // the mask).
            const int qb = n_seg & 1;
            const bool got = next_segment(g, n_seg) && wait(&q_full[qb], (n_seg >> 1) & 1, vfail, a.wait_ns);
            if (any_of(1, 128, !got)) break;
            ++n_seg;
            uint64_t l2[NC / 2];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) l2[i] = 0;
            const int hist = g.kv - g.nq;  // keys before the new tokens
            const int clear = a.mode == QVG_MASK_NONE ? g.kv : min(g.kv, hist);
            bool late = false;  // this thread gave up a wait: all agree on that at the next barrier
            for (int t = g.t0; t < g.t1; ++t, ++it, rv.next()) {
                const int bf = it & 1;
                const bool first = t == g.t0;
                bool ok = !late && wait(&v_full[rv.i], rv.parity, vfail, a.wait_ns);  // (the scales)
                const uint8_t *sc = base + (sc0 - sm) + rv.i * C::kScales;
                uint32_t kb = 0, vb = 0;
                if constexpr (BITS == 8) {
                    kb = sc[r];
                    vb = sc[128 + r];
                } else {
#pragma unroll
                    for (int j = 0; j < C::G; ++j) {
                        kb = max(kb, static_cast<uint32_t>(sc[r * C::G + j]));
                        vb = max(vb, static_cast<uint32_t>(sc[128 * C::G + r * C::G + j]));
                    }
                }
                const int key = t * kTile + r;
                if (key >= g.kv) kb = vb = 127u;  // (whatever is there)
                // 4 bits: the operands are 2^6 times the values over the largest scale
                const float ka = scale_of(kb) * (BITS == 8 ? a.scale_log2 : a.scale_log2 * 0x1p-6f);
                const bool v_nan = vb == 255u;  // weighed as 1, and made a NaN below
                const float sv = v_nan ? 1.0f : scale_of(vb) * (BITS == 8 ? 1.0f : 0x1p-6f);
                const float lsv = v_nan ? 0.0f : static_cast<float>(static_cast<int>(vb) - (BITS == 8 ? 127 : 133));
                const bool part = (t + 1) * kTile > clear;
                const uint64_t ka2 = pk2(ka, ka), lo2 = pk2(0.0625f, 0.0625f);
                uint32_t hidden = 0;  // columns that do not see this key, where that can be
                if (part)
                    hidden = hidden_rows<NC>(a, g.r * NB, s_tok[qb], s_mw, r, g.q0, key >= g.kv, key - hist,
                                             max(0, t * kTile - hist) >> 5);
                ok = ok && wait(&s_full[bf], (it >> 1) & 1, vfail, a.wait_ns);
                umma::tc_fence_after();
                const uint32_t t_s = tmem + t_lane + bf * 2 * NB;
                float y[NC];  // logits (base 2) less the reference
                for (int set = 0;;) {  // (the answer of set_references)
#pragma unroll
                    for (int c = 0; c < NC; c += 16) {
                        uint32_t v[16], u[16];  // against Q's hi and lo rows
                        tmem_ld_pair(t_s + c, NB, v, u);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 qs = *reinterpret_cast<const float4 *>(&s_qs[qb][c + 4 * i]);
                            const float4 nm = *reinterpret_cast<const float4 *>(&s_nm[c + 4 * i]);
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
#pragma unroll
                        for (int c = 0; c < NC; ++c) y[c] = (hidden >> c) & 1u ? -INFINITY : y[c];
                    }
                    if (set == 1) break;
                    float top4[4] = {y[0], y[1], y[2], y[3]};
#pragma unroll
                    for (int c = 4; c < NC; ++c) top4[c & 3] = fmaxf(top4[c & 3], y[c]);
                    const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                    if (!any_of(1, 128, first || !ok || top + fmaxf(lsv, kLeastV) > kTop)) break;
                    if (!first) ok = ok && wait(&pv_done, (it - 1) & 1, vfail, a.wait_ns);  // O's latest
                    set = set_references<NC, NB>(t_s, t_o + t_lane, s_qs[qb], s_nm, reinterpret_cast<float *>(p_base), s_red, s_dl, r,
                                                 ka, lsv, hidden, first, ok, set == 0 ? 120.0f : INFINITY);
                    dead = set == 0;
                    if (dead) break;
#pragma unroll
                    for (int i = 0; i < NC / 2; ++i) l2[i] = mul2(l2[i], pk2(s_dl[2 * i], s_dl[2 * i + 1]));
                }
                if (dead) break;
                umma::tc_fence_before();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&s_free[bf]);
                if (BITS == 8 && part)
                    clean_values<D>(base + (vr0 - sm) + rv.i * C::kRaw, max(0, min(hist, g.kv) - t * kTile), g.kv - t * kTile, r);
                auto place = [&](int z, int c) {  // part z of columns c .. c + 15 in this thread's row of weights
                    return prow + ((((z * NB + c) >> 4) ^ (r & 7)) << 4);
                };
                const uint64_t sv2 = pk2(sv, sv);
#pragma unroll
                for (int c = 0; c < NC; c += 16) {
                    uint32_t h[3][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int e = c + 4 * k + 2 * i;
                            const uint64_t p = pk2(ex2(y[e]), ex2(y[e + 1]));
                            l2[e / 2] = add2(l2[e / 2], p);
                            float wa, wb;
                            up2(mul2(p, sv2), wa, wb);
                            w[i] = f16x2(wa, wb);
                        }
                        three_parts(w[0], w[1], h[0][k], h[1][k], h[2][k]);
                    }
                    // (the last tile's weights have been used up by now)
                    if (c == 0 && it > 0 && !wait(&pv_done, (it - 1) & 1, vfail, a.wait_ns)) late = true;
#pragma unroll
                    for (int z = 0; z < 3; ++z) *reinterpret_cast<uint4 *>(place(z, c)) = make_uint4(h[z][0], h[z][1], h[z][2], h[z][3]);
                }
                if (v_nan) {  // a NaN for the rows that see this key, and only for them
#pragma unroll 1
                    for (int c = 0; c < NC; ++c)
                        if (!((hidden >> c) & 1u)) place(0, c & 16)[c & 15] = 0x7F;
                }
                umma::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    umma::mbar_arrive(&p_full);
                    umma::mbar_arrive(&v_empty[rv.i]);
                }
            }
            if (dead) break;
            // ---- the segment's sums; the weights' buffer is free: l's column sums go through it ----
            bool ok = !late && wait(&pv_done, (it - 1) & 1, vfail, a.wait_ns);
            float *scratch = reinterpret_cast<float *>(p_base);
            if (ok) {
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) *reinterpret_cast<uint64_t *>(scratch + r * NC + 2 * i) = l2[i];
            }
            dead = any_of(1, 128, !ok);
            if (dead) break;
            reduce_columns<NC, false>(scratch, s_red, r);
            any_of(1, 128, false);
            umma::tc_fence_after();
            const int slot = cta * 2 + (g.t0 > 0 ? 0 : 1);
            const bool whole = g.whole();
            if (r < NB) {
                float l = 0.0f;
                for (int i = 0; i < 128 / NC; ++i) l += s_red[i][r];
                const float m = -s_nm[r];
                s_dl[r] = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
                s_nm[r] = 0.0f;  // for the next unit
                const long long row = s_row[qb][r];
                if (!whole) {
                    a.pm[static_cast<long long>(slot) * NB + r] = m;
                    a.pl[static_cast<long long>(slot) * NB + r] = l;
                } else if (a.lse && row >= 0) {
                    a.lse[(row % a.Hq) * a.total_q + row / a.Hq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                }
            }
            any_of(1, 128, false);
#pragma unroll 1
            for (int c = 0; c < NB; c += 8) {
                uint32_t x[3][8];
                tmem_ld8x3(t_o + t_lane + c, NB, x[0], x[1], x[2]);
                if (r >= D) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const long long row = s_row[qb][c + i];
                    if (row < 0) continue;
                    const float o = ((__uint_as_float(x[2][i]) + __uint_as_float(x[1][i])) + __uint_as_float(x[0][i])) * s_dl[c + i];
                    if (!whole)
                        a.po[(static_cast<long long>(slot) * NB + c + i) * D + r] = o;
                    else if (a.out32)
                        a.out32[row * D + r] = o;
                    else
                        a.out16[row * D + r] = f32_to_bf16(o);
                }
            }
            umma::tc_fence_before();
            any_of(1, 128, false);  // everything of this segment has been read
            if (lane == 0) umma::mbar_arrive(&m_free[qb]);
        }
    } else if (warp == 0) {
        // ---- loads: lane i fetches a tile's i-th piece (a page, or 128 tokens of one); the scales, 16 bytes at a
        // time, go by plain asynchronous copies of all lanes (issuing a bulk copy takes a warp about 90 clocks) ----
        const int pr_log2 = min(a.page_log2, 7), pr = 1 << pr_log2;
        Segment g;
        Ring<SK> rk;
        Ring<SV> rv;
        int it = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            // the block table, 32 entries at a time, the next 32 on their way while these are used
            const int32_t *row = a.table + g.b * a.table_stride;
            const int pages = (g.kv + (1 << a.page_log2) - 1) >> a.page_log2;
            int have = (g.t0 * kTile) >> a.page_log2 & ~31;  // entry of lane 0's `now`
            auto entries = [&](int e) { return e + lane < pages ? row[e + lane] : 0; };
            int now = entries(have), then = entries(have + 32);
            for (int t = g.t0; t < g.t1; ++t, ++it, rk.next(), rv.next()) {
                if ((t * kTile) >> a.page_log2 >= have + 32) {  // (a tile's entries never straddle 32)
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
                        ok = ok && wait(which ? &v_empty[rv.i] : &k_empty[rk.i], (which ? rv.parity : rk.parity) ^ 1u, vfail, a.wait_ns);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (lane == 0) umma::mbar_arrive_expect_tx(full, bytes);
                    __syncwarp();
                    if (good) {
                        if constexpr (BITS == 8)
                            tma_load_4d(dst, which ? &vmap : &kmap, off, g.h, page, full);
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
                    const int c = v ? i - 8 * C::G : i, first = c * (16 / C::G);  // part c begins with this key's
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
    } else if (warp == 1) {
        // ---- S = K Q^T -------------------------------------------------------------------
        constexpr uint32_t id = idesc_f8(128, 2 * NB, 0);
        const uint64_t dq = desc_rows8<D>(q0);
        Segment g;
        Ring<SK> rk;
        int it = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            if (lane == 0) {
                ok = wait(&q_full[n_seg & 1], (n_seg >> 1) & 1, vfail, a.wait_ns);
                for (int t = g.t0; ok && t < g.t1; ++t, ++it, rk.next()) {
                    const int bf = it & 1;
                    ok = BITS == 8 ? wait(&k_full[rk.i], rk.parity, vfail, a.wait_ns) : wait(&ko_full, it & 1, vfail, a.wait_ns);
                    if (it >= 2) ok = ok && wait(&s_free[bf], ((it >> 1) - 1) & 1, vfail, a.wait_ns);
                    if (!ok) break;
                    umma::tc_fence_after();
                    const uint64_t dk = desc_rows8<D>(BITS == 8 ? kr0 + rk.i * C::kRaw : k80);
#pragma unroll
                    for (int s = 0; s < D / 32; ++s) mma_f8(tmem + bf * 2 * NB, dk + 2 * s, dq + 2 * s, id, s != 0);
                    umma::mma_commit(&s_full[bf]);
                    umma::mma_commit(BITS == 8 ? &k_empty[rk.i] : &ko_done);
                    // test hook: with S in flight, wait for what never comes
                    if (it == 0 && a.inject) ok = wait(&never, 0, vfail, a.wait_ns);
                }
                umma::mma_commit(&q_free);
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            ++n_seg;
        }
        if (lane == 0) umma::mma_commit(&drain);
        __syncwarp();
    } else if (warp == 2) {
        // ---- O += V^T P^T (its own warp: starting a batch of products takes longer than the batch) ----
        constexpr uint32_t id = idesc_f8(128, 3 * NB, 1) | (1u << 15) | (1u << 16);  // both MN-major
        const uint64_t dp = desc_rows8<128>(p0);
        Segment g;
        Ring<SV> rv;
        int it = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            if (lane == 0) {
                for (int t = g.t0; ok && t < g.t1; ++t, ++it, rv.next()) {
                    // (4 bits: the loaded codes' buffer may be in its next use by now)
                    ok = BITS == 8 ? wait(&v_full[rv.i], rv.parity, vfail, a.wait_ns) : wait(&vo_full, it & 1, vfail, a.wait_ns);
                    ok = ok && wait(&p_full, it & 1, vfail, a.wait_ns);
                    if (!ok) break;
                    umma::tc_fence_after();
                    // d = 64: the accumulator's upper 64 rows repeat the lower ones and are not read
                    const uint64_t dv = desc_rows8<D>(BITS == 8 ? vr0 + rv.i * C::kRaw : v80);
#pragma unroll
                    for (int s = 0; s < kTile / 32; ++s) mma_f8(t_o, dv + s * (32 * D / 16), dp + s * 256, id, !(t == g.t0 && s == 0));
                    umma::mma_commit(&pv_done);
                    if (BITS == 8) umma::mma_commit(&v_empty[rv.i]);
                }
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        // all products issued, S's too, complete before TMEM goes back
        if (lane == 0) {
            umma::mma_commit(&drain);
            umma::mbar_wait(&drain, 0, kDrainNs);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ---- this CTA's part of the line, unit by unit, and each unit's Q rows ------------------------
        Line<NB> line(a, s_chunk);
        bool ok = true;
        for (int n_seg = 0; ok; ++n_seg) {
            Segment g;
            line.next(a, g);
            const int i = n_seg & (kRing - 1);
            if (n_seg >= kRing) ok = wait(&seg_free[i], ((n_seg / kRing) - 1) & 1, vfail, a.wait_ns);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane == 0) {
                s_seg[i] = g;
                umma::mbar_arrive(&seg_full[i]);
            }
            if (g.t1 == 0) break;
            // Q's rows, once the last unit's products with its own are done
            const int qb = n_seg & 1;
            if (n_seg >= 1) ok = wait(&q_free, (n_seg - 1) & 1, vfail, a.wait_ns);
            if (n_seg >= 2) ok = ok && wait(&m_free[qb], ((n_seg >> 1) - 1) & 1, vfail, a.wait_ns);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            make_q<D, NB>(a, g, base + (q0 - sm), s_qs[qb], s_tok[qb], s_row[qb]);
            if (lane == 0) umma::mbar_arrive(&q_full[qb]);
        }
        if (lane == 0) a.desc[cta] = ok ? line.cut : make_int4(-1, 0, 0, 0);
    } else if (BITS == 4) {
        // ---- 4-bit codes into e4m3 operands, two warps for K and two for V: one (row, 32-channel group) a step, its
        // scale relative to the row's largest.  A word's eight magnitudes are two byte permutes of the group's eight
        // levels. ----
        constexpr int GR = D / 32, kThreads = C::kConv > 0 ? C::kConv * 16 : 32;
        const int which = (warp - 8) / (kThreads / 32), w = (warp - 8) % (kThreads / 32) * 32 + lane;
        Segment g;
        Ring<SK> rk;
        Ring<SV> rv;
        int it = 0, n_seg = 0;
        bool ok = true;
        while (ok && next_segment(g, n_seg)) {
            ++n_seg;
            for (int t = g.t0; t < g.t1; ++t, ++it, rk.next(), rv.next()) {
                ok = wait(&v_full[rv.i], rv.parity, vfail, a.wait_ns);  // (K's scales come with V's codes)
                if (!which) ok = ok && wait(&k_full[rk.i], rk.parity, vfail, a.wait_ns);
                if (it >= 1) ok = ok && wait(which ? &pv_done : &ko_done, (it - 1) & 1, vfail, a.wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint8_t *src = base + ((which ? vr0 + rv.i * C::kRaw : kr0 + rk.i * C::kRaw) - sm);
                const uint8_t *scales = base + (sc0 - sm) + rv.i * C::kScales + which * 128 * GR;
                uint8_t *dst = base + ((which ? v80 : k80) - sm);
#pragma unroll 2
                for (int i = 0; i < kTile * GR / kThreads; ++i) {
                    const int idx = w + kThreads * i, row = idx / GR, gq = idx % GR;
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + idx * 16);
                    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
                    const uint8_t *sc = scales + row * GR;
                    uint32_t top, mine;
                    if constexpr (GR == 4) {
                        const uint32_t all = *reinterpret_cast<const uint32_t *>(sc);
                        const uint32_t m = __vmaxu4(all, all >> 16);
                        top = max(m & 0xFFu, (m >> 8) & 0xFFu);
                        mine = (all >> (8 * gq)) & 0xFFu;
                    } else {
                        const uint32_t all = *reinterpret_cast<const uint16_t *>(sc);
                        top = max(all & 0xFFu, all >> 8);
                        mine = (all >> (8 * gq)) & 0xFFu;
                    }
                    const uint2 lv = s_lv[min(top - mine, 15u)];
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
                if (lane == 0) {
                    umma::mbar_arrive(which ? &vo_full : &ko_full);
                    if (!which) umma::mbar_arrive(&k_empty[rk.i]);
                    umma::mbar_arrive(&v_empty[rv.i]);
                }
            }
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
    if (warp == 2) {
        umma::tc_fence_after();
        umma::tmem_dealloc(tmem, C::kTmem);
    }
}

}  // namespace pa
}  // namespace qvg
