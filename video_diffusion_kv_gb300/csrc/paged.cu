// paged.cu -- the paged token cache: quantise tokens into their slots
// (rotating K on the way) and read slots back.  Formats: see qvg_paged in qvg.h.
#include "paged.cuh"
#include "rope.cuh"

namespace qvg {

qvg_status check_paged(const qvg_paged *c, bool shape_only) {
    if (!c || c->H < 1 || c->num_pages < 1 || (c->bits != 8 && c->bits != 4)) return QVG_ERR_INVALID_ARG;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
        return QVG_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return QVG_ERR_UNSUPPORTED;
    if (shape_only) return QVG_OK;
    for (const void *b : {c->k_codes, c->k_scales, c->v_codes, c->v_scales})
        if (!b || reinterpret_cast<uintptr_t>(b) % 16 != 0) return QVG_ERR_INVALID_ARG;
    return QVG_OK;
}

namespace {

constexpr int kWarps = 8;

struct PagedArgs {
    uint8_t *codes[2], *scales[2];  // K, V
    int H, page_log2;
    long long n_slots;
    int *err;
};

PagedArgs paged_args(const qvg_paged *c) {
    PagedArgs a{};
    a.codes[0] = c->k_codes;
    a.codes[1] = c->v_codes;
    a.scales[0] = c->k_scales;
    a.scales[1] = c->v_scales;
    a.H = c->H;
    a.page_log2 = __builtin_ctz(static_cast<unsigned>(c->page_size));
    a.n_slots = static_cast<long long>(c->num_pages) * c->page_size;
    a.err = device_error_word();
    return a;
}

// Row (page, head, offset) of a slot and head.
__device__ __forceinline__ size_t row_of(const PagedArgs &a, long long slot, int h) {
    const long long page = slot >> a.page_log2, off = slot & ((1 << a.page_log2) - 1);
    return static_cast<size_t>(((page * a.H + h) << a.page_log2) + off);
}

// 16 channels of one row (packed bf16 pairs) into their codes.  The lanes of
// a row are neighbours (LANES of them).  8 bits: one scale for the row.
// 4 bits: one for 32 channels, i.e. two lanes.  An infinity
// or a NaN marks every group of the row.
template <int BITS, int LANES>
__device__ __forceinline__ void quantise16(const uint32_t (&x)[8], uint8_t *codes, uint8_t *scales, size_t row, int u,
                                           bool live) {
    uint32_t m2 = 0;  // largest magnitudes of the even and the odd channels, as bit patterns
#pragma unroll
    for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, x[i] & 0x7FFF7FFFu);
    uint32_t amax = max(m2 & 0xFFFFu, m2 >> 16);
    constexpr int kSpan = BITS == 8 ? LANES : 2;
#pragma unroll
    for (int o = 1; o < kSpan; o <<= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    uint32_t row_max = amax;
#pragma unroll
    for (int o = kSpan; o < LANES; o <<= 1) row_max = max(row_max, __shfl_xor_sync(0xFFFFFFFFu, row_max, o));
    const uint32_t sb = row_max >= 0x7F80u ? 255u : scale_byte<BITS>(amax);
    const float inv = sb == 255u ? 0.0f : scale_inverse(sb);
    const uint32_t keep = sb == 255u ? 0u : 0xFFFFFFFFu;  // a row with an infinity or a NaN: codes 0
    // Under the largest scale a magnitude above 1.875 2^127 (1.75 2^127 at 4
    // bits) would round up to 2^128: the code below it is the last finite one.
    const bool top = sb == (BITS == 8 ? 247u : 253u);
    constexpr float kLast = BITS == 8 ? 240.0f : 3.0f;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t xi = x[i] & keep;
        float lo = __uint_as_float(xi << 16) * inv, hi = __uint_as_float(xi & 0xFFFF0000u) * inv;
        if (top) {
            lo = fminf(fmaxf(lo, -kLast), kLast);
            hi = fminf(fmaxf(hi, -kLast), kLast);
        }
        w[i] = BITS == 8 ? e4m3x2(lo, hi) : e2m1x2(lo, hi);
    }
    if (!live) return;
    if constexpr (BITS == 8) {
        *reinterpret_cast<uint4 *>(codes + (row * LANES + u) * 16) =
            make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        if (u == 0) scales[row] = static_cast<uint8_t>(sb);
    } else {
        *reinterpret_cast<uint2 *>(codes + (row * LANES + u) * 8) =
            make_uint2(w[0] | w[1] << 8 | w[2] << 16 | w[3] << 24, w[4] | w[5] << 8 | w[6] << 16 | w[7] << 24);
        if ((u & 1) == 0) scales[row * (LANES / 2) + u / 2] = static_cast<uint8_t>(sb);
    }
}

// How K is rotated on its way: not at all, pairs of neighbouring channels
// (a lane has both), halves whose 16-byte pieces line up (pairs % 8 == 0), or
// any halves.
enum { kNoRope = 0, kPairs = 1, kHalves = 2, kAnyHalves = 3 };

// One warp per token (blockIdx.y: a share of its heads); a lane holds 16
// consecutive channels, D / 16 lanes a head, 512 / D heads side by side.
//   The token's cosines and sines are made once per warp (pairs / 32 angles a
// lane) and kept in registers for the lane's 16 channels.  With halves the K
// row goes through shared memory, from which each lane takes its channels'
// partners, 16 bytes at a time where they line up (2 bytes at a time, it took
// 2.3 times as long).  The rotated row is rounded to bf16, as qvg_rope would
// store it.
// Bound by HBM: reads 4 H D bytes a token, writes 2 H D bits / 8 + scales.
// 37,440 tokens of 16 heads of 128 into the 4-bit cache with K rotated, and back
// as bf16 (0.78 GB in all): 188 us, 4.1 TB/s, 61 % of a plain copy's rate, 109 us of
// it this kernel (3.5 TB/s: neither HBM nor, at 65 %, the issue slots are full; a warp
// loads a few heads, works on them and stores them before it loads the next; the
// rotation in 64 registers, four blocks an SM; three: 197 us, five: 209 us); 48
// tokens of 8 heads: 6 us.
template <int D, int BITS, int ROPE>
__global__ void __launch_bounds__(kWarps * 32, ROPE == kNoRope ? 5 : 4)
    k_paged_append(const __grid_constant__ RopeArgs r, PagedArgs a, const uint16_t *__restrict__ k, const uint16_t *__restrict__ v, int n,
                   long long ks, long long vs, const int64_t *__restrict__ slots, const int32_t *__restrict__ positions,
                   int heads_per_block) {
    constexpr int LANES = D / 16, SIDE = 32 / LANES;
    constexpr bool SHARED = ROPE == kHalves || ROPE == kAnyHalves;
    __shared__ float2 s_cs[ROPE ? kWarps : 1][ROPE ? QVG_ROPE_MAX_PAIRS : 1];
    __shared__ __align__(16) uint16_t s_row[SHARED ? kWarps : 1][SHARED ? SIDE * D : 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= n) return;
    const long long slot = slots[t];
    if (slot < 0) return;
    if (slot >= a.n_slots) {
        if (lane == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
        return;
    }
    const int u = lane % LANES, hs = lane / LANES;
    float co[ROPE == kPairs ? 8 : 16], si[ROPE == kPairs ? 8 : 16];  // si with the sign of the channel's place in its pair
    const int turned = r.pairs - u * 8;  // kPairs: the lane's pairs that turn, from its first on
    int from[2];  // where the lane's two runs of 8 channels have their partners in the row
    if constexpr (ROPE != kNoRope) {
        for (int i = lane; i < r.pairs; i += 32)
            s_cs[warp][i] = rope_cos_sin(r.step[i], positions[static_cast<long long>(t) * r.axes + r.axis[i]], r.mscale, false);
        __syncwarp();
        if constexpr (ROPE == kPairs) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 cs = u * 8 + i < r.pairs ? s_cs[warp][u * 8 + i] : make_float2(1.0f, 0.0f);
                co[i] = cs.x;
                si[i] = cs.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int c = u * 16 + i;
                const bool second = c >= r.pairs;
                const float2 cs = c < 2 * r.pairs ? s_cs[warp][second ? c - r.pairs : c] : make_float2(1.0f, 0.0f);
                co[i] = cs.x;
                si[i] = second ? cs.y : -cs.y;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = u * 16 + 8 * h;
                from[h] = c < r.pairs ? c + r.pairs : c < 2 * r.pairs ? c - r.pairs : c;
            }
        }
    }
    const int h0 = blockIdx.y * heads_per_block, h1 = min(a.H, h0 + heads_per_block);
    const uint16_t *kr = k + t * ks, *vr = v + t * vs;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int hb = h0; hb < h1; hb += SIDE) {
        const int h = hb + hs;
        const bool live = h < h1;
        const uint4 *pk = reinterpret_cast<const uint4 *>(kr + static_cast<long long>(h) * D + u * 16);
        const uint4 *pv = reinterpret_cast<const uint4 *>(vr + static_cast<long long>(h) * D + u * 16);
        const uint4 k0 = live ? __ldcs(pk) : zero, k1 = live ? __ldcs(pk + 1) : zero;
        const uint4 v0 = live ? __ldcs(pv) : zero, v1 = live ? __ldcs(pv + 1) : zero;
        uint32_t xk[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
        const uint32_t xv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        if constexpr (ROPE == kPairs) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 t = rope_turn(__uint_as_float(xk[i] << 16), __uint_as_float(xk[i] & 0xFFFF0000u), co[i], si[i]);
                const __nv_bfloat162 y = __floats2bfloat162_rn(t.x, t.y);
                // (a pair that does not turn stays as it is: 0 times its partner would make +0 of -0)
                xk[i] = i < turned ? *reinterpret_cast<const uint32_t *>(&y) : xk[i];
            }
        }
        if constexpr (SHARED) {
            uint16_t *row = s_row[warp] + hs * D;
            __syncwarp();  // the previous heads' partners have been read
            reinterpret_cast<uint4 *>(row + u * 16)[0] = k0;
            reinterpret_cast<uint4 *>(row + u * 16)[1] = k1;
            __syncwarp();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pw[4];
                if constexpr (ROPE == kHalves) {
                    const uint4 p = *reinterpret_cast<const uint4 *>(row + from[half]);
                    pw[0] = p.x, pw[1] = p.y, pw[2] = p.z, pw[3] = p.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w = 0;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int c = u * 16 + 8 * half + 2 * i + e;
                            const int q = c < r.pairs ? c + r.pairs : c < 2 * r.pairs ? c - r.pairs : c;
                            w |= static_cast<uint32_t>(row[q]) << (16 * e);
                        }
                        pw[i] = w;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = 8 * half + 2 * i;
                    const uint32_t x = xk[e / 2];
                    const __nv_bfloat162 y =
                        __floats2bfloat162_rn(fmaf(__uint_as_float(x << 16), co[e], __fmul_rn(__uint_as_float(pw[i] << 16), si[e])),  // as rope_turn
                                              fmaf(__uint_as_float(x & 0xFFFF0000u), co[e + 1], __fmul_rn(__uint_as_float(pw[i] & 0xFFFF0000u), si[e + 1])));
                    xk[e / 2] = *reinterpret_cast<const uint32_t *>(&y);
                }
            }
        }
        const size_t at = live ? row_of(a, slot, h) : 0;
        quantise16<BITS, LANES>(xk, a.codes[0], a.scales[0], at, u, live);
        quantise16<BITS, LANES>(xv, a.codes[1], a.scales[1], at, u, live);
    }
}

// One warp per token, lanes as in k_paged_append; K and V one after the
// other.  Bound by HBM: reads the codes and scales, writes n H D elements
// for each of K and V.  37,440 tokens of 16 heads of 128, 8 bits, as bf16 (0.46
// GB): 79 us, 5.8 TB/s, 86 % of a plain copy's rate; 4 bits (0.39 GB): 78 us, 5 TB/s,
// as long, so there the instructions of the conversion count too.
template <int D, int BITS, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) k_paged_read(PagedArgs a, const int64_t *__restrict__ slots, int n,
                                                           void *__restrict__ k_out, void *__restrict__ v_out,
                                                           int heads_per_block) {
    constexpr int LANES = D / 16, SIDE = 32 / LANES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= n) return;
    const long long slot = slots[t];
    const bool in = slot >= 0 && slot < a.n_slots;
    if (slot >= a.n_slots && lane == 0 && blockIdx.y == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
    const int u = lane % LANES, hs = lane / LANES;
    const int h0 = blockIdx.y * heads_per_block, h1 = min(a.H, h0 + heads_per_block);
#pragma unroll 4
    for (int h = h0 + hs; h < h1; h += SIDE) {
        const size_t row = in ? row_of(a, slot, h) : 0;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            void *out = which ? v_out : k_out;
            if (!out) continue;
            float f[16];
            if (in) {
                uint32_t w[8];  // fp16 pairs
                float s;
                if constexpr (BITS == 8) {
                    const uint4 c = *reinterpret_cast<const uint4 *>(a.codes[which] + (row * LANES + u) * 16);
                    const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = e4m3x2_to_f16x2(cw[i / 2] >> (16 * (i & 1)));
                    s = scale_of(a.scales[which][row]);
                } else {
                    const uint2 c = *reinterpret_cast<const uint2 *>(a.codes[which] + (row * LANES + u) * 8);
                    const uint32_t cw[2] = {c.x, c.y};
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = e2m1x2_to_f16x2((cw[i / 4] >> (8 * (i & 3))) & 0xFFu);
                    s = scale_of(a.scales[which][row * (LANES / 2) + u / 2]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                    f[2 * i] = p.x * s;
                    f[2 * i + 1] = p.y * s;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = 0.0f;
            }
            const size_t at = (static_cast<size_t>(t) * a.H + h) * D + u * 16;
            if constexpr (BF16) {
                uint32_t b[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {  // exact: at most four significant bits
                    const __nv_bfloat162 y = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                    b[i] = *reinterpret_cast<const uint32_t *>(&y);
                }
                uint4 *q = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at);
                q[0] = make_uint4(b[0], b[1], b[2], b[3]);
                q[1] = make_uint4(b[4], b[5], b[6], b[7]);
            } else {
                float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
            }
        }
    }
}

// Heads per block and the grid's second extent: one block takes all heads
// unless the tokens alone leave the SMs without about four blocks each.
dim3 token_grid(int n, int H, int side, int *per) {
    const int blocks = ceil_div(n, kWarps);
    const int shares = std::max(1, std::min(ceil_div(H, side), 4 * sm_count_current() / blocks));
    *per = ceil_div(ceil_div(H, side), shares) * side;
    return dim3(blocks, ceil_div(H, *per));
}

template <int D, int BITS>
qvg_status launch_append(const qvg_paged *c, const uint16_t *k, const uint16_t *v, int n, long long ks, long long vs,
                         const int64_t *slots, const qvg_rope_plan *plan, const int32_t *positions, cudaStream_t st) {
    const PagedArgs a = paged_args(c);
    int per;
    const dim3 grid = token_grid(n, c->H, 512 / D, &per);
    const RopeArgs r = plan ? rope_args(plan, false) : RopeArgs{};
    if (!plan)
        k_paged_append<D, BITS, kNoRope><<<grid, kWarps * 32, 0, st>>>(r, a, k, v, n, ks, vs, slots, positions, per);
    else if (r.layout == QVG_ROPE_INTERLEAVED)
        k_paged_append<D, BITS, kPairs><<<grid, kWarps * 32, 0, st>>>(r, a, k, v, n, ks, vs, slots, positions, per);
    else if (r.pairs % 8 == 0)
        k_paged_append<D, BITS, kHalves><<<grid, kWarps * 32, 0, st>>>(r, a, k, v, n, ks, vs, slots, positions, per);
    else
        k_paged_append<D, BITS, kAnyHalves><<<grid, kWarps * 32, 0, st>>>(r, a, k, v, n, ks, vs, slots, positions, per);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

template <int D, int BITS>
qvg_status launch_read(const qvg_paged *c, const int64_t *slots, int n, void *k_out, void *v_out, int out_dtype,
                       cudaStream_t st) {
    const PagedArgs a = paged_args(c);
    int per;
    const dim3 grid = token_grid(n, c->H, 512 / D, &per);
    if (out_dtype == QVG_OUT_BF16)
        k_paged_read<D, BITS, true><<<grid, kWarps * 32, 0, st>>>(a, slots, n, k_out, v_out, per);
    else
        k_paged_read<D, BITS, false><<<grid, kWarps * 32, 0, st>>>(a, slots, n, k_out, v_out, per);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

bool misaligned(const void *p, uintptr_t to) { return !p || reinterpret_cast<uintptr_t>(p) % to != 0; }

}  // namespace
}  // namespace qvg

using namespace qvg;

extern "C" {

qvg_status qvg_paged_bytes(int32_t H, int32_t d, int32_t page_size, int32_t num_pages, int32_t bits, size_t *codes,
                           size_t *scales) {
    if (!codes || !scales) return QVG_ERR_INVALID_ARG;
    qvg_paged c{};
    c.H = H;
    c.d = d;
    c.page_size = page_size;
    c.num_pages = num_pages;
    c.bits = bits;
    const qvg_status s = check_paged(&c, true);
    if (s != QVG_OK) return s;
    const size_t rows = static_cast<size_t>(num_pages) * H * page_size;
    *codes = rows * (static_cast<size_t>(d) * bits / 8);
    *scales = rows * (bits == 8 ? 1 : d / 32);
    return QVG_OK;
}

qvg_status qvg_paged_append(const qvg_paged *cache, const void *k_bf16, const void *v_bf16, int32_t n,
                            int64_t k_stride, int64_t v_stride, const int64_t *slots, const qvg_rope_plan *plan,
                            const int32_t *positions, void *stream) {
    const qvg_status s = check_paged(cache, false);
    if (s != QVG_OK) return s;
    const int64_t row = static_cast<int64_t>(cache->H) * cache->d;
    if (n < 0 || k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0) return QVG_ERR_INVALID_ARG;
    if (plan && !rope_plan_ok(plan, cache->d)) return QVG_ERR_INVALID_ARG;
    if (n == 0) return QVG_OK;
    if (misaligned(k_bf16, 16) || misaligned(v_bf16, 16) || misaligned(slots, 8) || (plan && misaligned(positions, 4)))
        return QVG_ERR_INVALID_ARG;
    const uint16_t *k = static_cast<const uint16_t *>(k_bf16), *v = static_cast<const uint16_t *>(v_bf16);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache->d == 64)
        return cache->bits == 8 ? launch_append<64, 8>(cache, k, v, n, k_stride, v_stride, slots, plan, positions, st)
                                : launch_append<64, 4>(cache, k, v, n, k_stride, v_stride, slots, plan, positions, st);
    return cache->bits == 8 ? launch_append<128, 8>(cache, k, v, n, k_stride, v_stride, slots, plan, positions, st)
                            : launch_append<128, 4>(cache, k, v, n, k_stride, v_stride, slots, plan, positions, st);
}

qvg_status qvg_paged_read(const qvg_paged *cache, const int64_t *slots, int32_t n, void *k_out, void *v_out,
                          int32_t out_dtype, void *stream) {
    const qvg_status s = check_paged(cache, false);
    if (s != QVG_OK) return s;
    if (n < 0 || (out_dtype != QVG_OUT_F32 && out_dtype != QVG_OUT_BF16)) return QVG_ERR_INVALID_ARG;
    if (n == 0 || (!k_out && !v_out)) return QVG_OK;
    if (misaligned(slots, 8) || (k_out && misaligned(k_out, 16)) || (v_out && misaligned(v_out, 16)))
        return QVG_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache->d == 64)
        return cache->bits == 8 ? launch_read<64, 8>(cache, slots, n, k_out, v_out, out_dtype, st)
                                : launch_read<64, 4>(cache, slots, n, k_out, v_out, out_dtype, st);
    return cache->bits == 8 ? launch_read<128, 8>(cache, slots, n, k_out, v_out, out_dtype, st)
                            : launch_read<128, 4>(cache, slots, n, k_out, v_out, out_dtype, st);
}

}  // extern "C"
