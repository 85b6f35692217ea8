// latent.cu -- the latent cache: write tokens into their slots (rotating the
// shared key part on the way) and read slots back.  Formats: see qvg_latent in
// qvg.h.
#include "latent.cuh"
#include "rope.cuh"

namespace qvg {

qvg_status check_latent(const qvg_latent *c, bool shape_only) {
    if (!c || c->num_pages < 1 || c->dr < 0 || c->dr > 128 || c->dr % 8 != 0) return QVG_ERR_INVALID_ARG;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
        return QVG_ERR_INVALID_ARG;
    if (c->dc != 64 && c->dc != 128 && c->dc != 192 && c->dc != 256) return QVG_ERR_UNSUPPORTED;
    if (shape_only) return QVG_OK;
    if (!c->c || reinterpret_cast<uintptr_t>(c->c) % 16 != 0) return QVG_ERR_INVALID_ARG;
    if (c->dr > 0 && (!c->kr || reinterpret_cast<uintptr_t>(c->kr) % 16 != 0)) return QVG_ERR_INVALID_ARG;
    return QVG_OK;
}

namespace {

constexpr int kWarps = 8;

struct LatentArgs {
    uint16_t *c, *kr;
    int dc, dr;
    long long n_slots;
    int *err;
};

LatentArgs latent_args(const qvg_latent *c) {
    return {static_cast<uint16_t *>(c->c), static_cast<uint16_t *>(c->kr), c->dc, c->dr,
            static_cast<long long>(c->num_pages) * c->page_size, device_error_word()};
}

__device__ __forceinline__ bool not_finite(uint4 v) {  // any of eight bf16 numbers
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad = bad || (x[i] & 0x7F80u) == 0x7F80u || (x[i] & 0x7F800000u) == 0x7F800000u;
    return bad;
}

// One warp per token: lane i holds channels 8 i .. of the latent, and of the
// key part.  A key part that turns goes through shared memory, from which a
// lane takes its channels' partners; the token's cosines and sines are made by
// the warp, one pair a lane.  A token that holds an infinity or a NaN (before
// the rotation or after) becomes NaN throughout.
// Bound by HBM: 4 (dc + dr) bytes a token.  A warp takes two tokens, whose slots,
// rows and positions are all asked for before any is waited for (one token, its
// slot first: 25 us for 37,440 tokens of 256 + 64 channels, 48.7 MB; so 13).
template <bool HALF>
__device__ __forceinline__ uint4 turned(const RopeArgs &r, uint4 v, const float2 *cs, const uint16_t *row, int lane) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ch = lane * 8 + 2 * i;
        if (!HALF) {
            if (ch >= 2 * r.pairs) continue;
            const float2 y = rope_turn(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u), cs[ch / 2].x, cs[ch / 2].y);
            w[i] = f32_to_bf16(y.x) | static_cast<uint32_t>(f32_to_bf16(y.y)) << 16;
        } else {
            uint32_t got = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int x = ch + e;
                const uint16_t own = static_cast<uint16_t>(w[i] >> (16 * e));
                uint16_t y = own;
                if (x < r.pairs)
                    y = f32_to_bf16(rope_turn(bf16_to_f32(own), bf16_to_f32(row[x + r.pairs]), cs[x].x, cs[x].y).x);
                else if (x < 2 * r.pairs)
                    y = f32_to_bf16(rope_turn(bf16_to_f32(row[x - r.pairs]), bf16_to_f32(own), cs[x - r.pairs].x, cs[x - r.pairs].y).y);
                got |= static_cast<uint32_t>(y) << (16 * e);
            }
            w[i] = got;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int N>  // tokens of a warp
__global__ void __launch_bounds__(kWarps * 32)
    k_latent_append(const __grid_constant__ RopeArgs r, LatentArgs a, const uint16_t *__restrict__ c, const uint16_t *__restrict__ kr,
                    int n, long long cs, long long ks, const int64_t *__restrict__ slots, const int32_t *__restrict__ positions) {
    __shared__ float2 s_cs[kWarps][N][QVG_ROPE_MAX_PAIRS];
    __shared__ __align__(16) uint16_t s_row[kWarps][N][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x * kWarps + warp) * N;
    const bool in_c = lane * 8 < a.dc, in_kr = lane * 8 < a.dr;
    long long slot[N];
    uint4 vc[N], vk[N];
    int32_t p0[N], p1[N];  // positions of the lane's two pairs
    const uint64_t step0 = r.step[lane], step1 = r.step[lane + 32];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const long long t = t0 + e;
        const bool live = t < n;
        slot[e] = live ? slots[t] : -1;
        vc[e] = live && in_c ? __ldcs(reinterpret_cast<const uint4 *>(c + t * cs) + lane) : make_uint4(0, 0, 0, 0);
        vk[e] = live && in_kr ? __ldcs(reinterpret_cast<const uint4 *>(kr + t * ks) + lane) : make_uint4(0, 0, 0, 0);
        p0[e] = live && lane < r.pairs ? positions[t * r.axes + r.axis[lane]] : 0;
        p1[e] = live && lane + 32 < r.pairs ? positions[t * r.axes + r.axis[lane + 32]] : 0;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (slot[e] < 0) continue;
        if (slot[e] >= a.n_slots) {
            if (lane == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
            continue;
        }
        bool bad = not_finite(vc[e]) || not_finite(vk[e]);
        if (r.pairs > 0) {
            if (lane < r.pairs) s_cs[warp][e][lane] = rope_cos_sin(step0, p0[e], r.mscale, false);
            if (lane + 32 < r.pairs) s_cs[warp][e][lane + 32] = rope_cos_sin(step1, p1[e], r.mscale, false);
            if (in_kr) *reinterpret_cast<uint4 *>(&s_row[warp][e][lane * 8]) = vk[e];
            __syncwarp();
            if (in_kr && lane * 8 < 2 * r.pairs) {
                vk[e] = r.layout == QVG_ROPE_INTERLEAVED ? turned<false>(r, vk[e], s_cs[warp][e], s_row[warp][e], lane)
                                                         : turned<true>(r, vk[e], s_cs[warp][e], s_row[warp][e], lane);
                bad = bad || not_finite(vk[e]);
            }
        }
        if (__any_sync(0xFFFFFFFFu, bad)) vc[e] = vk[e] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
        if (in_c) *(reinterpret_cast<uint4 *>(a.c + slot[e] * a.dc) + lane) = vc[e];
        if (in_kr) *(reinterpret_cast<uint4 *>(a.kr + slot[e] * a.dr) + lane) = vk[e];
    }
}

// One warp per token.  Bound by HBM.
__global__ void __launch_bounds__(kWarps * 32) k_latent_read(LatentArgs a, const int64_t *__restrict__ slots, int n,
                                                            uint16_t *__restrict__ c_out, uint16_t *__restrict__ kr_out) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= n) return;
    const long long slot = slots[t];
    const bool in = slot >= 0 && slot < a.n_slots;
    if (slot >= a.n_slots && lane == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (c_out && lane * 8 < a.dc)
        *(reinterpret_cast<uint4 *>(c_out + static_cast<long long>(t) * a.dc) + lane) =
            in ? *(reinterpret_cast<const uint4 *>(a.c + slot * a.dc) + lane) : zero;
    if (kr_out && lane * 8 < a.dr)
        *(reinterpret_cast<uint4 *>(kr_out + static_cast<long long>(t) * a.dr) + lane) =
            in ? *(reinterpret_cast<const uint4 *>(a.kr + slot * a.dr) + lane) : zero;
}

bool misaligned(const void *p, uintptr_t to) { return !p || reinterpret_cast<uintptr_t>(p) % to != 0; }

}  // namespace
}  // namespace qvg

using namespace qvg;

extern "C" {

qvg_status qvg_latent_bytes(int32_t dc, int32_t dr, int32_t page_size, int32_t num_pages, size_t *c, size_t *kr) {
    if (!c || !kr) return QVG_ERR_INVALID_ARG;
    const qvg_latent l{dc, dr, page_size, num_pages, nullptr, nullptr};
    const qvg_status s = check_latent(&l, true);
    if (s != QVG_OK) return s;
    const size_t rows = static_cast<size_t>(num_pages) * page_size;
    *c = rows * dc * 2;
    *kr = rows * dr * 2;
    return QVG_OK;
}

qvg_status qvg_latent_append(const qvg_latent *cache, const void *c_bf16, const void *k_rope_bf16, int32_t n,
                             int64_t c_stride, int64_t kr_stride, const int64_t *slots, const qvg_rope_plan *plan,
                             const int32_t *positions, void *stream) {
    const qvg_status s = check_latent(cache, false);
    if (s != QVG_OK) return s;
    if (n < 0 || c_stride < cache->dc || c_stride % 8 != 0) return QVG_ERR_INVALID_ARG;
    if (cache->dr > 0 && (kr_stride < cache->dr || kr_stride % 8 != 0)) return QVG_ERR_INVALID_ARG;
    if (plan && !rope_plan_ok(plan, cache->dr)) return QVG_ERR_INVALID_ARG;
    if (n == 0) return QVG_OK;
    if (misaligned(c_bf16, 16) || misaligned(slots, 8) || (cache->dr > 0 && misaligned(k_rope_bf16, 16)) ||
        (plan && misaligned(positions, 4)))
        return QVG_ERR_INVALID_ARG;
    const RopeArgs r = plan ? rope_args(plan, false) : RopeArgs{};
    const uint16_t *c = static_cast<const uint16_t *>(c_bf16), *kr = static_cast<const uint16_t *>(k_rope_bf16);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // two tokens a warp once that still leaves every SM four blocks
    if (n >= 8 * kWarps * sm_count_current())
        k_latent_append<2><<<ceil_div(n, 2 * kWarps), kWarps * 32, 0, st>>>(r, latent_args(cache), c, kr, n, c_stride, kr_stride, slots, positions);
    else
        k_latent_append<1><<<ceil_div(n, kWarps), kWarps * 32, 0, st>>>(r, latent_args(cache), c, kr, n, c_stride, kr_stride, slots, positions);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

qvg_status qvg_latent_read(const qvg_latent *cache, const int64_t *slots, int32_t n, void *c_out, void *kr_out,
                           void *stream) {
    const qvg_status s = check_latent(cache, false);
    if (s != QVG_OK) return s;
    if (n < 0) return QVG_ERR_INVALID_ARG;
    if (cache->dr == 0) kr_out = nullptr;
    if (n == 0 || (!c_out && !kr_out)) return QVG_OK;
    if (misaligned(slots, 8) || (c_out && misaligned(c_out, 16)) || (kr_out && misaligned(kr_out, 16))) return QVG_ERR_INVALID_ARG;
    k_latent_read<<<ceil_div(n, kWarps), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(
        latent_args(cache), slots, n, static_cast<uint16_t *>(c_out), static_cast<uint16_t *>(kr_out));
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

}  // extern "C"
