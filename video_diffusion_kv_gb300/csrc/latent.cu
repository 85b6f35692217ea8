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
constexpr int kAppendBlocks = 4;  // blocks an SM, at most: what its registers hold

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

// A warp takes tokens one after the other, the next one's slot, rows and positions
// on their way meanwhile.  Lane i holds channels 8 i .. of the latent and, of the
// key part, the pairs i and i + 32 (with halves two channels dims / 2 apart; a pair
// past the rotated ones is two neighbours), so a pair turns within its lane; the lane's
// steps and axes stay in registers.  A token that holds an infinity or a NaN (before
// the rotation or after) becomes NaN throughout.
// Bound by the instructions (215 a token, most of them the angles') beside HBM, 4 (dc + dr)
// bytes a token: 37,440 tokens of 256 + 64 channels, 48.7 MB, three axes: 12 us, 4.1 TB/s.  (One token
// a warp, its channels in eights and the partners through shared memory: 25 us.)
struct Token {
    long long slot;
    uint4 c;
    uint32_t k[2];   // the lane's pairs
    int32_t pos[2];
};

constexpr int kMostTokens = 1 << 30;  // of a call: the warps' indices step past the last one in 32 bits

template <bool HALF>
__global__ void __launch_bounds__(kWarps * 32)
    k_latent_append(const __grid_constant__ RopeArgs r, LatentArgs a, const uint16_t *__restrict__ c, const uint16_t *__restrict__ kr,
                    int n, long long cs, long long ks, const int64_t *__restrict__ slots, const int32_t *__restrict__ positions) {
    const int lane = threadIdx.x & 31, step = gridDim.x * kWarps;
    const bool in_c = lane * 8 < a.dc;
    bool in[2], turns[2];
    int lo[2], hi[2];  // channels of the pairs
    uint64_t angle[2];
    int axis[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int p = lane + 32 * i;
        in[i] = 2 * p < a.dr;
        turns[i] = p < r.pairs;
        lo[i] = HALF && turns[i] ? p : 2 * p;
        hi[i] = HALF && turns[i] ? p + r.pairs : 2 * p + 1;
        angle[i] = turns[i] ? r.step[p] : 0;
        axis[i] = turns[i] ? r.axis[p] : 0;
    }
    auto fetch = [&](int t, Token &x) {
        x.slot = -1;
        if (t >= n) return;
        x.slot = slots[t];
        if (in_c) x.c = __ldcs(reinterpret_cast<const uint4 *>(c + t * cs) + lane);
        const uint16_t *k = kr + t * ks;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!in[i]) continue;
            x.k[i] = HALF ? k[lo[i]] | static_cast<uint32_t>(k[hi[i]]) << 16 : reinterpret_cast<const uint32_t *>(k)[lane + 32 * i];
            if (turns[i]) x.pos[i] = positions[static_cast<long long>(t) * r.axes + axis[i]];
        }
    };
    Token next;
    next.c = make_uint4(0, 0, 0, 0);
    next.k[0] = next.k[1] = 0;
    next.pos[0] = next.pos[1] = 0;
    int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    fetch(t, next);
    for (; t < n; t += step) {
        Token x = next;
        fetch(t + step, next);
        if (x.slot < 0) continue;
        if (x.slot >= a.n_slots) {
            if (lane == 0) raise_error(a.err, QVG_ERR_INVALID_ARG);
            continue;
        }
        bool bad = not_finite(x.c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bad = bad || (x.k[i] & 0x7F80u) == 0x7F80u || (x.k[i] & 0x7F800000u) == 0x7F800000u;
            if (!turns[i]) continue;
            const float2 cs2 = rope_cos_sin(angle[i], x.pos[i], r.mscale, false);
            const float2 y = rope_turn(__uint_as_float(x.k[i] << 16), __uint_as_float(x.k[i] & 0xFFFF0000u), cs2.x, cs2.y);
            x.k[i] = f32_to_bf16(y.x) | static_cast<uint32_t>(f32_to_bf16(y.y)) << 16;
            bad = bad || (x.k[i] & 0x7F80u) == 0x7F80u || (x.k[i] & 0x7F800000u) == 0x7F800000u;
        }
        if (__any_sync(0xFFFFFFFFu, bad)) {
            x.c = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
            x.k[0] = x.k[1] = 0x7FFF7FFFu;
        }
        if (in_c) *(reinterpret_cast<uint4 *>(a.c + x.slot * a.dc) + lane) = x.c;
        uint16_t *k = a.kr + x.slot * a.dr;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!in[i]) continue;
            if (HALF) {
                k[lo[i]] = static_cast<uint16_t>(x.k[i]);
                k[hi[i]] = static_cast<uint16_t>(x.k[i] >> 16);
            } else {
                reinterpret_cast<uint32_t *>(k)[lane + 32 * i] = x.k[i];
            }
        }
    }
}

// One warp per token: two loads and two stores a lane.  Bound by HBM.
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
    if (n > kMostTokens) return QVG_ERR_UNSUPPORTED;
    const RopeArgs r = plan ? rope_args(plan, false) : RopeArgs{};
    const uint16_t *c = static_cast<const uint16_t *>(c_bf16), *kr = static_cast<const uint16_t *>(k_rope_bf16);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int blocks = std::min(ceil_div(n, kWarps), kAppendBlocks * sm_count_current());
    if (plan && r.layout == QVG_ROPE_HALF)
        k_latent_append<true><<<blocks, kWarps * 32, 0, st>>>(r, latent_args(cache), c, kr, n, c_stride, kr_stride, slots, positions);
    else
        k_latent_append<false><<<blocks, kWarps * 32, 0, st>>>(r, latent_args(cache), c, kr, n, c_stride, kr_stride, slots, positions);
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
    if (n > kMostTokens) return QVG_ERR_UNSUPPORTED;
    k_latent_read<<<ceil_div(n, kWarps), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(
        latent_args(cache), slots, n, static_cast<uint16_t *>(c_out), static_cast<uint16_t *>(kr_out));
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

}  // extern "C"
