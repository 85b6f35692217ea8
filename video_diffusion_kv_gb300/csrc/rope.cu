// rope.cu -- rotary positions: the plan (host) and the rotation of a
// tensor's heads.
#include <cmath>

#include "rope.cuh"

namespace qvg {

bool rope_plan_ok(const qvg_rope_plan *plan, int d) {
    if (!plan || plan->dims < 2 || plan->dims % 2 != 0 || plan->dims > d || plan->dims > 2 * QVG_ROPE_MAX_PAIRS ||
        plan->axes < 1 || plan->axes > QVG_ROPE_MAX_AXES ||
        (plan->layout != QVG_ROPE_HALF && plan->layout != QVG_ROPE_INTERLEAVED) || !std::isfinite(plan->mscale))
        return false;
    for (int i = 0; i < plan->dims / 2; ++i)
        if (plan->axis[i] >= plan->axes) return false;
    return true;
}

RopeArgs rope_args(const qvg_rope_plan *plan, bool transpose) {
    RopeArgs r{};
    r.pairs = plan->dims / 2;
    for (int i = 0; i < r.pairs; ++i) {
        r.step[i] = plan->step[i];
        r.axis[i] = plan->axis[i];
    }
    r.axes = plan->axes;
    r.layout = plan->layout;
    r.mscale = plan->mscale;
    r.transpose = transpose;
    return r;
}

namespace {

// Sixteen bytes of elements <-> floats.
__device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(uint4 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

template <typename T>
__device__ __forceinline__ float load1(const T *p);
template <>
__device__ __forceinline__ float load1(const float *p) { return *p; }
template <>
__device__ __forceinline__ float load1(const uint16_t *p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = f32_to_bf16(v); }

constexpr int kWarps = 8;

// One warp per token (blockIdx.y: a share of its heads).  The warp first
// puts the token's cosines and sines into shared memory, pairs / 32 angles a
// lane: they serve every head.  Then a lane owns two 16-byte pieces that
// hold whole pairs (HALF: the same piece of both halves; INTERLEAVED: 32
// consecutive bytes) and goes through the heads.
//   VEC: pieces line up (pairs a multiple of the elements in 16 bytes, all
// rows 16-byte aligned).  Otherwise a lane owns single pairs.
// Bound by HBM: 2 n H d bytes-per-element, each read and written once.  37,440
// tokens of 16 heads of 128, bf16, three axes (0.31 GB): 56 us, 5.4 TB/s, 80 % of
// a plain copy's rate; 2,639 fp32 tokens of 24 heads (65 MB): 12 us, 80 % too (a call
// takes 13 to 20, the host's part); 64 tokens of 32 heads: 4 us.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) k_rope(const __grid_constant__ RopeArgs r, const T *x, int n, int H,
                                                     int d, long long xs, const int32_t *__restrict__ positions,
                                                     T *out, long long os, int heads_per_block) {
    constexpr int E = 16 / sizeof(T);  // elements in 16 bytes
    __shared__ float2 s_cs[kWarps][QVG_ROPE_MAX_PAIRS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= n) return;
    float2 *cs = s_cs[warp];
    const int h0 = blockIdx.y * heads_per_block, h1 = min(H, h0 + heads_per_block);
    const T *xr = x + t * xs;
    T *yr = out + t * os;
    const bool half = r.layout == QVG_ROPE_HALF;
    auto angles = [&]() {
        for (int i = lane; i < r.pairs; i += 32)
            cs[i] = rope_cos_sin(r.step[i], positions[static_cast<long long>(t) * r.axes + r.axis[i]], r.mscale, r.transpose);
        __syncwarp();
    };
    if constexpr (VEC) {
        const int units = d / (2 * E);  // lanes on one head; 32 / units heads side by side
        const int u = lane % units, step = 32 / units;
        const int rot = r.pairs / E;  // units that rotate; the others copy
        const bool turn = u < rot, live = turn || x != out;
        const int c0 = half && turn ? u * E : 2 * E * u, c1 = half && turn ? r.pairs + u * E : c0 + E;
        constexpr int AHEAD = 4;  // heads on their way at once, the first ones while the angles are made
        uint4 v0[AHEAD], v1[AHEAD];
        auto fetch = [&](int h) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (live && h + i * step < h1) {
                    const T *p = xr + static_cast<long long>(h + i * step) * d;
                    v0[i] = __ldcs(reinterpret_cast<const uint4 *>(p + c0));
                    v1[i] = __ldcs(reinterpret_cast<const uint4 *>(p + c1));
                }
        };
        int h = h0 + lane / units;
        fetch(h);
        angles();
        float2 a[E];
#pragma unroll
        for (int i = 0; i < E; ++i) a[i] = turn ? cs[u * E + i] : make_float2(1.0f, 0.0f);
        for (; h < h1; h += AHEAD * step) {
#pragma unroll
            for (int b = 0; b < AHEAD; ++b) {
                if (!live || h + b * step >= h1) break;
                if (turn) {
                    float f0[E], f1[E];
                    unpack(v0[b], f0);
                    unpack(v1[b], f1);
                    if (half) {
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            const float2 y = rope_turn(f0[i], f1[i], a[i].x, a[i].y);
                            f0[i] = y.x;
                            f1[i] = y.y;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < E / 2; ++i) {
                            const float2 e = a[E / 2 + i];
                            const float2 y0 = rope_turn(f0[2 * i], f0[2 * i + 1], a[i].x, a[i].y);
                            const float2 y1 = rope_turn(f1[2 * i], f1[2 * i + 1], e.x, e.y);
                            f0[2 * i] = y0.x;
                            f0[2 * i + 1] = y0.y;
                            f1[2 * i] = y1.x;
                            f1[2 * i + 1] = y1.y;
                        }
                    }
                    v0[b] = pack(f0);
                    v1[b] = pack(f1);
                }
                T *q = yr + static_cast<long long>(h + b * step) * d;
                *reinterpret_cast<uint4 *>(q + c0) = v0[b];
                *reinterpret_cast<uint4 *>(q + c1) = v1[b];
            }
            fetch(h + AHEAD * step);
        }
    } else {
        angles();
        for (int h = h0; h < h1; ++h) {
            const T *p = xr + static_cast<long long>(h) * d;
            T *q = yr + static_cast<long long>(h) * d;
            for (int i = lane; i < d / 2; i += 32) {
                if (i < r.pairs) {
                    const int c0 = half ? i : 2 * i, c1 = half ? r.pairs + i : 2 * i + 1;
                    const float2 y = rope_turn(load1(p + c0), load1(p + c1), cs[i].x, cs[i].y);
                    store1(q + c0, y.x);
                    store1(q + c1, y.y);
                } else if (x != out) {
                    q[2 * i] = p[2 * i];
                    q[2 * i + 1] = p[2 * i + 1];
                }
            }
        }
    }
}

template <typename T>
qvg_status launch_rope(const RopeArgs &r, const void *x, int n, int H, int d, long long xs, const int32_t *positions,
                       void *out, long long os, cudaStream_t st) {
    constexpr int E = 16 / sizeof(T);
    const bool vec = r.pairs % E == 0 && xs % E == 0 && os % E == 0 &&
                     ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    // Few tokens: their heads spread over more blocks, until the grid holds
    // about four blocks per SM; a share is at least the heads a warp takes
    // side by side.
    const int blocks = ceil_div(n, kWarps), side = std::max(1, 64 * E / d);
    int shares = std::max(1, std::min({ceil_div(H, side), 4 * sm_count_current() / blocks, 65535}));
    const int per = ceil_div(ceil_div(H, side), shares) * side;
    shares = ceil_div(H, per);
    const dim3 grid(blocks, shares);
    if (vec)
        k_rope<T, true><<<grid, kWarps * 32, 0, st>>>(r, static_cast<const T *>(x), n, H, d, xs, positions,
                                                      static_cast<T *>(out), os, per);
    else
        k_rope<T, false><<<grid, kWarps * 32, 0, st>>>(r, static_cast<const T *>(x), n, H, d, xs, positions,
                                                       static_cast<T *>(out), os, per);
    QVG_LAUNCH_CHECK();
    return QVG_OK;
}

}  // namespace
}  // namespace qvg

using namespace qvg;

extern "C" {

qvg_status qvg_rope_plan_init(qvg_rope_plan *plan, int32_t axes, const int32_t *axis_dims, int32_t layout,
                              double base, int32_t scaling, double factor, double original, double fast,
                              double slow, uint32_t scaled_axes, float mscale) {
    if (!plan || !axis_dims || axes < 1 || axes > QVG_ROPE_MAX_AXES) return QVG_ERR_INVALID_ARG;
    if ((layout != QVG_ROPE_HALF && layout != QVG_ROPE_INTERLEAVED) || scaling < QVG_ROPE_PLAIN ||
        scaling > QVG_ROPE_PARTS)
        return QVG_ERR_INVALID_ARG;
    if (!std::isfinite(base) || base < 1.0 || !std::isfinite(factor) || factor < 1.0 || !std::isfinite(mscale))
        return QVG_ERR_INVALID_ARG;
    if (scaling == QVG_ROPE_PARTS &&
        (!std::isfinite(original) || original <= 0.0 || !std::isfinite(fast) || !std::isfinite(slow) || fast <= slow))
        return QVG_ERR_INVALID_ARG;
    int64_t total = 0;
    for (int a = 0; a < axes; ++a) {
        if (axis_dims[a] < 2 || axis_dims[a] % 2 != 0) return QVG_ERR_INVALID_ARG;
        total += axis_dims[a];
    }
    if (total > 2 * QVG_ROPE_MAX_PAIRS) return QVG_ERR_INVALID_ARG;
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    qvg_rope_plan p{};
    p.dims = static_cast<int32_t>(total);
    p.axes = axes;
    p.layout = layout;
    p.mscale = mscale;
    int at = 0;
    for (int a = 0; a < axes; ++a) {
        const int n = axis_dims[a];
        const int how = (scaled_axes >> a) & 1u ? scaling : QVG_ROPE_PLAIN;
        const double b = how == QVG_ROPE_NTK && n > 2 ? base * std::pow(factor, static_cast<double>(n) / (n - 2)) : base;
        for (int i = 0; i < n / 2; ++i, ++at) {
            double f = std::pow(b, -2.0 * i / n);
            if (how == QVG_ROPE_LINEAR) f /= factor;
            if (how == QVG_ROPE_PARTS) {
                const double turns = original * f / kTwoPi;
                const double keep = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
                f = f * keep + f / factor * (1.0 - keep);
            }
            // turns per position, at most 1 / 2 pi: the product stays below 2^62
            p.step[at] = static_cast<uint64_t>(std::ldexp(f / kTwoPi, 64) + 0.5);
            p.axis[at] = static_cast<uint8_t>(a);
        }
    }
    *plan = p;
    return QVG_OK;
}

qvg_status qvg_rope(const qvg_rope_plan *plan, const void *x, int32_t dtype, int32_t n, int32_t H, int32_t d,
                    int64_t x_stride, const int32_t *positions, int32_t transpose, void *out, int64_t out_stride,
                    void *stream) {
    if (dtype != QVG_OUT_F32 && dtype != QVG_OUT_BF16) return QVG_ERR_INVALID_ARG;
    if (n < 0 || H < 1 || (transpose != 0 && transpose != 1)) return QVG_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return QVG_ERR_UNSUPPORTED;
    if (!rope_plan_ok(plan, d)) return QVG_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(H) * d;
    if (x_stride < row || out_stride < row) return QVG_ERR_INVALID_ARG;
    if (n == 0) return QVG_OK;
    const uintptr_t el = dtype == QVG_OUT_F32 ? 4 : 2;
    if (!x || !out || !positions || reinterpret_cast<uintptr_t>(x) % el != 0 ||
        reinterpret_cast<uintptr_t>(out) % el != 0 || reinterpret_cast<uintptr_t>(positions) % 4 != 0)
        return QVG_ERR_INVALID_ARG;
    if (x == out && x_stride != out_stride) return QVG_ERR_INVALID_ARG;
    const RopeArgs r = rope_args(plan, transpose != 0);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == QVG_OUT_F32 ? launch_rope<float>(r, x, n, H, d, x_stride, positions, out, out_stride, st)
                                : launch_rope<uint16_t>(r, x, n, H, d, x_stride, positions, out, out_stride, st);
}

}  // extern "C"
