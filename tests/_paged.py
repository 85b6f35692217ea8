"""Plain 64-bit forms of the token-wise operators (numpy), for their tests:
rotary positions, the paged cache's formats, attention over pages."""
import math

import numpy as np
import torch

MAGS = {
    8: np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:-1]),
    4: np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]),
}
TOP = {8: 448.0, 4: 6.0}


def bf16(a):
    """Values rounded to bf16 (nearest even), as float64."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).double().numpy()


# ---- rotary positions ------------------------------------------------------------

def frequencies(axis_dims, base=10000.0, scaling="plain", factor=1.0, original=1.0, fast=32.0, slow=1.0, scaled=None):
    f, axis = [], []
    for a, n in enumerate(axis_dims):
        how = scaling if scaled is None or a in scaled else "plain"
        b = base * factor ** (n / (n - 2)) if how == "ntk" and n > 2 else base
        for i in range(n // 2):
            w = b ** (-2.0 * i / n)
            if how == "linear":
                w /= factor
            if how == "parts":
                k = min(1.0, max(0.0, (original * w / (2 * math.pi) - slow) / (fast - slow)))
                w *= k + (1 - k) / factor
            f.append(w)
            axis.append(a)
    return np.array(f), np.array(axis)


def rope(x, positions, f, axis, layout, mscale=1.0, transpose=False):
    """x [n][H][d] float64; positions [n][axes]."""
    m = len(f)
    ang = positions[:, axis].astype(np.float64) * f * (-1 if transpose else 1)
    c, s = mscale * np.cos(ang)[:, None], mscale * np.sin(ang)[:, None]
    y = x.copy()
    ia = np.arange(m) if layout == 0 else 2 * np.arange(m)
    ib = ia + m if layout == 0 else ia + 1
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


# ---- the cache's formats -----------------------------------------------------------

def quantise(x, bits):
    """x [..., d] float64 -> (values of the codes, scale bytes), groups of d (8
    bits) or 32 (4 bits).  A row with an infinity or a NaN: 0 and 255."""
    d = x.shape[-1]
    g = x.reshape(*x.shape[:-1], 1 if bits == 8 else d // 32, -1)
    bad = np.broadcast_to(~np.isfinite(g).all(-1).all(-1, keepdims=True), g.shape[:-1])
    g = np.where(bad[..., None], 0.0, g)
    top = np.abs(g).max(-1)
    m, e = np.frexp(top / TOP[bits])  # top / TOP = m 2^e with m in [0.5, 1): the smallest power of two above is 2^e, or 2^(e-1) at m = 0.5
    e = np.where(m == 0.5, e - 1, e)
    e = np.where(top == 0, -126, np.clip(e, -126, 127))
    y = np.ldexp(g, -e[..., None])
    mags = MAGS[bits]
    at = np.clip(np.searchsorted(mags, np.abs(y)), 1, len(mags) - 1)
    lo, hi = mags[at - 1], mags[at]
    up, down = hi - np.abs(y), np.abs(y) - lo
    r = np.where((down > up) | ((down == up) & (at % 2 == 0)), hi, lo)
    # codes stand for finite values: under the largest scale the last one is
    # the largest below 2^128
    last = mags[mags * np.exp2(float(120 if bits == 8 else 126)) < 2.0 ** 128].max()
    r = np.where(e[..., None] == (120 if bits == 8 else 126), np.minimum(r, last), r) * np.sign(y)
    return r.reshape(x.shape), np.where(bad, 255, e + 127).astype(np.uint8)


def code_values(codes, bits):
    """Values of code bytes [..., d bits / 8]."""
    if bits == 8:
        mags = np.append(MAGS[8], np.nan)
        return np.where(codes & 128, -1.0, 1.0) * mags[codes & 127]
    nib = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    return np.where(nib & 8, -1.0, 1.0) * MAGS[4][nib & 7]


def dequantise(values, scales):
    """values [..., d] of codes, scale bytes [..., groups] -> float64."""
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return (values.reshape(*scales.shape, values.shape[-1] // scales.shape[-1]) * s[..., None]).reshape(values.shape)


def held(cache):
    """(K, V) float64 [pages][H][page][d] that a PagedKV holds."""
    out = []
    for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        out.append(dequantise(code_values(c.cpu().numpy(), cache.bits), s.cpu().numpy()))
    return out


# ---- attention -----------------------------------------------------------------------

def attention(q, k, v, see, scale=None):
    """q [T][Hq][d], k, v [L][H][d] float64, see [T][L] bool -> (out [T][Hq][d],
    lse [Hq][T]); keys that a row does not see do not enter at all."""
    T, Hq, d = q.shape
    g = Hq // k.shape[1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, lse = np.zeros((T, Hq, d)), np.full((Hq, T), -np.inf)
    for t in range(T):
        js = np.nonzero(see[t])[0]
        if len(js) == 0:
            continue
        for h in range(Hq):
            with np.errstate(invalid="ignore"):
                s = (k[js, h // g] @ q[t, h]) * scale
                m = s.max()
                p = np.exp(s - m)
                out[t, h] = p @ v[js, h // g] / p.sum()
                lse[h, t] = m + np.log(p.sum())
    return out, lse


def tree_rows(parents):
    """[T][T] bool: token j is token t or an ancestor of it."""
    T = len(parents)
    m = np.zeros((T, T), bool)
    for t in range(T):
        if parents[t] >= 0:
            m[t] = m[parents[t]]
        m[t, t] = True
    return m
