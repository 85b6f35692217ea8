"""Measured calls of the token-wise operators: rotary positions, the paged
8-bit / 4-bit token cache (written as tokens arrive, read back) and attention
of a few new tokens (one, a drafted tree, a short chunk) over its pages.

Each case is one call, or one run of calls, as a program that serves an
autoregressive video model makes it.  Head counts, head sizes and token grids
are those of the workloads in video_diffusion_kv_gb300/synth.py (16 heads of
128 with chunks of 3 frames of 30 x 52 tokens; 24 heads with frames of 22 x 40;
8 heads and 288 frames; 2 heads of 64), or generic grouped-query shapes.

`run` has two sides that take the same state: elementary torch operations in
32 bits (angles in 64), and, with `own`, the calls of the package.

Formats of the token cache (the same bytes on both sides):
  codes   uint8 [pages][H][page][d bits / 8]; 8 bits: the fp8 number e4m3,
          4 bits: the fp4 number e2m1, channel 2i in the low half of byte i.
  scales  uint8 [pages][H][page][1 or d / 32]: a power of two, 2^(byte - 127),
          the smallest for which no value of the group exceeds the format's
          largest (448; 6).  The group is the head's row (8 bits) or 32
          channels of it (4 bits).
"""
import math
import random

import torch

own = False

DEV = "cuda"
TOP = {8: 448.0, 4: 6.0}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of e2m1
LOG2E = 1.4426950408889634


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # 64 drafted tokens' queries at far positions: a launch-latency call between two layers
        rope_case("rope_step", n=64, H=32, d=128, axes="128", layout="half", scaling="parts", factor=8.0, far=300000),
        # a whole 24-frame clip's queries, rotated by frame, row and column
        rope_case("rope_clip", n=37440, H=16, d=128, axes="44,42,42", layout="interleaved", far=24),
        # the gradient of a training step's fp32 queries, half of each head rotated, odd token count
        rope_case("rope_grad", n=2639, H=24, d=128, axes="64", layout="half", dtype="f32", transpose=True, scaling="linear",
                  factor=4.0, far=40000),
        # 48 drafted tokens' keys (rotated on the way) and values into the 8-bit cache
        append_case("append_step", n=48, H=8, d=128, bits=8, page=64, axes="128", far=100000),
        # a clip's keys and values into the 4-bit cache, and back as bf16
        append_case("append_read_4bit", n=37440, H=16, d=128, bits=4, page=128, axes="44,42,42", far=24, back=True),
        # the 8-bit cache of a clip read back, pages in any order
        read_case("read_clip", n=37440, H=16, d=128, bits=8, page=128),
        # one token over a short history of the tiny model: latency
        attn_case("attn_token_tiny", B=1, H=2, G=1, d=64, bits=8, page=32, q=(1, 1), kv=(1000, 1000)),
        # one token over a one-minute rollout (288 frames of 30 x 52)
        attn_case("attn_token_long", B=1, H=8, G=4, d=128, bits=8, page=128, q=(1, 1), kv=(449280, 449280)),
        # a decode batch of ragged histories
        attn_case("attn_token_batch", B=48, H=8, G=8, d=128, bits=8, page=16, q=(1, 1), kv=(700, 24000)),
        # drafted trees of 17 to 48 tokens, verified in one call
        attn_case("attn_tree", B=16, H=8, G=4, d=128, bits=8, page=64, q=(17, 48), kv=(2000, 12000), mask="tree"),
        # small trees over the 4-bit cache, one KV head per query head
        attn_case("attn_tree_4bit", B=24, H=16, G=1, d=128, bits=4, page=32, q=(5, 13), kv=(4000, 16000), mask="tree"),
        # the tokens of one 22 x 40 frame over 24 frames of history, causal
        attn_case("attn_frame", B=1, H=24, G=1, d=128, bits=8, page=128, q=(880, 880), kv=(21120, 21120)),
    ]


def rope_case(name, n, H, d, axes, layout, far, dtype="bf16", transpose=False, scaling="none", factor=1.0):
    return {"name": name, "op": "rope", "n": n, "H": H, "d": d, "axes": axes, "layout": layout, "far": far,
            "dtype": dtype, "transpose": transpose, "scaling": scaling, "factor": factor}


def append_case(name, n, H, d, bits, page, axes, far, back=False):
    return {"name": name, "op": "append", "n": n, "H": H, "d": d, "bits": bits, "page": page, "axes": axes,
            "layout": "half", "far": far, "scaling": "none", "factor": 1.0, "back": back}


def read_case(name, n, H, d, bits, page):
    return {"name": name, "op": "read", "n": n, "H": H, "d": d, "bits": bits, "page": page}


def attn_case(name, B, H, G, d, bits, page, q, kv, mask="causal"):
    return {"name": name, "op": "attn", "B": B, "H": H, "G": G, "d": d, "bits": bits, "page": page,
            "q_lo": q[0], "q_hi": q[1], "kv_lo": kv[0], "kv_hi": kv[1], "mask": mask}


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "read", "attn", "attn", "attn"))
    d = rng.choice((64, 128, 128))
    if op in ("rope", "append"):
        axes = rng.choice(("%d" % d, "%d" % (d // 2), "44,42,42" if d == 128 else "24,20,20", "32,32"))
        far = rng.choice((24, 5000, 300000))
        n = spread(rng, 1, 37440)
        H = rng.choice((1, 2, 5, 8, 16))
    if op == "rope":
        c = rope_case("", n, H, d, axes, rng.choice(("half", "interleaved")), far, rng.choice(("bf16", "f32")),
                      rng.random() < 0.5)
        c["scaling"] = rng.choice(("none", "linear", "ntk", "parts"))
        c["factor"] = 1.0 if c["scaling"] == "none" else rng.choice((2.0, 5.5, 16.0))
    elif op == "append":
        bits = rng.choice((8, 4))
        c = append_case("", n, H, d, bits, rng.choice((16, 32, 64, 128, 256)), axes, far, bits == 4)
    elif op == "read":
        c = read_case("", spread(rng, 1, 37440), rng.choice((1, 2, 5, 8, 16)), d, rng.choice((8, 4)), rng.choice((16, 32, 64, 128, 256)))
    else:
        B, H, G = spread(rng, 1, 40), rng.choice((1, 2, 3, 8)), rng.choice((1, 2, 4, 7, 8))
        q_hi = spread(rng, 1, 64)
        most = min(200000, 4000000 // (B * H), 120000000 // (B * H * G * q_hi))  # keeps a pass under the largest listed one
        kv_hi = spread(rng, max(q_hi, min(300, most)), max(q_hi, most))
        c = attn_case("", B, H, G, d, rng.choice((8, 4)), rng.choice((16, 32, 64, 128, 256)), (max(1, q_hi // 3), q_hi),
                      (max(q_hi, kv_hi // 8), kv_hi), rng.choice(("causal", "tree")))
    del c["name"]
    return c


def ragged(lo, hi, count, odd):
    """`count` lengths between lo and hi, both ends among them, in a fixed mixed order."""
    rng = random.Random(1000 * count + odd)
    got = [hi] if count == 1 else [lo + (hi - lo) * i // (count - 1) for i in range(count)]
    rng.shuffle(got)
    return got


def work(c):
    if c["op"] == "rope":
        el = c["n"] * c["H"] * c["d"]
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2 * el * size + 4 * c["n"] * len(dims_of(c)), "flops": 3 * c["n"] * c["H"] * sum(dims_of(c))}
    if c["op"] in ("append", "read"):
        rows = c["n"] * c["H"]
        held = 2 * rows * (c["d"] * c["bits"] // 8 + groups(c))
        plain = 2 * rows * c["d"] * 2
        if c["op"] == "read":
            return {"bytes": held + plain + 8 * c["n"], "flops": 2 * rows * c["d"]}
        got = {"bytes": held + plain + 8 * c["n"] + 4 * c["n"] * len(dims_of(c)), "flops": 2 * rows * c["d"] * 3}
        if c["back"]:
            got = {"bytes": got["bytes"] + held + plain + 8 * c["n"], "flops": got["flops"] + 2 * rows * c["d"]}
        return got
    nq, kv = ragged(c["q_lo"], c["q_hi"], c["B"], 1), ragged(c["kv_lo"], c["kv_hi"], c["B"], 2)
    pairs = sum(a * b for a, b in zip(nq, kv)) * c["H"] * c["G"]
    rows = sum(nq) * c["H"] * c["G"]
    held = 2 * sum(kv) * c["H"] * (c["d"] * c["bits"] // 8 + groups(c))
    table = 4 * sum(-(-x // c["page"]) for x in kv)
    return {"bytes": held + table + rows * (4 * c["d"] + 4), "flops": 4 * pairs * c["d"]}


def dims_of(c):
    return [int(x) for x in c["axes"].split(",")]


def groups(c):
    return 1 if c["bits"] == 8 else c["d"] // 32


# ---- rotary plan ---------------------------------------------------------------------

BASE, ORIGINAL, FAST, SLOW = 10000.0, 4096.0, 32.0, 1.0


def mscale_of(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "parts" else 1.0


def frequencies(c):
    """Radians a position adds to each pair, axis by axis."""
    got = []
    for n in dims_of(c):
        for i in range(n // 2):
            base = BASE
            if c["scaling"] == "ntk" and n > 2:
                base = BASE * c["factor"] ** (n / (n - 2))
            f = base ** (-2.0 * i / n)
            if c["scaling"] == "linear":
                f /= c["factor"]
            if c["scaling"] == "parts":
                turns = ORIGINAL * f / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - SLOW) / (FAST - SLOW)))
                f = f * keep + f / c["factor"] * (1 - keep)
            got.append(f)
    return got


def axis_of_pair(c):
    return [a for a, n in enumerate(dims_of(c)) for _ in range(n // 2)]


def rope_state(c, g):
    axes = len(dims_of(c))
    if axes == 3:  # frame, row and column of a 30 x 52 grid
        t = torch.arange(c["n"], device=DEV)
        pos = torch.stack((t // 1560 + int(torch.randint(0, c["far"], (1,), generator=g, device=DEV)), t % 1560 // 52, t % 52), 1)
    else:
        first = torch.randint(0, c["far"], (1, axes), generator=g, device=DEV)
        pos = first + torch.arange(c["n"], device=DEV)[:, None]
    s = {"positions": pos.to(torch.int32).contiguous(), "freq": torch.tensor(frequencies(c), dtype=torch.float64, device=DEV),
         "axis": torch.tensor(axis_of_pair(c), device=DEV), "mscale": mscale_of(c), "layout": c["layout"]}
    if own:
        import video_diffusion_kv_gb300 as qvg
        s["plan"] = qvg.RopePlan(dims_of(c), layout=qvg.QVG_ROPE_HALF if c["layout"] == "half" else qvg.QVG_ROPE_INTERLEAVED, base=BASE,
                                 scaling={"none": qvg.QVG_ROPE_PLAIN, "linear": qvg.QVG_ROPE_LINEAR, "ntk": qvg.QVG_ROPE_NTK,
                                          "parts": qvg.QVG_ROPE_PARTS}[c["scaling"]],
                                 factor=c["factor"], original=ORIGINAL, fast=FAST, slow=SLOW, mscale=mscale_of(c))
    return s


def rotated(x, s, transpose=False):
    """x [n][H][d] with its first channels rotated, in 32 bits (angles in 64)."""
    angle = s["positions"].double()[:, s["axis"]] * s["freq"]
    cos, sin = ((f(angle) * s["mscale"]).float()[:, None] for f in (torch.cos, torch.sin))
    sin = -sin if transpose else sin
    m, x = s["freq"].numel(), x.float()
    y = x.clone()
    if s["layout"] == "half":
        a, b = x[..., :m], x[..., m:2 * m]
        y[..., :m], y[..., m:2 * m] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:2 * m:2], x[..., 1:2 * m:2]
        y[..., 0:2 * m:2], y[..., 1:2 * m:2] = a * cos - b * sin, b * cos + a * sin
    return y


# ---- the cache's formats, plain ------------------------------------------------------

def quantised(x, bits):
    """(codes uint8, scale bytes uint8) of x [..., d] in 32 bits."""
    d = x.shape[-1]
    grp = x.float().reshape(*x.shape[:-1], 1 if bits == 8 else d // 32, -1)
    frac, e = torch.frexp(grp.abs().amax(-1))
    e = (e - (9 if bits == 8 else 3) + (frac > (0.875 if bits == 8 else 0.75))).clamp(-126, 127)
    e = torch.where(frac == 0, torch.full_like(e, -126), e)
    y = torch.ldexp(grp, -e[..., None]).reshape(x.shape)
    if bits == 8:
        codes = y.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        m = y.abs()
        up = (m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)
        nib = (up + 8 * torch.signbit(y)).to(torch.uint8)
        codes = nib[..., 0::2] | (nib[..., 1::2] << 4)
    return codes, (e + 127).to(torch.uint8)


def values(codes, scales, bits):
    """What codes [..., d bits / 8] and scales [..., groups] stand for, in 32 bits."""
    if bits == 8:
        y = codes.view(torch.float8_e4m3fn).float()
    else:
        nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
        level = torch.tensor(LEVELS, device=codes.device)
        y = torch.where(nib >= 8, -level[nib & 7], level[nib & 7])
    s = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    return (y.reshape(*scales.shape, -1) * s[..., None]).reshape(y.shape)


def rows_of(slots, H, page):
    """Index (page, head, offset) of each (token, head) row."""
    return (slots // page)[:, None], torch.arange(H, device=slots.device)[None], (slots % page)[:, None]


# ---- inputs --------------------------------------------------------------------------

def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def keys_values(n, H, d, g):
    """bf16 K and V rows with a few channels that stand out, as video models' have."""
    def one(by):
        ch = torch.where(torch.rand(H, d, generator=g, device=DEV) < 0.02, by, 1.0)
        return (torch.randn(n, H, d, generator=g, device=DEV) * ch).bfloat16()
    return one(8.0), one(10.0)


def empty_pages(c, pages):
    shape = (pages, c["H"], c["page"])
    one = lambda last: torch.zeros(*shape, last, dtype=torch.uint8, device=DEV)  # noqa: E731
    nb = c["d"] * c["bits"] // 8
    return [one(nb), one(groups(c)), one(nb), one(groups(c))]


def handle(c, buffers):
    import video_diffusion_kv_gb300 as qvg
    return qvg.PagedKV(c["H"], c["d"], c["page"], buffers[0].shape[0], bits=c["bits"], buffers=buffers)


def prepare(c, seed):
    g = gen(seed)
    if c["op"] == "rope":
        s = rope_state(c, g)
        x = torch.randn(c["n"], c["H"], c["d"], generator=g, device=DEV)
        s.update(x=x.bfloat16() if c["dtype"] == "bf16" else x)
        return {"case": c, **s}
    if c["op"] in ("append", "read"):
        pages = -(-c["n"] // c["page"]) + 2
        order = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(c["n"], device=DEV) + c["page"] // 3  # the first page is already partly filled
        slots = order[t // c["page"]] * c["page"] + t % c["page"]
        buffers = empty_pages(c, pages)
        s = {"case": c, "slots": slots, "buffers": buffers}
        if c["op"] == "append":  # keys and values as a fused projection leaves them: rows of one wider tensor
            both = torch.stack(keys_values(c["n"], c["H"], c["d"], g), 1)
            s.update(rope_state(c, g), k=both[:, 0], v=both[:, 1])
        else:
            kv = torch.stack(keys_values(pages * c["page"], c["H"], c["d"], g))
            codes, scales = quantised(kv, c["bits"])
            for i, x in enumerate((codes[0], scales[0], codes[1], scales[1])):
                buffers[i].copy_(x.view(pages, c["page"], c["H"], -1).transpose(1, 2))
        if own:
            s["cache"] = handle(c, buffers)
        return s
    B, H, d, page = c["B"], c["H"], c["d"], c["page"]
    nq, kv = ragged(c["q_lo"], c["q_hi"], B, 1), ragged(c["kv_lo"], c["kv_hi"], B, 2)
    need = [-(-x // page) for x in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.zeros(B, max(need), dtype=torch.int32, device=DEV)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    buffers = empty_pages(c, pages)
    for p in range(0, pages, max(1, 400000 // page)):  # a part at a time: the fp32 rows take four times the cache
        m = min(max(1, 400000 // page), pages - p)
        k, v = keys_values(m * page, H, d, g)
        for i, x in ((0, k), (2, v)):
            for j, y in enumerate(quantised(x, c["bits"])):
                buffers[i + j][p:p + m] = y.view(m, page, H, -1).transpose(1, 2)
    total, first = sum(nq), [sum(nq[:b]) for b in range(B)]
    s = {"case": c, "buffers": buffers, "table": table, "q": torch.randn(total, H * c["G"], d, generator=g, device=DEV).bfloat16(),
         "kv_len": torch.tensor(kv, dtype=torch.int32, device=DEV),
         "cu_q": torch.tensor(first + [total], dtype=torch.int32, device=DEV)}
    if c["mask"] == "tree":  # every drafted token hangs on an earlier one or on the history (-1)
        r = random.Random(seed)
        s["parents"] = torch.tensor([r.randrange(max(-1, t - 6), t) for m in nq for t in range(m)], dtype=torch.int32, device=DEV)
    if own:
        s["cache"] = handle(c, buffers)
    return s


# ---- one pass ------------------------------------------------------------------------

def run(s):
    return (own_calls if own else plain)(s)


def own_calls(s):
    import video_diffusion_kv_gb300 as qvg
    c = s["case"]
    if c["op"] == "rope":
        return qvg.rope(s["plan"], s["x"], s["positions"], transpose=c["transpose"])
    if c["op"] == "read":
        return qvg.paged_read(s["cache"], s["slots"])
    if c["op"] == "append":
        qvg.paged_append(s["cache"], s["k"], s["v"], s["slots"], plan=s["plan"], positions=s["positions"])
        return qvg.paged_read(s["cache"], s["slots"]) if c["back"] else held(s)
    mask = qvg.tree_mask(s["parents"], c["q_hi"], cu_q=s["cu_q"]) if c["mask"] == "tree" else None
    return qvg.paged_attention(s["cache"], s["q"], s["table"], s["kv_len"], c["q_hi"], cu_q=s["cu_q"], mask=mask,
                               mask_mode=qvg.QVG_MASK_TREE if c["mask"] == "tree" else qvg.QVG_MASK_CAUSAL, want_lse=True)


def held(s):
    """The 8-bit cache's state: codes as the fp8 numbers they are, scale bytes."""
    k, ks, v, vs = s["buffers"]
    return k.view(torch.float8_e4m3fn), ks, v.view(torch.float8_e4m3fn), vs


def plain(s):
    c = s["case"]
    if c["op"] == "rope":
        return rotated(s["x"], s, c["transpose"]).to(s["x"].dtype)
    if c["op"] == "attn":
        return plain_attention(s)
    at = rows_of(s["slots"], c["H"], c["page"])
    k, ks, v, vs = s["buffers"]
    if c["op"] == "append":
        k[at], ks[at] = quantised(rotated(s["k"], s).bfloat16(), c["bits"])
        v[at], vs[at] = quantised(s["v"], c["bits"])
        if not c["back"]:
            return held(s)
    return values(k[at], ks[at], c["bits"]).bfloat16(), values(v[at], vs[at], c["bits"]).bfloat16()


def ancestors(parents, cu, b, t, B, n):
    """[B][n][n]: whether token j is token t or one of its ancestors."""
    up = torch.zeros(B, n, n, device=DEV)
    has = parents >= 0
    up[b[has], t[has], parents[has].long()] = 1
    eye = torch.eye(n, device=DEV).expand(B, n, n)
    return torch.linalg.solve_triangular(eye - up, eye, upper=False, unitriangular=True) > 0.5


def plain_attention(s):
    c, cu, table = s["case"], s["cu_q"].long(), s["table"].long()
    B, H, G, d, n = c["B"], c["H"], c["G"], c["d"], c["q_hi"]
    row = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(cu, row, right=True) - 1
    t = row - cu[b]
    q = torch.zeros(B, n, H, G, d, device=DEV)
    q[b, t] = s["q"].float().view(-1, H, G, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(B, H, G * n, d)

    def all_rows(codes, scales):
        x = values(codes[table], scales[table], c["bits"])  # [B][pages][H][page][d]
        return x.transpose(1, 2).reshape(B, H, -1, d)

    k = all_rows(*s["buffers"][:2])
    key = torch.arange(k.shape[2], device=DEV)
    nq, kv = cu[1:] - cu[:-1], s["kv_len"].long()
    j = key[None] - (kv - nq)[:, None]  # key's number among the new tokens; below 0: history
    if c["mask"] == "tree":
        seen = ancestors(s["parents"], cu, b, t, B, n)
        inside = j.clamp(0, n - 1)[:, None].expand(B, n, -1)
        see = torch.where(j[:, None] < 0, True, seen.gather(2, inside))
    else:
        see = j[:, None] <= torch.arange(n, device=DEV)[None, :, None]
    see = see & (key[None] < kv[:, None])[:, None]
    x = q @ k.transpose(-1, -2) / math.sqrt(d)
    del k
    x = x.view(B, H, G, n, -1).masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    den = p.sum(-1)
    o = p.view(B, H, G * n, -1) @ all_rows(*s["buffers"][2:])
    o = o.view(B, H, G, n, d) / torch.where(den == 0, 1.0, den)[..., None]
    lse = den.log() + m[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4)[b, t], lse.permute(0, 3, 1, 2)[b, t]
    return o.reshape(-1, H * G, d).bfloat16(), lse.reshape(-1, H * G).t().contiguous()


# ---- 64 bits -------------------------------------------------------------------------

def exact_rope(x, s, c, sign):
    x = x.double()
    pair = torch.arange(s["freq"].numel(), device=DEV)
    lo, hi = (pair, pair + len(pair)) if c["layout"] == "half" else (2 * pair, 2 * pair + 1)
    z = torch.complex(x[..., lo], x[..., hi])
    turn = sign * s["positions"].double()[:, s["axis"]] * s["freq"]
    z = z * torch.polar(torch.full_like(turn, s["mscale"]), turn)[:, None]
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def exact_values(x, bits):
    """(what the cache holds for x in 64 bits, codes' values, scale exponents), by search among the format's numbers."""
    if bits == 8:
        mags = sorted({(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)} - {480.0})
    else:
        mags = list(LEVELS)
    mags = torch.tensor(mags, dtype=torch.float64, device=DEV)
    g = x.double().reshape(*x.shape[:-1], 1 if bits == 8 else x.shape[-1] // 32, -1)
    top = g.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top == 0, 1e-300, top) / TOP[bits])).clamp(-126, 127)
    e = torch.where(top > TOP[bits] * torch.exp2(e), e + 1, torch.where(top <= TOP[bits] * torch.exp2(e - 1), e - 1, e)).clamp(-126, 127)
    y = g * torch.exp2(-e)
    at = torch.searchsorted(mags, y.abs().contiguous()).clamp(1, len(mags) - 1)
    a, b = mags[at - 1], mags[at]
    upper = (y.abs() - a > b - y.abs()) | ((y.abs() - a == b - y.abs()) & (at % 2 == 0))  # a tie goes to the even code
    r = torch.where(upper, b, a) * torch.sign(y)
    return (r * torch.exp2(e)).reshape(x.shape), r.reshape(x.shape), e[..., 0]


def exact_dequant(codes, scales, bits):
    """What the bytes stand for in 64 bits, from a table of all codes."""
    if bits == 8:
        table = torch.tensor([(-1.0 if v & 128 else 1.0) * ((v & 7) / 8 + (1 if v & 120 else 0)) * 2.0 ** (max(v >> 3 & 15, 1) - 7)
                              for v in range(256)], dtype=torch.float64, device=DEV)[:, None]
    else:
        one = [(-1.0 if v & 8 else 1.0) * LEVELS[v & 7] for v in range(16)]
        table = torch.tensor([[one[v & 15], one[v >> 4]] for v in range(256)], dtype=torch.float64, device=DEV)
    y = table[codes.long()].flatten(-2)
    s = torch.exp2(scales.double() - 127)
    return (y.reshape(*scales.shape, -1) * s[..., None]).reshape(y.shape)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return exact_rope(s["x"], s, c, -1 if c["transpose"] else 1)
    if c["op"] == "attn":
        return exact_attention(s, c)
    at = rows_of(s["slots"], c["H"], c["page"])
    if c["op"] == "read":
        return tuple(exact_dequant(s["buffers"][i][at], s["buffers"][i + 1][at], c["bits"]) for i in (0, 2))
    k = exact_rope(s["k"], s, c, 1).bfloat16()
    (kx, kr, ke), (vx, vr, ve) = exact_values(k, c["bits"]), exact_values(s["v"], c["bits"])
    if c["back"]:
        return kx, vx
    out = [torch.zeros(*b.shape, dtype=torch.float64, device=DEV) for b in s["buffers"]]
    out[0][at], out[2][at] = kr, vr
    return out[0], None, out[2], None


def exact_attention(s, c):
    H, G, d = c["H"], c["G"], c["d"]
    nq, kv = ragged(c["q_lo"], c["q_hi"], c["B"], 1), ragged(c["kv_lo"], c["kv_hi"], c["B"], 2)
    outs, lses, first = [], [], 0
    for b in range(c["B"]):
        pages = s["table"][b, :-(-kv[b] // c["page"])].long()
        rows = [exact_dequant(s["buffers"][i][pages], s["buffers"][i + 1][pages], c["bits"]).transpose(0, 1).reshape(H, -1, d)[:, :kv[b]] for i in (0, 2)]
        see = torch.ones(nq[b], kv[b], dtype=torch.bool, device=DEV)
        new = torch.zeros(nq[b], nq[b], dtype=torch.bool)
        up = s["parents"][first:first + nq[b]].tolist() if c["mask"] == "tree" else list(range(-1, nq[b] - 1))
        for t in range(nq[b]):
            if up[t] >= 0:
                new[t] = new[up[t]]
            new[t, t] = True
        see[:, kv[b] - nq[b]:] = new.to(DEV)
        q = s["q"][first:first + nq[b]].double().view(-1, H, G, d)
        out, lse = torch.empty(nq[b], H, G, d, dtype=torch.float64, device=DEV), torch.empty(H, G, nq[b], dtype=torch.float64, device=DEV)
        for h in range(H):
            x = torch.einsum("tgd,kd->gtk", q[:, h], rows[0][h]) / math.sqrt(d)
            x = x.masked_fill(~see, -math.inf)
            lse[h] = torch.logsumexp(x, -1)
            out[:, h] = torch.einsum("gtk,kd->tgd", torch.softmax(x, -1), rows[1][h])
        outs.append(out.view(-1, H * G, d))
        lses.append(lse.view(H * G, -1))
        first += nq[b]
    return torch.cat(outs), torch.cat(lses, 1)
