"""Measured calls of the latent token cache and of the pages' bookkeeping: a
paged cache of one latent vector a token (written as tokens arrive), attention
over it in the absorbed form (new tokens' queries against the latents), the
expanded form for prompts (keys and values projected per head, one rotated key
part shared by the heads), sequences that fork, grow and are freed by page
with copies on write, and the compaction of kept tokens.

Each case is one call, or one run of calls, as a program that serves an
autoregressive model makes it.  Head counts, token grids, batches and history
lengths are those of the workloads in video_diffusion_kv_gb300/synth.py (16
heads, chunks of 3 frames of 30 x 52 tokens, clips of 24 frames, rollouts of
288), or generic shapes; latents of 64 to 256 channels.

`run` has two sides that take the same state: elementary torch operations in
32 bits (angles in 64), and, with `own`, the calls of the package.

The latent cache: c bf16 [pages][page][dc], kr bf16 [pages][page][dr]; slot s
is token s % page of page s / page.  A pool counts how many sequences hold
each page (refs int32 [pages], 0: free).
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # 48 new tokens' latents, the shared key rotated on the way: a launch-latency call between two layers
        append_case("latent_append_step", n=48, dc=256, dr=64, page=64, axes="64", layout="half", far=100000),
        # a whole 24-frame clip's latents, rotated by frame, row and column
        append_case("latent_append_clip", n=37440, dc=256, dr=64, page=128, axes="24,20,20", layout="interleaved", far=24),
        # one token over a short history: latency
        attn_case("latent_token_short", B=1, Hq=16, dc=128, dr=32, page=32, q=(1, 1), kv=(1000, 1000)),
        # one token over a one-minute rollout (288 frames of 30 x 52)
        attn_case("latent_token_long", B=1, Hq=16, dc=256, dr=64, page=128, q=(1, 1), kv=(449280, 449280)),
        # a decode batch of ragged histories
        attn_case("latent_token_batch", B=48, Hq=32, dc=256, dr=64, page=64, q=(1, 1), kv=(700, 24000)),
        # drafted trees of 17 to 48 tokens, verified in one call, small pages
        attn_case("latent_tree", B=16, Hq=16, dc=256, dr=64, page=16, q=(17, 48), kv=(2000, 12000), mask="tree"),
        # the tokens of a three-frame chunk as one prompt
        expand_case("expanded_prompt", B=1, H=16, dn=128, dr=64, dv=128, q=(4680, 4680), past=(0, 0)),
        # a batch of ragged prompts, one of them a single token, after a cached part
        expand_case("expanded_ragged", B=12, H=8, dn=64, dr=32, dv=64, q=(1, 1100), past=(0, 1700)),
        # a beam of 4 for each of 6 sequences: freed, forked anew, one more token each, the shared last pages copied
        fork_case("pages_beam", kind="kv", P=6, F=3, page=64, H=8, d=128, bits=8, kv=(300, 2400), new=(1, 1)),
        # 64 long histories, each continued in three ways by a drafted run
        fork_case("pages_fork_batch", kind="latent", P=64, F=3, page=32, H=1, d=256, bits=16, kv=(2000, 24000), new=(5, 48)),
        # drafted trees written to the cache, then the accepted tokens moved together
        compact_case("compact_tree", kind="latent", B=32, page=16, H=1, d=256, bits=16, kv=(500, 3000), tree=(17, 48), share=0.3),
        # histories copied to pages of their own, from which two tokens in five are dropped
        compact_case("compact_evict", kind="kv", B=8, page=128, H=8, d=128, bits=8, kv=(5000, 20000), tree=(0, 0), share=0.6),
    ]


def append_case(name, n, dc, dr, page, axes, layout, far):
    return {"name": name, "op": "append", "n": n, "dc": dc, "dr": dr, "page": page, "axes": axes, "layout": layout, "far": far}


def attn_case(name, B, Hq, dc, dr, page, q, kv, mask="causal"):
    return {"name": name, "op": "attn", "B": B, "Hq": Hq, "dc": dc, "dr": dr, "page": page, "q_lo": q[0], "q_hi": q[1],
            "kv_lo": kv[0], "kv_hi": kv[1], "mask": mask}


def expand_case(name, B, H, dn, dr, dv, q, past, mask="causal"):
    return {"name": name, "op": "expand", "B": B, "H": H, "dn": dn, "dr": dr, "dv": dv, "q_lo": q[0], "q_hi": q[1],
            "past_lo": past[0], "past_hi": past[1], "mask": mask}


def fork_case(name, kind, P, F, page, H, d, bits, kv, new):
    """P sequences, F forks of each; kind "kv": K and V of H heads of d; "latent": latents of d and 64 rotated channels."""
    return {"name": name, "op": "fork", "kind": kind, "P": P, "F": F, "page": page, "H": H, "d": d, "bits": bits,
            "kv_lo": kv[0], "kv_hi": kv[1], "new_lo": new[0], "new_hi": new[1]}


def compact_case(name, kind, B, page, H, d, bits, kv, tree, share):
    """tree: drafted tokens at the end, a `share` of them accepted; without: a `share` of the history kept."""
    return {"name": name, "op": "compact", "kind": kind, "B": B, "page": page, "H": H, "d": d, "bits": bits,
            "kv_lo": kv[0], "kv_hi": kv[1], "tree_lo": tree[0], "tree_hi": tree[1], "share": share}


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


PAGES = (16, 32, 64, 128, 256)


def draw(rng):
    op = rng.choice(("append", "attn", "attn", "attn", "expand", "expand", "fork", "compact"))
    page = rng.choice(PAGES)
    dc = rng.choice((64, 128, 192, 256))
    if op == "append":
        dr, axes = rng.choice(((32, "32"), (64, "64"), (64, "32"), (64, "24,20,20"), (128, "44,42,42")))
        c = append_case("", spread(rng, 1, 37440), dc, dr, page, axes, rng.choice(("half", "interleaved")), rng.choice((24, 5000, 300000)))
    elif op == "attn":
        B, Hq = spread(rng, 1, 40), rng.choice((1, 2, 5, 8, 16, 24, 40))
        q_hi = spread(rng, 1, 64)
        most = min(400000, 560000 // B, 50000000 // (B * Hq * q_hi))  # keeps a pass under the largest listed one
        kv_hi = spread(rng, max(q_hi, min(300, most)), max(q_hi, most))
        c = attn_case("", B, Hq, dc, rng.choice((32, 64, 128)), page, (max(1, q_hi // 3), q_hi), (max(q_hi, kv_hi // 8), kv_hi),
                      rng.choice(("causal", "tree")))
    elif op == "expand":
        B, H = spread(rng, 1, 16), rng.choice((1, 2, 3, 8, 16))
        q_hi = spread(rng, 1, min(4000, int(math.sqrt(300000000 / (B * H)))))
        past = rng.choice((0, spread(rng, 1, max(1, min(4000, 300000000 // (B * H * q_hi) - q_hi)))))
        c = expand_case("", B, H, rng.choice((64, 128)), rng.choice((32, 64)), rng.choice((64, 128)), (max(1, q_hi // 9), q_hi),
                        (past // 3, past), rng.choice(("causal", "causal", "none")))
    else:
        kind = rng.choice(("kv", "latent"))
        H, d, bits = (rng.choice((1, 2, 8)), rng.choice((64, 128)), 8) if kind == "kv" else (1, dc, 16)
        if op == "fork":
            P, F = spread(rng, 1, 60), rng.choice((1, 2, 3))
            kv_hi = spread(rng, 20, min(24000, 600000 // P))
            new = spread(rng, 1, 100)
            c = fork_case("", kind, P, F, page, H, d, bits, (max(1, kv_hi // 8), kv_hi), (max(1, new // 4), new))
        else:
            B = spread(rng, 1, 30)
            tree = rng.choice((0, spread(rng, 2, 64))) if kind == "latent" else 0
            kv_hi = spread(rng, max(64, tree), min(20000, 90000 // B))
            c = compact_case("", kind, B, page, H, d, bits, (max(1, tree, kv_hi // 4), kv_hi), (max(1, tree // 3) if tree else 0, tree),
                             rng.choice((0.1, 0.5, 0.9)))
    del c["name"]
    return c


def ragged(lo, hi, count, odd):
    """`count` lengths between lo and hi, both ends among them, in a fixed mixed order."""
    rng = random.Random(1000 * count + odd)
    got = [hi] if count == 1 else [lo + (hi - lo) * i // (count - 1) for i in range(count)]
    rng.shuffle(got)
    return got


def up(a, b):
    return -(-a // b)


def row_bytes(c):
    """Bytes a token takes in the cache."""
    return 2 * c["H"] * (c["d"] * c["bits"] // 8 + 1) if c["kind"] == "kv" else 2 * (c["d"] + 64)


def work(c):
    if c["op"] == "append":
        turned = sum(dims_of(c))
        return {"bytes": 4 * c["n"] * (c["dc"] + c["dr"]) + c["n"] * (8 + 4 * len(dims_of(c))), "flops": 3 * c["n"] * turned}
    if c["op"] == "attn":
        nq, kv = ragged(c["q_lo"], c["q_hi"], c["B"], 1), ragged(c["kv_lo"], c["kv_hi"], c["B"], 2)
        pairs = sum(a * b for a, b in zip(nq, kv)) * c["Hq"]
        rows = sum(nq) * c["Hq"]
        held = 2 * sum(kv) * (c["dc"] + c["dr"]) + 4 * sum(up(x, c["page"]) for x in kv)
        return {"bytes": held + rows * (2 * (2 * c["dc"] + c["dr"]) + 4), "flops": 2 * pairs * (2 * c["dc"] + c["dr"])}
    if c["op"] == "expand":
        nq, past = ragged(c["q_lo"], c["q_hi"], c["B"], 1), ragged(c["past_lo"], c["past_hi"], c["B"], 2)
        seen = sum(t * p + (t * (t + 1) // 2 if c["mask"] == "causal" else t * t) for t, p in zip(nq, past)) * c["H"]
        q, k = sum(nq), sum(nq) + sum(past)
        return {"bytes": 2 * q * c["H"] * (c["dn"] + c["dr"] + c["dv"]) + 4 * q * c["H"] + 2 * k * (c["H"] * (c["dn"] + c["dv"]) + c["dr"]),
                "flops": 2 * seen * (c["dn"] + c["dr"] + c["dv"])}
    if c["op"] == "fork":
        kv = ragged(c["kv_lo"], c["kv_hi"], c["P"], 2)
        new = ragged(c["new_lo"], c["new_hi"], c["P"] * c["F"], 3)
        shared = c["F"] * sum(x % c["page"] != 0 for x in kv)
        entries = c["F"] * sum(up(x, c["page"]) for x in kv)
        return {"bytes": 2 * shared * c["page"] * row_bytes(c) + 24 * entries + 4 * pool_pages(c) + 8 * sum(new), "flops": entries}
    kv = ragged(c["kv_lo"], c["kv_hi"], c["B"], 2)
    if c["tree_hi"]:
        t = ragged(c["tree_lo"], c["tree_hi"], c["B"], 1)
        return {"bytes": 2 * row_bytes(c) * (sum(t) + sum(int(x * c["share"]) for x in t)) + 12 * sum(t), "flops": 3 * 64 * sum(t)}
    pages = sum(up(x, c["page"]) for x in kv)
    return {"bytes": 2 * row_bytes(c) * (pages * c["page"] + sum(int(x * c["share"]) for x in kv)) + 4 * sum(kv), "flops": sum(kv)}


def dims_of(c):
    return [int(x) for x in c["axes"].split(",")]


# ---- rotary plan ---------------------------------------------------------------------

BASE = 10000.0


def frequencies(dims):
    return [BASE ** (-2.0 * i / n) for n in dims for i in range(n // 2)]


def rope_state(dims, layout, pos):
    s = {"positions": pos.to(torch.int32).contiguous(), "freq": torch.tensor(frequencies(dims), dtype=torch.float64, device=DEV),
         "axis": torch.tensor([a for a, n in enumerate(dims) for _ in range(n // 2)], device=DEV), "layout": layout}
    if own:
        import video_diffusion_kv_gb300 as qvg
        s["plan"] = qvg.RopePlan(dims, layout=qvg.QVG_ROPE_HALF if layout == "half" else qvg.QVG_ROPE_INTERLEAVED, base=BASE)
    return s


def rotated(x, s):
    """x [n][channels] with its first channels rotated, in 32 bits (angles in 64)."""
    angle = s["positions"].double()[:, s["axis"]] * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    m, x = s["freq"].numel(), x.float()
    y = x.clone()
    lo, hi = (slice(0, m), slice(m, 2 * m)) if s["layout"] == "half" else (slice(0, 2 * m, 2), slice(1, 2 * m, 2))
    a, b = x[:, lo], x[:, hi]
    y[:, lo], y[:, hi] = a * cos - b * sin, b * cos + a * sin
    return y


# ---- inputs --------------------------------------------------------------------------

def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def latents(n, dc, dr, g):
    """bf16 [n][dc + dr], as a down projection leaves a token's latent and its shared key; a few channels stand out."""
    ch = torch.where(torch.rand(dc + dr, generator=g, device=DEV) < 0.02, 5.0, 1.0)
    return (torch.randn(n, dc + dr, generator=g, device=DEV) * ch).bfloat16()


def tables(lens, room, page, pages, g):
    """int32 [B][...]: pages for `lens` tokens (the table has columns for `room`), in any order."""
    order = torch.randperm(pages, generator=g, device=DEV).int()
    need = [up(x, page) for x in lens]
    table = torch.zeros(len(lens), max(up(x, page) for x in room), dtype=torch.int32, device=DEV)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table


def cache_buffers(c, pages, g):
    """Buffers of a filled cache: [codes, scales] of K and V, or [c, kr]."""
    if c["kind"] == "latent":
        return [latents(pages * c["page"], n, 0, g).view(pages, c["page"], n) for n in (c["d"], 64)]
    got = []
    for _ in range(2):
        shape = (pages, c["H"], c["page"])
        got.append(torch.cat([(100 * torch.randn(min(4096, pages - p), *shape[1:], c["d"], generator=g, device=DEV)).clamp(-448, 448)
                              .to(torch.float8_e4m3fn).view(torch.uint8) for p in range(0, pages, 4096)]))
        got.append(torch.randint(115, 125, (*shape, 1), generator=g, device=DEV, dtype=torch.uint8))
    return got


def handle(c, buffers):
    import video_diffusion_kv_gb300 as qvg
    if c.get("kind") == "kv":
        return qvg.PagedKV(c["H"], c["d"], c["page"], buffers[0].shape[0], bits=c["bits"], buffers=buffers)
    return qvg.LatentKV(buffers[0].shape[2], buffers[1].shape[2], c["page"], buffers[0].shape[0], buffers=buffers)


def starts(counts):
    got = [0]
    for x in counts:
        got.append(got[-1] + x)
    return torch.tensor(got, dtype=torch.int32, device=DEV)


def parents_of(nq, seed):
    """Every drafted token hangs on an earlier one or on the history (-1)."""
    r = random.Random(seed)
    return torch.tensor([r.randrange(max(-1, t - 6), t) for m in nq for t in range(m)], dtype=torch.int32, device=DEV)


def prepare(c, seed):
    g = gen(seed)
    return {"append": prepare_append, "attn": prepare_attn, "expand": prepare_expand, "fork": prepare_fork,
            "compact": prepare_compact}[c["op"]](c, seed, g)


def prepare_append(c, seed, g):
    dims, n, page = dims_of(c), c["n"], c["page"]
    if len(dims) == 3:  # frame, row and column of a 30 x 52 grid
        t = torch.arange(n, device=DEV)
        pos = torch.stack((t // 1560 + int(torch.randint(0, c["far"], (1,), generator=g, device=DEV)), t % 1560 // 52, t % 52), 1)
    else:
        pos = torch.randint(0, c["far"], (1, len(dims)), generator=g, device=DEV) + torch.arange(n, device=DEV)[:, None]
    pages = up(n, page) + 2
    order = torch.randperm(pages, generator=g, device=DEV)
    t = torch.arange(n, device=DEV) + page // 3  # the first page is already partly filled
    both = latents(n, c["dc"], c["dr"], g)
    buffers = [torch.zeros(pages, page, w, dtype=torch.bfloat16, device=DEV) for w in (c["dc"], c["dr"])]
    s = {"case": c, "slots": order[t // page] * page + t % page, "c": both[:, :c["dc"]], "kr": both[:, c["dc"]:], "buffers": buffers,
         **rope_state(dims, c["layout"], pos)}
    if own:
        s["cache"] = handle(c, buffers)
    return s


def prepare_attn(c, seed, g):
    B, page = c["B"], c["page"]
    nq, kv = ragged(c["q_lo"], c["q_hi"], B, 1), ragged(c["kv_lo"], c["kv_hi"], B, 2)
    pages = sum(up(x, page) for x in kv) + 3
    buffers = [latents(pages * page, n, 0, g).view(pages, page, n) for n in (c["dc"], c["dr"])]
    total = sum(nq)
    # queries in the latents' space as a product per head leaves them: [heads][tokens][channels]
    q = torch.randn(c["Hq"], total, c["dc"], generator=g, device=DEV).bfloat16().transpose(0, 1)
    s = {"case": c, "buffers": buffers, "table": tables(kv, kv, page, pages, g), "q": q,
         "q_rope": torch.randn(total, c["Hq"], c["dr"], generator=g, device=DEV).bfloat16(),
         "kv_len": torch.tensor(kv, dtype=torch.int32, device=DEV), "cu_q": starts(nq), "scale": 1 / math.sqrt(128 + c["dr"])}
    if c["mask"] == "tree":
        s["parents"] = parents_of(nq, seed)
    if own:
        s["cache"] = handle(c, buffers)
    return s


def prepare_expand(c, seed, g):
    nq, past = ragged(c["q_lo"], c["q_hi"], c["B"], 1), ragged(c["past_lo"], c["past_hi"], c["B"], 2)
    H, total, keys = c["H"], sum(nq), sum(nq) + sum(past)
    # rows of the fused projections: each head's plain and rotated query channels, each head's key and value
    q = torch.randn(total, H, c["dn"] + c["dr"], generator=g, device=DEV).bfloat16()
    kv = torch.randn(keys, H, c["dn"] + c["dv"], generator=g, device=DEV).bfloat16()
    return {"case": c, "q": q[..., :c["dn"]], "q_rope": q[..., c["dn"]:], "k": kv[..., :c["dn"]], "v": kv[..., c["dn"]:],
            "k_rope": latents(keys, 0, c["dr"], g), "cu_q": starts(nq), "cu_k": starts([a + b for a, b in zip(nq, past)]),
            "scale": 1 / math.sqrt(c["dn"] + c["dr"])}


def pool_pages(c):
    kv = ragged(c["kv_lo"], c["kv_hi"], c["P"], 2)
    grown = c["P"] * c["F"] * (up(c["new_hi"], c["page"]) + 1)
    return 2 * (sum(up(x, c["page"]) for x in kv) + grown)


def prepare_fork(c, seed, g):
    P, F, page = c["P"], c["F"], c["page"]
    kv, new = ragged(c["kv_lo"], c["kv_hi"], P, 2), ragged(c["new_lo"], c["new_hi"], P * F, 3)
    pages = pool_pages(c)
    table = torch.zeros(P * (F + 1), up(c["kv_hi"] + c["new_hi"], page), dtype=torch.int32, device=DEV)
    mine = tables(kv, kv, page, pages, g)
    table[:P, :mine.shape[1]] = mine
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    for b, x in enumerate(kv):
        refs[mine[b, :up(x, page)].long()] = 1
    first = list(range(P)) * F
    s = {"case": c, "table": table, "refs": refs, "kv_len": torch.tensor(kv + [0] * (P * F), dtype=torch.int32, device=DEV),
         "parents": torch.tensor(first, dtype=torch.int32, device=DEV),
         "children": torch.arange(P, P * (F + 1), dtype=torch.int32, device=DEV), "cu_new": starts([0] * P + new), "total": sum(new),
         "buffers": cache_buffers(c, pages, g)}
    plain_fork(s)  # the forks of the step before, which a pass frees first
    if own:
        import video_diffusion_kv_gb300 as qvg
        s["cache"], s["pool"] = handle(c, s["buffers"]), qvg.PagePool(pages, refs=refs)
    return s


def prepare_compact(c, seed, g):
    B, page = c["B"], c["page"]
    kv = ragged(c["kv_lo"], c["kv_hi"], B, 2)
    r = random.Random(seed)
    pages = sum(up(x, page) for x in kv) * (1 if c["tree_hi"] else 2) + 2
    if c["tree_hi"]:
        t = ragged(c["tree_lo"], c["tree_hi"], B, 1)
        first = [a - b for a, b in zip(kv, t)]
        kept = [[f + i for i in sorted(r.sample(range(n), int(n * c["share"])))] for f, n in zip(first, t)]
    else:
        first = [min(4, x) for x in kv]  # the first tokens stay where they are
        kept = [sorted(r.sample(range(f, x), min(x - f, int(x * c["share"])))) for f, x in zip(first, kv)]
    keep = torch.full((B, max(1, max(map(len, kept)))), -1, dtype=torch.int32)
    for b, k in enumerate(kept):
        keep[b, :len(k)] = torch.tensor(k, dtype=torch.int32)
    s = {"case": c, "first": torch.tensor(first, dtype=torch.int32, device=DEV), "keep": keep.to(DEV),
         "n_keep": torch.tensor([len(k) for k in kept], dtype=torch.int32, device=DEV), "buffers": cache_buffers(c, pages, g)}
    if c["tree_hi"]:
        s["table"] = tables(kv, kv, page, pages, g)
        b = torch.repeat_interleave(torch.arange(B), torch.tensor(t))
        at = torch.cat([torch.arange(f, x) for f, x in zip(first, kv)])
        s["slots"] = s["table"].cpu()[b, at // page].long().to(DEV) * page + (at % page).to(DEV)
        both = latents(sum(t), c["d"], 64, g)
        s.update(c=both[:, :c["d"]], kr=both[:, c["d"]:], **rope_state([64], "half", at[:, None].to(DEV)))
    else:
        two = tables(kv + kv, kv, page, pages, g)
        s["table"] = two[B:].contiguous()
        s["copies"] = torch.cat([torch.stack((two[b, :up(x, page)], two[B + b, :up(x, page)]), 1) for b, x in enumerate(kv)]).contiguous()
    if own:
        s["cache"] = handle(c, s["buffers"])
    return s


# ---- one pass ------------------------------------------------------------------------

def run(s):
    return (own_calls if own else plain)(s)


def values(s):
    """The cache's state: latents, or codes as the fp8 numbers they are and scale bytes."""
    return [b.view(torch.float8_e4m3fn) if b.dtype == torch.uint8 and b.shape[-1] > 1 else b for b in s["buffers"]]


def own_calls(s):
    import video_diffusion_kv_gb300 as qvg
    c = s["case"]
    if c["op"] == "append":
        qvg.latent_append(s["cache"], s["c"], s["kr"], s["slots"], plan=s["plan"], positions=s["positions"])
        return values(s)
    if c["op"] == "attn":
        mask = qvg.tree_mask(s["parents"], c["q_hi"], cu_q=s["cu_q"]) if c["mask"] == "tree" else None
        return qvg.latent_attention(s["cache"], s["q"], s["q_rope"], s["table"], s["kv_len"], c["q_hi"], s["scale"], cu_q=s["cu_q"], mask=mask,
                                    mask_mode=qvg.QVG_MASK_TREE if c["mask"] == "tree" else qvg.QVG_MASK_CAUSAL, want_lse=True)
    if c["op"] == "expand":
        return qvg.expanded_attention(s["q"], s["q_rope"], s["k"], s["k_rope"], s["v"], c["q_hi"], scale=s["scale"], cu_q=s["cu_q"],
                                      cu_k=s["cu_k"], mask_mode=qvg.QVG_MASK_CAUSAL if c["mask"] == "causal" else qvg.QVG_MASK_NONE,
                                      want_lse=True)
    if c["op"] == "fork":
        qvg.pages_release(s["pool"], c["page"], s["table"], s["kv_len"], s["children"])
        qvg.pages_fork(s["pool"], c["page"], s["table"], s["kv_len"], s["parents"], s["children"])
        slots, copies = qvg.pages_reserve(s["pool"], c["page"], s["table"], s["kv_len"], cu_new=s["cu_new"], total=s["total"])
        qvg.pages_copy(s["cache"], copies)
        return [slots, copies, s["table"], s["kv_len"], s["refs"]] + values(s)
    if c["tree_hi"]:
        qvg.latent_append(s["cache"], s["c"], s["kr"], s["slots"], plan=s["plan"], positions=s["positions"])
    else:
        qvg.pages_copy(s["cache"], s["copies"])
    qvg.paged_compact(s["cache"], s["table"], s["first"], s["keep"], s["n_keep"])
    return values(s)


def plain(s):
    return {"append": plain_append, "attn": plain_attention, "expand": plain_expanded, "fork": plain_fork, "compact": plain_compact}[s["case"]["op"]](s)


def plain_append(s):
    page, (c, kr) = s["case"]["page"], s["buffers"]
    at = s["slots"] // page, s["slots"] % page
    c[at] = s["c"]
    kr[at] = rotated(s["kr"], s).bfloat16()
    return values(s)


def ancestors(parents, b, t, B, n):
    """[B][n][n]: whether token j is token t or one of its ancestors."""
    step = torch.zeros(B, n, n, device=DEV)
    has = parents >= 0
    step[b[has], t[has], parents[has].long()] = 1
    eye = torch.eye(n, device=DEV).expand(B, n, n)
    return torch.linalg.solve_triangular(eye - step, eye, upper=False, unitriangular=True) > 0.5


def softmax_rows(x, v):
    """(weights times v, log-sum-exp) of logits x (-inf: not seen); a row that sees nothing is 0."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    den = p.sum(-1)
    return p @ v / torch.where(den == 0, 1.0, den)[..., None], den.log() + m[..., 0]


def plain_attention(s):
    c, cu, table = s["case"], s["cu_q"].long(), s["table"].long()
    B, Hq, dc, n = c["B"], c["Hq"], c["dc"], c["q_hi"]
    row = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(cu, row, right=True) - 1
    t = row - cu[b]
    q = torch.zeros(B, n, Hq, dc + c["dr"], device=DEV)
    q[b, t] = torch.cat((s["q"], s["q_rope"]), -1).float()
    q = q.transpose(1, 2).reshape(B, Hq * n, -1)
    k = torch.cat([x[table].flatten(1, 2) for x in s["buffers"]], -1).float()
    key = torch.arange(k.shape[1], device=DEV)
    nq, kv = cu[1:] - cu[:-1], s["kv_len"].long()
    j = key[None] - (kv - nq)[:, None]  # key's number among the new tokens; below 0: history
    if c["mask"] == "tree":
        inside = j.clamp(0, n - 1)[:, None].expand(B, n, -1)
        see = torch.where(j[:, None] < 0, True, ancestors(s["parents"], b, t, B, n).gather(2, inside))
    else:
        see = j[:, None] <= torch.arange(n, device=DEV)[None, :, None]
    see = see & (key[None] < kv[:, None])[:, None]
    x = (q @ k.transpose(1, 2)).mul_(s["scale"])
    x = x.view(B, Hq, n, -1).masked_fill_(~see[:, None], -math.inf).view(B, Hq * n, -1)
    o, lse = softmax_rows(x, k[..., :dc])
    o, lse = o.view(B, Hq, n, dc).transpose(1, 2)[b, t], lse.view(B, Hq, n).transpose(1, 2)[b, t]
    return o.bfloat16(), lse.t().contiguous()


def plain_expanded(s):
    c = s["case"]
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    outs, lses = [], []
    for b in range(c["B"]):
        q = torch.cat((s["q"], s["q_rope"]), -1)[cq[b]:cq[b + 1]].float().transpose(0, 1)
        k = torch.cat((s["k"], s["k_rope"][:, None].expand(-1, c["H"], -1)), -1)[ck[b]:ck[b + 1]].float().transpose(0, 1)
        x = (q @ k.transpose(1, 2)).mul_(s["scale"])
        if c["mask"] == "causal":
            T, L = x.shape[1:]
            x.masked_fill_(torch.arange(L, device=DEV)[None] > torch.arange(T, device=DEV)[:, None] + L - T, -math.inf)
        o, lse = softmax_rows(x, s["v"][ck[b]:ck[b + 1]].float().transpose(0, 1))
        outs.append(o.transpose(0, 1).bfloat16())
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses, 1)


def plain_fork(s):
    c, page, table, refs, kv_len = s["case"], s["case"]["page"], s["table"], s["refs"], s["kv_len"]
    column = torch.arange(table.shape[1], device=DEV)

    def held(seqs):  # the pages that sequences hold, one entry for each holding
        m = column < ((kv_len[seqs] + page - 1) // page)[:, None]
        return m, table[seqs][m].long()

    kids, parents = s["children"].long(), s["parents"].long()
    refs.index_add_(0, held(kids)[1], torch.full_like(refs[held(kids)[1]], -1))  # freed
    kv_len[kids] = 0
    m, pages = held(parents)  # forked
    table[kids] = torch.where(m, table[parents], table[kids])
    refs.index_add_(0, pages, torch.ones_like(refs[pages]))
    kv_len[kids] = kv_len[parents]
    L, n = kv_len.long(), (s["cu_new"][1:] - s["cu_new"][:-1]).long()  # new tokens
    old = up(L, page)
    seq = torch.arange(len(L), device=DEV)
    last = table[seq, (old - 1).clamp(min=0)].long()
    shared = (n > 0) & (L % page != 0) & (refs[last] > 1)
    rank = ((last[:, None] == last[None]) & shared[None] & (seq[None] < seq[:, None])).sum(1)
    cow = shared & (rank < refs[last] - 1)
    need = up(L + n, page) - old + cow
    upto = need.cumsum(0)
    k = torch.arange(int(upto[-1]), device=DEV)
    b = torch.searchsorted(upto, k, right=True)
    free = (refs == 0).nonzero()[:len(k), 0]
    j = k - (upto - need)[b] - cow[b].long()  # -1: the copy of the last page
    table[b, old[b] + j] = free.int()
    refs.index_add_(0, last[cow], torch.full_like(refs[last[cow]], -1))
    refs[free] = 1
    copies = torch.where(cow[:, None], torch.stack((last, table[seq, (old - 1).clamp(min=0)].long()), 1), -1).int()
    row = torch.arange(s["total"], device=DEV)
    b = torch.searchsorted(s["cu_new"].long(), row, right=True) - 1
    at = L[b] + row - s["cu_new"].long()[b]
    slots = table[b, at // page].long() * page + at % page
    kv_len += n.int()
    src, dst = copies[cow].long().unbind(1)
    for x in s["buffers"]:
        x[dst] = x[src]
    return [slots, copies, table, kv_len, refs] + values(s)


def plain_compact(s):
    c, page, table = s["case"], s["case"]["page"], s["table"].long()
    if c["tree_hi"]:
        plain_append(s)
    else:
        src, dst = s["copies"].long().unbind(1)
        for x in s["buffers"]:
            x[dst] = x[src]
    b, i = (torch.arange(s["keep"].shape[1], device=DEV) < s["n_keep"][:, None]).nonzero().unbind(1)
    src, dst = s["keep"][b, i].long(), s["first"].long()[b] + i
    for x in s["buffers"]:
        if c["kind"] == "kv":
            x[table[b, dst // page], :, dst % page] = x[table[b, src // page], :, src % page]
        else:
            x[table[b, dst // page], dst % page] = x[table[b, src // page], src % page]
    return values(s)


# ---- 64 bits -------------------------------------------------------------------------

def exact_rope(x, s):
    x = x.double()
    pair = torch.arange(s["freq"].numel(), device=DEV)
    lo, hi = (pair, pair + len(pair)) if s["layout"] == "half" else (2 * pair, 2 * pair + 1)
    turn = s["positions"].double()[:, s["axis"]] * s["freq"]
    z = torch.complex(x[:, lo], x[:, hi]) * torch.polar(torch.ones_like(turn), turn)
    y = x.clone()
    y[:, lo], y[:, hi] = z.real, z.imag
    return y


def exact(c, seed):
    s = prepare(c, seed)
    return {"append": exact_append, "attn": exact_attention, "expand": exact_expanded, "fork": exact_fork,
            "compact": exact_compact}[c["op"]](s, c)


def exact_append(s, c):
    out = [b.double().flatten(0, 1) for b in s["buffers"]]
    out[0][s["slots"]] = s["c"].double()
    out[1][s["slots"]] = exact_rope(s["kr"], s)
    return [o.view(b.shape) for o, b in zip(out, s["buffers"])]


def exact_rows(q, k, v, see, scale):
    """q [T][H][n], k [L][H or 1][n], v [L][H or 1][m] in 64 bits, see [T][L] -> (out [T][H][m], lse [H][T])."""
    T, H = q.shape[:2]
    out, lse = torch.empty(T, H, v.shape[2], dtype=torch.float64, device=DEV), torch.empty(H, T, dtype=torch.float64, device=DEV)
    for h in range(H):
        kh, vh = k[:, h % k.shape[1]].double(), v[:, h % v.shape[1]].double()
        for t in range(0, T, 1024):
            x = (q[t:t + 1024, h].double() @ kh.T * scale).masked_fill(~see[t:t + 1024], -math.inf)
            lse[h, t:t + 1024] = torch.logsumexp(x, -1)
            out[t:t + 1024, h] = torch.softmax(x, -1) @ vh
    return out, lse


def exact_attention(s, c):
    nq, kv = ragged(c["q_lo"], c["q_hi"], c["B"], 1), ragged(c["kv_lo"], c["kv_hi"], c["B"], 2)
    outs, lses, first = [], [], 0
    for b in range(c["B"]):
        pages = s["table"][b, :up(kv[b], c["page"])].long()
        latent, kr = (x[pages].flatten(0, 1)[:kv[b], None] for x in s["buffers"])
        new = torch.zeros(nq[b], nq[b], dtype=torch.bool)
        above = s["parents"][first:first + nq[b]].tolist() if c["mask"] == "tree" else list(range(-1, nq[b] - 1))
        for t in range(nq[b]):
            if above[t] >= 0:
                new[t] = new[above[t]]
            new[t, t] = True
        see = torch.ones(nq[b], kv[b], dtype=torch.bool, device=DEV)
        see[:, kv[b] - nq[b]:] = new.to(DEV)
        q = torch.cat((s["q"][first:first + nq[b]], s["q_rope"][first:first + nq[b]]), -1)
        o, l = exact_rows(q, torch.cat((latent, kr), -1), latent, see, s["scale"])
        outs.append(o)
        lses.append(l)
        first += nq[b]
    return torch.cat(outs), torch.cat(lses, 1)


def exact_expanded(s, c):
    nq, past = ragged(c["q_lo"], c["q_hi"], c["B"], 1), ragged(c["past_lo"], c["past_hi"], c["B"], 2)
    outs, lses, q0, k0 = [], [], 0, 0
    for T, P in zip(nq, past):
        L = T + P
        see = torch.ones(T, L, dtype=torch.bool, device=DEV)
        see = torch.tril(see, P) if c["mask"] == "causal" else see
        q = torch.cat((s["q"][q0:q0 + T], s["q_rope"][q0:q0 + T]), -1)
        k = torch.cat((s["k"][k0:k0 + L], s["k_rope"][k0:k0 + L, None].expand(-1, c["H"], -1)), -1)
        o, l = exact_rows(q, k, s["v"][k0:k0 + L], see, s["scale"])
        outs.append(o)
        lses.append(l)
        q0, k0 = q0 + T, k0 + L
    return torch.cat(outs), torch.cat(lses, 1)


def exact_fork(s, c):
    """One sequence after the other, on the host."""
    page = c["page"]
    table, refs, L = s["table"].tolist(), s["refs"].tolist(), s["kv_len"].tolist()
    cu = s["cu_new"].tolist()
    for b in s["children"].tolist():
        for p in table[b][:up(L[b], page)]:
            refs[p] -= 1
        L[b] = 0
    for a, b in zip(s["parents"].tolist(), s["children"].tolist()):
        L[b] = L[a]
        for i in range(up(L[a], page)):
            table[b][i] = table[a][i]
            refs[table[a][i]] += 1
    free = iter([p for p, r in enumerate(refs) if r == 0])  # what becomes free in this call is not given out by it
    slots, copies = [], []
    for b in range(len(L)):
        pair = [-1, -1]
        for i in range(L[b], L[b] + cu[b + 1] - cu[b]):
            if i % page == 0:
                table[b][i // page] = next(free)
                refs[table[b][i // page]] = 1
            elif refs[table[b][i // page]] > 1:
                pair = [table[b][i // page], next(free)]
                refs[pair[0]] -= 1
                refs[pair[1]] = 1
                table[b][i // page] = pair[1]
            slots.append(table[b][i // page] * page + i % page)
        L[b] += cu[b + 1] - cu[b]
        copies.append(pair)
    held = values({"buffers": [x.clone() for x in s["buffers"]]})
    for a, b in copies:
        if a >= 0:
            for x in held:
                x.view(torch.uint8)[b].copy_(x.view(torch.uint8)[a])
    whole = [torch.tensor(x, dtype=d) for x, d in ((slots, torch.int64), (copies, torch.int32), (table, torch.int32), (L, torch.int32),
                                                   (refs, torch.int32))]
    return whole + [x.double() if x.is_floating_point() else x for x in held]


def exact_compact(s, c):
    page = c["page"]
    held = [x.double() if x.is_floating_point() else x.clone() for x in values(s)]
    if c["tree_hi"]:
        held = exact_append({**s, "buffers": held}, c)
    else:
        for a, b in s["copies"].tolist():
            for x in held:
                x[b] = x[a]
    table = s["table"].tolist()
    for b, n in enumerate(s["n_keep"].tolist()):
        src = s["keep"][b, :n].tolist()
        dst = range(s["first"][b].item(), s["first"][b].item() + n)
        where = [torch.tensor([[table[b][i // page], i % page] for i in at], dtype=torch.long, device=DEV).view(-1, 2).unbind(1) for at in (src, dst)]
        for x in held:
            rows = x.transpose(1, 2) if c["kind"] == "kv" else x
            rows[where[1]] = rows[where[0]]
    return held
