"""The latent cache on the GPU (append, read, attention in the absorbed form)
and attention of prompts in the expanded form, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import video_diffusion_kv_gb300 as qvg

import _paged as ref

pytestmark = pytest.mark.gpu

NONE, CAUSAL, TREE = qvg.QVG_MASK_NONE, qvg.QVG_MASK_CAUSAL, qvg.QVG_MASK_TREE


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert qvg.get_status() == qvg.QVG_OK


def starts(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


# ---- the plain form and its bounds -------------------------------------------------

def check_rows(got, got_lse, q, k, v, see, scale, out_bf16):
    """got [T][H][m], got_lse [H][T] or None, against q [T][H][n], k [L][H or
    1][n], v [L][H or 1][m] (float64), see [T][L].  Bounds, per row (p: the
    weights, summing to 1):
      a logit is off by D = scale n 2^-23 sum |q||k| (an fp32 sum of n exact
      products, in any order, cut off rather than rounded) + 8 2^-24 max|s|
      (the base-2 form's roundings of the logit and of the reference);
      a weight by 2 D + 2^-20 (2^x) + 2^-8 (rounded to bf16) of itself; weights
      and their sum over L keys by L 2^-23 more; and the output by half a step
      of its type.
      lse: D + 2^-20 + L 2^-24 (the sum) + 2^-22 |lse|."""
    T, H = q.shape[:2]
    half = 2.0 ** -8 if out_bf16 else 2.0 ** -24
    worst = 0.0
    for h in range(H):
        kh, vh = k[:, h % k.shape[1]], v[:, h % v.shape[1]]
        for t0 in range(0, T, 64):
            qq, ss, row = q[t0:t0 + 64, h], see[t0:t0 + 64], got[t0:t0 + 64, h]
            some = ss.any(1)
            assert (row[~some] == 0).all()
            if got_lse is not None:
                assert (got_lse[h, t0:t0 + 64][~some] == -np.inf).all()
            if not some.any():
                continue
            qq, ss, row = qq[some], ss[some], row[some]
            s = np.where(ss, qq @ kh.T * scale, -np.inf)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            den = p.sum(1, keepdims=True)
            p /= den
            want, lse = p @ vh, (m + np.log(den))[:, 0]
            n, L = q.shape[2], len(kh)
            top = np.where(ss, np.abs(s), 0).max(1)
            dd = (scale * n * 2.0 ** -23 * np.where(ss, np.abs(qq) @ np.abs(kh).T, 0)).max(1) + 8 * 2.0 ** -24 * top
            rel = 2 * dd + 2.0 ** -20 + 2.0 ** -8 + L * 2.0 ** -23
            bound = rel[:, None] * (p @ np.abs(vh)) + half * np.abs(want) + 1e-37
            err = np.abs(row - want)
            assert np.isfinite(row).all()
            assert (err <= bound).all(), (h, t0, float((err / bound).max()))
            worst = max(worst, float((err / bound).max()))
            if got_lse is not None:
                lb = dd + 2.0 ** -20 + L * 2.0 ** -24 + 2.0 ** -22 * np.abs(lse)
                e = np.abs(got_lse[h, t0:t0 + 64][some] - lse)
                assert (e <= lb).all(), (h, t0, float((e / lb).max()))
    return worst


def seen(T, L, mode, rows=None):
    j, t = np.arange(L)[None] - (L - T), np.arange(T)[:, None]
    if mode == NONE:
        return np.ones((T, L), bool)
    if mode == CAUSAL:
        return j <= t
    return np.where(j < 0, True, rows[t, np.clip(j, 0, T - 1)])


class Batch:
    """A latent cache with B sequences on shuffled pages and their new tokens'
    queries.  Slots of no sequence, and each last page behind its sequence,
    hold NaN; table entries past the last page are no pages."""

    def __init__(self, Hq, dc, dr, page, nq, kv, seed=0, q_scale=1.0, c_scale=1.0):
        g = np.random.default_rng(seed)
        need = [-(-n // page) for n in kv]
        pages = sum(need) + 2
        order = g.permutation(pages)
        self.Hq, self.dc, self.dr, self.nq, self.kv, self.page = Hq, dc, dr, nq, kv, page
        self.cache = qvg.LatentKV(dc, dr, page, pages)
        self.cache.c.fill_(math.nan)
        self.cache.kr.fill_(math.nan)
        table = np.full((len(kv), max(need + [1])), -7, np.int32)
        self.slots, at = [], 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
            t = np.arange(kv[b])
            self.slots.append(table[b, t // page].astype(np.int64) * page + t % page)
        dev = lambda *s: torch.from_numpy(g.standard_normal(s)).to("cuda", torch.bfloat16)  # noqa: E731
        rows, total = sum(kv), sum(nq)
        self.c, self.kr = dev(rows, dc) * c_scale, dev(rows, dr)
        self.all_slots = torch.from_numpy(np.concatenate(self.slots + [np.zeros(0, np.int64)])).cuda()
        if rows:
            qvg.latent_append(self.cache, self.c, self.kr if dr else None, self.all_slots)
        self.table = torch.from_numpy(table).cuda()
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")
        self.cu_q = starts(nq)
        self.q, self.q_rope = dev(total, Hq, dc) * q_scale, (dev(total, Hq, dr) if dr else None)
        self.scale = 1 / math.sqrt(dc / 2 + dr)

    def run(self, mode=CAUSAL, **kw):
        kw.setdefault("want_lse", True)
        kw.setdefault("cu_q", self.cu_q)
        return qvg.latent_attention(self.cache, self.q, self.q_rope, self.table, self.kv_len, max(self.nq), self.scale, mask_mode=mode, **kw)

    def check(self, out, lse, mode, rows=None, skip=()):
        c, kr = (x.double().cpu().flatten(0, 1).numpy() for x in (self.cache.c, self.cache.kr))
        q = torch.cat((self.q, self.q_rope), -1) if self.dr else self.q
        q, got = q.double().cpu().numpy(), out.double().cpu().numpy()
        got_lse = None if lse is None else lse.double().cpu().numpy()
        first = 0
        for b, T in enumerate(self.nq):
            at = self.slots[b]
            if b not in skip:
                k = np.concatenate((c[at], kr[at]), 1)[:, None] if self.dr else c[at][:, None]
                part = slice(first, first + T)
                check_rows(got[part], None if lse is None else got_lse[:, part], q[part], k, c[at][:, None],
                           seen(T, self.kv[b], mode, None if rows is None else rows[b]), self.scale, out.dtype == torch.bfloat16)
            first += T


def trees(nq, seed):
    """(parents on the device, mask rows, seen rows per sequence)."""
    r = np.random.default_rng(seed)
    parents = [[int(r.integers(max(-1, t - 4), t)) for t in range(n)] for n in nq]
    dev = torch.tensor([p for x in parents for p in x], dtype=torch.int32, device="cuda")
    return qvg.tree_mask(dev, max(nq), cu_q=starts(nq)), [ref.tree_rows(p) for p in parents]


# ---- append and read -------------------------------------------------------------------

@pytest.mark.parametrize("layout", [qvg.QVG_ROPE_HALF, qvg.QVG_ROPE_INTERLEAVED])
@pytest.mark.parametrize("dc,dr,dims,page", [
    (64, 8, (4, 2), 16), (128, 24, (16,), 32), (192, 64, (24, 20, 20), 64), (256, 64, (64,), 128), (256, 128, (44, 42, 42), 256),
    (256, 128, (126,), 16), (64, 40, (30,), 16),
])
def test_append_rotates(layout, dc, dr, dims, page):
    """Latents to the bit; rotated key parts within the angle's and the
    products' roundings (cos and sin off by 2^-24 + 2 pi 2^-28, three fp32
    roundings) and half a bf16 step; channels past the rotated ones, slots of no token and skipped
    tokens as they were."""
    g = np.random.default_rng(dc + dr)
    n, plan = 77, qvg.RopePlan(dims, layout=layout)
    cache = qvg.LatentKV(dc, dr, page, -(-n // page) + 3)
    cache.c.fill_(3.0)
    cache.kr.fill_(5.0)
    both = torch.from_numpy(g.standard_normal((n, dc + dr + 8))).to("cuda", torch.bfloat16)
    c, kr = both[:, :dc], both[:, dc:dc + dr]
    pos = g.integers(0, 400000, (n, len(dims))).astype(np.int32)
    slots = g.permutation(cache.num_pages * page)[:n].astype(np.int64)
    slots[5] = -1
    qvg.latent_append(cache, c, kr, torch.from_numpy(slots).cuda(), plan=plan, positions=torch.from_numpy(pos).cuda())
    got_c, got_kr = cache.c.view(-1, dc).cpu(), cache.kr.view(-1, dr).double().cpu().numpy()
    live = slots >= 0
    assert torch.equal(got_c[slots[live]], c.cpu()[live])
    f, axis = ref.frequencies(dims)
    x = kr.double().cpu().numpy()
    want = ref.rope(x[:, None], pos, f, axis, layout)[:, 0]
    if layout == qvg.QVG_ROPE_HALF:
        m = sum(dims) // 2
        size = x.copy()
        size[:, :m] = size[:, m:2 * m] = np.abs(x[:, :m]) + np.abs(x[:, m:2 * m])
    else:
        size = x.copy()
        size[:, 0:sum(dims):2] = size[:, 1:sum(dims):2] = np.abs(x[:, 0:sum(dims):2]) + np.abs(x[:, 1:sum(dims):2])
    bound = 2.0 ** -8 * np.abs(want) + (4 * 2.0 ** -24 + 2 * math.pi * 2.0 ** -28) * np.abs(size) * 1.01
    assert (np.abs(got_kr[slots[live]] - want[live]) <= bound[live]).all()
    np.testing.assert_array_equal(got_kr[slots[live]][:, sum(dims):], x[live][:, sum(dims):])
    rest = np.setdiff1d(np.arange(cache.num_pages * page), slots)
    assert (got_c[rest] == 3).all() and (got_kr[rest] == 5).all()
    back_c, back_kr = qvg.latent_read(cache, torch.from_numpy(slots).cuda())
    assert torch.equal(back_c.cpu()[live], got_c[slots[live]]) and (back_c[5] == 0).all() and (back_kr[5] == 0).all()
    np.testing.assert_array_equal(back_kr.double().cpu().numpy()[live], got_kr[slots[live]])


def test_append_without_a_plan_without_key_parts_and_non_finite():
    for dr in (0, 16):
        cache = qvg.LatentKV(128, dr, 16, 2)
        x = torch.randn(6, 128 + dr, device="cuda").bfloat16()
        x[1, 3], x[2, 127] = math.inf, math.nan
        if dr:
            x[4, 130] = -math.inf
        c, kr = x[:, :128].contiguous(), x[:, 128:].contiguous()
        qvg.latent_append(cache, c, kr if dr else None, torch.arange(6, device="cuda"))
        bad = [1, 2] + ([4] if dr else [])
        for t in range(6):
            if t in bad:
                assert cache.c[0, t].isnan().all() and cache.kr[0, t].isnan().all()
            else:
                assert torch.equal(cache.c[0, t], c[t]) and torch.equal(cache.kr[0, t], kr[t])


def test_slots_beyond_the_cache():
    cache = qvg.LatentKV(64, 8, 16, 2)
    c, kr = torch.ones(2, 64, device="cuda").bfloat16(), torch.ones(2, 8, device="cuda").bfloat16()
    slots = torch.tensor([32, 31], device="cuda")
    qvg.latent_append(cache, c, kr, slots)
    assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG
    assert (cache.c.view(-1, 64)[31] == 1).all() and cache.c.sum() == 64
    got, _ = qvg.latent_read(cache, slots)
    assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG
    assert (got[0] == 0).all() and (got[1] == 1).all()
    qvg.latent_append(cache, c[:0], kr[:0], slots[:0])
    assert qvg.latent_read(cache, slots[:0])[0].shape == (0, 64)


# ---- absorbed form ----------------------------------------------------------------------

@pytest.mark.parametrize("Hq,dc,dr,page,nq,kv", [
    (1, 64, 0, 16, (1,), (1,)),
    (1, 64, 8, 16, (1, 1, 1, 1, 1), (1, 63, 64, 65, 129)),
    (5, 128, 32, 32, (1, 1, 1), (300, 17, 1000)),
    (16, 256, 64, 64, (1, 3, 2), (64, 700, 65)),
    (8, 192, 40, 128, (5,), (513,)),
    (24, 256, 128, 256, (9, 16), (255, 1030)),
    (3, 256, 72, 16, (50, 1), (400, 900)),
])
@pytest.mark.parametrize("mode", [NONE, CAUSAL, TREE])
def test_shapes_and_masks(Hq, dc, dr, page, nq, kv, mode):
    b = Batch(Hq, dc, dr, page, nq, kv, seed=dc + dr)
    kw, rows = {}, None
    if mode == TREE:
        kw["mask"], rows = trees(nq, 3)
    out, lse = b.run(mode, **kw)
    assert qvg.get_status() == qvg.QVG_OK
    b.check(out, lse, mode, rows)
    o32, _ = b.run(mode, out_dtype=qvg.QVG_OUT_F32, **kw)
    b.check(o32, None, mode, rows)


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 127, 128, 129, 300])
def test_row_counts(rows):
    b = Batch(1, 128, 64, 32, (rows, 1), (700, 200), seed=rows)
    out, lse = b.run()
    b.check(out, lse, CAUSAL)


def test_long_and_ragged():
    b = Batch(16, 256, 64, 64, (1,) * 9, (1, 30000, 64, 5, 9000, 4097, 0, 128, 777), seed=5)
    out, lse = b.run()
    b.check(out, lse, CAUSAL)


def test_thousands_of_sequences():
    n = 2500
    b = Batch(2, 64, 16, 16, (1,) * n, tuple(i % 40 for i in range(n)), seed=6)
    out, lse = b.run()
    b.check(out, lse, CAUSAL)


@pytest.mark.parametrize("short", [1, 2, 3])
@pytest.mark.parametrize("idle", [0, 1, 40, 700])
@pytest.mark.parametrize("dc,dr,page", [(64, 0, 64), (256, 64, 16)])
def test_a_short_unit_before_a_long_one(short, idle, dc, dr, page):
    """Parts of the line that begin with a unit of 1, 2 or 3 tiles before one of
    many, the next unit found at once or behind sequences without new tokens
    (so that its Q and its first tiles are asked for at the same time)."""
    parts = torch.cuda.get_device_properties(0).multi_processor_count if idle < 100 else 12
    nq = ((1,) + (0,) * idle + (1,)) * parts
    kv = ((64 * short,) + (70,) * idle + (64 * 20 - 3,)) * parts
    b = Batch(3, dc, dr, page, nq, kv, seed=short)
    out, lse = b.run()
    assert qvg.get_status() == qvg.QVG_OK
    b.check(out, lse, CAUSAL)
    for _ in range(5):
        again, again_lse = b.run()
        assert torch.equal(again, out) and torch.equal(again_lse, lse)
    assert qvg.get_status() == qvg.QVG_OK


@pytest.mark.parametrize("dc,dr", [(64, 0), (128, 64), (256, 128)])
def test_many_units_a_part(dc, dr):
    """Units of one or two tiles, a dozen or more after one another in each
    part: each one's Q takes the place of the last one's."""
    n = 1600
    b = Batch(20, dc, dr, 32, tuple(1 + i % 7 for i in range(n)), tuple(7 + (11 * i) % 120 for i in range(n)), seed=dc)
    out, lse = b.run()
    b.check(out, lse, CAUSAL)
    for _ in range(5):
        again, again_lse = b.run()
        assert torch.equal(again, out) and torch.equal(again_lse, lse)


@pytest.mark.parametrize("mode", [NONE, CAUSAL, TREE])
@pytest.mark.parametrize("nq,kv", [((5, 16), (3, 1)), ((40, 7), (10, 6)), ((200, 140), (150, 0))])
def test_more_new_tokens_than_keys(mode, nq, kv):
    b = Batch(4, 64, 16, 16, nq, kv, seed=7)
    kw, rows = {}, None
    if mode == TREE:  # masks count the new tokens, of which the first have no key
        kw["mask"], rows = trees(nq, 4)
        rows = [r[:, T - min(T, L):] if L else r[:, :0] for r, T, L in zip(rows, nq, kv)]
    out, lse = b.run(mode, **kw)
    if mode == TREE:
        got, got_lse, first = out.double().cpu().numpy(), lse.double().cpu().numpy(), 0
        c = b.cache.c.double().cpu().numpy().reshape(-1, 64)
        kr = b.cache.kr.double().cpu().numpy().reshape(-1, 16)
        q = torch.cat((b.q, b.q_rope), -1).double().cpu().numpy()
        for i, T in enumerate(nq):
            at, part = b.slots[i], slice(first, first + T)
            check_rows(got[part], got_lse[:, part], q[part], np.concatenate((c[at], kr[at]), 1)[:, None], c[at][:, None], rows[i], b.scale, True)
            first += T
    else:
        b.check(out, lse, mode)


def test_masks_that_leave_a_row_empty():
    """Mask words of 0: only the history is left; without one, nothing."""
    b = Batch(4, 128, 32, 16, (6, 5), (40, 5), seed=8)
    mask = torch.zeros(11, 1, dtype=torch.int32, device="cuda")
    mask[2] = -1
    out, lse = b.run(TREE, mask=mask)
    rows = [np.zeros((6, 6), bool), np.zeros((5, 5), bool)]
    rows[0][2] = True
    b.check(out, lse, TREE, rows)
    assert (out[6:] == 0).all() and (lse[:, 6:] == -math.inf).all()


@pytest.mark.parametrize("dc,dr", [(64, 0), (256, 64), (192, 128)])
@pytest.mark.parametrize("T", [1, 9, 70])
def test_unseen_keys_have_no_influence(dc, dr, T):
    """Whatever unseen slots hold (NaN, infinities, huge numbers), in the
    sequence's last page, among the new tokens, and where no page is."""
    b = Batch(4, dc, dr, 16, (T, T), (T + 61, 1200), seed=9)
    mask = torch.zeros(2 * T, -(-T // 32), dtype=torch.int32, device="cuda")  # every new token sees the history and itself
    for t in range(T):
        bit = 1 << (t % 32)
        mask[[t, T + t], t // 32] = bit - (1 << 32) if bit >= 1 << 31 else bit
    rows = [np.eye(T, dtype=bool)] * 2
    want, want_lse = b.run(TREE, mask=mask)
    b.check(want, want_lse, TREE, rows)
    for bad in (math.nan, math.inf, -math.inf, 3e38):
        at = b.slots[1][-T:][T // 2]  # a new token of sequence 1
        keep = b.cache.c.view(-1, dc)[at].clone()
        b.cache.c.view(-1, dc)[at, ::3] = bad
        out, lse = b.run(TREE, mask=mask)
        others = [t for t in range(2 * T) if t != T + T // 2]
        assert torch.equal(out[others], want[others]) and torch.equal(lse[:, others], want_lse[:, others])
        if not bad == 3e38:
            assert out[T + T // 2].isnan().any()
        if math.isnan(bad):
            assert out[T + T // 2].isnan().all() and lse[:, T + T // 2].isnan().all()
        b.cache.c.view(-1, dc)[at] = keep
        at = b.slots[0][0]  # a key that all of sequence 0 sees
        keep = b.cache.c.view(-1, dc)[at].clone()
        b.cache.c.view(-1, dc)[at] = math.nan
        out, lse = b.run(TREE, mask=mask)
        assert out[:T].isnan().all() and lse[:, :T].isnan().all() and torch.equal(out[T:], want[T:])
        b.cache.c.view(-1, dc)[at] = keep
    out, lse = b.run(TREE, mask=mask)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_non_finite_query():
    b = Batch(4, 128, 32, 32, (3, 2), (300, 90), seed=10)
    want, _ = b.run()
    b.q[1, 2, 5] = math.nan
    b.q_rope[4, 0, 1] = math.inf
    out, lse = b.run()
    bad = [(1, 2), (4, 0)]
    for t in range(5):
        for h in range(4):
            if (t, h) in bad:
                assert out[t, h].isnan().all() and lse[h, t].isnan()
            else:
                assert torch.equal(out[t, h], want[t, h])


@pytest.mark.parametrize("keys", [1, 64, 65, 9000])
@pytest.mark.parametrize("T", [1, 5])
def test_infinite_query_over_keys_of_one_sign(keys, T):
    """Where every key that a row sees turns an infinity of its q to -inf, the
    softmax has no value: NaN, as with one key of another sign, in whole units
    and in joined ones; a row that sees no key stays 0."""
    b = Batch(4, 64, 16, 64, (T, T), (keys, 20), seed=30)
    for x in (b.cache.c, b.cache.kr):
        x.view(-1, x.shape[-1])[torch.from_numpy(b.slots[0]).cuda(), 3] = 2.0
    none = max(0, T - keys)  # new tokens in front of the first key
    want, want_lse = b.run()
    for part in ("q", "q_rope"):
        for sign in (math.inf, -math.inf):
            x = getattr(b, part)
            keep = x.clone()
            x[:T, 1, 3] = sign
            out, lse = b.run()
            assert out[none:T, 1].isnan().all() and lse[1, none:T].isnan().all()
            assert (out[:none] == 0).all() and (lse[:, :none] == -math.inf).all()
            for h in (0, 2, 3):
                assert torch.equal(out[:T, h], want[:T, h]) and torch.equal(lse[h, :T], want_lse[h, :T])
            assert torch.equal(out[T:], want[T:]) and torch.equal(lse[:, T:], want_lse[:, T:])
            x.copy_(keep)


def test_logits_beyond_fp32_in_a_part_of_the_keys():
    """Keys whose logit falls below fp32's range weigh nothing beside others,
    also where all keys of a part are such."""
    b = Batch(2, 64, 0, 64, (1,), (30000,), seed=31)
    b.q[:] = 0
    b.q[:, :, 0] = 2.0 ** 100
    at = torch.from_numpy(b.slots[0]).cuda()
    b.cache.c.view(-1, 64)[at, 0] = -(2.0 ** 100)
    last = at[29000:29100]
    b.cache.c.view(-1, 64)[last, 0] = 0
    out, lse = b.run(out_dtype=qvg.QVG_OUT_F32)
    want = b.cache.c.view(-1, 64)[last].double().mean(0)
    # equal weights of 1 (exact in bf16), fp32 sums over 30,000 keys
    assert ((out[0].double() - want).abs() <= 30000 * 2.0 ** -23 * b.cache.c.view(-1, 64)[last].double().abs().mean(0) + 1e-30).all()
    assert (lse - math.log(100)).abs().max() <= 2.0 ** -18
    b.cache.c.view(-1, 64)[last, 0] = -(2.0 ** 100)
    out, lse = b.run()
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("kw", [dict(q_scale=30.0), dict(c_scale=2.0 ** -60), dict(c_scale=2.0 ** 60, q_scale=2.0 ** -62), dict(q_scale=2.0 ** -20)])
def test_magnitudes(kw):
    b = Batch(8, 128, 32, 32, (3, 20), (300, 1500), seed=11, **kw)
    out, lse = b.run()
    b.check(out, lse, CAUSAL)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("T", [1, 40])
def test_growing_and_falling_logits(sign, T):
    """The reference moves in many tiles of every part, or starts far from 0."""
    b = Batch(4, 64, 16, 64, (T,), (6000,), seed=12)
    c = torch.zeros(6000, 64, device="cuda")
    c[:, 0] = sign * torch.linspace(1, 3000, 6000, device="cuda")
    c[:, 1:] = torch.randn(6000, 63, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    qvg.latent_append(b.cache, c.bfloat16(), b.kr, b.all_slots)
    b.q[:, :, 0] = 2.0
    out, lse = b.run()
    b.check(out, lse, CAUSAL)


def test_one_key_far_above_the_rest():
    b = Batch(2, 64, 8, 16, (1,), (3000,), seed=13)
    at = int(b.slots[0][1700])
    b.cache.c.view(-1, 64)[at] = 0
    b.cache.c.view(-1, 64)[at, 5] = 4096.0
    b.q[:, :, 5] = 64.0
    out, _ = b.run()
    assert torch.equal(out[0, 0], b.cache.c.view(-1, 64)[at])


def test_strides_uniform_queries_and_rows_behind():
    b = Batch(6, 128, 32, 32, (3, 3), (100, 333), seed=14)
    want, want_lse = b.run()
    b.check(want, want_lse, CAUSAL)
    # heads outermost, as a product per head leaves them; key parts as slices of wider rows
    q = b.q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((6, 6, 32 + 24), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[..., 8:40] = b.q_rope
    out, lse = qvg.latent_attention(b.cache, q, wide[..., 8:40], b.table, b.kv_len, 3, b.scale, want_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # a padded batch: rows from cu_q[B] on are neither read nor written
    pad = lambda x: torch.cat((x, torch.full_like(x, math.nan)))  # noqa: E731
    out = torch.full((12, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    qvg.latent_attention(b.cache, pad(b.q), pad(b.q_rope), b.table, b.kv_len, 3, b.scale, cu_q=b.cu_q, out=out)
    assert torch.equal(out[:6], want) and (out[6:] == 7).all()


def test_same_bits_each_time_on_any_stream_and_in_a_graph():
    b = Batch(16, 256, 64, 16, (1, 1, 20), (4000, 20, 900), seed=15)
    want, want_lse = b.run()
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    got = [b.run(stream=s) for _ in range(4) for s in side]
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    other = Batch(16, 256, 64, 16, (7, 1, 14), (130, 2500, 700), seed=16)
    plain, plain_lse = other.run()
    pages = max(b.cache.num_pages, other.cache.num_pages)
    cache = qvg.LatentKV(256, 64, 16, pages)
    table = torch.zeros(3, max(b.table.shape[1], other.table.shape[1]), dtype=torch.int32, device="cuda")
    q, qr, kv, cu = b.q.clone(), b.q_rope.clone(), b.kv_len.clone(), b.cu_q.clone()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two captured calls, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, qvg.latent_attention(cache, q, qr, table, kv, 20, b.scale, cu_q=cu, want_lse=True)))
    for x, w, l in ((b, want, want_lse), (other, plain, plain_lse), (b, want, want_lse)):
        cache.c[:x.cache.num_pages], cache.kr[:x.cache.num_pages] = x.cache.c, x.cache.kr
        table[:, :x.table.shape[1]] = x.table
        q.copy_(x.q), qr.copy_(x.q_rope), kv.copy_(x.kv_len), cu.copy_(x.cu_q)
        for graph, (o, got_lse) in graphs:
            o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, w) and torch.equal(got_lse, l)


@pytest.mark.parametrize("B,rows,keys", [(1, 128 * 256, 1 << 30), (2, 128 * 128, 1 << 30), (32, 128 * 8, 1 << 30), (33, 128 * 8, 1 << 30),
                                         (40, 128 * 512, 1 << 24), (1000, 128 * 17, 1 << 24)])
def test_a_batch_beyond_the_line_is_refused(B, rows, keys):
    """Batches of 2^32 tiles and more (the fixed cost of a block of rows counted
    in), one sequence or many, are reported and left out: nothing is written, and it takes no time."""
    cost = keys // 64 + 5
    assert B * (rows // 128) * cost >= 2 ** 32 - 1
    cache = qvg.LatentKV(64, 0, 256, 1)
    q = torch.zeros(B * rows, 1, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, keys // 256, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()  # every page the same one
    kv_len = torch.full((B,), keys, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    _, lse = qvg.latent_attention(cache, q, None, table, kv_len, rows, 0.1, out=out, want_lse=True)
    assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG
    assert (out == 7).all()
    kv_len.fill_(100)
    _, lse = qvg.latent_attention(cache, q, None, table, kv_len, rows, 0.1, out=out, want_lse=True)
    assert qvg.get_status() == qvg.QVG_OK
    assert (out == 0).all() and (lse[:, -1] - math.log(100)).abs().max() < 1e-5


def test_bad_device_arguments_are_reported():
    def status(**kw):
        b = Batch(4, 64, 16, 16, (2, 1), (40, 30), seed=17)
        for n, x in kw.items():
            getattr(b, n).copy_(torch.tensor(x, dtype=torch.int32))
        b.run()
        return qvg.get_status()
    assert status() == qvg.QVG_OK
    assert status(kv_len=[49, 30]) == qvg.QVG_ERR_INVALID_ARG  # longer than its table row
    assert status(kv_len=[-1, 30]) == qvg.QVG_ERR_INVALID_ARG
    assert status(table=[[0, 99, 1], [0, 1, 2]]) == qvg.QVG_ERR_INVALID_ARG
    assert status(table=[[0, -1, 1], [0, 1, 2]]) == qvg.QVG_ERR_INVALID_ARG
    assert status(cu_q=[0, 3, 3]) == qvg.QVG_ERR_INVALID_ARG  # 3 new tokens, max_q 2
    assert status(cu_q=[0, 2, 9]) == qvg.QVG_ERR_INVALID_ARG
    assert status(cu_q=[0, 2, 1]) == qvg.QVG_ERR_INVALID_ARG


@pytest.mark.parametrize("T", [1, 40])
def test_wait_timeout_is_reported_and_recovers(T):
    b = Batch(16, 256, 64, 64, (T, 1), (3000, 500), seed=18)
    want, want_lse = b.run()
    qvg.debug_set_wait(1_000_000, True)
    try:
        b.run()
    finally:
        qvg.debug_set_wait(0, False)
    assert qvg.get_status() == qvg.QVG_ERR_TIMEOUT
    assert qvg.get_status() == qvg.QVG_OK
    out, lse = b.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_offsets_past_32_bits():
    """Pages at the end of a cache whose latents pass 2^32 elements."""
    dc, dr, page = 256, 8, 256
    pages = (1 << 32) // (page * dc) + 9
    b = Batch(4, dc, dr, page, (2,), (700,), seed=19)
    want, want_lse = b.run()
    big = qvg.LatentKV(dc, dr, page, pages)
    n = b.cache.num_pages
    slots = b.all_slots + (pages - n) * page
    qvg.latent_append(big, b.c, b.kr, slots)
    out, lse = qvg.latent_attention(big, b.q, b.q_rope, b.table.clamp(min=0) + (pages - n), b.kv_len, 2, b.scale, cu_q=b.cu_q, want_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    c, _ = qvg.latent_read(big, slots)
    assert torch.equal(c, b.c)


# ---- expanded form -----------------------------------------------------------------------

class Prompt:
    def __init__(self, H, dn, dr, dv, nq, past, seed=0, fused=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        total, keys = sum(nq), sum(nq) + sum(past)
        self.H, self.dn, self.dr, self.dv, self.nq, self.past = H, dn, dr, dv, nq, past
        q, kv = rnd(total, H, dn + dr), rnd(keys, H, dn + dv)
        self.q, self.k, self.v = q[..., :dn], kv[..., :dn], kv[..., dn:]
        self.q_rope, self.k_rope = (q[..., dn:], rnd(keys, dr)) if dr else (None, None)
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.kv = [max(0, a + b) for a, b in zip(nq, past)]
        self.cu_q, self.cu_k = starts(nq), starts(self.kv)

    def run(self, mode=CAUSAL, **kw):
        kw.setdefault("want_lse", True)
        return qvg.expanded_attention(self.q, self.q_rope, self.k, self.k_rope, self.v, max(self.nq), cu_q=self.cu_q, cu_k=self.cu_k,
                                      mask_mode=mode, **kw)

    def check(self, out, lse, mode, scale=None):
        q, k = self.q, self.k
        if self.dr:
            q, k = torch.cat((q, self.q_rope), -1), torch.cat((k, self.k_rope[:, None].expand(-1, self.H, -1)), -1)
        q, k, v, got, got_lse = (x.double().cpu().numpy() for x in (q, k, self.v, out, lse))
        q0 = k0 = 0
        for T, L in zip(self.nq, self.kv):
            check_rows(got[q0:q0 + T], got_lse[:, q0:q0 + T], q[q0:q0 + T], k[k0:k0 + L], v[k0:k0 + L], seen(T, L, mode),
                       1 / math.sqrt(self.dn + self.dr) if scale is None else scale, out.dtype == torch.bfloat16)
            q0, k0 = q0 + T, k0 + L


@pytest.mark.parametrize("mode", [NONE, CAUSAL])
@pytest.mark.parametrize("H,dn,dr,dv,nq,past", [
    (1, 64, 0, 64, (1,), (0,)),
    (2, 64, 8, 64, (1, 63, 64, 65), (0, 0, 3, 64)),
    (3, 128, 64, 128, (130, 1, 257), (0, 700, 31)),
    (2, 128, 32, 64, (300, 0, 129), (5, 9, 0)),
    (1, 64, 40, 128, (513, 20), (0, 1000)),
    (2, 128, 0, 128, (127, 128, 256), (1, 64, 300)),
])
def test_prompts(mode, H, dn, dr, dv, nq, past):
    p = Prompt(H, dn, dr, dv, nq, past, seed=dn + dr)
    out, lse = p.run(mode)
    assert qvg.get_status() == qvg.QVG_OK
    p.check(out, lse, mode)
    o32, l32 = p.run(mode, out_dtype=qvg.QVG_OUT_F32, scale=0.2)
    p.check(o32, l32, mode, scale=0.2)


def test_long_prompt():
    p = Prompt(2, 128, 64, 128, (1500,), (900,), seed=20)
    out, lse = p.run()
    p.check(out, lse, CAUSAL)


@pytest.mark.parametrize("dn,dr,dv", [(128, 64, 128), (128, 0, 64), (64, 8, 64)])
@pytest.mark.parametrize("mode", [NONE, CAUSAL])
def test_groups_of_many_blocks(mode, dn, dr, dv):
    """Blocks of two groups over many keys, several a SM one after the other,
    with two stages of K and with more: the second group begins after the first
    one's weights, however far that has got meanwhile."""
    p = Prompt(150, dn, dr, dv, (256, 200, 130), (700, 0, 1300), seed=28)
    out, lse = p.run(mode)
    for _ in range(10):
        again, again_lse = p.run(mode)
        assert torch.equal(again, out) and torch.equal(again_lse, lse)
    assert qvg.get_status() == qvg.QVG_OK
    p.H, keep = 3, [0, 77, 149]
    p.q, p.k, p.v = (x[:, keep] for x in (p.q, p.k, p.v))
    p.q_rope = p.q_rope[:, keep] if dr else None
    p.check(out[:, keep], lse[keep], mode)


@pytest.mark.parametrize("rows", [1, 129, 140])
def test_a_group_with_far_fewer_keys(rows):
    """Blocks whose second group has no row, or a few, beside a first one over
    many keys, and one whose first group sees far less: the group that is done
    gives back the stages that it has no use for."""
    p = Prompt(160, 128, 64, 128, (rows, 256), (2500, -100), seed=33)
    out, lse = p.run()
    for _ in range(5):
        again, again_lse = p.run()
        assert torch.equal(again, out) and torch.equal(again_lse, lse)
    assert qvg.get_status() == qvg.QVG_OK
    p.H, keep = 2, [0, 159]
    p.q, p.k, p.v, p.q_rope = (x[:, keep] for x in (p.q, p.k, p.v, p.q_rope))
    p.check(out[:, keep], lse[keep], CAUSAL)


@pytest.mark.parametrize("B", [20, 300, 1200])
def test_many_ragged_prompts(B):
    """Blocks of rows that are ranked by length, and more of them than that."""
    nq = tuple((37 * i) % 90 if i % 11 else 300 for i in range(B))
    p = Prompt(2, 64, 8, 64, nq, tuple((13 * i) % 70 for i in range(B)), seed=B)
    out, lse = p.run()
    p.check(out, lse, CAUSAL)
    p.cu_k[5] = p.cu_k[4] - 1  # a length below 0
    p.run()
    assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG


@pytest.mark.parametrize("B", [1, 2])
@pytest.mark.parametrize("nq,bound", [(700, 65536), (700, 65537), (700, 131072), (3000, 1 << 30), (1, 100000), (70000, 100000)])
def test_prompts_below_a_loose_bound(B, nq, bound):
    """max_q far above the new tokens that there are (a captured call's bound):
    every row is computed, and nothing behind them."""
    p = Prompt(1, 64, 0, 64, (nq,) * B, (0,) * B, seed=29)
    want, want_lse = p.run()
    out = torch.full((B * nq, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    call = lambda: qvg.expanded_attention(p.q, None, p.k, None, p.v, bound, cu_q=p.cu_q, cu_k=p.cu_k, out=out, want_lse=True)  # noqa: E731
    _, lse = call()
    assert qvg.get_status() == qvg.QVG_OK
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    if nq <= 3000:
        p.check(out, lse, CAUSAL)
    p.cu_q[B] = B * nq + 1  # a row that is not there
    call()
    assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG


def test_prompts_with_more_new_tokens_than_keys():
    p = Prompt(2, 64, 16, 64, (300, 40, 7), (-200, -40, -3), seed=21)  # 100, 0 and 4 keys
    for mode in (NONE, CAUSAL):
        out, lse = p.run(mode)
        p.check(out, lse, mode)
    none = Prompt(1, 64, 0, 64, (5,), (-5,), seed=22)  # no keys at all
    out, lse = none.run()
    assert (out == 0).all() and (lse == -math.inf).all()


def test_prompts_strides_uniform_and_rows_behind():
    p = Prompt(3, 64, 16, 128, (70, 70), (20, 20), seed=23)
    want, want_lse = p.run()
    p.check(want, want_lse, CAUSAL)
    q = Prompt(3, 64, 16, 128, (70, 70), (20, 20), seed=23, fused=False)
    heads = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    out, lse = qvg.expanded_attention(heads(q.q), q.q_rope, q.k, q.k_rope, heads(q.v), 70, max_k=90, want_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    pad = lambda x: torch.cat((x, torch.full_like(x, math.nan)))  # noqa: E731
    out = torch.full((280, 3, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    qvg.expanded_attention(pad(p.q), pad(p.q_rope), pad(p.k), pad(p.k_rope), pad(p.v), 70, cu_q=p.cu_q, cu_k=p.cu_k, out=out)
    assert torch.equal(out[:140], want) and (out[140:] == 7).all()


def test_prompt_keys_that_are_not_seen():
    """NaN in keys and values after a row's last key, and in the next
    sequence, does not reach it; rows that see it become NaN."""
    p = Prompt(2, 64, 16, 64, (200, 90), (0, 10), seed=24)
    want, want_lse = p.run()
    for name in ("k", "v"):
        for bad in (math.nan, math.inf):
            x = getattr(p, name)
            keep = x[150].clone()
            x[150, :, 7] = bad
            out, lse = p.run()
            assert torch.equal(out[:150], want[:150]) and torch.equal(lse[:, :150], want_lse[:, :150])
            assert torch.equal(out[200:], want[200:])
            if math.isnan(bad):
                assert out[150:200].isnan().any(-1).all()
            x[150] = keep
    p.v[200] = math.nan  # the first key of the second sequence
    out, lse = p.run()
    assert torch.equal(out[:200], want[:200]) and out[200:].isnan().all()


@pytest.mark.parametrize("dr", [0, 16])
@pytest.mark.parametrize("part", ["q", "q_rope"])
@pytest.mark.parametrize("sign", [math.inf, -math.inf])
def test_infinite_query_of_prompts(part, sign, dr):
    """NaN whatever the signs of the keys that a row sees (a prompt's first row
    sees one); a row that sees none stays 0."""
    if part == "q_rope" and dr == 0:
        return
    p = Prompt(2, 64, dr, 64, (300, 7, 5), (0, 70, -3), seed=32)
    (p.k[:, :, 3] if part == "q" else p.k_rope[:, 3:4]).fill_(2.0)
    want, want_lse = p.run()
    getattr(p, part)[:, 1, 3] = sign
    out, lse = p.run()
    none = slice(307, 310)  # (5 new tokens, 2 keys)
    assert (out[none] == 0).all() and (lse[:, none] == -math.inf).all()
    assert torch.equal(out[:, 0], want[:, 0]) and torch.equal(lse[0], want_lse[0])
    some = [t for t in range(312) if not 307 <= t < 310]
    assert out[some, 1].isnan().all() and lse[1, some].isnan().all()


def test_prompts_on_streams_in_a_graph_and_out_of_time():
    p = Prompt(4, 128, 64, 128, (300, 5, 140), (0, 40, 200), seed=25)
    want, want_lse = p.run()
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    got = [p.run(stream=s) for _ in range(3) for s in side]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(l, want_lse) for o, l in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = p.run()
    p.cu_q.copy_(starts([100, 5, 340])), p.cu_k.copy_(starts([60, 45, 580]))  # other lengths; 340 > max_q
    graph.replay()
    assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG
    p.cu_q.copy_(starts(p.nq)), p.cu_k.copy_(starts(p.kv))
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(l, want_lse) and qvg.get_status() == qvg.QVG_OK
    qvg.debug_set_wait(1_000_000, True)
    try:
        p.run()
    finally:
        qvg.debug_set_wait(0, False)
    assert qvg.get_status() == qvg.QVG_ERR_TIMEOUT
    out, _ = p.run()
    assert qvg.get_status() == qvg.QVG_OK and torch.equal(out, want)


def test_both_forms_agree():
    """The absorbed form over cached latents is the expanded form over keys and
    values projected from them, with the key projections in the queries and the value
    projections after: a layer in 64 bits, each form within the roundings of its own bf16 inputs."""
    H, dc, dr, dn, dv, L, T = 4, 128, 32, 64, 64, 300, 20
    g = torch.Generator(device="cuda").manual_seed(26)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    c, kr, wk, wv = rnd(L, dc).bfloat16(), rnd(L, dr).bfloat16(), rnd(H, dn, dc) / math.sqrt(dc), rnd(H, dv, dc) / math.sqrt(dc)
    q, qr = rnd(T, H, dn).bfloat16(), rnd(T, H, dr).bfloat16()
    scale = 1 / math.sqrt(dn + dr)
    k, v = torch.einsum("lc,hnc->lhn", c.double(), wk), torch.einsum("lc,hnc->lhn", c.double(), wv)
    x = (torch.einsum("thn,lhn->htl", q.double(), k) + torch.einsum("thr,lr->htl", qr.double(), kr.double())) * scale
    x = x.masked_fill(torch.arange(L, device="cuda")[None] > torch.arange(T, device="cuda")[:, None] + L - T, -math.inf)
    p = torch.softmax(x, -1)
    want = torch.einsum("htl,lhn->thn", p, v)
    mean = torch.einsum("htl,lhn->thn", p, v.abs())
    cache = qvg.LatentKV(dc, dr, 64, 8)
    qvg.latent_append(cache, c, kr, torch.arange(L, device="cuda"))
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None].contiguous()
    kv_len = torch.tensor([L], dtype=torch.int32, device="cuda")
    q_abs = torch.einsum("thn,hnc->thc", q.double(), wk)
    o, _ = qvg.latent_attention(cache, q_abs.bfloat16(), qr, table, kv_len, T, scale, out_dtype=qvg.QVG_OUT_F32)
    got = torch.einsum("thc,hnc->thn", o.double(), wv)
    # The rounding of q_abs moves a logit by at most 2^-8 scale |q_abs| |c|, a weight by twice that of itself, plus 2^-8 (and
    # fp32's) for its own rounding; an output by that share of the mean of |c| through |wv|.
    dl = 2.0 ** -8 * scale * torch.einsum("thc,lc->htl", q_abs.abs(), c.double().abs()).amax(-1).t()
    size = torch.einsum("htl,lc,hnc->thn", p, c.double().abs(), wv.abs())
    assert ((got - want).abs() <= ((2 * dl + 2.0 ** -8 + 2.0 ** -12)[..., None] * size)).all()
    o, _ = qvg.expanded_attention(q, qr, k.bfloat16(), kr, v.bfloat16(), T, max_k=L, out_dtype=qvg.QVG_OUT_F32)
    # likewise: k's rounding in the logits, v's and the weights' in the sum
    dl = 2.0 ** -8 * scale * torch.einsum("thn,lhn->htl", q.double().abs(), k.abs()).amax(-1).t()
    assert ((o.double() - want).abs() <= (2 * dl + 2 * 2.0 ** -8 + 2.0 ** -12)[..., None] * mean).all()


def test_a_run_of_calls():
    """Append a prompt, attend to it in the expanded form, then drafted tokens:
    room, append, tree mask, absorbed attention, the accepted ones moved
    together, the rest given back, and another token: the last attention is
    that of the accepted sequence written in one go."""
    dc, dr, page, H = 128, 32, 16, 4
    g = torch.Generator(device="cuda").manual_seed(27)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    plan = qvg.RopePlan((32,))
    cache, pool = qvg.LatentKV(dc, dr, page, 40), qvg.PagePool(40)
    table = torch.zeros(2, 12, dtype=torch.int32, device="cuda")
    kv_len = torch.zeros(2, dtype=torch.int32, device="cuda")
    lens, drafts, path = (70, 33), (6, 4), ((0, 2, 5), (1,))
    c, kr = rnd(sum(lens), dc), rnd(sum(lens), dr)
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    slots, copies = qvg.pages_reserve(pool, page, table, kv_len, cu_new=starts(lens), total=sum(lens))
    qvg.pages_copy(cache, copies)
    qvg.latent_append(cache, c, kr, slots, plan=plan, positions=pos)
    parents = torch.tensor([-1, 0, 0, 1, 2, 2, -1, -1, 1, 1], dtype=torch.int32, device="cuda")
    depth = torch.tensor([0, 1, 1, 2, 2, 2, 0, 0, 1, 1])
    dpos = (torch.repeat_interleave(torch.tensor(lens), torch.tensor(drafts)) + depth).int().cuda()
    dc_, dkr = rnd(10, dc), rnd(10, dr)
    slots, copies = qvg.pages_reserve(pool, page, table, kv_len, cu_new=starts(drafts), total=10)
    qvg.latent_append(cache, dc_, dkr, slots, plan=plan, positions=dpos)
    mask = qvg.tree_mask(parents, 6, cu_q=starts(drafts))
    q, qr = rnd(10, H, dc), rnd(10, H, dr)
    drafted, _ = qvg.latent_attention(cache, q, qr, table, kv_len, 6, 0.1, cu_q=starts(drafts), mask_mode=TREE, mask=mask)
    keep = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    for b in range(2):
        keep[b, :len(path[b])] = torch.tensor([lens[b] + i for i in path[b]])
    n_keep = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    qvg.paged_compact(cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), keep, n_keep)
    qvg.pages_release(pool, page, table, kv_len, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                      keep=torch.tensor([73, 34], dtype=torch.int32, device="cuda"))
    slots, copies = qvg.pages_reserve(pool, page, table, kv_len)
    last_c, last_kr = rnd(2, dc), rnd(2, dr)
    qvg.latent_append(cache, last_c, last_kr, slots, plan=plan, positions=kv_len - 1)
    q1, qr1 = rnd(2, H, dc), rnd(2, H, dr)
    out, lse = qvg.latent_attention(cache, q1, qr1, table, kv_len, 1, 0.1, want_lse=True)
    assert qvg.get_status() == qvg.QVG_OK and kv_len.tolist() == [74, 35]
    assert int((pool.refs > 0).sum()) == 5 + 3 and int(pool.refs.max()) == 1
    # the same tokens written in one go, on other pages
    plain = qvg.LatentKV(dc, dr, page, 12)
    t2 = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)
    first = (0, 70)
    for b in range(2):
        d0 = 0 if b == 0 else 6
        cc = torch.cat([c[first[b]:first[b] + lens[b]], dc_[[d0 + i for i in path[b]]], last_c[b:b + 1]])
        kk = torch.cat([kr[first[b]:first[b] + lens[b]], dkr[[d0 + i for i in path[b]]], last_kr[b:b + 1]])
        n = len(cc)
        at = t2[b, torch.arange(n, device="cuda") // page].long() * page + torch.arange(n, device="cuda") % page
        qvg.latent_append(plain, cc, kk, at, plan=plan, positions=torch.arange(n, dtype=torch.int32, device="cuda"))
    want, want_lse = qvg.latent_attention(plain, q1, qr1, t2, kv_len, 1, 0.1, want_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert torch.isfinite(drafted.float()).all()
