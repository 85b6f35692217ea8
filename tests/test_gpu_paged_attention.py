"""Attention over the paged cache on the GPU, against the plain 64-bit form
over what the cache holds (tests/_paged.py)."""
import math

import numpy as np
import pytest
import torch

import video_diffusion_kv_gb300 as qvg

import _paged as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert qvg.get_status() == qvg.QVG_OK


class Batch:
    """A cache with B sequences on shuffled pages, and their new tokens' q.
    Slots of no sequence hold bytes that are no numbers (codes and scales
    0xFF), as does each last page behind its sequence."""

    def __init__(self, H, G, d, bits, page, nq, kv, seed=0, k_scale=1.0, v_scale=1.0, q_scale=1.0):
        g = np.random.default_rng(seed)
        need = [-(-n // page) for n in kv]
        pages = sum(need) + 2
        order = g.permutation(pages)
        self.H, self.G, self.d, self.nq, self.kv, self.page = H, G, d, nq, kv, page
        self.cache = qvg.PagedKV(H, d, page, pages, bits)
        for t in (self.cache.k_codes, self.cache.k_scales, self.cache.v_codes, self.cache.v_scales):
            t.fill_(0xFF)
        table = np.full((len(kv), max(need + [1])), -7, np.int32)  # entries past the last page are not read
        self.slots, at = [], 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
            t = np.arange(kv[b])
            self.slots.append(table[b, t // page].astype(np.int64) * page + t % page)
        rows = sum(kv)
        if rows:
            bf = lambda s: torch.from_numpy(g.standard_normal((rows, H, d)) * s).to("cuda", torch.bfloat16)  # noqa: E731
            spread = np.exp2(g.integers(-3, 4, size=(rows, H, 1)) * 0.5)
            self.k, self.v = bf(k_scale * spread), bf(v_scale * spread[:, :, ::-1])
            qvg.paged_append(self.cache, self.k, self.v, torch.from_numpy(np.concatenate(self.slots)).cuda())
        self.table = torch.from_numpy(table).cuda()
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")
        self.cu_q = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32, device="cuda")
        self.q = torch.from_numpy(g.standard_normal((sum(nq), H * G, d)) * q_scale).to("cuda", torch.bfloat16)

    def see(self, b, mode, rows=None):
        T, L = self.nq[b], self.kv[b]
        j = np.arange(L)[None] - (L - T)
        t = np.arange(T)[:, None]
        if mode == qvg.QVG_MASK_NONE:
            return np.ones((T, L), bool)
        if mode == qvg.QVG_MASK_CAUSAL:
            return j <= t
        return np.where(j < 0, True, rows[t, np.clip(j, 0, T - 1)])

    def check(self, out, lse, mode, rows=None, scale=None, nan_ok=False):
        """Every row against the plain form.  Bounds, per row (p: the weights):
        a logit is off by
          D = scale (2^-21 max|q| sum|k| + 2 d 2^-23 sum |q||k|) + 8 2^-24 |s|
        (Q's fp8 pair, 2^-17 with many rows; fp32 sums of 2 d products; the base-2 form's roundings
        of the logit), so a weight by 2 D + 2^-20 (2^x) of itself; a weight
        times V's scale by 2^-11 (fp16) and 2^-9 (three e5m2 parts) more or,
        far below the largest, by 2^-25 of the largest (half of e5m2's smallest
        step, 2^-17, against 2^8), against codes up to twice the largest's
        own; sums over the keys: L 2^-24."""
        k_all, v_all = (x.transpose(0, 2, 1, 3).reshape(-1, self.H, self.d) for x in ref.held(self.cache))
        got, q = out.double().cpu().numpy(), self.q.double().cpu().numpy()
        got_lse = None if lse is None else lse.double().cpu().numpy()
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        rows_in_block = max(self.nq) * self.G
        q_step = 2.0 ** -21 if rows_in_block <= (64 if self.cache.bits == 8 else 32) else 2.0 ** -17
        half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
        first = 0
        for b, T in enumerate(self.nq):
            k, v = k_all[self.slots[b]], v_all[self.slots[b]]
            see = self.see(b, mode, None if rows is None else rows[b])
            for t in range(T):
                js = np.nonzero(see[t])[0]
                row = got[first + t]
                if len(js) == 0:
                    assert (row == 0).all() and (got_lse is None or (got_lse[:, first + t] == -np.inf).all())
                    continue
                kk, vv = np.repeat(k[js], self.G, 1).transpose(1, 0, 2), np.repeat(v[js], self.G, 1).transpose(1, 0, 2)
                qq = q[first + t][:, None]
                s = (kk * qq).sum(-1) * scale
                m = s.max(-1, keepdims=True)
                p = np.exp(s - m)
                den = p.sum(-1, keepdims=True)
                want, want_lse = ((p / den)[..., None] * vv).sum(1), (m + np.log(den))[:, 0]
                dd = scale * (q_step * np.abs(qq).max(-1) * np.abs(kk).sum(-1) + 2 * self.d * 2.0 ** -23 * np.abs(kk * qq).sum(-1))
                dd = (dd + 8 * 2.0 ** -24 * np.abs(s)).max(-1, keepdims=True)
                rel = 2 * dd + 2.0 ** -20 + 2.0 ** -11 + 2.0 ** -9 + len(js) * 2.0 ** -24
                mean = ((p / den)[..., None] * np.abs(vv)).sum(1)
                lost = len(js) * 2.0 ** -24 * np.abs((p / den)[..., None] * np.abs(vv).max(-1, keepdims=True)).max(1)
                bound = rel * mean + lost + half * np.abs(want) + 1e-37
                err = np.abs(row - want)
                assert (err <= bound).all(), (b, t, float((err / bound).max()))
                if got_lse is not None:
                    lb = dd[:, 0] + 2.0 ** -20 + len(js) * 2.0 ** -24 + 2.0 ** -21 * np.abs(want_lse)
                    e = np.abs(got_lse[:, first + t] - want_lse)
                    assert (e <= lb).all(), (b, t, float((e / lb).max()))
            first += T

    def run(self, mode=qvg.QVG_MASK_CAUSAL, **kw):
        kw.setdefault("want_lse", True)
        kw.setdefault("cu_q", self.cu_q)
        return qvg.paged_attention(self.cache, self.q, self.table, self.kv_len, max(self.nq), mask_mode=mode, **kw)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,G,page,nq,kv", [
    (1, 1, 16, (1,), (1,)),
    (2, 1, 16, (1, 1, 1, 1), (1, 127, 128, 129)),
    (3, 4, 32, (1, 1, 1), (300, 17, 1000)),
    (2, 7, 64, (1, 3, 2), (64, 700, 65)),
    (1, 8, 128, (5,), (513,)),
    (2, 2, 256, (9, 16), (255, 1030)),
])
def test_decode_shapes(bits, d, H, G, page, nq, kv):
    """A few new tokens, causal, at lengths around the tile and the page."""
    b = Batch(H, G, d, bits, page, nq, kv, seed=d + bits)
    out, lse = b.run()
    assert qvg.get_status() == qvg.QVG_OK
    b.check(out, lse, qvg.QVG_MASK_CAUSAL)
    o32, _ = b.run(out_dtype=qvg.QVG_OUT_F32)
    b.check(o32, None, qvg.QVG_MASK_CAUSAL)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("mode", [qvg.QVG_MASK_NONE, qvg.QVG_MASK_CAUSAL, qvg.QVG_MASK_TREE])
@pytest.mark.parametrize("H,G,d,page,nq,kv", [
    (2, 1, 128, 16, (33, 1, 64), (33, 1, 200)),   # no history at all
    (1, 4, 64, 64, (40, 7), (400, 90)),           # several row blocks
    (2, 8, 128, 32, (25,), (1000,)),
    (1, 3, 128, 128, (1, 65, 2, 31), (5, 1100, 129, 640)),
])
def test_masks(bits, mode, H, G, d, page, nq, kv):
    g = np.random.default_rng(1)
    b = Batch(H, G, d, bits, page, nq, kv, seed=2)
    mask, rows = None, None
    if mode == qvg.QVG_MASK_TREE:
        parents = [np.array([g.integers(-1, t) if t else -1 for t in range(T)], np.int32) for T in nq]
        rows = [ref.tree_rows(p) for p in parents]
        mask = qvg.tree_mask(torch.from_numpy(np.concatenate(parents)).cuda(), max(nq), cu_q=b.cu_q)
        bits_of = mask.cpu().numpy().view(np.uint32)
        first = 0
        for r in rows:
            for t in range(len(r)):
                got = [(bits_of[first + t, j >> 5] >> (j & 31)) & 1 for j in range(mask.shape[1] * 32)]
                assert got[:len(r)] == list(r[t].astype(int)) and not any(got[len(r):])
            first += len(r)
    out, lse = b.run(mode, mask=mask)
    assert qvg.get_status() == qvg.QVG_OK
    b.check(out, lse, mode, rows)


def test_rows_that_see_nothing():
    """Mask rows of zeros over a sequence with no history, and kv_len 0."""
    b = Batch(2, 2, 128, 8, 16, (5, 3, 4), (5, 0, 200), seed=3)
    rows = [np.eye(5, dtype=bool), np.zeros((3, 3), bool), np.tri(4, dtype=bool)]
    rows[0][[1, 4]] = False
    words = np.zeros((12, 1), np.uint32)
    for i, r in enumerate(np.concatenate([np.pad(r, ((0, 0), (0, 32 - r.shape[1]))) for r in rows])):
        words[i, 0] = sum(int(x) << j for j, x in enumerate(r))
    mask = torch.from_numpy(words.view(np.int32)).cuda()
    out, lse = b.run(qvg.QVG_MASK_TREE, mask=mask)
    assert qvg.get_status() == qvg.QVG_OK
    o, l = out.cpu(), lse.cpu()
    for i in (1, 4, 5, 6, 7):
        assert (o[i] == 0).all() and (l[:, i] == -math.inf).all()
    b.nq, b.kv, b.slots = (5, 3, 4), (5, 0, 200), b.slots
    b.check(out, lse, qvg.QVG_MASK_TREE, rows)


@pytest.mark.parametrize("bits", [8, 4])
def test_unseen_keys_have_no_influence(bits):
    """Infinities and NaN in the K and V rows of masked drafts change no row
    that does not see them; rows that do are NaN."""
    b = Batch(2, 2, 64, bits, 32, (6, 3), (70, 200), seed=4)
    mask = torch.tensor([[1 << t] for t in range(6)] + [[1], [3], [7]], dtype=torch.int32, device="cuda")
    want, want_lse = b.run(qvg.QVG_MASK_TREE, mask=mask)
    bad = torch.full((2, 2, 64), 1.0, dtype=torch.bfloat16, device="cuda")
    bad[0, :, 3], bad[1, :, 60] = math.inf, math.nan
    at = torch.from_numpy(b.slots[0][[64 + 1, 64 + 4]]).cuda()
    good = torch.zeros_like(bad)
    for k, v in ((bad, good), (good, bad), (bad, bad)):
        qvg.paged_append(b.cache, k, v, at)
        out, lse = b.run(qvg.QVG_MASK_TREE, mask=mask)
        keep = [i for i in range(9) if i not in (1, 4)]
        assert torch.equal(out[keep], want[keep]) and torch.equal(lse[:, keep], want_lse[:, keep])
        assert out[[1, 4]].isnan().all()
    assert qvg.get_status() == qvg.QVG_OK


def test_slots_never_written():
    """New tokens whose slots hold codes and scales that are no numbers change
    no row that does not see them."""
    b = Batch(2, 2, 128, 8, 32, (6,), (70,), seed=21)
    mask = torch.tensor([[1 << t] for t in range(6)], dtype=torch.int32, device="cuda")
    want, want_lse = b.run(qvg.QVG_MASK_TREE, mask=mask)
    for s in b.slots[0][[64 + 1, 64 + 4]]:
        for t in (b.cache.k_codes, b.cache.v_codes):
            t[s // 32, :, s % 32] = torch.randint(0, 256, (2, 128), device="cuda").to(torch.uint8) | 0x7E
    out, lse = b.run(qvg.QVG_MASK_TREE, mask=mask)
    keep = [0, 2, 3, 5]
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[:, keep], want_lse[:, keep])


def test_non_finite_query():
    b = Batch(2, 4, 128, 8, 16, (3,), (300,), seed=5)
    want, _ = b.run()
    b.q[1, 2, 7], b.q[2, 5, 0] = math.nan, math.inf
    out, lse = b.run()
    nan = torch.zeros(3, 8, dtype=torch.bool)
    nan[1, 2], nan[2, 5] = True, True
    assert (out.cpu().isnan().all(-1) == nan).all() and (lse.cpu().isnan().t() == nan).all()
    assert torch.equal(out.cpu()[~nan], want.cpu()[~nan])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kw", [dict(k_scale=30.0), dict(v_scale=2.0 ** -20), dict(v_scale=2.0 ** 30), dict(q_scale=2.0 ** 20, k_scale=2.0 ** -18),
                                dict(k_scale=2.0 ** -30)])
def test_magnitudes(bits, kw):
    """Peaked and flat rows, V far from 1, large Q with small K."""
    b = Batch(1, 2, 128, bits, 64, (2, 1), (900, 300), seed=6, **kw)
    out, lse = b.run()
    b.check(out, lse, qvg.QVG_MASK_CAUSAL)


def test_channels_of_unlike_size():
    """Q rows whose channels span 2^14, in one block with rows 2^12 larger."""
    b = Batch(1, 4, 128, 8, 16, (4,), (400,), seed=7)
    g = torch.Generator(device="cuda").manual_seed(1)
    b.q *= torch.exp2(torch.randint(-14, 1, (128,), generator=g, device="cuda").float()).bfloat16()
    b.q[:, 1] *= 2.0 ** -12
    out, lse = b.run()
    b.check(out, lse, qvg.QVG_MASK_CAUSAL)


def test_one_key_far_above_the_rest():
    """A first token that takes nearly all weight, and many keys 2^-18 and
    less below it, all pointing the same way: their sum still counts."""
    b = Batch(1, 1, 64, 8, 128, (1,), (60000,), seed=8, k_scale=2.0 ** -6)
    first = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    first[0, 0, 0] = 13.0 * 8
    v = first * 0 + 1.0
    qvg.paged_append(b.cache, first, -v, torch.from_numpy(b.slots[0][:1]).cuda())
    rest = torch.from_numpy(b.slots[0][1:]).cuda()
    k = torch.zeros(len(rest), 1, 64, dtype=torch.bfloat16, device="cuda")
    qvg.paged_append(b.cache, k, k + 1.0, rest)
    b.q.fill_(0)
    b.q[0, 0, 0] = 1.0
    out, lse = b.run(out_dtype=qvg.QVG_OUT_F32)
    b.check(out, lse, qvg.QVG_MASK_CAUSAL)
    assert float(out[0, 0, 0]) > -0.8  # the rest's share is 0.12


def test_growing_logits():
    """Keys whose logits climb from tile to tile: references are raised many
    times, in one CTA's run and across cuts."""
    for L in (3000, 40000):
        b = Batch(1, 2, 128, 8, 64, (2,), (L,), seed=9)
        t = torch.arange(L, device="cuda")
        k = torch.randn(L, 1, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
        k[:, 0, 0] = t / L * 400.0
        qvg.paged_append(b.cache, k.bfloat16(), b.v, torch.from_numpy(b.slots[0]).cuda())
        b.q[:, 0, 0], b.q[:, 1, 0] = 1.0, -2.0
        out, lse = b.run()
        b.check(out, lse, qvg.QVG_MASK_CAUSAL)


@pytest.mark.parametrize("bits", [8, 4])
def test_long_and_ragged(bits):
    """Cut units: few long sequences, and many ragged ones."""
    b = Batch(2, 4, 128, bits, 16, (1, 4), (20011, 9000), seed=10)
    out, lse = b.run()
    b.check(out, lse, qvg.QVG_MASK_CAUSAL)
    g = np.random.default_rng(11)
    kv = [int(x) for x in g.integers(1, 700, size=600)]
    b = Batch(1, 2, 64, bits, 32, [1] * 600, kv, seed=11)
    out, lse = b.run()
    b.check(out, lse, qvg.QVG_MASK_CAUSAL)


def test_uniform_queries_strides_scale():
    """cu_q left out, q as a view of a fused projection, a scale of its own,
    outputs and workspace given."""
    b = Batch(2, 2, 128, 8, 64, (3, 3), (100, 260), seed=12)
    wide = torch.zeros(6, 9, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:6] = b.q
    ws = torch.empty(qvg.paged_workspace_size(b.cache, 4, 2, 3), dtype=torch.uint8, device="cuda")
    out = torch.empty(6, 4, 128, dtype=torch.float32, device="cuda")
    got, lse = qvg.paged_attention(b.cache, wide[:, 2:6], b.table, b.kv_len, 3, scale=0.25, out_dtype=qvg.QVG_OUT_F32,
                                   want_lse=True, out=out, workspace=ws)
    assert got is out
    b.check(out, lse, qvg.QVG_MASK_CAUSAL, scale=0.25)


def test_rows_behind_the_last_sequence():
    """A padded batch: rows of q, out and mask past cu_q[B] stay as they were;
    a sequence without new tokens takes no row."""
    b = Batch(1, 2, 64, 8, 16, (2, 0, 3), (50, 20, 40), seed=13)
    q = torch.full((9, 2, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    q[:5] = b.q
    out = torch.full((9, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    qvg.paged_attention(b.cache, q, b.table, b.kv_len, 4, cu_q=b.cu_q, out=out)
    assert (out[5:] == 5).all()
    b.check(out[:5], None, qvg.QVG_MASK_CAUSAL)
    parents = torch.full((9,), -1, dtype=torch.int32, device="cuda")
    mask = torch.full((9, 2), 77, dtype=torch.int32, device="cuda")
    qvg.tree_mask(parents, 4, cu_q=b.cu_q, out=mask)
    assert (mask[5:] == 77).all() and mask[:5].tolist() == [[1, 0], [2, 0], [1, 0], [2, 0], [4, 0]]


def test_bad_device_arguments_are_reported():
    """Pages outside the cache, lengths past the table, more new tokens than
    promised, parents that do not come first: reported once, nothing else
    breaks, and the next call is clean."""
    b = Batch(2, 1, 64, 8, 16, (1, 2, 1), (40, 100, 30), seed=14)
    good, _ = b.run()
    assert qvg.get_status() == qvg.QVG_OK
    for what in ("page", "negative page", "length", "negative length", "queries", "descending"):
        table, kv, cu = b.table.clone(), b.kv_len.clone(), b.cu_q.clone()
        if what == "page":
            table[1, 3] = b.cache.num_pages
        if what == "negative page":
            table[1, 0] = -1
        if what == "length":
            kv[1] = 16 * table.shape[1] + 1
        if what == "negative length":
            kv[1] = -5
        if what == "queries":
            cu[2] = cu[3] = 5  # more than there are rows
        if what == "descending":
            cu[3] = 2
        out, _ = qvg.paged_attention(b.cache, b.q, table, kv, 2, cu_q=cu)
        assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG, what
        assert torch.equal(out[0], good[0]), what
    parents = torch.tensor([0, -1, 1, -2], dtype=torch.int32, device="cuda")
    mask = qvg.tree_mask(parents, 2, cu_q=b.cu_q)
    assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG
    assert mask[:, 0].tolist() == [1, 1, 2, 1]
    again, _ = b.run()
    assert qvg.get_status() == qvg.QVG_OK and torch.equal(again, good)


def test_wait_timeout_is_reported_and_recovers():
    """The library's bounded-wait hook: every CTA stops, TMEM and copies in
    flight are waited for, the status says so once, the next call is whole."""
    b = Batch(2, 4, 128, 8, 64, (3, 1), (3000, 500), seed=15)
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


def test_same_bits_each_time_on_any_stream():
    b = Batch(2, 4, 128, 8, 16, (1, 1, 6), (4000, 20, 900), seed=16)
    want, want_lse = b.run()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):  # two calls at once, a workspace each
        got += [b.run(stream=s) for s in side]
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, want_lse)


def test_captured_call_with_other_lengths():
    """One captured step (rotate, append, tree mask, attention) replayed with
    other lengths, tables, slots and drafts gives the bits of a plain call."""
    plan = qvg.RopePlan((64, 32, 32))
    a, b = (Batch(2, 2, 128, 8, 32, nq, kv, seed=s) for nq, kv, s in (((4, 2), (40, 300), 17), ((1, 5), (600, 170), 18)))
    assert a.q.shape == b.q.shape
    pages = max(a.cache.num_pages, b.cache.num_pages)
    width = max(a.table.shape[1], b.table.shape[1])
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = torch.randn(6, 2, 2, 128, device="cuda", generator=g).bfloat16()
    pos = torch.randint(0, 999, (6, 3), device="cuda", generator=g, dtype=torch.int32)

    def inputs(x):
        big = qvg.PagedKV(2, 128, 32, pages)
        for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
            getattr(big, n)[:x.cache.num_pages] = getattr(x.cache, n)
        table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
        table[:, :x.table.shape[1]] = x.table.clamp(min=0)
        new = np.concatenate([x.slots[i][x.kv[i] - x.nq[i]:] for i in range(2)])
        parents = torch.tensor([t - 1 if t % 3 else -1 for n in x.nq for t in range(n)], dtype=torch.int32, device="cuda")
        return big, table, torch.from_numpy(new).cuda(), parents

    def step(cache, q, table, slots, parents, kv_len, cu_q):
        rq = qvg.rope(plan, q, pos)
        qvg.paged_append(cache, kv[:, 0], kv[:, 1], slots, plan=plan, positions=pos)
        mask = qvg.tree_mask(parents, 5, cu_q=cu_q)
        return qvg.paged_attention(cache, rq, table, kv_len, 5, cu_q=cu_q, mask_mode=qvg.QVG_MASK_TREE, mask=mask, want_lse=True)

    sets = []
    for x in (a, b):
        cache, table, slots, parents = inputs(x)
        sets.append((cache, x.q, table, slots, parents, x.kv_len, x.cu_q))
    want = [step(*s) for s in sets]
    static = [qvg.PagedKV(2, 128, 32, pages)] + [torch.zeros_like(t) for t in sets[0][1:]]
    static[5].fill_(1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = step(*static)
    for s, (o, l) in zip(sets, want):
        for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
            getattr(static[0], n).copy_(getattr(s[0], n))
        for d, t in zip(static[1:], s[1:]):
            d.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, l)
    assert qvg.get_status() == qvg.QVG_OK


def test_offsets_past_32_bits():
    """Pages at the end of a cache whose codes pass 4 GB."""
    H, d, page = 8, 128, 128
    pages = (1 << 32) // (H * page * d) + 9
    b = Batch(H, 1, d, 8, page, (2,), (700,), seed=19)
    want, want_lse = b.run()
    big = qvg.PagedKV(H, d, page, pages, 8)
    n = b.cache.num_pages
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(big, name)[-n:] = getattr(b.cache, name)
    out, lse = qvg.paged_attention(big, b.q, b.table.clamp(min=0) + (pages - n), b.kv_len, 2, cu_q=b.cu_q, want_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_joins_the_compressed_history():
    """Attention over compressed chunks and over the pages of the chunk being
    generated, joined by their log-sum-exps, is attention over both."""
    p = qvg.Params(C=16, L=1, bits=4, group=32, iters=4, seed=3)
    H, d, n = 2, 64, 256
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(n, H, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    kc, vc = qvg.CompressedKV(p, H, d, n, 1), qvg.CompressedKV(p, H, d, n, 1)
    qvg.compress_chunk(p, k, kc)
    qvg.compress_chunk(p, v, vc)
    b = Batch(H, 1, d, 8, 16, (5,), (37,), seed=20)
    o2, l2 = b.run(out_dtype=qvg.QVG_OUT_F32)
    o1, l1, _ = qvg.attention(p, b.q, kc, vc, want_lse=True)
    w = torch.sigmoid(l1.double() - l2.double()).t()[..., None]
    got = w * o1.double() + (1 - w) * o2.double()
    kh, vh = (qvg.decompress(p, c, 0, n).double().cpu().numpy() for c in (kc, vc))
    k_all, v_all = (x.transpose(0, 2, 1, 3).reshape(-1, H, d)[b.slots[0]] for x in ref.held(b.cache))
    see = np.concatenate([np.ones((5, n), bool), b.see(0, qvg.QVG_MASK_CAUSAL)], 1)
    want, _ = ref.attention(b.q.double().cpu().numpy(), np.concatenate([kh, k_all]), np.concatenate([vh, v_all]), see)
    # the compressed side's own bar: 2e-3 of the largest output (fp16 operands)
    assert np.abs(got.cpu().numpy() - want).max() <= 2e-3 * np.abs(want).max()


# ---- many rows a sequence -------------------------------------------------------------------------


def check_on_device(b, out, lse, mode, rows=None):
    """Batch.check's plain form and bounds, sequence by sequence on the GPU in
    64 bits (for batches that are too long for the host's loop).  Below 2^-90
    V's scale is not in the reference: a weight, of up to 2^98 of its row's
    sum, is off by at most 2^-17 (half of e5m2's smallest step) against codes
    up to 448, n 2^-106 over n keys."""
    k_all, v_all = (torch.from_numpy(x).cuda().transpose(1, 2).reshape(-1, b.H, b.d) for x in ref.held(b.cache))
    q_step = 2.0 ** -21 if max(b.nq) * b.G <= (64 if b.cache.bits == 8 else 32) else 2.0 ** -17
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    scale, first = 1 / math.sqrt(b.d), 0
    for i, (T, L) in enumerate(zip(b.nq, b.kv)):
        if T == 0:
            continue
        at = torch.from_numpy(b.slots[i]).cuda()
        see = torch.from_numpy(b.see(i, mode, None if rows is None else rows[i])).cuda()
        q = b.q[first:first + T].double().view(T, b.H, b.G, b.d)
        got, got_lse = out[first:first + T].double().view(T, b.H, b.G, b.d), lse[:, first:first + T].double().view(b.H, b.G, T)
        first += T
        if L == 0:
            assert bool((got_lse == -math.inf).all()) and bool((got == 0).all())
            continue
        k, v = k_all[at], v_all[at]
        s = torch.einsum("thgd,lhd->hgtl", q, k) * scale
        s = s.masked_fill(~see, -math.inf)
        m = s.amax(-1, keepdim=True).clamp(min=-1e300)
        p = torch.exp(s - m)
        den = p.sum(-1, keepdim=True)
        want_lse = (m + den.log())[..., 0]
        w = p / den.clamp(min=1e-300)
        n = see.sum(-1).double()
        absqk = torch.einsum("thgd,lhd->hgtl", q.abs(), k.abs())
        dd = scale * (q_step * q.abs().amax(-1).permute(1, 2, 0)[..., None] * k.abs().sum(-1).t()[:, None, None] + 2 * b.d * 2.0 ** -23 * absqk)
        dd = (dd + 8 * 2.0 ** -24 * s.abs().masked_fill(~see, 0)).masked_fill(~see, 0).amax(-1)
        rel = 2 * dd + 2.0 ** -20 + 2.0 ** -11 + 2.0 ** -9 + n * 2.0 ** -24
        back = lambda x: x.permute(2, 0, 1)[..., None]  # noqa: E731
        want = torch.einsum("hgtl,lhd->thgd", w, v)
        mean = torch.einsum("hgtl,lhd->thgd", w, v.abs())
        lost = n * 2.0 ** -24 * (w * v.abs().amax(-1).t()[:, None, None]).amax(-1)
        bound = back(rel) * mean + back(lost) + half * want.abs() + back(n.expand_as(rel)) * 2.0 ** -106
        err = (got - want).abs()
        assert bool((err <= bound).all()), (i, float((err / bound).max()))
        some = n > 0
        assert bool((got_lse[:, :, ~some] == -math.inf).all()) and bool((got[~some] == 0).all())
        lb = dd + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -21 * want_lse.abs()
        assert bool(((got_lse - want_lse).abs() <= lb)[:, :, some].all())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mode", [qvg.QVG_MASK_NONE, qvg.QVG_MASK_CAUSAL, qvg.QVG_MASK_TREE])
def test_many_rows_many_units(bits, d, mode):
    """Several row blocks in one CTA's run, second halves of them with and
    without rows, sequences without new tokens, without history, without keys."""
    g = np.random.default_rng(100 + d)
    nq = [int(x) for x in g.choice([0, 1, 31, 32, 33, 64, 65, 75, 97], size=230)]
    kv = [max(n, int(x)) for n, x in zip(nq, g.integers(0, 500, size=230))]
    nq[0], kv[0], nq[7], kv[7] = 97, 97, 64, 64
    b = Batch(2, 4, d, bits, 32, nq, kv, seed=22)
    mask = rows = None
    if mode == qvg.QVG_MASK_TREE:
        rows = [np.eye(T, dtype=bool) | (g.random((T, T)) < 0.5) for T in nq]
        rows[0][[0, 40, 96]] = False  # no history: rows that see nothing
        words = np.zeros((sum(nq), (max(nq) + 31) // 32), np.uint32)
        first = 0
        for T, r in zip(nq, rows):
            for j in range(T):
                words[first:first + T, j >> 5] |= r[:, j].astype(np.uint32) << np.uint32(j & 31)
            first += T
        mask = torch.from_numpy(words.view(np.int32)).cuda()
    out, lse = b.run(mode, mask=mask)
    assert qvg.get_status() == qvg.QVG_OK
    check_on_device(b, out, lse, mode, rows)
    again, lse2 = b.run(mode, mask=mask)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rows", [15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 600])
def test_row_counts(bits, rows):
    """Either side of every size at which another kernel or block begins."""
    b = Batch(1, 1, 128, bits, 64, (rows, 1, rows // 2), (rows + 300, 200, rows), seed=23)
    out, lse = b.run()
    check_on_device(b, out, lse, qvg.QVG_MASK_CAUSAL)
    b = Batch(2, 3, 64, bits, 16, (-(-rows // 3),), (3000,), seed=24)
    out, lse = b.run()
    check_on_device(b, out, lse, qvg.QVG_MASK_CAUSAL)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_unseen_keys_have_no_influence_on_many_rows(bits, G, d):
    """The same with 17 to 32 rows and more: masked drafts that are not finite,
    and slots that were never written."""
    b = Batch(2, G, d, bits, 32, (6, 3), (70, 200), seed=25)
    mask = torch.tensor([[1 << t] for t in range(6)] + [[1], [3], [7]], dtype=torch.int32, device="cuda")
    want, want_lse = b.run(qvg.QVG_MASK_TREE, mask=mask)
    bad = torch.full((2, 2, d), 1.0, dtype=torch.bfloat16, device="cuda")
    bad[0, :, 3], bad[1, :, 60] = math.inf, math.nan
    at = torch.from_numpy(b.slots[0][[64 + 1, 64 + 4]]).cuda()
    good = torch.zeros_like(bad)
    keep = [i for i in range(9) if i not in (1, 4)]
    for k, v in ((bad, good), (good, bad), (bad, bad)):
        qvg.paged_append(b.cache, k, v, at)
        out, lse = b.run(qvg.QVG_MASK_TREE, mask=mask)
        assert torch.equal(out[keep], want[keep]) and torch.equal(lse[:, keep], want_lse[:, keep])
        assert out[[1, 4]].isnan().all()
    for s in b.slots[0][[64 + 1, 64 + 4]]:
        for t in (b.cache.k_codes, b.cache.v_codes):
            t[s // 32, :, s % 32] = torch.randint(0, 256, t.shape[-1:], device="cuda").to(torch.uint8) | 0x7E
        for t in (b.cache.k_scales, b.cache.v_scales):
            t[s // 32, :, s % 32] = int(s) * 37 % 256
    out, lse = b.run(qvg.QVG_MASK_TREE, mask=mask)
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[:, keep], want_lse[:, keep])
    assert qvg.get_status() == qvg.QVG_OK


@pytest.mark.parametrize("T", [7, 60])
def test_non_finite_query_among_many_rows(T):
    b = Batch(2, 4, 128, 8, 16, (T,), (300,), seed=26)
    want, _ = b.run()
    b.q[1, 2, 7], b.q[2, 5, 0], b.q[T - 1, 7, 127] = math.nan, math.inf, -math.inf
    out, lse = b.run()
    nan = torch.zeros(T, 8, dtype=torch.bool)
    nan[1, 2], nan[2, 5], nan[T - 1, 7] = True, True, True
    assert (out.cpu().isnan().all(-1) == nan).all() and (lse.cpu().isnan().t() == nan).all()
    assert torch.equal(out.cpu()[~nan], want.cpu()[~nan])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T", [12, 70])
@pytest.mark.parametrize("kw", [dict(k_scale=30.0), dict(v_scale=2.0 ** -20), dict(v_scale=2.0 ** -80), dict(v_scale=2.0 ** 30),
                                dict(q_scale=2.0 ** 20, k_scale=2.0 ** -18), dict(k_scale=2.0 ** -30)])
def test_magnitudes_with_many_rows(bits, T, kw):
    b = Batch(1, 2, 128, bits, 64, (T, 1), (900, 300), seed=27, **kw)
    out, lse = b.run()
    check_on_device(b, out, lse, qvg.QVG_MASK_CAUSAL)


@pytest.mark.parametrize("T", [12, 70])
@pytest.mark.parametrize("v_scale", [1.0, 2.0 ** -70, 2.0 ** -122])
def test_growing_logits_with_many_rows(T, v_scale):
    """References raised from tile to tile, by a little and by far more than
    the weights' types hold; with V so small that the sum would overflow first."""
    for L, top in ((3000, 400.0), (9000, 3e4)):
        b = Batch(1, 2, 128, 8, 64, (T,), (L,), seed=28, v_scale=v_scale)
        t = torch.arange(L, device="cuda")
        k = torch.randn(L, 1, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
        k[:, 0, 0] = t / L * top
        qvg.paged_append(b.cache, k.bfloat16(), b.v, torch.from_numpy(b.slots[0]).cuda())
        b.q[:, 0, 0], b.q[:, 1, 0] = 1.0, -2.0
        out, lse = b.run()
        check_on_device(b, out, lse, qvg.QVG_MASK_CAUSAL)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T", [6, 80])
def test_many_rows_padded_captured_and_out_of_time(bits, T):
    """A padded batch, several streams at once, a replayed graph, and the
    library's bounded-wait hook, for the kernels of more than 16 rows."""
    b = Batch(2, 4, 128, bits, 32, (T, 0, T // 2), (1500, 40, 700), seed=29)
    want, want_lse = b.run()
    check_on_device(b, want, want_lse, qvg.QVG_MASK_CAUSAL)
    n = sum(b.nq)
    q = torch.full((n + 5, 8, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    q[:n] = b.q
    out = torch.full_like(q, 5.0)
    qvg.paged_attention(b.cache, q, b.table, b.kv_len, T, cu_q=b.cu_q, out=out)
    assert (out[n:] == 5).all() and torch.equal(out[:n], want)
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    got = [b.run(stream=s) for _ in range(3) for s in side]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(l, want_lse) for o, l in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = b.run()
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    qvg.debug_set_wait(1_000_000, True)
    try:
        b.run()
    finally:
        qvg.debug_set_wait(0, False)
    assert qvg.get_status() == qvg.QVG_ERR_TIMEOUT
    again, _ = b.run()
    assert qvg.get_status() == qvg.QVG_OK and torch.equal(again, want)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T", [1, 12, 70])
def test_logits_far_below_zero(bits, T):
    """Every key's logit far below 0, in every cut of the sequence: the first
    reference is as far below."""
    b = Batch(1, 2, 128, bits, 64, (T,), (5000,), seed=30)
    k = torch.randn(5000, 1, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    k[:, 0, 0] = 3000.0
    qvg.paged_append(b.cache, k.bfloat16(), b.v, torch.from_numpy(b.slots[0]).cuda())
    b.q[:, :, 0] = -4.0
    out, lse = b.run()
    check_on_device(b, out, lse, qvg.QVG_MASK_CAUSAL)


def test_tree_masks_of_long_trees():
    """Chains and bushes up to the largest tree, rows wider than they need be,
    and row counts that do not fit the tensors."""
    g = np.random.default_rng(31)
    T = 8192
    chain = torch.arange(T, dtype=torch.int32, device="cuda") - 1
    m = qvg.tree_mask(chain, T).cpu().numpy().view(np.uint32)
    t, w = np.arange(T)[:, None], np.arange(T // 32)[None]
    full = np.clip(t + 1 - 32 * w, 0, 32)
    assert (m == ((1 << full.astype(np.uint64)) - 1).astype(np.uint32)).all()
    parents = np.array([-1] + [int(g.integers(max(-1, i - 40), i)) for i in range(1, 700)], np.int32)
    rows = ref.tree_rows(parents)
    out = torch.full((700, 30), -1, dtype=torch.int32, device="cuda")
    qvg.tree_mask(torch.from_numpy(parents).cuda(), 700, out=out)
    bits = np.unpackbits(out.cpu().numpy().view(np.uint8), axis=1, bitorder="little")
    assert (bits[:, :700] == rows).all() and not bits[:, 700:].any()
    assert qvg.get_status() == qvg.QVG_OK
    for cu in ([0, 5, 900], [0, 5, 3], [-3, 2, 4], [2**31 - 1, -2**31, 7]):
        out.fill_(-1)
        qvg.tree_mask(torch.from_numpy(parents).cuda(), 20, cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out)
        assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG, cu
        assert (out[20:] == -1).all()


@pytest.mark.parametrize("G", [1, 8, 64])
def test_nothing_to_do(G):
    """No new tokens in any sequence; no keys in any; pages shared by sequences."""
    b = Batch(1, G, 64, 8, 16, (2, 1), (40, 30), seed=32)
    out = torch.full((3, G, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    qvg.paged_attention(b.cache, b.q, b.table, b.kv_len, 2, cu_q=torch.zeros_like(b.cu_q), out=out)
    assert (out == 5).all()
    out, lse = qvg.paged_attention(b.cache, b.q, b.table, torch.zeros_like(b.kv_len), 2, cu_q=b.cu_q, want_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    b.table[1] = b.table[0]
    b.slots[1] = b.slots[0][:30]
    out, lse = b.run()
    check_on_device(b, out, lse, qvg.QVG_MASK_CAUSAL)
    assert qvg.get_status() == qvg.QVG_OK


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("mode", [qvg.QVG_MASK_NONE, qvg.QVG_MASK_CAUSAL, qvg.QVG_MASK_TREE])
@pytest.mark.parametrize("nq,kv", [((5, 16), (3, 1)), ((40, 7), (10, 6)), ((200, 140), (150, 1))])
def test_more_new_tokens_than_keys(bits, mode, nq, kv):
    """The first T - L new tokens have no key of their own."""
    g = np.random.default_rng(33)
    b = Batch(2, 1, 128, bits, 16, nq, kv, seed=33)
    mask = rows = None
    if mode == qvg.QVG_MASK_TREE:
        parents = [np.array([g.integers(-1, t) if t else -1 for t in range(T)], np.int32) for T in nq]
        rows = [ref.tree_rows(p) for p in parents]
        mask = qvg.tree_mask(torch.from_numpy(np.concatenate(parents)).cuda(), max(nq), cu_q=b.cu_q)
    out, lse = b.run(mode, mask=mask)
    assert qvg.get_status() == qvg.QVG_OK
    check_on_device(b, out, lse, mode, rows)


def test_thousands_of_sequences():
    """More sequences than a warp's list holds at once, some without keys,
    some without new tokens."""
    g = np.random.default_rng(34)
    kv = [int(x) for x in g.choice([0, 1, 17, 128, 129, 300], size=2500)]
    nq = [int(x) for x in g.integers(0, 3, size=2500)]
    b = Batch(1, 2, 64, 8, 16, nq, kv, seed=34)
    out, lse = b.run()
    assert qvg.get_status() == qvg.QVG_OK
    check_on_device(b, out, lse, qvg.QVG_MASK_CAUSAL)


# ---- waits that run out ---------------------------------------------------------------------------


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("G", [1, 32, 128])
def test_wait_that_ends_while_the_work_is_handed_out(bits, G):
    """A bound of a nanosecond, and lists of sequences that take from some ten
    to a thousand microseconds to go through, so that waits run out before,
    while and after the first unit is handed out: each call ends, and the
    next one is whole."""
    b = Batch(1, G, 64, bits, 16, (1, 1), (20, 16), seed=35)
    want, want_lse = b.run()
    status = None
    for n in [int(2 ** (11 + i / 8)) for i in range(33)] + [1 << 16]:
        kv = torch.zeros(n, dtype=torch.int32, device="cuda")  # one new token each, and hardly any keys
        kv[:8] = 16
        table = b.table[:1, :1].expand(n, 1).contiguous()
        q = b.q[:1].expand(n, G, 64).contiguous()
        qvg.debug_set_wait(1, False)
        try:
            qvg.paged_attention(b.cache, q, table, kv, 1)
        finally:
            qvg.debug_set_wait(0, False)
        status = qvg.get_status()
        assert status in (qvg.QVG_OK, qvg.QVG_ERR_TIMEOUT), n
    assert status == qvg.QVG_ERR_TIMEOUT
    out, lse = b.run()
    assert qvg.get_status() == qvg.QVG_OK
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("G", [1, 8, 32])
def test_wait_that_ends_among_short_trees(bits, G):
    """Trees of four tokens in sequences of one tile: the wait runs out with
    the first unit's products in flight and the next units' rows not there
    yet, while every tile needs mask rows.  The status says so, the next call is whole."""
    g = np.random.default_rng(36)
    n = 900
    b = Batch(2, G, 64, bits, 16, [4] * n, [int(x) for x in g.integers(4, 129, size=n)], seed=36)
    parents = torch.from_numpy(np.concatenate([[-1] + [g.integers(-1, t) for t in range(1, 4)] for _ in range(n)]).astype(np.int32)).cuda()
    mask = qvg.tree_mask(parents, 4, cu_q=b.cu_q)
    want, want_lse = b.run(qvg.QVG_MASK_TREE, mask=mask)
    assert qvg.get_status() == qvg.QVG_OK
    for limit, inject in ((1_000_000, True), (20_000, True), (1, True), (1, False)):
        qvg.debug_set_wait(limit, inject)
        try:
            b.run(qvg.QVG_MASK_TREE, mask=mask)
        finally:
            qvg.debug_set_wait(0, False)
        assert qvg.get_status() in ((qvg.QVG_ERR_TIMEOUT,) if inject else (qvg.QVG_OK, qvg.QVG_ERR_TIMEOUT))
        out, lse = b.run(qvg.QVG_MASK_TREE, mask=mask)
        assert qvg.get_status() == qvg.QVG_OK
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 70])
def test_wait_that_ends_with_copies_in_flight(bits, d, T):
    """Long sequences, whose copies run ahead of the products: K's of a tile
    may be out when the wait for V's room ends (4 bits and many rows: K's room
    is free once converted, V's waits for products).  The calls right behind,
    on the same and on another stream, get their own bytes."""
    b = Batch(2, 1, d, bits, 16, (T, T), (30000, 20000), seed=37)
    want, want_lse = b.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for limit in (1, 30_000, 200_000, 1_000_000):
        qvg.debug_set_wait(limit, True)
        try:
            b.run()
        finally:
            qvg.debug_set_wait(0, False)
        got += [b.run(), b.run(stream=side)]
    assert qvg.get_status() == qvg.QVG_ERR_TIMEOUT
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, want_lse)


# ---- V of very unlike sizes -----------------------------------------------------------------------


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T", [1, 12, 70])
@pytest.mark.parametrize("e", [60, 118])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_values_of_very_unlike_size(bits, T, e, order):
    """Keys of equal weight whose V rows are 0 or around 2^e: the reference of
    the weights follows V's scale, by more than 2^126, and every key still
    counts in the sum; within a CTA's run (many sequences) and across cuts."""
    for n, L in ((60, 1000), (1, 20000)):
        b = Batch(2, 2, 64, bits, 64, [T] * n, [L] * n, seed=38)
        t = torch.arange(L, device="cuda")
        big = {"rising": t >= L // 2, "falling": t < L // 2, "mixed": t % 777 == 500}[order].repeat(n)
        v = torch.randn(L * n, 2, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)) * 2.0 ** e
        qvg.paged_append(b.cache, torch.zeros_like(b.k), (v * big[:, None, None]).bfloat16(), torch.from_numpy(np.concatenate(b.slots)).cuda())
        out, lse = b.run(out_dtype=qvg.QVG_OUT_F32)
        check_on_device(b, out, lse, qvg.QVG_MASK_CAUSAL)
    assert qvg.get_status() == qvg.QVG_OK


# ---- the weights' own precision --------------------------------------------------------------------


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T", [16, 30, 200])
def test_precision_of_a_weight(bits, T):
    """Each row sees two keys that share no channel of V, so that an fp32
    output is one weight times one value.  Q has four significant bits (exact
    in its fp8 pair).  Bounds: the logits' fp32 sums (of 2 d products, 2^-23
    each; the base-2 form 8 2^-24 of the logit), twice for two of them; ex2 2^-20; the weight as fp16,
    2^-11 of itself, and with few rows as three e5m2 parts, 2^-9 more; fp32
    roundings of the result 2^-22; far below the largest 2^-25 of it."""
    H, d = 8, 64
    b = Batch(H, 1, d, bits, 16, (T,), (T,), seed=39, k_scale=0.4)
    g = torch.Generator(device="cuda").manual_seed(7)
    b.q.copy_(torch.randint(-15, 16, b.q.shape, device="cuda", generator=g) / 8)
    v = torch.ones(T, H, d, device="cuda")
    v[:, :, 0] = 0.0
    v[0] = 0.0
    v[0, :, 0] = 1.0
    k = b.k.clone()
    k[0] = (b.q.float().mean(0) * 4).bfloat16()  # often the larger logit, not always
    qvg.paged_append(b.cache, k, v.bfloat16(), torch.from_numpy(b.slots[0]).cuda())
    words = torch.zeros(T, -(-T // 32), dtype=torch.int64, device="cuda")
    t = torch.arange(T, device="cuda")
    words[t, t // 32] |= 1 << (t % 32)
    words[:, 0] |= 1
    mask = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    out, lse = b.run(qvg.QVG_MASK_TREE, mask=mask, out_dtype=qvg.QVG_OUT_F32)
    assert qvg.get_status() == qvg.QVG_OK
    kk, vv = (x.transpose(0, 2, 1, 3).reshape(-1, H, d)[b.slots[0]] for x in ref.held(b.cache))
    q = b.q.double().cpu().numpy()
    see = np.eye(T, dtype=bool)
    see[:, 0] = True
    want, want_lse = ref.attention(q, kk, vv, see)
    s0, st = np.abs(q * kk[:1]).sum(-1), np.abs(q * kk).sum(-1)
    logit = (2 * d * 2.0 ** -23 + 8 * 2.0 ** -24) * np.maximum(s0, st) / math.sqrt(d)
    few = T <= (64 if bits == 8 else 32)
    rel = 2 * logit + 2.0 ** -20 + 2.0 ** -11 + (2.0 ** -9 if few else 0) + 2.0 ** -22
    bound = rel[..., None] * np.abs(want) + 2.0 ** -25 * np.abs(want).max()
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= bound).all(), float((err / bound).max())
    lb = logit.T + 2.0 ** -20 + 2.0 ** -21 * np.abs(want_lse)
    assert (np.abs(lse.double().cpu().numpy() - want_lse) <= lb).all()


@pytest.mark.parametrize("bits,G", [(8, 1), (4, 1), (8, 70)])
def test_longest_sequence(bits, G):
    """One page that a whole block table points to.  2^31 - 4096 keys are
    served: the page's own attention, with log of the repeats in the lse.
    One more is reported (the numbers of a tile's keys would pass 32 bits).
    Bounds: a CTA has up to 2^24 / 152 tiles.  With few rows a thread owns a
    key of each tile, so a sum has one addition a tile; with many a thread owns a row and keeps
    four sums of 32 keys a tile each; 2^-24 an addition.  The products go
    into O in eight steps a tile, 2^-23 each."""
    b = Batch(1, G, 64, bits, 256, (1,), (256,), seed=40)
    most = 2 ** 31 - 4096
    table = b.table[:, :1].expand(1, (1 << 23)).contiguous()
    kv = torch.tensor([most], dtype=torch.int32, device="cuda")
    out, lse = qvg.paged_attention(b.cache, b.q, table, kv, 1, out_dtype=qvg.QVG_OUT_F32, want_lse=True)
    assert qvg.get_status() == qvg.QVG_OK
    k, v = (x.transpose(0, 2, 1, 3).reshape(-1, 1, 64)[b.slots[0]] for x in ref.held(b.cache))
    want, want_lse = ref.attention(b.q.double().cpu().numpy(), k, v, np.ones((1, 256), bool))
    tiles = 2.0 ** 24 / 152
    sums = tiles * (32 if G > 64 else 1) * 2.0 ** -24
    assert np.abs(lse.double().cpu().numpy() - want_lse - math.log(most / 256)).max() <= sums + 2.0 ** -9
    bound = (sums + tiles * 8 * 2.0 ** -23 + 2.0 ** -8) * np.abs(v).max()
    assert np.abs(out.double().cpu().numpy() - want).max() <= bound
    for n in (most + 1, 2 ** 31 - 128, 2 ** 31 - 1):
        kv.fill_(n)
        qvg.paged_attention(b.cache, b.q, table, kv, 1)
        assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG, n
    again, _ = b.run()
    assert qvg.get_status() == qvg.QVG_OK
