"""CPU-side checks of the latent cache, of attention over it and of prompts,
and of the pages' calls: sizes and every refusal that is found on the host
before anything is launched (no GPU is needed; the pointers are never
followed)."""
import ctypes as ct
import math

import pytest
import torch

import video_diffusion_kv_gb300 as qvg
from video_diffusion_kv_gb300 import build as qbuild

BAD, UNS, WS = qvg.QVG_ERR_INVALID_ARG, qvg.QVG_ERR_UNSUPPORTED, qvg.QVG_ERR_WORKSPACE
P, ODD = 0x10000, 0x10001


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qvg.lib()


def latent(dc=128, dr=32, page=16, pages=4, c=P, kr=P):
    return ct.byref(qvg._Latent(dc, dr, page, pages, c, kr))


def view(data=P, token=4096, head=256):
    return ct.byref(qvg._View(data, token, head))


@pytest.mark.parametrize("kw,status", [
    (dict(dc=96), UNS), (dict(dc=320), UNS), (dict(dc=0), UNS), (dict(dr=-8), BAD), (dict(dr=136), BAD), (dict(dr=12), BAD),
    (dict(page=8), BAD), (dict(page=48), BAD), (dict(page=512), BAD), (dict(pages=0), BAD),
])
def test_cache_shapes(lib, kw, status):
    a = dict(dc=128, dr=32, page=16, pages=4, **{})
    a.update(kw)
    x, y = ct.c_size_t(7), ct.c_size_t(7)
    assert lib.qvg_latent_bytes(a["dc"], a["dr"], a["page"], a["pages"], ct.byref(x), ct.byref(y)) == status
    assert (x.value, y.value) == (7, 7)
    assert lib.qvg_latent_append(latent(**kw), P, P, 1, 128, 32, P, None, None, None) == status
    with pytest.raises(qvg.QvgError):
        qvg.LatentKV(a["dc"], a["dr"], a["page"], a["pages"], device="cpu")


def test_sizes_and_buffers(lib):
    assert qvg.latent_bytes(192, 24, 32, 5) == (5 * 32 * 384, 5 * 32 * 48)
    assert qvg.latent_bytes(64, 0, 16, 1) == (2048, 0)
    assert qvg.latent_bytes(256, 128, 256, 2 ** 20) == (2 ** 37, 2 ** 36)
    c = qvg.LatentKV(64, 8, 16, 3, device="cpu")
    assert c.c.shape == (3, 16, 64) and c.kr.shape == (3, 16, 8) and c.nbytes == 3 * 16 * 144
    own = [torch.zeros(3 * 16 * 64, dtype=torch.bfloat16), torch.zeros(3 * 16 * 8, dtype=torch.bfloat16)]
    assert qvg.LatentKV(64, 8, 16, 3, buffers=own).c.data_ptr() == own[0].data_ptr()
    both = torch.zeros(3 * 16 * 64, dtype=torch.bfloat16)
    for buffers in (own[:1], own + own[:1], [own[0][:-1], own[1]], [own[0].float(), own[1]], [both, both[:3 * 16 * 8]]):
        with pytest.raises(ValueError):
            qvg.LatentKV(64, 8, 16, 3, buffers=buffers)
    assert lib.qvg_latent_bytes(64, 8, 16, 3, None, ct.byref(ct.c_size_t())) == BAD


def test_append_and_read_refusals(lib):
    ok = dict(cache=latent(), c=P, kr=P, n=1, cs=128, ks=32, slots=P, plan=None, pos=None)

    def call(**kw):
        a = {**ok, **kw}
        return lib.qvg_latent_append(a["cache"], a["c"], a["kr"], a["n"], a["cs"], a["ks"], a["slots"], a["plan"], a["pos"], None)
    plan = qvg.RopePlan((32,))
    wide = qvg.RopePlan((34,))
    for kw in (dict(cache=None), dict(cache=latent(c=None)), dict(cache=latent(kr=None)), dict(cache=latent(c=0x10008)), dict(c=None), dict(c=0x10002),
               dict(kr=None), dict(kr=0x10008), dict(n=-1), dict(cs=120), dict(cs=132), dict(ks=24), dict(ks=36), dict(slots=None), dict(slots=0x10004),
               dict(plan=wide._ref, pos=P), dict(plan=plan._ref, pos=None), dict(plan=plan._ref, pos=ODD)):
        assert call(**kw) == BAD, kw
    assert call(n=0, c=None, slots=None) == qvg.QVG_OK
    assert lib.qvg_latent_read(latent(), P, -1, P, P, None) == BAD
    assert lib.qvg_latent_read(latent(), None, 1, P, P, None) == BAD
    assert lib.qvg_latent_read(latent(), P, 1, 0x10008, P, None) == BAD
    assert lib.qvg_latent_read(latent(), P, 1, P, 0x10008, None) == BAD
    assert lib.qvg_latent_read(latent(), P, 1, None, None, None) == qvg.QVG_OK
    assert lib.qvg_latent_read(latent(), P, 2 ** 30 + 1, P, P, None) == UNS
    assert lib.qvg_latent_append(latent(), P, P, 2 ** 30 + 1, 128, 32, P, None, None, None) == UNS
    assert lib.qvg_latent_read(latent(), None, 0, P, P, None) == qvg.QVG_OK


def test_latent_attention_refusals(lib):
    need = ct.c_size_t()
    assert lib.qvg_latent_workspace_size(128, 32, ct.byref(need)) == qvg.QVG_OK and need.value > 0
    assert lib.qvg_latent_workspace_size(100, 32, ct.byref(need)) == UNS
    assert lib.qvg_latent_workspace_size(128, 32, None) == BAD
    ok = dict(cache=latent(), q=view(), qr=view(), total=4, Hq=16, B=2, max_q=2, cu=P, table=P, stride=4, kv=P, mode=1, mask=None, words=0, scale=0.1,
              out=P, dtype=1, lse=P, ws=0x10000, size=1 << 40)

    def call(**kw):
        a = {**ok, **kw}
        return lib.qvg_latent_attention(a["cache"], a["q"], a["qr"], a["total"], a["Hq"], a["B"], a["max_q"], a["cu"], a["table"], a["stride"], a["kv"],
                                        a["mode"], a["mask"], a["words"], a["scale"], a["out"], a["dtype"], a["lse"], a["ws"], a["size"], None)
    for kw in (dict(cache=None), dict(cache=latent(c=None)), dict(q=None), dict(q=view(None)), dict(q=view(0x10008)), dict(q=view(token=120)),
               dict(q=view(token=4097)), dict(q=view(head=120)), dict(q=view(head=132)), dict(qr=None), dict(qr=view(head=24)), dict(total=-1), dict(Hq=0),
               dict(B=-1), dict(max_q=-1), dict(cu=ODD), dict(cu=None, total=3), dict(table=None), dict(table=ODD), dict(stride=0), dict(kv=None),
               dict(mode=3), dict(mode=-1), dict(mode=2), dict(mode=2, mask=P, words=0), dict(mode=2, mask=ODD, words=1), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(out=None), dict(out=0x10008), dict(dtype=2), dict(lse=ODD)):
        assert call(**kw) == BAD, kw
    assert call(cache=latent(dc=72)) == UNS
    assert call(max_q=2 ** 27, total=2 ** 30) == UNS
    assert call(cache=latent(pages=2 ** 28)) == UNS
    for kw in (dict(ws=None), dict(ws=0x10080), dict(size=100)):
        assert call(**kw) == WS, kw
    for kw in (dict(B=0), dict(max_q=0), dict(total=0)):
        assert call(q=None, out=None, **kw) == qvg.QVG_OK
    # one token or one head: the stride that is never taken may be anything
    assert call(total=1, q=view(token=3), ws=None) == WS and call(Hq=1, q=view(head=3), ws=None) == WS
    assert call(cache=latent(dr=0, kr=None), qr=None, ws=None) == WS


def test_expanded_attention_refusals(lib):
    ok = dict(q=view(), qr=view(), k=view(), kr=view(), v=view(), tq=4, tk=9, H=4, dn=128, dr=32, dv=64, B=2, max_q=2, max_k=4, cu=P, ck=P, mode=1,
              scale=0.0, out=P, dtype=1, lse=P)

    def call(**kw):
        a = {**ok, **kw}
        return lib.qvg_expanded_attention(*(a[n] for n in ("q", "qr", "k", "kr", "v", "tq", "tk", "H", "dn", "dr", "dv", "B", "max_q", "max_k", "cu", "ck",
                                                           "mode", "scale", "out", "dtype", "lse")), None)
    for kw in (dict(q=None), dict(q=view(0x10008)), dict(qr=None), dict(k=None), dict(k=view(token=120)), dict(kr=None), dict(kr=view(token=24)),
               dict(v=None), dict(v=view(head=56)), dict(v=view(head=68)), dict(tq=-1), dict(tk=-1), dict(H=0), dict(dr=-8), dict(dr=12), dict(B=-1),
               dict(max_q=-1), dict(max_k=-1), dict(cu=None, tq=3), dict(ck=None, tk=7), dict(cu=ODD), dict(ck=ODD), dict(mode=2), dict(mode=-1),
               dict(scale=math.nan), dict(out=None), dict(out=0x10008), dict(dtype=5), dict(lse=ODD)):
        assert call(**kw) == BAD, kw
    for kw in (dict(dn=96), dict(dv=256), dict(dr=72), dict(B=2 ** 20, H=2 ** 12), dict(B=2 ** 20, H=2 ** 10, max_q=2 ** 20, tq=2 ** 30), dict(max_q=2 ** 31 - 100), dict(tk=2 ** 31 - 64)):
        assert call(**kw) == UNS, kw
    for kw in (dict(B=0), dict(max_q=0), dict(tq=0)):
        assert call(q=None, out=None, **kw) == qvg.QVG_OK


def pool(pages=8, refs=P):
    return ct.byref(qvg._PagePool(pages, refs))


def seqs(B=3, page=16, stride=4, table=P, kv=P):
    return ct.byref(qvg._Sequences(B, page, stride, table, kv))


def test_page_calls_refusals(lib):
    fork = lambda p=pool(), s=seqs(), a=P, b=P, n=2: lib.qvg_pages_fork(p, s, a, b, n, None)  # noqa: E731
    cut = lambda p=pool(), s=seqs(), a=P, b=P, n=2: lib.qvg_pages_release(p, s, a, b, n, None)  # noqa: E731
    grow = lambda p=pool(), s=seqs(), cu=P, new=0, total=6, slots=P, copies=P, ws=P, size=1 << 20: \
        lib.qvg_pages_reserve(p, s, cu, new, total, slots, copies, ws, size, None)  # noqa: E731
    for call in (fork, cut, grow):
        for kw in (dict(p=None), dict(p=pool(0)), dict(p=pool(refs=None)), dict(p=pool(refs=ODD)), dict(s=None), dict(s=seqs(B=-1)), dict(s=seqs(page=24)),
                   dict(s=seqs(stride=0)), dict(s=seqs(table=None)), dict(s=seqs(table=ODD)), dict(s=seqs(kv=None)), dict(s=seqs(kv=ODD))):
            assert call(**kw) == BAD, kw
    for call in (fork, cut):
        assert call(n=-1) == BAD and call(a=None) == BAD and call(a=ODD) == BAD and call(b=ODD) == BAD and call(s=seqs(B=0)) == BAD
        assert call(n=0, a=None, b=None) == qvg.QVG_OK
    assert fork(b=None) == BAD
    for kw in (dict(cu=ODD), dict(total=-1), dict(cu=None, new=-1), dict(cu=None, new=3), dict(slots=None), dict(slots=0x10004), dict(copies=None),
               dict(copies=0x10004), dict(s=seqs(B=0))):
        assert grow(**kw) == BAD, kw
    for kw in (dict(ws=None), dict(ws=0x10008), dict(size=8)):
        assert grow(**kw) == WS, kw
    assert grow(s=seqs(B=0, table=None, kv=None), total=0) == qvg.QVG_OK
    most = 2 ** 31 - 2049  # (one less reaches the workspace's check)
    assert fork(n=2 ** 20 + 1) == UNS and cut(n=2 ** 20 + 1) == UNS
    assert grow(total=most + 1) == UNS and grow(p=pool(most + 1)) == UNS and grow(s=seqs(B=most + 1)) == UNS
    assert grow(total=most, ws=None) == WS and grow(p=pool(most)) == WS
    size = ct.c_size_t()
    assert lib.qvg_pages_workspace_size(8, 3, ct.byref(size)) == qvg.QVG_OK and size.value >= 4 * (2 * 8 + 3)
    assert lib.qvg_pages_workspace_size(0, 3, ct.byref(size)) == BAD
    assert lib.qvg_pages_workspace_size(8, -1, ct.byref(size)) == BAD
    assert lib.qvg_pages_workspace_size(8, 3, None) == BAD


def rows(n=2, page=16, pages=4, base=(P, P), heads=(1, 1), row_bytes=(256, 64)):
    r = qvg._PageRows(page, pages, n)
    for i in range(min(2, n)):
        r.base[i], r.heads[i], r.row_bytes[i] = base[i], heads[i], row_bytes[i]
    return ct.byref(r)


def test_moves_refusals(lib):
    r = qvg._PageRows()
    assert lib.qvg_latent_rows(latent(), ct.byref(r)) == qvg.QVG_OK
    assert (r.n, r.page_size, r.num_pages, list(r.heads)[:2], list(r.row_bytes)[:2]) == (2, 16, 4, [1, 1], [256, 64])
    assert lib.qvg_latent_rows(latent(dr=0, kr=None), ct.byref(r)) == qvg.QVG_OK and r.n == 1
    for bits, d, want in ((8, 128, [128, 128, 1, 1]), (4, 128, [64, 64, 4, 4]), (4, 64, [32, 32, 2, 2]), (8, 64, [64, 64, 1, 1])):
        p = qvg._Paged(3, d, 16, 4, bits, P, 0x20000, 0x30000, 0x40000)
        assert lib.qvg_paged_rows(ct.byref(p), ct.byref(r)) == qvg.QVG_OK
        assert (r.n, list(r.heads), list(r.row_bytes), list(r.base)) == (4, [3] * 4, want, [P, 0x30000, 0x20000, 0x40000])
    assert lib.qvg_paged_rows(None, ct.byref(r)) == BAD and lib.qvg_paged_rows(ct.byref(p), None) == BAD
    assert lib.qvg_latent_rows(latent(c=None), ct.byref(r)) == BAD and lib.qvg_latent_rows(latent(), None) == BAD
    copy = lambda r=rows(), c=P, n=1: lib.qvg_pages_copy(r, c, n, None)  # noqa: E731
    pack = lambda r=rows(), t=P, stride=4, B=2, first=P, keep=P, ks=3, n=P: lib.qvg_paged_compact(r, t, stride, B, first, keep, ks, n, None)  # noqa: E731
    for call in (copy, pack):
        for bad in (None, rows(n=0), rows(n=5), rows(page=20), rows(pages=0), rows(base=(None, P)), rows(base=(0x10008, P)), rows(heads=(0, 1)),
                    rows(row_bytes=(8, 64)), rows(row_bytes=(24, 64)), rows(row_bytes=(0, 64)), rows(row_bytes=(-16, 64))):
            assert call(r=bad) == BAD
    assert copy(n=-1) == BAD and copy(c=None) == BAD and copy(c=ODD) == BAD and copy(n=0, c=None) == qvg.QVG_OK
    for kw in (dict(t=None), dict(t=ODD), dict(stride=0), dict(B=-1), dict(first=None), dict(keep=None), dict(keep=ODD), dict(ks=-1), dict(n=None)):
        assert pack(**kw) == BAD, kw
    assert pack(B=65536) == UNS and copy(n=2 ** 31 - 65535) == UNS
    assert pack(B=0, t=None) == qvg.QVG_OK and pack(ks=0, keep=None) == qvg.QVG_OK


def test_compaction_refuses_more_kept_tokens_than_its_indices_hold(lib):
    pack = lambda ks, B=2, first=P: lib.qvg_paged_compact(rows(), P, 4, B, first, P, ks, P, None)  # noqa: E731
    for ks in (2 ** 31 - 2048, 2 ** 31 - 1):
        assert pack(ks) == UNS and pack(ks, B=1) == UNS
    assert pack(2 ** 31 - 2049, first=None) == BAD  # (no limit: the next check's answer)


def test_rows_of_more_bytes_than_63_bits(lib):
    big = 2 ** 31 - 16
    for kw in (dict(heads=(big, 1), row_bytes=(big, 64)), dict(heads=(1, big), row_bytes=(256, big), pages=2 ** 20),
               dict(heads=(2 ** 20, 1), row_bytes=(2 ** 24, 64), pages=2 ** 30, page=256)):
        assert lib.qvg_pages_copy(rows(**kw), P, 1, None) == BAD
        assert lib.qvg_paged_compact(rows(**kw), P, 4, 2, P, P, 3, P, None) == BAD


def test_attention_refuses_more_sequences_than_its_walks_hold(lib):
    def latent_call(B, ws=None):
        return lib.qvg_latent_attention(latent(), view(), view(), 4, 16, B, 2, P, P, 4, P, 1, None, 0, 0.1, P, 1, P, ws, 0, None)

    def prompt_call(B, max_q=2, total=4, H=1):
        return lib.qvg_expanded_attention(view(), view(), view(), view(), view(), total, 9, H, 128, 32, 64, B, max_q, 4, P, P, 1, 0.0, P, 1, P, None)
    for B in (2 ** 20 + 1, 2 ** 30 + 1, 2 ** 31 - 20, 2 ** 31 - 1):
        assert latent_call(B) == UNS and prompt_call(B) == UNS
        assert prompt_call(B, max_q=300, total=2 ** 31 - 1) == UNS  # (the blocks pass 31 bits)
    assert latent_call(2 ** 20) == WS  # (no limit: the next check's answer)


def test_no_gradient_is_lost_without_a_word(lib):
    """There is no backward pass: inputs that require a gradient are refused
    where gradients are recorded, and not otherwise (the next check, for a
    CUDA device, answers then)."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    cache = qvg.LatentKV(64, 8, 16, 2, device="cpu")
    calls = (
        (lambda **a: qvg.latent_append(cache, slots=torch.zeros(3, dtype=torch.int64), **a), dict(c=bf(3, 64), k_rope=bf(3, 8))),
        (lambda **a: qvg.latent_attention(cache, block_table=i32(2, 3), kv_len=i32(2), max_q=2, scale=0.1, cu_q=i32(3), **a),
         dict(q=bf(4, 2, 64), q_rope=bf(4, 2, 8))),
        (lambda **a: qvg.expanded_attention(max_q=2, cu_q=i32(3), cu_k=i32(3), **a),
         dict(q=bf(4, 2, 64), q_rope=bf(4, 2, 8), k=bf(6, 2, 64), k_rope=bf(6, 8), v=bf(6, 2, 64))))
    for call, inputs in calls:
        for name in inputs:
            some = {**inputs, name: inputs[name].clone().requires_grad_()}
            with pytest.raises(ValueError, match="no gradient"):
                call(**some)
            with torch.no_grad(), pytest.raises(ValueError) as e:
                call(**some)
            assert "gradient" not in str(e.value)
        with pytest.raises(ValueError) as e:
            call(**inputs)
        assert "gradient" not in str(e.value)


def test_counts_beyond_32_bits_are_not_cut_off(lib):
    """(Shapes of expanded tensors: nothing of that size is allocated.)"""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    many = torch.zeros(1, dtype=torch.int32).expand(2 ** 32 + 1)
    cache, pool_ = qvg.LatentKV(64, 8, 16, 2, device="cpu"), qvg.PagePool(4, device="cpu")
    t, n = i32(2, 3), i32(2)
    for call in (lambda: qvg.latent_attention(cache, bf(4, 2, 64), bf(4, 2, 8), t, n, 2 ** 32, 0.1, cu_q=i32(3)),
                 lambda: qvg.expanded_attention(bf(4, 2, 64), None, bf(6, 2, 64), None, bf(6, 2, 64), 2 ** 32 + 1, cu_q=i32(3), cu_k=i32(3)),
                 lambda: qvg.expanded_attention(bf(4, 2, 64), None, bf(6, 2, 64), None, bf(6, 2, 64), 2, cu_q=i32(3), cu_k=i32(3), max_k=2 ** 33),
                 lambda: qvg.pages_fork(pool_, 16, t, n, many, many), lambda: qvg.pages_release(pool_, 16, t, n, many),
                 lambda: qvg.pages_release(pool_, 16, many[:, None].expand(-1, 3), many, i32(1)),
                 lambda: qvg.pages_reserve(pool_, 16, t, n, n_new=2 ** 32), lambda: qvg.pages_reserve(pool_, 16, t, n, cu_new=i32(3), total=2 ** 32),
                 lambda: qvg.pages_copy(cache, many[:, None].expand(-1, 2)),
                 lambda: qvg.paged_compact(cache, t, n, i32(1).expand(2, 2 ** 32), n)):
        with pytest.raises(ValueError, match="32-bit counts"):
            call()


def test_python_refusals(lib):
    """Shapes, types and devices are checked before the library is called."""
    c = qvg.LatentKV(64, 8, 16, 2, device="cpu")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    slots = torch.zeros(3, dtype=torch.int64)
    plan = qvg.RopePlan((8,))
    for args, kw in (((bf(3, 65), bf(3, 8), slots), {}), ((bf(3, 64).float(), bf(3, 8), slots), {}), ((bf(3, 64), None, slots), {}),
                     ((bf(3, 64), bf(2, 8), slots), {}), ((bf(2, 64), bf(2, 8), slots), {}), ((bf(64, 3).t(), bf(3, 8), slots), {}),
                     ((bf(3, 64), bf(3, 8), slots.int()), {}), ((bf(3, 64), bf(3, 8), slots), dict(plan=plan)),
                     ((bf(3, 64), bf(3, 8), slots), dict(plan=plan, positions=i32(2))),
                     ((bf(3, 64), bf(3, 8), slots), {})):  # the last: no CUDA device
        with pytest.raises(ValueError):
            qvg.latent_append(c, *args, **kw)
    with pytest.raises(ValueError):
        qvg.latent_read(c, slots, c_out=bf(2, 64))
    ok = dict(q=bf(4, 2, 64), q_rope=bf(4, 2, 8), block_table=i32(2, 3), kv_len=i32(2), max_q=2, scale=0.1, cu_q=i32(3))
    for kw in (dict(q=bf(4, 2, 63)), dict(q=bf(4, 128)), dict(q=bf(4, 64, 2).transpose(1, 2)), dict(q_rope=None), dict(q_rope=bf(4, 3, 8)),
               dict(block_table=i32(3, 3)), dict(cu_q=i32(2)), dict(mask_mode=2), dict(mask_mode=2, mask=i32(3, 1)), dict(out=bf(4, 2, 32)),
               dict(kv_len=slots[:2]), dict(workspace=i32(4)), dict()):
        with pytest.raises(ValueError):
            qvg.latent_attention(c, **{**ok, **kw})
    ok = dict(q=bf(4, 2, 64), q_rope=bf(4, 2, 8), k=bf(6, 2, 64), k_rope=bf(6, 8), v=bf(6, 2, 64), max_q=2, cu_q=i32(3), cu_k=i32(3))
    for kw in (dict(q=bf(4, 64)), dict(k=bf(6, 3, 64)), dict(v=bf(5, 2, 64)), dict(q_rope=None), dict(k_rope=None), dict(k_rope=bf(6, 2, 8)),
               dict(k_rope=bf(5, 8)), dict(cu_k=i32(4)), dict(cu_q=None, cu_k=None, max_k=2), dict(cu_k=None, max_k=2), dict(out=bf(4, 2, 32)),
               dict(q=bf(4, 2, 64).float()), dict()):
        with pytest.raises(ValueError):
            qvg.expanded_attention(**{**ok, **kw})
    with pytest.raises(ValueError):
        qvg.PagePool(0, device="cpu")
    with pytest.raises(ValueError):
        qvg.PagePool(4, refs=i32(3))
    pool_ = qvg.PagePool(4, device="cpu")
    t, n = i32(2, 3), i32(2)
    for call in (lambda: qvg.pages_fork(pool_, 16, t, i32(3), i32(1), i32(1)), lambda: qvg.pages_fork(pool_, 16, t, n, i32(1), i32(2)),
                 lambda: qvg.pages_fork(pool_, 16, t, n, i32(1), slots[:1]), lambda: qvg.pages_release(pool_, 16, t, n, i32(1), keep=i32(2)),
                 lambda: qvg.pages_release(pool_, 16, t.long(), n, i32(1)), lambda: qvg.pages_reserve(pool_, 16, t, n, cu_new=i32(3)),
                 lambda: qvg.pages_reserve(pool_, 16, t, n, cu_new=i32(2), total=1), lambda: qvg.pages_reserve(pool_, 16, t, n, n_new=-1),
                 lambda: qvg.pages_reserve(pool_, 16, t, n, slots=slots), lambda: qvg.pages_reserve(pool_, 16, t, n),
                 lambda: qvg.pages_copy(c, i32(3)), lambda: qvg.pages_copy(c, i32(3, 3)), lambda: qvg.pages_copy(c, i32(3, 2)),
                 lambda: qvg.paged_compact(c, t, i32(3), i32(2, 2), n), lambda: qvg.paged_compact(c, t, n, i32(2), n),
                 lambda: qvg.paged_compact(c, t, n, i32(2, 2), n)):
        with pytest.raises(ValueError):
            call()
