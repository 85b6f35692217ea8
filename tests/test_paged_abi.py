"""CPU-side checks of the token-wise operators: the rotary plan's angles, the
paged cache's sizes, and every refusal (found on the host before anything is
launched: no GPU is needed, and the pointers below are never followed)."""
import ctypes as ct
import math

import numpy as np
import pytest
import torch

import video_diffusion_kv_gb300 as qvg
from video_diffusion_kv_gb300 import build as qbuild

import _paged as ref

BAD, UNS, WS = qvg.QVG_ERR_INVALID_ARG, qvg.QVG_ERR_UNSUPPORTED, qvg.QVG_ERR_WORKSPACE
P = ct.c_void_p(0x10000)


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qvg.lib()


def steps(plan):
    m = plan.dims // 2
    return np.array([plan._c.step[i] for i in range(m)], dtype=np.float64) / 2.0 ** 64 * 2 * math.pi, \
        np.array([plan._c.axis[i] for i in range(m)])


@pytest.mark.parametrize("kw,ref_kw", [
    (dict(), dict()),
    (dict(scaling=qvg.QVG_ROPE_LINEAR, factor=4.0), dict(scaling="linear", factor=4.0)),
    (dict(scaling=qvg.QVG_ROPE_NTK, factor=5.5, base=500.0), dict(scaling="ntk", factor=5.5, base=500.0)),
    (dict(scaling=qvg.QVG_ROPE_PARTS, factor=8.0, original=4096.0), dict(scaling="parts", factor=8.0, original=4096.0)),
    (dict(scaling=qvg.QVG_ROPE_LINEAR, factor=2.0, scaled_axes=1), dict(scaling="linear", factor=2.0, scaled=(0,))),
])
@pytest.mark.parametrize("dims", [(128,), (2,), (44, 42, 42), (16, 8, 8, 6)])
def test_plan_frequencies(lib, dims, kw, ref_kw):
    """Steps are the formulas' frequencies, to a double's precision (a few
    roundings of 2^-53 each) and the rounding to a whole number of 2^-64 turns
    (half of one: 2 pi 2^-65 radians)."""
    plan = qvg.RopePlan(dims, **kw)
    f, axis = ref.frequencies(dims, **ref_kw)
    got, got_axis = steps(plan)
    np.testing.assert_allclose(got, f, rtol=1e-14, atol=2 * math.pi * 2.0 ** -65)
    np.testing.assert_array_equal(got_axis, axis)
    assert (plan.dims, plan.axes) == (sum(dims), len(dims))


@pytest.mark.parametrize("dims,kw", [
    ((), {}), ((2,) * 5, {}), ((3,), {}), ((0,), {}), ((-2,), {}), ((130,), {}), ((64, 66), {}),
    ((64,), dict(layout=2)), ((64,), dict(scaling=4)), ((64,), dict(scaling=-1)), ((64,), dict(base=0.5)),
    ((64,), dict(base=math.nan)), ((64,), dict(factor=0.5)), ((64,), dict(factor=math.inf)),
    ((64,), dict(mscale=math.nan)), ((64,), dict(scaling=3, original=0.0)),
    ((64,), dict(scaling=3, original=10.0, fast=1.0, slow=1.0)),
])
def test_plan_refusals(lib, dims, kw):
    with pytest.raises(qvg.QvgError) as e:
        qvg.RopePlan(dims, **kw)
    assert e.value.status == BAD


def test_rope_refusals(lib):
    plan = qvg.RopePlan((64,))
    call = lambda plan=plan._ref, x=P, dt=1, n=4, H=2, d=64, xs=128, pos=P, tr=0, out=P, os=128: lib.qvg_rope(  # noqa: E731
        plan, x, dt, n, H, d, xs, pos, tr, out, os, None)
    for kw in (dict(plan=None), dict(dt=2), dict(n=-1), dict(H=0), dict(xs=127), dict(os=64), dict(x=None), dict(out=None),
               dict(pos=None), dict(tr=2), dict(x=ct.c_void_p(0x10001)), dict(dt=0, out=ct.c_void_p(0x10002)),
               dict(pos=ct.c_void_p(0x10002)), dict(xs=136)):  # the last: in place with two strides
        assert call(**kw) == BAD, kw
    assert call(d=96) == UNS
    assert call(n=0, x=None, out=None, pos=None) == qvg.QVG_OK
    wide = qvg.RopePlan((128,))
    assert call(plan=wide._ref) == BAD  # rotates more channels than the head has
    broken = qvg._RopePlan.from_buffer_copy(plan._c)
    broken.axis[3] = 1
    assert call(plan=ct.byref(broken)) == BAD


def test_paged_sizes(lib):
    assert qvg.paged_bytes(8, 128, 64, 10, 8) == (10 * 8 * 64 * 128, 10 * 8 * 64)
    assert qvg.paged_bytes(3, 64, 16, 7, 4) == (7 * 3 * 16 * 32, 7 * 3 * 16 * 2)
    # sizes past 32 bits
    assert qvg.paged_bytes(32, 128, 128, 1 << 17, 8) == (32 << 31, 32 << 24)
    for kw in (dict(H=0), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(num_pages=0), dict(bits=2)):
        with pytest.raises(qvg.QvgError) as e:
            qvg.paged_bytes(**{**dict(H=2, d=64, page_size=16, num_pages=4, bits=8), **kw})
        assert e.value.status == BAD
    with pytest.raises(qvg.QvgError) as e:
        qvg.paged_bytes(2, 96, 16, 4, 8)
    assert e.value.status == UNS


def fake(H=2, d=64, page=16, pages=4, bits=8, ptrs=(0x1000,) * 4):
    return qvg._Paged(H, d, page, pages, bits, *ptrs)


BAD_CACHES = [dict(H=0), dict(page=24), dict(pages=0), dict(bits=3), dict(ptrs=(None, 0x1000, 0x1000, 0x1000)),
              dict(ptrs=(0x1000, 0x1008, 0x1000, 0x1000)), dict(ptrs=(0x1000, 0x1000, 0x1000, None))]


def test_append_refusals(lib):
    plan = qvg.RopePlan((64,))

    def call(c=None, k=P, v=P, n=4, ks=128, vs=128, slots=P, plan=None, pos=None):
        c = fake() if c is None else c
        return lib.qvg_paged_append(ct.byref(c), k, v, n, ks, vs, slots, plan, pos, None)
    for kw in BAD_CACHES:
        assert call(fake(**kw)) == BAD, kw
    assert call(fake(d=32)) == UNS
    assert lib.qvg_paged_append(None, P, P, 4, 128, 128, P, None, None, None) == BAD
    for kw in (dict(n=-1), dict(ks=120), dict(ks=132), dict(vs=127), dict(k=None), dict(v=None), dict(slots=None),
               dict(k=ct.c_void_p(0x10008)), dict(v=ct.c_void_p(0x10004)), dict(slots=ct.c_void_p(0x10004)),
               dict(plan=plan._ref), dict(plan=plan._ref, pos=ct.c_void_p(0x10001)),
               dict(plan=qvg.RopePlan((128,))._ref, pos=P)):
        assert call(**kw) == BAD, kw
    assert call(n=0, k=None, v=None, slots=None) == qvg.QVG_OK


def test_read_refusals(lib):
    def call(c=None, slots=P, n=4, k=P, v=P, dt=1):
        c = fake() if c is None else c
        return lib.qvg_paged_read(ct.byref(c), slots, n, k, v, dt, None)
    for kw in BAD_CACHES:
        assert call(fake(**kw)) == BAD, kw
    for kw in (dict(n=-1), dict(dt=3), dict(slots=None), dict(k=ct.c_void_p(0x10008)), dict(v=ct.c_void_p(0x10002))):
        assert call(**kw) == BAD, kw
    assert call(n=0, slots=None) == qvg.QVG_OK
    assert call(k=None, v=None) == qvg.QVG_OK


def test_python_refusals(lib):
    """The binding refuses what it can see before the library is called."""
    plan = qvg.RopePlan((64,))
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(4, 1, dtype=torch.int32)
    for args in ((x.half(), pos), (x[0], pos), (x.transpose(0, 1), pos), (x, pos[:3]), (x, pos.long()), (x, None), (x, pos)):
        with pytest.raises(ValueError):  # the last: not on a CUDA device
            qvg.rope(plan, *args)
    c = qvg.PagedKV(2, 64, 16, 4, device="cpu")
    assert c.nbytes == 2 * (4 * 2 * 16 * 64 + 4 * 2 * 16)
    slots = torch.zeros(4, dtype=torch.int64)
    for kw in (dict(k=x[:3]), dict(k=x.float()), dict(slots=slots.int()), dict(slots=slots[:2]), dict(plan=plan), dict()):
        with pytest.raises(ValueError):
            qvg.paged_append(c, **{**dict(k=x, v=x, slots=slots), **kw})
    with pytest.raises(ValueError):
        qvg.paged_read(c, slots.int())
    with pytest.raises(ValueError):
        qvg.paged_read(c, slots, k_out=torch.zeros(4, 2, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        qvg.PagedKV(2, 64, 16, 4, buffers=[torch.zeros(8, dtype=torch.uint8)] * 4)


def test_tree_mask_refusals(lib):
    call = lambda par=P, cu=None, B=2, mq=40, tq=80, w=2, m=P: lib.qvg_tree_mask(par, cu, B, mq, tq, w, m, None)  # noqa: E731
    for kw in (dict(B=-1), dict(mq=-1), dict(w=1), dict(par=None), dict(m=None), dict(m=ct.c_void_p(0x10002)),
               dict(tq=-1), dict(tq=79), dict(cu=ct.c_void_p(0x10001))):
        assert call(**kw) == BAD, kw
    assert call(mq=8193, tq=20000, w=300) == UNS
    assert call(B=0, par=None, m=None) == qvg.QVG_OK


def test_paged_workspace(lib):
    size = ct.c_size_t(0)
    for kw, code in ((dict(), 0), (dict(H=0), BAD), (dict(Hq=3), BAD), (dict(B=-1), BAD), (dict(mq=-1), BAD), (dict(d=80), UNS)):
        a = {**dict(H=2, d=64, Hq=4, B=3, mq=5), **kw}
        assert lib.qvg_paged_workspace_size(a["H"], a["d"], a["Hq"], a["B"], a["mq"], ct.byref(size)) == code, kw
    assert lib.qvg_paged_workspace_size(2, 64, 4, 3, 5, None) == BAD
    assert size.value > 0


def test_paged_attention_refusals(lib):
    need = ct.c_size_t(0)
    assert lib.qvg_paged_workspace_size(2, 64, 4, 3, 40, ct.byref(need)) == qvg.QVG_OK

    def call(c=None, q=P, qs=256, tq=120, Hq=4, B=3, mq=40, cu=None, table=P, ts=8, kv=P, mode=1, mask=None, words=0, scale=0.0,
             out=P, dt=1, lse=None, ws=P, wb=need.value):
        c = fake() if c is None else c
        return lib.qvg_paged_attention(ct.byref(c), q, qs, tq, Hq, B, mq, cu, table, ts, kv, mode, mask, words, scale, out, dt, lse,
                                       ws, wb, None)
    for kw in BAD_CACHES:
        assert call(fake(**kw)) == BAD, kw
    assert call(fake(d=32)) == UNS
    for kw in (dict(qs=255), dict(qs=260), dict(Hq=3), dict(Hq=0), dict(B=-1), dict(mq=-1), dict(tq=-1), dict(tq=119),
               dict(ts=0), dict(mode=3), dict(mode=2), dict(mode=2, mask=P, words=1), dict(mode=2, mask=ct.c_void_p(0x10002), words=2),
               dict(scale=math.nan), dict(scale=math.inf), dict(dt=2), dict(q=None), dict(out=None), dict(table=None), dict(kv=None),
               dict(q=ct.c_void_p(0x10008)), dict(out=ct.c_void_p(0x10008)), dict(kv=ct.c_void_p(0x10002)),
               dict(cu=ct.c_void_p(0x10002)), dict(lse=ct.c_void_p(0x10002))):
        assert call(**kw) == BAD, kw
    for kw in (dict(ws=None), dict(wb=need.value - 1), dict(ws=ct.c_void_p(0x10080))):
        assert call(**kw) == WS, kw
    for kw in (dict(B=0), dict(mq=0), dict(tq=0, B=0)):
        assert call(**{**kw, **dict(q=None, out=None, table=None, kv=None, ws=None, wb=0)}) == qvg.QVG_OK, kw


def test_python_attention_refusals(lib):
    c = qvg.PagedKV(2, 64, 16, 4, device="cpu")
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    table, kv = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(q=q.float()), dict(q=q[..., :32]), dict(table=table[:1]), dict(table=table[0]), dict(kv=kv.long()),
               dict(cu_q=kv), dict(mask_mode=2), dict(mask_mode=2, mask=torch.zeros(3, 1, dtype=torch.int32)),
               dict(out=torch.zeros(4, 2, 64, dtype=torch.bfloat16)), dict(workspace=torch.zeros(9)), dict()):
        a = {**dict(q=q, table=table, kv=kv), **kw}
        q_, t_, k_ = a.pop("q"), a.pop("table"), a.pop("kv")
        with pytest.raises(ValueError):
            qvg.paged_attention(c, q_, t_, k_, 2, **a)
    par = torch.zeros(4, dtype=torch.int32)
    for args, kw in (((par, 3), {}), ((par, 0), {}), ((par, 2), dict(out=torch.zeros(3, 1, dtype=torch.int32))), ((par.long(), 2), {}),
                     ((par, 2), {})):
        with pytest.raises(ValueError):
            qvg.tree_mask(*args, **kw)


def test_positions_by_axis_are_refused(lib):
    """positions are [n, axes]: [axes, n] has as many elements, and would be
    read in the wrong order."""
    plan = qvg.RopePlan((24, 20, 20))
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache, slots = qvg.PagedKV(2, 64, 16, 4, device="cpu"), torch.zeros(4, dtype=torch.int64)
    for shape, good in (((4, 3), True), ((2, 2, 3), True), ((3, 4), False), ((12,), False), ((4, 3, 1), False)):
        pos = torch.zeros(*shape, dtype=torch.int32)
        for call in (lambda: qvg.rope(plan, x, pos), lambda: qvg.paged_append(cache, x, x, slots, plan=plan, positions=pos)):
            with pytest.raises(ValueError, match="CUDA tensors" if good else "positions must be"):
                call()
    one = qvg.RopePlan((64,))
    for shape in ((4,), (4, 1), (1, 4)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            qvg.rope(one, x, torch.zeros(*shape, dtype=torch.int32))


def test_paged_buffers_given(lib):
    """Four buffers that share no byte; they may be parts of one allocation."""
    codes, scales = qvg.paged_bytes(2, 64, 16, 4, 8)
    sizes = [codes, scales, codes, scales]
    arena = torch.zeros(sum(sizes) + 16, dtype=torch.uint8)
    parts = list(arena[:sum(sizes)].split(sizes))
    c = qvg.PagedKV(2, 64, 16, 4, buffers=parts)
    assert c.v_codes.data_ptr() == parts[2].data_ptr() and c.nbytes == sum(sizes)
    for bad in (parts[:3], parts + [parts[0].clone()], [parts[0], parts[1], parts[0], parts[3]],
                [parts[0], parts[1], arena[codes:2 * codes], parts[3]], [parts[0], parts[1], parts[2], parts[1]]):
        with pytest.raises(ValueError, match="four buffers|overlap"):
            qvg.PagedKV(2, 64, 16, 4, buffers=bad)


def test_rope_refuses_out_where_a_gradient_is_wanted(lib):
    plan = qvg.RopePlan((64,))
    x = torch.zeros(4, 2, 64, requires_grad=True)
    pos = torch.zeros(4, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="no gradient through out"):
        qvg.rope(plan, x, pos, out=torch.zeros(4, 2, 64))
    with pytest.raises(ValueError, match="CUDA tensors"):
        qvg.rope(plan, x, pos)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensors"):
        qvg.rope(plan, x, pos, out=torch.zeros(4, 2, 64))
    with pytest.raises(ValueError, match="a plan needs positions"):
        qvg.rope(plan, x, None)
