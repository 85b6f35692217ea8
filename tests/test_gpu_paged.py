"""Rotary positions and the paged token cache on the GPU, against plain
64-bit forms (tests/_paged.py)."""
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


SCALINGS = {
    "plain": (dict(), dict()),
    "linear": (dict(scaling=qvg.QVG_ROPE_LINEAR, factor=4.0), dict(scaling="linear", factor=4.0)),
    "ntk": (dict(scaling=qvg.QVG_ROPE_NTK, factor=5.5), dict(scaling="ntk", factor=5.5)),
    "parts": (dict(scaling=qvg.QVG_ROPE_PARTS, factor=8.0, original=4096.0, mscale=1.25),
              dict(scaling="parts", factor=8.0, original=4096.0)),
}


def values(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def positions_of(n, axes, seed, far):
    g = np.random.default_rng(seed)
    p = g.integers(-far, far + 1, size=(n, axes)).astype(np.int32)
    if n > 2:
        p[0], p[1], p[2] = 0, -2 ** 31, 2 ** 31 - 1  # the ends of the type
    return p


# y = x0 c + x1 s in fp32: c and s within 4 ulp (sincospif's 2 ulp bound, the
# 2^-28-turn rest of the angle = 2.4e-8 rad, the mscale product), two products
# and a sum: at most 8 roundings of 2^-24 of |x0| + |x1| each, times mscale;
# a bf16 result adds half a step, 2^-8 of the result.
def rope_bound(x, want, mscale, dtype):
    b = 8 * 2.0 ** -24 * 2 * np.abs(x).max(-1, keepdims=True) * mscale
    return b + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [qvg.QVG_ROPE_HALF, qvg.QVG_ROPE_INTERLEAVED])
@pytest.mark.parametrize("d,dims", [(128, (128,)), (128, (44, 42, 42)), (128, (64,)), (64, (64,)), (64, (24, 20, 20)),
                                    (64, (22,)), (128, (2,)), (128, (16, 6, 6, 4))])
@pytest.mark.parametrize("n,H,how", [(1, 1, "plain"), (37, 5, "parts"), (5, 24, "linear"), (130, 3, "ntk")])
def test_rope(dtype, layout, d, dims, n, H, how):
    kw, ref_kw = SCALINGS[how]
    plan = qvg.RopePlan(dims, layout=layout, **kw)
    f, axis = ref.frequencies(dims, **ref_kw)
    x = values((n, H, d), n + H, dtype)
    pos = positions_of(n, len(dims), n, 10 ** 6)
    ms = kw.get("mscale", 1.0)
    for tr in (False, True):
        got = qvg.rope(plan, x.cuda(), torch.from_numpy(pos).cuda(), transpose=tr)
        # angles in exact turns: the plan's own steps, whose frequencies the
        # CPU tests check (at position 2^31 a double's frequency is itself off)
        turns = np.array([[(int(p[axis[i]]) * plan._c.step[i]) % 2 ** 64 / 2.0 ** 64 for i in range(len(f))] for p in pos])
        want = rope_turns(x.double().numpy(), turns, layout, ms, tr)
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= rope_bound(x.double().numpy(), want, ms, dtype)).all()
        # and at ordinary positions, the formula itself
        near = np.abs(pos).max(-1) <= 10 ** 6
        want = ref.rope(x.double().numpy(), pos, f, axis, layout, ms, tr)[near]
        err = np.abs(got.double().cpu().numpy()[near] - want)
        assert (err <= rope_bound(x.double().numpy()[near], want, ms, dtype)).all()


def rope_turns(x, turns, layout, mscale, transpose):
    m = turns.shape[1]
    turns = (turns + 0.5) % 1 - 0.5
    c, s = mscale * np.cos(2 * np.pi * turns)[:, None], mscale * np.sin(2 * np.pi * turns)[:, None] * (-1 if transpose else 1)
    ia = np.arange(m) if layout == 0 else 2 * np.arange(m)
    ib = ia + m if layout == 0 else ia + 1
    y = x.copy()
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    return y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dims", [(128,), (64,), (42,)])
def test_rope_strided_and_in_place(dtype, dims):
    """Rows of a fused projection, an output with its own stride, and in place
    give the bits of the plain call; what lies between rows stays."""
    plan = qvg.RopePlan(dims)
    wide = values((9, 3 * 4, 128), 1, dtype).cuda()
    x = wide[:, 4:8]
    pos = torch.arange(9, dtype=torch.int32, device="cuda") * 1000
    want = qvg.rope(plan, x.contiguous(), pos)
    assert torch.equal(qvg.rope(plan, x, pos), want)
    keep = wide.clone()
    got = qvg.rope(plan, x, pos, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
    assert torch.equal(wide[:, :4], keep[:, :4]) and torch.equal(wide[:, 8:], keep[:, 8:])
    out = torch.full((9, 5, 128), 7.0, dtype=dtype, device="cuda")
    qvg.rope(plan, want, pos, transpose=True, out=out[:, :4])
    assert (out[:, 4] == 7).all()
    # an element's offset from 16 bytes takes the narrow kernel
    flat = torch.zeros(9 * 512 + 1, dtype=dtype, device="cuda")
    odd = flat[1:].view(9, 4, 128)
    odd.copy_(keep[:, 4:8])
    assert torch.equal(qvg.rope(plan, odd, pos), want)


def test_rope_gradient():
    """transpose=True is the gradient: <dy, R x> = <R^T dy, x>, and central
    differences of a scalar loss (linear in x, so exact up to fp32 rounding)."""
    plan = qvg.RopePlan((64,), layout=qvg.QVG_ROPE_INTERLEAVED, mscale=1.5)
    x, dy = (values((6, 2, 128), s, torch.float32).cuda() for s in (1, 2))
    pos = torch.arange(6, dtype=torch.int32, device="cuda") * 12345
    gx = qvg.rope(plan, dy, pos, transpose=True)
    a = (dy.double() * qvg.rope(plan, x, pos).double()).sum()
    b = (gx.double() * x.double()).sum()
    terms = (dy.double() * qvg.rope(plan, x, pos).double()).abs().sum()
    assert abs(a - b) <= 32 * 2.0 ** -24 * terms
    for i, h, c in ((0, 0, 0), (3, 1, 17), (5, 0, 63), (2, 1, 100)):
        e = torch.zeros_like(x)
        e[i, h, c] = 1.0
        diff = (dy.double() * (qvg.rope(plan, x + e, pos).double() - qvg.rope(plan, x - e, pos).double())).sum() / 2
        # |x| + 1 <= 6, |dy| <= 6, mscale 1.5: two channels change, 8 roundings of 2^-24 each, and x +- 1 is rounded
        assert abs(diff - gx[i, h, c].double()) <= 2 * 10 * 2.0 ** -24 * 6 * 6 * 1.5 * 2


def test_rope_autograd():
    """The pair of calls as an autograd function: the gradients of a loss over
    rotated queries are those of the plain form in 64 bits."""
    plan = qvg.RopePlan((44, 42, 42))
    pos = torch.from_numpy(positions_of(33, 3, 5, 500)[3:]).cuda()

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return qvg.rope(plan, x, pos)

        @staticmethod
        def backward(ctx, dy):
            return qvg.rope(plan, dy.contiguous(), pos, transpose=True)

    x = values((30, 4, 128), 3, torch.float32).cuda().requires_grad_()
    Rope.apply(x).pow(3).sum().backward()
    f, axis = ref.frequencies((44, 42, 42))
    xd = x.detach().double().cpu().numpy()
    y = ref.rope(xd, pos.cpu().numpy(), f, axis, 0)
    want = ref.rope(3 * y ** 2, pos.cpu().numpy(), f, axis, 0, transpose=True)
    # y is off by 16 2^-24 max|x|; 3 y^2 by 6 |y| times that and 2 roundings; then the rotation's own bound
    top = np.abs(xd).max() * np.sqrt(2)
    bound = 2 * (6 * top * 16 * 2.0 ** -24 * top + 3 * top ** 2 * 20 * 2.0 ** -24)
    assert np.abs(x.grad.double().cpu().numpy() - want).max() <= bound


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("transpose", [False, True])
def test_rope_keeps_the_gradient(dtype, transpose):
    """The gradient of a loss over qvg.rope of a part of a fused projection
    reaches the projection and is the transposed rotation, for dy as a tensor
    and as an expanded scalar; no_grad and inputs without one are as before."""
    plan = qvg.RopePlan((24, 20, 20), layout=qvg.QVG_ROPE_INTERLEAVED, mscale=1.25)
    pos = torch.from_numpy(positions_of(30, 3, 5, 500)[3:]).cuda()
    wide = values((27, 6, 128), 8, dtype).cuda().requires_grad_()
    x = wide[:, 2:5]
    y = qvg.rope(plan, x, pos, transpose=transpose)
    assert y.requires_grad and torch.equal(y.detach(), qvg.rope(plan, x.detach(), pos, transpose=transpose))
    dy = values((27, 3, 128), 9, dtype).cuda()
    y.backward(dy)
    want = torch.zeros_like(wide)
    want[:, 2:5] = qvg.rope(plan, dy, pos, transpose=not transpose)
    assert torch.equal(wide.grad, want)
    f, axis = ref.frequencies((24, 20, 20))
    formula = ref.rope(dy.double().cpu().numpy(), pos.cpu().numpy(), f, axis, 1, 1.25, not transpose)
    err = np.abs(want[:, 2:5].double().cpu().numpy() - formula)
    assert (err <= rope_bound(dy.double().cpu().numpy(), formula, 1.25, dtype)).all()
    wide.grad = None
    qvg.rope(plan, x, pos, transpose=transpose).sum().backward()
    assert torch.equal(wide.grad[:, 2:5], qvg.rope(plan, torch.ones_like(dy), pos, transpose=not transpose))
    with torch.no_grad():
        assert not qvg.rope(plan, x, pos).requires_grad
        out = torch.empty_like(y)
        assert torch.equal(qvg.rope(plan, x, pos, transpose=transpose, out=out), y)
    assert not qvg.rope(plan, dy, pos).requires_grad


def test_rope_gradient_by_differences():
    """A loss that is not linear: autograd against central differences in
    64 bits of the plain form, and the second derivative through the graph."""
    plan = qvg.RopePlan((64,))
    pos = torch.arange(5, dtype=torch.int32, device="cuda") * 77
    x = values((5, 2, 64), 10, torch.float32).cuda().requires_grad_()
    g, = torch.autograd.grad(qvg.rope(plan, x, pos).pow(3).sum(), x, create_graph=True)
    f, axis = ref.frequencies((64,))
    xd, pn = x.detach().double().cpu().numpy(), pos.cpu().numpy()[:, None]
    loss = lambda a: (ref.rope(a, pn, f, axis, 0) ** 3).sum()  # noqa: E731
    top = np.abs(xd).max() * np.sqrt(2)
    for i, h, c in ((0, 0, 0), (3, 1, 17), (4, 0, 63)):
        e = np.zeros_like(xd)
        e[i, h, c] = 1e-4
        # a cubic's central difference is off by its third derivative's step: 1e-8 times a few; g as in test_rope_autograd
        bound = 2 * (6 * top * 16 * 2.0 ** -24 * top + 3 * top ** 2 * 20 * 2.0 ** -24) + 1e-6
        assert abs((loss(xd + e) - loss(xd - e)) / 2e-4 - float(g[i, h, c].detach())) <= bound
    # H u for u = 1: R^T (6 y R u), each rotation off by 16 2^-24 of its largest input, products by 2^-24
    hu, = torch.autograd.grad(g.sum(), x)
    ones = np.ones_like(xd)
    mid = 6 * ref.rope(xd, pn, f, axis, 0) * ref.rope(ones, pn, f, axis, 0)
    want = ref.rope(mid, pn, f, axis, 0, transpose=True)
    assert np.abs(hu.double().cpu().numpy() - want).max() <= 64 * 2.0 ** -24 * 6 * top * 2 * 2


def test_rope_gradient_on_a_stream_and_captured():
    """Forward and backward on a side stream, and captured into a graph that
    is replayed with other inputs while the eager graph of the leaf lives."""
    plan = qvg.RopePlan((128,))
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    x = values((40, 3, 128), 11, torch.float32).cuda().requires_grad_()
    step = lambda t: torch.autograd.grad(qvg.rope(plan, t, pos).pow(2).sum(), t)[0]  # noqa: E731
    want = step(x)
    alive = qvg.rope(plan, x, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(x)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    other = torch.zeros_like(x).requires_grad_()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = step(other)
    with torch.no_grad():
        other.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, want) and alive.requires_grad


# ---- the cache --------------------------------------------------------------------------

def rows(n, H, d, seed):
    """Rows of many magnitudes: ordinary, tiny, huge, all zero, ties of both
    formats, one large channel."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, H, d)) * np.exp2(g.integers(-40, 40, size=(n, H, 1)))
    x[::7] = g.standard_normal((len(x[::7]), H, d))
    x[1::11, :, d // 3] = 3e38
    x[2::11] = 0.0
    x[3::11] = g.integers(-32, 33, size=(len(x[3::11]), H, d)) / 8  # ties of e2m1, exact in e4m3
    x[4::11] = g.integers(-256, 257, size=(len(x[4::11]), H, d)) * 2.0 ** -3  # ties of e4m3
    x[5::11] = g.standard_normal((len(x[5::11]), H, d)) * 2.0 ** -128  # bf16 subnormals
    x[6::11, :, 0] = -448.0
    return ref.bf16(x)


def make(H, d, page, pages, bits, fill=0xA5):
    c = qvg.PagedKV(H, d, page, pages, bits)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(fill)
    return c


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("n,H,d,page", [(1, 1, 64, 16), (2, 1, 64, 16), (3, 2, 128, 16), (77, 5, 64, 32), (200, 3, 128, 64), (33, 16, 128, 256),
                                        (300, 1, 128, 128)])
def test_append_and_read(bits, n, H, d, page):
    """Codes and scales bit for bit; nothing beside the slots is written; what
    is read back is exactly what they stand for, in both types."""
    pages = -(-n // page) + 2
    c = make(H, d, page, pages, bits)
    g = np.random.default_rng(n)
    slots = g.permutation(pages * page)[:n].astype(np.int64)
    k, v = rows(n, H, d, 1), rows(n, H, d, 2)
    slots[n // 2:n // 2 + 1] = -1  # skipped
    to = lambda a: torch.from_numpy(a).to("cuda", torch.bfloat16)  # noqa: E731
    qvg.paged_append(c, to(k), to(v), torch.from_numpy(slots).cuda())
    live = slots >= 0
    at = slots[live] // page, slice(None), slots[live] % page
    free = np.ones(pages * page, bool)
    free[slots[live]] = False
    for x, codes, scales in ((k, c.k_codes, c.k_scales), (v, c.v_codes, c.v_scales)):
        r, s = ref.quantise(x, bits)
        codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
        np.testing.assert_array_equal(scales[at], s[live])
        np.testing.assert_array_equal(ref.code_values(codes[at], bits), r[live])
        for b in (codes, scales):
            rest = b.transpose(0, 2, 1, 3).reshape(pages * page, -1)[free]
            assert (rest == 0xA5).all()
    for dt in (qvg.QVG_OUT_BF16, qvg.QVG_OUT_F32):
        kk, vv = qvg.paged_read(c, torch.from_numpy(slots).cuda(), out_dtype=dt)
        for x, got in ((k, kk), (v, vv)):
            want = ref.dequantise(*ref.quantise(x, bits))
            want[~live] = 0.0
            np.testing.assert_array_equal(got.double().cpu().numpy(), want)
            # a value is off by half a step of its code at most
            half = 2.0 ** -4 if bits == 8 else 0.25
            grp = np.abs(x).reshape(n, H, -1, d if bits == 8 else 32).max(-1, keepdims=True)
            floor = np.maximum(grp * 2.0 ** (-10 - 7 if bits == 8 else -1 - 1), 2.0 ** -127 * 2.0 ** (-9 if bits == 8 else -1))
            err = np.abs(want - x).reshape(n, H, -1, d if bits == 8 else 32)
            assert (err <= np.maximum(half * np.abs(x).reshape(err.shape), floor))[live].all()


@pytest.mark.parametrize("bits", [8, 4])
def test_non_finite_rows(bits):
    """A row with an infinity or a NaN holds codes 0 and scale bytes 255 and
    reads as NaN; its neighbours are untouched."""
    x = rows(8, 2, 64, 3)
    x[1, 0, 5], x[2, 1, 40], x[3, 0, 63] = np.inf, np.nan, -np.inf
    c = make(2, 64, 16, 1, bits)
    slots = torch.arange(8, device="cuda")
    t = torch.from_numpy(x).to("cuda", torch.bfloat16)
    qvg.paged_append(c, t, t, slots)
    r, s = ref.quantise(x, bits)
    assert (s == 255).sum() == 3 * s.shape[-1]
    np.testing.assert_array_equal(c.k_scales[0, :, :8].cpu().numpy(), s.transpose(1, 0, 2))
    np.testing.assert_array_equal(ref.code_values(c.v_codes[0, :, :8].cpu().numpy(), bits), r.transpose(1, 0, 2))
    kk, _ = qvg.paged_read(c, slots)
    np.testing.assert_array_equal(kk.double().cpu().numpy(), ref.dequantise(r, s))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("layout", [qvg.QVG_ROPE_HALF, qvg.QVG_ROPE_INTERLEAVED])
@pytest.mark.parametrize("d,dims", [(128, (128,)), (128, (44, 42, 42)), (64, (22,)), (64, (64,)), (128, (96,))])
def test_append_rotates(bits, layout, d, dims):
    """K rotated on the way is K rotated by qvg_rope and then appended, byte
    for byte; V is not rotated.  Keys and values may be views of one tensor."""
    plan = qvg.RopePlan(dims, layout=layout, mscale=1.125)
    both = values((50, 2, 3, d), 4, torch.bfloat16).cuda()
    k, v = both[:, 0], both[:, 1]
    pos = torch.from_numpy(positions_of(50, len(dims), 9, 10 ** 5)).cuda()
    slots = torch.randperm(64, device="cuda")[:50]
    a, b = make(3, d, 32, 2, bits), make(3, d, 32, 2, bits)
    qvg.paged_append(a, k, v, slots, plan=plan, positions=pos)
    qvg.paged_append(b, qvg.rope(plan, k, pos), v.contiguous(), slots)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("layout", [qvg.QVG_ROPE_HALF, qvg.QVG_ROPE_INTERLEAVED])
@pytest.mark.parametrize("d,dims", [(128, (128,)), (128, (44, 20)), (64, (22,)), (128, (96,))])
def test_append_rotates_zeros_of_either_sign(bits, layout, d, dims):
    """The same where many channels are 0 or -0 beside values of either sign,
    among the rotated channels and the others."""
    plan = qvg.RopePlan(dims, layout=layout)
    g = torch.Generator().manual_seed(12)
    x = torch.randn(300, 2, d, generator=g)
    x = torch.where(torch.rand(x.shape, generator=g) < 0.6, torch.copysign(torch.zeros(()), x), x).bfloat16().cuda()
    pos = torch.from_numpy(positions_of(300, len(dims), 13, 1000)).cuda()
    slots = torch.arange(300, device="cuda")
    a, b = make(2, d, 16, 20, bits), make(2, d, 16, 20, bits)
    qvg.paged_append(a, x, x, slots, plan=plan, positions=pos)
    qvg.paged_append(b, qvg.rope(plan, x, pos), x, slots)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_slots_beyond_the_cache():
    """A slot past the end is skipped (append) or zeros (read) and reported
    once; the other tokens are served."""
    c = make(1, 64, 16, 2, 8)
    x = values((4, 1, 64), 5, torch.bfloat16).cuda()
    slots = torch.tensor([3, 32, 7, 2 ** 40], device="cuda")
    qvg.paged_append(c, x, x, slots)
    assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG
    assert qvg.get_status() == qvg.QVG_OK
    kk, vv = qvg.paged_read(c, slots)
    assert qvg.get_status() == qvg.QVG_ERR_INVALID_ARG
    want = ref.dequantise(*ref.quantise(x.double().cpu().numpy(), 8))
    want[[1, 3]] = 0
    np.testing.assert_array_equal(kk.double().cpu().numpy(), want)
    np.testing.assert_array_equal(vv.double().cpu().numpy(), want)


def test_offsets_past_32_bits():
    """A cache whose K codes pass 4 GB: the last page holds what is written."""
    H, d, page = 32, 128, 128
    pages = (1 << 32) // (H * page * d) + 9
    c = qvg.PagedKV(H, d, page, pages, 8)
    n = 40
    x = values((n, H, d), 6, torch.bfloat16).cuda()
    slots = torch.arange(n, device="cuda") + (pages - 1) * page
    qvg.paged_append(c, x, x, slots)
    kk, vv = qvg.paged_read(c, slots)
    want = ref.dequantise(*ref.quantise(x.double().cpu().numpy(), 8))
    np.testing.assert_array_equal(kk.double().cpu().numpy(), want)
    np.testing.assert_array_equal(vv.double().cpu().numpy(), want)
    assert int(c.k_codes[:-1].count_nonzero()) == 0


def test_streams_and_graph():
    """Calls on a side stream while the current one is busy, and a captured
    rotate + append + read replayed with other inputs."""
    plan = qvg.RopePlan((128,))
    c = make(4, 128, 64, 2, 8)
    x = values((60, 4, 128), 7, torch.bfloat16).cuda()
    pos = torch.arange(60, dtype=torch.int32, device="cuda")
    slots = torch.arange(60, device="cuda") + 5
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = qvg.rope(plan, x, pos, stream=side)
    qvg.paged_append(c, y, x, slots, stream=side)
    a, b = qvg.paged_read(c, slots, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = [t.clone() for t in (a, b)]
    graph = torch.cuda.CUDAGraph()
    xs, ps = torch.zeros_like(x), torch.zeros_like(pos)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        qvg.paged_append(c, xs, xs, slots, plan=plan, positions=ps)
        ka, va = qvg.paged_read(c, slots)
    xs.copy_(x)
    ps.copy_(pos)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ka, want[0]) and torch.equal(va, want[1])
