"""Python binding of libqvg: compressed video KV cache (QVG / QVG-Pro with
QuantWM QSAC / PSAC) on one GB300, and the operators of single tokens: rotary
positions, a paged 8-bit / 4-bit cache, and attention over its pages.

Argument marshalling only: every step of compression, reconstruction,
attention, the QuantWM statistics and the token-wise operators runs in the CUDA kernels of
``libqvg.so``; PyTorch provides device memory and streams.  There is no
fallback: if the library is missing or no CUDA device is present, the calls
raise.  rope() carries gradients; nothing else here does.

Names follow the C ABI in ``include/qvg.h``.
"""
from __future__ import annotations

import ctypes as ct
import dataclasses
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqvg.so")

QVG_OK, QVG_ERR_INVALID_ARG, QVG_ERR_UNSUPPORTED, QVG_ERR_CUDA = 0, 1, 2, 3
QVG_ERR_TIMEOUT, QVG_ERR_WORKSPACE, QVG_ERR_CAPACITY = 4, 5, 6
QVG_QSAC, QVG_PSAC, QVG_GIVEN_CENTROIDS, QVG_OUTLIER, QVG_KEEP_MEANS = 1, 2, 4, 8, 16
QVG_TILE = 128
QVG_PSAC_RANK = 8
QVG_CACHE_NBUF = 14
QVG_OUT_F32, QVG_OUT_BF16 = 0, 1
QVG_OP_COMPRESS, QVG_OP_ATTENTION, QVG_OP_PSAC_BASIS = 0, 1, 2
QVG_ROPE_HALF, QVG_ROPE_INTERLEAVED = 0, 1
QVG_ROPE_PLAIN, QVG_ROPE_LINEAR, QVG_ROPE_NTK, QVG_ROPE_PARTS = 0, 1, 2, 3
QVG_ROPE_MAX_PAIRS, QVG_ROPE_MAX_AXES = 64, 4
QVG_MASK_NONE, QVG_MASK_CAUSAL, QVG_MASK_TREE = 0, 1, 2

EXPORTED = (
    "qvg_status_string", "qvg_cache_bytes", "qvg_workspace_size", "qvg_compress_chunk",
    "qvg_decompress", "qvg_attention", "quantwm_query_stats", "quantwm_psac_basis",
    "qvg_get_status", "qvg_last_cuda_error", "qvg_compress_chunk_noalloc", "qvg_attention_ar",
    "qvg_debug_set_wait", "qvg_rope_plan_init", "qvg_rope", "qvg_paged_bytes", "qvg_paged_append",
    "qvg_paged_read", "qvg_tree_mask", "qvg_paged_workspace_size", "qvg_paged_attention",
)
NOALLOC_SCRATCH_BYTES = 32 << 20

BUFFER_NAMES = ("codes", "scales", "ids", "cent", "chunk_start", "chunk_len", "tile_chunk",
                "psac_p", "psac_s", "psac_basis", "outl_val", "outl_idx", "anchor", "chunk_anchor")


class QvgError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, status_string(status), status))


class _Params(ct.Structure):
    _fields_ = [("C", ct.c_int32), ("L", ct.c_int32), ("bits", ct.c_int32),
                ("group", ct.c_int32), ("iters", ct.c_int32), ("scale_mode", ct.c_int32),
                ("flags", ct.c_int32), ("anchor_every", ct.c_int32), ("seed", ct.c_uint64)]


class _Cache(ct.Structure):
    _fields_ = [("H", ct.c_int32), ("d", ct.c_int32), ("capacity_tokens", ct.c_int32),
                ("max_chunks", ct.c_int32), ("n_chunks", ct.c_int32), ("n_tokens", ct.c_int32),
                ("codes", ct.c_void_p), ("scales", ct.c_void_p), ("ids", ct.c_void_p),
                ("cent", ct.c_void_p), ("chunk_start", ct.c_void_p), ("chunk_len", ct.c_void_p),
                ("tile_chunk", ct.c_void_p), ("psac_p", ct.c_void_p), ("psac_s", ct.c_void_p),
                ("psac_basis", ct.c_void_p), ("outl_val", ct.c_void_p), ("outl_idx", ct.c_void_p),
                ("anchor", ct.c_void_p), ("chunk_anchor", ct.c_void_p)]


class _RopePlan(ct.Structure):
    _fields_ = [("dims", ct.c_int32), ("axes", ct.c_int32), ("layout", ct.c_int32), ("mscale", ct.c_float),
                ("step", ct.c_uint64 * QVG_ROPE_MAX_PAIRS), ("axis", ct.c_uint8 * QVG_ROPE_MAX_PAIRS)]


class _Paged(ct.Structure):
    _fields_ = [("H", ct.c_int32), ("d", ct.c_int32), ("page_size", ct.c_int32), ("num_pages", ct.c_int32),
                ("bits", ct.c_int32), ("k_codes", ct.c_void_p), ("k_scales", ct.c_void_p),
                ("v_codes", ct.c_void_p), ("v_scales", ct.c_void_p)]


_lib = None


def lib():
    """Load libqvg.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libqvg.so is not built; run __graft_entry__.build() "
                               "or python video_diffusion_kv_gb300/build.py")
        L = ct.CDLL(LIB_PATH)
        L.qvg_status_string.restype = ct.c_char_p
        L.qvg_status_string.argtypes = [ct.c_int]
        vp, i32, sz = ct.c_void_p, ct.c_int32, ct.c_size_t
        L.qvg_cache_bytes.argtypes = [vp, i32, i32, i32, i32, vp]
        L.qvg_workspace_size.argtypes = [vp, i32, i32, i32, i32, i32, vp]
        L.qvg_compress_chunk.argtypes = [vp, vp, i32, vp, vp, vp, vp, sz, vp]
        L.qvg_compress_chunk_noalloc.argtypes = [vp, vp, i32, vp, vp, vp, vp]
        L.qvg_decompress.argtypes = [vp, vp, i32, i32, vp, i32, vp]
        L.qvg_attention.argtypes = [vp, vp, i32, i32, vp, vp, ct.c_float, vp, i32, vp, vp, vp, sz, vp]
        L.qvg_attention_ar.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, i32, ct.c_float, vp, i32, vp, vp, vp,
                                       sz, vp]
        L.quantwm_query_stats.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp]
        L.quantwm_psac_basis.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp]
        i64, dbl = ct.c_int64, ct.c_double
        L.qvg_rope_plan_init.argtypes = [vp, i32, vp, i32, dbl, i32, dbl, dbl, dbl, dbl, ct.c_uint32, ct.c_float]
        L.qvg_rope.argtypes = [vp, vp, i32, i32, i32, i32, i64, vp, i32, vp, i64, vp]
        L.qvg_paged_bytes.argtypes = [i32, i32, i32, i32, i32, vp, vp]
        L.qvg_paged_append.argtypes = [vp, vp, vp, i32, i64, i64, vp, vp, vp, vp]
        L.qvg_paged_read.argtypes = [vp, vp, i32, vp, vp, i32, vp]
        L.qvg_tree_mask.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp]
        L.qvg_paged_workspace_size.argtypes = [i32, i32, i32, i32, i32, vp]
        L.qvg_paged_attention.argtypes = [vp, vp, i64, i32, i32, i32, i32, vp, vp, i32, vp, i32, vp, i32, ct.c_float,
                                          vp, i32, vp, vp, sz, vp]
        L.qvg_get_status.argtypes = [vp]
        L.qvg_debug_set_wait.argtypes = [ct.c_uint64, i32]
        L.qvg_last_cuda_error.restype = ct.c_char_p
        L.qvg_last_cuda_error.argtypes = []
        _lib = L
    return _lib


def status_string(s):
    return lib().qvg_status_string(int(s)).decode()


def _check(s, where):
    if s != QVG_OK:
        if s == QVG_ERR_CUDA:
            where = "%s [%s]" % (where, lib().qvg_last_cuda_error().decode())
        raise QvgError(s, where)


@dataclasses.dataclass
class Params:
    """Method parameters (see qvg_params in include/qvg.h)."""
    C: int = 256
    L: int = 1
    bits: int = 2
    group: int = 64
    iters: int = 8
    scale_mode: int = 0
    flags: int = 0
    seed: int = 0
    anchor_every: int = 0

    def c(self):
        return _Params(self.C, self.L, self.bits, self.group, self.iters, self.scale_mode,
                       self.flags, self.anchor_every, self.seed)


def _ptr(t):
    return None if t is None else ct.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ct.c_void_p(s.cuda_stream)


def kv_bytes_uncompressed(layers, kv_heads, head_dim, tokens, bytes_per_elt=2):
    """KV cache size before compression: 2 (K and V) x layers x KV heads x
    head_dim x tokens x bytes per element ("The 2-bit quantisation trap",
    section 1)."""
    return 2 * layers * kv_heads * head_dim * tokens * bytes_per_elt


def cache_bytes(params: Params, H, d, capacity_tokens, max_chunks):
    """Per-buffer byte sizes of one compressed tensor (dict)."""
    out = (ct.c_size_t * QVG_CACHE_NBUF)()
    p = params.c()
    _check(lib().qvg_cache_bytes(ct.byref(p), H, d, capacity_tokens, max_chunks, out), "qvg_cache_bytes")
    return dict(zip(BUFFER_NAMES, [int(v) for v in out]))


def workspace_size(params: Params, op, n, H, d, Hq=None):
    b = ct.c_size_t(0)
    p = params.c()
    _check(lib().qvg_workspace_size(ct.byref(p), op, n, H, d, Hq or H, ct.byref(b)), "qvg_workspace_size")
    return int(b.value)


class CompressedKV:
    """One compressed tensor (K or V) of one layer: device buffers allocated
    with torch at the sizes libqvg reports, plus the host-side counters."""

    def __init__(self, params: Params, H, d, capacity_tokens, max_chunks, device="cuda"):
        import torch
        capacity_tokens = -(-capacity_tokens // QVG_TILE) * QVG_TILE
        self.params = dataclasses.replace(params)
        self.H, self.d = H, d
        self.capacity_tokens, self.max_chunks = capacity_tokens, max_chunks
        sizes = cache_bytes(params, H, d, capacity_tokens, max_chunks)
        self.sizes = sizes
        self.buffers = {}
        for name in BUFFER_NAMES:
            n = sizes[name]
            self.buffers[name] = torch.zeros(max(n, 0), dtype=torch.uint8, device=device) if n else None
        self.n_chunks = 0
        self.n_tokens = 0

    @property
    def nbytes(self):
        return sum(self.sizes.values())

    def c(self):
        b = self.buffers
        return _Cache(self.H, self.d, self.capacity_tokens, self.max_chunks, self.n_chunks,
                      self.n_tokens, *[_ptr(b[n]) for n in BUFFER_NAMES])

    def reset(self, n_chunks=0, n_tokens=0):
        self.n_chunks, self.n_tokens = n_chunks, n_tokens

    def view(self, name, dtype, shape):
        """Typed view of one buffer (for inspection and checkpointing)."""
        return self.buffers[name].view(dtype).view(*shape)

    def centroid_slot(self, chunk):
        """bf16 [L, H, C, d] view of one chunk's centroids."""
        import torch
        p = self.params
        cent = self.view("cent", torch.bfloat16, (p.L, self.H, self.max_chunks, p.C, self.d))
        return cent[:, :, chunk]


def compress_chunk(params: Params, x, cache: CompressedKV, qsac_w=None, psac_basis=None,
                   workspace=None, stream=None):
    """Append one chunk x (bf16 [N, H, d], contiguous, on the GPU) to cache.
    Returns the first token slot of the chunk.  With QVG_KEEP_MEANS in
    params.flags, pass a workspace and read the fp32 means from it with
    kept_means()."""
    import torch
    assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.dim() == 3
    N = x.shape[0]
    need = workspace_size(params, QVG_OP_COMPRESS, N, cache.H, cache.d)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    c = cache.c()
    p = params.c()
    slot0 = cache.n_tokens
    s = lib().qvg_compress_chunk(ct.byref(p), _ptr(x), N, _ptr(qsac_w), _ptr(psac_basis), ct.byref(c),
                                 _ptr(workspace), workspace.numel(), _stream(stream))
    _check(s, "qvg_compress_chunk")
    cache.n_chunks, cache.n_tokens = c.n_chunks, c.n_tokens
    return slot0


def kept_means(params: Params, workspace, H, d):
    """fp32 [L, H, C, d] view of the centroid means a QVG_KEEP_MEANS
    compression left at the start of its workspace."""
    import torch
    n = params.L * H * params.C * d
    return workspace[:4 * n].view(torch.float32).view(params.L, H, params.C, d)


def compress_chunk_noalloc(params: Params, x, cache: CompressedKV, qsac_w=None, psac_basis=None,
                           stream=None):
    """compress_chunk without a workspace argument: for callers that cannot
    allocate device memory, the library uses its own fixed 32 MiB device
    scratch (see qvg_compress_chunk_noalloc in include/qvg.h; calls that
    overlap on the GPU race on it).  Returns the first token slot."""
    import torch
    assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.dim() == 3
    c = cache.c()
    p = params.c()
    slot0 = cache.n_tokens
    s = lib().qvg_compress_chunk_noalloc(ct.byref(p), _ptr(x), x.shape[0], _ptr(qsac_w), _ptr(psac_basis),
                                         ct.byref(c), _stream(stream))
    _check(s, "qvg_compress_chunk_noalloc")
    cache.n_chunks, cache.n_tokens = c.n_chunks, c.n_tokens
    return slot0


def decompress(params: Params, cache: CompressedKV, tok0, ntok, out_dtype=QVG_OUT_F32, out=None,
               stream=None):
    import torch
    dt = torch.float32 if out_dtype == QVG_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((ntok, cache.H, cache.d), dtype=dt, device=cache.buffers["codes"].device)
    c = cache.c()
    p = params.c()
    _check(lib().qvg_decompress(ct.byref(p), ct.byref(c), tok0, ntok, _ptr(out), out_dtype, _stream(stream)),
           "qvg_decompress")
    return out


def attention(params: Params, q, kc: CompressedKV, vc: CompressedKV, scale=0.0,
              out_dtype=QVG_OUT_F32, want_lse=False, want_top1=False, out=None, workspace=None,
              stream=None, allow_split=True):
    """O = softmax(scale Q K_hat^T) V_hat over every cached token.
    q: bf16 [Nq, Hq, d].  Returns (out, lse or None, top1 or None).
    allow_split=False passes no workspace, so the cache is never split over
    extra CTAs."""
    import torch
    assert q.dtype == torch.bfloat16 and q.is_contiguous() and q.dim() == 3
    Nq, Hq, d = q.shape
    dt = torch.float32 if out_dtype == QVG_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((Nq, Hq, d), dtype=dt, device=q.device)
    lse = torch.empty((Hq, Nq), dtype=torch.float32, device=q.device) if want_lse else None
    top1 = torch.empty((Hq, Nq), dtype=torch.int32, device=q.device) if want_top1 else None
    need = workspace_size(params, QVG_OP_ATTENTION, Nq, kc.H, d, Hq) if allow_split else 0
    if not allow_split:
        workspace = None
    elif need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    k, v = kc.c(), vc.c()
    p = params.c()
    s = lib().qvg_attention(ct.byref(p), _ptr(q), Nq, Hq, ct.byref(k), ct.byref(v), float(scale),
                            _ptr(out), out_dtype, _ptr(lse), _ptr(top1), _ptr(workspace),
                            0 if workspace is None else workspace.numel(), _stream(stream))
    _check(s, "qvg_attention")
    return out, lse, top1


def attention_ar(params: Params, q, kc: CompressedKV, vc: CompressedKV, k_cur, v_cur, scale=0.0,
                 out_dtype=QVG_OUT_F32, want_lse=False, want_top1=False, out=None, workspace=None,
                 stream=None):
    """One autoregressive step: softmax(scale Q [K_hat; K_cur]^T) [V_hat; V_cur]
    over the cached tokens and the current chunk's raw bf16 rows.
    q: bf16 [Nq, Hq, d]; k_cur, v_cur: bf16 [n_cur, H, d].  Returns
    (out, lse or None, top1 or None); current-chunk token j is slot
    kc.n_tokens + j in top1."""
    import torch
    assert q.dtype == torch.bfloat16 and q.is_contiguous() and q.dim() == 3
    for x in (k_cur, v_cur):
        assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.dim() == 3
    assert k_cur.shape == v_cur.shape and k_cur.shape[1:] == (kc.H, kc.d)
    Nq, Hq, d = q.shape
    n_cur = k_cur.shape[0]
    dt = torch.float32 if out_dtype == QVG_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((Nq, Hq, d), dtype=dt, device=q.device)
    lse = torch.empty((Hq, Nq), dtype=torch.float32, device=q.device) if want_lse else None
    top1 = torch.empty((Hq, Nq), dtype=torch.int32, device=q.device) if want_top1 else None
    need = workspace_size(params, QVG_OP_ATTENTION, Nq, kc.H, d, Hq)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    k, v = kc.c(), vc.c()
    p = params.c()
    s = lib().qvg_attention_ar(ct.byref(p), _ptr(q), Nq, Hq, ct.byref(k), ct.byref(v), _ptr(k_cur), _ptr(v_cur),
                               n_cur, float(scale), _ptr(out), out_dtype, _ptr(lse), _ptr(top1), _ptr(workspace),
                               0 if workspace is None else workspace.numel(), _stream(stream))
    _check(s, "qvg_attention_ar")
    return out, lse, top1


class RopePlan:
    """Rotary positions of one model (qvg_rope_plan_init): `axis_dims` channels
    per position axis, the first sum(axis_dims) of each head.  A host object;
    it may be shared by streams and devices."""

    def __init__(self, axis_dims, layout=QVG_ROPE_HALF, base=10000.0, scaling=QVG_ROPE_PLAIN, factor=1.0,
                 original=0.0, fast=32.0, slow=1.0, scaled_axes=0xFFFFFFFF, mscale=1.0):
        self._c = _RopePlan()
        dims = (ct.c_int32 * max(1, len(axis_dims)))(*axis_dims)
        _check(lib().qvg_rope_plan_init(ct.byref(self._c), len(axis_dims), dims, layout, base, scaling, factor,
                                        original, fast, slow, scaled_axes, mscale), "qvg_rope_plan_init")
        self._ref = ct.byref(self._c)
        self.dims, self.axes, self.layout = self._c.dims, self._c.axes, layout


def _heads(x, where):
    """(tokens, heads, channels, token stride) of a [n, H, d] tensor whose
    heads and channels are contiguous."""
    if x.dim() != 3:
        raise ValueError("%s: a [tokens, heads, channels] tensor is wanted" % where)
    n, H, d = x.shape
    s = x.stride()
    if (s[2] != 1 and d > 1) or (s[1] != d and H > 1):
        raise ValueError("%s: heads and channels must be contiguous" % where)
    return n, H, d, (s[0] if n > 1 else H * d)


def _on(dev, where, **tensors):
    """Checks (dtype, contiguity, device) of the tensors handed to a call that
    runs on `dev`."""
    for name, (t, dtype) in tensors.items():
        if t is None:
            continue
        if t.dtype != dtype:
            raise ValueError("%s: %s is %s, %s is wanted" % (where, name, t.dtype, dtype))
        if t.device != dev:
            raise ValueError("%s: %s is on %s, not on %s" % (where, name, t.device, dev))
        if not t.is_contiguous():
            raise ValueError("%s: %s must be contiguous" % (where, name))


class _Device:
    """Makes `dev` the current device of the calling thread, where it is not
    already (the library works on the current device)."""
    __slots__ = ("dev", "was")

    def __init__(self, dev):
        self.dev, self.was = dev, None

    def __enter__(self):
        import torch
        if self.dev.type != "cuda":
            raise ValueError("CUDA tensors are wanted, got one on %s" % self.dev)
        was = torch.cuda.current_device()
        if self.dev.index != was:
            self.was = was
            torch.cuda.set_device(self.dev)

    def __exit__(self, *exc):
        if self.was is not None:
            import torch
            torch.cuda.set_device(self.was)


def _raw_stream(stream, dev):
    """The CUDA stream of a call on `dev`: the given one, or torch's current."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _empty(shape, dtype, dev, stream):
    """An output or workspace for a kernel on `stream` (None: the current
    stream), from that stream's own memory: memory that the current stream
    has given back may still be in use there."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _positions(plan, positions, n, where):
    if positions is None:
        raise ValueError("%s: a plan needs positions" % where)
    if positions.numel() != n * plan.axes or (n > 0 and plan.axes > 1 and positions.shape[-1] != plan.axes):
        raise ValueError("%s: positions must be int32 [%d, %d]" % (where, n, plan.axes))


_rope_autograd = None


def _rope_with_gradient(plan, x, positions, transpose, stream):
    """rope as a node of torch's graph (the class is made at its first use:
    torch is imported by the calls)."""
    global _rope_autograd
    if _rope_autograd is None:
        import torch

        class Rope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, positions, plan, transpose, stream):
                ctx.plan, ctx.transpose = plan, transpose
                ctx.save_for_backward(positions)
                return rope(plan, x, positions, transpose=transpose, stream=stream)

            @staticmethod
            def backward(ctx, dy):  # torch runs it on the stream that was current in forward
                positions, = ctx.saved_tensors
                return rope(ctx.plan, dy.contiguous(), positions, transpose=not ctx.transpose), None, None, None, None

        _rope_autograd = Rope
    return _rope_autograd.apply(x, positions, plan, transpose, stream)


def rope(plan: RopePlan, x, positions, transpose=False, out=None, stream=None):
    """Rotate x (bf16 or fp32 [n, H, d]; tokens may be strided) at positions
    (int32 [n, axes], or [n] with one axis).  transpose=True turns the angles'
    signs: the gradient with respect to x.  out may be x itself.  Where x
    requires a gradient, the result has one (without `out`)."""
    import torch
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("rope: no gradient through out; leave it out, or call under torch.no_grad()")
        return _rope_with_gradient(plan, x, positions, transpose, stream)
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("rope: bf16 or fp32 is wanted, got %s" % x.dtype)
    n, H, d, xs = _heads(x, "rope")
    if out is None:
        out = _empty((n, H, d), x.dtype, x.device, stream)
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
        raise ValueError("rope: out must match x")
    _, _, _, os_ = _heads(out, "rope")
    _positions(plan, positions, n, "rope")
    _on(x.device, "rope", positions=(positions, torch.int32))
    with _Device(x.device):
        _check(lib().qvg_rope(plan._ref, x.data_ptr(), QVG_OUT_F32 if x.dtype == torch.float32 else QVG_OUT_BF16, n, H,
                              d, xs, positions.data_ptr(), 1 if transpose else 0, out.data_ptr(), os_,
                              _raw_stream(stream, x.device)), "qvg_rope")
    return out


def paged_bytes(H, d, page_size, num_pages, bits):
    """(codes, scales) bytes of one of a paged cache's two tensors."""
    a, b = ct.c_size_t(0), ct.c_size_t(0)
    _check(lib().qvg_paged_bytes(H, d, page_size, num_pages, bits, ct.byref(a), ct.byref(b)), "qvg_paged_bytes")
    return int(a.value), int(b.value)


class PagedKV:
    """K and V of one layer in pages of fp8 (bits=8) or fp4 (bits=4) codes
    with power-of-two scales (qvg_paged in include/qvg.h).  `buffers`: the four
    uint8 tensors (k codes, k scales, v codes, v scales) where the caller
    allocates them."""

    def __init__(self, H, d, page_size, num_pages, bits=8, device="cuda", buffers=None):
        import torch
        sizes = paged_bytes(H, d, page_size, num_pages, bits)
        self.H, self.d, self.page_size, self.num_pages, self.bits = H, d, page_size, num_pages, bits
        rows = (num_pages, H, page_size)
        shapes = [rows + (d * bits // 8,), rows + (1 if bits == 8 else d // 32,)] * 2
        if buffers is None:
            buffers = [torch.zeros(s, dtype=torch.uint8, device=device) for s in shapes]
        if len(buffers) != 4:
            raise ValueError("PagedKV: four buffers are wanted (k codes, k scales, v codes, v scales), got %d" % len(buffers))
        for t, need in zip(buffers, sizes * 2):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() != need or t.device != buffers[0].device:
                raise ValueError("PagedKV: each buffer must be contiguous uint8 of the size paged_bytes reports")
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel()) for t in buffers)
        if any(end > start for (_, end), (start, _) in zip(spans, spans[1:])):
            raise ValueError("PagedKV: the buffers overlap")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = (t.view(s) for t, s in zip(buffers, shapes))
        self.device = self.k_codes.device
        self._c = _Paged(H, d, page_size, num_pages, bits, self.k_codes.data_ptr(), self.k_scales.data_ptr(),
                         self.v_codes.data_ptr(), self.v_scales.data_ptr())
        self._ref = ct.byref(self._c)
        self._workspace = {}  # paged_attention's scratch bytes by (Hq, max_q): no sequence count changes them

    @property
    def nbytes(self):
        return sum(t.numel() for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales))


def paged_append(cache: PagedKV, k, v, slots, plan=None, positions=None, stream=None):
    """Quantise k and v (bf16 [n, H, d]; tokens may be strided) into the slots
    (int64 [n]; negative: skip).  With a RopePlan, K is rotated at `positions`
    on the way.  A slot beyond the cache is reported by get_status()."""
    import torch
    n, H, d, ks = _heads(k, "paged_append")
    _, _, _, vs = _heads(v, "paged_append")
    if k.shape != v.shape or (H, d) != (cache.H, cache.d) or slots.numel() != n:
        raise ValueError("paged_append: k, v must be [n, %d, %d] and slots [n]" % (cache.H, cache.d))
    if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16 or k.device != cache.device or v.device != cache.device:
        raise ValueError("paged_append: k and v must be bf16 on the cache's device")
    _on(cache.device, "paged_append", slots=(slots, torch.int64), positions=(positions, torch.int32))
    if plan is not None:
        _positions(plan, positions, n, "paged_append")
    with _Device(cache.device):
        _check(lib().qvg_paged_append(cache._ref, k.data_ptr(), v.data_ptr(), n, ks, vs, slots.data_ptr(),
                                      None if plan is None else plan._ref,
                                      None if plan is None else positions.data_ptr(), _raw_stream(stream, cache.device)),
               "qvg_paged_append")


def paged_read(cache: PagedKV, slots, out_dtype=QVG_OUT_BF16, k_out=None, v_out=None, stream=None):
    """The rows that the slots (int64 [n]; negative: zeros) hold: (K, V), each
    bf16 or fp32 [n, H, d]."""
    import torch
    n = slots.numel()
    dt = torch.float32 if out_dtype == QVG_OUT_F32 else torch.bfloat16
    shape = (n, cache.H, cache.d)
    k_out = _empty(shape, dt, cache.device, stream) if k_out is None else k_out
    v_out = _empty(shape, dt, cache.device, stream) if v_out is None else v_out
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError("paged_read: outputs must be [n, %d, %d]" % (cache.H, cache.d))
    _on(cache.device, "paged_read", slots=(slots, torch.int64), k_out=(k_out, dt), v_out=(v_out, dt))
    with _Device(cache.device):
        _check(lib().qvg_paged_read(cache._ref, slots.data_ptr(), n, k_out.data_ptr(), v_out.data_ptr(), out_dtype,
                                    _raw_stream(stream, cache.device)), "qvg_paged_read")
    return k_out, v_out


def tree_mask(parents, max_q, cu_q=None, out=None, stream=None):
    """Mask rows of drafted trees (int32 [total_q, ceil(max_q / 32)], read as
    unsigned bits): a token sees itself and its ancestors.  parents: int32
    [total_q], the parent's number within the sequence's new tokens or -1;
    cu_q: int32 [B + 1], or None when every sequence has max_q tokens."""
    import torch
    total, words = parents.numel(), max(1, -(-max_q // 32))
    if cu_q is None and (max_q < 1 or total % max_q != 0):
        raise ValueError("tree_mask: without cu_q every sequence has max_q tokens")
    if out is None:
        out = _empty((total, words), torch.int32, parents.device, stream)
    elif out.dim() != 2 or out.shape[0] != total or out.shape[1] < words:
        raise ValueError("tree_mask: out must be [total_q, words] with at least %d words" % words)
    B = total // max_q if cu_q is None else cu_q.numel() - 1
    _on(parents.device, "tree_mask", parents=(parents, torch.int32), cu_q=(cu_q, torch.int32), out=(out, torch.int32))
    with _Device(parents.device):
        _check(lib().qvg_tree_mask(parents.data_ptr(), None if cu_q is None else cu_q.data_ptr(), B, max_q, total,
                                   out.shape[1], out.data_ptr(), _raw_stream(stream, parents.device)), "qvg_tree_mask")
    return out


def paged_workspace_size(cache: PagedKV, Hq, B, max_q):
    """Scratch bytes of paged_attention."""
    b = ct.c_size_t(0)
    with _Device(cache.device):
        _check(lib().qvg_paged_workspace_size(cache.H, cache.d, Hq, B, max_q, ct.byref(b)), "qvg_paged_workspace_size")
    return int(b.value)


def paged_attention(cache: PagedKV, q, block_table, kv_len, max_q, cu_q=None, mask_mode=QVG_MASK_CAUSAL, mask=None,
                    scale=0.0, out_dtype=QVG_OUT_BF16, want_lse=False, out=None, workspace=None, stream=None):
    """Attention of the new tokens q (bf16 [total_q, Hq, d]; tokens may be
    strided), which are the last ones of their sequences, over the cache.
    block_table: int32 [B, pages]; kv_len: int32 [B], new tokens included;
    cu_q: int32 [B + 1] (None: max_q tokens each); mask: tree_mask's rows, with
    mask_mode QVG_MASK_TREE.  Returns (out, lse or None).  Two calls that run
    at once need a workspace each (None: one per call)."""
    import torch
    total, Hq, d, qs = _heads(q, "paged_attention")
    B = kv_len.numel()
    dt = torch.float32 if out_dtype == QVG_OUT_F32 else torch.bfloat16
    if q.dtype != torch.bfloat16 or q.device != cache.device or d != cache.d:
        raise ValueError("paged_attention: q must be bf16 [total_q, Hq, %d] on the cache's device" % cache.d)
    if block_table.dim() != 2 or block_table.shape[0] != B or (cu_q is not None and cu_q.numel() != B + 1):
        raise ValueError("paged_attention: block_table must be [B, pages], kv_len [B], cu_q [B + 1]")
    if mask_mode == QVG_MASK_TREE and (mask is None or mask.dim() != 2 or mask.shape[0] < total):
        raise ValueError("paged_attention: QVG_MASK_TREE needs mask rows [total_q, words]")
    if out is None:
        out = _empty((total, Hq, d), dt, q.device, stream)
    elif out.shape != (total, Hq, d):
        raise ValueError("paged_attention: out must be [total_q, Hq, d]")
    _on(q.device, "paged_attention", block_table=(block_table, torch.int32), kv_len=(kv_len, torch.int32),
        cu_q=(cu_q, torch.int32), mask=(mask, torch.int32), out=(out, dt), workspace=(workspace, torch.uint8))
    lse = _empty((Hq, total), torch.float32, q.device, stream) if want_lse else None
    if workspace is None:
        need = cache._workspace.get((Hq, max_q))
        if need is None:
            need = cache._workspace[Hq, max_q] = paged_workspace_size(cache, Hq, B, max_q)
        workspace = _empty((need,), torch.uint8, q.device, stream)
    with _Device(q.device):
        _check(lib().qvg_paged_attention(
            cache._ref, q.data_ptr(), qs, total, Hq, B, max_q, None if cu_q is None else cu_q.data_ptr(),
            block_table.data_ptr(), block_table.shape[1], kv_len.data_ptr(), mask_mode,
            None if mask is None else mask.data_ptr(), 0 if mask is None else mask.shape[1], scale, out.data_ptr(),
            out_dtype, None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
            _raw_stream(stream, q.device)), "qvg_paged_attention")
    return out, lse


def query_stats(q, H, M=None, w=None, count=None, accumulate=False, stream=None):
    """History-query statistics: returns (M fp32 [H,d,d], w fp32 [H,d], count int64 [1])."""
    import torch
    assert q.dtype == torch.bfloat16 and q.is_contiguous() and q.dim() == 3
    n, Hq, d = q.shape
    dev = q.device
    if M is None:
        M = torch.zeros((H, d, d), dtype=torch.float32, device=dev)
    if w is None:
        w = torch.zeros((H, d), dtype=torch.float32, device=dev)
    if count is None:
        count = torch.zeros(1, dtype=torch.int64, device=dev)
    _check(lib().quantwm_query_stats(_ptr(q), n, Hq, H, d, int(accumulate), _ptr(M), _ptr(w), _ptr(count),
                                     _stream(stream)), "quantwm_query_stats")
    return M, w, count


def psac_basis(M, count, rank=QVG_PSAC_RANK, stream=None):
    """Returns (U fp32 [H,d,rank], eigvals fp32 [H,rank], energy_frac fp32 [H])."""
    import torch
    H, d, _ = M.shape
    U = torch.empty((H, d, rank), dtype=torch.float32, device=M.device)
    eig = torch.empty((H, rank), dtype=torch.float32, device=M.device)
    frac = torch.empty((H,), dtype=torch.float32, device=M.device)
    _check(lib().quantwm_psac_basis(_ptr(M), _ptr(count), H, d, rank, _ptr(U), _ptr(eig), _ptr(frac),
                                    _stream(stream)), "quantwm_psac_basis")
    return U, eig, frac


def get_status(stream=None):
    """Synchronise with `stream` (default: the whole device) and return (and
    clear) the device-side error status."""
    return lib().qvg_get_status(None if stream is None else ct.c_void_p(stream.cuda_stream))


def debug_set_wait(limit_ns=0, inject=False):
    """Bound of the device-side waits of the kernels this host thread launches
    next (0: the default 2 s) and the failure-path test hook (see
    qvg_debug_set_wait in include/qvg.h)."""
    _check(lib().qvg_debug_set_wait(int(limit_ns), int(bool(inject))), "qvg_debug_set_wait")


def compression_ratio(params: Params, H, d, tokens_per_chunk, n_chunks, with_psac=False):
    """bf16 bytes / compressed bytes for n_chunks chunks, counting codes,
    fp16 scales, 1-byte ids, bf16 centroids, the outlier side list (fp16
    value + 1-byte channel per group and stage, with QVG_OUTLIER),
    (optionally) the PSAC data, and anchor chunks (anchor_every > 0) at
    their bf16 size, at the stored sizes (padding slots, and the slots an
    anchor chunk reserves in the compressed buffers, excluded)."""
    n_anchor = -(-n_chunks // params.anchor_every) if params.anchor_every > 0 else 0
    n_comp = n_chunks - n_anchor
    N = tokens_per_chunk * n_comp
    side = 3 * d / params.group if params.flags & QVG_OUTLIER else 0
    per_tok = params.L * (d * params.bits / 8 + 2 * d / params.group + (1 if params.C > 0 else 0) + side)
    if with_psac:
        per_tok += QVG_PSAC_RANK + 2
    comp = H * N * per_tok + params.L * H * n_comp * params.C * d * 2
    if with_psac:
        comp += n_comp * H * d * QVG_PSAC_RANK * 4
    comp += n_anchor * tokens_per_chunk * H * d * 2
    return (H * tokens_per_chunk * n_chunks * d * 2) / comp
