"""The calls around the attention: norm and rotation of queries and keys, the
paged K/V cache, attention of new tokens over it, forks of sequences and their
pages, and the verification of drafts (``include/ra.h``).

As in the package's other calls, the functions only marshal arguments.  All
tensors of a call are on the current CUDA device; a call with tensors of
another device is refused.  Tensors that a call allocates belong to the stream
it runs on.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field
from typing import NamedTuple

import torch

from . import _check, _dtype_code, _native, _stream
from ._native import RA_BF16, RA_E4M3, RA_F32, RaCacheC, RaRopeC

_CACHE_TYPES = {torch.float32: RA_F32, torch.bfloat16: RA_BF16, torch.float8_e4m3fn: RA_E4M3}


_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else \
    torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _here(t: torch.Tensor) -> int:
    """The current device, which has to be the tensor's."""
    index = t.get_device()
    if index < 0 or index != _device():
        raise ValueError("tensors must be on the current CUDA device")
    return index


def _on_stream(stream, index: int) -> int:
    """The handle of the given stream, or of the device's current one."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(index)
    return _stream(stream)


def _dev(t: torch.Tensor, index: int, dtype=None, shape=None, what: str = "tensor") -> int:
    """The address of a contiguous tensor on the current device."""
    if t.get_device() != index:
        raise ValueError(f"{what} must be on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _rows(t: torch.Tensor, index: int, dtype, shape, what: str):
    """Address and batch, head, token strides of a [B, H, N, d] tensor (None:
    dense)."""
    if t.get_device() != index:
        raise ValueError(f"{what} must be on the current CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), None
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"the last dimension of {what} must be contiguous")
    return t.data_ptr(), _Strides(*st[:3])


_Strides = ctypes.c_int64 * 3


class _on:
    """Allocations inside belong to `stream` (None: the current one)."""

    def __init__(self, stream):
        self.ctx = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


# ---------------------------------------------------------- norm and rotation
@dataclass(frozen=True)
class RaRope:
    """A rotation plan (see `new_rope`); a backward pass takes it as the forward
    had it, so its field is not assigned anew."""

    c: RaRopeC = field(repr=False)

    def __post_init__(self):
        object.__setattr__(self, "ref", ctypes.byref(self.c))

    @property
    def rot(self) -> int:
        return self.c.rot

    @property
    def axes(self) -> int:
        return self.c.axes


def new_rope(inv_freq, axis=None, interleaved: bool = False, axes: int | None = None) -> RaRope:
    """Rotation plan: pair i of the first 2 * len(inv_freq) elements of a head
    turns by positions[axis[i]] * inv_freq[i] radians.

    inv_freq     floats (radians per position), a multiple of 4 of them.
    axis         the position axis of each pair (default: all axis 0).
    interleaved  pairs (2i, 2i + 1) instead of (i, i + rot / 2).
    axes         number of position axes (default: 1 + max(axis))."""
    freq = [float(f) for f in inv_freq]
    n = len(freq)
    ax = [0] * n if axis is None else [int(a) for a in axis]
    if len(ax) != n:
        raise ValueError("axis must have one entry per frequency")
    if axes is None:
        axes = 1 + max(ax, default=0)
    c = RaRopeC()
    code = _native.lib().ra_rope_init(ctypes.byref(c), (ctypes.c_double * max(n, 1))(*freq),
                                      (ctypes.c_int32 * max(n, 1))(*ax), 2 * n, axes,
                                      1 if interleaved else 0)
    _check(code, "ra_rope_init")
    return RaRope(c)


def _plan(rope, positions, B, N, index):
    if rope is None or rope.c.rot == 0:
        return None, None
    if positions is None:
        raise ValueError("a rotation needs positions")
    shape = positions.shape
    if shape != (rope.c.axes, B, N) and not (rope.c.axes == 1 and shape == (B, N)):
        raise ValueError(f"positions must have shape {(rope.axes, B, N)}, got {tuple(shape)}")
    return rope.ref, _dev(positions, index, torch.int64, what="positions")


def _weight(w, d, dtype, index, what):
    return None if w is None else _dev(w, index, dtype, (d,), what)


def ra_qk_norm_rope(q, k, rope: RaRope | None = None, positions=None, q_weight=None,
                    k_weight=None, eps: float | None = 1e-6, q_out=None, k_out=None, stream=None):
    """RMS norm of every head row of q [B, Hq, N, d] and k [B, Hk, N, d]
    (views of a projection are read through their strides) and rotation by
    positions [axes, B, N] int64 ([B, N] for one axis), in one pass.
    eps=None: rotation only.  Returns dense (q_out, k_out)."""
    B, Hq, N, d = q.shape
    Hk = k.shape[1]
    dt, index = q.dtype, _here(q)
    code = _dtype_code(q)
    qp, qs = _rows(q, index, dt, (B, Hq, N, d), "q")
    kp, ks = _rows(k, index, dt, (B, Hk, N, d), "k")
    plan, pos = _plan(rope, positions, B, N, index)
    if q_out is None or k_out is None:
        with _on(stream):
            if q_out is None:
                q_out = torch.empty((B, Hq, N, d), device=q.device, dtype=dt)
            if k_out is None:
                k_out = torch.empty((B, Hk, N, d), device=q.device, dtype=dt)
    res = _native.lib().ra_qk_norm_rope(
        qp, qs, kp, ks, _weight(q_weight, d, dt, index, "q_weight"),
        _weight(k_weight, d, dt, index, "k_weight"), plan, pos,
        _dev(q_out, index, dt, (B, Hq, N, d), "q_out"),
        _dev(k_out, index, dt, (B, Hk, N, d), "k_out"), B, Hq, Hk, N, d,
        -1.0 if eps is None else eps, code, _on_stream(stream, index))
    _check(res, "ra_qk_norm_rope")
    return q_out, k_out


def ra_qk_norm_rope_backward_workspace_bytes(d: int) -> int:
    return int(_native.lib().ra_qk_norm_rope_backward_workspace_bytes(d))


def ra_qk_norm_rope_backward(q, k, dq_out, dk_out, rope: RaRope | None = None, positions=None,
                             q_weight=None, k_weight=None, eps: float | None = 1e-6, dq=None,
                             dk=None, workspace=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ra_qk_norm_rope for the
    output gradients dq_out, dk_out (dense).  dq, dk have the strides of q, k
    where those are without gaps, else they are dense; the weights' gradients
    are fp32 (None without a weight)."""
    B, Hq, N, d = q.shape
    Hk = k.shape[1]
    dt, index = q.dtype, _here(q)
    code = _dtype_code(q)
    qp, qs = _rows(q, index, dt, (B, Hq, N, d), "q")
    kp, ks = _rows(k, index, dt, (B, Hk, N, d), "k")
    wq = _weight(q_weight, d, dt, index, "q_weight")
    wk = _weight(k_weight, d, dt, index, "k_weight")
    plan, pos = _plan(rope, positions, B, N, index)
    dwq = dwk = None
    with _on(stream):
        if dq is None:
            dq = torch.empty_like(q)
        if dk is None:
            dk = torch.empty_like(k)
        if wq is not None:
            dwq = torch.empty(d, device=q.device, dtype=torch.float32)
        if wk is not None:
            dwk = torch.empty(d, device=q.device, dtype=torch.float32)
        if workspace is None and (wq is not None or wk is not None):
            workspace = torch.empty(max(0, ra_qk_norm_rope_backward_workspace_bytes(d)),
                                    device=q.device, dtype=torch.uint8)
    dqp, dqs = _rows(dq, index, dt, (B, Hq, N, d), "dq")
    dkp, dks = _rows(dk, index, dt, (B, Hk, N, d), "dk")
    res = _native.lib().ra_qk_norm_rope_backward(
        qp, qs, kp, ks, wq, wk, plan, pos, _dev(dq_out, index, dt, (B, Hq, N, d), "dq_out"),
        _dev(dk_out, index, dt, (B, Hk, N, d), "dk_out"), dqp, dqs, dkp, dks,
        None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(),
        None if workspace is None else _dev(workspace, index, torch.uint8, what="workspace"),
        0 if workspace is None else workspace.numel(), B, Hq, Hk, N, d,
        -1.0 if eps is None else eps, code, _on_stream(stream, index))
    _check(res, "ra_qk_norm_rope_backward")
    return dq, dk, dwq, dwk


# ------------------------------------------------------------------ the cache
class _Found(NamedTuple):
    """A cache's fields, checked."""

    places: tuple
    c: RaCacheC
    ref: object  # to c
    heads: int
    d: int
    index: int


@dataclass
class RaCache:
    """Pages of K and V, [pages, heads, page, d] (float32, bfloat16, or
    float8_e4m3fn with exponent bytes k_exp, v_exp [pages, heads, page]).  A
    call takes the tensors that the fields hold then."""

    k: torch.Tensor
    v: torch.Tensor
    k_exp: torch.Tensor | None = None
    v_exp: torch.Tensor | None = None

    def __post_init__(self):
        self._check()

    def __setattr__(self, name, value):
        object.__setattr__(self, "_found", None)  # checked anew by the next call
        object.__setattr__(self, name, value)

    @property
    def heads(self) -> int:
        return self.k.shape[1]

    @property
    def d(self) -> int:
        return self.k.shape[3]

    def _places(self):
        """What a tensor changed in place shows: addresses and sizes."""
        k, v, ke, ve = self.k, self.v, self.k_exp, self.v_exp
        return (k.data_ptr(), v.data_ptr(), 0 if ke is None else ke.data_ptr(),
                0 if ve is None else ve.data_ptr(), k.numel(), v.numel())

    def _check(self):
        k, v = self.k, self.v
        if k.dtype not in _CACHE_TYPES:
            raise TypeError(f"unsupported cache dtype {k.dtype}")
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v must be [pages, heads, page, d] of one dtype")
        index = k.device.index
        ptrs = [_dev(k, index, what="k"), _dev(v, index, what="v"), None, None]
        if k.dtype == torch.float8_e4m3fn:
            for i, (t, what) in enumerate(((self.k_exp, "k_exp"), (self.v_exp, "v_exp"))):
                if t is None:
                    raise ValueError("an 8-bit cache needs k_exp and v_exp")
                ptrs[2 + i] = _dev(t, index, torch.uint8, tuple(k.shape[:3]), what)
        elif self.k_exp is not None or self.v_exp is not None:
            raise ValueError("only an 8-bit cache has exponents")
        pages, heads, page, d = k.shape
        c = RaCacheC(*ptrs, pages, heads, page, d, _CACHE_TYPES[k.dtype])
        object.__setattr__(self, "_found", _Found(self._places(), c, ctypes.byref(c), heads, d, index))

    def found(self, index) -> _Found:
        """The fields as the C calls take them, on device `index`."""
        f = self._found
        if f is None or f.places != self._places():
            self._check()
            f = self._found
        if f.index != index:
            raise ValueError("the cache must be on the current CUDA device")
        return f


def new_cache(pages: int, heads: int, page: int, d: int, dtype=torch.bfloat16,
              device=None) -> RaCache:
    """Allocate a cache (uninitialised pages)."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    k, v = (torch.empty((pages, heads, page, d), device=dev, dtype=dtype) for _ in range(2))
    if dtype != torch.float8_e4m3fn:
        return RaCache(k, v)
    return RaCache(k, v, *(torch.empty((pages, heads, page), device=dev, dtype=torch.uint8)
                           for _ in range(2)))


def _sequences(table, lens, count, B: int, index: int):
    if table.dim() != 2 or table.shape[0] != B:
        raise ValueError("table must be [B, width]")
    return (_dev(table, index, torch.int32, what="table"), table.shape[1],
            _dev(lens, index, torch.int32, (B,), "lens"),
            None if count is None else _dev(count, index, torch.int32, (B,), "count"))


def ra_cache_write(cache: RaCache, k, v, table, lens, count=None, stream=None) -> RaCache:
    """Append new tokens: k, v [B, heads, T, d] (views are read through their
    strides), token t < count[b] goes to position lens[b] + t of sequence b.
    An 8-bit cache is quantised as it is written.  lens is not advanced."""
    B, heads, T, d = k.shape
    index = _here(k)
    c = cache.found(index)
    tab, width, ln, cnt = _sequences(table, lens, count, B, index)
    kp, ks = _rows(k, index, k.dtype, (B, c.heads, T, c.d), "k")
    vp, vs = _rows(v, index, k.dtype, (B, c.heads, T, c.d), "v")
    res = _native.lib().ra_cache_write(c.ref, kp, ks, vp, vs, tab, width, ln, cnt, B, T,
                                       _dtype_code(k), _on_stream(stream, index))
    _check(res, "ra_cache_write")
    return cache


def ra_cache_read(cache: RaCache, table, lens, first: int, n: int, dtype=None, k=None, v=None,
                  stream=None):
    """Positions first .. first + n - 1 of every sequence as dense (k, v)
    [B, heads, n, d]; rows at or behind lens[b] are 0.  dtype: the result's
    (default: that of a given k or v, the cache's, or bfloat16 for 8 bits)."""
    B = table.shape[0]
    index = _here(table)
    c = cache.found(index)
    tab, width, ln, _ = _sequences(table, lens, None, B, index)
    if dtype is None:
        given = k if k is not None else v
        if given is not None:
            dtype = given.dtype
        else:
            dtype = torch.bfloat16 if c.c.dtype == RA_E4M3 else cache.k.dtype
    shape = (B, c.heads, n, c.d)
    if k is None or v is None:
        with _on(stream):
            if k is None:
                k = torch.empty(shape, device=cache.k.device, dtype=dtype)
            if v is None:
                v = torch.empty(shape, device=cache.k.device, dtype=dtype)
    res = _native.lib().ra_cache_read(c.ref, tab, width, ln, first, n,
                                      _dev(k, index, dtype, shape, "k"),
                                      _dev(v, index, dtype, shape, "v"), B, _dtype_code(k),
                                      _on_stream(stream, index))
    _check(res, "ra_cache_read")
    return k, v


def ra_cache_attention_workspace_bytes(B: int, Hq: int, heads: int, T: int, d: int) -> int:
    return int(_native.lib().ra_cache_attention_workspace_bytes(B, Hq, heads, T, d))


def ra_cache_attention(q, cache: RaCache, table, lens, count=None, mask=None, out=None, lse=None,
                       workspace=None, stream=None):
    """Attention of the newest tokens q [B, Hq, T, d] over the cache that
    ra_cache_write has put them in: query t sees the context (positions below
    lens[b]) and of the new tokens those with mask[b, t, j] (bool [B, T, T],
    or [T, T] for all sequences; None: j <= t).  Hq is a multiple of the
    cache's heads.  `workspace` (uint8, ra_cache_attention_workspace_bytes) is
    allocated when not given.  Returns (out [B, Hq, T, d], lse [B, Hq, T])."""
    return _attend(None, q, cache, table, lens, count, mask, out, lse, workspace, stream)


def ra_cache_attention_shared_workspace_bytes(B: int, Hq: int, heads: int, T: int, d: int) -> int:
    return int(_native.lib().ra_cache_attention_shared_workspace_bytes(B, Hq, heads, T, d))


def ra_cache_attention_shared(q, cache: RaCache, table, lens, shared, count=None, mask=None, out=None,
                              lse=None, workspace=None, stream=None):
    """ra_cache_attention for sequences that share prefixes, each read once for
    all of them: shared [B] (int32) > 0 are the tokens that sequence b has in
    common with the one before it (the next lower one with lens >= 0), else a
    group begins at b.  `workspace`: ra_cache_attention_shared_workspace_bytes.
    Short prefixes (below some 50000 repeated tokens in all) take longer shared
    than read again, which a table as wide as they are long shows to the call; in
    one much wider, ra_cache_attention is the call for them.  Over an 8-bit cache
    a prefix's probabilities are bf16, not f16, where B x T x Hq / heads > 16."""
    if shared is None:
        raise ValueError("shared must be an int32 tensor [B]")
    return _attend(shared, q, cache, table, lens, count, mask, out, lse, workspace, stream)


def _attend(shared, q, cache, table, lens, count, mask, out, lse, workspace, stream):
    B, Hq, T, d = q.shape
    index = _here(q)
    c = cache.found(index)
    tab, width, ln, cnt = _sequences(table, lens, count, B, index)
    if d != c.d:
        raise ValueError(f"q has head width {d}, the cache {c.d}")
    mp, ms = None, 0
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"mask must be bool or uint8, got {mask.dtype}")
        if mask.dim() == 2:
            mp = _dev(mask, index, shape=(T, T), what="mask")
        else:
            mp, ms = _dev(mask, index, shape=(B, T, T), what="mask"), T * T
    lib = _native.lib()
    size = lib.ra_cache_attention_workspace_bytes if shared is None else \
        lib.ra_cache_attention_shared_workspace_bytes
    if out is None or lse is None or workspace is None:
        with _on(stream):
            if out is None:
                out = torch.empty((B, Hq, T, d), device=q.device, dtype=q.dtype)
            if lse is None:
                lse = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
            if workspace is None:
                workspace = torch.empty(max(int(size(B, Hq, c.heads, T, d)), 0), device=q.device,
                                        dtype=torch.uint8)
    rest = (cnt, mp, ms, _dev(out, index, q.dtype, (B, Hq, T, d), "out"),
            _dev(lse, index, torch.float32, (B, Hq, T), "lse"),
            _dev(workspace, index, torch.uint8, what="workspace"), workspace.numel(), B, Hq, T,
            _dtype_code(q), _on_stream(stream, index))
    qp = _dev(q, index, shape=(B, Hq, T, d), what="q")
    if shared is None:
        _check(lib.ra_cache_attention(qp, c.ref, tab, width, ln, *rest), "ra_cache_attention")
    else:
        res = lib.ra_cache_attention_shared(qp, c.ref, tab, width, ln,
                                            _dev(shared, index, torch.int32, (B,), "shared"), *rest)
        _check(res, "ra_cache_attention_shared")
    return out, lse


# ------------------------------------------------------ pages that are shared
def _table(ref, table, held, lens, index):
    """Addresses and sizes of a table and its counts: (ref, pages, table, held,
    lens, width, B)."""
    if table.dim() != 2 or ref.dim() != 1:
        raise ValueError("table must be [B, width] and ref [pages]")
    B, width = table.shape
    return (_dev(ref, index, torch.int32, what="ref"), ref.shape[0],
            _dev(table, index, torch.int32, what="table"), _dev(held, index, torch.int32, (B,), "held"),
            None if lens is None else _dev(lens, index, torch.int32, (B,), "lens"), width, B)


def ra_pages_fork(ref, table, held, lens, source, page: int, table_out=None, held_out=None,
                  lens_out=None, stream=None):
    """Rows that continue sequences source [n] (int32; < 0: an empty row):
    they hold the same pages, whose counts in ref rise.  Returns (table_out
    [n, width], held_out [n], lens_out [n])."""
    index = _here(table)
    r, pages, tab, hl, ln, width, B = _table(ref, table, held, lens, index)
    n = source.shape[0]
    if table_out is None or held_out is None or lens_out is None:
        with _on(stream):
            if table_out is None:
                table_out = torch.empty((n, width), device=table.device, dtype=torch.int32)
            if held_out is None:
                held_out = torch.empty(n, device=table.device, dtype=torch.int32)
            if lens_out is None:
                lens_out = torch.empty(n, device=table.device, dtype=torch.int32)
    res = _native.lib().ra_pages_fork(
        r, pages, tab, hl, ln, width, page, B, _dev(source, index, torch.int32, (n,), "source"), n,
        _dev(table_out, index, torch.int32, (n, width), "table_out"),
        _dev(held_out, index, torch.int32, (n,), "held_out"),
        _dev(lens_out, index, torch.int32, (n,), "lens_out"), _on_stream(stream, index))
    _check(res, "ra_pages_fork")
    return table_out, held_out, lens_out


def ra_pages_reserve(ref, table, held, lens, page: int, T: int, count=None, granted=None, src=None,
                     dst=None, stream=None):
    """Room for count[b] (None: T) new tokens of every sequence: table, held
    and ref are updated.  Returns (granted, src, dst), int32 [B] each: the new
    tokens that have room (the `count` of the calls that follow), and the pages
    that ra_cache_copy has to copy in every layer's cache before they are
    written."""
    index = _here(table)
    r, pages, tab, hl, ln, width, B = _table(ref, table, held, lens, index)
    if granted is None or src is None or dst is None:
        with _on(stream):
            granted, src, dst = (torch.empty(B, device=table.device, dtype=torch.int32) if t is None
                                 else t for t in (granted, src, dst))
    res = _native.lib().ra_pages_reserve(
        r, pages, tab, hl, ln, None if count is None else _dev(count, index, torch.int32, (B,), "count"),
        width, page, B, T, _dev(granted, index, torch.int32, (B,), "granted"),
        _dev(src, index, torch.int32, (B,), "src"), _dev(dst, index, torch.int32, (B,), "dst"),
        _on_stream(stream, index))
    _check(res, "ra_pages_reserve")
    return granted, src, dst


def ra_pages_trim(ref, table, held, lens, page: int, stream=None) -> None:
    """Give back the pages behind lens[b] tokens (all of them for lens[b] < 0,
    and of every sequence for lens=None): table, held and ref are updated."""
    index = _here(table)
    r, pages, tab, hl, ln, width, B = _table(ref, table, held, lens, index)
    res = _native.lib().ra_pages_trim(r, pages, tab, hl, ln, width, page, B, _on_stream(stream, index))
    _check(res, "ra_pages_trim")


def ra_cache_copy(cache: RaCache, src, dst, stream=None) -> RaCache:
    """Page dst[i] becomes a copy of page src[i] (int32 [n]; pairs with a
    negative number are passed over)."""
    index = _here(src)
    c = cache.found(index)
    n = src.shape[0]
    res = _native.lib().ra_cache_copy(c.ref, _dev(src, index, torch.int32, (n,), "src"),
                                      _dev(dst, index, torch.int32, (n,), "dst"), n,
                                      _on_stream(stream, index))
    _check(res, "ra_cache_copy")
    return cache


def ra_cache_compact(cache: RaCache, table, lens, path, kept, stream=None) -> RaCache:
    """Move the kept new tokens together: the rows at position lens[b] +
    path[b, j] go to lens[b] + j, j < kept[b] (path int32 [B, T], rising, as
    ra_verify_drafts returns it).  lens is not advanced."""
    B, T = path.shape
    index = _here(path)
    c = cache.found(index)
    tab, width, ln, _ = _sequences(table, lens, None, B, index)
    res = _native.lib().ra_cache_compact(c.ref, tab, width, ln,
                                         _dev(path, index, torch.int32, (B, T), "path"),
                                         _dev(kept, index, torch.int32, (B,), "kept"), B, T,
                                         _on_stream(stream, index))
    _check(res, "ra_cache_compact")
    return cache


# ------------------------------------------------------- verification of drafts
def ra_verify_drafts(probs, tokens, uniform, parent=None, draft_probs=None, count=None, path=None,
                     kept=None, token=None, stream=None):
    """Which drafts stay, and the token after them.  probs [B, T, V]: the
    model's distribution after node t (float32 or bfloat16, rows that add up to
    1); node 0 is the newest settled token, tokens [B, T] (int64) the drafts,
    parent [B, T] (int32; None: a chain) the node that each follows;
    draft_probs: what they were drawn from (None: they were chosen); uniform
    [B, T] float32 in [0, 1), which resolves probabilities to 2^-24.  A row of
    draft_probs that no draft was drawn from is not read.  Returns (path [B, T] int32: the nodes that stay,
    -1 behind them; kept [B] int32: their number, node 0 counted; token [B]
    int64)."""
    B, T, V = probs.shape
    index = _here(probs)
    if path is None or kept is None or token is None:
        with _on(stream):
            if path is None:
                path = torch.empty((B, T), device=probs.device, dtype=torch.int32)
            if kept is None:
                kept = torch.empty(B, device=probs.device, dtype=torch.int32)
            if token is None:
                token = torch.empty(B, device=probs.device, dtype=torch.int64)
    res = _native.lib().ra_verify_drafts(
        _dev(probs, index, what="probs"),
        None if draft_probs is None else _dev(draft_probs, index, probs.dtype, (B, T, V), "draft_probs"),
        _dev(tokens, index, torch.int64, (B, T), "tokens"),
        None if parent is None else _dev(parent, index, torch.int32, (B, T), "parent"),
        None if count is None else _dev(count, index, torch.int32, (B,), "count"),
        _dev(uniform, index, torch.float32, (B, T), "uniform"),
        _dev(path, index, torch.int32, (B, T), "path"), _dev(kept, index, torch.int32, (B,), "kept"),
        _dev(token, index, torch.int64, (B,), "token"), B, T, V, _dtype_code(probs),
        _on_stream(stream, index))
    _check(res, "ra_verify_drafts")
    return path, kept, token
