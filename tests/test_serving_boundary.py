"""The calls around the attention on the host: argument checks, the rotation
plan's integers, workspace sizes, and the binding's own refusals (no GPU)."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import long_context_ra_gb300 as ra
from long_context_ra_gb300 import _native
from long_context_ra_gb300.build import build

BF16, F32, E4M3 = _native.RA_BF16, _native.RA_F32, _native.RA_E4M3
INV, UNS, MIS, ARCH, OK = (_native.RA_ERR_INVALID_ARG, _native.RA_ERR_UNSUPPORTED,
                           _native.RA_ERR_MISALIGNED, _native.RA_ERR_ARCH, _native.RA_OK)
A = 1 << 20  # a stand-in address, never dereferenced


@pytest.fixture(scope="module")
def L():
    build()
    return _native.lib()


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


def test_page_status_has_a_name(L):
    assert L.ra_status_string(_native.RA_ERR_PAGE).startswith(b"RA_ERR_PAGE")


# ------------------------------------------------------------------ the plan
def plan(freq, axis=None, rot=None, axes=1, inter=0):
    c = _native.RaRopeC()
    n = len(freq)
    code = _native.lib().ra_rope_init(
        ctypes.byref(c), (ctypes.c_double * max(n, 1))(*freq),
        None if axis is None else (ctypes.c_int32 * n)(*axis), 2 * n if rot is None else rot, axes,
        inter)
    return code, c


PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164, 10 ** 70)


@pytest.mark.parametrize("f", [1.0, 0.5, -1.0, 10000.0 ** -0.37, 1e-12, 5e-324, 0.0, 7.25, 123456789.125, -3.7e-5,
                               2.0 ** 30 + 0.5])
def test_turns_are_the_rounded_fraction(L, f):
    code, c = plan([f, 1.0, 1.0, 1.0])
    assert code == OK
    exact = Fraction(abs(f)) / (2 * PI) * 2 ** 64
    want = math.floor(exact + Fraction(1, 2)) % 2 ** 64
    want = (2 ** 64 - want) % 2 ** 64 if f < 0 else want
    # 1 / 2 pi is kept to 130 bits: exact but for a last place of large f
    diff = (c.turns[0] - want) % 2 ** 64
    assert min(diff, 2 ** 64 - diff) <= (0 if abs(f) < 2.0 ** 16 else 1)


def test_plan_refusals(L):
    assert plan([1.0] * 4, [0, 1, 2, 0], axes=3, inter=1)[0] == OK
    assert plan([1.0] * 3)[0] == UNS                         # rot 6
    assert plan([1.0] * 132)[0] == UNS                       # rot 264
    assert plan([1.0] * 4, axes=9)[0] == UNS
    assert plan([1.0] * 4, axes=0)[0] == INV
    assert plan([1.0] * 4, inter=2)[0] == INV
    assert plan([1.0] * 4, [0, 1, 2, 0], axes=2)[0] == INV   # axis out of range
    assert plan([1.0] * 4, [0, -1, 0, 0])[0] == INV
    assert plan([math.inf, 1, 1, 1])[0] == INV
    assert plan([math.nan, 1, 1, 1])[0] == INV
    assert plan([2.0 ** 31, 1, 1, 1])[0] == INV
    assert L.ra_rope_init(None, None, None, 0, 1, 0) == INV
    assert plan([])[0] == OK                                 # no rotation
    with pytest.raises(ra.RaError):
        ra.new_rope([1.0] * 3)
    with pytest.raises(ValueError):
        ra.new_rope([1.0] * 4, axis=[0])


# ----------------------------------------------------------------- the norm
def norm(L, back=False, q=A, k=A, qs=None, ks=None, wq=A, wk=A, rope="plan", pos=A, qo=A, ko=A, B=2,
         Hq=4, Hk=2, N=16, d=64, eps=1e-6, dt=BF16, dq=A, dk=A, dqs=None, dwq=A, dwk=A, ws=A, n=None):
    r = plan([1.0] * 32)[1] if rope == "plan" else rope
    rp = None if r is None else ctypes.byref(r)
    if not back:
        return L.ra_qk_norm_rope(q, qs, k, ks, wq, wk, rp, pos, qo, ko, B, Hq, Hk, N, d, eps, dt, None)
    n = L.ra_qk_norm_rope_backward_workspace_bytes(d) if n is None else n
    return L.ra_qk_norm_rope_backward(q, qs, k, ks, wq, wk, rp, pos, qo, ko, dq, dqs, dk, None, dwq, dwk,
                                      ws, n, B, Hq, Hk, N, d, eps, dt, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(qo=None), INV), (dict(pos=None), INV), (dict(B=-1), INV),
    (dict(Hk=-1), INV), (dict(N=-1), INV), (dict(d=0), INV), (dict(dt=E4M3), INV), (dict(dt=9), INV),
    (dict(eps=math.nan), INV), (dict(eps=-1.0), INV),            # weights without a norm
    (dict(d=60), UNS), (dict(d=264), UNS), (dict(d=56), UNS),    # rot 64 > 56
    (dict(N=1 << 31), UNS), (dict(Hq=1 << 15), UNS),
    (dict(q=A + 4), MIS), (dict(wq=A + 2), MIS), (dict(ko=A + 4), MIS), (dict(pos=A + 4), MIS),
    (dict(qs=i64(64, 2, 64)), MIS), (dict(dt=F32, q=A + 8), MIS),
    (dict(B=0), ARCH), (dict(), ARCH), (dict(rope=None, pos=None), ARCH), (dict(Hk=0, k=None, ko=None), ARCH),
    (dict(qs=i64(6 * 16 * 64, 64, 6 * 64)), ARCH),
])
def test_norm_checks(L, back, kw, code):
    if code == ARCH and "B" in kw and not back:
        code = OK  # no row and nothing to write
    extra = dict(dk=None) if back and kw.get("Hk") == 0 else {}
    assert norm(L, back, **kw, **extra) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dwq=None), INV), (dict(wk=None), INV), (dict(ws=None), INV), (dict(n=100), INV),
    (dict(dq=None), INV), (dict(dqs=i64(4096, 0, 64)), INV), (dict(dqs=i64(0, 1024, 64)), INV),
    (dict(dqs=i64(4096, 1024, 0)), INV), (dict(dqs=i64(4096, 1024, 6)), MIS), (dict(ws=A + 8), MIS),
    (dict(dwq=A + 2), MIS),
    (dict(wq=None, wk=None, dwq=None, dwk=None, ws=None, n=0), ARCH),
    (dict(wq=None, wk=None, dwq=None, dwk=None, ws=None, n=0, N=0), OK),
])
def test_norm_backward_checks(L, kw, code):
    assert norm(L, True, **kw) == code


def test_norm_rejects_a_bad_plan(L):
    r = plan([1.0] * 4)[1]
    for field, value, code in (("rot", 12, UNS), ("rot", -8, INV), ("axes", 0, INV), ("interleaved", 3, INV),
                               ("rot", 512, UNS)):
        bad = _native.RaRopeC.from_buffer_copy(r)
        setattr(bad, field, value)
        assert norm(L, rope=bad) == code, field
    bad = _native.RaRopeC.from_buffer_copy(r)
    bad.axis[3] = 1
    assert norm(L, rope=bad) == INV
    assert L.ra_qk_norm_rope_backward_workspace_bytes(60) == -1
    assert L.ra_qk_norm_rope_backward_workspace_bytes(264) == -1


# ---------------------------------------------------------------- the cache
def cache(k=A, v=A, ke=None, ve=None, pages=10, heads=2, page=16, d=64, dt=BF16):
    return _native.RaCacheC(k, v, ke, ve, pages, heads, page, d, dt)


CACHE_RULES = [
    (dict(k=None), INV), (dict(v=None), INV), (dict(pages=-1), INV), (dict(heads=0), INV), (dict(page=0), INV),
    (dict(d=0), INV), (dict(dt=5), INV), (dict(dt=F32), UNS), (dict(d=60), UNS), (dict(d=264), UNS),
    (dict(page=24), UNS), (dict(page=4), UNS), (dict(page=2048), UNS), (dict(heads=1 << 15), UNS),
    (dict(pages=1 << 31), UNS), (dict(k=A + 8), MIS), (dict(v=A + 8), MIS),
    (dict(dt=E4M3), INV), (dict(dt=E4M3, ke=A), INV), (dict(dt=E4M3, ke=A, ve=A), ARCH), (dict(), ARCH),
]


def write(L, c, k=A, v=A, ks=None, table=A, width=4, lens=A, count=None, B=3, T=2, dt=BF16):
    return L.ra_cache_write(ctypes.byref(c) if c else None, k, ks, v, None, table, width, lens, count, B, T, dt,
                            None)


def read(L, c, table=A, width=4, lens=A, first=0, n=8, k=A, v=A, B=3, dt=BF16):
    return L.ra_cache_read(ctypes.byref(c) if c else None, table, width, lens, first, n, k, v, B, dt, None)


def attend(L, c, q=A, table=A, width=4, lens=A, count=None, mask=None, ms=0, out=A, lse=A, ws=A, n=None, B=3,
           Hq=4, T=2, dt=BF16):
    if n is None:
        n = max(0, L.ra_cache_attention_workspace_bytes(B, max(Hq, 0), 1, max(T, 0), 64))
    return L.ra_cache_attention(q, ctypes.byref(c) if c else None, table, width, lens, count, mask, ms, out, lse,
                                ws, n, B, Hq, T, dt, None)


@pytest.mark.parametrize("call", [write, read, attend])
@pytest.mark.parametrize("kw,code", CACHE_RULES)
def test_cache_rules(L, call, kw, code):
    assert call(L, cache(**kw)) == code


@pytest.mark.parametrize("call", [write, read, attend])
def test_sequence_rules(L, call):
    assert call(L, None) == INV
    assert call(L, cache(), lens=None) == INV
    assert call(L, cache(), table=None) == INV
    assert call(L, cache(), width=-1) == INV
    assert call(L, cache(), B=-1) == INV
    assert call(L, cache(), dt=E4M3) == INV
    assert call(L, cache(), dt=F32) == UNS          # fp32 over a bf16 cache
    assert call(L, cache(), table=A + 2) == MIS
    assert call(L, cache(), lens=A + 2) == MIS
    assert call(L, cache(), B=0, lens=None, table=None) == OK
    assert call(L, cache(), table=None, width=0) == ARCH  # a table without pages is a table


def test_write_and_read_rules(L):
    c = cache()
    assert write(L, c, k=None) == INV
    assert write(L, c, T=-1) == INV
    assert write(L, c, T=0, k=None, v=None) == OK
    assert write(L, c, k=A + 8) == MIS
    assert write(L, c, ks=i64(256, 4, 64)) == MIS   # 8-element rows of bf16
    assert write(L, c, ks=i64(256, 64, 128)) == ARCH
    assert write(L, c, count=A + 1) == MIS
    assert write(L, c, B=1 << 16, T=1 << 16) == UNS
    assert read(L, c, first=-1) == INV
    assert read(L, c, n=-1) == INV
    assert read(L, c, n=0, k=None) == OK
    assert read(L, c, v=None) == INV
    assert read(L, c, k=A + 8) == MIS
    assert read(L, c, n=1 << 31) == UNS
    assert read(L, c, first=1 << 40) == ARCH        # behind every sequence: zeros


def test_attention_rules(L):
    c = cache()
    assert attend(L, c, q=None) == INV
    assert attend(L, c, out=None) == INV
    assert attend(L, c, lse=None) == INV
    assert attend(L, c, ws=None) == INV
    assert attend(L, c, n=64) == INV
    assert attend(L, c, Hq=3) == INV                # 2 key heads
    assert attend(L, c, Hq=-2) == INV
    assert attend(L, c, mask=A, ms=3) == INV        # T * T = 4
    assert attend(L, c, mask=A, ms=4) == ARCH
    assert attend(L, c, mask=A, ms=0) == ARCH
    assert attend(L, cache(d=80)) == UNS            # bf16 head width
    assert attend(L, cache(d=80, dt=F32), dt=F32, n=1 << 40) == ARCH
    assert attend(L, c, q=A + 8) == MIS
    assert attend(L, c, out=A + 8) == MIS
    assert attend(L, c, ws=A + 16) == MIS
    assert attend(L, c, T=0) == OK
    assert attend(L, c, Hq=0) == OK
    w = L.ra_cache_attention_workspace_bytes
    assert w(-1, 4, 2, 1, 64) == -1 and w(1, 3, 2, 1, 64) == -1 and w(1, 4, 0, 1, 64) == -1
    assert w(1, 4, 2, 1, 264) == -1 and w(1, 4, 2, 1, 64) > 0


# --------------------------------------------------------------- the binding
def test_binding_refuses_host_tensors_and_wrong_caches(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ra.ra_qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        ra.RaCache(x, x)
    with pytest.raises(TypeError):
        ra.RaCache(x.half(), x.half())
    with pytest.raises(ValueError):
        ra.RaCache(x, x[:, :1])


def test_a_cache_follows_its_fields(monkeypatch):
    """A call takes the tensors that the cache has then: a field assigned anew
    or a storage that moved reaches it, and what does not fit is refused."""
    seen = []

    class Lib:
        def ra_cache_read(self, ref, *rest):
            c = ctypes.cast(ref, ctypes.POINTER(_native.RaCacheC)).contents
            seen.append((c.k, c.v, c.k_exp, c.v_exp, c.pages, c.dtype))
            return 0

    from long_context_ra_gb300 import serving
    monkeypatch.setattr(serving, "_here", lambda t: None)
    monkeypatch.setattr(serving, "_dev", lambda t, *a, **kw: t.data_ptr())
    monkeypatch.setattr(serving, "_on_stream", lambda *a: 0)
    monkeypatch.setattr(_native, "lib", Lib)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)

    def call(c, code=_native.RA_BF16):
        ra.ra_cache_read(c, table, lens, 0, 4, dtype=torch.bfloat16)
        want = tuple(None if t is None else t.data_ptr() for t in (c.k, c.v, c.k_exp, c.v_exp))
        assert seen[-1] == want + (c.k.shape[0], code)

    pool = lambda pages: torch.zeros(pages, 2, 16, 64, dtype=torch.bfloat16)
    c = ra.RaCache(pool(4), pool(4))
    call(c)
    c.k = pool(4)
    call(c)
    c.v = pool(4)
    call(c)
    before = c.k.data_ptr()
    held = c.k.untyped_storage()
    held.resize_(1 << 26)                       # in place: the storage moves
    assert c.k.data_ptr() != before
    call(c)
    c.k, c.v = pool(9), pool(9)                 # grown: both sides, then the call
    call(c)
    c.k = pool(5)
    with pytest.raises(ValueError):
        call(c)
    c.v = pool(5)
    call(c)
    c.k_exp = torch.zeros(5, 2, 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        call(c)
    c.k, c.v = (x.to(torch.float8_e4m3fn) for x in (c.k, c.v))
    with pytest.raises(ValueError):
        call(c)
    c.v_exp = torch.zeros(5, 2, 16, dtype=torch.uint8)
    call(c, _native.RA_E4M3)
    assert (c.heads, c.d) == (2, 64)


def test_a_rotation_plan_stays_as_it_is():
    """The calls hold its address, and a gradient needs the forward's angles."""
    a, b = ra.new_rope([1.0] * 4), ra.new_rope([0.5] * 8)
    with pytest.raises(AttributeError):
        a.c = b.c
    c = ctypes.cast(a.ref, ctypes.POINTER(_native.RaRopeC)).contents
    assert a.rot == c.rot == 8
