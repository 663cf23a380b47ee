"""Forks, pages, moves and the verification of drafts on the host: argument
checks and the binding's own refusals (no GPU)."""
import ctypes

import pytest
import torch

import long_context_ra_gb300 as ra
from long_context_ra_gb300 import _native
from long_context_ra_gb300.build import build

BF16, F32, E4M3 = _native.RA_BF16, _native.RA_F32, _native.RA_E4M3
INV, UNS, MIS, ARCH, OK = (_native.RA_ERR_INVALID_ARG, _native.RA_ERR_UNSUPPORTED,
                           _native.RA_ERR_MISALIGNED, _native.RA_ERR_ARCH, _native.RA_OK)
A = 1 << 20  # stand-in addresses, never dereferenced
FAR = 1 << 30


@pytest.fixture(scope="module")
def L():
    build()
    return _native.lib()


def fork(L, ref=A, pages=10, table=A, held=A, lens=A, width=4, page=16, B=3, source=A, n=5, to=FAR, ho=FAR, lo=FAR):
    return L.ra_pages_fork(ref, pages, table, held, lens, width, page, B, source, n, to, ho, lo, None)


def reserve(L, ref=A, pages=10, table=A, held=A, lens=A, width=4, page=16, B=3, count=None, T=2, g=A, s=A, d=A):
    return L.ra_pages_reserve(ref, pages, table, held, lens, count, width, page, B, T, g, s, d, None)


def trim(L, ref=A, pages=10, table=A, held=A, lens=A, width=4, page=16, B=3):
    return L.ra_pages_trim(ref, pages, table, held, lens, width, page, B, None)


@pytest.mark.parametrize("call", [fork, reserve, trim])
@pytest.mark.parametrize("kw,code", [
    (dict(ref=None), INV), (dict(table=None), INV), (dict(held=None), INV), (dict(pages=-1), INV),
    (dict(width=-1), INV), (dict(B=-1), INV), (dict(page=0), INV), (dict(page=-16), INV), (dict(page=24), UNS),
    (dict(page=4), UNS), (dict(page=2048), UNS), (dict(pages=1 << 31), UNS), (dict(width=1 << 30), UNS),
    (dict(ref=A + 2), MIS), (dict(table=A + 1), MIS), (dict(held=A + 2), MIS), (dict(lens=A + 2), MIS),
    (dict(), ARCH), (dict(width=0, table=None), ARCH), (dict(pages=0, ref=None), ARCH),
])
def test_table_rules(L, call, kw, code):
    extra = dict(to=None) if call is fork and kw.get("width") == 0 else {}
    assert call(L, **kw, **extra) == code


def test_fork_rules(L):
    assert fork(L, lens=None) == INV
    assert fork(L, n=-1) == INV
    assert fork(L, n=0, source=None, to=None, ho=None, lo=None) == OK
    assert fork(L, source=None) == INV
    assert fork(L, to=None) == INV
    assert fork(L, ho=None) == INV
    assert fork(L, lo=None) == INV
    assert fork(L, source=A + 2) == MIS
    assert fork(L, to=FAR + 2) == MIS
    assert fork(L, n=1 << 30) == UNS
    assert fork(L, B=0, table=None, held=None, lens=None) == ARCH  # every row is empty
    # new rows over the old ones: 3 x 4 columns at A
    assert fork(L, to=A) == INV
    assert fork(L, to=A + 44) == INV
    assert fork(L, to=A - 76) == INV
    assert fork(L, to=A + 48) == ARCH
    assert fork(L, to=A - 80) == ARCH
    apart = dict(ref=FAR + 4096, source=FAR + 8192, table=FAR + 12288)
    assert fork(L, ho=A + 8, **apart) == INV and fork(L, ho=A + 12, **apart) == ARCH
    assert fork(L, lo=A - 16, **apart) == INV and fork(L, lo=A - 20, **apart) == ARCH


def test_reserve_rules(L):
    assert reserve(L, lens=None) == INV
    assert reserve(L, T=-1) == INV
    assert reserve(L, g=None) == INV
    assert reserve(L, s=None) == INV
    assert reserve(L, d=None) == INV
    assert reserve(L, count=A + 2) == MIS
    assert reserve(L, g=A + 2) == MIS
    assert reserve(L, B=8193) == UNS
    assert reserve(L, B=8192) == ARCH
    assert reserve(L, T=0) == ARCH                     # granted, src and dst are written
    assert reserve(L, B=0, table=None, held=None, lens=None, g=None, s=None, d=None) == OK


def test_trim_rules(L):
    assert trim(L, lens=None) == ARCH                  # everything goes
    assert trim(L, B=0, table=None, held=None, lens=None) == OK


def cache(k=A, v=A, ke=None, ve=None, pages=10, heads=2, page=16, d=64, dt=BF16):
    return _native.RaCacheC(k, v, ke, ve, pages, heads, page, d, dt)


def copy(L, c, src=A, dst=A, n=3):
    return L.ra_cache_copy(ctypes.byref(c) if c else None, src, dst, n, None)


def compact(L, c, table=A, width=4, lens=A, path=A, kept=A, B=3, T=2):
    return L.ra_cache_compact(ctypes.byref(c) if c else None, table, width, lens, path, kept, B, T, None)


@pytest.mark.parametrize("call", [copy, compact])
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(pages=-1), INV), (dict(heads=0), INV), (dict(page=0), INV),
    (dict(d=0), INV), (dict(dt=5), INV), (dict(d=60), UNS), (dict(d=264), UNS), (dict(page=24), UNS),
    (dict(page=4), UNS), (dict(heads=1 << 15), UNS), (dict(pages=1 << 31), UNS), (dict(k=A + 8), MIS),
    (dict(dt=E4M3), INV), (dict(dt=E4M3, ke=A), INV), (dict(dt=E4M3, ke=A, ve=A + 4), MIS),
    (dict(dt=E4M3, ke=A, ve=A), ARCH), (dict(dt=F32), ARCH), (dict(), ARCH),
])
def test_cache_rules(L, call, kw, code):
    assert call(L, cache(**kw)) == code


def test_copy_and_compact_rules(L):
    c = cache()
    assert copy(L, None) == INV
    assert copy(L, c, n=-1) == INV
    assert copy(L, c, src=None) == INV
    assert copy(L, c, dst=None) == INV
    assert copy(L, c, src=A + 2) == MIS
    assert copy(L, c, n=0, src=None, dst=None) == OK
    assert compact(L, None) == INV
    assert compact(L, c, lens=None) == INV
    assert compact(L, c, path=None) == INV
    assert compact(L, c, kept=None) == INV
    assert compact(L, c, kept=A + 1) == MIS
    assert compact(L, c, T=-1) == INV
    assert compact(L, c, B=1 << 16, T=1 << 16) == UNS
    assert compact(L, c, T=0, path=None) == OK
    assert compact(L, c, B=0, lens=None, table=None) == OK


def verify(L, p=A, q=A, tok=A, par=A, cnt=None, u=A, path=A, kept=A, token=A, B=3, T=4, V=100, dt=F32):
    return L.ra_verify_drafts(p, q, tok, par, cnt, u, path, kept, token, B, T, V, dt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(p=None), INV), (dict(tok=None), INV), (dict(u=None), INV), (dict(path=None), INV), (dict(kept=None), INV),
    (dict(token=None), INV), (dict(B=-1), INV), (dict(T=0), INV), (dict(V=0), INV), (dict(dt=E4M3), INV),
    (dict(dt=9), INV), (dict(T=1025), UNS), (dict(V=1 << 31), UNS), (dict(B=(1 << 24) + 1), UNS),
    (dict(p=A + 4), MIS), (dict(q=A + 8), MIS), (dict(tok=A + 4), MIS), (dict(token=A + 4), MIS),
    (dict(u=A + 2), MIS), (dict(cnt=A + 2), MIS), (dict(), ARCH), (dict(q=None, par=None, dt=BF16), ARCH),
    (dict(B=0, p=None, tok=None), OK),
])
def test_verify_rules(L, kw, code):
    assert verify(L, **kw) == code


def test_binding_refuses_host_tensors(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    i = torch.zeros(3, dtype=torch.int32)
    t = torch.zeros(3, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ra.ra_pages_fork(i, t, i, i, i, 16)
    with pytest.raises(ValueError):
        ra.ra_pages_reserve(i, t, i, i, 16, 1)
    with pytest.raises(ValueError):
        ra.ra_pages_trim(i, t, i, None, 16)
    with pytest.raises(ValueError):
        ra.ra_verify_drafts(torch.zeros(1, 2, 3), torch.zeros(1, 2, dtype=torch.int64), torch.zeros(1, 2))


def attend(L, c, q=A, table=A, width=4, lens=A, shared=A, count=None, mask=None, ms=0, out=A, lse=A, ws=A, n=None,
           B=3, Hq=4, T=2, dt=BF16):
    if n is None:
        n = max(0, L.ra_cache_attention_shared_workspace_bytes(B, max(Hq, 0), 1, max(T, 0), 64))
    return L.ra_cache_attention_shared(q, ctypes.byref(c) if c else None, table, width, lens, shared, count, mask,
                                       ms, out, lse, ws, n, B, Hq, T, dt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(out=None), INV), (dict(lse=None), INV), (dict(ws=None), INV), (dict(n=64), INV),
    (dict(Hq=3), INV), (dict(Hq=-2), INV), (dict(mask=A, ms=3), INV), (dict(B=-1), INV), (dict(T=-1), INV),
    (dict(lens=None), INV), (dict(table=None), INV), (dict(shared=None), INV), (dict(dt=E4M3), INV),
    (dict(dt=F32), UNS), (dict(q=A + 8), MIS), (dict(out=A + 8), MIS), (dict(ws=A + 16), MIS), (dict(shared=A + 2), MIS),
    (dict(count=A + 2), MIS), (dict(T=0), OK), (dict(Hq=0), OK), (dict(B=0, lens=None, table=None, shared=None), OK),
    (dict(), ARCH), (dict(mask=A, ms=4), ARCH),
])
def test_shared_attention_rules(L, kw, code):
    assert attend(L, cache(), **kw) == code


def test_shared_attention_of_other_caches(L):
    assert attend(L, None) == INV
    assert attend(L, cache(d=80)) == UNS
    assert attend(L, cache(d=80, dt=F32), dt=F32, n=1 << 40) == ARCH
    w, plain = L.ra_cache_attention_shared_workspace_bytes, L.ra_cache_attention_workspace_bytes
    assert w(-1, 4, 2, 1, 64) == -1 and w(1, 3, 2, 1, 64) == -1 and w(1, 4, 0, 1, 64) == -1
    assert w(1, 4, 2, 1, 264) == -1
    for sizes in ((1, 4, 2, 1, 64), (96, 32, 8, 1, 128), (3000, 8, 8, 1, 64), (8, 32, 8, 300, 128)):
        assert w(*sizes) >= plain(*sizes)
    with pytest.raises(ValueError):
        ra.ra_cache_attention_shared(None, None, None, None, None)


@pytest.mark.parametrize("out", ["to", "ho", "lo"])
@pytest.mark.parametrize("near", ["ref", "table", "held", "lens", "source"])
def test_fork_refuses_what_lies_over_its_inputs(L, out, near):
    size = dict(ref=10, table=12, held=3, lens=3, source=5)[near]
    far = {k: A + i * 4096 for i, k in enumerate(("ref", "table", "held", "lens", "source"))}
    assert fork(L, **far, **{out: far[near] + 4 * (size - 1)}) == INV
    assert fork(L, **far, **{out: far[near] - 4 * (4 if out != "to" else 19)}) == INV
    assert fork(L, **far, **{out: far[near] + 4 * size}) == ARCH
    assert fork(L, **far, **{out: far[near] - 4 * (5 if out != "to" else 20)}) == ARCH


@pytest.mark.parametrize("sizes", [(32, 32, 8, 512, 128), (64, 8, 8, 129, 64), (1, 32, 8, 1, 128), (1, 4, 4, 128, 80),
                                   (2049, 32, 8, 4, 128), (100000, 8, 1, 1, 64), (0, 8, 1, 1, 64), (9, 2, 1, 200, 256)])
def test_batches_that_never_share_need_the_plain_workspace(L, sizes):
    """More than 128 query rows of a key head and sequence, a single sequence, or
    more than 2048: no state of a prefix is kept for the join."""
    want = L.ra_cache_attention_workspace_bytes(*sizes)
    assert L.ra_cache_attention_shared_workspace_bytes(*sizes) == want
    # one that may share keeps two fp32 states a row
    rows = 16 * 32 * 8
    assert L.ra_cache_attention_shared_workspace_bytes(16, 32, 8, 8, 128) >= 2 * rows * 130 * 4
