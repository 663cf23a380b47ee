"""ra_cache_write and ra_cache_read: the bits of the cache and of what is
read back, over pages, ragged lengths, strides, and calls that point outside
the cache.  Copies are exact; an 8-bit row is the nearest-even rounding of
the row over its power-of-two scale, so equality is asked for throughout."""
import math

import pytest
import torch

import long_context_ra_gb300 as ra
import serve_ref as R
from long_context_ra_gb300 import _native

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn

SHAPES = [
    # lens, count, T, heads, page, d
    ([0], None, 1, 1, 8, 8),
    ([5, 0, 130], [1, 1, 1], 1, 2, 16, 64),
    ([7, 63, 64, 0], [33, 0, 40, 17], 40, 3, 64, 128),
    ([1000, 3], [129, 1], 129, 2, 128, 80),
    ([31, -1, 12], None, 5, 4, 32, 256),
]


def bits(t):
    return t.view(torch.uint8) if t is not None and t.dtype == E4M3 else t


def filled_cache(pages, heads, page, d, dtype, seed):
    """A cache whose every byte has a known value."""
    c = ra.new_cache(pages, heads, page, d, dtype)
    g = torch.Generator(device=DEV).manual_seed(seed)
    for t in (c.k, c.v):
        t.copy_(torch.randn(t.shape, device=DEV, generator=g))
    if c.k_exp is not None:
        for t in (c.k_exp, c.v_exp):
            t.copy_(torch.randint(120, 130, t.shape, device=DEV, generator=g))
    return c


def new_tokens(B, heads, T, d, dtype, seed, strided):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(B, T, 2 * heads, d, device=DEV, generator=g)
    x *= torch.exp(2 * torch.randn(B, T, 2 * heads, 1, device=DEV, generator=g))
    x = x.to(dtype).transpose(1, 2)
    k, v = x[:, :heads], x[:, heads:]
    return (k, v) if strided else (k.contiguous(), v.contiguous())


def expected(cache, table, lens, count, k, v):
    """The cache's tensors (8-bit ones as float64 values) after the write."""
    out = []
    for held, exps, x in ((cache.k, cache.k_exp, k), (cache.v, cache.v_exp, v)):
        vals = held.cpu().float().double() if held.dtype == E4M3 else held.cpu().clone()
        marks = None if exps is None else exps.cpu().clone()
        for b, n in enumerate(lens):
            if n < 0:
                continue
            for t in range(x.shape[2] if count is None else count[b]):
                p = int(table[b, (n + t) // held.shape[2]])
                o = (n + t) % held.shape[2]
                row = x[b, :, t].cpu()
                if marks is None:
                    vals[p, :, o] = row
                else:
                    vals[p, :, o], marks[p, :, o] = R.quantise(row)
        out += [vals, marks]
    return out


@pytest.mark.parametrize("strided", [True, False])
@pytest.mark.parametrize("dtype,held", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, E4M3),
                                        (torch.float32, torch.float32), (torch.float32, E4M3)])
@pytest.mark.parametrize("shape", SHAPES)
def test_write_and_read(shape, dtype, held, strided):
    lens, count, T, heads, page, d = shape
    B = len(lens)
    total = [n + (T if count is None else count[b]) if n >= 0 else 0 for b, n in enumerate(lens)]
    table, pages = R.make_paged(total, page, 3)
    cache = filled_cache(pages, heads, page, d, held, 4)
    k, v = new_tokens(B, heads, T, d, dtype, 5, strided)
    want = expected(cache, table, lens, count, k, v)
    tab = table.to(DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cnt = None if count is None else torch.tensor(count, dtype=torch.int32, device=DEV)
    ra.ra_cache_write(cache, k, v, tab, ln, cnt)
    for got, w in zip((cache.k, cache.k_exp, cache.v, cache.v_exp), want):
        if w is not None:
            g = got.cpu().float().double() if got.dtype == E4M3 else got.cpu()
            assert torch.equal(g, w)
    # read back: every position, and a window that starts and ends inside pages
    now = torch.tensor(total, dtype=torch.int32, device=DEV)
    paged = R.PagedCpu(cache, table)
    for first, n in ((0, max(total) + 3), (max(total) // 3, max(1, max(total) // 2))):
        rk, rv = ra.ra_cache_read(cache, tab, now, first, n, dtype=dtype)
        assert rk.dtype == dtype and rk.shape == (B, heads, n, d)
        for b in range(B):
            wk, wv = paged.rows(b, total[b])
            for r, w in ((rk, wk), (rv, wv)):
                full = torch.zeros(heads, first + n, d, dtype=torch.float64)
                m = min(total[b], first + n)
                full[:, :m] = w[:, :m]
                assert torch.equal(r[b].cpu().double(), full[:, first:])
    assert ra.ra_last_device_status() == 0


def test_written_8_bit_rows_are_stable():
    """A row that is read and written again keeps its values."""
    table, pages = R.make_paged([200], 16, 1)
    tab = table.to(DEV)
    zero, n = (torch.tensor([x], dtype=torch.int32, device=DEV) for x in (0, 200))
    cache = filled_cache(pages, 2, 16, 128, E4M3, 2)
    k, v = new_tokens(1, 2, 200, 128, torch.bfloat16, 3, False)
    ra.ra_cache_write(cache, k, v, tab, zero)
    a = ra.ra_cache_read(cache, tab, n, 0, 200)
    ra.ra_cache_write(cache, *a, tab, zero)
    b = ra.ra_cache_read(cache, tab, n, 0, 200)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_extreme_rows():
    """Zero rows, the scale's borders, the smallest and largest magnitudes,
    infinities and NaN."""
    d = 16
    x = torch.zeros(1, 1, 12, d, device=DEV)
    x[0, 0, 1] = 448.0                                  # exactly the largest value: scale 1
    x[0, 0, 2] = 448.0 * (1 + 2.0 ** -20)               # just above: scale 2
    x[0, 0, 3, 0], x[0, 0, 3, 1] = 3e38, 1e-30
    x[0, 0, 4] = 1e-38
    x[0, 0, 5] = 1e-45                                  # below fp32's normal range
    x[0, 0, 6, 3], x[0, 0, 6, 4] = math.inf, 2.0
    x[0, 0, 7, 5], x[0, 0, 7, 6] = math.nan, -3.0
    x[0, 0, 8] = torch.linspace(-1.75, 1.75, d)
    x[0, 0, 9] = torch.tensor([1.0, 1.0625, 1.1875, 1.0 / 64, 1 / 512, 3 / 1024, 1 / 1024, 0.0] * 2)
    x[0, 0, 10] = -math.inf
    x[0, 0, 11, 0], x[0, 0, 11, 1:] = 256.0, 2.0 ** -10  # a tie at the smallest code: to even, zero
    table, pages = R.make_paged([12], 8, 1)
    cache = filled_cache(pages, 1, 8, d, E4M3, 2)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    ra.ra_cache_write(cache, x, x, table.to(DEV), zero)
    want, e = R.quantise(torch.where(x[0, 0].isfinite(), x[0, 0], torch.sign(x[0, 0]) * 3e38).cpu())
    full, e = R.quantise(x[0, 0].cpu())
    for t in range(12):
        p, o = int(table[0, t // 8]), t % 8
        got = cache.k[p, 0, o].cpu().float().double()
        assert int(cache.k_exp[p, 0, o]) == int(e[t]), t
        for i in range(d):
            xi = float(x[0, 0, t, i])
            if math.isnan(xi):
                assert math.isnan(got[i])
            elif math.isinf(xi):
                assert got[i] == math.copysign(448.0, xi)
            else:
                assert got[i] == full[t, i], (t, i)


@pytest.mark.parametrize("what", ["page", "negative page", "width", "count"])
def test_positions_outside_the_cache_touch_nothing(what):
    """A page number or position outside the cache skips the token, reads as
    zero and is reported once; everything else of the call is done."""
    lens, T, page = [6, 20], 4, 8
    table, pages = R.make_paged([n + T for n in lens], page, 9, width_extra=0)
    cache = filled_cache(pages, 2, page, 64, torch.bfloat16, 1)
    ok = filled_cache(pages, 2, page, 64, torch.bfloat16, 1)
    k, v = new_tokens(2, 2, T, 64, torch.bfloat16, 2, True)
    count = [T, T]
    bad = table.clone()
    skipped = {}
    if what == "page":
        bad[0, 1] = pages
        skipped = {0: [2, 3]}  # positions 8, 9
    elif what == "negative page":
        bad[0, 1] = -1
        skipped = {0: [2, 3]}
    elif what == "width":
        lens = [6, 24 - 2]     # positions 22 .. 25 of a table of 24
        skipped = {1: [2, 3]}
    else:
        count = [T, T + 3]     # only T tokens exist
    tab = bad.to(DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ra.ra_cache_write(cache, k, v, tab, ln, torch.tensor(count, dtype=torch.int32, device=DEV))
    assert ra.ra_last_device_status() == _native.RA_ERR_PAGE
    assert ra.ra_last_device_status() == 0
    for b in range(2):
        for t in range(T):
            if t in skipped.get(b, []):
                continue
            p, o = int(bad[b, (lens[b] + t) // page]), (lens[b] + t) % page
            ok.k[p, :, o], ok.v[p, :, o] = k[b, :, t], v[b, :, t]
    assert torch.equal(cache.k, ok.k) and torch.equal(cache.v, ok.v)
    if what != "count":
        now = ln + T
        rk, _ = ra.ra_cache_read(cache, tab, now, 0, 30)
        assert ra.ra_last_device_status() == _native.RA_ERR_PAGE
        for b, ts in skipped.items():
            for t in ts:
                assert not rk[b, :, lens[b] + t].any()


@pytest.mark.parametrize("first", [200, 2 ** 31 - 1, 2 ** 31, 2 ** 62, 2 ** 63 - 1, 2 ** 63 - 40])
def test_reading_behind_the_end_gives_zeros(first):
    cache = filled_cache(4, 2, 64, 64, torch.bfloat16, 9)
    table = torch.tensor([[2, 0, 3], [1, 0, 2]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([190, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    k, v = ra.ra_cache_read(cache, table, lens[:1].repeat(2), first, 70)
    assert not k.any() and not v.any()
    assert _native.lib().ra_last_device_status(None) == _native.RA_OK
    # a length beyond the table: zeros too, and the status says so
    k, v = ra.ra_cache_read(cache, table, lens, first, 70)
    assert not k.any() and not v.any()
    assert _native.lib().ra_last_device_status(None) == (
        _native.RA_ERR_PAGE if first < 2 ** 31 - 1 else _native.RA_OK)


def test_rows_of_other_sequences_and_pages_are_left():
    """Guard rows: only the new tokens' rows change."""
    table, pages = R.make_paged([40], 16, 11, spare=4)
    cache = filled_cache(pages, 2, 16, 64, E4M3, 1)
    before = [t.clone() for t in (bits(cache.k), cache.k_exp, bits(cache.v), cache.v_exp)]
    k, v = new_tokens(1, 2, 4, 64, torch.bfloat16, 2, True)
    ra.ra_cache_write(cache, k, v, table.to(DEV), torch.tensor([14], dtype=torch.int32, device=DEV))
    live = torch.zeros(pages, 16, dtype=torch.bool, device=DEV)
    for p in range(14, 18):
        live[int(table[0, p // 16]), p % 16] = True
    for now, then in zip((bits(cache.k), cache.k_exp, bits(cache.v), cache.v_exp), before):
        changed = (now != then).flatten(3).any(-1) if now.dim() == 4 else now != then
        assert not (changed & ~live[:, None]).any()
