"""ra_cache_attention against the 64-bit softmax over the cache's values.

Tolerances, before any run.  With A = sum p |v| / l per element and S = tau
sum |q||k| of a row's largest key: the scores carry (d + 8) 2^-24 S (d
products, fp32 sums), which moves every p by twice that relatively (p and l);
the hardware exponentials 2^-20; sums over n keys at most n 2^-24.  On the
tensor cores p is rounded once (2^-8 for bf16, 2^-11 for the f16 of an 8-bit
cache: 2^-8 covers both), and the result once more (its own half step).
    |out - want| <= half |want| + A (round_p + 2 (d + 8) 2^-24 S + 2^-20 + n 2^-24)
    |lse - want| <= (d + 8) 2^-24 S + 2^-20 + n 2^-24 + 2^-23 |want|"""
import math

import pytest
import torch

import long_context_ra_gb300 as ra
import serve_ref as R
from long_context_ra_gb300 import _native

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn
ROUND_P = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def make(lens, count, T, Hq, heads, page, d, dtype, held, seed, scale=1.0):
    """Queries, a cache whose used positions hold random rows and whose other
    rows are NaN, and the table."""
    B = len(lens)
    total = [n + (T if count is None else count[b]) if n >= 0 else 0 for b, n in enumerate(lens)]
    table, pages = R.make_paged(total, page, seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    cache = ra.new_cache(pages, heads, page, d, held)
    for t, e, s in ((cache.k, cache.k_exp, scale), (cache.v, cache.v_exp, 1.0)):
        t.copy_(torch.full(t.shape, math.nan, device=DEV))
        if e is not None:
            e.fill_(255)
    n = max(max(total), 1)
    x = torch.randn(B, heads, n, 2, d, device=DEV, generator=g)
    x *= torch.exp(torch.randn(B, heads, n, 2, 1, device=DEV, generator=g))
    x = x.to(dtype)
    zero = torch.tensor([0 if t > 0 else -1 for t in total], dtype=torch.int32, device=DEV)
    ra.ra_cache_write(cache, (x[:, :, :, 0] * scale).contiguous(), x[:, :, :, 1].contiguous(),
                      table.to(DEV), zero, torch.tensor(total, dtype=torch.int32, device=DEV))
    q = torch.randn(B, Hq, T, d, device=DEV, generator=g).to(dtype)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cnt = None if count is None else torch.tensor(count, dtype=torch.int32, device=DEV)
    return q, cache, table, ln, cnt


def check(got, q, cache, table, lens, count, mask):
    out, lse = got
    want, wl, mag, size = R.attention(q, R.PagedCpu(cache, table), lens, count,
                                      None if mask is None else mask.cpu())
    dtype, d = q.dtype, q.shape[-1]
    n = max(lens) + q.shape[2]
    common = 2.0 ** -20 + n * R.U + 0 * size
    score = (d + 8) * R.U * size
    assert torch.equal(wl == -math.inf, lse.cpu().double() == -math.inf)
    live = wl > -math.inf
    el = (lse.cpu().double() - wl).abs()[live]
    assert (el <= (score + common + 2.0 ** -23 * wl.abs())[live]).all(), el.max()
    tol = R.EPS_HALF[dtype] * want.abs() + mag * (ROUND_P[dtype] + 2 * score + common)[..., None]
    err = (out.cpu().double() - want).abs()
    assert (err <= tol).all(), (err - tol).max()
    assert not out[~live.to(DEV)].any()


TYPES = [(torch.float32, torch.float32, 80), (torch.float32, E4M3, 256), (torch.float32, torch.float32, 8),
         (torch.bfloat16, torch.bfloat16, 64), (torch.bfloat16, torch.bfloat16, 128),
         (torch.bfloat16, E4M3, 64), (torch.bfloat16, E4M3, 128)]

SHAPES = [
    # lens, count, T, Hq, heads, page
    ([0], None, 1, 1, 1, 8),                      # a first token: it sees itself alone
    ([1], None, 1, 4, 2, 16),
    ([127, 128, 129, 1000], None, 1, 8, 2, 64),   # borders of tiles and pages
    ([3000], None, 1, 5, 5, 16),                  # one long row, split
    ([700, 5, 0, 333], [3, 1, 3, 2], 3, 12, 2, 32),
    ([513, -1, 40], [17, 17, 0], 17, 4, 2, 128),  # sequences that take no part
    ([900, 250], None, 33, 6, 3, 64),             # 66 rows a head
    ([1500], None, 61, 16, 2, 1024),              # 488 rows a head
    ([300, 2000, 77], [40, 64, 9], 64, 8, 2, 16),  # 256 rows a head, ragged
]


@pytest.mark.parametrize("dtype,held,d", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_causal(shape, dtype, held, d):
    lens, count, T, Hq, heads, page = shape
    q, cache, table, ln, cnt = make(lens, count, T, Hq, heads, page, d, dtype, held, 1)
    got = ra.ra_cache_attention(q, cache, table.to(DEV), ln, cnt)
    assert ra.ra_last_device_status() == 0
    check(got, q, cache, table, lens, count, None)


def tree(B, T, seed):
    g = torch.Generator().manual_seed(seed)
    m = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            p = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            if p >= 0:
                m[b, i] = m[b, p]
            m[b, i, i] = True
    return m


@pytest.mark.parametrize("dtype,held,d", TYPES)
@pytest.mark.parametrize("shape", SHAPES[4:])
@pytest.mark.parametrize("shared", [False, True])
def test_tree(shape, dtype, held, d, shared):
    lens, count, T, Hq, heads, page = shape
    q, cache, table, ln, cnt = make(lens, count, T, Hq, heads, page, d, dtype, held, 2)
    mask = tree(1, T, 3)[0] if shared else tree(len(lens), T, 3)
    got = ra.ra_cache_attention(q, cache, table.to(DEV), ln, cnt, mask.to(DEV))
    assert ra.ra_last_device_status() == 0
    check(got, q, cache, table, lens, count, mask)


@pytest.mark.parametrize("dtype,held,d", TYPES[3:] + TYPES[:1])
@pytest.mark.parametrize("T", [3, 40])
def test_masks_that_leave_rows_empty(T, dtype, held, d):
    """Rows whose mask shows no drafted token: with a context they see that,
    without one they are empty; a mask that is all false likewise."""
    lens, count, Hq, heads, page = [50, 0, 0, 128], None, 4, 2, 16
    q, cache, table, ln, cnt = make(lens, count, T, Hq, heads, page, d, dtype, held, 4)
    mask = torch.rand(4, T, T, generator=torch.Generator().manual_seed(5)) < 0.3
    mask[:, 1] = False
    mask[2] = False
    got = ra.ra_cache_attention(q, cache, table.to(DEV), ln, cnt, mask.to(DEV))
    check(got, q, cache, table, lens, count, mask)


@pytest.mark.parametrize("dtype,held,d", TYPES[3:] + TYPES[:1])
@pytest.mark.parametrize("T", [2, 40])
def test_unseen_rows_may_hold_anything(T, dtype, held, d):
    """NaN and infinities in drafted rows that some queries do not see do not
    reach those queries."""
    lens, Hq, heads, page = [70, 128], 4, 2, 16
    q, cache, table, ln, _ = make(lens, None, T, Hq, heads, page, d, dtype, held, 6)
    mask = tree(2, T, 7)
    mask[:, 1:, 0] = False  # token 0 is seen by itself alone
    mask[:, 0] = False
    mask[:, 0, 0] = True
    want = ra.ra_cache_attention(q, cache, table.to(DEV), ln, None, mask.to(DEV))
    for value in (math.nan, math.inf):
        bad = ra.RaCache(cache.k.clone(), cache.v.clone(),
                         *(None if e is None else e.clone() for e in (cache.k_exp, cache.v_exp)))
        for b in range(2):
            p, o = int(table[b, lens[b] // page]), lens[b] % page
            for t in (bad.k, bad.v):
                t[p, :, o] = torch.full((heads, d), value, device=DEV).to(held)
            if held == E4M3 and value == math.inf:  # an 8-bit row is infinite by its exponent
                for t, e in ((bad.k, bad.k_exp), (bad.v, bad.v_exp)):
                    t[p, :, o] = torch.ones(heads, d, device=DEV).to(held)
                    e[p, :, o] = 255
        out, lse = ra.ra_cache_attention(q, bad, table.to(DEV), ln, None, mask.to(DEV))
        assert torch.equal(out[:, :, 1:], want[0][:, :, 1:])
        assert torch.equal(lse[:, :, 1:], want[1][:, :, 1:])
        # the query that sees it: not finite (an 8-bit row of one sign times an
        # infinite scale may score -inf, which is no weight at all)
        if held != E4M3 or math.isnan(value):
            assert not torch.isfinite(out[:, :, 0].float()).any()


@pytest.mark.parametrize("dtype,held,d", TYPES[3:] + TYPES[:1])
@pytest.mark.parametrize("T", [1, 24, 70])
def test_growing_scores_and_unlike_scales(T, dtype, held, d):
    """Scores that rise along the keys (the running maximum moves in every
    tile) and value rows of magnitudes 2^-20 .. 2^20."""
    lens, Hq, heads, page = [2500], 8, 2, 64
    q, cache, table, ln, _ = make(lens, None, T, Hq, heads, page, d, dtype, held, 8)
    n = lens[0] + T
    g = torch.Generator(device=DEV).manual_seed(9)
    k = torch.randn(1, heads, n, d, device=DEV, generator=g)
    k += q.float().reshape(heads, -1, d).mean(1)[None, :, None] * torch.linspace(0, 12, n, device=DEV)[None, None, :, None]
    v = torch.randn(1, heads, n, d, device=DEV, generator=g)
    v *= torch.exp2(40 * torch.rand(1, 1, n, 1, device=DEV, generator=g) - 20)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    ra.ra_cache_write(cache, k.to(dtype), v.to(dtype), table.to(DEV), zero)
    got = ra.ra_cache_attention(q, cache, table.to(DEV), ln)
    check(got, q, cache, table, lens, None, None)


@pytest.mark.parametrize("dtype,held,d", [TYPES[0], TYPES[4], TYPES[6]])
def test_large_ragged_batch(dtype, held, d):
    """More sequences than a block has threads, lengths from none to long."""
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(-1, 60, (700,), generator=g).tolist()
    lens[13], lens[699] = 1500, 900
    q, cache, table, ln, cnt = make(lens, None, 1, 2, 1, 16, d, dtype, held, 12)
    got = ra.ra_cache_attention(q, cache, table.to(DEV), ln)
    check(got, q, cache, table, lens, None, None)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("held", [torch.bfloat16, E4M3])
def test_bad_pages_leave_their_keys_out(held, T):
    lens, Hq, heads, page, d = [200, 90], 4, 2, 16, 128
    q, cache, table, ln, _ = make(lens, None, T, Hq, heads, page, d, torch.bfloat16, held, 13)
    bad = table.clone()
    bad[0, 0], bad[0, 5] = cache.k.shape[0], -7
    out, lse = ra.ra_cache_attention(q, cache, bad.to(DEV), ln)
    assert ra.ra_last_device_status() == _native.RA_ERR_PAGE
    assert ra.ra_last_device_status() == 0
    # the other sequence is as it was; the first sees the other 12 pages' keys
    good = ra.ra_cache_attention(q, cache, table.to(DEV), ln)
    assert torch.equal(out[1], good[0][1]) and torch.equal(lse[1], good[1][1])
    keep = [p for i, p in enumerate(table[0].tolist()) if i not in (0, 5)]
    less = table.clone()
    less[0] = torch.tensor(keep + [-1, -1])
    alone = ra.ra_cache_attention(q[:1].contiguous(), cache, less[:1].to(DEV).contiguous(), ln[:1] - 2 * page)
    torch.testing.assert_close(out[:1].float(), alone[0].float(), atol=2e-2, rtol=2.0 ** -6)
    torch.testing.assert_close(lse[:1], alone[1], atol=1e-4, rtol=1e-5)


def test_results_repeat_and_do_not_depend_on_the_workspace():
    lens = [3000, 17, 1200]
    for T, held in ((1, E4M3), (40, torch.bfloat16)):
        q, cache, table, ln, _ = make(lens, None, T, 8, 2, 64, 128, torch.bfloat16, held, 14)
        n = ra.ra_cache_attention_workspace_bytes(3, 8, 2, T, 128)
        first = ra.ra_cache_attention(q, cache, table.to(DEV), ln)
        for fill in (0, 255):
            ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
            again = ra.ra_cache_attention(q, cache, table.to(DEV), ln, workspace=ws)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def with_value(cache, table, places, head, column, value):
    """A copy of the cache with `value` in one column of V at the given
    (sequence, position) places of one key head."""
    v = cache.v.clone()
    page = v.shape[2]
    for b, n in places:
        p = int(table[b, n // page])
        if v.dtype == E4M3:
            assert math.isnan(value)
            v.view(torch.uint8)[p, head, n % page, column] = 0x7f
        else:
            v[p, head, n % page, column] = value
    return ra.RaCache(cache.k, v, cache.k_exp, cache.v_exp)


def check_one_column(got, want, g, head, column, lens, count, T):
    """Column `column` of the rows of key head `head` is not finite; all else
    has the bits of `want`."""
    live = torch.zeros(got[0].shape[:3], dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        if n >= 0:
            live[b, :, :T if count is None else count[b]] = True
    assert not got[0][:, head * g:(head + 1) * g, :, column][live[:, head * g:(head + 1) * g]].isfinite().any()
    same = torch.ones(got[0].shape, dtype=torch.bool, device=DEV)
    same[:, head * g:(head + 1) * g, :, column] = False
    same |= ~live[..., None]
    assert torch.equal(got[0][same], want[0][same]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype,held,d,value", [
    (*t, x) for t in TYPES[3:] + TYPES[:1] for x in (math.nan, math.inf)
    if t[1] != E4M3 or math.isnan(x)])   # an 8-bit code is finite or NaN
@pytest.mark.parametrize("T", [1, 3, 40, 100])
def test_context_values_that_are_not_finite(dtype, held, d, value, T):
    """A NaN or an infinity in the last rows of the context, which share a tile
    with the new tokens, reaches every query, in its column only."""
    lens, Hq, heads, page = [70, 2000, 200, 2, -1], 4, 2, 16
    count = [T, T, max(1, T // 2), T, T]
    q, cache, table, ln, cnt = make(lens, count, T, Hq, heads, page, d, dtype, held, 15)
    want = ra.ra_cache_attention(q, cache, table.to(DEV), ln, cnt)
    for back, column, head in ((1, 5, 0), (2, d - 1, 1)):
        bad = with_value(cache, table, [(b, n - back) for b, n in enumerate(lens) if n > 0], head, column, value)
        got = ra.ra_cache_attention(q, bad, table.to(DEV), ln, cnt)
        check_one_column(got, want, 2, head, column, lens, count, T)
    assert ra.ra_last_device_status() == 0


def check_weight_zero(places, T, dtype, held, d):
    """For each (top, at) of `places` a sequence of 3000 in which key `top`
    scores 200 or more above all others, whose weights so are 0 in fp32: a NaN
    in the value row at `at`, which every query sees, makes its column NaN."""
    Hq, heads, page, n = 4, 2, 32, 3000
    lens = [n] * len(places)
    B = len(lens)
    table, pages = R.make_paged([n + T] * B, page, 16)
    cache = ra.new_cache(pages, heads, page, d, held)
    g = torch.Generator(device=DEV).manual_seed(17)
    k = torch.zeros(B, heads, n + T, d, device=DEV, dtype=dtype)
    v = torch.randn(B, heads, n + T, d, device=DEV, generator=g).to(dtype)
    for b, (top, _) in enumerate(places):
        k[b, :, top] = 8
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    ra.ra_cache_write(cache, k, v, table.to(DEV), zero)
    q = torch.full((B, Hq, T, d), 4.0, device=DEV, dtype=dtype)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = ra.ra_cache_attention(q, cache, table.to(DEV), ln)
    bad = with_value(cache, table, [(b, at) for b, (_, at) in enumerate(places)], 1, 7, math.nan)
    got = ra.ra_cache_attention(q, bad, table.to(DEV), ln)
    check_one_column(got, want, 2, 1, 7, lens, None, T)


@pytest.mark.parametrize("dtype,held,d", TYPES[:3])
@pytest.mark.parametrize("T", [1, 3, 24, 100])
def test_nan_at_weight_zero_in_the_last_tile(T, dtype, held, d):
    """Both keys in the tile that holds the end of the context."""
    check_weight_zero([(2999, 2998), (2998, 3000)], T, dtype, held, d)


@pytest.mark.parametrize("dtype,held,d", TYPES[:2] + TYPES[3:])
@pytest.mark.parametrize("T", [1, 3, 24, 100])
def test_nan_at_weight_zero_in_another_part(T, dtype, held, d):
    """The two keys in the same or in other tiles, which other warps, streams
    or blocks may work on: their states are joined with weight 0."""
    check_weight_zero([(0, 40), (40, 0), (5, 2990), (2990, 5), (100, 164), (64, 2999), (2999, 2998),
                       (2998, 3000)], T, dtype, held, d)


LONG = [
    ([0], None, 300, 4, 2, 64),                    # a prompt without a context
    ([77, -1, 500], [257, 3, 140], 257, 4, 2, 16),  # chunks of two prompts, 514 rows a head
    ([33], None, 520, 3, 3, 128),
]


@pytest.mark.parametrize("dtype,held,d", TYPES)
@pytest.mark.parametrize("shape", LONG)
def test_chunks_of_a_prompt(shape, dtype, held, d):
    """More new tokens than a tile has rows."""
    lens, count, T, Hq, heads, page = shape
    q, cache, table, ln, cnt = make(lens, count, T, Hq, heads, page, d, dtype, held, 18)
    got = ra.ra_cache_attention(q, cache, table.to(DEV), ln, cnt)
    assert ra.ra_last_device_status() == 0
    check(got, q, cache, table, lens, count, None)


@pytest.mark.parametrize("dtype,held,d", TYPES[3:] + TYPES[:1])
@pytest.mark.parametrize("at", [0, 127, 150, 256])
def test_a_new_value_that_is_not_finite_in_a_chunk(at, dtype, held, d):
    """It reaches the tokens from its own on, in its column, and no bit of the
    ones before, whichever tile of rows they are in."""
    lens, T, Hq, heads, page, column = [100, 0], 257, 4, 2, 32, 9
    q, cache, table, ln, _ = make(lens, None, T, Hq, heads, page, d, dtype, held, 19)
    want = ra.ra_cache_attention(q, cache, table.to(DEV), ln)
    bad = with_value(cache, table, [(b, n + at) for b, n in enumerate(lens)], 1, column, math.nan)
    out, lse = ra.ra_cache_attention(q, bad, table.to(DEV), ln)
    assert out[:, 2:, at:, column].isnan().all()
    same = torch.ones(out.shape, dtype=torch.bool, device=DEV)
    same[:, 2:, at:, column] = False
    assert torch.equal(out[same], want[0][same]) and torch.equal(lse, want[1])
