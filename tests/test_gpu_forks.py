"""Pages that several sequences hold, and the moves in the cache that follow:
whole numbers and bits, equal to a model on the host."""
import random

import pytest
import torch

import fork_ref as F
import long_context_ra_gb300 as ra
import serve_ref as R
from long_context_ra_gb300 import _native

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAGE = _native.RA_ERR_PAGE


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rows_to_gpu(rows, width):
    t = torch.tensor([r[0] for r in rows], dtype=torch.int32, device=DEV).view(len(rows), width)
    return t, i32([r[1] for r in rows]), i32([r[2] for r in rows])


def same(model, rows, ref, table, held):
    assert ref.tolist() == model.ref
    assert held.tolist() == [r[1] for r in rows]
    assert table.tolist() == [list(r[0]) for r in rows]
    assert (ra.ra_last_device_status() == PAGE) == model.bad
    model.bad = False


def copy_rows(rows):
    return [(list(t), h, n) for t, h, n in rows]


@pytest.mark.parametrize("seed", range(12))
def test_a_run_of_steps(seed):
    """Prompts, forks, drafts, rejections, ends, in any order, in a pool that
    is sometimes too small."""
    r = random.Random(seed)
    page = r.choice([8, 16, 64])
    width, pages = r.randint(3, 12), r.choice([20, 60, 200])
    m = F.Pages(pages, width, page)
    ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
    rows = [([-1] * width, 0, 0) for _ in range(r.randint(1, 6))]
    table, held, lens = rows_to_gpu(rows, width)
    for step in range(40):
        B = len(rows)
        what = r.choice(["reserve", "reserve", "fork", "trim", "end"])
        if what == "reserve":
            T = r.choice([0, 1, 1, 5, 3 * page])
            count = None if r.random() < 0.4 else [r.randint(0, T) for _ in range(B)]
            got = ra.ra_pages_reserve(ref, table, held, lens, page, T, None if count is None else i32(count))
            want = m.reserve(rows, T, count)
            assert [x.tolist() for x in got] == [list(x) for x in want]
            same(m, rows, ref, table, held)
            # some of the new tokens stay
            rows = [(t, h, n if n < 0 else n + r.randint(0, g)) for (t, h, n), g in zip(rows, want[0])]
            lens = i32([x[2] for x in rows])
        elif what == "fork":
            source = [r.randint(-1, B - 1) if r.random() < 0.9 else B for _ in range(r.randint(1, 9))]
            new = m.fork(rows, source)
            t2, h2, l2 = ra.ra_pages_fork(ref, table, held, lens, i32(source), page)
            assert l2.tolist() == [x[2] for x in new]
            same(m, new, ref, t2, h2)
            m.trim(rows)
            ra.ra_pages_trim(ref, table, held, None, page)
            same(m, rows, ref, table, held)
            rows, table, held, lens = new, t2, h2, l2
        elif what == "trim":
            m.trim(rows, [x[2] for x in rows])
            ra.ra_pages_trim(ref, table, held, lens, page)
            same(m, rows, ref, table, held)
        else:
            b = r.randrange(B)
            n = r.choice([-1, max(0, rows[b][2] - r.randint(0, page))])  # ended, or taken back
            rows[b] = (rows[b][0], rows[b][1], n)
            lens = i32([x[2] for x in rows])


def test_the_last_holder_keeps_its_page():
    """Three that share a partial page and all ask: two copies, the third
    stays.  With a fourth that does not ask: three copies."""
    for n, asking in ((3, [1, 1, 1]), (4, [1, 1, 0, 1])):
        m = F.Pages(30, 4, 8)
        rows = [([5, 6, -1, -1], 2, 13)]
        m.ref[5] = m.ref[6] = 1
        new = m.fork(rows, [0] * n)
        m.trim(rows)
        assert m.ref[6] == n
        ref = i32(m.ref)
        table, held, lens = rows_to_gpu(new, 4)
        got = ra.ra_pages_reserve(ref, table, held, lens, 8, 1, i32(asking))
        want = m.reserve(new, 1, asking)
        assert [x.tolist() for x in got] == [list(x) for x in want]
        assert got[1].tolist() == ([6, 6, -1] if n == 3 else [6, 6, -1, 6])
        same(m, new, ref, table, held)


@pytest.mark.parametrize("B,page,T,pages", [(1, 8, 4000, 600), (700, 16, 1, 40000), (3000, 8, 9, 70000),
                                            (8192, 64, 1, 20000), (40, 1024, 300, 41)])
def test_many_sequences_and_pages(B, page, T, pages):
    r = random.Random(B)
    width = F.up(T, page) + 3
    m = F.Pages(pages, width, page)
    for p in r.sample(range(pages), pages // 3 if pages > 100 else 0):
        m.ref[p] = 1  # held elsewhere
    rows = [([-1] * width, 0, 0) for _ in range(B)]
    free = [p for p, x in enumerate(m.ref) if x == 0]
    for b in range(0, B, 3):  # some have a page with a few tokens, which the next one shares
        p = free.pop(r.randrange(len(free)))
        m.ref[p] = 1
        rows[b] = ([p] + [-1] * (width - 1), 1, r.randint(1, page))
        if b + 1 < B and b % 2:
            m.ref[p] = 2
            rows[b + 1] = ([p] + [-1] * (width - 1), 1, rows[b][2])
    ref = i32(m.ref)
    table, held, lens = rows_to_gpu(rows, width)
    got = ra.ra_pages_reserve(ref, table, held, lens, page, T)
    want = m.reserve(rows, T)
    assert [x.tolist() for x in got] == [list(x) for x in want]
    same(m, rows, ref, table, held)
    m.trim(rows, [x[2] for x in rows])
    ra.ra_pages_trim(ref, table, held, lens, page)
    same(m, rows, ref, table, held)


def test_what_is_left_out():
    """A row that would pass the width, one whose context is not held, one that
    shares a page behind its next token, bad page numbers, counts above T: each
    is left out alone."""
    m = F.Pages(16, 3, 8)
    for p, n in ((0, 1), (1, 1), (2, 2), (3, 2), (4, 1)):
        m.ref[p] = n
    rows = [([0, -1, -1], 1, 3), ([1, -1, -1], 1, 5), ([2, 3, -1], 2, 4), ([2, 3, -1], 2, 12), ([99, -1, -1], 1, 2),
            ([-5, -1, -1], 1, 2), ([4, -1, -1], 1, 20)]
    count = [30, 2, 6, 1, 1, 1, 1]
    ref = i32(m.ref)
    table, held, lens = rows_to_gpu(rows, 3)
    got = ra.ra_pages_reserve(ref, table, held, lens, 8, 7, i32(count))
    want = m.reserve(rows, 7, count)
    assert [x.tolist() for x in got] == [list(x) for x in want]
    assert m.bad
    assert got[0].tolist() == [7, 2, 0, 1, 0, 0, 0]
    same(m, rows, ref, table, held)
    new = m.fork(rows, [0, 4, 5, 6, -1, 7, 1])
    t2, h2, l2 = ra.ra_pages_fork(ref, table, held, lens, i32([0, 4, 5, 6, -1, 7, 1]), 8)
    assert m.bad and l2.tolist() == [x[2] for x in new]
    same(m, new, ref, t2, h2)
    m.trim(rows)
    ra.ra_pages_trim(ref, table, held, None, 8)
    assert m.bad  # numbers that are no pages
    same(m, rows, ref, table, held)


def test_counts_that_disagree_stay_inside():
    """More holders than ref says: nothing is written outside, and a count does
    not fall below 0."""
    ref = i32([2, 0, 0, 0])
    table, held, lens = i32([[0, -1]] * 5), i32([1] * 5), i32([3] * 5)
    ra.ra_pages_reserve(ref, table, held, lens, 8, 1)
    ra.ra_last_device_status()
    assert ((table >= -1) & (table < 4)).all()
    ref = i32([1, 0])
    table, held = i32([[0], [0], [1]]), i32([1, 7, 1])
    ra.ra_pages_trim(ref, table, held, None, 8)
    assert ref.tolist() == [0, 0] and held.tolist() == [0, 0, 0] and (table == -1).all()
    assert ra.ra_last_device_status() == PAGE


def test_empty_tables():
    ref = torch.zeros(0, dtype=torch.int32, device=DEV)
    table = torch.zeros(2, 0, dtype=torch.int32, device=DEV)
    held, lens = i32([0, 0]), i32([0, -1])
    t, h, n = ra.ra_pages_fork(ref, table, held, lens, i32([0, 1, 0]), 8)
    assert t.shape == (3, 0) and h.tolist() == [0, 0, 0] and n.tolist() == [0, -1, 0]
    assert ra.ra_last_device_status() == 0
    assert ra.ra_pages_reserve(ref, table, held, lens, 8, 1)[0].tolist() == [0, 0]
    assert ra.ra_last_device_status() == PAGE          # no column for a token
    assert ra.ra_pages_reserve(ref, table, held, lens, 8, 0)[0].tolist() == [0, 0]
    assert ra.ra_last_device_status() == 0


# --------------------------------------------------------------- copy, compact
HELD = [(torch.float32, 8), (torch.float32, 200), (torch.bfloat16, 64), (torch.bfloat16, 8), (torch.bfloat16, 136),
        (torch.float8_e4m3fn, 8), (torch.float8_e4m3fn, 24), (torch.float8_e4m3fn, 128), (torch.float8_e4m3fn, 256)]


def filled(pages, heads, page, d, held, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = ra.new_cache(pages, heads, page, d, held)
    for t in (c.k, c.v, c.k_exp, c.v_exp):
        if t is not None:
            x = t.view(torch.uint8)
            x.copy_(torch.randint(0, 256, x.shape, generator=g, device=DEV, dtype=torch.uint8))  # any bits, NaN too
    return c


def bits(c):
    return [t.view(torch.uint8).view(*c.k.shape[:3], -1).cpu().clone()
            for t in (c.k, c.v, c.k_exp, c.v_exp) if t is not None]


@pytest.mark.parametrize("held,d", HELD)
@pytest.mark.parametrize("heads,page,pages", [(1, 8, 5), (3, 64, 9), (8, 256, 6)])
def test_copy(held, d, heads, page, pages):
    c = filled(pages, heads, page, d, held, 1)
    want = bits(c)
    src, dst = [0, -1, 2, 0, 1, -7], [3, 1, -1, 4, -9, -2]
    for x in want:
        x[3], x[4] = x[0], x[0]
    ra.ra_cache_copy(c, i32(src), i32(dst))
    assert ra.ra_last_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(bits(c), want))
    ra.ra_cache_copy(c, i32([pages, 1, 0]), i32([1, pages + 3, 2]))  # outside: passed over, and said
    for x in want:
        x[2] = x[0]
    assert ra.ra_last_device_status() == PAGE
    assert all(torch.equal(a, b) for a, b in zip(bits(c), want))


def test_copy_of_many_pairs():
    """More pairs than a grid has rows."""
    n = 70000
    c = filled(2 * n, 1, 8, 8, torch.float8_e4m3fn, 2)
    want = bits(c)
    for x in want:
        x[n:] = x[:n]
    at = torch.arange(n, device=DEV, dtype=torch.int32)
    ra.ra_cache_copy(c, at, at + n)
    assert all(torch.equal(a, b) for a, b in zip(bits(c), want))


def moved(want, table, lens, path, kept, page):
    """One row after another, in order."""
    for x in want:
        for b, n in enumerate(lens):
            for j in range(kept[b]):
                a, z = n + path[b][j], n + j
                x[table[b][z // page], :, z % page] = x[table[b][a // page], :, a % page]


@pytest.mark.parametrize("held,d", HELD)
@pytest.mark.parametrize("heads,page,T", [(2, 8, 1), (1, 16, 7), (5, 8, 64), (2, 32, 300)])
def test_compact(held, d, heads, page, T):
    r = random.Random(T * d)
    lens = [0, 37, 5, 16, 3, -1]
    total = [max(n, 0) + T for n in lens]
    table, pages = R.make_paged(total, page, 3)
    c = filled(pages, heads, page, d, held, 4)
    want = bits(c)
    kept, path = [], []
    for b in range(len(lens)):
        k = r.randint(0, T) if b else T
        p = sorted(r.sample(range(T), k))  # overlapping moves: a row is read, then written over
        kept.append(k)
        path.append(p + [r.choice([-1, 0, 99999])] * (T - k))
    moved(want, table.tolist(), lens, path, [k if n >= 0 else 0 for n, k in zip(lens, kept)], page)
    ra.ra_cache_compact(c, table.to(DEV), i32(lens), i32(path), i32(kept))
    assert ra.ra_last_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(bits(c), want))


def test_compact_refuses_paths_that_do_not_rise():
    """A sequence's moves end at the first bad entry; counts above T and
    positions outside the table are said as well."""
    page, T = 8, 140
    lens = [0, 4, 9, 2]
    table, pages = R.make_paged([n + T for n in lens], page, 5)
    table[3, 3] = -1                                   # positions 24 .. 31
    c = filled(pages, 2, page, 16, torch.bfloat16, 6)
    want = bits(c)
    path = [list(range(T)) for _ in lens]
    path[0] = [0, 3, 3, 7] + [9] * (T - 4)             # stops at 2
    path[1] = [2, 5, T, 6] + [7] * (T - 4)             # stops at 2
    path[2] = [i + 1 for i in range(T - 1)] + [0]      # the last one falls; behind 128, too
    kept = [4, 4, T + 5, 0]
    moved(want, table.tolist(), lens, path, [2, 2, T - 1, 0], page)
    ra.ra_cache_compact(c, table.to(DEV), i32(lens), i32(path), i32(kept))
    assert ra.ra_last_device_status() == PAGE
    assert all(torch.equal(a, b) for a, b in zip(bits(c), want))
    # sources and places on a page that is not there are passed over, the others move
    p3 = [1] + list(range(20, 30))
    for x in want:
        for j, node in enumerate(p3):
            a, z = 2 + node, 2 + j
            if not 24 <= a < 32:
                x[table[3][z // page], :, z % page] = x[table[3][a // page], :, a % page]
    full = p3 + [-1] * (T - len(p3))
    ra.ra_cache_compact(c, table.to(DEV), i32(lens), i32([full] * 4), i32([0, 0, 0, len(p3)]))
    assert ra.ra_last_device_status() == PAGE
    assert all(torch.equal(a, b) for a, b in zip(bits(c), want))


def test_offsets_beyond_32_bits():
    """Pages behind 2^32 bytes of a side."""
    heads, page, d = 16, 1024, 128
    pages = (1 << 32) // (heads * page * d * 2) + 3    # bf16: 4 MiB a page
    c = ra.new_cache(pages, heads, page, d)
    c.k[:2].normal_(), c.v[:2].normal_()
    last = pages - 1
    ra.ra_cache_copy(c, i32([1]), i32([last]))
    assert torch.equal(c.k[last], c.k[1]) and torch.equal(c.v[last], c.v[1])
    table = i32([[0, last]])
    row = c.k[last, :, 9].clone(), c.v[last, :, 9].clone()
    ra.ra_cache_compact(c, table, i32([1024]), i32([[0, 9] + [-1] * 8]), i32([2]))
    assert torch.equal(c.k[last, :, 1], row[0]) and torch.equal(c.v[last, :, 1], row[1])
    assert ra.ra_last_device_status() == 0
