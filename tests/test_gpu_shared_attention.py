"""ra_cache_attention_shared against the 64-bit softmax over the cache's
values, each sequence by its own table row.

Tolerances are those of test_gpu_cache_attention, derived there: a state over a
prefix and one over the rest are joined as the parts of a divided row are, with
one more weight of relative error 2^-20, which the bound for the hardware
exponentials (2^-20 on every p, of which the kernels' own ex2 takes 2^-22) and
the n 2^-24 of the sums hold."""
import math

import pytest
import torch

import long_context_ra_gb300 as ra
import serve_ref as R
from long_context_ra_gb300 import _native
from test_gpu_cache_attention import TYPES, check, check_one_column, tree, with_value

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def wide(table, cache):
    """The table with columns of no page behind: as large as one must be for
    prefixes to be shared rather than read again."""
    _, heads, page, d = cache.k.shape
    column = (table.shape[0] - 1) * page * heads * 2 * d * cache.k.element_size()
    more = (160 << 20) // max(column, 1) + 1
    return torch.cat([table, torch.full((table.shape[0], more), -1, dtype=torch.int32)], 1).to(DEV)


def make(groups, count, T, Hq, heads, page, d, dtype, held, seed, same_pages=True):
    """groups: (prefix, [own context tokens of each sequence; None: lens = -1]).
    The prefix of a group is the same in all of its sequences: whole pages are
    the first one's (or equal copies), the rest of it equal copies; all that no
    sequence holds is NaN."""
    lens, shared, of = [], [], []
    for g, (prefix, own) in enumerate(groups):
        began = False
        for n in own:
            of.append(g)
            lens.append(-1 if n is None else prefix + n)
            shared.append(prefix if began else (0 if len(lens) > 1 else 99999))
            began = began or n is not None
    B = len(lens)
    total = [n + (T if count is None else count[b]) if n >= 0 else 0 for b, n in enumerate(lens)]
    table, pages = R.make_paged(total, page, seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    cache = ra.new_cache(pages, heads, page, d, held)
    for t, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        t.copy_(torch.full(t.shape, math.nan, device=DEV))
        if e is not None:
            e.fill_(255)
    n = max(max(total), 1)
    x = torch.randn(B, heads, n, 2, d, device=DEV, generator=g)
    x *= torch.exp(torch.randn(B, heads, n, 2, 1, device=DEV, generator=g))
    lead = {}
    for b in range(B):
        if lens[b] < 0:
            continue
        a, prefix = lead.setdefault(of[b], b), groups[of[b]][0]
        x[b, :, :prefix] = x[a, :, :prefix]
        if same_pages:
            table[b, :prefix // page] = table[a, :prefix // page]
    zero = i32([0 if t > 0 else -1 for t in total])
    x = x.to(dtype)
    ra.ra_cache_write(cache, x[:, :, :, 0].contiguous(), x[:, :, :, 1].contiguous(), table.to(DEV), zero, i32(total))
    q = torch.randn(B, Hq, T, d, device=DEV, generator=g).to(dtype)
    return q, cache, table, lens, i32(shared), None if count is None else i32(count)


SHAPES = [
    # groups, count, T, Hq, heads, page
    ([(300, [5, 0, 60])], None, 1, 8, 2, 16),                            # few rows: 12
    ([(700, list(range(20)))], None, 1, 8, 2, 64),                       # one tile of rows: 80
    ([(700, list(range(40)))], None, 1, 4, 1, 128),                      # two tiles: 160
    ([(2000, [3, 130, 70] * 23)], None, 1, 32, 8, 32),                   # two units and a rest
    ([(140, [3, None, 5]), (0, [7]), (600, [None, 9, 400, None, 0, 1])], None, 2, 6, 2, 8),  # ragged, some take no part
    ([(384, [0, 0, 1]), (1000, [300] * 4)], [3, 0, 1, 3, 2, 0, 3], 3, 3, 1, 64),   # 9 rows a sequence, counts
    ([(300, [10, 200, 30, 7, 9, 11])], [17, 4, 0, 17, 1, 9], 17, 4, 2, 128),       # 34 rows a sequence
    ([(520, [10, 200, 30, 7, 9])], None, 32, 8, 2, 64),                  # 128 rows: two sequences to a unit
    ([(1000, [50, 0]), (200, [30] * 3)], None, 21, 3, 1, 256),           # 63 rows, pages longer than a tile
    ([(2500, [1, 1, 1])], None, 1, 2, 1, 1024),                          # pages of 1024
    ([(100, [5, 6, 7])], None, 1, 4, 2, 16),                             # shorter than a tile: nothing in common
    ([(257, [b % 5 for b in range(2)]) for _ in range(50)], None, 1, 4, 2, 16),    # many groups of two
    ([(50000, [9, 1])], None, 1, 1, 1, 256),                             # a long one, divided among all
    ([(256, [40, 3])], None, 65, 4, 2, 16),                              # more rows than two fit a unit
]


@pytest.mark.parametrize("dtype,held,d", TYPES)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_causal(shape, dtype, held, d):
    groups, count, T, Hq, heads, page = SHAPES[shape]
    q, cache, table, lens, shared, cnt = make(groups, count, T, Hq, heads, page, d, dtype, held, 1)
    got = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared, cnt)
    assert ra.ra_last_device_status() == 0
    check(got, q, cache, table, lens, count, None)
    # a small table: each reads its own pages, as without sharing
    if (len(lens) - 1) * table.shape[1] * page * heads * 2 * d * cache.k.element_size() >= 160 << 20:
        return
    got = ra.ra_cache_attention_shared(q, cache, table.to(DEV), i32(lens), shared, cnt)
    want = ra.ra_cache_attention(q, cache, table.to(DEV), i32(lens), cnt)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype,held,d", TYPES)
@pytest.mark.parametrize("shape", [4, 5, 6, 7, 8])
@pytest.mark.parametrize("one_mask", [False, True])
def test_tree(shape, one_mask, dtype, held, d):
    groups, count, T, Hq, heads, page = SHAPES[shape]
    q, cache, table, lens, shared, cnt = make(groups, count, T, Hq, heads, page, d, dtype, held, 2)
    mask = tree(1, T, 3)[0] if one_mask else tree(len(lens), T, 3)
    if not one_mask and len(lens) > 2:
        mask[2] = False                      # new tokens that see the context alone
    got = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared, cnt, mask.to(DEV))
    assert ra.ra_last_device_status() == 0
    check(got, q, cache, table, lens, count, mask)


@pytest.mark.parametrize("held,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (E4M3, 64), (E4M3, 128)])
@pytest.mark.parametrize("Hq,T", [(1, 1), (7, 1), (2, 4), (9, 1), (3, 5), (16, 1), (2, 12)])
def test_rows_of_a_small_unit(Hq, T, held, d):
    """1 to 24 rows of a key head: the decode kernel works on one half of its 16 rows or on both."""
    q, cache, table, lens, shared, cnt = make([(300, [70, 9]), (0, [200, 0, None, 1])], None, T, 2 * Hq, 2, 32, d,
                                              torch.bfloat16, held, 6)
    got = ra.ra_cache_attention(q, cache, table.to(DEV), i32(lens))
    check(got, q, cache, table, lens, None, None)
    got = ra.ra_cache_attention_shared(q[:2].contiguous(), cache, wide(table[:2], cache), i32(lens[:2]), shared[:2])
    check(got, q[:2], cache, table[:2], lens[:2], None, None)
    assert ra.ra_last_device_status() == 0


WIDE = [(torch.float32, torch.float32, 80, 1), (torch.bfloat16, torch.bfloat16, 64, 1),
        (torch.bfloat16, torch.bfloat16, 128, 12), (torch.bfloat16, E4M3, 128, 40)]


@pytest.mark.parametrize("dtype,held,d,T", WIDE)
def test_the_common_part_is_the_first_ones(dtype, held, d, T):
    """Equal copies: once the others' copies of the whole tiles are spoilt, the
    result stays, so they are not read."""
    groups = [(300, [5, 90, 3, 8, 0])]
    q, cache, table, lens, shared, _ = make(groups, None, T, 2, 1, 16, d, dtype, held, 4, same_pages=False)
    want = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared)
    check(want, q, cache, table, lens, None, None)
    for b in range(1, len(lens)):
        for p in table[b, :256 // 16].tolist():
            cache.v.view(torch.uint8)[p] = 0x7f
            cache.k.view(torch.uint8)[p] = 0x7f
    got = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype,held,d,T", WIDE)
def test_entries_of_all_kinds(dtype, held, d, T):
    """Entries above the lengths, negative ones, a smaller one that holds for
    its group: what is in common is never more than they say."""
    groups = [(512, [8, 100, 0, 30]), (400, [3, 3, 70])]
    q, cache, table, lens, shared, _ = make(groups, None, T, 2, 1, 32, d, dtype, held, 5)
    plain = ra.ra_cache_attention(q, cache, table.to(DEV), i32(lens))
    for entries in ([7, 1 << 30, 512, 512, -3, 1 << 30, 400], [0, 512, 130, 512, 0, 400, 127],
                    [-5, -1, 0, 512, 0, 0, 0], [0] * 7):
        if max(entries) > 1000:  # more than is in common would be wrong: only where the lengths cut it
            entries = [min(e, 512 if b < 4 else 400) if e > 1000 else e for b, e in enumerate(entries)]
        got = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), i32(entries))
        check(got, q, cache, table, lens, None, None)
    one = [(512, [0, 0])]
    q, cache, table, lens, shared, _ = make(one, None, T, 2, 1, 32, d, dtype, held, 6)
    got = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), i32([0, 1 << 30]))  # cut by lens
    check(got, q, cache, table, lens, None, None)
    assert plain[0].isfinite().all()


@pytest.mark.parametrize("dtype,held,d,T", WIDE)
def test_many_sequences(dtype, held, d, T):
    """As many as the plan takes, and one more (which shares nothing)."""
    T = min(T, 2)
    for B in (2048, 2049):
        own = [b % 3 for b in range(B)]
        groups = [(128, own[:1500]), (0, own[1500:1700]), (260, own[1700:])]
        q, cache, table, lens, shared, _ = make(groups, None, T, 1, 1, 128, d, dtype, held, 7)
        got = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared)
        want = ra.ra_cache_attention(q, cache, table.to(DEV), i32(lens))
        some = list(range(0, B, 97)) + [1499, 1500, 1699, 1700, B - 1]
        assert ra.ra_last_device_status() == 0
        check((got[0][some], got[1][some]), q[some], cache, table[some], [lens[b] for b in some], None, None)
        torch.testing.assert_close(got[1], want[1], atol=1e-4, rtol=1e-5)


@pytest.mark.parametrize("dtype,held,d,T", WIDE)
def test_values_that_are_not_finite_in_a_prefix(dtype, held, d, T):
    """A NaN in a value row of the prefix reaches every query of its group, in
    its column only."""
    groups = [(300, [5, 70, 0]), (0, [400]), (290, [3, 9])]
    q, cache, table, lens, shared, _ = make(groups, None, T, 4, 2, 16, d, dtype, held, 8)
    want = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared)
    for at in (0, 255, 256, 285):
        places = [(b, at) for b in range(6)]
        bad = with_value(cache, table, places, 1, 7, math.nan)
        got = ra.ra_cache_attention_shared(q, bad, wide(table, bad), i32(lens), shared)
        check_one_column(got, want, 2, 1, 7, lens, None, T)


@pytest.mark.parametrize("dtype,held,d,T", WIDE)
def test_weights_of_0_between_prefix_and_rest(dtype, held, d, T):
    """A key that takes all weight in the one, a NaN in the other."""
    for top, at in ((5, 310), (310, 5), (200, 201), (301, 302)):
        groups = [(300, [20, 30, 40])]
        q, cache, table, lens, shared, _ = make(groups, None, T, 2, 1, 64, d, dtype, held, 9)
        n = max(lens)
        k = torch.zeros(3, 1, n + T, d, device=DEV, dtype=dtype)
        v = torch.randn(3, 1, n + T, d, device=DEV).to(dtype)
        v[1:, :, :300] = v[:1, :, :300]
        k[:, :, top] = 8
        ra.ra_cache_write(cache, k, v, table.to(DEV), i32([0] * 3), i32([x + T for x in lens]))
        q = torch.full_like(q, 4.0)
        want = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared)
        bad = with_value(cache, table, [(b, at) for b in range(3)], 0, 7, math.nan)
        got = ra.ra_cache_attention_shared(q, bad, wide(table, bad), i32(lens), shared)
        check_one_column(got, want, 2, 0, 7, lens, None, T)


@pytest.mark.parametrize("dtype,held,d,T", WIDE)
def test_drafts_that_are_not_seen(dtype, held, d, T):
    """NaN in a new token's rows does not reach the queries that do not see it."""
    T = max(T, 3)
    groups = [(300, [5, 70, 0])]
    q, cache, table, lens, shared, _ = make(groups, None, T, 2, 1, 16, d, dtype, held, 10)
    mask = tree(3, T, 7)
    mask[:, 1:, 0] = False
    want = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared, None, mask.to(DEV))
    for t in (cache.k, cache.v):
        for b, n in enumerate(lens):
            t[int(table[b, n // 16]), :, n % 16] = torch.full((1, d), math.nan, device=DEV).to(held)
    got = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared, None, mask.to(DEV))
    assert torch.equal(got[0][:, :, 1:], want[0][:, :, 1:]) and torch.equal(got[1][:, :, 1:], want[1][:, :, 1:])
    assert not got[0][:, :, 0].isfinite().any()


@pytest.mark.parametrize("dtype,held,d,T", WIDE)
def test_bad_pages(dtype, held, d, T):
    """Pages of a prefix and of an own part that are not there: their keys are
    left out, for all who share them, and it is said."""
    groups = [(512, [60, 70, 80])]
    q, cache, table, lens, shared, _ = make(groups, None, T, 2, 1, 16, d, dtype, held, 11)
    bad = table.clone()
    bad[:, 3], bad[1, 33] = cache.k.shape[0] + 5, -1
    got = ra.ra_cache_attention_shared(q, cache, wide(bad, cache), i32(lens), shared)
    assert ra.ra_last_device_status() == _native.RA_ERR_PAGE
    want = ra.ra_cache_attention(q, cache, bad.to(DEV), i32(lens))
    assert ra.ra_last_device_status() == _native.RA_ERR_PAGE
    torch.testing.assert_close(got[0].float(), want[0].float(), atol=2e-2, rtol=2.0 ** -6)
    torch.testing.assert_close(got[1], want[1], atol=1e-4, rtol=1e-5)
    # a table that is too short for the sequences
    got = ra.ra_cache_attention_shared(q, cache, wide(table[:, :20], cache), i32(lens), shared)
    assert ra.ra_last_device_status() == _native.RA_ERR_PAGE
    want = ra.ra_cache_attention(q, cache, table[:, :20].contiguous().to(DEV), i32(lens))
    torch.testing.assert_close(got[1], want[1], atol=1e-4, rtol=1e-5)
    # a count above T
    ra.ra_last_device_status()
    got = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared, i32([T, T + 1, T]))
    assert ra.ra_last_device_status() == _native.RA_ERR_PAGE
    check(got, q, cache, table, lens, None, None)


@pytest.mark.parametrize("dtype,held,d,T", WIDE)
def test_repeats_and_does_not_depend_on_the_workspace(dtype, held, d, T):
    groups = [(3000, [5, 700, 0, 9]), (800, [3, 9])]
    q, cache, table, lens, shared, _ = make(groups, None, T, 4, 2, 64, d, dtype, held, 12)
    n = ra.ra_cache_attention_shared_workspace_bytes(6, 4, 2, T, d)
    first = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared)
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        again = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype,held,d,T", WIDE)
def test_graph_follows_lengths_and_entries(dtype, held, d, T):
    groups = [(640, [50, 60, 70]), (0, [10]), (512, [9, 8])]
    q, cache, table, lens, shared, _ = make(groups, None, T, 2, 1, 32, d, dtype, held, 13)
    tab, ln, sh = wide(table, cache), i32(lens), shared.clone()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    ws = torch.empty(ra.ra_cache_attention_shared_workspace_bytes(6, 2, 1, T, d), dtype=torch.uint8, device=DEV)
    ra.ra_cache_attention_shared(q, cache, tab, ln, sh, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.ra_cache_attention_shared(q, cache, tab, ln, sh, out=out, lse=lse, workspace=ws)
    for cut, entries in ((0, shared.tolist()), (3, [0, 200, 640, 0, 0, 300]), (8, [0] * 6)):
        now = [n - cut for n in lens]
        ln.copy_(i32(now)), sh.copy_(i32(entries))
        out.fill_(math.nan), lse.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        check((out, lse), q, cache, table, now, None, None)


def test_a_wait_that_runs_out_is_said():
    """A tile that is never loaded, in the launch of the prefixes and in that of
    the own parts: the status, and a working context after it."""
    groups = [(1024, [200, 300, 100])]
    q, cache, table, lens, shared, _ = make(groups, None, 33, 2, 1, 64, 128, torch.bfloat16, torch.bfloat16, 14)
    try:
        ra.ra_watchdog_config(1 << 20, 0)
        ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared)
        assert ra.ra_last_device_status() == _native.RA_ERR_TIMEOUT
    finally:
        ra.ra_watchdog_config(0, -1)
    got = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared)
    assert ra.ra_last_device_status() == 0
    check(got, q, cache, table, lens, None, None)
