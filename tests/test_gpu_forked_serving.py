"""Several continuations of one context, as a program carries them: a prompt,
samples forked from it, steps of drafted trees (room, copies, norm and
rotation, write, attention over the shared prefix, verification, the kept rows
together, pages given back), the end; the same steps as one captured graph;
streams, graphs side by side, large caches, queries that are not finite."""
import math
import random

import numpy as np
import pytest
import torch

import fork_ref as F
import long_context_ra_gb300 as ra
import serve_ref as R
from long_context_ra_gb300._native import RA_ERR_PAGE
from test_gpu_cache_attention import check, tree
from test_gpu_shared_attention import make, wide

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def rnd(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, device=DEV, generator=g).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """Samples of one prompt over the caches of two layers with one table."""

    heads, Hq, d, page, V = 2, 8, 64, 16, 97

    def __init__(self, prompt, samples, held, columns):
        self.caches = [ra.new_cache(samples * 12 + prompt // self.page + 8, self.heads, self.page, self.d, held)
                       for _ in range(2)]
        for c in self.caches:
            for t in (c.k, c.v):
                t.view(torch.uint8).zero_()
            if c.k_exp is not None:
                c.k_exp.zero_(), c.v_exp.zero_()
        self.ref = torch.zeros(self.caches[0].k.shape[0], dtype=torch.int32, device=DEV)
        table = torch.full((1, columns), -1, dtype=torch.int32, device=DEV)
        held0, lens = i32([0]), i32([0])
        granted, src, dst = ra.ra_pages_reserve(self.ref, table, held0, lens, self.page, prompt)
        assert granted.tolist() == [prompt] and src.tolist() == dst.tolist() == [-1]
        self.rows = []
        for i, c in enumerate(self.caches):
            kv = rnd(20 + i, 2, 1, self.heads, prompt, self.d, dtype=BF16)
            ra.ra_cache_write(c, kv[0], kv[1], table, lens)
            self.rows.append(kv)
        lens += prompt
        out = ra.ra_pages_fork(self.ref, table, held0, lens, i32([0] * samples), self.page)
        ra.ra_pages_trim(self.ref, table, held0, None, self.page)
        self.table, self.held, self.lens = out
        self.shared = i32([0] + [prompt] * (samples - 1))
        self.rope = ra.new_rope([10000.0 ** (-2 * i / self.d) for i in range(self.d // 2)])
        self.head = rnd(30, self.Hq * self.d, self.V) * 0.2

    def step(self, x, tokens, uniform, parent, mask, depth):
        """x [layers, B, T, Hq + 2 heads, d]: the projections of the drafts."""
        T = tokens.shape[1]
        granted, src, dst = ra.ra_pages_reserve(self.ref, self.table, self.held, self.lens, self.page, T)
        pos = self.lens[:, None].long() + depth
        outs = []
        for c, y in zip(self.caches, x):
            ra.ra_cache_copy(c, src, dst)
            y = y.transpose(1, 2)
            q, k = ra.ra_qk_norm_rope(y[:, :self.Hq], y[:, self.Hq:self.Hq + self.heads], self.rope, pos)
            ra.ra_cache_write(c, k, y[:, self.Hq + self.heads:], self.table, self.lens, granted)
            out, lse = ra.ra_cache_attention_shared(q, c, self.table, self.lens, self.shared, granted, mask)
            outs.append((q, k, out, lse))
        probs = torch.softmax(outs[-1][2].transpose(1, 2).flatten(2).float() @ self.head, -1)
        path, kept, token = ra.ra_verify_drafts(probs, tokens, uniform, parent, count=granted)
        for c in self.caches:
            ra.ra_cache_compact(c, self.table, self.lens, path, kept)
        self.lens += kept
        ra.ra_pages_trim(self.ref, self.table, self.held, self.lens, self.page)
        return outs, probs, path, kept, token


def drafts(server, B, T, seed):
    r = np.random.RandomState(seed)
    parent = np.full((B, T), -1, dtype=np.int32)
    mask, depth = torch.zeros(B, T, T, dtype=torch.bool), torch.zeros(B, T, dtype=torch.int64)
    for b in range(B):
        for t in range(T):
            if t:
                parent[b, t] = r.randint(max(0, t - 3), t)
                mask[b, t] = mask[b, parent[b, t]]
                depth[b, t] = depth[b, parent[b, t]] + 1
            mask[b, t, t] = True
    x = rnd(seed, 2, B, T, server.Hq + 2 * server.heads, server.d, dtype=BF16)
    tokens = torch.from_numpy(r.randint(0, server.V, (B, T))).to(DEV)
    # small numbers accept: half of the drafts or so stay
    u = (torch.rand(B, T, generator=torch.Generator().manual_seed(seed)) ** 6).to(DEV)
    return x, tokens, u, torch.from_numpy(parent).to(DEV), mask.to(DEV), depth.to(DEV)


def read(server, layer, dtype):
    n = int(server.lens.max())
    return ra.ra_cache_read(server.caches[layer], server.table, server.lens, 0, n, dtype=dtype)


@pytest.mark.parametrize("held", [BF16, E4M3])
@pytest.mark.parametrize("columns", [64, 6000])   # prefixes are read by each, or once for all
def test_steps_of_samples(held, columns):
    B, T, prompt = 6, 9, 300
    s = Server(prompt, B, held, columns)
    first = s.ref.clone()
    assert int(first.sum()) == B * F.up(prompt, s.page)
    want = [[[kv[side][0].repeat(1, 1, 1) for side in range(2)] for _ in range(B)] for kv in s.rows]  # [heads, n, d]
    for i in range(6):
        args = drafts(s, B, T, 100 + i)
        lens = s.lens.tolist()
        table0, before = s.table.clone(), None
        outs, probs, path, kept, token = s.step(*args)
        assert ra.ra_last_device_status() == 0
        u, tok, par = args[2], args[1], args[3]
        for b in range(B):
            w = F.verify(probs[b].double().cpu().numpy(), None, tok[b].cpu().numpy(), par[b].tolist(), T,
                         u[b].double().cpu().numpy())
            if w[2] > 2.0 ** -40:
                assert (path[b, :int(kept[b])].tolist(), int(token[b])) == (w[0], w[1])
        for layer, (q, k, out, lse) in enumerate(outs):
            v = args[0][layer].transpose(1, 2)[:, s.Hq + s.heads:]
            for b in range(B):
                nodes = path[b, :int(kept[b])].long()
                for side, new in enumerate((k, v)):
                    want[layer][b][side] = torch.cat([want[layer][b][side], new[b][:, nodes]], 1)
            got = read(s, layer, BF16)
            for b in range(B):
                n = int(s.lens[b])
                assert n == want[layer][b][0].shape[1]
                for side in range(2):
                    x, y = got[side][b, :, :n], want[layer][b][side]
                    if held == E4M3:  # a row is off by half a step of 8 bits, or of the smallest one
                        top = y.float().abs().amax(-1, keepdim=True)
                        assert ((x.float() - y.float()).abs() <= y.float().abs() * 2.0 ** -4 + top * 2.0 ** -17).all()
                    else:
                        assert torch.equal(x, y)
            # the step's attention, in 64 bits over what the cache held then
            if i == 5 and layer == 1 and held == BF16:
                for b in (0, 3):
                    n = lens[b]
                    kk = torch.cat([want[1][b][0][:, :n], k[b]], 1)
                    vv = torch.cat([want[1][b][1][:, :n], v[b]], 1)
                    seen = torch.cat([torch.ones(T, n, dtype=torch.bool, device=DEV), args[4][b]], 1)
                    qq = q[b].double().view(s.heads, s.Hq // s.heads, T, s.d)
                    sc = torch.einsum("hgtd,hnd->hgtn", qq, kk.double()) / math.sqrt(s.d)
                    p = torch.softmax(sc.masked_fill(~seen, -math.inf), -1)
                    o = torch.einsum("hgtn,hnd->hgtd", p, vv.double()).reshape(s.Hq, T, s.d)
                    mag = torch.einsum("hgtn,hnd->hgtd", p, vv.double().abs()).reshape(s.Hq, T, s.d)
                    tol = 2.0 ** -8 * o.abs() + mag * (2.0 ** -8 + 2.0 ** -12)
                    assert ((out[b].double() - o).abs() <= tol).all()
        # nobody holds more than it needs, and every page that is held is counted
        assert s.held.tolist() == [F.up(n, s.page) for n in s.lens.tolist()]
        count = torch.zeros_like(s.ref)
        for row, h in zip(s.table.tolist(), s.held.tolist()):
            for p in row[:h]:
                count[p] += 1
            assert row[h:] == [-1] * (columns - h)
        assert torch.equal(count, s.ref)
    ra.ra_pages_trim(s.ref, s.table, s.held, None, s.page)
    assert not s.ref.any() and ra.ra_last_device_status() == 0


@pytest.mark.parametrize("held", [BF16, E4M3])
@pytest.mark.parametrize("columns", [64, 6000])
def test_a_captured_step(held, columns):
    """The step as one graph, replayed while the samples grow at unlike pace,
    against the same steps without a graph: equal bits everywhere."""
    B, T, prompt = 5, 8, 270
    servers = [Server(prompt, B, held, columns) for _ in range(2)]
    args = [t.clone() for t in drafts(servers[0], B, T, 1)]
    warm = Server(prompt, B, held, columns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm.step(*args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = servers[0].step(*args)
    for i in range(5):
        for t, new in zip(args, drafts(servers[0], B, T, 200 + i)):
            t.copy_(new)
        graph.replay()
        want = servers[1].step(*args)
        torch.cuda.synchronize()
        for a, b in zip(res[1:], want[1:]):
            assert torch.equal(a, b)
        for x, y in zip(res[0], want[0]):
            assert all(torch.equal(a, b) for a, b in zip(x, y))
        for a, b in zip(servers[0].caches, servers[1].caches):
            assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8))
            assert torch.equal(a.v.view(torch.uint8), b.v.view(torch.uint8))
        for name in ("ref", "table", "held", "lens"):
            assert torch.equal(getattr(servers[0], name), getattr(servers[1], name)), name
    assert ra.ra_last_device_status() == 0


def test_a_beam_search_step():
    """Beams that go on, some twice, others not at all: a fork into a second
    table, a release of the first, and copies where two write into one page."""
    page, width = 8, 6
    m = F.Pages(60, width, page)
    rows = [([-1] * width, 0, 0)]
    m.reserve(rows, 19)
    rows = [(rows[0][0], rows[0][1], 19)]
    rows, old = m.fork(rows, [0] * 4), rows
    m.trim(old)
    cache = ra.new_cache(60, 1, page, 8, torch.float32)
    cache.k.copy_(torch.arange(60 * page, device=DEV).view(60, 1, page, 1).expand_as(cache.k).float())
    cache.v.copy_(-cache.k)
    ref, lens = i32(m.ref), i32([19] * 4)
    table, held = i32([r[0] for r in rows]), i32([r[1] for r in rows])
    r = random.Random(3)
    for _ in range(8):
        source = [r.randrange(4) for _ in range(4)]
        new = m.fork(rows, source)
        m.trim(rows)
        want = m.reserve(new, 1)
        t, h, n = ra.ra_pages_fork(ref, table, held, lens, i32(source), page)
        ra.ra_pages_trim(ref, table, held, None, page)
        got = ra.ra_pages_reserve(ref, t, h, n, page, 1)
        keys = cache.k.clone()
        ra.ra_cache_copy(cache, got[1], got[2])
        assert [x.tolist() for x in got] == [list(x) for x in want]
        for a, z in zip(want[1], want[2]):
            if a >= 0:
                keys[z] = keys[a]
        assert torch.equal(cache.k, keys) and torch.equal(cache.v, -keys)
        rows = [(a, b, c + g) for (a, b, c), g in zip(new, want[0])]
        n += got[0]
        table, held, lens = t, h, n
        assert ref.tolist() == m.ref and table.tolist() == [list(x[0]) for x in rows]
        if sum(want[0]) == 0:
            break
    assert not m.bad or ra.ra_last_device_status()


@pytest.mark.parametrize("pages", [60, 16, 8, 7])
def test_beams_say_when_pages_run_out(pages):
    """The status of every step is that of a model: a page error in the step that
    finds too few free pages, nothing in the others."""
    page, width, n = 8, 6, 4
    m = F.Pages(pages, width, page)
    rows = [([-1] * width, 0, 0)]
    m.reserve(rows, 19)
    rows = [(rows[0][0], rows[0][1], 19)]
    rows, old = m.fork(rows, [0] * n), rows
    m.trim(old)
    ref, lens = i32(m.ref), i32([19] * n)
    table, held = i32([r[0] for r in rows]), i32([r[1] for r in rows])
    r, said = random.Random(pages), []
    assert ra.ra_last_device_status() == 0
    for _ in range(12):
        source, m.bad = [r.randrange(n) for _ in range(n)], False
        new = m.fork(rows, source)
        m.trim(rows)
        want = m.reserve(new, 1)
        t, h, ln = ra.ra_pages_fork(ref, table, held, lens, i32(source), page)
        ra.ra_pages_trim(ref, table, held, None, page)
        got = ra.ra_pages_reserve(ref, t, h, ln, page, 1)
        said.append(ra.ra_last_device_status())
        assert (said[-1] == RA_ERR_PAGE) == m.bad and said[-1] in (0, RA_ERR_PAGE)
        assert [x.tolist() for x in got] == [list(x) for x in want]
        rows = [(a, b, c + g) for (a, b, c), g in zip(new, want[0])]
        ln += got[0]
        table, held, lens = t, h, ln
        assert ref.tolist() == m.ref and table.tolist() == [list(x[0]) for x in rows]
    assert (RA_ERR_PAGE in said) == (pages <= 8)


# --------------------------------------------------------- graphs and streams
CASES = [(BF16, BF16, 64, 1), (BF16, BF16, 128, 12), (BF16, BF16, 128, 40), (BF16, E4M3, 128, 1), (torch.float32, torch.float32, 80, 1)]


@pytest.mark.parametrize("dtype,held,d,T", CASES)
def test_the_next_kernel_sees_the_whole_result(dtype, held, d, T):
    """Launches of a call begin before those ahead of them have ended; what
    follows on the stream comes after all of them."""
    q, cache, table, lens, shared, _ = make([(640, [50] * 19), (0, [700] * 3)], None, T, 8, 2, 64, d, dtype, held, 3)
    tab, ln = wide(table, cache), i32(lens)
    out, lse = ra.ra_cache_attention_shared(q, cache, tab, ln, shared)
    torch.cuda.synchronize()
    assert out.abs().amax(-1).min() > 0
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(ra.ra_cache_attention_shared_workspace_bytes(22, 8, 2, T, d), device=DEV, dtype=torch.uint8)
    copies = []
    for _ in range(20):
        out2.zero_()
        lse2.zero_()
        ws.fill_(255)
        ra.ra_cache_attention_shared(q, cache, tab, ln, shared, out=out2, lse=lse2, workspace=ws)
        copies.append((out2.clone(), lse2.clone()))
    for o, s in copies:
        assert torch.equal(o, out) and torch.equal(s, lse)


@pytest.mark.parametrize("dtype,held,d,T", CASES)
def test_two_graphs_run_side_by_side(dtype, held, d, T):
    q, cache, table, lens, shared, _ = make([(900, [50, 60, 70, 5, 0])], None, T, 8, 2, 64, d, dtype, held, 4)
    tab, ln = wide(table, cache), i32(lens)
    n = ra.ra_cache_attention_shared_workspace_bytes(5, 8, 2, T, d)
    runs = []
    for i in range(2):
        x = rnd(30 + i, *q.shape, dtype=dtype)
        want = ra.ra_cache_attention_shared(x, cache, tab, ln, shared)
        out, lse, ws = torch.empty_like(want[0]), torch.empty_like(want[1]), torch.empty(n, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ra.ra_cache_attention_shared(x, cache, tab, ln, shared, out=out, lse=lse, workspace=ws)
        runs.append((graph, torch.cuda.Stream(), want, out, lse, x, ws))
    for _ in range(10):
        for graph, s, *_ in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, want, out, lse, *_ in runs:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_calls_on_a_given_stream():
    """stream=: work and the calls' own allocations belong to that stream."""
    q, cache, table, lens, shared, _ = make([(300, [5, 9, 40])], None, 4, 4, 2, 16, 64, BF16, BF16, 5)
    tab, ln = wide(table, cache), i32(lens)
    probs = torch.softmax(rnd(6, 3, 4, 1001), -1)
    tokens, u = torch.randint(0, 1001, (3, 4), device=DEV), torch.rand(3, 4, device=DEV)
    ref = torch.zeros(cache.k.shape[0], dtype=torch.int32, device=DEV)
    short, held = torch.full((3, 4), -1, dtype=torch.int32, device=DEV), i32([0] * 3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [ra.ra_cache_attention_shared(q, cache, tab, ln, shared, stream=s) for _ in range(3)]
    seen = [ra.ra_verify_drafts(probs, tokens, u, stream=s) for _ in range(3)]
    zero, source, src, dst, path0 = i32([0] * 3), i32([2, 0]), i32([1]), i32([0]), i32([[0, 2, -1, -1]] * 3)
    torch.cuda.synchronize()
    got = ra.ra_pages_reserve(ref, short, held, zero, 16, 20, stream=s)
    forks = ra.ra_pages_fork(ref, short, held, zero, source, 16, stream=s)
    copied = cache.k.clone(), cache.v.clone()
    torch.cuda.synchronize()
    ra.ra_cache_copy(cache, src, dst, stream=s)
    ra.ra_cache_compact(cache, tab, ln, path0, zero, stream=s)
    ra.ra_pages_trim(ref, short, held, None, 16, stream=s)
    s.synchronize()
    assert got[0].tolist() == [20] * 3 and not ref.any() and forks[2].tolist() == [0, 0]
    assert torch.equal(cache.k[0].view(torch.uint8), copied[0][1].view(torch.uint8))
    cache.k.copy_(copied[0]), cache.v.copy_(copied[1])
    want, path = ra.ra_cache_attention_shared(q, cache, tab, ln, shared), ra.ra_verify_drafts(probs, tokens, u)
    assert all(torch.equal(o, want[0]) and torch.equal(z, want[1]) for o, z in outs)
    assert all(torch.equal(x, y) for r in seen for x, y in zip(r, path))


# ----------------------------------------------------- values and large caches
@pytest.mark.parametrize("dtype,held,d,T", CASES)
def test_queries_that_are_not_finite_stay_in_their_rows(dtype, held, d, T):
    """Rows of several sequences share a tile: a NaN or an infinity in one
    query reaches no other row's bits."""
    q, cache, table, lens, shared, _ = make([(640, [5, 70, 0, 9])], None, T, 6, 2, 32, d, dtype, held, 6)
    tab, ln = wide(table, cache), i32(lens)
    bad = q.clone()
    bad[0, 2, T - 1, 5] = math.nan
    bad[0, 3, 0, 7] = math.inf
    bad[2, 5] = math.nan
    want = ra.ra_cache_attention_shared(q, cache, tab, ln, shared)
    got = ra.ra_cache_attention_shared(bad, cache, tab, ln, shared)
    same = torch.ones(q.shape[:3], dtype=torch.bool, device=DEV)
    same[0, 2, T - 1] = same[0, 3, 0] = False
    same[2, 5] = False
    assert torch.equal(got[0][same], want[0][same]) and torch.equal(got[1][same], want[1][same])
    assert got[0][~same].isnan().any(-1).all()


@pytest.mark.parametrize("dtype,held,d,T", CASES)
def test_growing_scores_and_unlike_scales(dtype, held, d, T):
    """Scores that rise along the keys by some hundred, so that references move
    from tile to tile and between prefix and rest; values of 2^-20 .. 2^20."""
    lens_own = [40, 0, 130]
    q, cache, table, lens, shared, _ = make([(1500, lens_own)], None, T, 4, 2, 64, d, dtype, held, 7)
    n = max(lens) + T
    g = torch.Generator(device=DEV).manual_seed(9)
    one = q.float()[:1].expand(3, -1, -1, -1)
    k = torch.randn(1, 2, n, d, device=DEV, generator=g).repeat(3, 1, 1, 1)
    k += one.reshape(3, 2, -1, d).mean(2)[:, :, None] * torch.linspace(0, 25, n, device=DEV)[None, None, :, None]
    v = torch.randn(1, 2, n, d, device=DEV, generator=g).repeat(3, 1, 1, 1)
    v *= torch.exp2(40 * torch.rand(1, 1, n, 1, device=DEV, generator=g) - 20)
    ra.ra_cache_write(cache, k.to(dtype), v.to(dtype), table.to(DEV), i32([0] * 3), i32([x + T for x in lens]))
    got = ra.ra_cache_attention_shared(q, cache, wide(table, cache), i32(lens), shared)
    check(got, q, cache, table, lens, None, None)


@pytest.mark.parametrize("held,T", [(BF16, 1), (BF16, 12), (E4M3, 12)])
def test_rows_behind_two_to_the_32_bytes(held, T):
    """A cache of over 2^32 bytes a side, the sequences in its last pages."""
    heads, d, page = 8, 128, 128
    q, small, table, lens, shared, _ = make([(640, [5, 200, 0])], None, T, 16, heads, page, d, BF16, held, 8)
    used = small.k.shape[0]
    pages = (1 << 32) // (heads * page * d * (2 if held == BF16 else 1)) + used
    large = ra.new_cache(pages, heads, page, d, held)
    for a, b in ((small.k, large.k), (small.v, large.v), (small.k_exp, large.k_exp), (small.v_exp, large.v_exp)):
        if a is not None:
            b[-used:] = a
    last = torch.where(table >= 0, table + pages - used, table)
    res = [ra.ra_cache_attention_shared(q, c, wide(t, c), i32(lens), shared) for c, t in ((small, table), (large, last))]
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert ra.ra_last_device_status() == 0
