"""The calls around the attention together, as a program uses them: the norm
and rotation before the differentiable attention; decode steps and drafted
trees over a cache; a context read back for ra_fold; caches of a sequence's
parts merged by ra_merge; captured and replayed steps; other streams; a cache
beyond 2^32 bytes; a stalled CTA."""
import math
import time

import pytest
import torch

import long_context_ra_gb300 as ra
import serve_ref as R
from gpu_util import check_same
from long_context_ra_gb300 import _native
from long_context_ra_gb300.autograd import attention, qk_norm_rope

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn
BF16 = torch.bfloat16


def rnd(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, device=DEV, generator=g).to(dtype)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rope_of(d, base=10000.0, **kw):
    return ra.new_rope([base ** (-2 * i / d) for i in range(d // 2)], **kw)


# ------------------------------------------------------------- training chain
def plain_chain(q, k, v, wq, wk, pos, inv, eps=1e-6):
    """The chain in torch operations on 64-bit tensors, differentiable."""
    ang = pos.double()[..., None] * torch.tensor(inv, dtype=torch.float64, device=pos.device)
    c, s = ang.cos()[:, None], ang.sin()[:, None]

    def one(x, w):
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w
        a, b = x.chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k = one(q, wq), one(k, wk)
    return torch.softmax(q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1]), -1) @ v


def test_norm_rope_before_attention_trains():
    """Gradients of projection views and weights through qk_norm_rope and
    attention, fp32, against torch's autograd of the same chain in 64 bits.
    The fp32 path's relative error is about 1e-6 per stage; 1e-4 of the largest
    gradient leaves room for the softmax's sums."""
    B, N, H, d = 1, 96, 3, 40
    inv = [10000.0 ** (-2 * i / d) for i in range(d // 2)]
    rope = ra.new_rope(inv)
    pos = torch.arange(N, device=DEV)[None] + 1000
    proj = rnd(1, B, N, 3 * H, d).requires_grad_()
    wq, wk = ((1 + 0.2 * rnd(2 + i, d)).requires_grad_() for i in range(2))
    q, k, v = (proj[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    up = rnd(5, B, H, N, d)
    qn, kn = qk_norm_rope(q, k, rope, pos, wq, wk)
    out, _ = attention(qn, kn, v, P=3)
    (out * up).sum().backward()
    proj64, wq64, wk64 = (t.detach().double().requires_grad_() for t in (proj, wq, wk))
    q, k, v = (proj64[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    (plain_chain(q, k, v, wq64, wk64, pos, inv) * up.double()).sum().backward()
    for got, want in ((proj.grad, proj64.grad), (wq.grad, wq64.grad), (wk.grad, wk64.grad)):
        assert (got.double() - want).abs().max() <= 1e-4 * want.abs().max()


def test_norm_rope_gradients_are_the_library_backward():
    shape = (2, 4, 129, 128)
    q, k = (rnd(10 + i, *shape, dtype=BF16).requires_grad_() for i in range(2))
    w = (1 + 0.1 * rnd(12, 128)).to(BF16).requires_grad_()
    rope, pos = rope_of(128), torch.arange(129, device=DEV).expand(2, 129).contiguous()
    ups = [rnd(13 + i, *shape, dtype=BF16) for i in range(2)]
    a, b = qk_norm_rope(q, k, rope, pos, w, w)     # one weight for both sides
    torch.autograd.backward([a, b], ups)
    dq, dk, dwq, dwk = ra.ra_qk_norm_rope_backward(q.detach(), k.detach(), *ups, rope, pos, w.detach(),
                                                   w.detach())
    assert torch.equal(q.grad, dq) and torch.equal(k.grad, dk)
    assert torch.equal(w.grad, dwq.to(BF16) + dwk.to(BF16))
    with pytest.raises(RuntimeError):               # no second derivative
        a, _ = qk_norm_rope(q, k, rope, pos, w, w)
        g, = torch.autograd.grad(a.float().sum(), q, create_graph=True)
        g.float().sum().backward()


# ------------------------------------------------------------------- decoding
@pytest.mark.parametrize("held", [BF16, E4M3])
@pytest.mark.parametrize("g", [1, 5])
def test_decode_steps(held, g):
    """A prompt and then single tokens of two sequences: norm and rotation,
    write, attention, each step against the 64-bit attention over the cache."""
    heads, d, page, prompt, steps = 2, 128, 16, 45, 4
    B, Hq = 2, heads * g
    table, pages = R.make_paged([prompt + steps] * B, page, 1)
    tab = table.to(DEV)
    cache = ra.new_cache(pages, heads, page, d, held)
    rope, w = rope_of(d), (1 + 0.1 * rnd(2, d)).to(BF16)
    lens = i32(0, 0)
    for step in range(steps + 1):
        T = prompt if step == 0 else 1
        x = rnd(100 + step, B, T, Hq + 2 * heads, d, dtype=BF16).transpose(1, 2)
        pos = (lens[:, None] + torch.arange(T, device=DEV)).long()
        q, k = ra.ra_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + heads], rope, pos, w, w)
        ra.ra_cache_write(cache, k, x[:, Hq + heads:], tab, lens)
        out, lse = ra.ra_cache_attention(q, cache, tab, lens)
        n = lens.tolist()
        want, wl, mag, size = R.attention(q, R.PagedCpu(cache, table), n, None, None)
        tol = 2.0 ** -8 * want.abs() + mag * (2.0 ** -8 + 2 * 136 * R.U * size + 2.0 ** -18)[..., None]
        assert ((out.cpu().double() - want).abs() <= tol).all()
        assert (lse.cpu().double() - wl).abs().max() <= 1e-4
        lens += T
    assert ra.ra_last_device_status() == 0


def test_accepted_path_of_a_tree_continues_the_sequence():
    """Drafted tokens attend along their path: a chain's queries equal those of
    the same tokens decoded one by one."""
    heads, Hq, d, page, L = 2, 8, 128, 32, 70
    parent = [-1, 0, 0, 1, 3, 2]                     # nodes 0, 1, 3, 4 are a path
    T = len(parent)
    mask = torch.zeros(T, T, dtype=torch.bool)
    for i, p in enumerate(parent):
        if p >= 0:
            mask[i] = mask[p]
        mask[i, i] = True
    table, pages = R.make_paged([L + T], page, 3)
    tab = table.to(DEV)
    q = rnd(1, 1, Hq, T, d, dtype=BF16)
    kv = rnd(2, 2, 1, heads, L + T, d, dtype=BF16)
    cache = ra.new_cache(pages, heads, page, d, E4M3)
    ra.ra_cache_write(cache, kv[0], kv[1], tab, i32(0))
    out, lse = ra.ra_cache_attention(q, cache, tab, i32(L), None, mask.to(DEV))
    one = ra.new_cache(pages, heads, page, d, E4M3)
    ra.ra_cache_write(one, kv[0][:, :, :L], kv[1][:, :, :L], tab, i32(0))
    for at, node in enumerate((0, 1, 3, 4)):
        ra.ra_cache_write(one, kv[0][:, :, L + node:L + node + 1], kv[1][:, :, L + node:L + node + 1], tab,
                          i32(L + at))
        o, s = ra.ra_cache_attention(q[:, :, node:node + 1].contiguous(), one, tab, i32(L + at))
        check_same(o[:, :, 0], out[:, :, node], BF16, "tree path", 2e-2)
        check_same(s[:, :, 0], lse[:, :, node], torch.float32, "tree path lse", 1e-4, relative=False)


# ------------------------------------------- with the fold and the merge
@pytest.mark.parametrize("held", [BF16, E4M3])
def test_context_read_back_folds_to_the_same(held):
    """Blocks read back from the cache, folded into a state in the ring's
    manner, give the attention over the cache."""
    heads, d, page, L, T = 2, 128, 64, 512, 128
    table, pages = R.make_paged([L], page, 5)
    tab = table.to(DEV)
    cache = ra.new_cache(pages, heads, page, d, held)
    k, v = (rnd(20 + i, 1, heads, L, d, dtype=BF16) for i in range(2))
    ra.ra_cache_write(cache, k, v, tab, i32(0))
    q = rnd(22, 1, heads, T, d, dtype=BF16)
    st = ra.ra_state_init(ra.new_state(heads * T, d))
    for first in range(0, L, 128):
        kb, vb = ra.ra_cache_read(cache, tab, i32(L), first, 128)
        ra.ra_fold(st, q.reshape(heads, T, d), kb.reshape(heads, 128, d), vb.reshape(heads, 128, d), batch=heads)
    out, lse = ra.ra_merge([st])
    # all T queries see the L context keys only: drafts that see nothing of one another
    none = torch.zeros(T, T, dtype=torch.bool, device=DEV)
    wide, npages = R.make_paged([L + T], page, 5)
    wide[0, : L // page] = table[0, : L // page]
    wide[0, L // page:] = wide[0, L // page - 1]     # the drafts' rows are not looked at: seen by none
    got, gl = ra.ra_cache_attention(q, cache, wide.to(DEV), i32(L), None, none)
    check_same(got.reshape(-1, d), out, BF16, "cache attention vs folds", 2e-2)
    check_same(gl.reshape(-1), lse, torch.float32, "lse", 1e-4, relative=False)


def test_caches_of_two_parts_merge_to_the_whole():
    """out and lse are a state (m = lse, l = 1, o = out): the context kept in
    two caches (as two ranks would) merges to that of one."""
    heads, Hq, d, page, L = 2, 6, 64, 16, 400
    q = rnd(1, 1, Hq, 1, d, dtype=BF16)
    kv = rnd(2, 2, 1, heads, L + 1, d, dtype=BF16)
    whole, states = None, []
    for a, b in ((0, L + 1), (0, 250), (250, L + 1)):
        table, pages = R.make_paged([b - a], page, a)
        cache = ra.new_cache(pages, heads, page, d)
        ra.ra_cache_write(cache, kv[0][:, :, a:b], kv[1][:, :, a:b], table.to(DEV), i32(0))
        out, lse = ra.ra_cache_attention(q, cache, table.to(DEV), i32(b - a - 1))
        if whole is None:
            whole = (out, lse)
        else:
            states.append(ra.RaState(lse.reshape(-1).clone(), torch.ones(Hq, device=DEV),
                                     out.float().reshape(Hq, d)))
    out, lse = ra.ra_merge(states)
    check_same(out, whole[0].reshape(Hq, d), BF16, "merged parts", 2e-2)
    check_same(lse, whole[1].reshape(-1), torch.float32, "merged lse", 1e-4, relative=False)


# --------------------------------------------------------- graphs and streams
def test_captured_decode_step_follows_lengths_and_contents():
    """One graph of a whole decode step, replayed while the sequences grow;
    each replay equals the eager calls bit for bit.  A second graph with a
    workspace of its own runs beside it."""
    heads, Hq, d, page, B, most = 2, 8, 128, 16, 3, 400
    table, pages = R.make_paged([most] * B, page, 7)
    tab = table.to(DEV)
    caches = [ra.new_cache(pages, heads, page, d, E4M3) for _ in range(2)]
    for c in caches:
        c.k.view(torch.uint8).zero_(), c.v.view(torch.uint8).zero_(), c.k_exp.zero_(), c.v_exp.zero_()
    rope = rope_of(d)
    x = rnd(1, B, Hq + 2 * heads, 1, d, dtype=BF16)
    lens = i32(0, 100, 250)
    pos = torch.zeros(B, 1, dtype=torch.int64, device=DEV)
    q, k = torch.empty(B, Hq, 1, d, dtype=BF16, device=DEV), torch.empty(B, heads, 1, d, dtype=BF16, device=DEV)
    n = ra.ra_cache_attention_workspace_bytes(B, Hq, heads, 1, d)
    bufs = [(torch.empty_like(q), torch.empty(B, Hq, 1, device=DEV),
             torch.empty(n, dtype=torch.uint8, device=DEV)) for _ in range(2)]

    def step(c, b):
        pos.copy_(lens[:, None])
        ra.ra_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + heads], rope, pos, q_out=q, k_out=k)
        ra.ra_cache_write(c, k, x[:, Hq + heads:], tab, lens)
        ra.ra_cache_attention(q, c, tab, lens, out=b[0], lse=b[1], workspace=b[2])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(caches[0], bufs[0])
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for b in (bufs[0],):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(caches[0], b)
        graphs.append(gr)
    for i in range(4):
        x.copy_(rnd(50 + i, *x.shape, dtype=BF16))
        graphs[0].replay()
        got = [t.clone() for t in bufs[0][:2]]
        step(caches[1], bufs[1])
        torch.cuda.synchronize()
        assert torch.equal(got[0], bufs[1][0]) and torch.equal(got[1], bufs[1][1])
        lens += 1
    for a, b in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert ra.ra_last_device_status() == 0


@pytest.mark.parametrize("T", [1, 40])
def test_two_captured_graphs_run_side_by_side(T):
    """Two graphs of attention calls on two streams at once, each with its own
    workspace, against the eager results."""
    heads, Hq, d, page, L = 2, 8, 128, 64, 3000
    table, pages = R.make_paged([L + T], page, 9)
    tab, lens = table.to(DEV), i32(L)
    cache = ra.new_cache(pages, heads, page, d)
    ra.ra_cache_write(cache, *rnd(1, 2, 1, heads, L + T, d, dtype=BF16), tab, i32(0))
    n = ra.ra_cache_attention_workspace_bytes(1, Hq, heads, T, d)
    runs = []
    for i in range(2):
        q = rnd(30 + i, 1, Hq, T, d, dtype=BF16)
        want = ra.ra_cache_attention(q, cache, tab, lens)
        out, lse, ws = (torch.empty_like(want[0]), torch.empty_like(want[1]),
                        torch.empty(n, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ra.ra_cache_attention(q, cache, tab, lens, out=out, lse=lse, workspace=ws)
        runs.append((gr, torch.cuda.Stream(), want, out, lse, q, ws))
    for _ in range(10):
        for gr, s, *_ in runs:
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for _, _, want, out, lse, *_ in runs:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype,held,B,T", [(BF16, BF16, 38, 1), (BF16, E4M3, 38, 1), (BF16, BF16, 19, 20),
                                            (BF16, E4M3, 19, 40), (torch.float32, torch.float32, 76, 1)])
def test_the_next_kernel_sees_the_whole_result(dtype, held, B, T):
    """Equal lengths and as many units as CTAs: no unit is shared, so nothing
    is joined, and what follows on the stream still comes after every CTA."""
    heads, page, n = 8, 64, 1500
    per = -(-(n + T) // page)
    cache = ra.new_cache(B * per, heads, page, 64, held)
    table = torch.arange(B * per, dtype=torch.int32, device=DEV).reshape(B, per)
    x = rnd(3, 2, B, heads, n + T, 64, dtype=dtype)
    ra.ra_cache_write(cache, x[0], x[1], table, i32(*[0] * B))
    q = rnd(4, B, heads * (4 if T > 1 else 1), T, 64, dtype=dtype)
    lens = i32(*[n] * B)
    out, lse = ra.ra_cache_attention(q, cache, table, lens)
    torch.cuda.synchronize()
    assert out.abs().amax(-1).min() > 0
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(ra.ra_cache_attention_workspace_bytes(B, q.shape[1], heads, T, 64), device=DEV,
                     dtype=torch.uint8)
    copies = []
    for _ in range(20):
        out2.zero_()
        lse2.zero_()
        ra.ra_cache_attention(q, cache, table, lens, out=out2, lse=lse2, workspace=ws)
        copies.append((out2.clone(), lse2.clone()))
    for o, s in copies:
        assert torch.equal(o, out) and torch.equal(s, lse)


@pytest.mark.parametrize("dtype,held", [(BF16, BF16), (BF16, E4M3), (torch.float32, torch.float32)])
@pytest.mark.parametrize("T", [1, 9, 40, 100])
def test_queries_that_are_not_finite_stay_in_their_rows(dtype, held, T):
    """Kernels work on rows of several tokens and heads together; a NaN or an
    infinity in one query reaches no other row's bits."""
    B, heads, g, d, page = 2, 2, 3, 64, 32
    n = 200 + T
    per = -(-n // page)
    cache = ra.new_cache(B * per, heads, page, d, held)
    table = torch.arange(B * per, dtype=torch.int32, device=DEV).reshape(B, per)
    x = rnd(7, 2, B, heads, n, d, dtype=dtype)
    ra.ra_cache_write(cache, x[0], x[1], table, i32(0, 0))
    q = rnd(8, B, heads * g, T, d, dtype=dtype)
    bad = q.clone()
    bad[0, 2, T - 1, 5] = math.nan
    bad[0, 3, 0, 7] = math.inf
    bad[1, 5] = math.nan
    want = ra.ra_cache_attention(q, cache, table, i32(200, 77))
    got = ra.ra_cache_attention(bad, cache, table, i32(200, 77))
    same = torch.ones(B, heads * g, T, dtype=torch.bool, device=DEV)
    same[0, 2, T - 1] = same[0, 3, 0] = False
    same[1, 5] = False
    assert torch.equal(got[0][same], want[0][same]) and torch.equal(got[1][same], want[1][same])
    assert got[0][~same].isnan().any(-1).all()


def test_calls_on_a_given_stream():
    """stream=: work and the call's own allocations belong to that stream."""
    heads, Hq, d, page, L, T = 2, 8, 64, 32, 700, 20
    table, pages = R.make_paged([L + T], page, 11)
    tab, zero, lens = table.to(DEV), i32(0), i32(L)
    cache = ra.new_cache(pages, heads, page, d, E4M3)
    kv = rnd(1, 2, 1, heads, L + T, d, dtype=BF16)
    q = rnd(2, 1, Hq, T, d, dtype=BF16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ra.ra_cache_write(cache, kv[0], kv[1], tab, zero, stream=s)
    outs = [ra.ra_cache_attention(q, cache, tab, lens, stream=s) for _ in range(5)]
    back = ra.ra_cache_read(cache, tab, lens, 0, L, stream=s)
    s.synchronize()
    want = ra.ra_cache_attention(q, cache, tab, lens)
    assert all(torch.equal(o, want[0]) and torch.equal(z, want[1]) for o, z in outs)
    assert torch.equal(back[0], ra.ra_cache_read(cache, tab, lens, 0, L)[0])


# ---------------------------------------------------------------- large caches
@pytest.mark.parametrize("held", [BF16, E4M3])
@pytest.mark.parametrize("T", [1, 40])
def test_rows_behind_two_to_the_32_bytes(held, T):
    """A cache of over 2^32 bytes a side, a sequence in its last pages."""
    heads, Hq, d, page, L = 8, 16, 128, 128, 600
    row = d * (2 if held == BF16 else 1)
    pages = (1 << 32) // (heads * page * row) + 16
    cache = ra.new_cache(pages, heads, page, d, held)
    small_table, n = R.make_paged([L + T], page, 13, spare=0)
    small = ra.new_cache(n, heads, page, d, held)
    last = small_table.clone()
    last[last >= 0] += pages - n
    kv = rnd(1, 2, 1, heads, L + T, d, dtype=BF16)
    q = rnd(2, 1, Hq, T, d, dtype=BF16)
    res = []
    for c, t in ((small, small_table), (cache, last)):
        ra.ra_cache_write(c, kv[0], kv[1], t.to(DEV), i32(0))
        res.append((*ra.ra_cache_attention(q, c, t.to(DEV), i32(L)), *ra.ra_cache_read(c, t.to(DEV), i32(L), 0, L)))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert ra.ra_last_device_status() == 0


# -------------------------------------------------------------------- watchdog
@pytest.mark.parametrize("held", [BF16, E4M3])
@pytest.mark.parametrize("T", [10, 40])
def test_stalled_cta_of_the_tree_kernel_times_out(held, T):
    """The CTA that loads nothing gives up its waits, the call reports it and
    the next call is right."""
    heads, Hq, d, page, L = 1, 8, 128, 64, 1500
    table, pages = R.make_paged([L + T], page, 15)
    tab, lens = table.to(DEV), i32(L)
    cache = ra.new_cache(pages, heads, page, d, held)
    ra.ra_cache_write(cache, *rnd(1, 2, 1, heads, L + T, d, dtype=BF16), tab, i32(0))
    q = rnd(2, 1, Hq, T, d, dtype=BF16)
    want = ra.ra_cache_attention(q, cache, tab, lens)
    assert ra.ra_last_device_status() == 0
    try:
        ra.ra_watchdog_config(20_000_000, 1)
        t0 = time.perf_counter()
        ra.ra_cache_attention(q, cache, tab, lens)
        assert ra.ra_last_device_status() == _native.RA_ERR_TIMEOUT
        assert time.perf_counter() - t0 < 5.0
    finally:
        ra.ra_watchdog_config(0, -1)
    again = ra.ra_cache_attention(q, cache, tab, lens)
    assert ra.ra_last_device_status() == 0
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("T", [10, 40])
def test_a_timeout_is_reported_over_a_missing_page(T):
    """A page outside the cache leaves the other results valid, a timeout does
    not: with both since the last look, the timeout is what is reported."""
    heads, Hq, d, page, L = 1, 8, 128, 64, 1500
    table, pages = R.make_paged([L + T], page, 15)
    tab, lens = table.to(DEV), i32(L)
    cache = ra.new_cache(pages, heads, page, d)
    ra.ra_cache_write(cache, *rnd(1, 2, 1, heads, L + T, d, dtype=BF16), tab, i32(0))
    q = rnd(2, 1, Hq, T, d, dtype=BF16)
    bad = table.clone()
    bad[0, 3] = pages
    assert ra.ra_last_device_status() == 0
    ra.ra_cache_read(cache, bad.to(DEV), lens, 0, L)
    torch.cuda.synchronize()
    try:
        ra.ra_watchdog_config(20_000_000, 1)
        ra.ra_cache_attention(q, cache, tab, lens)
        torch.cuda.synchronize()
        ra.ra_cache_read(cache, bad.to(DEV), lens, 0, L)   # nor does a page behind it hide it
        assert ra.ra_last_device_status() == _native.RA_ERR_TIMEOUT
    finally:
        ra.ra_watchdog_config(0, -1)
    assert ra.ra_last_device_status() == 0
    ra.ra_cache_read(cache, bad.to(DEV), lens, 0, L)
    assert ra.ra_last_device_status() == _native.RA_ERR_PAGE


# -------------------------------------------------------------------- refusals
def test_the_binding_refuses_what_does_not_fit():
    cache = ra.new_cache(4, 2, 16, 64)
    tab, lens = torch.zeros(1, 4, dtype=torch.int32, device=DEV), i32(3)
    q = rnd(1, 1, 4, 2, 64, dtype=BF16)
    kv = rnd(2, 1, 2, 2, 64, dtype=BF16)
    with pytest.raises(ValueError):
        ra.ra_cache_attention(q.transpose(1, 2), cache, tab, lens)            # not dense
    with pytest.raises(ValueError):
        ra.ra_cache_attention(rnd(1, 1, 4, 2, 128, dtype=BF16), cache, tab, lens)  # head width
    with pytest.raises(ra.RaError):
        ra.ra_cache_attention(rnd(1, 1, 3, 2, 64, dtype=BF16), cache, tab, lens)   # 3 heads over 2
    with pytest.raises(ra.RaError):
        ra.ra_cache_attention(q.float(), cache, tab, lens)                    # fp32 over bf16
    with pytest.raises(TypeError):
        ra.ra_cache_attention(q, cache, tab.long(), lens)
    with pytest.raises(TypeError):
        ra.ra_cache_attention(q, cache, tab, lens, mask=torch.zeros(2, 2, device=DEV))
    with pytest.raises(ValueError):
        ra.ra_cache_attention(q, cache, tab, lens, mask=torch.ones(3, 3, dtype=torch.bool, device=DEV))
    with pytest.raises(ValueError):
        ra.ra_cache_attention(q, cache, tab, i32(1, 2))
    with pytest.raises(ra.RaError):
        ra.ra_cache_attention(q, cache, tab, lens, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        ra.ra_cache_write(cache, kv, kv.float(), tab, lens)
    with pytest.raises(ValueError):
        ra.ra_cache_write(cache, kv[:, :1], kv[:, :1], tab, lens)
    with pytest.raises(ValueError):
        ra.ra_cache_write(cache, kv.transpose(2, 3).contiguous().transpose(2, 3), kv, tab, lens)
    with pytest.raises(ValueError):
        ra.ra_qk_norm_rope(q, q, rope_of(64))                                 # no positions
    with pytest.raises(ValueError):
        ra.ra_qk_norm_rope(q, q, rope_of(64), torch.zeros(2, 2, dtype=torch.int64, device=DEV))
    with pytest.raises(TypeError):
        ra.ra_qk_norm_rope(q, q, q_weight=torch.ones(64, device=DEV))         # fp32 weight of bf16 rows
    with pytest.raises(ValueError):
        ra.RaCache(cache.k, cache.v, k_exp=torch.zeros(4, 2, 16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        ra.RaCache(cache.k.to(E4M3), cache.v.to(E4M3))
    assert ra.ra_last_device_status() == 0
