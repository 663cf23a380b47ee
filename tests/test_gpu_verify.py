"""ra_verify_drafts against the definition in 64 bits: the same decisions.

The kernel's sums are off by 2^-47 relative (pairs of floats) and a few
roundings of 64 bits; a test only asks that no input lies nearer to a border
than 2^-40, which the reference measures, before it compares."""
import math

import numpy as np
import pytest
import torch

import fork_ref as F
import long_context_ra_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda"
BORDER = 2.0 ** -40


def trees(B, T, r, wide):
    parent = np.full((B, T), -1, dtype=np.int32)
    for t in range(1, T):
        parent[:, t] = r.randint(0 if wide else max(0, t - 3), t, size=B)
    return parent


def make(B, T, V, dtype, tree, draft, seed, sharp=3.0, noise=0.7, wide=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.RandomState(seed)
    logits = torch.randn(B, T, V, generator=g, device=DEV) * sharp
    p = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits + noise * torch.randn(B, T, V, generator=g, device=DEV), -1).to(dtype)
    parent = trees(B, T, r, wide) if tree else None
    above = torch.from_numpy(parent if tree else np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1))).clamp(min=0)
    rows = q.gather(1, above.long().to(DEV)[..., None].expand(B, T, V)).view(B * T, V)
    tokens = torch.multinomial(rows.float().clamp(min=1e-30), 1, generator=g).view(B, T)
    u = torch.rand(B, T, generator=g, device=DEV)
    return p, (q if draft else None), tokens, parent, u


def reference(p, q, tokens, parent, count, u):
    p64, q64 = (None if x is None else x.double().cpu().numpy() for x in (p, q))
    tok, uu = tokens.cpu().numpy(), u.double().cpu().numpy()
    B, T, _ = p64.shape
    paths, kept, after, margins = [], [], [], []
    for b in range(B):
        c = T if count is None else min(count[b], T)
        if c <= 0:
            path, token, margin = [], -1, 1.0
        else:
            path, token, margin = F.verify(p64[b], None if q64 is None else q64[b], tok[b],
                                           None if parent is None else parent[b], c, uu[b])
        paths.append(path + [-1] * (T - len(path)))
        kept.append(len(path))
        after.append(token)
        margins.append(margin)
    return paths, kept, after, np.array(margins)


def check(p, q, tokens, parent, u, count=None):
    par = None if parent is None else torch.from_numpy(np.ascontiguousarray(parent)).to(DEV)
    cnt = None if count is None else torch.tensor(count, dtype=torch.int32, device=DEV)
    path, kept, token = ra.ra_verify_drafts(p, tokens, u, par, q, cnt)
    want = reference(p, q, tokens, parent, count, u)
    clear = want[3] > BORDER
    assert clear.mean() > 0.9
    for got, w in zip((path, kept, token), want):
        got, w = got.cpu().numpy(), np.array(w)
        assert (got == w)[clear].all(), np.argwhere(got != w)[:5]
    return path, kept, token


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 2, 2), (5, 4, 7), (9, 9, 130), (3, 33, 1001), (64, 6, 257),
                                   (700, 3, 40)])
def test_small(B, T, V, tree, draft, dtype):
    args = make(B, T, V, dtype, tree, draft, B + T + V)
    check(*args)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,T,V", [(1, 3, 200003), (2, 5, 131072), (200, 2, 30011), (620, 2, 5000), (3, 40, 32768)])
def test_long_rows(B, T, V, draft, dtype):
    """1 to 8 CTAs to a sequence, rows that begin anywhere in 16 bytes."""
    args = make(B, T, V, dtype, T > 2, draft, V)
    check(*args)


def test_one_long_row_per_warp():
    """Runs of more than 32 pieces a lane: one CTA to a sequence."""
    p, q, tokens, parent, u = make(1, 2, 300000, torch.float32, False, True, 4)
    B = 640
    u = torch.rand(B, 2, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5))
    check(p.expand(B, -1, -1).contiguous(), q.expand(B, -1, -1).contiguous(), tokens.expand(B, -1).contiguous(),
          None, u)


@pytest.mark.parametrize("draft", [True, False])
def test_wide_trees(draft):
    """Many drafts below a node, equal ones among them: sums after each refusal."""
    p, q, tokens, parent, u = make(40, 60, 50, torch.float32, True, draft, 8, sharp=1.0, noise=2.0, wide=True)
    parent[:, 1:20] = 0
    path, kept, token = check(p, q, tokens, parent, u)
    u[:, 1:] = 0.999
    check(p, q, tokens, parent, u)


def test_counts_and_nodes_that_are_none():
    p, q, tokens, parent, u = make(8, 9, 64, torch.float32, True, True, 3)
    u[:, 1:] *= 0.2
    tokens[0, 1], tokens[1, 2], tokens[2, 3] = -1, 64, 1 << 40
    parent[3, 2], parent[4, 3], parent[5, 1], parent[6, 4] = 2, -3, 5, 100
    none = np.array(parent)
    for b, t in ((3, 2), (4, 3), (5, 1), (6, 4)):
        none[b, t] = -1
    count = [9, 9, 9, 9, 9, 40, 0, -2]
    cnt = torch.tensor(count, dtype=torch.int32, device=DEV)
    got = ra.ra_verify_drafts(p, tokens, u, torch.from_numpy(parent).to(DEV), q, cnt)
    want = reference(p, q, tokens, none, count, u)
    for a, w in zip(got, want):
        assert a.tolist() == list(w)
    assert got[1].tolist()[6:] == [0, 0] and got[2].tolist()[6:] == [-1, -1]


def test_rows_that_are_special():
    """One token has it all; both distributions are the same; nothing is left;
    zeros, NaN and infinities; u at both ends."""
    V, T = 37, 3
    p = torch.zeros(9, T, V, device=DEV)
    q = torch.zeros(9, T, V, device=DEV)
    tokens = torch.full((9, T), 5, device=DEV)
    u = torch.full((9, T), 1.0 - 2.0 ** -24, device=DEV)
    flat = torch.full((V,), 1.0 / 32, device=DEV)
    flat[32:] = 0.0
    p[0, :, 5] = q[0, :, 5] = 1.0            # certain: stays
    p[1], q[1] = flat, flat                  # equal: all stay
    p[2, :, 7] = 1.0                         # the draft is impossible
    q[2] = flat
    q[3], p[3] = flat, flat * 0.5            # p below q everywhere: nothing is left, p itself
    p[4], q[4] = 0.0, flat                   # a row without mass
    p[5], q[5] = math.nan, flat
    p[6], q[6] = flat, flat
    p[6, 2, 3] = math.inf
    p[7], q[7] = flat, flat
    u[7] = 0.0                               # the first token with any mass
    p[7, 2, :4] = 0.0
    p[8], q[8] = flat, flat
    u[8] = math.nan                          # refused; the last token with any mass
    path, kept, token = ra.ra_verify_drafts(p, tokens, u, None, q)
    assert kept.tolist() == [3, 3, 1, 1, 1, 1, 3, 3, 1]
    assert token.tolist() == [5, 31, 7, 31, -1, -1, -1, 4, 31]
    assert path.tolist()[0] == [0, 1, 2] and path.tolist()[2] == [0, -1, -1]
    # chosen drafts: what is refused is out, and equal drafts are refused once more
    p = torch.zeros(1, 3, 4, device=DEV)
    p[0, 0] = torch.tensor([0.25, 0.5, 0.25, 0.0])
    tok = torch.tensor([[0, 1, 1]], device=DEV)
    par = torch.tensor([[-1, 0, 0]], dtype=torch.int32, device=DEV)
    uu = torch.tensor([[0.5, 0.5, 0.0]], device=DEV)
    path, kept, token = ra.ra_verify_drafts(p, tok, uu, par)
    # u = 0.5 < 0.5 is false; then r = (1/4, 0, 1/4), 0 < 0 is false; cum 1/4 > 1/4 is false
    assert kept.tolist() == [1] and token.tolist() == [2]


def test_borders_between_tokens():
    """u just at and beside the borders of the cumulative sums: fp32 sums would
    take the neighbouring token."""
    V, B = 50000, 256
    g = torch.Generator(device=DEV).manual_seed(2)
    row = torch.softmax(torch.randn(V, generator=g, device=DEV) * 2, -1)
    upto = np.cumsum(row.double().cpu().numpy())
    at = np.random.RandomState(0).randint(0, V, B)
    border = (upto[at] / upto[-1]).astype(np.float32)
    u = torch.from_numpy(np.nextafter(border, np.where(np.arange(B) % 2 == 0, 0, 1).astype(np.float32))).to(DEV)[:, None]
    p = row.expand(B, 1, V).contiguous()
    tokens = torch.zeros(B, 1, dtype=torch.int64, device=DEV)
    check(p, None, tokens, None, u)


def test_the_first_token_is_the_models():
    """Over many random numbers the token behind node 0 has the model's
    distribution, drawn drafts or chosen ones: within 6 standard deviations."""
    B, V = 1 << 16, 6
    g = torch.Generator(device=DEV).manual_seed(11)
    p = torch.tensor([0.4, 0.05, 0.3, 0.0, 0.2, 0.05], device=DEV).expand(B, 3, V).contiguous()
    qrow = torch.tensor([0.1, 0.5, 0.1, 0.1, 0.1, 0.1], device=DEV)
    q = qrow.expand(B, 3, V).contiguous()
    par = torch.tensor([-1, 0, 0], dtype=torch.int32, device=DEV).expand(B, 3).contiguous()
    u = torch.rand(B, 3, generator=g, device=DEV)
    drawn = torch.multinomial(qrow.expand(B, V), 3, replacement=True, generator=g)
    chosen = torch.tensor([0, 2, 1], device=DEV).expand(B, 3).contiguous()
    for tokens, draft in ((drawn, q), (chosen, None)):
        path, kept, token = ra.ra_verify_drafts(p, tokens, u, par, draft)
        second = path[:, 1].long()
        first = torch.where(kept > 1, tokens.gather(1, second.clamp(min=0)[:, None])[:, 0], token)
        share = torch.bincount(first, minlength=V).double().cpu() / B
        want = p[0, 0].double().cpu()
        assert ((share - want).abs() <= 6 * (want * (1 - want) / B).sqrt() + 1e-12).all(), share


def test_the_same_bits_every_time():
    args = make(20, 12, 20011, torch.bfloat16, True, True, 6)
    par = torch.from_numpy(args[3]).to(DEV)
    a = ra.ra_verify_drafts(args[0], args[2], args[4], par, args[1])
    for _ in range(3):
        b = ra.ra_verify_drafts(args[0], args[2], args[4], par, args[1])
        assert all(torch.equal(x, y) for x, y in zip(a, b))
