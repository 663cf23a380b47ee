"""ra_verify_drafts on rows of which little is left, that are long, or that hold
what no decision needs, against the definition in 64 bits.

Inputs are placed beside a border on purpose: 2^-39.5 to 2^-38 of the decision's
value away from it, which the documented 2^-40 has to tell apart."""
import math

import numpy as np
import pytest
import torch

import fork_ref as F
import long_context_ra_gb300 as ra
from test_gpu_verify import check, make

pytestmark = pytest.mark.gpu
DEV = "cuda"
ONE = np.float32(1.0 - 2.0 ** -24)  # the largest uniform number
NEAR, FAR = 2.0 ** -39.5, 2.0 ** -38


def beside(others, around, stays, r):
    """(p, u), fp32, such that u (others + p) lies NEAR to FAR of p below
    (`stays`) or above it; `others` in 64 bits."""
    while True:
        p = (around * r.uniform(0.5, 1.5, 1 << 17)).astype(np.float32)
        u = (p / (others + p.astype(np.float64))).astype(np.float32)
        off = (u.astype(np.float64) * (others + p.astype(np.float64)) - p) / p
        good = np.flatnonzero((np.abs(off) > NEAR) & (np.abs(off) < FAR) & ((off < 0) == stays))
        if len(good):
            return p[good[0]], u[good[0]]


def run(p, tokens, u, parent):
    """One tree for all sequences, chosen drafts."""
    B, T = u.shape
    return check(torch.from_numpy(p).to(DEV), None, torch.from_numpy(tokens).to(DEV),
                 np.tile(np.array(parent, dtype=np.int32), (B, 1)), torch.from_numpy(u).to(DEV))


@pytest.mark.parametrize("V", [257, 20011])
@pytest.mark.parametrize("left", [3, 7, 10, 16, 22])
@pytest.mark.parametrize("more", [0, 1, 3])
def test_little_is_left_of_a_chosen_row(left, more, V):
    """The first draft has 1 - 2^-left of the row and is refused, `more` others
    have some of the rest and are refused too; the next one is beside its border."""
    B, T = 24, 3 + more
    r = np.random.RandomState(left * 10 + more)
    p = np.zeros((B, T, V), dtype=np.float32)
    tokens = np.tile(np.arange(T), (B, 1))
    u = np.full((B, T), ONE)
    for b in range(B):
        row = np.exp(2 * r.randn(V))
        row = (row / row.sum() * 2.0 ** -left).astype(np.float32)
        rest = np.float64(2.0 ** -left)
        for t in range(1, T - 1):
            row[t] = np.float32(1.0 - 2.0 ** -left) if t == 1 else np.float32(rest * r.uniform(0.2, 0.6))
        row[T - 1] = 0
        others = math.fsum(row[[i for i in range(V) if not 1 <= i < T]].tolist())
        row[T - 1], u[b, T - 1] = beside(others, others * r.uniform(0.2, 2), b % 2 == 0, r)
        u[b, 0] = r.rand()
        p[b] = row
    path, kept, _ = run(p, tokens, u, [-1] + [0] * (T - 1))
    assert kept.tolist() == [2 - b % 2 for b in range(B)]


@pytest.mark.parametrize("V", [40, 5003])
def test_a_row_that_is_used_up_step_by_step(V):
    """Three refused drafts leave 2^-67 of the row; one of probability 0 is no
    node of the path, and the next token is the one that is left."""
    B, T = 64, 5
    r = np.random.RandomState(V)
    p = np.zeros((B, T, V), dtype=np.float32)
    u = np.full((B, T), ONE)
    tokens = np.zeros((B, T), dtype=np.int64)
    for b in range(B):
        at = r.permutation(V)[:5]
        p[b, :, at[0]] = 1.0 - 2.0 ** -23
        for i in range(1, 4):  # each is refused: what is left behind it is some 2^-22 of it
            p[b, :, at[i]] = r.uniform(0.6, 1.0) * 2.0 ** (-1 - 22 * i)
        tokens[b, 1:] = at[[0, 1, 2, 4]]
        u[b, 0], u[b, 4] = r.rand(), 0.5
    path, kept, token = run(p, tokens, u, [-1, 0, 0, 0, 0])
    for b in range(B):  # whatever is kept has a probability
        assert all(p[b, 0, tokens[b, t]] > 0 for t in path[b].tolist() if t > 0)
        if int(kept[b]) == 1:
            assert p[b, 0, int(token[b])] > 0
    assert (kept == 1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_refused_draft_that_is_not_finite(dtype):
    """A chosen draft with a NaN for its probability is refused and out of the
    row: the drafts and the token after it are those of the rest."""
    B, T, V = 6, 3, 50
    g = torch.Generator(device=DEV).manual_seed(1)
    p = torch.softmax(torch.randn(B, T, V, generator=g, device=DEV), -1).to(dtype)
    p[:, 0, 7] = math.nan
    tokens = torch.tensor([[0, 7, 3]], device=DEV).expand(B, T).contiguous()
    u = torch.rand(B, T, generator=g, device=DEV)
    rest = p[:, 0].double().nan_to_num(0.0)
    total = rest.sum(-1)
    u[:, 2] = (rest[:, 3] / total * torch.tensor([0.5, 2.0] * 3, device=DEV)).float()
    par = torch.tensor([[-1, 0, 0]], dtype=torch.int32, device=DEV).expand(B, T).contiguous()
    path, kept, token = ra.ra_verify_drafts(p, tokens, u, par)
    assert kept.tolist() == [2, 1] * 3
    assert path[::2, 1].tolist() == [2] * 3
    rest[1::2, 3] = 0.0
    rest[::2] = p[::2, 2].double()
    upto = rest.cumsum(-1)
    want = (upto > u[:, :1].double() * upto[:, -1:]).double().argmax(-1)
    assert torch.equal(token, want)


@pytest.mark.parametrize("value", [math.nan, math.inf, -1.0, 1e30])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tree", [False, True])
def test_rows_of_draft_probs_that_nothing_was_drawn_from(tree, dtype, value):
    """A node without drafts has no row of draft_probs: what lies there does not
    matter, in a chain that stays whole, at the leaves of trees, for a node 0
    that stands alone."""
    B, T, V = 20, 6, 301
    p, q, tokens, parent, u = make(B, T, V, dtype, tree, True, 9)
    u[:, 1:] *= 0.05
    count = [T - b % T for b in range(B)]
    for b in range(B):
        above = {parent[b, t] if tree else t - 1 for t in range(1, count[b])}
        for t in set(range(T)) - above:
            q[b, t] = value
    path, kept, token = check(p, q, tokens, parent, u, count)
    assert (kept > 1).any() and (token >= 0).all()


def test_a_row_of_draft_probs_that_is_needed():
    """A NaN in the row that refused a draft was drawn from: no next token."""
    p, q, tokens, parent, u = make(3, 2, 50, torch.float32, False, True, 2)
    u[:, 1] = float(ONE)
    p[:, 0, :] = 1.0 / 50
    q[:, 0] = torch.softmax(torch.arange(50.0, device=DEV) * 0.1, -1)
    tokens[:, 1] = 49
    q[1, 0, 3] = math.nan
    par = torch.tensor([[-1, 0]] * 3, dtype=torch.int32, device=DEV)
    path, kept, token = ra.ra_verify_drafts(p, tokens, u, par, q)
    assert kept.tolist() == [1, 1, 1] and token.tolist()[1] == -1 and min(token.tolist()[::2]) >= 0


def test_the_longest_row():
    """V = 2^31 - 1: the last token's place in the second row, which begins 14
    bytes behind a multiple of 16, lies behind 2^31."""
    V = 2 ** 31 - 1
    p = torch.zeros(1, 3, V, dtype=torch.bfloat16, device=DEV)
    p[0, 0, V - 2] = 1.0
    p[0, 1, V - 1], p[0, 1, V - 3], p[0, 1, 5] = 0.5, 0.25, 0.25
    tokens = torch.tensor([[0, V - 2, V - 1]], device=DEV)
    u = torch.tensor([[0.6, 0.5, 0.9]], device=DEV)
    path, kept, token = ra.ra_verify_drafts(p, tokens, u)
    assert path.tolist() == [[0, 1, -1]] and kept.tolist() == [2] and token.tolist() == [V - 3]


def test_a_long_row_with_a_peak():
    """Some 2^13 small probabilities behind one that has a good part of the row, in
    one thread's part of it."""
    B, T, V = 6, 3, 1 << 26
    r = np.random.RandomState(3)
    g = torch.Generator(device=DEV).manual_seed(3)
    p = torch.zeros(B, T, V, device=DEV)
    tokens = torch.tensor([[0, 1, 0]], device=DEV).expand(B, T).contiguous()
    par = torch.tensor([[-1, 0, 0]], dtype=torch.int32, device=DEV).expand(B, T).contiguous()
    u = torch.full((B, T), float(ONE), device=DEV)
    for b in range(B):
        row = torch.exp(torch.randn(V, generator=g, device=DEV))
        p[b, 0] = row * (0.4 / row.sum(dtype=torch.float64)).float()
        p[b, 0, 1], p[b, 0, 0] = 0.25, 0.0
        others = float(p[b, 0].sum(dtype=torch.float64)) - 0.25
        x, y = beside(others, others, b % 2 == 0, r)
        p[b, 0, 0], u[b, 2] = float(x), float(y)
    path, kept, _ = ra.ra_verify_drafts(p, tokens, u, par)
    assert kept.tolist() == [2, 1] * 3 and path[::2, 1].tolist() == [2] * 3
