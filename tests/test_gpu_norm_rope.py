"""ra_qk_norm_rope and its backward against 64-bit references.

Tolerances, before any run.  A bf16 result is rounded once: 2^-8 |want|.  The
fp32 arithmetic before it: the sum of squares of a row takes 8 products a
lane and at most 5 exchanges (13 roundings, halved by the root), then mean,
eps, rsqrt (2 steps), the two products with r and w, cosine and sine (2 steps
each, and 2^-24 of the angle's half turn) and the rotation's three roundings:
below 32 half steps of the row's largest normalised element.  The backward
runs the same terms twice and subtracts: below 64 half steps of the sizes
that it subtracts.  A weight gradient adds at most 256 terms in a chain (rows
of one thread, groups of a block) of 24 half steps each: below 280 half steps
of the sum of magnitudes."""
import math

import pytest
import torch

import long_context_ra_gb300 as ra
import serve_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"

SHAPES = [
    # B, N, Hq, Hk, d, rot, axes, interleaved
    (1, 1, 1, 1, 8, 8, 1, False),
    (5, 1, 8, 2, 64, 64, 1, False),
    (2, 37, 3, 1, 128, 128, 1, True),
    (1, 129, 4, 4, 80, 80, 1, False),
    (2, 33, 5, 2, 128, 96, 3, True),
    (1, 65, 2, 1, 256, 256, 3, False),
    (3, 17, 7, 3, 104, 8, 2, False),
    (1, 300, 2, 2, 16, 0, 1, False),
]


def case(shape, dtype, seed, strided=True, norm=True, far=1 << 20):
    B, N, Hq, Hk, d, rot, axes, inter = shape
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, device=DEV, generator=g)
    both = (rnd(B, N, Hq + Hk, d) * 2).to(dtype)
    q, k = both[:, :, :Hq].transpose(1, 2), both[:, :, Hq:].transpose(1, 2)
    if not strided:
        q, k = q.contiguous(), k.contiguous()
    wq, wk = ((1 + 0.3 * rnd(d)).to(dtype) for _ in range(2)) if norm else (None, None)
    inv = [10000.0 ** (-i / max(1, rot // 2)) for i in range(rot // 2)]
    axis = [i * axes // max(1, rot // 2) for i in range(rot // 2)]
    pos = torch.randint(-far, far, (axes, B, N), device=DEV, generator=g)
    rope = ra.new_rope(inv, axis, inter, axes=axes)
    angle = R.rotation(pos, inv, axis) if rot else None
    return q, k, wq, wk, rope, pos, angle


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, norm, dtype):
    q, k, wq, wk, rope, pos, angle = case(shape, dtype, 1, norm=norm)
    eps = 1e-5 if norm else None
    got = ra.ra_qk_norm_rope(q, k, rope, pos, wq, wk, eps)
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        assert y.is_contiguous() and y.shape == x.shape and y.dtype == dtype
        want = R.norm_rope(x, w, eps, angle, shape[7])
        tol = R.EPS_HALF[dtype] * want.abs() + 32 * R.U * want.abs().amax(-1, keepdim=True) * math.sqrt(2)
        assert ((R.f64(y) - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, norm, dtype):
    q, k, wq, wk, rope, pos, angle = case(shape, dtype, 2, norm=norm)
    eps = 1e-5 if norm else None
    g = torch.Generator(device=DEV).manual_seed(3)
    dys = [torch.randn(x.shape, device=DEV, generator=g).to(dtype) for x in (q, k)]
    dq, dk, dwq, dwk = ra.ra_qk_norm_rope_backward(q, k, *dys, rope, pos, wq, wk, eps)
    for x, w, dy, dx, dw in ((q, wq, dys[0], dq, dwq), (k, wk, dys[1], dk, dwk)):
        assert dx.shape == x.shape and dx.dtype == dtype
        want, want_w, size, terms = R.norm_rope_backward(x, w, eps, angle, shape[7], dy)
        tol = R.EPS_HALF[dtype] * want.abs() + 64 * R.U * math.sqrt(2) * size
        assert ((R.f64(dx) - want).abs() <= tol).all()
        if norm:
            assert dw.dtype == torch.float32
            assert ((R.f64(dw) - want_w).abs() <= 280 * R.U * math.sqrt(2) * terms).all()
        else:
            assert dw is None


@pytest.mark.parametrize("shape", SHAPES[1:5])
def test_gradient_against_differences(shape):
    """The fp32 gradient against central differences of the 64-bit forward
    along a random direction (their own error is h^2 of the third derivative,
    far below the fp32 one at h = 1e-5)."""
    q, k, wq, wk, rope, pos, angle = case(shape, torch.float32, 4)
    g = torch.Generator(device=DEV).manual_seed(5)
    dys = [torch.randn(x.shape, device=DEV, generator=g) for x in (q, k)]
    dq, dk, dwq, dwk = ra.ra_qk_norm_rope_backward(q, k, *dys, rope, pos, wq, wk, 1e-5)
    for x, w, dy, dx, dw in ((q, wq, dys[0], dq, dwq), (k, wk, dys[1], dk, dwk)):
        f = lambda xx, ww: (R.norm_rope(xx, ww, 1e-5, angle, shape[7]) * R.f64(dy)).sum()
        cg = torch.Generator().manual_seed(6)
        vx = torch.randn(x.shape, generator=cg, dtype=torch.float64)
        vw = torch.randn(w.shape, generator=cg, dtype=torch.float64)
        h = 1e-5
        want = (f(R.f64(x) + h * vx, R.f64(w) + h * vw) - f(R.f64(x) - h * vx, R.f64(w) - h * vw)) / (2 * h)
        got = (R.f64(dx) * vx).sum() + (R.f64(dw) * vw).sum()
        _, _, size, terms = R.norm_rope_backward(x, w, 1e-5, angle, shape[7], dy)
        tol = (66 * R.U * math.sqrt(2) * size * vx.abs()).sum() + (280 * R.U * terms * vw.abs()).sum()
        assert abs(got - want) <= tol + 1e-8 * abs(want)


def test_views_and_dense_inputs_agree_and_gradients_keep_the_layout():
    shape = (2, 33, 5, 2, 128, 96, 3, True)
    a, b = case(shape, torch.bfloat16, 7), case(shape, torch.bfloat16, 7, strided=False)
    assert not a[0].is_contiguous() and b[0].is_contiguous()
    for x, y in zip(ra.ra_qk_norm_rope(*a[:2], a[4], a[5], a[2], a[3]),
                    ra.ra_qk_norm_rope(*b[:2], b[4], b[5], b[2], b[3])):
        assert torch.equal(x, y)
    dys = [torch.randn_like(x) for x in b[:2]]
    ga = ra.ra_qk_norm_rope_backward(*a[:2], *dys, a[4], a[5], a[2], a[3])
    gb = ra.ra_qk_norm_rope_backward(*b[:2], *dys, b[4], b[5], b[2], b[3])
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))


def test_shared_heads_of_an_expanded_key():
    """An input whose heads are one broadcast row (stride 0) is read as such;
    its gradient is dense."""
    shape = (1, 5, 2, 1, 64, 64, 1, False)
    q, k, wq, wk, rope, pos, angle = case(shape, torch.float32, 8)
    k4 = k.expand(1, 4, 5, 64)
    _, y = ra.ra_qk_norm_rope(q, k4, rope, pos, wq, wk)
    _, one = ra.ra_qk_norm_rope(q, k, rope, pos, wq, wk)
    assert torch.equal(y, one.expand(1, 4, 5, 64))
    dy = torch.randn(1, 4, 5, 64, device=DEV)
    _, dk, _, _ = ra.ra_qk_norm_rope_backward(q, k4, torch.zeros(1, 2, 5, 64, device=DEV), dy, rope,
                                              pos, wq, wk)
    assert dk.is_contiguous()
    want, _, size, _ = R.norm_rope_backward(k4, wk, 1e-6, angle, False, dy)
    assert ((R.f64(dk) - want).abs() <= R.U * want.abs() + 64 * R.U * math.sqrt(2) * size).all()


def test_far_positions_keep_their_angles():
    """Positions up to 2^40: the angle is the exact fraction of a turn, so the
    result stays within the forward's tolerance (the reference takes the
    product in exact integers)."""
    from fractions import Fraction

    inv = [1.0, 0.5, 0.1, 1e-3]
    pos = torch.tensor([[[(1 << 40) + 12345, -(1 << 39) - 7, 1 << 31, 123456789]]], device=DEV)
    two_pi = Fraction(2) * Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    angle = torch.tensor([[[float((int(p) * Fraction(f)) % two_pi) for f in inv]
                           for p in pos[0, 0].tolist()]], dtype=torch.float64)
    x = torch.randn(1, 1, 4, 8, device=DEV)
    y, _ = ra.ra_qk_norm_rope(x, x, ra.new_rope(inv), pos, eps=None)
    want = R.rotate(R.f64(x), angle, False)
    # the plan's 64-bit turns: half a step of 2^-64 turns per position unit
    tol = 32 * R.U * want.abs().amax(-1, keepdim=True) * 2 + 2 * math.pi * (1 << 41) * 2.0 ** -65 * 4
    assert ((R.f64(y) - want).abs() <= tol).all()


def test_zero_rows_and_empty_sides():
    q = torch.zeros(1, 2, 3, 64, device=DEV)
    k = torch.empty(1, 0, 3, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    y, e = ra.ra_qk_norm_rope(q, k, q_weight=w, eps=1e-6)
    assert e.shape == (1, 0, 3, 64) and torch.equal(y, q)
    dq, dk, dwq, _ = ra.ra_qk_norm_rope_backward(q, k, torch.ones_like(q), k, q_weight=w, eps=1e-6)
    assert torch.allclose(dq, torch.full_like(q, 1e3), rtol=1e-6)  # r = 1 / sqrt(eps)
    assert torch.equal(dwq, torch.zeros(64, device=DEV))
    none = torch.empty(0, 2, 3, 64, device=DEV)
    out = ra.ra_qk_norm_rope_backward(none, none, none, none, q_weight=w, k_weight=w)
    assert torch.equal(out[2], torch.zeros(64, device=DEV)) and out[0].shape == none.shape


def test_gradients_repeat_bit_for_bit():
    shape = (2, 1111, 8, 2, 128, 128, 1, False)
    q, k, wq, wk, rope, pos, _ = case(shape, torch.bfloat16, 9)
    dys = [torch.randn(x.shape, device=DEV).to(x.dtype) for x in (q, k)]
    first = ra.ra_qk_norm_rope_backward(q, k, *dys, rope, pos, wq, wk)
    for _ in range(3):
        again = ra.ra_qk_norm_rope_backward(q, k, *dys, rope, pos, wq, wk)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_on_another_stream():
    shape = (1, 129, 4, 4, 80, 80, 1, False)
    q, k, wq, wk, rope, pos, _ = case(shape, torch.bfloat16, 10)
    want = ra.ra_qk_norm_rope(q, k, rope, pos, wq, wk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ra.ra_qk_norm_rope(q, k, rope, pos, wq, wk, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [
    (1, 1, 2, 1, 64, 64, 1, False),
    (1, 33, 4, 2, 128, 128, 1, False),
    (2, 37, 3, 1, 128, 96, 3, True),
    (1, 37, 2, 2, 24, 24, 1, False),   # 3 lanes of 4 hold a row
    (3, 301, 5, 1, 80, 0, 1, False),
])
def test_backward_without_an_epsilon(shape, dtype):
    """eps = 0, and token counts that leave groups of the last block without a
    token: no row is zero, so every gradient is finite, within the same bounds."""
    q, k, wq, wk, rope, pos, angle = case(shape, dtype, 12)
    g = torch.Generator(device=DEV).manual_seed(13)
    dys = [torch.randn(x.shape, device=DEV, generator=g).to(dtype) for x in (q, k)]
    dq, dk, dwq, dwk = ra.ra_qk_norm_rope_backward(q, k, *dys, rope, pos, wq, wk, 0.0)
    for x, w, dy, dx, dw in ((q, wq, dys[0], dq, dwq), (k, wk, dys[1], dk, dwk)):
        want, want_w, size, terms = R.norm_rope_backward(x, w, 0.0, angle, shape[7], dy)
        tol = R.EPS_HALF[dtype] * want.abs() + 64 * R.U * math.sqrt(2) * size
        assert ((R.f64(dx) - want).abs() <= tol).all()
        assert ((R.f64(dw) - want_w).abs() <= 280 * R.U * math.sqrt(2) * terms).all()
