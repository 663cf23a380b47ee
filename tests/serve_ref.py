"""Plain 64-bit references of the calls around the attention, on the CPU:
the norm and rotation of queries and keys with its gradients, the 8-bit rows
of the cache, and the attention of new tokens over a paged cache.  They share
no code with the library."""
from __future__ import annotations

import math

import torch

EPS_HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a rounding step
U = 2.0 ** -24  # half a step of fp32 arithmetic


def f64(t):
    return None if t is None else t.detach().double().cpu()


# ---------------------------------------------------------- norm and rotation
def rotation(positions, inv_freq, axis):
    """Angles [B, N, pairs] of positions [axes, B, N]."""
    pos = positions.cpu().double()
    return torch.stack([pos[a] * f for a, f in zip(axis, inv_freq)], -1)


def rotate(x, angle, interleaved, sign=1.0):
    """The first 2 * pairs elements of x [B, H, N, d] turned by sign * angle."""
    pairs = angle.shape[-1]
    y = x.clone()
    c, s = angle.cos()[:, None], sign * angle.sin()[:, None]
    for i in range(pairs):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        y[..., p] = x[..., p] * c[..., i] - x[..., q] * s[..., i]
        y[..., q] = x[..., q] * c[..., i] + x[..., p] * s[..., i]
    return y


def norm_rope(x, w, eps, angle, interleaved):
    x = f64(x)
    if eps is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
        if w is not None:
            x = x * f64(w)
    return rotate(x, angle, interleaved) if angle is not None else x


def norm_rope_backward(x, w, eps, angle, interleaved, dy):
    """dx, dw, and the sizes their errors scale with (per element of dx: the
    terms it is the difference of; per element of dw: the sum of |terms|)."""
    x, dy = f64(x), f64(dy)
    dz = rotate(dy, angle, interleaved, -1.0) if angle is not None else dy
    if eps is None:
        return dz, None, dz.abs().amax(-1, keepdim=True), None
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    n = x * r
    g = dz * f64(w) if w is not None else dz
    mean = (g * n).mean(-1, keepdim=True)
    size = r * (g.abs().amax(-1, keepdim=True) +
                n.abs().amax(-1, keepdim=True) * (g * n).abs().mean(-1, keepdim=True))
    terms = dz * n
    return r * (g - n * mean), terms.sum((0, 1, 2)), size, terms.abs().sum((0, 1, 2))


# ------------------------------------------------------------------ the cache
def quantise(x):
    """(8-bit values as float64, exponent bytes) of rows of x [..., d]."""
    x = f64(x)
    top = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    f, ex = torch.frexp(top)                       # top = f 2^ex, f in [0.5, 1)
    e = (ex - 9 + (f > 0.875).int()).clamp(-126, 120)
    e = torch.where(top > 0, e, torch.full_like(e, -126))
    y = x * torch.exp2(-e.double())[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(2.0 ** -6, 448.0))) - 3)
    y = torch.round(y / step) * step               # halves to even
    return y.clamp(-448.0, 448.0), (e + 127).to(torch.uint8)


class PagedCpu:
    """Where each sequence's positions lie, and the cache's values in 64 bits."""

    def __init__(self, cache, table):
        self.k, self.v = (self._values(t, e) for t, e in ((cache.k, cache.k_exp),
                                                          (cache.v, cache.v_exp)))
        self.table = table.cpu().tolist()
        self.page = cache.k.shape[2]

    @staticmethod
    def _values(t, e):
        x = t.cpu().float().double()
        return x if e is None else x * torch.exp2(e.cpu().double()[..., None] - 127)

    def rows(self, b, n):
        """K and V rows 0 .. n - 1 of sequence b: [heads, n, d] each."""
        at = [(self.table[b][p // self.page], p % self.page) for p in range(n)]
        pages = torch.tensor([a for a, _ in at], dtype=torch.long)
        place = torch.tensor([o for _, o in at], dtype=torch.long)
        return (self.k[pages, :, place].transpose(0, 1), self.v[pages, :, place].transpose(0, 1))


def attention(q, paged, lens, count, mask):
    """out, lse, and per row the bounds that errors scale with:
    (sum p |v| / l per element, sum |q||k| tau of the largest key)."""
    q = f64(q)
    B, Hq, T, d = q.shape
    heads = paged.k.shape[1]
    g = Hq // heads
    out = torch.zeros(B, Hq, T, d, dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    size = torch.zeros(B, Hq, T, dtype=torch.float64)
    for b in range(B):
        L = lens[b]
        if L < 0:
            continue
        c = T if count is None else count[b]
        k, v = paged.rows(b, L + c)
        for t in range(c):
            sees = torch.ones(L + c, dtype=torch.bool)
            for j in range(c):
                sees[L + j] = (j <= t) if mask is None else bool(mask[b if mask.dim() == 3 else 0][t, j]
                                                               if mask.dim() == 3 else mask[t, j])
            if not sees.any():
                continue
            for h in range(Hq):
                kk, vv = k[h // g][sees], v[h // g][sees]
                s = kk @ q[b, h, t] / math.sqrt(d)
                m = s.max()
                p = (s - m).exp()
                out[b, h, t] = p @ vv / p.sum()
                mag[b, h, t] = p @ vv.abs() / p.sum()
                lse[b, h, t] = m + p.sum().log()
                size[b, h, t] = (kk.abs() @ q[b, h, t].abs()).max() / math.sqrt(d)
    return out, lse, mag, size


def make_paged(lens_total, page, seed, spare=3, width_extra=1):
    """A scrambled page table (int32 [B, width], -1 behind the last page) for
    sequences of the given total lengths, and the number of pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lens_total]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).tolist()
    width = max(max(need, default=0), 0) + width_extra
    table = torch.full((len(lens_total), width), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = order.pop()
    return table, pages
