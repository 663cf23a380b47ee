"""Cases of the serving-path operators: the norm and rotation of queries and
keys (and its backward), the write into and the read from a paged K/V cache,
and attention of drafted tokens over that cache.

Each case has a plain form in elementary torch operations and the calls a
program makes of the library (`own`); `exact` evaluates the definitions in 64
bits.  Attention tensors are [B, H, N, d]; a cache holds pages of
[heads, page, d], reached through a table of page numbers per sequence.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token of each of a few sequences: the latency of a decode step
        dict(name="norm decode", kind="norm", dtype="bf16", B=5, N=1, Hq=8, Hk=2, d=64, rot=64, axes=1,
             interleaved=False, norm=True, far=1 << 20),
        # a prompt of grouped-query heads before the attention of 32 heads
        dict(name="norm prompt", kind="norm", dtype="bf16", B=1, N=32768, Hq=32, Hk=8, d=128, rot=128, axes=1,
             interleaved=False, norm=True, far=1 << 20),
        # training on images: positions of time, height and width, part of each head rotated, an odd length
        dict(name="norm backward", kind="norm_backward", dtype="bf16", B=2, N=16381, Hq=32, Hk=8, d=128, rot=96,
             axes=3, interleaved=True, norm=True, far=4096),
        # the new token of 64 sequences goes into an 8-bit cache
        dict(name="write decode", kind="write", dtype="bf16", cache="e4m3", B=64, T=1, Hk=8, d=128, page=64,
             longest=8192, ragged=True),
        # two prompts of unlike length are quantised into the cache
        dict(name="write prompt", kind="write", dtype="bf16", cache="e4m3", B=2, T=32768, Hk=8, d=128, page=64,
             longest=4099, ragged=True),
        # a short block of a few sequences is read for a continued prompt
        dict(name="read block", kind="read", dtype="bf16", cache="bf16", B=3, n=384, first=513, Hk=2, d=64, page=16,
             longest=1024, ragged=True),
        # a whole long sequence is read back from 8 bits
        dict(name="read long", kind="read", dtype="bf16", cache="e4m3", B=1, n=131072, first=0, Hk=8, d=128, page=128,
             longest=131072, ragged=False),
        # one new token of one short sequence: the smallest call
        dict(name="attend one", kind="attend", dtype="bf16", cache="bf16", B=1, T=1, Hq=8, Hk=8, d=64, page=16,
             longest=1021, ragged=False, mask="causal"),
        # a decode step of 32 sequences of unlike length over an 8-bit cache
        dict(name="attend batch", kind="attend", dtype="bf16", cache="e4m3", B=32, T=1, Hq=32, Hk=8, d=128, page=64,
             longest=32768, ragged=True, mask="causal"),
        # trees of 32 drafted tokens of 8 sequences
        dict(name="attend tree", kind="attend", dtype="bf16", cache="bf16", B=8, T=32, Hq=32, Hk=8, d=128, page=64,
             longest=16384, ragged=True, mask="tree"),
        # a tree over one sequence of a million tokens in 8 bits
        dict(name="attend long tree", kind="attend", dtype="bf16", cache="e4m3", B=1, T=61, Hq=64, Hk=8, d=128,
             page=128, longest=1048576, ragged=False, mask="tree"),
        # the 32-bit path: a few tokens, a head width of no special size
        dict(name="attend f32", kind="attend", dtype="f32", cache="f32", B=2, T=3, Hq=6, Hk=3, d=80, page=16,
             longest=4096, ragged=True, mask="tree"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw(rng):
    kind = rng.choice(["norm", "norm_backward", "write", "read", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind.startswith("norm"):
        d = rng.choice([64, 128, 8 * rng.randint(2, 32)])
        axes = rng.choice([1, 1, 3])
        return dict(kind=kind, dtype=dtype, B=_log(rng, 1, 64), N=_log(rng, 1, 32768), Hq=_log(rng, 1, 64),
                    Hk=_log(rng, 1, 16), d=d, rot=d if rng.random() < 0.5 else 8 * rng.randint(1, d // 8),
                    axes=axes, interleaved=rng.random() < 0.5, norm=rng.random() < 0.75,
                    far=_log(rng, 4096, 1 << 20))
    cache = rng.choice([dtype, "e4m3"])
    d = rng.choice([64, 128]) if dtype == "bf16" else 8 * rng.randint(2, 32)
    c = dict(kind=kind, dtype=dtype, cache=cache, B=_log(rng, 1, 64), Hk=_log(rng, 1, 16), d=d,
             page=2 ** rng.randint(4, 8), ragged=rng.random() < 0.75)
    if kind == "write":
        return dict(c, T=_log(rng, 1, 32768), longest=_log(rng, 1, 8192))
    if kind == "read":
        longest = _log(rng, 16, 131072)
        return dict(c, longest=longest, n=_log(rng, 1, longest), first=rng.randrange(longest))
    return dict(c, T=_log(rng, 1, 128), Hq=c["Hk"] * rng.randint(1, 8), longest=_log(rng, 1, 262144),
                mask=rng.choice(["causal", "tree"]))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if c["kind"] == "attend":
            # the padded scores of the plain form stay below those of the largest listed case
            if w["flops"] > (3e10 if c["dtype"] == "f32" else 1e12) or w["bytes"] > 2e9:
                continue
            if c["B"] * c["longest"] * max(c["T"] * c["Hq"], c["Hk"] * c["d"]) > 4e9:
                continue
        elif w["bytes"] > 1e9 or c["B"] * c.get("longest", 0) * c.get("Hk", 0) * c["d"] > 1e9:
            continue
        return c


def _lens(case):
    """Tokens in the cache before the call, per sequence: `longest` for the
    first, spread below it for the others of a ragged batch."""
    B, L = case["B"], case["longest"]
    if not case["ragged"]:
        return [L] * B
    return [max(1, L - (L * 7 * b) // (8 * B) - (13 * b) % 29) for b in range(B)]


def _counts(case):
    """New tokens per sequence: all T for the first, fewer for some others."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [max(1, T - (T * (b % 4)) // 6) for b in range(B)]


def work(case):
    c = case
    e = SIZE[c["dtype"]]
    if c["kind"] in ("norm", "norm_backward"):
        rows = c["B"] * c["N"] * (c["Hq"] + c["Hk"])
        back = c["kind"] == "norm_backward"
        return {"bytes": rows * c["d"] * e * (3 if back else 2) + c["axes"] * c["B"] * c["N"] * 8,
                "flops": rows * (c["d"] * (10 if back else 4) + 3 * c["rot"])}
    heads, d, s = c["Hk"], c["d"], SIZE[c["cache"]]
    held = d * s + (1 if c["cache"] == "e4m3" else 0)  # one row of the cache
    if c["kind"] == "write":
        rows = 2 * heads * sum(_counts(c))
        return {"bytes": rows * (d * e + held), "flops": 2 * rows * d}
    if c["kind"] == "read":
        seen = sum(min(c["n"], max(0, n - c["first"])) for n in _lens(c))
        return {"bytes": 2 * heads * (seen * held + c["B"] * c["n"] * d * e), "flops": 2 * heads * seen * d}
    g = c["Hq"] // heads
    lens, cnt = _lens(c), _counts(c)
    keys = sum(n + t for n, t in zip(lens, cnt))
    pairs = sum(t * (n + (t + 1) / 2) for n, t in zip(lens, cnt))
    return {"bytes": 2 * heads * keys * held + c["B"] * c["Hq"] * c["T"] * (2 * d * e + 4),
            "flops": 4.0 * heads * g * pairs * d}


# ------------------------------------------------------------- their inputs
class State(dict):
    __getattr__ = dict.__getitem__


def _rnd(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _axis_of_pairs(case):
    """The axis that turns each pair: runs of pairs for time, height, width."""
    pairs, axes = case["rot"] // 2, case["axes"]
    return [min(axes - 1, i * axes // pairs) for i in range(pairs)]


def _inv_freq(case):
    """Angle per position of each pair: base 10000 within the pair's axis."""
    axis = _axis_of_pairs(case)
    out, seen = [], {}
    for a in axis:
        i = seen.get(a, 0)
        seen[a] = i + 1
        out.append(10000.0 ** (-i / axis.count(a)))
    return out


def _table(case, tokens, g):
    """Pages of each sequence in scrambled order, -1 behind the last one."""
    page = case["page"]
    need = [-(-n // page) for n in tokens]
    width, pages = max(need), sum(need) + 2
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)
    have = torch.tensor(need, device=DEV)
    start = torch.cumsum(have, 0) - have
    at = (start[:, None] + col).clamp_(max=pages - 1)
    return torch.where(col < have[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32)), pages


def _power(amax):
    """The exponent e of the smallest scale 2^e that keeps amax within 448."""
    f, x = torch.frexp(amax)
    return (x - 9 + (f > 0.875).to(x.dtype)).clamp(-126, 120)


def _to_8_bits(x):
    """x [..., d] -> (codes, one exponent byte per row)."""
    e = _power(x.abs().amax(-1))
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _pool(case, pages, g):
    """A cache's pages as earlier steps left them."""
    shape = (pages, case["Hk"], case["page"], case["d"])
    made = []
    for scale in (1.0, 0.5):
        x = _rnd(g, *shape) * scale
        x *= torch.exp(0.5 * _rnd(g, *shape[:3], 1))
        if case["cache"] == "e4m3":
            made += _to_8_bits(x)
        else:
            made += [x.to(TYPES[case["cache"]]), None]
    return made


def _tree(case, seed):
    """Ancestor masks of random trees: node i hangs below an earlier node or the context."""
    B, T = case["B"], case["T"]
    r = np.random.RandomState(seed % (1 << 31))
    m = np.zeros((B, T, T), dtype=bool)
    at = np.arange(B)
    for i in range(T):
        p = np.maximum(r.randint(-1, i, size=B) if i else np.full(B, -1), i - 4 if i > 4 else -1)
        m[:, i] = np.where((p >= 0)[:, None], m[at, p], False)
        m[:, i, i] = True
    return torch.from_numpy(m).to(DEV)


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    dt = TYPES[c["dtype"]]
    s = State(case=c)
    if own:
        import long_context_ra_gb300 as ra

        s.update(ra=ra)
    if c["kind"] in ("norm", "norm_backward"):
        B, N, Hq, Hk, d = c["B"], c["N"], c["Hq"], c["Hk"], c["d"]
        # heads of one projection of every token: views, as the matrix product leaves them
        both = (_rnd(g, B, N, Hq + Hk, d) * 1.5).to(dt)
        s.update(q=both[:, :, :Hq].transpose(1, 2), k=both[:, :, Hq:].transpose(1, 2))
        s.update(wq=(1 + 0.1 * _rnd(g, d)).to(dt) if c["norm"] else None,
                 wk=(1 + 0.1 * _rnd(g, d)).to(dt) if c["norm"] else None)
        far = torch.randint(0, c["far"], (c["axes"], B, 1), generator=g, device=DEV)
        s.update(positions=(far + torch.arange(N, device=DEV)).contiguous())
        s.update(inv_freq=torch.tensor(_inv_freq(c), dtype=torch.float64, device=DEV),
                 axis=torch.tensor(_axis_of_pairs(c), device=DEV))
        if own:
            s.update(rope=s.ra.new_rope(_inv_freq(c), axis=_axis_of_pairs(c), interleaved=c["interleaved"]))
        if c["kind"] == "norm":
            s.update(q_out=torch.empty(B, Hq, N, d, dtype=dt, device=DEV),
                     k_out=torch.empty(B, Hk, N, d, dtype=dt, device=DEV))
        else:
            s.update(dq_out=_rnd(g, B, Hq, N, d).to(dt), dk_out=_rnd(g, B, Hk, N, d).to(dt))
        return s
    lens = _lens(c)
    counts = [0] * c["B"] if c["kind"] == "read" else _counts(c)
    table, pages = _table(c, [n + t for n, t in zip(lens, counts)], g)
    pool = _pool(c, pages, g)
    s.update(table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), pool=pool)
    if c["kind"] != "read":
        s.update(count=torch.tensor(counts, dtype=torch.int32, device=DEV) if c["ragged"] else None)
    if own:
        s.update(cache=s.ra.RaCache(k=pool[0], v=pool[2], k_exp=pool[1], v_exp=pool[3]))
    if c["kind"] == "write":
        new = _rnd(g, c["B"], c["T"], 2 * c["Hk"], c["d"]) * torch.exp(0.5 * _rnd(g, c["B"], c["T"], 2 * c["Hk"], 1))
        new = new.to(dt).transpose(1, 2)  # [B, heads of k and v, T, d], a view
        s.update(k=new[:, : c["Hk"]], v=new[:, c["Hk"]:])
    elif c["kind"] == "read":
        shape = (c["B"], c["Hk"], c["n"], c["d"])
        s.update(k=torch.empty(shape, dtype=dt, device=DEV), v=torch.empty(shape, dtype=dt, device=DEV))
    else:
        B, T, Hq = c["B"], c["T"], c["Hq"]
        s.update(q=(_rnd(g, B, Hq, T, c["d"]) * 1.5).to(dt), mask=_tree(c, seed) if c["mask"] == "tree" else None)
        if own:
            n = s.ra.ra_cache_attention_workspace_bytes(B, Hq, c["Hk"], T, c["d"])
            s.update(out=torch.empty_like(s.q), lse=torch.empty(B, Hq, T, device=DEV),
                     workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    return s


# ----------------------------------------------------------- the plain forms
def _pairs(x, case):
    r = case["rot"]
    if case["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2]
    return x[..., : r // 2], x[..., r // 2: r]


def _unpair(a, b, rest, case):
    if case["interleaved"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _angles(s):
    """Cosine and sine per token and pair, the angle taken in 64 bits."""
    pos = s.positions[s.axis]  # [pairs, B, N]
    a = (pos.double() * s.inv_freq[:, None, None]).permute(1, 2, 0)[:, None]  # [B, 1, N, pairs]
    return a.cos().float(), a.sin().float()


def _plain_norm(x, w, cos, sin, case):
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    a, b = _pairs(x, case)
    return _unpair(a * cos - b * sin, b * cos + a * sin, x[..., case["rot"]:], case)


def _plain_norm_backward(x, w, dy, cos, sin, case):
    x, dy = x.float(), dy.float()
    a, b = _pairs(dy, case)
    dz = _unpair(a * cos + b * sin, b * cos - a * sin, dy[..., case["rot"]:], case)
    if not case["norm"]:
        return dz, None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    dn = dz * w.float()
    dx = r * dn - x * (r * r * r) * (dn * x).mean(-1, keepdim=True)
    return dx, (dz * x * r).sum((0, 1, 2), dtype=torch.float64).float()


def _positions_in_cache(s, t0, n):
    """Page and place of positions t0[b] .. t0[b] + n - 1 (clamped into the table)."""
    page = s.case["page"]
    at = t0[:, None].long() + torch.arange(n, device=DEV)
    col = (at // page).clamp_(max=s.table.shape[1] - 1)
    return at, s.table.long().gather(1, col), at % page


def _plain_write(s):
    c = s.case
    _, pages, place = _positions_in_cache(s, s.lens, c["T"])
    live = torch.arange(c["T"], device=DEV) < (s.count[:, None] if s.count is not None else c["T"])
    pages, place = pages[live], place[live]
    for x, held, exps in ((s.k, s.pool[0], s.pool[1]), (s.v, s.pool[2], s.pool[3])):
        x = x.transpose(1, 2)[live].float()  # [tokens, heads, d]
        if exps is None:
            held[pages, :, place] = x.to(held.dtype)
        else:
            codes, e = _to_8_bits(x)
            held.view(torch.uint8)[pages, :, place] = codes.view(torch.uint8)
            exps[pages, :, place] = e
    return [t for t in s.pool if t is not None]


def _gathered(held, exps, pages, place):
    """Rows of the cache at the given pages and places, in 32 bits: [B, heads, n, d]."""
    if exps is None:
        return held[pages, :, place].permute(0, 2, 1, 3).float()
    x = held.view(torch.uint8)[pages, :, place].view(torch.float8_e4m3fn).float()
    return torch.ldexp(x, exps[pages, :, place].int()[..., None] - 127).permute(0, 2, 1, 3)


def _plain_read(s):
    c = s.case
    at, pages, place = _positions_in_cache(s, torch.full_like(s.lens, c["first"]), c["n"])
    live = (at < s.lens[:, None])[:, None, :, None]
    pages = pages.clamp(min=0)
    dt = TYPES[c["dtype"]]
    return [torch.where(live, _gathered(x, e, pages, place), 0.0).to(dt)
            for x, e in ((s.pool[0], s.pool[1]), (s.pool[2], s.pool[3]))]


def _plain_attend(s):
    c = s.case
    B, T, Hq, Hk, d = c["B"], c["T"], c["Hq"], c["Hk"], c["d"]
    n = c["longest"] + T
    at, pages, place = _positions_in_cache(s, torch.zeros_like(s.lens), n)
    count = s.count if s.count is not None else torch.full_like(s.lens, T)
    pages = pages.clamp(min=0)
    k = _gathered(s.pool[0], s.pool[1], pages, place)
    v = _gathered(s.pool[2], s.pool[3], pages, place)
    q = s.q.float().reshape(B, Hk, (Hq // Hk) * T, d)
    # key at position p: the context is seen by all, drafted tokens by the mask
    draft = at - s.lens[:, None]  # [B, n]
    seen = s.mask if s.mask is not None else torch.ones(T, T, dtype=torch.bool, device=DEV).tril().expand(B, T, T)
    seen = seen.gather(2, draft.clamp(0, T - 1)[:, None].expand(B, T, n))
    seen = (draft < 0)[:, None] | (seen & (draft < count[:, None])[:, None])
    live = torch.arange(T, device=DEV) < count[:, None]  # [B, T]
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(B, Hk, Hq // Hk, T, n)
    scores.masked_fill_(~(seen & live[:, :, None])[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hk, -1, n), v).view(B, Hk, Hq // Hk, T, d)
    out = torch.where(total > 0, out / total, 0.0).view(B, Hq, T, d)
    lse = (top + total.log()).view(B, Hq, T)
    return [out.to(s.q.dtype), lse]


# --------------------------------------------------------------- one pass
def run(s):
    c = s.case
    if c["kind"] == "norm":
        eps = EPS if c["norm"] else None
        if own:
            return s.ra.ra_qk_norm_rope(s.q, s.k, s.rope, s.positions, s.wq, s.wk, eps, q_out=s.q_out, k_out=s.k_out)
        cos, sin = _angles(s)
        return [s.q_out.copy_(_plain_norm(s.q, s.wq, cos, sin, c)), s.k_out.copy_(_plain_norm(s.k, s.wk, cos, sin, c))]
    if c["kind"] == "norm_backward":
        eps = EPS if c["norm"] else None
        if own:
            return s.ra.ra_qk_norm_rope_backward(s.q, s.k, s.dq_out, s.dk_out, s.rope, s.positions, s.wq, s.wk, eps)
        cos, sin = _angles(s)
        dq, dwq = _plain_norm_backward(s.q, s.wq, s.dq_out, cos, sin, c)
        dk, dwk = _plain_norm_backward(s.k, s.wk, s.dk_out, cos, sin, c)
        return [dq.to(s.q.dtype), dk.to(s.k.dtype), dwq, dwk]
    if c["kind"] == "write":
        if own:
            s.ra.ra_cache_write(s.cache, s.k, s.v, s.table, s.lens, s.count)
            return [t for t in s.pool if t is not None]
        return _plain_write(s)
    if c["kind"] == "read":
        if own:
            return s.ra.ra_cache_read(s.cache, s.table, s.lens, c["first"], c["n"], k=s.k, v=s.v)
        return _plain_read(s)
    if own:
        return s.ra.ra_cache_attention(s.q, s.cache, s.table, s.lens, s.count, s.mask, out=s.out, lse=s.lse,
                                       workspace=s.workspace)
    return _plain_attend(s)


# ------------------------------------------------------- the same in 64 bits
def _exact_rotation(s, sign):
    c = s.case
    turn = torch.stack([s.positions[a].double() * f for a, f in zip(_axis_of_pairs(c), _inv_freq(c))], -1)
    turn = torch.polar(torch.ones_like(turn), sign * turn)[:, None]

    def rotate(x):
        r = c["rot"]
        first = x[..., :r]
        z = first.unflatten(-1, (r // 2, 2)) if c["interleaved"] else first.unflatten(-1, (2, r // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        z = z if c["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., r:]], -1)

    return rotate


def _exact_norm(s):
    rotate, out = _exact_rotation(s, 1.0), []
    for x, w in ((s.q, s.wq), (s.k, s.wk)):
        x = x.double()
        if w is not None:
            x = x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
        out.append(rotate(x))
    return out


def _exact_norm_backward(s):
    back, grads, weights = _exact_rotation(s, -1.0), [], []
    for x, w, dy in ((s.q, s.wq, s.dq_out), (s.k, s.wk, s.dk_out)):
        dz = back(dy.double())
        if w is None:
            grads.append(dz)
            weights.append(None)
            continue
        x = x.double()
        size = ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        unit = x / size
        weights.append((dz * unit).sum((0, 1, 2)))
        dn = dz * w.double()
        grads.append((dn - unit * (dn * unit).sum(-1, keepdim=True) / x.shape[-1]) / size)
    return grads + weights


def _exact_codes(x):
    """8-bit values (nearest, ties to even) and exponent bytes of rows of x."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 448)).clamp(-126, 120)
    e = torch.where(torch.exp2(e) * 448 < top, e + 1, torch.where(torch.exp2(e - 1) * 448 >= top, e - 1, e))
    e = e.clamp(-126, 120)
    y = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, (e[..., 0] + 127).to(torch.uint8)


def _exact_write(s):
    c, out = s.case, []
    counts = s.count.tolist() if s.count is not None else [c["T"]] * c["B"]
    table, page = s.table.cpu().numpy(), c["page"]
    for x, held, exps in ((s.k, s.pool[0], s.pool[1]), (s.v, s.pool[2], s.pool[3])):
        vals = held.float() if exps is not None else held.clone()
        marks = exps.clone() if exps is not None else None
        for b, (n, t) in enumerate(zip(s.lens.tolist(), counts)):
            at = np.arange(n, n + t)
            pages = torch.from_numpy(table[b, at // page].astype(np.int64)).to(DEV)
            place = torch.from_numpy(at % page).to(DEV)
            rows = x[b, :, :t].transpose(0, 1)
            if exps is None:
                vals[pages, :, place] = rows.to(vals.dtype)
            else:
                codes, e = _exact_codes(rows.double())
                vals[pages, :, place] = codes.float()
                marks[pages, :, place] = e
        out += [vals] + ([marks] if marks is not None else [])
    return out


def _sequence(s, b, tokens, side):
    """Rows 0 .. tokens - 1 of sequence b in 64 bits: [heads, tokens, d]."""
    held, exps = s.pool[2 * side], s.pool[2 * side + 1]
    pages = s.table[b, : -(-tokens // s.case["page"])].long()
    x = held[pages].double()
    if exps is not None:
        x = x * torch.exp2(exps[pages].double()[..., None] - 127)
    return x.transpose(0, 1).reshape(s.case["Hk"], -1, s.case["d"])[:, :tokens]


def _exact_read(s):
    c, out = s.case, []
    for side in (0, 1):
        x = torch.zeros(c["B"], c["Hk"], c["n"], c["d"], dtype=torch.float64, device=DEV)
        for b, n in enumerate(s.lens.tolist()):
            seen = min(n, c["first"] + c["n"])
            if seen > c["first"]:
                x[b, :, : seen - c["first"]] = _sequence(s, b, seen, side)[:, c["first"]:]
        out.append(x)
    return out


def _exact_attend(s):
    c = s.case
    B, T, Hq, Hk, d = c["B"], c["T"], c["Hq"], c["Hk"], c["d"]
    g = Hq // Hk
    out = torch.zeros(B, Hq, T, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    counts = s.count.tolist() if s.count is not None else [T] * B
    for b, (n, t) in enumerate(zip(s.lens.tolist(), counts)):
        k, v = _sequence(s, b, n + t, 0), _sequence(s, b, n + t, 1)
        sees = s.mask[b, :t, :t] if s.mask is not None else torch.ones(t, t, device=DEV).tril() > 0
        for h in range(Hk):
            x = s.q[b, h * g: (h + 1) * g, :t].double().reshape(g * t, d) @ k[h].T / math.sqrt(d)
            x.view(g, t, n + t)[:, :, n:].masked_fill_(~sees, -math.inf)
            top = x.amax(-1, keepdim=True)
            p = (x - top).exp()
            total = p.sum(-1, keepdim=True)
            out[b, h * g: (h + 1) * g, :t] = (p @ v[h] / total).view(g, t, d)
            lse[b, h * g: (h + 1) * g, :t] = (top + total.log()).view(g, t)
    return [out, lse]


def exact(case, seed):
    if work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "write": _exact_write, "read": _exact_read,
            "attend": _exact_attend}[case["kind"]](s)
