"""Cases of the operators that carry several continuations of one context:
attention of sequences that share a prefix of a paged K/V cache, the forks of
sequences and the moves of their pages and rows, and the verification of
drafted tokens.

Each case has a plain form in elementary torch operations and the calls a
program makes of the library (`own`); `exact` evaluates the definitions in 64
bits.  Attention tensors are [B, H, T, d]; a cache holds pages of
[heads, page, d], reached through a table of page numbers per sequence.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of each of 3 continuations of a short prompt: the smallest call
        dict(name="attend few", kind="attend", dtype="bf16", cache="bf16", B=3, groups=1, T=1, Hq=8, Hk=2, d=64,
             page=16, prefix=1021, tail=77, ragged=False, mask="causal"),
        # a decode step of 32 samples that were drawn from one long prompt
        dict(name="attend samples", kind="attend", dtype="bf16", cache="bf16", B=32, groups=1, T=1, Hq=32, Hk=8,
             d=128, page=64, prefix=32768, tail=1024, ragged=True, mask="causal"),
        # a serving batch over an 8-bit cache: 6 instructions of unlike length, each before many requests
        dict(name="attend instructions", kind="attend", dtype="bf16", cache="e4m3", B=96, groups=6, T=1, Hq=32, Hk=8,
             d=128, page=64, prefix=16384, tail=2048, ragged=True, mask="causal"),
        # trees of 32 drafted tokens for 24 samples of one context
        dict(name="attend trees", kind="attend", dtype="bf16", cache="bf16", B=24, groups=1, T=32, Hq=32, Hk=8,
             d=128, page=128, prefix=65536, tail=512, ragged=True, mask="tree"),
        # the 32-bit path: beams of a few tokens, a head width of no special size
        dict(name="attend f32", kind="attend", dtype="f32", cache="f32", B=10, groups=2, T=3, Hq=6, Hk=3, d=80,
             page=16, prefix=2048, tail=129, ragged=True, mask="tree"),
        # 4 samples are started from one prompt
        dict(name="fork one", kind="fork", cache="bf16", B=1, n=4, T=1, heads=2, d=64, page=16, longest=1021),
        # a beam step: 96 beams of 32 prompts, each with room for a tree of drafts
        dict(name="fork beams", kind="fork", cache="bf16", B=32, n=96, T=32, heads=8, d=128, page=64, longest=16384),
        # the kept drafts of a few sequences move together
        dict(name="compact few", kind="compact", cache="bf16", B=3, T=9, heads=2, d=64, page=16, longest=1021),
        # the same after the trees of a large batch over an 8-bit cache
        dict(name="compact trees", kind="compact", cache="e4m3", B=192, T=64, heads=8, d=128, page=64, longest=4096),
        # a chain of 4 tokens of one sequence, drawn by a small model: the latency of a step
        dict(name="verify one", kind="verify", dtype="f32", B=1, T=5, V=32768, tree=False, draft=True),
        # chains of a large batch
        dict(name="verify batch", kind="verify", dtype="f32", B=128, T=6, V=131072, tree=False, draft=True),
        # trees of chosen tokens, a vocabulary of odd size
        dict(name="verify trees", kind="verify", dtype="bf16", B=32, T=32, V=100003, tree=True, draft=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw(rng):
    kind = rng.choice(["attend", "attend", "fork", "compact", "verify"])
    if kind == "verify":
        return dict(kind=kind, dtype=rng.choice(["bf16", "f32"]), B=_log(rng, 1, 128), T=_log(rng, 1, 64),
                    V=_log(rng, 100, 200000), tree=rng.random() < 0.5, draft=rng.random() < 0.5)
    cache = rng.choice(["bf16", "f32", "e4m3"])
    if kind == "fork":
        return dict(kind=kind, cache=cache, B=_log(rng, 1, 64), n=_log(rng, 1, 256), T=_log(rng, 1, 300),
                    heads=_log(rng, 1, 16), d=8 * rng.randint(2, 32), page=2 ** rng.randint(3, 8),
                    longest=_log(rng, 1, 16384))
    if kind == "compact":
        return dict(kind=kind, cache=cache, B=_log(rng, 1, 192), T=_log(rng, 1, 128), heads=_log(rng, 1, 16),
                    d=8 * rng.randint(2, 32), page=2 ** rng.randint(3, 8), longest=_log(rng, 1, 4096))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hk, B = _log(rng, 1, 16), _log(rng, 1, 96)
    return dict(kind=kind, dtype=dtype, cache=rng.choice([dtype, "e4m3"]), B=B,
                groups=min(B, _log(rng, 1, 8)), T=_log(rng, 1, 64), Hq=Hk * rng.randint(1, 8), Hk=Hk,
                d=rng.choice([64, 128]) if dtype == "bf16" else 8 * rng.randint(2, 32), page=2 ** rng.randint(4, 8),
                prefix=_log(rng, 16, 131072), tail=_log(rng, 1, 4096), ragged=rng.random() < 0.75,
                mask=rng.choice(["causal", "tree"]))


def draw(rng):
    while True:
        c = _draw(rng)
        if c["kind"] == "attend":
            # the plain form's scores and gathered rows stay below those of the largest listed case
            keys = c["B"] * (c["prefix"] + c["tail"] + c["T"])
            if keys * max(c["T"] * c["Hq"], c["Hk"] * c["d"]) > 1.7e9 or work(c)["flops"] > 8e11:
                continue
            if c["dtype"] == "f32" and work(c)["flops"] > 5e10:
                continue
        elif c["kind"] == "verify":
            if c["B"] * c["T"] * c["V"] > 1.1e8:
                continue
        elif c["B"] * c["longest"] * c["heads"] * c["d"] > 8.5e8 or work(c)["bytes"] > 2e8:
            continue
        return c


def _prefixes(case):
    """Tokens that the sequences of each group have in common."""
    G, L = case["groups"], case["prefix"]
    if not case["ragged"]:
        return [L] * G
    return [max(1, L - (L * 5 * g) // (8 * G) - (13 * g) % 29) for g in range(G)]


def _group_of(case):
    """The group of each sequence: runs, of unlike length where they are ragged."""
    B, G = case["B"], case["groups"]
    power = 1.5 if case["ragged"] else 1.0
    first = [max(g, int(B * (g / G) ** power)) for g in range(G)]
    return [sum(f <= b for f in first) - 1 for b in range(B)]


def _lens(case):
    """Tokens in the cache before the call, per sequence."""
    B = case["B"]
    if case["kind"] == "attend":
        tail = case["tail"]
        own_part = [tail if not case["ragged"] else max(0, tail - (tail * b) // B - (7 * b) % 5) for b in range(B)]
        pre = _prefixes(case)
        return [pre[g] + t for g, t in zip(_group_of(case), own_part)]
    L = case["longest"]
    return [max(1, L - (L * 7 * b) // (8 * B) - (13 * b) % 29) for b in range(B)]


def _counts(case):
    """New tokens per sequence: all T for the first, fewer for some others."""
    B, T = case["B"], case["T"]
    if not case.get("ragged", True):
        return [T] * B
    return [max(1, T - (T * (b % 4)) // 6) for b in range(B)]


def _sources(case):
    """The sequence that each fork continues: all in turn, some more than once."""
    return [(i * 5 // 3 if i % 7 else i) % case["B"] for i in range(case["n"])]


def _kept(case):
    """Drafts that stay per sequence, the first token among them: none to half of the tree."""
    return [1 + (b * 5 + 2) % max(1, (case["T"] + 1) // 2) for b in range(case["B"])]


def work(case):
    c = case
    if c["kind"] == "verify":
        # the rows at which each sequence stops
        return {"bytes": c["B"] * c["V"] * SIZE[c["dtype"]] * (2 if c["draft"] else 1), "flops": 2.0 * c["B"] * c["V"]}
    heads, d, s = c.get("heads") or c["Hk"], c["d"], SIZE[c["cache"]]
    held = d * s + (1 if c["cache"] == "e4m3" else 0)  # one row of the cache
    lens = _lens(c)
    if c["kind"] == "fork":
        at = [lens[b] for b in _sources(c)]
        partial = sum(n % c["page"] != 0 for n in at)
        columns = sum(-(-(n + c["T"]) // c["page"]) for n in at)
        return {"bytes": 4 * heads * partial * c["page"] * held + 4 * (3 * columns + c["n"] * 8), "flops": 0.0}
    if c["kind"] == "compact":
        moved = sum(k - 1 for k in _kept(c))
        return {"bytes": 4 * heads * moved * held + c["B"] * 8 + 4 * sum(_kept(c)), "flops": 0.0}
    g, of, cnt, pre = c["Hq"] // heads, _group_of(c), _counts(c), _prefixes(c)
    keys = sum(pre) + sum(n - pre[x] + t for n, x, t in zip(lens, of, cnt))
    pairs = sum(t * (n + (t + 1) / 2) for n, t in zip(lens, cnt))
    return {"bytes": 2 * heads * keys * held + c["B"] * c["Hq"] * c["T"] * (2 * d * SIZE[c["dtype"]] + 4),
            "flops": 4.0 * heads * g * pairs * d}


# ------------------------------------------------------------- their inputs
class State(dict):
    __getattr__ = dict.__getitem__


def _rnd(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _table(case, tokens, g, spare=2, columns=0, skip=None):
    """Pages of each sequence in scrambled order (none for the first `skip`
    columns), -1 elsewhere; their number, and that of all pages."""
    page = case["page"]
    need = [-(-n // page) for n in tokens]
    skip = torch.tensor(skip or [0] * len(need), device=DEV)
    have = torch.tensor(need, device=DEV)
    width, pages = max(max(need), columns), int((have - skip).sum()) + spare
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)
    start = torch.cumsum(have - skip, 0) - have
    at = (start[:, None] + col).clamp_(0, pages - 1)
    there = (col >= skip[:, None]) & (col < have[:, None])
    return torch.where(there, order[at], torch.full_like(at, -1, dtype=torch.int32)), need, pages


def _to_8_bits(x):
    """x [..., d] -> (codes, one exponent byte per row): the smallest scale 2^e that keeps the row within 448."""
    f, e = torch.frexp(x.abs().amax(-1))
    e = (e - 9 + (f > 0.875).to(e.dtype)).clamp(-126, 120)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _pool(case, pages, heads, g):
    """A cache's pages as earlier steps left them."""
    shape = (pages, heads, case["page"], case["d"])
    made = []
    for scale in (1.0, 0.5):
        x = _rnd(g, *shape) * scale
        x *= torch.exp(0.5 * _rnd(g, *shape[:3], 1))
        made += _to_8_bits(x) if case["cache"] == "e4m3" else [x.to(TYPES[case["cache"]]), None]
    return made


def _tree(case, seed):
    """Parents of the nodes of random trees [B, T] and their ancestor masks.
    Node 0 hangs below the context, every other one below an earlier node."""
    B, T = case["B"], case["T"]
    r = np.random.RandomState(seed % (1 << 31))
    parent = np.full((B, T), -1, dtype=np.int32)
    m = np.zeros((B, T, T), dtype=bool)
    at = np.arange(B)
    for i in range(T):
        if i:
            parent[:, i] = r.randint(max(0, i - 4), i, size=B)
            m[:, i] = m[at, parent[:, i]]
        m[:, i, i] = True
    return parent, torch.from_numpy(m).to(DEV)


def _bytes_of(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    s = State(case=c)
    if own:
        import long_context_ra_gb300 as ra

        s.update(ra=ra)
    if c["kind"] == "verify":
        return _prepare_verify(s, g, seed)
    heads = c.get("heads") or c["Hk"]
    lens = _lens(c)
    s.update(lens=_int(lens))
    if c["kind"] == "fork":
        # parents, and free pages for every fork: its partial page and its new tokens
        at = [lens[b] for b in _sources(c)]
        table, need, pages = _table(c, lens, g, spare=sum((n + c["T"]) // c["page"] + 1 - n // c["page"] for n in at),
                                    columns=-(-(max(lens) + c["T"]) // c["page"]))
        ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
        ref[table[table >= 0].long()] = 1
        n = c["n"]
        s.update(table=table, held=_int(need), ref=ref, source=_int(_sources(c)),
                 table_out=torch.full((n, table.shape[1]), -1, dtype=torch.int32, device=DEV),
                 held_out=_int([0] * n), lens_out=_int([-1] * n), granted=_int([0] * n), src=_int([-1] * n),
                 dst=_int([-1] * n))
    else:
        of = _group_of(c) if c["kind"] == "attend" else list(range(c["B"]))
        lead = [of.index(x) for x in of]
        common = [_prefixes(c)[x] if c["kind"] == "attend" else 0 for x in of]
        # whole pages of a prefix are the first sequence's
        table, need, pages = _table(c, [n + c["T"] for n in lens], g,
                                    skip=[0 if b == x else m // c["page"] for b, (x, m) in enumerate(zip(lead, common))])
    pool = _pool(c, pages, heads, g)
    s.update(pool=pool)
    if c["kind"] == "compact":
        # the path of a tree: node 0, then later nodes in order; none for some (a chain that was kept as it lies)
        kept, T = _kept(c), c["T"]
        r = np.random.RandomState(seed % (1 << 31))
        path = np.full((c["B"], T), -1, dtype=np.int32)
        for b, k in enumerate(kept):
            path[b, :k] = np.arange(k)
            if b % 5 != 4 and k > 1:
                path[b, 1:k] = np.sort(r.choice(np.arange(k, T), k - 1, replace=False)) if T - k >= k - 1 else path[b, 1:k]
        s.update(path=torch.from_numpy(path).to(DEV), kept=_int(kept))
    elif c["kind"] == "attend":
        lead, common = torch.tensor(lead, device=DEV), torch.tensor(common, device=DEV)
        col = torch.arange(table.shape[1], device=DEV)
        first = table[lead]
        table = torch.where(col < (common // c["page"])[:, None], first, table)
        # the last, partial page of a prefix is a copy of the first sequence's
        part = (col == (common // c["page"])[:, None]) & (common % c["page"] != 0)[:, None] & (first != table)
        to, source = table[part].long(), first[part].long()
        for x in pool:
            if x is not None:
                _bytes_of(x)[to] = _bytes_of(x)[source]
        B, T, Hq = c["B"], c["T"], c["Hq"]
        s.update(shared=torch.where(lead == torch.arange(B, device=DEV), 0, common).to(torch.int32),
                 count=_int(_counts(c)) if c["ragged"] else None,
                 q=(_rnd(g, B, Hq, T, c["d"]) * 1.5).to(TYPES[c["dtype"]]),
                 mask=_tree(c, seed)[1] if c["mask"] == "tree" else None)
        if own:
            n = s.ra.ra_cache_attention_shared_workspace_bytes(B, Hq, heads, T, c["d"])
            s.update(out=torch.empty_like(s.q), lse=torch.empty(B, Hq, T, device=DEV),
                     workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    if c["kind"] != "fork":
        s.update(table=table)
    if own:
        s.update(cache=s.ra.RaCache(k=pool[0], v=pool[2], k_exp=pool[1], v_exp=pool[3]))
    return s


def _prepare_verify(s, g, seed):
    """Distributions of a model over the next token behind every node, those of a
    smaller model that resembles it, and tokens that the smaller one drew."""
    c = s.case
    B, T, V = c["B"], c["T"], c["V"]
    dt = TYPES[c["dtype"]]
    logits = _rnd(g, B, T, V) * 4
    s.update(probs=torch.softmax(logits, -1).to(dt))
    small = torch.softmax(logits.add_(_rnd(g, B, T, V), alpha=0.7), -1).to(dt)
    parent = _tree(c, seed)[0] if c["tree"] else np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1))
    parent = torch.from_numpy(parent).to(DEV)
    rows = torch.arange(B, device=DEV)[:, None] * T + parent.clamp(min=0)
    # drawn by the largest of q / e, e from an exponential distribution
    e = torch.empty(V, device=DEV).exponential_(generator=g)
    flat, tokens = small.view(B * T, V), []
    for lot in torch.chunk(torch.arange(B * T, device=DEV), -(-B * T // 256)):
        shift = torch.randint(0, V, (1,), generator=g, device=DEV)
        draw_of = e[(torch.arange(V, device=DEV) + shift + 7919 * lot[:, None]) % V]
        tokens.append((flat[rows.view(-1)[lot]].float() / draw_of).argmax(-1))
    s.update(tokens=torch.cat(tokens).view(B, T), uniform=torch.rand(B, T, generator=g, device=DEV),
             parent=parent if c["tree"] else None, draft=small if c["draft"] else None,
             count=_int(_counts(c)) if c["tree"] else None)
    if own:
        s.update(path=torch.empty(B, T, dtype=torch.int32, device=DEV), kept=_int([0] * B),
                 token=torch.empty(B, dtype=torch.int64, device=DEV))
    return s


# ----------------------------------------------------------- the plain forms
def _positions(s, t0, n):
    """Page and place of positions t0[b] .. t0[b] + n - 1 (clamped into the table)."""
    page = s.case["page"]
    at = t0[:, None].long() + torch.arange(n, device=DEV)
    col = (at // page).clamp_(max=s.table.shape[1] - 1)
    return at, s.table.long().gather(1, col), at % page


def _gathered(held, exps, pages, place):
    """Rows of the cache at the given pages and places, in 32 bits: [B, heads, n, d]."""
    if exps is None:
        return held[pages, :, place].permute(0, 2, 1, 3).float()
    x = held.view(torch.uint8)[pages, :, place].view(torch.float8_e4m3fn).float()
    return torch.ldexp(x, exps[pages, :, place].int()[..., None] - 127).permute(0, 2, 1, 3)


def _plain_attend(s):
    c = s.case
    B, T, Hq, Hk, d = c["B"], c["T"], c["Hq"], c["Hk"], c["d"]
    n = c["prefix"] + c["tail"] + T
    at, pages, place = _positions(s, torch.zeros_like(s.lens), n)
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


def _plain_fork(s):
    """The forks of the last step go, new ones take their place and get room for T tokens."""
    c = s.case
    page, n, T = c["page"], c["n"], c["T"]
    width, pages = s.table.shape[1], s.ref.numel()
    col = torch.arange(width, device=DEV)
    one = torch.ones((), dtype=torch.int32, device=DEV)

    def held_by(table, held):
        """One at every page in the first `held` columns, the others in a place of their own."""
        return torch.where(col < held[:, None], table.long(), pages).flatten()

    def change(at, by):
        wide = torch.zeros(pages + 1, dtype=torch.int32, device=DEV)
        s.ref += wide.index_add_(0, at, (one * by).expand(at.numel()))[:pages]

    change(held_by(s.table_out, s.held_out), -1)
    source = s.source.long()
    s.lens_out.copy_(s.lens[source])
    held = (s.lens_out + page - 1) // page
    s.table_out.copy_(torch.where(col < held[:, None], s.table[source], -1))
    change(held_by(s.table_out, held), 1)
    # room: the page that the first new token falls into is replaced where others hold it too
    first, last = s.lens_out // page, (s.lens_out + T + page - 1) // page
    own_col = first.long().clamp(max=width - 1)[:, None]
    present = s.table_out.gather(1, own_col)[:, 0].long()
    inside = first < held
    at = torch.where(inside, present, pages)
    holders = torch.cat([s.ref, torch.zeros_like(s.ref[:1])])
    index = torch.arange(n, device=DEV)
    asking = torch.zeros(pages + 1, dtype=torch.int32, device=DEV).index_add_(0, at, one.expand(n))
    latest = torch.full((pages + 1,), -1, device=DEV).scatter_reduce_(0, at, index, "amax")
    keeps = (asking[at] == holders[at]) & (latest[at] == index)
    replaced = inside & (holders[at] > 1) & ~keeps
    fresh = (last - held).clamp(min=0)
    need = fresh + replaced
    upto = torch.cumsum(need, 0)
    free = torch.cumsum(s.ref == 0, 0)
    enough = (upto[-1] <= free[-1])
    # the k-th wanted page is the k-th free one
    k = torch.where(col >= held[:, None], (upto - need + replaced)[:, None] + col - held[:, None], -1)
    k = torch.where((col == first[:, None]) & replaced[:, None], (upto - need)[:, None], k)
    k = torch.where((col < last[:, None]) & enough, k, -1)
    got = torch.searchsorted(free, k.flatten() + 1).view(n, width).to(torch.int32)
    got = torch.where(k >= 0, got, -1)
    s.src.copy_(torch.where(replaced & enough & (s.lens_out % page != 0), present, -1))
    taken = replaced & enough
    change(torch.where(taken, at, pages), -1)
    change(torch.where(got >= 0, got.long(), pages).flatten(), 1)
    s.table_out.copy_(torch.where(got >= 0, got, s.table_out))
    s.dst.copy_(torch.where(s.src >= 0, s.table_out.gather(1, own_col)[:, 0], -1))
    s.granted.copy_(torch.where(enough, T, 0).expand(n))
    s.held_out.copy_(torch.where(enough, torch.maximum(held, last), held))
    copied = s.src >= 0
    to, of = s.dst[copied].long(), s.src[copied].long()
    for x in s.pool:
        if x is not None:
            _bytes_of(x)[to] = _bytes_of(x)[of]
    return _fork_results(s)


def _fork_results(s):
    return [s.ref, s.table_out, s.held_out, s.lens_out, s.granted, s.src, s.dst] + [t for t in s.pool if t is not None]


def _plain_compact(s):
    c = s.case
    live = torch.arange(c["T"], device=DEV) < s.kept[:, None]
    _, to, to_place = _positions(s, s.lens, c["T"])
    at = s.lens[:, None].long() + s.path.clamp(min=0)
    of, of_place = s.table.long().gather(1, at // c["page"]), at % c["page"]
    for x in s.pool:
        if x is not None:
            x = _bytes_of(x)
            x[to[live], :, to_place[live]] = x[of[live], :, of_place[live]]
    return [t for t in s.pool if t is not None]


def _plain_verify(s):
    c = s.case
    B, T, V = c["B"], c["T"], c["V"]
    b = torch.arange(B, device=DEV)
    count = s.count if s.count is not None else torch.full((B,), T, device=DEV)
    node = torch.zeros(B, dtype=torch.long, device=DEV)
    scale = torch.zeros(B, dtype=torch.float64, device=DEV)   # how much of the draft's row was taken away
    total = torch.ones(B, dtype=torch.float64, device=DEV)    # of what is left
    gone = torch.zeros(B, V, dtype=torch.bool, device=DEV)    # chosen tokens that were refused
    path = torch.full((B, T), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    kept = torch.ones(B, dtype=torch.long, device=DEV)

    def left():
        row = s.probs[b, node].double()
        if s.draft is None:
            return torch.where(gone, 0.0, row)
        return (row - scale[:, None] * s.draft[b, node].double()).clamp(min=0)

    # the decisions follow one another: each depends on those before it
    for t in range(1, T):
        above = s.parent[:, t] if s.parent is not None else torch.full((B,), t - 1, device=DEV)
        child = (above == node) & (t < count)
        x = s.tokens[:, t]
        px = s.probs[b, node, x].double()
        if s.draft is None:
            qx, rest = torch.ones_like(px), torch.where(gone[b, x], 0.0, px)
        else:
            qx = s.draft[b, node, x].double()
            rest = (px - scale * qx).clamp(min=0)
        yes = child & (s.uniform[:, t].double() * qx * total < rest)
        no = child & ~yes
        path.scatter_(1, torch.where(yes, kept, T - 1)[:, None],
                      torch.where(yes, t, path[:, T - 1])[:, None].to(torch.int32))
        kept += yes
        node = torch.where(yes, t, node)
        scale = torch.where(yes, 0.0, torch.where(no, scale + total, scale))
        gone &= ~yes[:, None]
        gone[b, x] |= no
        total = torch.where(yes, 1.0, torch.where(no, left().sum(-1), total))
    upto = torch.cumsum(left(), -1)
    upto = torch.where(upto[:, -1:] > 0, upto, torch.cumsum(s.probs[b, node].double(), -1))
    token = (upto <= s.uniform[:, :1].double() * upto[:, -1:]).sum(-1)
    token = torch.minimum(token, (upto < upto[:, -1:]).sum(-1))
    return [path, kept.to(torch.int32), token]


# --------------------------------------------------------------- one pass
def run(s):
    c = s.case
    if c["kind"] == "attend":
        if own:
            return s.ra.ra_cache_attention_shared(s.q, s.cache, s.table, s.lens, s.shared, s.count, s.mask, out=s.out,
                                                  lse=s.lse, workspace=s.workspace)
        return _plain_attend(s)
    if c["kind"] == "fork":
        if not own:
            return _plain_fork(s)
        s.ra.ra_pages_trim(s.ref, s.table_out, s.held_out, None, c["page"])
        s.ra.ra_pages_fork(s.ref, s.table, s.held, s.lens, s.source, c["page"], table_out=s.table_out,
                           held_out=s.held_out, lens_out=s.lens_out)
        s.ra.ra_pages_reserve(s.ref, s.table_out, s.held_out, s.lens_out, c["page"], c["T"], granted=s.granted,
                              src=s.src, dst=s.dst)
        s.ra.ra_cache_copy(s.cache, s.src, s.dst)
        return _fork_results(s)
    if c["kind"] == "compact":
        if own:
            s.ra.ra_cache_compact(s.cache, s.table, s.lens, s.path, s.kept)
            return [t for t in s.pool if t is not None]
        return _plain_compact(s)
    if own:
        return list(s.ra.ra_verify_drafts(s.probs, s.tokens, s.uniform, parent=s.parent, draft_probs=s.draft,
                                          count=s.count, path=s.path, kept=s.kept, token=s.token))
    return _plain_verify(s)


# ------------------------------------------------------- the same in 64 bits
def _sequence(s, b, tokens, side):
    """Rows 0 .. tokens - 1 of sequence b in 64 bits: [heads, tokens, d]."""
    held, exps = s.pool[2 * side], s.pool[2 * side + 1]
    pages = s.table[b, : -(-tokens // s.case["page"])].long()
    x = held[pages].double()
    if exps is not None:
        x = x * torch.exp2(exps[pages].double()[..., None] - 127)
    return x.transpose(0, 1).reshape(s.case["Hk"], -1, s.case["d"])[:, :tokens]


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


def _exact_fork(s):
    """Sequence by sequence, on the host."""
    c = s.case
    page, T = c["page"], c["T"]
    ref, table, lens = s.ref.tolist(), s.table.tolist(), s.lens.tolist()
    rows, at = [], [lens[b] for b in s.source.tolist()]
    for b, n in zip(s.source.tolist(), at):
        rows.append(table[b][: -(-n // page)])
        for p in rows[-1]:
            ref[p] += 1
    asks = {}  # who writes into a page that is there already
    for i, n in enumerate(at):
        if n // page < len(rows[i]):
            asks.setdefault(rows[i][n // page], []).append(i)
    go = {i for p, who in asks.items() if ref[p] > 1 for i in (who if len(who) < ref[p] else who[:-1])}
    free = iter([p for p, r in enumerate(ref) if r == 0])
    src, dst = [-1] * len(at), [-1] * len(at)
    for i, n in enumerate(at):
        if i in go:
            src[i] = rows[i][n // page]
            rows[i][n // page] = dst[i] = next(free)
        while len(rows[i]) * page < n + T:
            rows[i].append(next(free))
    ref = s.ref.tolist()
    for row in rows:
        for p in row:
            ref[p] += 1
    width = s.table.shape[1]
    wide = [row + [-1] * (width - len(row)) for row in rows]
    pool = [x.clone() for x in s.pool if x is not None]
    for a, z in zip(src, dst):
        if a >= 0:
            for x in pool:
                _bytes_of(x)[z] = _bytes_of(x)[a]
    return [_int(ref), _int(wide), _int([len(r) for r in rows]), _int(at), _int([T] * len(at)), _int(src), _int(dst)] + pool


def _exact_compact(s):
    page = s.case["page"]
    table, lens, path, kept = s.table.tolist(), s.lens.tolist(), s.path.tolist(), s.kept.tolist()
    pool = [x.clone() for x in s.pool if x is not None]
    for b, n in enumerate(lens):
        for j in range(kept[b]):
            a, z = n + path[b][j], n + j
            if a != z:
                for x in pool:
                    y = _bytes_of(x)
                    y[table[b][z // page], :, z % page] = y[table[b][a // page], :, a % page]
    return pool


def _exact_verify(s):
    """Sequence by sequence, on the host; rows are fetched as they are reached."""
    c, paths, tokens = s.case, [], []
    T = c["T"]
    parent = s.parent.tolist() if s.parent is not None else [list(range(-1, T - 1))] * c["B"]
    counts = s.count.tolist() if s.count is not None else [T] * c["B"]
    draws, drafted = s.uniform.double().tolist(), s.tokens.tolist()
    for b in range(c["B"]):
        at, path = 0, [0]
        while True:
            p = s.probs[b, at].double().cpu().numpy()
            q = s.draft[b, at].double().cpu().numpy() if s.draft is not None else None
            rest, total, below = p.copy(), 1.0, None
            for t in [t for t in range(at + 1, counts[b]) if parent[b][t] == at]:
                x = drafted[b][t]
                if draws[b][t] * (q[x] if q is not None else 1.0) * total < rest[x]:
                    below = t
                    break
                if q is not None:
                    rest = np.maximum(rest - total * q, 0.0)
                else:
                    rest[x] = 0.0
                total = math.fsum(rest)
            if below is None:
                break
            at = below
            path.append(at)
        upto = np.cumsum(rest if rest.sum() > 0 else p)
        tokens.append(min(int(np.searchsorted(upto, draws[b][0] * upto[-1], side="right")),
                          int(np.searchsorted(upto, upto[-1]))))
        paths.append(path + [-1] * (T - len(path)))
    return [_int(paths), _int([sum(i >= 0 for i in p) for p in paths]), torch.tensor(tokens, device=DEV)]


def exact(case, seed):
    if case["kind"] == "attend" and work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    return {"attend": _exact_attend, "fork": _exact_fork, "compact": _exact_compact,
            "verify": _exact_verify}[case["kind"]](s)
