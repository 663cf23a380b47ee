"""The documented serving example of samples of prompts, run as it stands: what
it leaves in the counts of the pages."""
import re
from pathlib import Path

import pytest
import torch

import long_context_ra_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUIDE = (Path(__file__).resolve().parent.parent / "README.md").read_text()


def block(word):
    (found,) = [b for b in re.findall(r"```python\n(.*?)```", GUIDE, re.S) if word in b]
    return found


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_samples_of_prompts_hold_what_they_need():
    heads, Hq, d, T, V, page = 2, 8, 64, 5, 50, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    cache = ra.new_cache(1024, heads, page, d)
    for t in (cache.k, cache.v):
        t.copy_(torch.randn(t.shape, device=DEV, generator=g))
    prompt = i32([300, 128])
    n = 6
    k, v = (torch.randn(n, heads, T, d, device=DEV, generator=g).bfloat16() for _ in range(2))
    env = dict(torch=torch, ra=ra, cache=cache, prompt=prompt, longest=300, T=T, k=k, v=v,
               table=torch.full((2, 12), -1, dtype=torch.int32, device=DEV), held=i32([0, 0]), lens=prompt.clone(),
               source=i32([0, 0, 0, 0, 1, 1]), shared=i32([0, 300, 300, 300, 0, 128]),
               q=torch.randn(n, Hq, T, d, device=DEV, generator=g).bfloat16(),
               tree=torch.ones(T, T, dtype=torch.bool, device=DEV).tril(),
               probs=torch.softmax(torch.randn(n, T, V, device=DEV, generator=g), -1),
               draft_probs=torch.full((n, T, V), 1.0 / V, device=DEV),
               tokens=torch.randint(0, V, (n, T), device=DEV, generator=g),
               uniform=torch.rand(n, T, device=DEV, generator=g), parent=None)
    exec(block("ra_pages_fork"), env)
    assert ra.ra_last_device_status() == 0
    ref, table, held = env["ref"], env["table"], env["held"]
    count = torch.zeros_like(ref)
    for row, h in zip(table.tolist(), held.tolist()):
        for p in row[:h]:
            count[p] += 1
    # whole pages of a prompt are held by its samples alone, and the one that it ended in by none or one
    assert torch.equal(ref, count)
    ra.ra_pages_trim(ref, table, held, None, page)
    assert not ref.any()
