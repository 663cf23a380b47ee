"""Waits that run out in every kernel that ra_cache_attention_shared launches
over stretches on the tensor cores: one tile of rows (two key tiles under way,
states exchanged) and two, prefixes and own parts in one launch or apart,
bf16 and 8-bit caches."""
import time

import pytest
import torch

import long_context_ra_gb300 as ra
from long_context_ra_gb300 import _native
from test_gpu_cache_attention import check
from test_gpu_shared_attention import i32, make, wide

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn

# sequences, T, Hq over 1 key head: rows of a sequence, of the batch
FORMS = {"one tile, own parts by the decode kernel": (6, 1, 8),      # 8, 48
         "two tiles, own parts by the decode kernel": (30, 2, 4),    # 8, 240
         "one tile for both": (3, 5, 8),                             # 40, 120
         "two tiles for both": (4, 20, 4)}                           # 80, 320


@pytest.mark.parametrize("held", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_a_stalled_cta_times_out_and_the_next_call_is_right(form, d, held):
    B, T, Hq = FORMS[form]
    groups = [(1024, [200 + 10 * b for b in range(B)])]
    q, cache, table, lens, shared, _ = make(groups, None, T, Hq, 1, 64, d, BF16, held, 14)
    tab, ln = wide(table, cache), i32(lens)
    want = ra.ra_cache_attention_shared(q, cache, tab, ln, shared)
    assert ra.ra_last_device_status() == 0
    check(want, q, cache, table, lens, None, None)
    try:
        ra.ra_watchdog_config(20_000_000, 0)
        t0 = time.perf_counter()
        ra.ra_cache_attention_shared(q, cache, tab, ln, shared)
        assert ra.ra_last_device_status() == _native.RA_ERR_TIMEOUT
        assert time.perf_counter() - t0 < 5.0
    finally:
        ra.ra_watchdog_config(0, -1)
    again = ra.ra_cache_attention_shared(q, cache, tab, ln, shared)
    assert ra.ra_last_device_status() == 0
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
