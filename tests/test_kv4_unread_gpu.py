"""Rows that a write to the 4-bit cache does not take are not read: a write of
no rows of a large padded buffer costs next to nothing."""
import pytest
import torch

import io_aware_exact_21_b200 as fa

pytestmark = pytest.mark.gpu

DEV = "cuda"


def device_ms(fn):
    """The fastest of several runs, by events around four calls."""
    best = float("inf")
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(4):
            fn()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / 4)
    return best


def unread_cases():
    """name -> (arguments under which no row of the buffer is taken)"""
    B, N = 4, 8192
    return {
        "lens 0": dict(lens=torch.zeros(B, dtype=torch.int32, device=DEV)),
        "no cache row": dict(starts=torch.full((B,), N, dtype=torch.int32, device=DEV)),
        "before the cache": dict(starts=torch.full((B,), -N, dtype=torch.int32, device=DEV)),
    }


@pytest.mark.parametrize("name", ["lens 0", "no cache row", "before the cache", "packed: no sequence"])
def test_rows_that_are_not_taken_cost_nothing(name):
    # 0.54 GB of rows, 80 us at the copy rate: launching the CTAs that find
    # nothing to do takes about a tenth of that
    B, N, H, d = 4, 8192, 32, 128
    x = torch.randn((B, N, H, d), device=DEV).to(torch.bfloat16)
    cache = fa.kv4_cache(B, N, H, d)
    full = device_ms(lambda: fa.quantize_kv4(x, x, cache))
    for t in cache.values():
        t.zero_()
    if name.startswith("packed"):
        rows, kw = x.view(B * N, H, d), dict(cu_seqlens=torch.full((B + 1,), 7, dtype=torch.int32, device=DEV))
    else:
        rows, kw = x, unread_cases()[name]
    none = device_ms(lambda: fa.quantize_kv4(rows, rows, cache, **kw))
    assert all(torch.count_nonzero(t) == 0 for t in cache.values())
    assert none < 0.4 * full, "%.1f us for no rows, %.1f us for all" % (1e3 * none, 1e3 * full)
