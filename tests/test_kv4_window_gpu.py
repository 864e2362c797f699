"""Chunks of queries under a window against the 4-bit cache: the rows read back
are those that the queries read, in a buffer with room for those alone."""
import pytest
import torch

import io_aware_exact_21_b200 as fa
from test_kv4_gpu import DEV, check, queries, random_cache

pytestmark = pytest.mark.gpu


def on_the_forward(q, cache, window, num_splits):
    """Whether the call reads rows back: its workspace then has room for them."""
    B, Nq, H, d = q.shape
    Hkv, Nk = cache["k_codes"].shape[1:3]
    rows = min(Nk, window + Nq)
    return fa.fa_fwd_kv4_workspace_size(B, H, Hkv, Nq, Nk, d, window, num_splits) >= 4 * B * rows * Hkv * d


@pytest.mark.parametrize("window", [1, 64, 130, 300, 519])
@pytest.mark.parametrize("num_splits", [1, 2, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_equals_the_bf16_cache(window, num_splits, d):
    # bit for bit the same chunk over the whole cache read back (lengths of whole
    # 128-key tiles, as without a window)
    cache = random_cache(2, 1032, 16, d, seed=13)
    lens = torch.tensor([1024, 384], dtype=torch.int32, device=DEV)
    q = queries(2, 150, 16, d, 5)
    assert on_the_forward(q, cache, window, num_splits)
    o, lse = fa.forward_kv4(q, cache, lens, causal=True, window=window, num_splits=num_splits)
    k, v = fa.dequantize_kv4(cache)
    o2, lse2 = fa.forward_kvcache(q, k, v, lens, causal=True, window=window, num_splits=num_splits)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window", [1, 2, 127, 128, 129, 700])
@pytest.mark.parametrize("Nq", [90, 257])
def test_where_the_window_starts(window, Nq):
    # lengths that put the first row read on, before and behind a tile's border,
    # and sequences shorter than the chunk
    edge = Nq + window - 1
    lens = [0, 1, Nq - 1, Nq, Nq + 1] + [min(1200, edge + t) for t in (-1, 0, 1, 127, 128, 129, 255, 256, 257)] + [1200]
    cache = random_cache(len(lens), 1200, 3, 64, seed=window + Nq)
    q = queries(len(lens), Nq, 9, 64, 3)
    assert on_the_forward(q, cache, window, 0)
    check(q, cache, torch.tensor(lens, dtype=torch.int32), True, window)


def test_a_workspace_as_large_as_asked_for():
    # what lies behind it stays as it was
    B, Nq, H, Hkv, Nk, d, window = 3, 300, 8, 4, 4096, 128, 100
    cache = random_cache(B, Nk, Hkv, d, seed=3)
    q = queries(B, Nq, H, d, 4)
    lens = torch.tensor([4096, 1111, 200], dtype=torch.int32, device=DEV)
    need = fa.fa_fwd_kv4_workspace_size(B, H, Hkv, Nq, Nk, d, window, 2)
    room = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device=DEV)
    o, lse = fa.forward_kv4(q, cache, lens, causal=True, window=window, num_splits=2, workspace=room[:need])
    assert torch.all(room[need:] == 0x5a)
    room.fill_(0xff)            # NaN everywhere: only what was read back is used
    o2, lse2 = fa.forward_kv4(q, cache, lens, causal=True, window=window, num_splits=2, workspace=room[:need])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
