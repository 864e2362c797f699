"""The workspace of a chunk under a window goes by the rows that the queries
read, not by the cache's room (no GPU)."""
import pytest

import io_aware_exact_21_b200 as fa


@pytest.mark.parametrize("B,H,Hkv,Nq,d,window", [(16, 8, 8, 512, 128, 1024), (4, 32, 8, 2000, 64, 1), (1, 8, 8, 700, 128, 65000)])
@pytest.mark.parametrize("num_splits", [1, 3])
def test_workspace_of_a_windowed_chunk(B, H, Hkv, Nq, d, window, num_splits):
    size = fa.fa_fwd_kv4_workspace_size
    parts = 0 if num_splits == 1 else num_splits * B * Nq * H * (d + 1) * 4 + 255
    rows = window + Nq + 127
    most = parts + 4 * B + 255 + 2 * (2 * B * rows * Hkv * d + 255)
    for Nk in (131072, 262144):
        assert 0 < size(B, H, Hkv, Nq, Nk, d, window, num_splits) <= most
        whole = size(B, H, Hkv, Nq, Nk, d, 0, num_splits)
        assert whole >= 4 * B * Nk * Hkv * d
        assert size(B, H, Hkv, Nq, Nk, d, Nk, num_splits) == whole          # as wide as the cache: none
