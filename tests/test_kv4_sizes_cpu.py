"""Sizes of the 4-bit cache's calls whose products pass 64 bits are refused
(nothing reaches a GPU)."""
import pytest

import io_aware_exact_21_b200 as fa

P = 0x10000      # a fake, 16-byte aligned address: the checks come before any use


@pytest.mark.parametrize("N,Hkv,d", [(1 << 27, 1 << 30, 128), (1 << 28, 1 << 30, 64), (1 << 30, 1 << 30, 64),
                                     ((1 << 31) - 1, 1 << 30, 128), (1 << 20, 1 << 28, 64)])
def test_rows_times_heads_times_channels(N, Hkv, d):
    for fn in (fa.fa_quantize_kv4, fa.fa_dequantize_kv4):
        for cu in (None, P):
            assert fn(P, P, P, P, P, P, 1, N, Hkv, 8, d, cu, None, None, 0) == -3
        assert fn(P, P, P, P, P, P, 1, N, Hkv, 0, d, None, None, None, 0) == -3
