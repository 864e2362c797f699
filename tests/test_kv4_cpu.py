"""The 4-bit key/value cache's argument checks, in the C ABI and in the
binding: what is refused on the host, and the sizes it derives (no GPU)."""
import pytest
import torch

import io_aware_exact_21_b200 as fa
from io_aware_exact_21_b200 import binding as bd

P = 0x10000      # a fake, 16-byte aligned address: the checks come before any use


def rows_args(**kw):
    args = dict(k=P, v=P, k_codes=P, k_words=P, v_codes=P, v_words=P, B=2, N=4, Hkv=3, Nk=64, d=128,
                cu_seqlens=None, starts=None, lens=None, stream=0)
    args.update(kw)
    return args


ROW_REFUSALS = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_codes=None), -1), (dict(v_words=None), -1),
    (dict(d=96), -2), (dict(d=256), -2), (dict(d=0), -2),
    (dict(B=-1), -3), (dict(N=-1), -3), (dict(Hkv=0), -3), (dict(Nk=-8), -3), (dict(Nk=60), -3),
    (dict(B=1 << 20, Nk=1 << 12), -3), (dict(B=1 << 16, N=1 << 16), -3),
    (dict(cu_seqlens=P, lens=P), -3), (dict(cu_seqlens=P, B=2049), -3),
    (dict(k=P + 8), -4), (dict(v_codes=P + 4), -4), (dict(k_words=P + 2), -4),
    (dict(cu_seqlens=P + 2), -4), (dict(starts=P + 1), -4), (dict(lens=P + 2), -4),
    (dict(N=0), 0), (dict(B=0), 0), (dict(N=0, k=None, v=None), 0),
    (dict(Nk=0, k_codes=None, k_words=None, v_codes=None, v_words=None), 0),
]


@pytest.mark.parametrize("kw,code", ROW_REFUSALS)
def test_rows_validation(kw, code):
    a = rows_args(**kw)
    assert fa.fa_quantize_kv4(**a) == code
    assert fa.fa_dequantize_kv4(**a) == code


def attend_args(**kw):
    args = dict(q=P, k_codes=P, k_words=P, v_codes=P, v_words=P, o=P, lse=P, B=2, H=6, Hkv=3, Nq=1, Nk=512,
                d=128, scale=0.1, causal=1, window=0, seqlens_k=None, num_splits=1, workspace=None,
                workspace_bytes=0, stream=0)
    args.update(kw)
    return args


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(o=None), -1), (dict(lse=None), -1), (dict(k_words=None), -1),
    (dict(d=32), -2),
    (dict(H=4), -3), (dict(H=0), -3), (dict(Hkv=0), -3), (dict(Nk=500), -3), (dict(Nq=-1), -3),
    (dict(B=-2), -3), (dict(num_splits=33), -3), (dict(num_splits=-1), -3),
    (dict(B=1 << 16, Nq=1 << 15), -3),
    (dict(q=P + 8), -4), (dict(v_codes=P + 8), -4), (dict(lse=P + 4), -4), (dict(seqlens_k=P + 2), -4),
    (dict(num_splits=2, workspace=P + 8, workspace_bytes=1 << 20), -4),
    (dict(causal=0, window=8), -5),
    (dict(num_splits=2), -6), (dict(num_splits=2, workspace=P, workspace_bytes=100), -6),
    (dict(Nq=100), -6), (dict(Nq=100, workspace=P, workspace_bytes=1000), -6),
    (dict(num_splits=0, Nk=65536), -6),
    (dict(scale=0.0), -9), (dict(scale=float("nan")), -9),
    (dict(Nq=0), 0), (dict(B=0), 0), (dict(Nq=0, q=None, o=None, lse=None), 0),
])
def test_attention_validation(kw, code):
    assert fa.fa_fwd_kv4(**attend_args(**kw)) == code


def test_sizes():
    # few rows: two partial results of 8 or 16 rows (d values, reference, sum)
    # to each range; a chunk: its splits' partials and the bf16 rows
    def up(n):
        return (n + 255) // 256 * 256

    size = fa.fa_fwd_kv4_workspace_size
    assert size(2, 8, 2, 1, 512, 128, 0, 1) == up(2 * (2 * 2) * 8 * 130 * 4)
    assert size(2, 8, 2, 1, 512, 128, 0, 4) == up(2 * (4 * 2 * 2) * 8 * 130 * 4)
    assert size(2, 8, 2, 3, 512, 64, 0, 4) == up(2 * (4 * 2 * 2) * 16 * 66 * 4)
    assert size(2, 8, 2, 7, 512, 64, 0, 3) == up(2 * (3 * 2 * 2 * 2) * 16 * 66 * 4)
    back = 2 * (2 * 512 * 2 * 128 * 2)
    assert size(2, 8, 2, 500, 512, 128, 0, 1) == back
    assert size(2, 8, 2, 500, 512, 128, 0, 3) == back + up(3 * 2 * 500 * 8 * 129 * 4)
    assert size(2, 8, 2, 1, 512, 128, 0, 0) == 0 and size(1, 8, 8, 1, 65536, 128, 0, 0) > 0
    assert size(1, 8, 8, 1, 65536, 128, 100, 0) == 0        # a window leaves few tiles: one kernel
    assert size(2, 8, 2, 1, 512, 128, 0, 0) >= 0 and size(2, 8, 2, 500, 512, 128, 0, 0) >= back
    assert size(2, 8, 3, 1, 512, 128, 0, 4) == 0       # 8 heads over 3: refused
    assert size(0, 8, 2, 1, 512, 128, 0, 4) == 0 and size(2, 8, 2, 1, 512, 128, 0, -1) == 0
    # shapes that the call refuses, products of sizes past 64 bits among them
    big = 2 ** 30
    assert size(big, big, big, 256, 1024, 64, 0, 0) == 0 and size(1, big, 1, big, 1024, 64, 0, 0) == 0
    assert size(2, 8, 2, 1, 508, 128, 0, 4) == 0 and size(2, 8, 2, 1, 512, 96, 0, 4) == 0
    assert fa.fa_fwd_kv4(**attend_args(B=big, H=big, Hkv=big, Nq=256)) == -3


# ------------------------------------------------------------- the binding --

@pytest.fixture
def calls(monkeypatch):
    rec = []
    lib = fa.load_library()

    class Library:
        def __getattr__(self, name):
            if name in ("fa_quantize_kv4", "fa_dequantize_kv4", "fa_fwd_kv4"):
                return lambda *args: rec.append((name, args)) or 0
            return getattr(lib, name)

    monkeypatch.setattr(bd, "_require_cuda", lambda t, name: None)
    monkeypatch.setattr(bd, "load_library", Library)
    monkeypatch.setattr(bd, "_stream", lambda stream: stream)
    return rec


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*values):
    return torch.tensor(values, dtype=torch.int32)


def test_cache_is_laid_out_and_rounded_up():
    c = fa.kv4_cache(3, 13, 2, 64, device="cpu")
    assert c["k_codes"].shape == (3, 2, 16, 32) and c["v_codes"].dtype == torch.uint8
    assert c["k_words"].shape == (3, 2, 16) and c["v_words"].dtype == torch.int16
    for bad in (dict(d=32), dict(rows=-1), dict(Hkv=0)):
        with pytest.raises(ValueError):
            fa.kv4_cache(**dict(dict(B=1, rows=8, Hkv=1, d=64, device="cpu"), **bad))


def test_binding_sizes(calls):
    c = fa.kv4_cache(3, 13, 2, 64, device="cpu")
    fa.quantize_kv4(bf(3, 5, 2, 64), bf(3, 5, 2, 64), c, starts=i32(0, 1, 2), lens=i32(5, 0, 3))
    assert calls[-1][0] == "fa_quantize_kv4" and calls[-1][1][6:11] == (3, 5, 2, 16, 64)
    fa.quantize_kv4(bf(9, 2, 64), bf(9, 2, 64), c, cu_seqlens=i32(0, 2, 2, 9))
    assert calls[-1][1][6:11] == (3, 9, 2, 16, 64)
    k, v = fa.dequantize_kv4(c)
    assert k.shape == v.shape == (3, 16, 2, 64) and calls[-1][1][6:11] == (3, 16, 2, 16, 64)
    k, v = fa.dequantize_kv4(c, rows=4, starts=i32(0, 4, 8))
    assert k.shape == (3, 4, 2, 64)
    k, v = fa.dequantize_kv4(c, rows=9, cu_seqlens=i32(0, 2, 2, 9))
    assert k.shape == (9, 2, 64)
    o, lse = fa.forward_kv4(bf(3, 2, 6, 64), c, seqlens_k=i32(1, 2, 3), causal=True)
    assert o.shape == (3, 2, 6, 64) and lse.shape == (3, 6, 2)
    assert calls[-1][1][7:13] == (3, 6, 2, 2, 16, 64)


def test_binding_refusals(calls):
    c = fa.kv4_cache(3, 16, 2, 64, device="cpu")
    x = bf(3, 5, 2, 64)
    bad = [
        lambda: fa.quantize_kv4(x, bf(3, 4, 2, 64), c),                       # unlike k and v
        lambda: fa.quantize_kv4(bf(2, 5, 2, 64), bf(2, 5, 2, 64), c),         # other batch than the cache
        lambda: fa.quantize_kv4(bf(3, 5, 2, 128), bf(3, 5, 2, 128), c),       # other d
        lambda: fa.quantize_kv4(x.float(), x.float(), c),
        lambda: fa.quantize_kv4(bf(3, 2, 5, 64).transpose(1, 2), x, c),       # not contiguous
        lambda: fa.quantize_kv4(x, x, c, starts=i32(0, 1)),
        lambda: fa.quantize_kv4(x, x, c, lens=torch.zeros(3, dtype=torch.int64)),
        lambda: fa.quantize_kv4(bf(9, 2, 64), bf(9, 2, 64), c, cu_seqlens=i32(0, 2, 9)),
        lambda: fa.quantize_kv4(bf(9, 2, 64), bf(9, 2, 64), c, cu_seqlens=i32(0, 2, 2, 9), lens=i32(1, 1, 1)),
        lambda: fa.quantize_kv4(x, x, dict(c, k_words=c["k_words"].to(torch.int32))),
        lambda: fa.quantize_kv4(x, x, dict(c, v_codes=c["v_codes"][:, :, :8].contiguous())),
        lambda: fa.quantize_kv4(x, x, {"k_codes": c["k_codes"]}),
        lambda: fa.dequantize_kv4(c, rows=4, out=(x, x)),
        lambda: fa.dequantize_kv4(c, cu_seqlens=i32(0, 2, 2, 9)),             # how many rows?
        lambda: fa.forward_kv4(bf(3, 1, 5, 64), c),                           # 5 heads over 2
        lambda: fa.forward_kv4(bf(2, 1, 4, 64), c),
        lambda: fa.forward_kv4(bf(3, 1, 4, 128), c),
        lambda: fa.forward_kv4(bf(3, 1, 4, 64), c, seqlens_k=i32(1, 2)),
        lambda: fa.forward_kv4(bf(3, 1, 4, 64), c, out=bf(3, 1, 2, 64)),
        lambda: fa.forward_kv4(bf(3, 1, 4, 64), c, num_splits=2,
                               workspace=torch.zeros(8, dtype=torch.uint8)),
    ]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()
    assert not calls
