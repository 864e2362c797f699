"""Attention over the 4-bit cache where the rows' weights p s^v differ much, or
hardly at all: against 64 bits, within bounds that go by |c - z|, what a row
stands for, not by c and z apart."""
import math

import pytest
import torch

import io_aware_exact_21_b200 as fa
from test_kv4_gpu import DEV, queries, random_cache, stands_for

pytestmark = pytest.mark.gpu


def scales(words):
    return (words & -16).view(torch.bfloat16).double()


def tight_reference(q, cache, lens, causal, window, scale):
    """(O, LSE, bound of |O error|) in float64, for the kernels that multiply the
    codes.

    Bounds.  x: each score is off by at most e = (d + 8) 2^-24 A (A = scale s_j
    sum |q| (c + z), the largest of the row) + 2^-21 (the exponential); the sum
    over n keys adds n 2^-24; so a normalised weight is off by 4 e relative at
    most, as in test_kv4_gpu.  w_j = p_j s^v_j is rounded to fp16: by 2^-11 of
    itself, or where it is small by 2^-21 of the row's largest w (the kernel
    keeps a row's largest above 2^-4, and fp16's smallest step is 2^-24).  The same
    rounded w multiply c and z, so both errors reach O times |c - z|: 2^-11
    sum p |v| and 2^-21 max w sum |c - z|.  The tensor core adds 16 products and
    the sum so far cut off 2^-23 below the largest; a code is an fp16 subnormal,
    whose product w c 2^-24 counts there as one of w 2^-14: in units of a code, 18
    2^-13 of the largest w of the 16, cut the same way for c and z, and 2^-23 of the
    sums, sum w (c + z), in each of n / 16 steps.  O is rounded to bf16: 2^-8.
    """
    B, Nq, H, d = q.shape
    G = H // cache["k_codes"].shape[1]
    O = torch.zeros((B, Nq, H, d), dtype=torch.float64, device=DEV)
    L = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device=DEV)
    bo = torch.zeros_like(O)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        pos = torch.arange(n - Nq, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None]
        ok = torch.ones((Nq, n), dtype=torch.bool, device=DEV)
        if causal:
            ok &= j <= pos
        if window > 0:
            ok &= j > pos - window
        for h in range(H):
            kc, kw = cache["k_codes"][b, h // G, :n], cache["k_words"][b, h // G, :n]
            vc, vw = cache["v_codes"][b, h // G, :n], cache["v_words"][b, h // G, :n]
            kk, vv, sv = stands_for(kc, kw), stands_for(vc, vw), scales(vw)
            qq = q[b, :, h].double()
            x = torch.where(ok, scale * (qq @ kk.T), -math.inf)
            some = ok.any(-1)
            L[b, h] = torch.logsumexp(x, -1)
            p = torch.where(ok, torch.exp(x - torch.where(some, L[b, h], 0.0)[:, None]), 0.0)
            O[b, :, h] = p @ vv
            both = lambda c, w: (torch.stack((c & 15, c >> 4), -1).flatten(-2).double()  # noqa: E731
                                 + (w & 15).double()[:, None])
            A = torch.where(ok, scale * (qq.abs() @ (scales(kw)[:, None] * both(kc, kw)).T), 0.0).amax(-1)
            e = (d + 8) * 2.0 ** -24 * A + 2.0 ** -21 + n * 2.0 ** -24
            w = p * sv
            steps = torch.where(sv[:, None] > 0, (vv / sv.clamp(min=2.0 ** -133)[:, None]).abs(), 0.0)
            bo[b, :, h] = (2.0 ** -8 * O[b, :, h].abs() + 1.01 * (
                (2.0 ** -11 + 4 * e)[:, None] * (p @ vv.abs())
                + 2.0 ** -21 * w.amax(-1, keepdim=True) * (ok.double() @ steps)
                + 18 * 2.0 ** -13 * (torch.nn.functional.pad(w, (0, -n % 16)).view(Nq, -1, 16)).amax(-1).sum(-1)[:, None]
                + (n / 16 + 1) * 2.0 ** -23 * (w @ both(vc, vw))))
    return O, L, bo


def runs_on_the_codes(q, cache, window, num_splits):
    B, Nq, H, d = q.shape
    Hkv, Nk = cache["k_codes"].shape[1:3]
    return fa.fa_fwd_kv4_workspace_size(B, H, Hkv, Nq, Nk, d, window, num_splits) < 2 * B * Nk * Hkv * d * 2


def check(q, cache, lens, causal, window=0, num_splits=0, codes=True):
    d = q.shape[-1]
    O, L, bo = tight_reference(q, cache, lens.tolist(), causal, window, d ** -0.5)
    assert not codes or runs_on_the_codes(q, cache, window, num_splits)
    o, lse = fa.forward_kv4(q, cache, seqlens_k=lens.to(DEV), causal=causal, window=window, num_splits=num_splits)
    assert fa.fa_get_device_error() == 0
    assert torch.isfinite(o).all()
    err = (o.double() - O).abs()
    assert (err <= bo).all(), "O: %.3g of its bound" % (err / bo.clamp(min=1e-300)).max()
    empty = torch.isneginf(L)
    assert torch.equal(torch.isneginf(lse), empty)
    return o, lse


def full(lens):
    return torch.tensor(lens, dtype=torch.int32)


SHAPES = [  # B, Nq, H, Hkv, Nk, d
    (2, 1, 8, 1, 1000, 128), (2, 3, 6, 2, 312, 64), (1, 16, 2, 1, 520, 128), (2, 1, 16, 1, 4096, 128),
    # above 32 rows to a key/value head, still on the codes
    (2, 40, 2, 2, 304, 128), (1, 33, 8, 4, 1000, 64), (1, 16, 16, 4, 2048, 128),
]


@pytest.mark.parametrize("B,Nq,H,Hkv,Nk,d", SHAPES)
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 100)])
@pytest.mark.parametrize("num_splits", [0, 1])
def test_ordinary_rows(B, Nq, H, Hkv, Nk, d, causal, window, num_splits):
    cache = random_cache(B, Nk, Hkv, d, seed=Nk + Nq)
    check(queries(B, Nq, H, d, 7), cache, full([Nk] * B), causal, window, num_splits)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("num_splits", [0, 1])
def test_equal_weights_of_rows_near_their_zero(d, num_splits):
    # each V row has one channel of 15 steps and all others at 0 or one step from
    # it, and the keys are alike, so that all weights round the same way: what
    # the rounding does must go with |c - z| (1), not with c (7 and 8)
    n = 512
    g = torch.Generator("cpu").manual_seed(3)
    v = torch.randint(-1, 2, (1, n, 1, d), generator=g).float()
    v[..., 0], v[..., 1] = 8.0, -7.0
    k = torch.zeros((1, n, 1, d))
    for t in range(12):
        # one key above the others by a little, in every warp's first tile: the
        # others' p are then 2^-y with another fraction each time
        k[0, ::64, 0, 0] = 0.25 + t / 8
        cache = fa.quantize_kv4(k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), fa.kv4_cache(1, n, 1, d))
        q = torch.zeros((1, 1, 4, d), dtype=torch.bfloat16, device=DEV)
        q[..., 0] = torch.tensor([1.0, 2.0, 3.0, 5.0], device=DEV)
        check(q, cache, full([n]), True, 0, num_splits)


UPS = [12, 20, 24, 31, 40, 64, 100, 120]


def raise_row(cache, at, up, b=0, hk=0):
    """V row `at` 2^up times as large, half of that by making the others smaller."""
    down = up // 2
    cache["v_words"] -= down << 7
    cache["v_words"][b, hk, at] += up << 7
    return cache


@pytest.mark.parametrize("up", UPS)
@pytest.mark.parametrize("B,Nq,H,Hkv,Nk,d", [(1, 2, 1, 1, 64, 128), (1, 4, 8, 2, 520, 128), (1, 3, 2, 2, 712, 64),
                                            (1, 16, 2, 1, 2048, 128)])
@pytest.mark.parametrize("num_splits", [0, 1, 3])
def test_a_large_row_that_a_mask_hides(up, B, Nq, H, Hkv, Nk, d, num_splits):
    # the last key is seen by the last query alone; the first key by the first
    # queries under a window
    q = queries(B, Nq, H, d, 5)
    check(q, raise_row(random_cache(B, Nk, Hkv, d, 8), Nk - 1, up), full([Nk]), True, 0, num_splits)
    window = min(Nk // 2, 40)
    at = Nk - Nq - window + 1         # the first key of query 0, before all others' windows
    check(q, raise_row(random_cache(B, Nk, Hkv, d, 9), at, up), full([Nk]), True, window, num_splits)
    if at > 0:                        # and one that no query sees, in a tile that they read
        check(q, raise_row(random_cache(B, Nk, Hkv, d, 9), at - 1, up), full([Nk]), True, window, num_splits)


@pytest.mark.parametrize("up", UPS)
@pytest.mark.parametrize("at", [0, 70, 511])
@pytest.mark.parametrize("low", [8.0, 20.0, 45.0, 70.0])
@pytest.mark.parametrize("num_splits", [0, 1])
def test_a_large_row_of_little_weight(up, at, low, num_splits):
    # one V row 2^up times the others, its key's weight 2^-low of theirs: either
    # may decide the result
    d, n = 128, 512
    g = torch.Generator("cpu").manual_seed(17)
    q = torch.randn((1, 1, 1, d), generator=g).to(torch.bfloat16)
    k = torch.randn((1, n, 1, d), generator=g) * 0.1
    k[0, at, 0] = -q[0, 0, 0].float() * (low * math.log(2.0) * d ** 0.5 / q.float().pow(2).sum())
    v = torch.randn((1, n, 1, d), generator=g) * 2.0 ** (-(up // 2))
    v[0, at] *= 2.0 ** up
    cache = fa.quantize_kv4(k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), fa.kv4_cache(1, n, 1, d))
    check(q.to(DEV), cache, full([n]), True, 0, num_splits)


@pytest.mark.parametrize("zero", [0, 2.0 ** -126])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("num_splits", [0, 1])
def test_a_row_of_zeros_takes_the_weight(zero, d, num_splits):
    # a key with nearly all the weight whose values are 0: the others' rows make
    # the result, at 2^-30 of its weight
    n = 300
    g = torch.Generator("cpu").manual_seed(18)
    q = torch.randn((1, 1, 2, d), generator=g).to(torch.bfloat16)
    q[0, 0, 1] = q[0, 0, 0]
    k = torch.randn((1, n, 1, d), generator=g) * 0.1
    k[0, 3, 0] = q[0, 0, 0].float() * (30 * math.log(2.0) * d ** 0.5 / q[0, 0, 0].float().pow(2).sum())
    v = torch.randn((1, n, 1, d), generator=g)
    v[0, 3] = 0
    cache = fa.quantize_kv4(k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), fa.kv4_cache(1, n, 1, d))
    if zero == 0:
        cache["v_words"][0, 0, 3] = 0         # as in a cache that nothing was written to
    check(q.to(DEV), cache, full([n]), True, 0, num_splits)


@pytest.mark.parametrize("num_splits", [0, 1])
@pytest.mark.parametrize("step", [-3, 3])
def test_scales_that_fall_or_grow_by_tiles(num_splits, step):
    # each 64-key tile's values 2^step times those of the one before
    n, d = 1600, 128
    cache = random_cache(1, n, 1, d, 10)
    tile = torch.arange(n, device=DEV) // 64
    cache["v_words"] += ((tile * step - step * 12) << 7).to(torch.int16)
    check(queries(1, 2, 4, d, 5), cache, full([n]), True, 0, num_splits)
    check(queries(1, 2, 4, d, 6), cache, full([n]), True, 64, num_splits)


def test_the_chunk_path_agrees():
    # the same rows, few queries on the codes and many read back
    d, n, up = 128, 520, 31
    cache = raise_row(random_cache(1, n, 20, d, 8), n - 1, up)
    cache["v_words"][:, 1:] = cache["v_words"][:, :1]
    q = queries(1, 250, 40, d, 5)
    assert not runs_on_the_codes(q, cache, 0, 1)
    o, _ = fa.forward_kv4(q, cache, causal=True, num_splits=1)
    few = q[:, -4:].contiguous()
    O, _, bo = tight_reference(few, cache, [n], True, 0, d ** -0.5)
    got, _ = check(few, cache, full([n]), True, 0, 1)
    assert ((o[:, -4:-1].double() - O[:, :-1]).abs() <= 8 * bo[:, :-1] + 2.0 ** -6 * O[:, :-1].abs().amax(-1, True)).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("Nq,H,Hkv", [(4, 2, 1), (12, 4, 2), (250, 40, 20)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("num_splits", [0, 1])
def test_a_nan_query_without_a_key(bad, Nq, H, Hkv, d, num_splits):
    # queries before the first key give O = 0 and LSE = -inf whatever they hold
    cache = random_cache(3, 304, Hkv, d, 19)
    lens = torch.tensor([2, 0, Nq - 1], dtype=torch.int32, device=DEV)
    q = queries(3, Nq, H, d, 20)
    clean, clean_lse = fa.forward_kv4(q, cache, lens, causal=True, num_splits=num_splits)
    for b, n in enumerate(lens.tolist()):
        q[b, :Nq - n, :, 3] = bad
    o, lse = fa.forward_kv4(q, cache, lens, causal=True, num_splits=num_splits)
    assert torch.equal(o, clean) and torch.equal(lse, clean_lse)
    for b, n in enumerate(lens.tolist()):
        assert torch.count_nonzero(o[b, :Nq - n]) == 0 and torch.isneginf(lse[b, :, :Nq - n]).all()
    # and one with keys makes its own row NaN alone
    q[0, Nq - 1, 0, 3] = bad
    o, _ = fa.forward_kv4(q, cache, lens, causal=True, num_splits=num_splits)
    assert torch.isnan(o[0, Nq - 1, 0]).all()
    o[0, Nq - 1, 0] = clean[0, Nq - 1, 0]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("channel", [0, 1, 37])
@pytest.mark.parametrize("large", [8.0, 64.0, 512.0])
@pytest.mark.parametrize("num_splits", [0, 1])
def test_queries_with_one_large_channel(d, channel, large, num_splits):
    # K has its zero in that channel, so that the others make the scores.  A
    # product q c is cut at 2^-13 of the largest |q| of its 16 channels, 18 numbers
    # to a step and d / 16 steps: x is off by 18 2^-13 (d / 16) scale s max |q|
    # beyond the rounding that grows with the sums themselves; where q's elements
    # lie within 2^6 of each other nothing is cut (8 bits of q and 4 of c on a grid
    # of 2^-23 below 2^-14 of the largest), which small parts of q make 2^-20 here.
    n = 1024
    cache = random_cache(1, n, 1, d, 5)
    q = queries(1, 1, 8, d, 7)
    q[..., channel] = q[..., channel].sign() * large
    codes, z = cache["k_codes"][..., channel // 2], (cache["k_words"] & 15).to(torch.uint8)
    codes.copy_((codes & 0x0f) | (z << 4) if channel % 2 else (codes & 0xf0) | z)
    x = d ** -0.5 * (q[0, 0].double() @ stands_for(cache["k_codes"], cache["k_words"])[0, 0].T)
    _, lse = fa.forward_kv4(q, cache, causal=True, num_splits=num_splits)
    top = (d ** -0.5 * scales(cache["k_words"])).max()
    A = top * 30 * q[0, 0].double().abs().sum(-1)
    bound = 18 * 2.0 ** -13 * (d / 16) * top * large + (d + 8) * 2.0 ** -24 * A + 2.0 ** -19
    assert ((lse[0, :, 0].double() - torch.logsumexp(x, -1)).abs() <= bound).all()


@pytest.mark.parametrize("spread", [4, 11, 40, 110])
@pytest.mark.parametrize("seed", range(12))
def test_random_scales(spread, seed):
    # every row's values another power of two, rows of zeros among them, NaN rows
    # where no query looks; heads, queries, lengths, masks and splits by the seed
    g = torch.Generator("cpu").manual_seed(1000 * spread + seed)
    pick = lambda *of: of[int(torch.randint(0, len(of), (1,), generator=g))]  # noqa: E731
    B, Hkv, G, Nq, d = pick(1, 3, 7), pick(1, 2), pick(1, 2, 3, 7), pick(1, 1, 2, 5), pick(64, 128)
    Nk = pick(8, 72, 520, 1800)
    causal, window = pick((False, 0), (True, 0), (True, 3), (True, 70), (True, 500))
    lens = torch.randint(0, Nk + 1, (B,), generator=g).to(torch.int32)
    cache = random_cache(B, Nk, Hkv, d, seed)
    up = torch.randint(-(spread // 2), spread // 2 + 1, (B, Hkv, Nk), generator=g)
    cache["v_words"] += (up << 7).to(torch.int16).to(DEV)
    cache["v_words"][torch.rand((B, Hkv, Nk), generator=g).to(DEV) < 0.05] = 0
    for b, n in enumerate(lens.tolist()):
        first = max(0, n - Nq - window + 1) if window else 0
        for name in ("k_words", "v_words"):
            cache[name][b, :, n:] = 0x7fc0
            cache[name][b, :, :first] = 0x7fc0
    clean = {n: t.clone() for n, t in cache.items()}
    for name in ("k_words", "v_words"):
        clean[name][clean[name] == 0x7fc0] = 0          # (0 * NaN in the reference's product)
    q = queries(B, Nq, G * Hkv, d, seed)
    num_splits = pick(0, 1, 3)
    O, L, bo = tight_reference(q, clean, lens.tolist(), causal, window, d ** -0.5)
    # (35 query rows to a key/value head at most: on the codes)
    o, lse = fa.forward_kv4(q, cache, lens.to(DEV), causal=causal, window=window, num_splits=num_splits)
    assert fa.fa_get_device_error() == 0
    err = (o.double() - O).abs()
    assert torch.isfinite(o).all() and (err <= bo).all(), "O: %.3g of its bound" % (err / bo.clamp(min=1e-300)).max()
    assert torch.equal(torch.isneginf(lse), torch.isneginf(L))
