"""The 4-bit key/value cache on the GPU: what is written and read back, bit by
bit against the definition, and attention over it against a float64 softmax of
the values the cache stands for, within bounds derived from the roundings."""
import math
from fractions import Fraction

import pytest
import torch

import io_aware_exact_21_b200 as fa

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAN_WORD = 0x7fc0


# ------------------------------------------------------- the definition --

def define_row(values):
    """(codes, word) of one row of finite bf16 values, in rational arithmetic."""
    x = [Fraction(v) for v in values]
    hi, lo = max([Fraction(0)] + x), min([Fraction(0)] + x)
    s = Fraction(1, 2 ** 126)
    if hi > lo:
        e = math.floor(math.log2(float((hi - lo) / 15))) - 5       # below the smallest that could do
        found = False
        while not found:
            for m in range(8, 16):
                cand = m * Fraction(2) ** e
                if cand >= s and 15 * cand >= hi - lo:
                    s, found = cand, True
                    break
            e += 1
    z = math.floor(-lo / s + Fraction(1, 2))
    codes = [min(15, math.floor(v / s + Fraction(1, 2)) + z) for v in x]
    word = (torch.tensor(float(s), dtype=torch.float32).view(torch.int32).item() >> 16) | z
    return codes, word


def define_rows(x):
    """Codes (one a channel) and words of finite rows [..., d], in float64 (exact
    here: the values of a row lie within 2^40 of each other)."""
    x = x.double()
    hi, lo = x.amax(-1).clamp(min=0), x.amin(-1).clamp(max=0)
    span = hi - lo
    e = torch.floor(torch.log2((span / 15).clamp(min=2.0 ** -126)))
    s = torch.full_like(span, math.inf)
    for up in (-1, 0, 1):
        for m in range(8, 16):
            cand = m * torch.exp2(e + up - 3)
            s = torch.where((15 * cand >= span) & (cand >= 2.0 ** -126) & (cand < s), cand, s)
    z = torch.floor(-lo / s + 0.5)
    c = (torch.floor(x / s[..., None] + 0.5) + z[..., None]).clamp(max=15)
    words = (s.float().view(torch.int32) >> 16) | z.int()
    return c.to(torch.uint8), words.to(torch.int16)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def stands_for(codes, words):
    """float64 values of cache rows (codes [.., d / 2], words [..])."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    s = (words & -16).view(torch.bfloat16).double()
    return s[..., None] * (c - (words & 15).double()[..., None])


def random_rows(shape, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.randn(shape, generator=g)
    x = x * torch.exp(torch.randn(shape[-1], generator=g))                 # unequal channels
    x = x * torch.exp2(torch.randint(-9, 10, shape[:-1], generator=g).float())[..., None]
    return x.to(torch.bfloat16)


def random_cache(B, rows, Hkv, d, seed):
    """A full cache of rows near N(0, 1), made by the definition."""
    g = torch.Generator(DEV).manual_seed(seed)
    c = fa.kv4_cache(B, rows, Hkv, d)
    for n in ("k", "v"):
        x = torch.randn(c[n + "_codes"].shape[:3] + (d,), generator=g, device=DEV)
        x = x * torch.exp(0.5 * torch.randn((Hkv, 1, d), generator=g, device=DEV))
        x = x * torch.exp(0.7 * torch.randn(x.shape[:3] + (1,), generator=g, device=DEV))
        codes, words = define_rows(x.to(torch.bfloat16))
        c[n + "_codes"].copy_(pack(codes))
        c[n + "_words"].copy_(words)
    return c


# ----------------------------------------------------------------- writing --

@pytest.mark.parametrize("d", [64, 128])
def test_special_rows(d):
    g = torch.Generator("cpu").manual_seed(1)
    base = torch.randn(d, generator=g).to(torch.bfloat16)
    rows = [torch.zeros(d), torch.ones(d), -torch.ones(d), base.abs(), -base.abs(), base * 2.0 ** 100,
            base * 2.0 ** -100, base * 2.0 ** -126, base * 2.0 ** -132]
    one = torch.zeros(d)
    one[7] = 3.0
    rows += [one, -one]
    ramp = torch.arange(d).float() % 31 - 15                       # s = 2: half steps everywhere
    rows += [ramp, -ramp, ramp / 2, ramp * 3, (torch.arange(d) % 16).float()]
    tiny = torch.full((d,), -(2.0 ** -60))
    tiny[0] = 15.0                                                 # 15 s is just too little
    rows += [tiny, -tiny]
    far = torch.full((d,), 2.0 ** -40)
    far[0], far[1], far[2] = -7.5, 7.5, -(2.0 ** -40)              # zero and half a step from it
    rows += [far, -far]
    top = torch.zeros(d)
    top[3], top[4] = 2.0 ** 126, -(2.0 ** 126)
    rows += [top]
    for seed in range(40):
        h = torch.Generator("cpu").manual_seed(100 + seed)
        rows.append(torch.randn(d, generator=h) * torch.exp2(torch.randint(-30, 30, (d,), generator=h).float()))
    x = torch.stack(rows).to(torch.bfloat16)
    N = x.shape[0]
    k = x.view(1, N, 1, d).to(DEV)
    cache = fa.quantize_kv4(k, (-k).contiguous(), fa.kv4_cache(1, N, 1, d))
    for name, y in (("k", x), ("v", -x)):
        codes, words = cache[name + "_codes"].cpu(), cache[name + "_words"].cpu()
        for i in range(N):
            want, word = define_row(y[i].tolist())
            assert words[0, 0, i].item() == word, (name, i)
            got = torch.stack((codes[0, 0, i] & 15, codes[0, 0, i] >> 4), -1).flatten().tolist()
            assert got == want, (name, i)
    # what is read back is what the definition says, and within half a step
    kb, vb = fa.dequantize_kv4(cache, rows=N)
    for name, y, back in (("k", x, kb), ("v", -x, vb)):
        val = stands_for(cache[name + "_codes"], cache[name + "_words"])[0, 0, :N].cpu()
        assert torch.equal(back[0, :, 0].double().cpu(), val)
        s = (cache[name + "_words"] & -16).view(torch.bfloat16).double()[0, 0, :N].cpu()
        assert ((val - y.double()).abs() <= s[:, None] / 2).all()


@pytest.mark.parametrize("B,N,H,d", [(1, 1, 1, 128), (1, 1, 1, 64), (3, 7, 5, 64), (2, 33, 3, 128), (5, 1, 16, 128),
                                     (2, 1000, 4, 128), (3, 777, 7, 64), (1, 20000, 2, 128)])
def test_write_and_read_every_row(B, N, H, d):
    k, v = random_rows((B, N, H, d), 2).to(DEV), random_rows((B, N, H, d), 3).to(DEV)
    cache = fa.quantize_kv4(k, v, fa.kv4_cache(B, N, H, d))
    for name, x in (("k", k), ("v", v)):
        codes, words = define_rows(x.transpose(1, 2))
        assert torch.equal(cache[name + "_words"][:, :, :N], words)
        assert torch.equal(cache[name + "_codes"][:, :, :N], pack(codes))
        assert (cache[name + "_codes"][:, :, N:] == 0).all() and (cache[name + "_words"][:, :, N:] == 0).all()
    for x, back in zip((k, v), fa.dequantize_kv4(cache, rows=N)):
        codes, words = define_rows(x)
        assert torch.equal(back.double(), stands_for(pack(codes), words))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_with_nan_or_infinity(d, bad):
    k = random_rows((1, 4, 2, d), 5)
    k[0, 1, 0, d - 1] = bad
    k[0, 2, 1, 0] = bad
    k = k.to(DEV)
    cache = fa.quantize_kv4(k, k, fa.kv4_cache(1, 8, 2, d))
    back = fa.dequantize_kv4(cache, rows=4)[0]
    nan = torch.isnan(back).all(-1)
    assert nan[0].tolist() == [[False, False], [True, False], [False, True], [False, False]]
    assert torch.equal(torch.isnan(back).any(-1), nan)
    assert cache["k_words"][0, 0, 1].item() == NAN_WORD


def sentinel_cache(B, rows, H, d):
    c = fa.kv4_cache(B, rows, H, d)
    for n in c:
        c[n].fill_(0x5a if n.endswith("codes") else 0x3f85)
    return c


def check_places(x, name, cache, places):
    """Exactly the rows of `places` {(b, cache row): index into x} are written."""
    H, cap = cache["k_codes"].shape[1:3]
    codes, words = define_rows(x)
    want_c = torch.full_like(cache[name + "_codes"], 0x5a)
    want_w = torch.full_like(cache[name + "_words"], 0x3f85)
    for (b, row), i in places.items():
        want_c[b, :, row] = pack(codes[i])
        want_w[b, :, row] = words[i]
    assert torch.equal(cache[name + "_codes"], want_c)
    assert torch.equal(cache[name + "_words"], want_w)


@pytest.mark.parametrize("d,N", [(64, 5), (128, 37), (128, 600)])
def test_starts_and_lens(d, N):
    # starts below zero and past the room, lens below zero and above N
    B, H, rows = 7, 3, 48
    starts = [0, 3, -2, 40, 48, 2 ** 31 - 1, -(2 ** 31)]
    lens = [N, 2, N + 9, -1, 3, N, 4]
    k, v = random_rows((B, N, H, d), 8).to(DEV), random_rows((B, N, H, d), 9).to(DEV)
    st, ln = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in (starts, lens))
    places = {(b, starts[b] + i): (b, i) for b in range(B) for i in range(max(0, min(N, lens[b])))
              if 0 <= starts[b] + i < rows}
    cache = fa.quantize_kv4(k, v, sentinel_cache(B, rows, H, d), starts=st, lens=ln)
    check_places(k, "k", cache, places)
    check_places(v, "v", cache, places)
    out = tuple(torch.full((B, N, H, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    fa.dequantize_kv4(cache, starts=st, lens=ln, out=out)
    for x, back in zip((k, v), out):
        codes, words = define_rows(x)
        want = torch.full((B, N, H, d), 7.0, dtype=torch.float64, device=DEV)
        val = stands_for(pack(codes), words)
        for b, i in places.values():
            want[b, i] = val[b, i]
        assert torch.equal(back.double(), want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[5, 0, 1, 40, 0, 17], [0, 0, 3], [300, 299, 1]])
def test_packed(d, lens):
    # empty sequences, rows past the last sequence (NaN), different starts
    B, H, rows, extra = len(lens), 2, 320, 5
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    T = int(cu[-1]) + extra
    k, v = random_rows((T, H, d), 8), random_rows((T, H, d), 9)
    k[T - extra:], v[T - extra:] = float("nan"), float("nan")
    k, v, cu_d = k.to(DEV), v.to(DEV), cu.to(DEV)
    starts = torch.arange(B, dtype=torch.int32) * 4
    places = {(b, int(starts[b]) + i): int(cu[b]) + i for b in range(B) for i in range(lens[b])
              if int(starts[b]) + i < rows}
    cache = fa.quantize_kv4(k, v, sentinel_cache(B, rows, H, d), starts=starts.to(DEV), cu_seqlens=cu_d)
    check_places(torch.nan_to_num(k), "k", cache, places)
    check_places(torch.nan_to_num(v), "v", cache, places)
    out = tuple(torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    fa.dequantize_kv4(cache, starts=starts.to(DEV), cu_seqlens=cu_d, out=out)
    codes, words = define_rows(torch.nan_to_num(k))
    want = torch.full((T, H, d), 7.0, dtype=torch.float64, device=DEV)
    val = stands_for(pack(codes), words)
    for i in places.values():
        want[i] = val[i]
    assert torch.equal(out[0].double(), want)


# --------------------------------------------------------------- attention --

def reference(q, cache, lens, causal, window, scale):
    """(O, LSE, bound of |O error|, bound of |LSE error|) in float64.

    Bounds.  Score: d products and a zero term in fp32, each addition off by at
    most 2^-24 of a partial sum that stays below A_ij = scale s_j sum |q| (c + z)
    (queries are exact, see the kernel), so |dx| <= (d + 8) 2^-24 max_j A_ij =: e
    (8: the later products and the exponent's fused multiply-add); the
    exponential and the sum over nk keys add 2^-21 + nk 2^-24.  The fp16 p s
    (few rows) is off by 2^-11, the bf16 p of the chunk path by
    2^-8, relative to each term of sum p s (c + z) / sum p (chunk: sum p |v|).
    O is then rounded to bf16: 2^-8.
    """
    B, Nq, H, d = q.shape
    Hkv = cache["k_codes"].shape[1]
    G = H // Hkv
    few = Nq * G <= 32          # more rows may run either way: both roundings
    O = torch.zeros((B, Nq, H, d), dtype=torch.float64, device=DEV)
    L = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device=DEV)
    bo, bl = torch.zeros_like(O), torch.zeros_like(L)
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
            kk, vv = stands_for(kc, kw), stands_for(vc, vw)
            qq = q[b, :, h].double()
            x = scale * (qq @ kk.T)
            x = torch.where(ok, x, -math.inf)
            some = ok.any(-1)
            L[b, h] = torch.logsumexp(x, -1)
            p = torch.where(ok, torch.exp(x - torch.where(some, L[b, h], 0.0)[:, None]), 0.0)
            O[b, :, h] = p @ vv
            mag = lambda c, w: ((w & -16).view(torch.bfloat16).double()[:, None] * (  # noqa: E731
                torch.stack((c & 15, c >> 4), -1).flatten(-2).double() + (w & 15).double()[:, None]))
            km, vm = mag(kc, kw), mag(vc, vw)
            A = torch.where(ok, scale * (qq.abs() @ km.T), 0.0).amax(-1)
            e = (d + 8) * 2.0 ** -24 * A + 2.0 ** -21 + n * 2.0 ** -24
            bo[b, :, h] = 2.0 ** -8 * O[b, :, h].abs() + (2.0 ** -11 + 4 * e)[:, None] * (p @ vm) * 1.01
            if not few:
                bo[b, :, h] += 2.0 ** -8 * (p @ vv.abs()) * 1.01
            bl[b, h] = 2 * e + 2.0 ** -22 * torch.where(some, L[b, h], 0.0).abs() + 2.0 ** -20
    return O, L, bo, bl


def queries(B, Nq, H, d, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn((B, Nq, H, d), generator=g, device=DEV).to(torch.bfloat16)


def hide_unused(cache, lens):
    """NaN words and full codes in every row past a sequence's length."""
    for b, n in enumerate(lens.tolist()):
        for name in ("k", "v"):
            cache[name + "_codes"][b, :, n:] = 255
            cache[name + "_words"][b, :, n:] = NAN_WORD
    return cache


def check(q, cache, lens, causal, window, num_splits=0, scale=None):
    d = q.shape[-1]
    O, L, bo, bl = reference(q, cache, lens.tolist(), causal, window, d ** -0.5 if scale is None else scale)
    o, lse = fa.forward_kv4(q, hide_unused(cache, lens), seqlens_k=lens.to(DEV), causal=causal,
                            window=window, num_splits=num_splits, scale=scale)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == 0
    err = (o.double() - O).abs()
    assert torch.isfinite(o).all()
    assert (err <= bo).all(), "O: %.3g of its bound" % (err / bo.clamp(min=1e-300)).max()
    empty = torch.isneginf(L)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (o.permute(0, 2, 1, 3)[empty] == 0).all()
    err = (lse.double() - L).abs()[~empty]
    assert (err <= bl[~empty]).all(), "LSE: %.3g of its bound" % (err / bl[~empty]).max()
    return o, lse


def some_lens(B, Nk, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randint(0, Nk + 1, (B,), generator=g).to(torch.int32)


SHAPES = [  # B, Nq, H, Hkv, Nk, d
    (1, 1, 1, 1, 8, 128), (2, 1, 2, 2, 64, 64), (3, 1, 4, 2, 40, 128), (2, 1, 8, 1, 1000, 128),
    (2, 3, 6, 2, 312, 64), (2, 2, 14, 2, 256, 128), (1, 16, 2, 1, 520, 128), (3, 5, 5, 5, 2000, 64),
    (2, 1, 16, 1, 4096, 128), (2, 4, 8, 1, 264, 64), (1, 32, 1, 1, 96, 128), (2, 3, 22, 2, 136, 128),
]
MASKS = [(False, 0), (True, 0), (True, 1), (True, 100)]


@pytest.mark.parametrize("B,Nq,H,Hkv,Nk,d", SHAPES)
@pytest.mark.parametrize("causal,window", MASKS)
@pytest.mark.parametrize("num_splits", [1, 3, 0])
def test_few_queries(B, Nq, H, Hkv, Nk, d, causal, window, num_splits):
    cache = random_cache(B, Nk, Hkv, d, seed=Nk + Nq)
    check(queries(B, Nq, H, d, 7), cache, some_lens(B, Nk, Nk + 5 * Nq), causal, window, num_splits)


CHUNKS = [(2, 40, 2, 2, 304, 128), (1, 129, 6, 2, 1000, 64), (2, 300, 4, 1, 520, 128), (3, 17, 14, 2, 400, 128),
          (1, 600, 2, 1, 2048, 128), (2, 96, 2, 2, 304, 64), (2, 97, 2, 2, 304, 64), (1, 33, 64, 1, 136, 128),
          # more blocks of 16 rows than run at once, and rows enough for the forward over the rows read back
          (2, 310, 8, 2, 520, 128), (3, 420, 4, 4, 1000, 64), (2, 150, 16, 16, 304, 128), (40, 97, 8, 8, 136, 64),
          (1, 1200, 8, 2, 136, 128),
          # groups of 3, 6, 16 and 256 heads: 1, 2, 16 and 128 of them share a block's rows
          (3, 250, 12, 4, 304, 64), (2, 200, 24, 4, 304, 128), (1, 100, 128, 8, 304, 64), (1, 40, 256, 1, 136, 64)]


@pytest.mark.parametrize("B,Nq,H,Hkv,Nk,d", CHUNKS)
@pytest.mark.parametrize("causal,window", MASKS)
@pytest.mark.parametrize("num_splits", [1, 3, 0])
def test_chunks(B, Nq, H, Hkv, Nk, d, causal, window, num_splits):
    cache = random_cache(B, Nk, Hkv, d, seed=Nk + Nq)
    check(queries(B, Nq, H, d, 7), cache, some_lens(B, Nk, Nk + 5 * Nq), causal, window, num_splits)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 9, 60])
def test_lengths_at_the_tiles_edges(d, Nq):
    lens = torch.tensor([0, 1, 2, 31, 32, 33, 63, 127, 128, 129, 255, 256, 257, 383, 384], dtype=torch.int32)
    cache = random_cache(len(lens), 384, 1, d, seed=4)
    for causal, window in ((True, 0), (True, 33), (False, 0)):
        check(queries(len(lens), Nq, 2, d, 3), {n: t.clone() for n, t in cache.items()}, lens, causal, window)


def test_more_splits_than_tiles_and_every_row_in_use():
    cache = random_cache(2, 200, 2, 128, seed=6)
    q = queries(2, 1, 4, 128, 2)
    lens = torch.tensor([200, 200], dtype=torch.int32)
    base, lse = check(q, cache, lens, True, 0, 32)
    o, l2 = fa.forward_kv4(q, cache, causal=True, num_splits=32)          # no lengths: all rows
    assert torch.equal(o, base) and torch.equal(l2, lse)


def test_no_rows_at_all():
    for Nq in (1, 100, 3000):
        o, lse = fa.forward_kv4(queries(2, Nq, 4, 64, 1), fa.kv4_cache(2, 0, 2, 64), causal=True)
        assert torch.count_nonzero(o) == 0 and torch.isneginf(lse).all()


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
def test_queries_of_any_size(size):
    # large queries against keys that are as much smaller, and rows of unlike
    # size beside each other in one tile
    cache = random_cache(1, 512, 1, 128, seed=8)
    e = int(math.log2(size))
    big = {**cache, "k_words": cache["k_words"] - (e << 7)}
    q = queries(1, 1, 8, 128, 5) * size
    lens = torch.tensor([512], dtype=torch.int32)
    o, lse = check(q, big, lens, True, 0)
    o1, lse1 = check(queries(1, 1, 8, 128, 5), cache, lens, True, 0)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)                  # powers of two change nothing
    if abs(e) <= 20:
        q[:, :, ::2] = queries(1, 1, 8, 128, 5)[:, :, ::2]
        check(q, cache, lens, True, 0, scale=2.0 ** (-max(0, e)))


@pytest.mark.parametrize("e", [-110, -60, 60, 100])
def test_values_of_any_size(e):
    cache = random_cache(2, 512, 2, 128, seed=9)
    q = queries(2, 3, 4, 128, 5)
    lens = torch.tensor([500, 77], dtype=torch.int32)
    shifted = {**cache, "v_words": cache["v_words"] + (e << 7)}
    o, _ = check(q, shifted, lens, True, 0)
    o1, _ = check(q, cache, lens, True, 0)
    back, o1 = o.double() * 2.0 ** -e, o1.double()
    if e >= -60:
        assert torch.equal(back, o1)          # a power of two changes no rounding
        return
    # Results around 2^-110 leave fp32's and bf16's normal ranges: a warp's
    # factor 2^(m - M) 2^-125 is held to 2^-150, that is 2^-23 of the heaviest
    # warp's terms (their sum is at most 2^11 bo, as bo holds 2^-11 of it), and
    # bf16 numbers under 2^-126 stand 2^-133 apart; besides, either rounding to
    # bf16 may fall to the other side: 2^-8 each.
    bo = reference(q, cache, lens.tolist(), True, 0, 128 ** -0.5)[2]
    assert ((back - o1).abs() <= 2.0 ** (-133 - e) + 2.0 ** -7 * o1.abs() + 2.0 ** -12 * bo).all()


def test_values_that_grow_along_the_cache():
    # each row's values 2^(1/8) larger than the last: the running scale moves
    # in every tile, and early rows fade out of fp16's range
    cache = random_cache(1, 1024, 1, 128, seed=10)
    cache["v_words"].fill_(0x3f87 - (60 << 7))
    cache["v_words"] += ((torch.arange(1024, device=DEV) // 8) << 7).to(torch.int16)
    lens = torch.tensor([1024], dtype=torch.int32)
    check(queries(1, 1, 2, 128, 5), cache, lens, True, 0)
    flipped = {**cache, "v_words": cache["v_words"].flip(-1).contiguous()}
    check(queries(1, 1, 2, 128, 5), flipped, lens, True, 0)


@pytest.mark.parametrize("Nq,Hkv", [(4, 2), (70, 2), (250, 20)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("num_splits", [1, 2])
def test_a_nan_row_reaches_only_the_queries_that_see_it(Nq, Hkv, which, num_splits):
    cache = random_cache(1, 304, Hkv, 128, seed=11)
    q = queries(1, Nq, 2 * Hkv, 128, 5)
    nk = 300
    lens = torch.tensor([nk], dtype=torch.int32, device=DEV)
    window = 40
    clean, _ = fa.forward_kv4(q, cache, lens, causal=True, window=window, num_splits=num_splits)
    at = nk - Nq + 1                      # seen by queries 1 .. window, not by query 0
    cache[which + "_words"][0, 1, at] = NAN_WORD
    cache[which + "_codes"][0, 1, at] = 0
    o, _ = fa.forward_kv4(q, cache, lens, causal=True, window=window, num_splits=num_splits)
    sees = torch.zeros(Nq, dtype=torch.bool, device=DEV)
    sees[1:1 + window] = True
    others = [h for h in range(2 * Hkv) if h // 2 != 1]
    assert torch.isnan(o[0, sees, 2:4]).all()
    assert torch.equal(o[0, ~sees], clean[0, ~sees]) and torch.equal(o[0, :, others], clean[0, :, others])


@pytest.mark.parametrize("Nq,H,Hkv", [(1, 4, 2), (70, 4, 2), (250, 40, 20)])
@pytest.mark.parametrize("num_splits", [0, 2])
def test_a_window_as_wide_as_the_cache_is_none(Nq, H, Hkv, num_splits):
    # also for queries that stand before the first key
    cache = random_cache(2, 304, Hkv, 128, seed=18)
    q = queries(2, Nq, H, 128, 6)
    lens = torch.tensor([304, 30], dtype=torch.int32, device=DEV)
    want, wlse = fa.forward_kv4(q, cache, lens, causal=True, num_splits=num_splits)
    for window in (304, 305, 2 ** 31 - 1):
        o, lse = fa.forward_kv4(q, cache, lens, causal=True, window=window, num_splits=num_splits)
        assert torch.equal(o, want) and torch.equal(lse, wlse)


def test_nan_queries_stay_alone():
    cache = random_cache(1, 256, 1, 64, seed=12)
    q = queries(1, 2, 8, 64, 5)
    clean, _ = fa.forward_kv4(q, cache, causal=True)
    q[0, 0, 3, 5] = float("nan")
    q[0, 1, 4, 0] = float("inf")
    o, _ = fa.forward_kv4(q, cache, causal=True)
    bad = torch.zeros((2, 8), dtype=torch.bool, device=DEV)
    bad[0, 3] = bad[1, 4] = True
    assert torch.isnan(o[0][bad]).all() and torch.equal(o[0][~bad], clean[0][~bad])


def test_chunk_equals_the_bf16_cache():
    # the values are bf16 numbers: the same chunk over the rows read back gives
    # the same bits (with lengths of whole 128-key tiles: the bf16 kernel reads a
    # last part of a tile together with rows before it, in another order)
    cache = random_cache(2, 520, 16, 128, seed=13)
    lens = torch.tensor([512, 384], dtype=torch.int32, device=DEV)
    q = queries(2, 150, 16, 128, 5)
    for ns in (1, 2):
        o, lse = fa.forward_kv4(q, cache, lens, causal=True, num_splits=ns)
        k, v = fa.dequantize_kv4(cache)
        o2, lse2 = fa.forward_kvcache(q, k, v, lens, causal=True, num_splits=ns)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_serving_loop():
    # a prompt in, then tokens one at a time: the cache is the one written at
    # once, and each step's attention is bit for bit that over it
    B, H, Hkv, d, prompt, steps = 3, 8, 2, 128, 45, 6
    total = prompt + steps
    k, v = random_rows((B, total, Hkv, d), 20).to(DEV), random_rows((B, total, Hkv, d), 21).to(DEV)
    whole = fa.quantize_kv4(k, v, fa.kv4_cache(B, total, Hkv, d))
    cache = fa.kv4_cache(B, total, Hkv, d)
    fa.quantize_kv4(k[:, :prompt].contiguous(), v[:, :prompt].contiguous(), cache)
    q = queries(B, total, H, d, 22)
    lens = torch.full((B,), prompt, dtype=torch.int32, device=DEV)
    o, _ = fa.forward_kv4(q[:, :prompt].contiguous(), cache, lens, causal=True)
    want, _ = fa.forward_kv4(q[:, :prompt].contiguous(), whole, lens, causal=True)
    assert torch.equal(o, want)
    for t in range(prompt, total):
        fa.quantize_kv4(k[:, t:t + 1].contiguous(), v[:, t:t + 1].contiguous(), cache, starts=lens)
        lens += 1
        qt = q[:, t:t + 1].contiguous()
        o, lse = fa.forward_kv4(qt, cache, lens, causal=True)
        want, wl = fa.forward_kv4(qt, whole, lens, causal=True)
        assert torch.equal(o, want) and torch.equal(lse, wl)
    for n in cache:
        assert torch.equal(cache[n], whole[n])


def test_two_runs_give_the_same_bits():
    cache = random_cache(4, 3000, 4, 128, seed=14)
    q = queries(4, 2, 8, 128, 5)
    for ns in (1, 7):
        a = fa.forward_kv4(q, cache, causal=True, num_splits=ns)
        b = fa.forward_kv4(q, cache, causal=True, num_splits=ns)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("Nq,H,Hkv", [(1, 4, 2), (200, 4, 2), (200, 24, 12)])
def test_step_in_a_graph_on_a_side_stream(Nq, H, Hkv):
    # write and attend captured once, replayed with other rows, lengths and
    # queries; a second graph with its own workspace is replayed between
    B, d, Nk = 2, 128, 1024
    side = torch.cuda.Stream()
    graphs = []
    for seed in (30, 31):
        cache = random_cache(B, Nk, Hkv, d, seed)
        st = dict(cache=cache, k=queries(B, Nq, Hkv, d, seed + 1), v=queries(B, Nq, Hkv, d, seed + 2),
                  q=queries(B, Nq, H, d, seed + 3), starts=torch.tensor([100, 700], dtype=torch.int32, device=DEV))
        st["lens"] = st["starts"] + Nq
        ns = 4
        st["ws"] = torch.empty(fa.fa_fwd_kv4_workspace_size(B, H, Hkv, Nq, Nk, d, 0, ns), dtype=torch.uint8, device=DEV)
        st["o"], st["lse"] = torch.empty_like(st["q"]), torch.empty((B, H, Nq), device=DEV)

        def step(st=st, ns=ns):
            fa.quantize_kv4(st["k"], st["v"], st["cache"], starts=st["starts"])
            fa.forward_kv4(st["q"], st["cache"], st["lens"], causal=True, num_splits=ns, out=st["o"],
                           lse=st["lse"], workspace=st["ws"])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        graphs.append((g, st))
    for r in range(3):
        for g, st in graphs:
            for n in ("q", "k", "v"):
                st[n].copy_(queries(*st[n].shape, 50 + r))
            st["starts"] += 17
            st["lens"] += 17
            g.replay()
        torch.cuda.synchronize()
        for g, st in graphs:
            plain = {n: t.clone() for n, t in st["cache"].items()}
            fa.quantize_kv4(st["k"], st["v"], plain, starts=st["starts"])
            o, lse = fa.forward_kv4(st["q"], plain, st["lens"], causal=True, num_splits=4)
            assert torch.equal(o, st["o"]) and torch.equal(lse, st["lse"])
            for n in plain:
                assert torch.equal(plain[n], st["cache"][n])


def test_offsets_past_32_bits():
    # a cache of over 2^31 code bytes (and 2^32 codes): the last rows of the
    # last head
    B, Hkv, d, Nk = 1, 2, 128, (1 << 24) + (1 << 20)
    cache = fa.kv4_cache(B, Nk, Hkv, d)
    assert cache["k_codes"].numel() > 2 ** 31
    N = 700
    k, v = queries(B, N, Hkv, d, 40), queries(B, N, Hkv, d, 41)
    starts = torch.tensor([Nk - N], dtype=torch.int32, device=DEV)
    fa.quantize_kv4(k, v, cache, starts=starts)
    codes, words = define_rows(k.transpose(1, 2))
    assert torch.equal(cache["k_codes"][:, :, -N:], pack(codes)) and torch.equal(cache["k_words"][:, :, -N:], words)
    assert torch.count_nonzero(cache["k_words"][:, :, :-N]) == 0
    back = fa.dequantize_kv4(cache, rows=N, starts=starts)[1]
    codes, words = define_rows(v)
    assert torch.equal(back.double(), stands_for(pack(codes), words))
    q = queries(B, 3, 4, d, 42)
    o, lse = fa.forward_kv4(q, cache, causal=True, window=N - 2)
    small = {n: t[:, :, -N - 4:].contiguous() for n, t in cache.items()}
    O, L, bo, bl = reference(q, small, [N + 4], True, N - 2, d ** -0.5)
    assert ((o.double() - O).abs() <= bo).all() and ((lse.double() - L).abs() <= bl).all()


def test_separate_streams():
    # separate caches on separate streams at once
    streams = [torch.cuda.Stream() for _ in range(3)]
    done = []
    for i, s in enumerate(streams):
        k = random_rows((2, 500, 4, 128), 60 + i).to(DEV)
        cache = fa.kv4_cache(2, 500, 4, 128)
        q = queries(2, 1, 8, 128, i)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            fa.quantize_kv4(k, k, cache)
            done.append((k, cache, q, fa.forward_kv4(q, cache, causal=True)))
    torch.cuda.synchronize()
    for k, cache, q, (o, lse) in done:
        codes, words = define_rows(k.transpose(1, 2))
        assert torch.equal(cache["v_codes"][:, :, :500], pack(codes))
        o2, lse2 = fa.forward_kv4(q, cache, causal=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)



def test_nothing_to_do():
    cache = random_cache(2, 64, 2, 64, seed=15)
    o, lse = fa.forward_kv4(queries(2, 0, 4, 64, 1), cache)
    assert o.shape == (2, 0, 4, 64) and lse.shape == (2, 4, 0)
    empty = fa.kv4_cache(0, 64, 2, 64)
    assert fa.forward_kv4(queries(0, 1, 4, 64, 1), empty)[0].shape == (0, 1, 4, 64)
    before = {n: t.clone() for n, t in cache.items()}
    none = torch.empty((2, 0, 2, 64), dtype=torch.bfloat16, device=DEV)
    fa.quantize_kv4(none, none, cache)
    fa.quantize_kv4(queries(2, 3, 2, 64, 1), queries(2, 3, 2, 64, 2), cache,
                    lens=torch.zeros(2, dtype=torch.int32, device=DEV))
    assert all(torch.equal(cache[n], before[n]) for n in cache)


@pytest.mark.parametrize("num_splits", [0, 4])
def test_a_wait_that_runs_out_is_reported(num_splits):
    # each warp's first K tile is left unloaded: the waits end, the host reads
    # the status, and the next call works
    cache = random_cache(2, 512, 2, 128, seed=16)
    q = queries(2, 1, 4, 128, 1)
    want, _ = fa.forward_kv4(q, cache, causal=True, num_splits=num_splits)
    torch.cuda.synchronize()
    assert fa.fa_debug_set_fault(3, 1000000) == 0
    try:
        fa.forward_kv4(q, cache, causal=True, num_splits=num_splits)
        assert fa.fa_get_device_error() == -8
    finally:
        assert fa.fa_debug_set_fault(0, 0) == 3
    o, _ = fa.forward_kv4(q, cache, causal=True, num_splits=num_splits)
    assert fa.fa_get_device_error() == 0 and torch.equal(o, want)


def test_lengths_of_many_sequences():
    # more sequences than a CTA has threads, most of them short or empty
    B, Hkv, d, Nk = 300, 1, 64, 72
    cache = random_cache(B, Nk, Hkv, d, seed=17)
    lens = some_lens(B, Nk, 3)
    lens[::3] = 0
    lens[100:180] = 0
    q = queries(B, 1, 2, d, 4)
    for ns in (0, 1, 7):
        check(q, {n: t.clone() for n, t in cache.items()}, lens, True, 0, ns)
    check(q, {n: t.clone() for n, t in cache.items()}, torch.zeros(B, dtype=torch.int32), True, 0, 3)


def test_tensors_of_another_device_are_refused(monkeypatch):
    # the library launches on the current device: tensors elsewhere are refused
    cache = random_cache(1, 64, 1, 64, seed=18)
    q = queries(1, 1, 1, 64, 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: fa.forward_kv4(q, cache), lambda: fa.dequantize_kv4(cache),
                 lambda: fa.quantize_kv4(q, q, cache)):
        with pytest.raises(ValueError, match="current device"):
            call()
