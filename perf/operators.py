"""Cases of the 4-bit key/value cache: writing new rows into it, reading rows
back, and attention over it, each with a plain form in elementary torch
operations and the call that a user makes (``own``).

A cache row is one token of one key/value head, x of d channels:
    hi = max(0, max x), lo = min(0, min x),
    s = the smallest number of 4 significant bits with 15 s >= hi - lo,
    z = floor(-lo / s + 1/2),  c = clamp(floor(x / s + 1/2) + z, 0, 15),
and stands for s (c - z), which bf16 holds exactly.  Codes are two to a byte
(even channel in the low half), [B, Hkv, rows, d / 2]; a row's 16-bit word is
the bf16 pattern of s with z in its low four bits, [B, Hkv, rows].
"""
import math

import torch

own = False
DEV = "cuda"
TINY = 2.0 ** -126


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one new token of each of 16 requests joins its cache (every decode step)
        {"name": "write_token_B16_H16_d128", "op": "write", "B": 16, "N": 1, "Hkv": 16, "d": 128,
         "rows": 8192, "packed": False, "least": 1},
        # a ragged chunk behind earlier rows, odd head count
        {"name": "write_chunk_B3_N1001_H5_d64", "op": "write", "B": 3, "N": 1001, "Hkv": 5, "d": 64,
         "rows": 2056, "packed": False, "least": 300},
        # a packed batch of prompts of 128 to 4096 tokens goes into empty caches
        {"name": "write_packed_B16_H32_d128", "op": "write", "B": 16, "N": 4096, "Hkv": 32, "d": 128,
         "rows": 4096, "packed": True, "least": 128},
        # a few rows are looked at again (a prefix moves to another program)
        {"name": "read_rows_B2_N17_H3_d64", "op": "read", "B": 2, "N": 17, "Hkv": 3, "d": 64,
         "rows": 1000, "least": 5},
        # a whole cache is read back
        {"name": "read_cache_B4_N8192_H16_d128", "op": "read", "B": 4, "N": 8192, "Hkv": 16, "d": 128,
         "rows": 8192, "least": 8192},
        # one request, a short cache, shared heads: latency
        {"name": "decode_B1_H16of2_Nk1000_d64", "op": "attend", "B": 1, "Nq": 1, "H": 16, "Hkv": 2,
         "d": 64, "rows": 1000, "least": 1000, "window": 0},
        # one token of 16 requests over caches of 4096 to 8192 tokens
        {"name": "decode_B16_H16_Nk8192_d128", "op": "attend", "B": 16, "Nq": 1, "H": 16, "Hkv": 16,
         "d": 128, "rows": 8192, "least": 4096, "window": 0},
        # the same with four query heads to a key/value head, some slots empty
        {"name": "decode_B32_H32of8_Nk8192_d128", "op": "attend", "B": 32, "Nq": 1, "H": 32, "Hkv": 8,
         "d": 128, "rows": 8192, "least": 0, "window": 0},
        # four drafted tokens a request, checked at once under a sliding window
        {"name": "draft_B24_Nq4_H32of8_w1024_d128", "op": "attend", "B": 24, "Nq": 4, "H": 32, "Hkv": 8,
         "d": 128, "rows": 4096, "least": 100, "window": 1024},
        # one request with a long context
        {"name": "decode_B1_H32of8_Nk131072_d128", "op": "attend", "B": 1, "Nq": 1, "H": 32, "Hkv": 8,
         "d": 128, "rows": 131072, "least": 131001, "window": 0},
        # a short chunk of a prompt behind a cached prefix
        {"name": "chunk_B2_Nq100_H16of4_Nk4096_d128", "op": "attend", "B": 2, "Nq": 100, "H": 16,
         "Hkv": 4, "d": 128, "rows": 4096, "least": 2000, "window": 0},
        # a 2048-token chunk after 6144 cached tokens
        {"name": "chunk_B4_Nq2048_H16_Nk8192_d128", "op": "attend", "B": 4, "Nq": 2048, "H": 16,
         "Hkv": 16, "d": 128, "rows": 8192, "least": 8192, "window": 0},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op != "attend":
        B = size(1, 32)
        N = 1 if op == "write" and rng.random() < 0.3 else size(1, 8192)
        N = max(1, min(N, 2 ** 28 // (B * Hkv * d)))
        rows = N + (size(1, 4096) if rng.random() < 0.7 else 0)
        case = {"op": op, "B": B, "N": N, "Hkv": Hkv, "d": d, "rows": rows,
                "least": rng.randint(0, N)}
        if op == "write":
            case["packed"] = rng.random() < 0.5
        return case
    G = rng.choice([1, 1, 2, 4, 7, 8])
    B = size(1, 32)
    Nq = rng.choice([1, 1, 1, rng.randint(2, 16), size(17, 1024)])
    rows = size(16, 65536)
    rows = max(1, min(rows, 2 ** 28 // (B * Hkv * d), 2 ** 30 // (B * Hkv * G * Nq)))
    window = rng.choice([0, 0, size(1, 4096)])
    return {"op": "attend", "B": B, "Nq": Nq, "H": Hkv * G, "Hkv": Hkv, "d": d, "rows": rows,
            "least": rng.randint(0, rows), "window": window}


def lengths(case, seed=None):
    """Rows of each sequence: spread evenly from ``least`` to the most, in an
    order of the seed's (case["B"] of them; the same numbers for every seed)."""
    most = case["N"] if case["op"] != "attend" else case["rows"]
    B, least = case["B"], min(case["least"], most)
    lens = [most] if B == 1 else [least + (most - least) * b // (B - 1) for b in range(B)]
    if seed is not None:
        g = torch.Generator("cpu").manual_seed(seed)
        lens = [lens[i] for i in torch.randperm(B, generator=g).tolist()]
    return lens


# ----------------------------------------------------------------- inputs --

def normal(shape, g, spread=0.0):
    """N(0, 1) in bf16; with spread, channels of unequal size as keys have them."""
    x = torch.randn(shape, generator=g, device=DEV)
    if spread:
        x = x * torch.exp(spread * torch.randn(shape[-2:], generator=g, device=DEV))
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    cap = (case["rows"] + 7) // 8 * 8
    lens = lengths(case, seed)
    state = {"case": case, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    names = ("k_codes", "k_words", "v_codes", "v_words")
    if case["op"] == "write":
        # caches that already hold something: random codes, scales near one
        state["cache"] = dict(zip(names, (
            torch.randint(0, 256, (B, Hkv, cap, d // 2), generator=g, device=DEV, dtype=torch.uint8),
            torch.full((B, Hkv, cap), 0x3f87, device=DEV, dtype=torch.int16),
            torch.randint(0, 256, (B, Hkv, cap, d // 2), generator=g, device=DEV, dtype=torch.uint8),
            torch.full((B, Hkv, cap), 0x3e98, device=DEV, dtype=torch.int16))))
        shape = [sum(lens), Hkv, d] if case["packed"] else [B, case["N"], Hkv, d]
        state["k"], state["v"] = normal(shape, g, 0.6), normal(shape, g)
        state["starts"] = torch.randint(0, case["rows"] - case["N"] + 1, (B,), generator=g, device=DEV,
                                        dtype=torch.int32)
        state["out"] = (torch.zeros(shape, dtype=torch.bfloat16, device=DEV),
                        torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
        if case["packed"]:
            cu = torch.zeros(B + 1, dtype=torch.int32)
            cu[1:] = torch.cumsum(torch.tensor(lens), 0)
            state["cu"] = cu.to(DEV)
        return state
    full = (B, cap, Hkv, d)
    state["cache"] = dict(zip(names, (t.contiguous() for t in (*quantise(normal(full, g, 0.6)),
                                                               *quantise(normal(full, g))))))
    if case["op"] == "read":
        shape = [B, case["N"], Hkv, d]
        state["starts"] = torch.randint(0, case["rows"] - case["N"] + 1, (B,), generator=g, device=DEV,
                                        dtype=torch.int32)
        state["out"] = (torch.zeros(shape, dtype=torch.bfloat16, device=DEV),
                        torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
    else:
        state["q"] = normal((B, case["Nq"], case["H"], d), g)
    return state


def work(case):
    B, Hkv, d, lens = case["B"], case["Hkv"], case["d"], lengths(case)
    wide, narrow = 2 * d, d // 2 + 2          # a row in bf16, in 4 bits with its word
    if case["op"] == "write":                 # new rows in, cache rows out; rows in, values out
        return {"bytes": sum(lens) * Hkv * 2 * (2 * wide + 2 * narrow), "flops": sum(lens) * Hkv * d * 8}
    if case["op"] == "read":
        return {"bytes": sum(lens) * Hkv * 2 * (wide + narrow), "flops": sum(lens) * Hkv * d * 4}
    Nq, H, window = case["Nq"], case["H"], case["window"]
    pairs = rows = 0
    for n in lens:
        first = max(0, n - Nq - window + 1) if window else 0
        rows += n - first
        for i in range(Nq):
            last = n - Nq + i
            pairs += max(0, last + 1 - max(0, last - window + 1 if window else 0))
    return {"bytes": rows * Hkv * 2 * narrow + 2 * B * Nq * H * wide + 4 * B * Nq * H,
            "flops": 4 * pairs * H * d}


# ------------------------------------------------------------- plain forms --

def quantise(x):
    """Codes and words of rows x [B, N, H, d], laid out [B, H, N, ..]."""
    x = x.transpose(1, 2).double()
    hi, lo = x.amax(-1).clamp(min=0), x.amin(-1).clamp(max=0)
    span = hi - lo
    span = torch.where((hi - span) - lo > 0, torch.nextafter(span, span + 1), span)
    half, exponent = torch.frexp(span / 15)                 # half in [0.5, 1)
    s = torch.ldexp(torch.ceil(half * 16), exponent - 4)
    s = torch.where(15 * s < span, s * (1 + 2.0 ** -40), s).clamp(min=TINY)
    z = torch.floor(-lo / s + 0.5)
    c = (torch.floor(x / s[..., None] + 0.5) + z[..., None]).clamp(0, 15).to(torch.uint8)
    words = s.to(torch.bfloat16).view(torch.int16) | z.to(torch.int16)
    return c[..., 0::2] | (c[..., 1::2] << 4), words


def values(codes, words):
    """What cache rows stand for, in 32 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    s = (words & -16).view(torch.bfloat16).float()
    return s[..., None] * (c - (words & 15).float()[..., None])


def places(state):
    """(sequence, cache row) of each row of the new rows, and which are taken."""
    case, starts, lens = state["case"], state["starts"].long(), state["lens"].long()
    if case.get("packed"):
        b = torch.repeat_interleave(torch.arange(case["B"], device=DEV), lens, output_size=state["k"].shape[0])
        i = torch.arange(b.numel(), device=DEV) - state["cu"].long()[b]
        return b, starts[b] + i, None
    b = torch.arange(case["B"], device=DEV)[:, None].expand(-1, case["N"])
    i = torch.arange(case["N"], device=DEV).expand(case["B"], -1)
    return b, starts[b] + i, i < lens[:, None]


def plain_write(state):
    cache = state["cache"]
    b, row, taken = places(state)
    if taken is not None:
        b, row = b[taken], row[taken]
    for name in ("k", "v"):
        x = state[name] if taken is None else state[name][taken]
        codes, words = quantise(x[None])                     # [1, H, rows, ..]
        cache[name + "_codes"][b, :, row] = codes[0].transpose(0, 1)
        cache[name + "_words"][b, :, row] = words[0].transpose(0, 1)
    return plain_read(state)


def plain_read(state):
    cache = state["cache"]
    b, row, taken = places(state)
    for name, out in zip(("k", "v"), state["out"]):
        x = values(cache[name + "_codes"][b, :, row], cache[name + "_words"][b, :, row])
        if taken is not None:
            x = torch.where(taken[..., None, None], x, out.float())
        out.copy_(x.to(torch.bfloat16))
    return state["out"]


def plain_attend(state):
    case, cache, q = state["case"], state["cache"], state["q"].float()
    B, Nq, H, d = q.shape
    Hkv, window = case["Hkv"], case["window"]
    k = values(cache["k_codes"], cache["k_words"])
    v = values(cache["v_codes"], cache["v_words"])
    rows = k.shape[2]
    q = q.view(B, Nq, Hkv, H // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(d))
    nk = state["lens"].long()[:, None, None]
    at = nk - Nq + torch.arange(Nq, device=DEV)[None, :, None]
    j = torch.arange(rows, device=DEV)[None, None, :]
    shown = (j < nk) & (j <= at)
    if window:
        shown = shown & (j > at - window)
    shown = shown.repeat_interleave(H // Hkv, 1)[:, None]
    x = torch.where(shown, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.where(shown, torch.exp(x - top.clamp(min=-1e30)), 0)
    total = p.sum(-1, keepdim=True)
    v = torch.where((torch.arange(rows, device=DEV) < nk[:, 0])[:, None, :, None], v, 0)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)

    def back(t):
        return t.view(B, Hkv, Nq, H // Hkv, -1).permute(0, 2, 1, 3, 4).reshape(B, Nq, H, -1)
    return back(o).to(torch.bfloat16), back(lse)[..., 0].transpose(1, 2).contiguous()


def run(state):
    op, case = state["case"]["op"], state["case"]
    if own:
        import io_aware_exact_21_b200 as fa
        if op == "attend":
            return fa.forward_kv4(state["q"], state["cache"], seqlens_k=state["lens"], causal=True,
                                  window=case["window"])
        where = {"starts": state["starts"]}
        where.update({"cu_seqlens": state["cu"]} if case.get("packed") else {"lens": state["lens"]})
        if op == "write":
            fa.quantize_kv4(state["k"], state["v"], state["cache"], **where)
        return fa.dequantize_kv4(state["cache"], out=state["out"], **where)
    return {"write": plain_write, "read": plain_read, "attend": plain_attend}[op](state)


# ------------------------------------------------- the definition in 64 bits --

def exact_row_values(x):
    """What rows x [..., d] become in the cache, by trying every scale and code."""
    x = x.double()
    hi, lo = x.amax(-1).clamp(min=0), x.amin(-1).clamp(max=0)
    # candidates m 2^e, m = 8..15, around (hi - lo) / 15; the smallest that is enough
    e = torch.floor(torch.log2(((hi - lo) / 15).clamp(min=TINY))) - 3
    s = torch.full_like(hi, math.inf)
    for shift in (-1, 0, 1):
        for m in range(8, 16):
            candidate = m * torch.exp2(e + shift)
            enough = (candidate >= TINY) & ((15 * candidate - hi) + lo >= 0)
            s = torch.where(enough & (candidate < s), candidate, s)
    s = torch.where(torch.isinf(s), TINY, s)
    z = torch.zeros_like(s)
    for n in range(1, 16):
        z = torch.where(-2 * lo >= (2 * n - 1) * s, n, z)
    got, best = torch.zeros_like(x), torch.full_like(x, math.inf)
    for c in range(16):
        value = ((c - z) * s)[..., None]
        nearer = (x - value).abs() <= best                    # of two as near, the upper
        got = torch.where(nearer, value, got)
        best = torch.where(nearer, (x - value).abs(), best)
    return got


def exact_cache_values(codes, words):
    s = torch.exp2((words.long() >> 7).double() - 127) * (1 + ((words.long() >> 4) & 7).double() / 8)
    z = (words & 15).double()
    got = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    got[..., 0::2] = s[..., None] * ((codes % 16).double() - z[..., None])
    got[..., 1::2] = s[..., None] * ((codes // 16).double() - z[..., None])
    return got


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "write":
        outs = []
        for x in (state["k"], state["v"]):
            got = torch.cat([exact_row_values(part) for part in x.flatten(0, -2).split(1 << 18)]).view(x.shape)
            if not case["packed"]:
                for b, n in enumerate(state["lens"].tolist()):
                    got[b, n:] = 0
            outs.append(got)
        return tuple(outs)
    cache = state["cache"]
    if case["op"] == "read":
        outs = []
        for name in ("k", "v"):
            got = torch.zeros(case["B"], case["N"], case["Hkv"], case["d"], dtype=torch.float64, device=DEV)
            for b, (at, n) in enumerate(zip(state["starts"].tolist(), state["lens"].tolist())):
                part = exact_cache_values(cache[name + "_codes"][b, :, at:at + n],
                                          cache[name + "_words"][b, :, at:at + n])
                got[b, :n] = part.transpose(0, 1)
            outs.append(got)
        return tuple(outs)
    q = state["q"].double()
    B, Nq, H, d = q.shape
    group, window = H // case["Hkv"], case["window"]
    o = torch.zeros_like(q)
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(state["lens"].tolist()):
        if n == 0:
            continue
        at = torch.arange(n - Nq, n, device=DEV)[:, None]
        key = torch.arange(n, device=DEV)[None]
        hidden = (key > at) | ((key <= at - window) if window else (key > at))
        seen = (~hidden).any(-1)
        for h in range(case["Hkv"]):
            k = exact_cache_values(cache["k_codes"][b, h, :n], cache["k_words"][b, h, :n])
            v = exact_cache_values(cache["v_codes"][b, h, :n], cache["v_words"][b, h, :n])
            for head in range(h * group, h * group + group):
                x = (q[b, :, head] @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
                lse[b, head] = torch.logsumexp(x, -1)
                w = torch.exp(x[seen] - lse[b, head][seen][:, None])
                o[b, seen, head] = w @ v
    return o, lse
