"""`stream=` with nothing preallocated: outputs and workspaces belong to the
stream that the call runs on, so that neither what the current stream still has
to do nor what it does next reaches them."""
import pytest
import torch

import io_aware_exact_21_b200 as fa

pytestmark = pytest.mark.gpu

DEV = "cuda"
BUSY = 200_000_000          # clock cycles of a wait on a stream, about 0.1 s


def randn(shape, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def handle(s, as_int):
    return s.cuda_stream if as_int else s


def full_cache(B, rows, Hkv, d, seed):
    return fa.quantize_kv4(randn((B, rows, Hkv, d), seed), randn((B, rows, Hkv, d), seed + 1), fa.kv4_cache(B, rows, Hkv, d))


def calls():
    """name -> call(stream) -> tuple of tensors, with inputs made beforehand."""
    cache = full_cache(2, 2048, 2, 128, 1)
    few, many = randn((2, 1, 8, 128), 3), randn((2, 700, 8, 128), 4)
    q, k, v, do = (randn((2, 512, 4, 128), 5 + i) for i in range(4))
    kc, vc = randn((2, 2048, 4, 128), 9), randn((2, 2048, 4, 128), 10)
    qd = randn((2, 1, 4, 128), 11)
    o, lse = fa.forward(q, k, v, causal=True)
    qz = fa.quantize_fp8(q, k, v)
    lens = torch.tensor([1000, 31], dtype=torch.int32, device=DEV)
    return {
        "dequantize_kv4": lambda s: fa.dequantize_kv4(cache, lens=lens, stream=s),
        "forward_kv4 ranges": lambda s: fa.forward_kv4(few, cache, causal=True, num_splits=8, stream=s),
        "forward_kv4 chunk": lambda s: fa.forward_kv4(many, cache, causal=True, stream=s),
        "forward_kvcache": lambda s: fa.forward_kvcache(qd, kc, vc, causal=True, num_splits=8, stream=s),
        "forward": lambda s: fa.forward(q, k, v, causal=True, stream=s),
        "forward_kv": lambda s: fa.forward_kv(q, kc, vc, causal=True, stream=s),
        "backward": lambda s: fa.backward(q, k, v, o, lse, do, causal=True, stream=s),
        "backward fused": lambda s: fa.backward(q, k, v, o, lse, do, causal=True, fused=True, stream=s),
        "quantize_fp8": lambda s: tuple(fa.quantize_fp8(q, k, v, stream=s).values()),
        "forward_fp8": lambda s: fa.forward_fp8(qz, 2, 512, 4, stream=s),
    }


NAMES = ["dequantize_kv4", "forward_kv4 ranges", "forward_kv4 chunk", "forward_kvcache", "forward", "forward_kv",
         "backward", "backward fused", "quantize_fp8", "forward_fp8"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_int", [False, True])
def test_the_current_stream_is_busy(name, as_int):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)                 # whatever is queued here comes late
    got = call(handle(side, as_int))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_int", [False, True])
def test_the_current_stream_takes_memory_at_once(name, as_int):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)             # the call's kernels come late
    got = call(handle(side, as_int))
    # all sizes that the call may have given back to the allocator, filled at once
    taken = [torch.full((n,), 0x7f, dtype=torch.uint8, device=DEV)
             for n in [1 << b for b in range(9, 26)] * 3]
    torch.cuda.synchronize()
    # (the call's kernels must not write to it, either)
    assert all(torch.all(t == 0x7f) for t in taken)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_replayed_graph_and_stream_argument():
    # captured with the capture's own stream given by hand
    cache = full_cache(1, 1024, 2, 128, 20)
    q = randn((1, 1, 8, 128), 21)
    want, wlse = fa.forward_kv4(q, cache, causal=True, num_splits=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        o, lse = fa.forward_kv4(q, cache, causal=True, num_splits=4, stream=side)
        k, v = fa.dequantize_kv4(cache, stream=side.cuda_stream)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wlse)
    k2, v2 = fa.dequantize_kv4(cache)
    assert torch.equal(k, k2) and torch.equal(v, v2)
