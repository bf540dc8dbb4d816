"""Calls on another stream than torch's current one that make their result
themselves: its memory is not one that queued work of either stream still uses."""
import pytest
import torch

import dense_gemm_blackwell_tcgen05_gb300 as g

pytestmark = pytest.mark.gpu

QUEUED = 20_000_000   # clocks that the current stream is kept busy: about 10 ms


def calls():
    gen = torch.Generator("cuda").manual_seed(1)
    ints = lambda *s: torch.randint(-3, 4, s, generator=gen, device="cuda").bfloat16()
    A, B, dD = ints(600, 256), ints(4, 512, 256), ints(600, 512)
    o = torch.tensor([0, 130, 130, 401, 600], dtype=torch.int32, device="cuda")
    G = torch.randn(2, 300, 520, generator=gen, device="cuda")
    ws = g.newton_schulz_workspace(2, 300, 520)
    X = torch.randn(300, 520, generator=gen, device="cuda")
    return {
        "grouped": lambda **k: g.matmul_grouped(A, B, o, **k),
        "dgrad": lambda **k: g.matmul_grouped_dgrad(dD, B, o, **k),
        "wgrad": lambda **k: g.matmul_grouped_wgrad(dD, A, o, out_dtype=torch.float32, **k),
        "newton_schulz": lambda **k: g.newton_schulz(G, workspace=ws, **k),
        "bf16": lambda **k: g.matmul_bf16(A, B[1], **k),
        "fused": lambda **k: g.matmul_fused(A, B[1], activation="relu", out_dtype=torch.float32, **k),
        "quantize": lambda **k: g.quantize_mxfp8(X, **k),
        "quantize_tiled": lambda **k: g.quantize_mxfp8_tiled(X, **k),
    }


NAMES = ["grouped", "dgrad", "wgrad", "newton_schulz", "bf16", "fused", "quantize", "quantize_tiled"]


def parts(result):
    return result if isinstance(result, (tuple, list)) else (result,)


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(parts(got), want))


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_writes(name):
    call, side = calls()[name], torch.cuda.Stream()
    want = [t.clone() for t in parts(call())]
    call(stream=side)                     # (first-call set-up)
    torch.cuda.synchronize()
    # blocks of the results' sizes, freed while the current stream has yet to write them
    junk = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(QUEUED)
    for t in junk:
        t.fill_(7)
    del junk, t
    got = call(stream=side)
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_reads(name):
    call, side = calls()[name], torch.cuda.Stream()
    want = [t.clone() for t in parts(call())]
    torch.cuda.synchronize()
    result = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(QUEUED)
    copies = [t.clone() for t in parts(result)]
    sizes = [(t.shape, t.dtype) for t in parts(result)]
    del result
    with torch.cuda.stream(side):
        others = [torch.full(shape, 7, dtype=dtype, device="cuda") for shape, dtype in sizes]
    torch.cuda.synchronize()
    assert same(copies, want) and len(others) == len(want)


def test_a_stream_that_is_only_a_handle():
    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    call, side = calls()["grouped"], torch.cuda.Stream()
    want = [t.clone() for t in parts(call())]
    torch.cuda.synchronize()
    got = call(stream=Handle(side))
    torch.cuda.synchronize()
    assert same(got, want)
