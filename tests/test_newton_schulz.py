"""newton_schulz against the formula in 64 bits.

Tolerance, on the 2-norm of the difference over that of the result.  A step
rounds three operands to fp16 (unit 2^-11): X, which meets Y = b P + c P^2, and
P and Y themselves.  With singular values near 1, |Y| is up to 2.8 against a
result of at least 0.68, so a rounding enters up to 4 times larger; rounding
errors of opposite sign cancel over a product's terms, so that the three
together stay within 4 * 2^-11 a step.  Rounding the result adds 2^-9 (bf16).
Directions of small singular values grow by up to 3.4445 a step: that they
carry no more than this is what the low-rank case is for."""
import numpy as np
import pytest
import torch

import dense_gemm_blackwell_tcgen05_gb300 as g

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


def tolerance(steps, dtype):
    return steps * 4 * 2.0 ** -11 + (2.0 ** -9 if dtype == torch.bfloat16 else 0.0)


def reference(G, steps=5, coefficients=g.NEWTON_SCHULZ_COEFFICIENTS, eps=1e-7):
    a, b, c = coefficients
    X = G.double()
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT if tall else X
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        P = X @ X.mT
        X = a * X + b * (P @ X) + c * (P @ (P @ X))
    return X.mT if tall else X


def close(got, want, tol):
    want = want.reshape(-1, *want.shape[-2:])
    got = got.double().reshape(want.shape)
    for i in range(want.shape[0]):
        err = ((got[i] - want[i]).norm() / want[i].norm()).item()
        assert err <= tol, f"matrix {i}: {err:.2e} > {tol:.2e}"


SIZES = [(1, 1), (1, 9), (9, 1), (7, 5), (64, 64), (128, 128), (127, 300), (129, 128), (256, 256), (255, 513),
         (300, 100), (640, 384), (520, 1040), (1041, 257)]


@pytest.mark.parametrize("rows, cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_random(rows, cols, dtype, out_dtype):
    gen = torch.Generator("cuda").manual_seed(rows + cols)
    G = torch.randn(rows, cols, device="cuda", generator=gen).to(dtype)
    for steps in (1, 5):
        O = g.newton_schulz(G, steps=steps, out_dtype=out_dtype)
        assert g.gemm_last_status(stream()) == g.GEMM_OK
        close(O, reference(G, steps), tolerance(steps, out_dtype))


@pytest.mark.parametrize("batch, rows, cols", [(3, 64, 200), (5, 200, 72), (2, 384, 384), (40, 16, 24)])
def test_batch_pitches(batch, rows, cols):
    """Batches with padded and odd pitches, an output that starts off any
    vector's alignment, and scales apart by 1e6."""
    gen = torch.Generator("cuda").manual_seed(batch)
    buf = torch.full((batch, rows + 1, cols + 3), float("nan"), device="cuda")
    G = buf[:, :rows, :cols]
    G.copy_(torch.randn(batch, rows, cols, device="cuda", generator=gen) *
            10.0 ** torch.linspace(-3, 3, batch, device="cuda")[:, None, None])
    want = reference(G)
    for pad, shift in ((0, 0), (1, 1), (4, 3)):
        flat = torch.full((batch * rows * (cols + pad) + shift,), float("nan"), dtype=torch.bfloat16, device="cuda")
        O = flat[shift:].view(batch, rows, cols + pad)[..., :cols]
        g.newton_schulz(G, out=O)
        assert g.gemm_last_status(stream()) == g.GEMM_OK
        close(O, want, tolerance(5, torch.bfloat16))
        O.fill_(float("nan"))
        assert flat.isnan().all(), "wrote outside the output"


@pytest.mark.parametrize("batch, rows, cols", [
    (1, 70, 2400), (1, 5000, 33), (2, 128, 2304), (1, 4100, 130), (4, 300, 2700), (3, 2900, 384), (5, 2047, 60),
    (4, 2700, 300), (20, 138, 670), (30, 300, 900), (24, 1300, 72)])
def test_long_sides(batch, rows, cols):
    """Long reductions of few tiles, and products whose best tiles differ."""
    gen = torch.Generator("cuda").manual_seed(rows - cols)
    G = torch.randn(batch, rows, cols, device="cuda", generator=gen)
    for dtype in (torch.float32, torch.bfloat16):
        O = g.newton_schulz(G, out_dtype=dtype)
        assert g.gemm_last_status(stream()) == g.GEMM_OK
        close(O, reference(G), tolerance(5, dtype))
        assert torch.equal(O, g.newton_schulz(G, out_dtype=dtype))


@pytest.mark.parametrize("rows, cols", [(512, 640), (640, 512), (96, 96)])
@pytest.mark.parametrize("kind", ["rank8", "decay"])
def test_small_singular_values(rows, cols, kind):
    gen = torch.Generator("cuda").manual_seed(1)
    if kind == "rank8":
        G = torch.randn(rows, 8, device="cuda", generator=gen) @ torch.randn(8, cols, device="cuda", generator=gen)
    else:
        m = min(rows, cols)
        q = lambda n: torch.linalg.qr(torch.randn(n, m, device="cuda", generator=gen))[0]
        G = (q(rows) / torch.arange(1, m + 1, device="cuda") ** 1.5) @ q(cols).T
    O = g.newton_schulz(G, out_dtype=torch.float32)
    close(O, reference(G), tolerance(5, torch.float32))


def test_other_coefficients():
    """The cubic Newton-Schulz iteration (1.5, -0.5, 0), which converges to
    the orthogonal factor itself."""
    gen = torch.Generator("cuda").manual_seed(2)
    G = torch.randn(96, 320, device="cuda", generator=gen)
    O = g.newton_schulz(G, steps=24, coefficients=(1.5, -0.5, 0.0), out_dtype=torch.float32)
    U, _, V = torch.linalg.svd(G.double(), full_matrices=False)
    # at the fixed point |Y| = 0.5 and the errors of earlier steps die out: one step's remain
    close(O, U @ V, tolerance(1, torch.float32))


@pytest.mark.parametrize("batch, rows, cols", [(1, 33, 47), (3, 130, 70), (2, 257, 600), (1, 70, 2400), (1, 2401, 65)])
def test_workspace_contents_do_not_matter(batch, rows, cols):
    gen = torch.Generator("cuda").manual_seed(rows)
    G = torch.randn(batch, rows, cols, device="cuda", generator=gen)
    bits = []
    for fill in (0, 0xFF, 0x7B):   # zeros, NaN, large numbers
        ws = g.newton_schulz_workspace(batch, rows, cols)
        ws.view(torch.uint8).fill_(fill)
        bits.append(g.newton_schulz(G, out_dtype=torch.float32, workspace=ws))
        assert g.gemm_last_status(stream()) == g.GEMM_OK
    assert not bits[0].isnan().any()
    assert torch.equal(bits[0], bits[1]) and torch.equal(bits[0], bits[2])


def test_zero_and_nonfinite_matrices():
    gen = torch.Generator("cuda").manual_seed(3)
    G = torch.randn(5, 160, 96, device="cuda", generator=gen)
    G[1] = 0.0
    G[2, 5, 7] = float("nan")
    G[3, 9, 1] = float("inf")
    O = g.newton_schulz(G, out_dtype=torch.float32)
    assert g.gemm_last_status(stream()) == g.GEMM_OK
    assert (O[1] == 0).all()
    assert O[2].isnan().any() and O[3].isnan().any()
    close(O[[0, 4]], reference(G[[0, 4]]), tolerance(5, torch.float32))


def test_empty():
    for shape in ((0, 4, 4), (2, 0, 5), (2, 5, 0)):
        assert g.newton_schulz(torch.zeros(shape, device="cuda")).shape == shape


def test_stream_graph_and_repeat():
    gen = torch.Generator("cuda").manual_seed(4)
    G = torch.randn(2, 300, 520, device="cuda", generator=gen)
    ws = g.newton_schulz_workspace(2, 300, 520)
    O = torch.empty(2, 300, 520, dtype=torch.float32, device="cuda")
    first = g.newton_schulz(G, out=O, workspace=ws).clone()
    for _ in range(3):
        ws.fill_(255)      # NaN in every half: the workspace needs no clearing
        assert torch.equal(g.newton_schulz(G, out=O, workspace=ws), first)
    s = torch.cuda.Stream()
    O.zero_()
    s.wait_stream(torch.cuda.current_stream())
    g.newton_schulz(G, out=O, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(O, first)
    with pytest.raises(ValueError):
        g.newton_schulz(G, out=O, stream=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.newton_schulz(G, out=O, workspace=ws)
    G.mul_(3.0)            # the same directions
    G[0] = G[1]
    graph.replay()
    assert g.gemm_last_status(stream()) == g.GEMM_OK
    close(O, reference(G), tolerance(5, torch.float32))


def test_tensor_refusals():
    G = torch.zeros(4, 8, device="cuda")
    with pytest.raises(TypeError):
        g.newton_schulz(G.half())
    with pytest.raises(ValueError):
        g.newton_schulz(G.T)
    with pytest.raises(ValueError):
        g.newton_schulz(G.cpu())
    with pytest.raises(ValueError):
        g.newton_schulz(G, out=torch.zeros(4, 9, device="cuda"))
    for kw in ({"steps": 0}, {"steps": 65}, {"eps": -1.0}, {"coefficients": (float("nan"), 0.0, 0.0)},
               {"workspace": torch.empty(256, dtype=torch.uint8, device="cuda")}):
        with pytest.raises(g.GemmError) as e:
            g.newton_schulz(G, **kw)
        assert e.value.status == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("rows, cols", [(96, 160), (300, 70), (64, 3000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1e-39, 1e-37, 1e-30, 1e-23, 1e-19, 1e-13, 1e15, 1e19, 1e24, 4e37])
def test_norms_whose_square_leaves_fp32(rows, cols, dtype, scale):
    """The norm is taken of any finite values: their squares need not be fp32 numbers."""
    gen = torch.Generator("cuda").manual_seed(rows)
    G = (torch.randn(rows, cols, device="cuda", generator=gen).double() * scale).to(dtype)
    assert G.isfinite().all() and (G != 0).any()
    O = g.newton_schulz(G, eps=0.0, out_dtype=torch.float32)
    assert g.gemm_last_status(stream()) == g.GEMM_OK
    close(O, reference(G, eps=0.0), tolerance(5, torch.float32))


def test_norms_of_mixed_magnitudes():
    """Parts of one matrix whose squares lie in different ranges, and matrices
    of a batch apart by 1e76; the default eps and none."""
    gen = torch.Generator("cuda").manual_seed(6)
    G = torch.randn(6, 130, 2100, device="cuda", generator=gen)
    G[0, :100] *= 1e-30
    G[1, 7:9] *= 1e25
    G[2] *= 1e-37
    G[2, 129] *= 1e17
    G[3, 64:] *= 1e18
    G[4] *= 1e38 / G[4].abs().max()
    G[5] *= 1e-38
    O = g.newton_schulz(G, eps=0.0, out_dtype=torch.float32)
    assert g.gemm_last_status(stream()) == g.GEMM_OK
    close(O, reference(G, eps=0.0), tolerance(5, torch.float32))
    O = g.newton_schulz(G[:5], out_dtype=torch.float32)
    close(O[[0, 1, 3, 4]], reference(G[[0, 1, 3, 4]]), tolerance(5, torch.float32))


@pytest.mark.parametrize("rows, cols", [(256, 256), (300, 70), (64, 3000), (384, 1030)])
@pytest.mark.parametrize("norm", [1e-9, 1e-11, 1e-12, 1e-14, 1e-20, 1e-36])
@pytest.mark.parametrize("steps", [1, 5, 12])
def test_norms_below_eps(rows, cols, norm, steps):
    """X = G / (|G| + eps) far below 1, as an idle expert's decayed momentum gives.

    As long as every step leaves |X| <= 2^-10 the products add less than 2^-17 of X,
    whose rounding to 16 bits does not show: what is left is X's own.  With entries
    of 1 / (8 sqrt m) or more times their power of two (m <= 384: 2^-7.3, and up to
    2 times less while a step's growth is counted in whole powers), halves of quantum
    2^-24 are off by 2^-25 at most: 2^-16 a step and for the first rounding."""
    gen = torch.Generator("cuda").manual_seed(rows + steps)
    G = torch.randn(rows, cols, device="cuda", generator=gen)
    G *= norm / G.norm()
    O = g.newton_schulz(G, steps=steps, out_dtype=torch.float32)
    assert g.gemm_last_status(stream()) == g.GEMM_OK
    small = norm / 1e-7 * 3.4445 ** steps <= 2.0 ** -10
    close(O, reference(G, steps), (steps + 1) * 2.0 ** -16 if small else tolerance(steps, torch.float32))


@pytest.mark.parametrize("rows, cols", [(200, 520), (520, 200), (1100, 1040)])
def test_batch_of_norms_around_eps(rows, cols):
    """Each matrix has its own power of two: nothing of one reaches another; the
    cubic's steps, a larger eps, a bf16 result."""
    gen = torch.Generator("cuda").manual_seed(8)
    G = torch.randn(6, rows, cols, device="cuda", generator=gen)
    norms = torch.tensor([1.0, 1e-8, 1e-12, 1e-16, 3e4, 0.0], device="cuda")
    G *= (norms / G.square().sum((1, 2)).sqrt())[:, None, None]
    for steps, coefficients, eps in ((5, g.NEWTON_SCHULZ_COEFFICIENTS, 1e-7), (14, (1.5, -0.5, 0.0), 1e-7),
                                     (7, g.NEWTON_SCHULZ_COEFFICIENTS, 50.0)):
        want = reference(G, steps, coefficients, eps)
        for dtype in (torch.float32, torch.bfloat16):
            O = g.newton_schulz(G, steps=steps, coefficients=coefficients, eps=eps, out_dtype=dtype)
            assert g.gemm_last_status(stream()) == g.GEMM_OK
            assert (O[5] == 0).all()
            close(O[:5], want[:5], tolerance(steps, dtype))


@pytest.mark.parametrize("batch, rows, cols, ctas, nt, lt", [
    (1, 2500, 2700, 2, 256, 256), (1, 2701, 2497, 2, 256, 256),    # every product on pairs, both orientations
    (4, 1101, 1490, 2, 256, 256), (4, 1490, 1101, 2, 256, 256),
    (12, 513, 770, 1, 128, 128), (8, 901, 700, 1, 128, 128),       # the symmetric ones on pairs
    (2, 1301, 1504, 2, 256, 256), (2, 1504, 1301, 2, 256, 256),    # the symmetric ones in tiles of 128 x 128
    (30, 900, 300, 1, 128, 128), (40, 200, 300, 1, 128, 128), (30, 300, 900, 1, 64, 128)])
def test_large_tiles(batch, rows, cols, ctas, nt, lt):
    """Sizes whose products take pairs and 128 x 128 tiles; the last product says so."""
    gen = torch.Generator("cuda").manual_seed(rows)
    G = torch.randn(batch, rows, cols, device="cuda", generator=gen)
    want = reference(G)
    for dtype, pad in ((torch.float32, 0), (torch.bfloat16, 1)):
        flat = torch.full((batch * rows * (cols + pad),), float("nan"), dtype=dtype, device="cuda")
        O = flat.view(batch, rows, cols + pad)[..., :cols]
        g.newton_schulz(G, out=O)
        assert g.gemm_last_status(stream()) == g.GEMM_OK
        s = g.gemm_last_schedule()
        assert (s["ctas_per_cluster"], s["dp_tiles"]) == (ctas, batch * -(-rows // nt) * -(-cols // lt))
        close(O, want, tolerance(5, dtype))
        assert torch.equal(O, g.newton_schulz(G, out_dtype=dtype))
        O.fill_(float("nan"))
        assert flat.isnan().all(), "wrote outside the output"
