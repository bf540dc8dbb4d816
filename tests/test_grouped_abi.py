"""Argument checks of the expert-training operators' C entry points, which
come before any device work: no GPU is needed."""
import pytest

import dense_gemm_blackwell_tcgen05_gb300 as g

FAKE = 0x7F0000000000   # never dereferenced: every case fails validation first
INVALID, ALIGN = g.GEMM_ERR_INVALID_ARG, g.GEMM_ERR_ALIGNMENT


def rows_call(entry, **k):
    """The forward entry point's arguments, or dgrad's with the roles of N and K swapped."""
    a = dict(X=FAKE, B=FAKE, out=FAKE, offsets=FAKE, groups=2, M=8, N=24, K=16, ldx=None, ldb=16, stride=24 * 16,
             ldo=None, dtype=g.DTYPE_BF16)
    a.update(k)
    fwd = entry is g.gemm_bf16_grouped
    ldx = a["ldx"] if a["ldx"] is not None else (a["K"] if fwd else a["N"])
    ldo = a["ldo"] if a["ldo"] is not None else (a["N"] if fwd else a["K"])
    return entry(a["X"], a["B"], a["out"], a["offsets"], a["groups"], a["M"], a["N"], a["K"], ldx, a["ldb"],
                 a["stride"], ldo, a["dtype"], 0)


@pytest.mark.parametrize("entry", [g.gemm_bf16_grouped, g.gemm_bf16_grouped_dgrad])
@pytest.mark.parametrize("change, want", [
    (dict(M=-1), INVALID), (dict(N=1 << 31), INVALID), (dict(K=-8), INVALID),
    (dict(groups=-1), INVALID), (dict(groups=g.MAX_GROUPS + 1), INVALID),
    (dict(dtype=2), INVALID), (dict(offsets=0), INVALID), (dict(offsets=FAKE + 2), ALIGN),
    (dict(X=0), INVALID), (dict(B=0), INVALID), (dict(out=0), INVALID),
    (dict(X=FAKE + 8), ALIGN), (dict(B=FAKE + 2), ALIGN), (dict(out=FAKE + 1), ALIGN),
    (dict(out=FAKE + 2, dtype=g.DTYPE_F32), ALIGN),
    (dict(ldx=8), INVALID), (dict(ldx=28), ALIGN), (dict(ldb=8), INVALID), (dict(ldb=20, stride=24 * 20), ALIGN),
    (dict(ldo=8), INVALID), (dict(stride=24 * 16 - 8), INVALID), (dict(stride=24 * 16 + 4), ALIGN),
    (dict(stride=1 << 40), INVALID),
    (dict(M=0), g.GEMM_OK), (dict(groups=0, offsets=0), g.GEMM_OK),
])
def test_rows_validation(entry, change, want):
    assert rows_call(entry, **change) == want


def wgrad_call(**k):
    a = dict(dD=FAKE, A=FAKE, out=FAKE, offsets=FAKE, groups=2, M=8, N=24, K=16, ldd=24, lda=16, ldo=16,
             stride=24 * 16, dtype=g.DTYPE_F32, accumulate=0)
    a.update(k)
    return g.gemm_bf16_grouped_wgrad(a["dD"], a["A"], a["out"], a["offsets"], a["groups"], a["M"], a["N"], a["K"],
                                     a["ldd"], a["lda"], a["ldo"], a["stride"], a["dtype"], a["accumulate"], 0)


@pytest.mark.parametrize("change, want", [
    (dict(M=-1), INVALID), (dict(groups=g.MAX_GROUPS + 1), INVALID), (dict(dtype=-1), INVALID),
    (dict(accumulate=2), INVALID), (dict(dD=0), INVALID), (dict(A=0), INVALID), (dict(out=0), INVALID),
    (dict(out=FAKE + 2), ALIGN), (dict(dD=FAKE + 4), ALIGN), (dict(ldd=28), ALIGN), (dict(lda=20), ALIGN),
    (dict(ldd=16), INVALID), (dict(ldo=15), INVALID), (dict(stride=24 * 16 - 1), INVALID),
    (dict(N=0), g.GEMM_OK), (dict(K=0), g.GEMM_OK), (dict(groups=0), g.GEMM_OK),
])
def test_wgrad_validation(change, want):
    assert wgrad_call(**change) == want


def ns_call(**k):
    a = dict(G=FAKE, O=FAKE, batch=2, rows=8, cols=16, ldg=16, sg=128, ldo=16, so=128, i=g.DTYPE_F32, o=g.DTYPE_BF16,
             steps=5, abc=g.NEWTON_SCHULZ_COEFFICIENTS, eps=1e-7, ws=FAKE, n=None)
    a.update(k)
    n = a["n"] if a["n"] is not None else max(0, g.gemm_newton_schulz_workspace_bytes(a["batch"], a["rows"], a["cols"]))
    return g.gemm_newton_schulz(a["G"], a["O"], a["batch"], a["rows"], a["cols"], a["ldg"], a["sg"], a["ldo"], a["so"],
                                a["i"], a["o"], a["steps"], *a["abc"], a["eps"], a["ws"], n, 0)


@pytest.mark.parametrize("change, want", [
    (dict(batch=-1), INVALID), (dict(batch=65536), INVALID), (dict(rows=-1), INVALID), (dict(cols=65537), INVALID),
    (dict(i=2), INVALID), (dict(o=7), INVALID), (dict(steps=0), INVALID), (dict(steps=65), INVALID),
    (dict(abc=(float("inf"), 0.0, 0.0)), INVALID), (dict(eps=-1e-7), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(G=0), INVALID), (dict(O=0), INVALID), (dict(ldg=15), INVALID), (dict(ldo=15), INVALID),
    (dict(sg=127), INVALID), (dict(so=127), INVALID), (dict(G=FAKE + 2), ALIGN), (dict(O=FAKE + 1), ALIGN),
    (dict(ws=0), INVALID), (dict(ws=FAKE + 16), ALIGN), (dict(n=1024), INVALID),
    (dict(batch=0), g.GEMM_OK), (dict(rows=0), g.GEMM_OK), (dict(cols=0), g.GEMM_OK),
])
def test_newton_schulz_validation(change, want):
    assert ns_call(**change) == want


def test_newton_schulz_workspace():
    f = g.gemm_newton_schulz_workspace_bytes
    assert f(1, 256, 256) >= 4 * 256 * 256 * 2 + 2 * 256 * 256 * 2
    assert f(-1, 4, 4) == INVALID and f(1, 65537, 4) == INVALID


@pytest.mark.parametrize("rows, ld", [((1 << 31) - 1, 1 << 33), (1 << 30, 1 << 33), ((1 << 31) - 1, (1 << 36) - 8),
                                      (1 << 28, 1 << 36)])
def test_stride_shorter_than_a_product_past_64_bits(rows, ld):
    """rows * pitch is compared as it is, not as what is left of it in 64 bits."""
    wide = (rows + 7) // 8 * 8
    for entry in (g.gemm_bf16_grouped, g.gemm_bf16_grouped_dgrad):
        assert rows_call(entry, N=rows, ldx=wide, ldo=wide, ldb=ld, stride=1 << 38) == INVALID
    assert wgrad_call(N=rows, ldd=wide, ldo=ld, stride=1 << 38) == INVALID
