"""Argument checks of the losses' C entry points, which come before any device
work, what the Python calls refuse, and the reference forms that the GPU tests
use, against automatic differentiation and differences: no GPU is needed."""
import pytest
import torch

import dense_gemm_blackwell_tcgen05_gb300 as g
from tests import loss_reference as ref

FAKE = 0x7F0000000000   # never dereferenced: every case fails validation first
INVALID, ALIGN, OK = g.GEMM_ERR_INVALID_ARG, g.GEMM_ERR_ALIGNMENT, g.GEMM_OK
NAN, INF = float("nan"), float("inf")
BIG = 1 << 40


def ce(**k):
    a = dict(A=FAKE, B=FAKE, targets=FAKE, loss=FAKE, lse=FAKE, M=8, N=24, K=16, lda=16, ldb=16, code=g.INDEX_I64, scale=1.0,
             smoothing=0.0, z=0.0, ws=FAKE, n=BIG)
    a.update(k)
    return g.gemm_bf16_cross_entropy(*a.values())


def ce_grad(**k):
    a = dict(dloss=FAKE, A=FAKE, B=FAKE, targets=FAKE, lse=FAKE, dA=FAKE, dB=FAKE, M=8, N=24, K=16, inc=1, lda=16, ldb=16,
             ld_da=16, ld_db=16, code=g.INDEX_I32, ca=g.DTYPE_BF16, cb=g.DTYPE_F32, scale=1.0, smoothing=0.0, z=0.0, acc=0,
             ws=FAKE, n=BIG)
    a.update(k)
    return g.gemm_bf16_cross_entropy_grad(*a.values())


def kd(**k):
    a = dict(A=FAKE, B=FAKE, teacher=FAKE, ids=FAKE, loss=FAKE, lse=FAKE, M=8, N=24, K=16, top=4, lda=16, ldb=16, ldt=4, ldi=4,
             ct=g.DTYPE_F32, ci=g.INDEX_I32, t=1.0, ws=FAKE, n=BIG)
    a.update(k)
    return g.gemm_bf16_distill(*a.values())


def kd_grad(**k):
    a = dict(dloss=FAKE, A=FAKE, B=FAKE, teacher=FAKE, ids=FAKE, lse=FAKE, dA=FAKE, dB=FAKE, M=8, N=24, K=16, top=4, inc=0,
             lda=16, ldb=16, ldt=4, ldi=4, ld_da=16, ld_db=16, ct=g.DTYPE_BF16, ci=g.INDEX_I64, ca=g.DTYPE_F32,
             cb=g.DTYPE_BF16, t=1.0, acc=0, ws=FAKE, n=BIG)
    a.update(k)
    return g.gemm_bf16_distill_grad(*a.values())


COMMON = [
    (dict(M=-1), INVALID), (dict(N=1 << 31), INVALID), (dict(K=-8), INVALID), (dict(N=0), INVALID),
    (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(A=FAKE + 8), ALIGN), (dict(B=FAKE + 2), ALIGN),
    (dict(lda=8), INVALID), (dict(lda=20), ALIGN), (dict(ldb=20), ALIGN), (dict(ldb=(1 << 36) + 8), INVALID),
    (dict(lse=0), INVALID), (dict(lse=FAKE + 2), ALIGN),
    (dict(ws=0), INVALID), (dict(ws=FAKE + 128), ALIGN), (dict(n=64), INVALID),
]
FORWARD = [(dict(loss=0), INVALID), (dict(loss=FAKE + 1), ALIGN), (dict(M=0), OK), (dict(M=0, N=0), OK)]
BACKWARD = [
    (dict(dloss=0), INVALID), (dict(dloss=FAKE + 2), ALIGN), (dict(inc=-1), INVALID), (dict(acc=2), INVALID),
    (dict(ca=2), INVALID), (dict(cb=-1), INVALID), (dict(dA=FAKE + 1), ALIGN), (dict(dB=FAKE + 1), ALIGN),
    (dict(ld_da=15), INVALID), (dict(ld_db=8), INVALID), (dict(dA=0, dB=0), OK), (dict(K=0), OK), (dict(M=0, N=0), OK),
    (dict(M=0, acc=1), OK), (dict(M=0, dB=0), OK),
]
TARGET = [
    (dict(targets=0), INVALID), (dict(targets=FAKE + 2), ALIGN), (dict(code=2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(scale=3e38), INVALID),
    (dict(smoothing=-0.1), INVALID), (dict(smoothing=1.5), INVALID), (dict(smoothing=NAN), INVALID),
    (dict(z=INF), INVALID), (dict(z=NAN), INVALID),
]
LIST = [
    (dict(top=0), INVALID), (dict(top=g.MAX_TOP + 1, ldt=2000, ldi=2000), INVALID), (dict(teacher=0), INVALID),
    (dict(ids=0), INVALID), (dict(teacher=FAKE + 1), ALIGN), (dict(ids=FAKE + 2), ALIGN), (dict(ldt=3), INVALID),
    (dict(ldi=3), INVALID), (dict(ct=2), INVALID), (dict(ci=-1), INVALID), (dict(t=0.0), INVALID), (dict(t=-1.0), INVALID),
    (dict(t=NAN), INVALID), (dict(t=INF), INVALID), (dict(t=1e-45), INVALID), (dict(t=3e-39), INVALID),
]


@pytest.mark.parametrize("call, change, want",
                         [(c, *x) for c in (ce, ce_grad, kd, kd_grad) for x in COMMON]
                         + [(c, *x) for c in (ce, kd) for x in FORWARD] + [(c, *x) for c in (ce_grad, kd_grad) for x in BACKWARD]
                         + [(c, *x) for c in (ce, ce_grad) for x in TARGET] + [(c, *x) for c in (kd, kd_grad) for x in LIST])
def test_validation(call, change, want):
    assert call(**change) == want


@pytest.mark.parametrize("call, change", [(ce, dict(targets=FAKE + 4)), (kd_grad, dict(ids=FAKE + 4)), (kd_grad, dict(dA=FAKE + 2)),
                                          (ce_grad, dict(dB=FAKE + 2))])
def test_alignment_follows_the_type(call, change):
    assert call(**change) == ALIGN


def test_workspace_bytes():
    for bad in ((-1, 8, 8), (8, 1 << 31, 8), (8, 8, -1)):
        assert g.gemm_bf16_cross_entropy_workspace_bytes(*bad, 0) == INVALID
        assert g.gemm_bf16_distill_workspace_bytes(*bad, 4, 1) == INVALID
    assert g.gemm_bf16_cross_entropy_workspace_bytes(8, 8, 8, 2) == INVALID
    assert g.gemm_bf16_distill_workspace_bytes(8, 8, 8, 0, 0) == INVALID
    assert g.gemm_bf16_distill_workspace_bytes(8, 8, 8, g.MAX_TOP + 1, 0) == INVALID
    assert g.gemm_bf16_cross_entropy_workspace_bytes(0, 8, 8, 1) == 0
    for M, N, K in ((1, 1, 1), (1, 1 << 28, 8), (128, 1 << 24, 96), (300, 5000, 96), (8192, 131072, 4096), (100000, 50021, 1040)):
        forward, back = (g.gemm_bf16_cross_entropy_workspace_bytes(M, N, K, x) for x in (0, 1))
        # nothing like the logits: what the header says, and room for vectors
        assert forward <= 2 * M * (K + 64) + M * N // 16 * 1.6 + 64 * M * 4 + 65536
        assert back <= 6 * M * (K + 64) + max(1 << 29, 2 * M * 4096) * 1.1 + 64 * M + 65536
        assert g.gemm_bf16_distill_workspace_bytes(M, N, K, 8, 0) > forward


# ------------------------------------------------------------------ Python

def cpu(M=8, N=24, K=16):
    return (torch.zeros(M, K, dtype=torch.bfloat16), torch.zeros(N, K, dtype=torch.bfloat16))


def test_python_refusals():
    A, B = cpu()
    t, f = torch.zeros(8, dtype=torch.int64), torch.zeros(8)
    teacher, ids = torch.zeros(8, 4), torch.zeros(8, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        g.matmul_cross_entropy(A, B, t)
    with pytest.raises(ValueError, match="CUDA"):
        g.matmul_cross_entropy_grad(f, A, B, t, f)
    with pytest.raises(ValueError, match="CUDA"):
        g.matmul_distill(A, B, teacher, ids)
    with pytest.raises(ValueError, match="CUDA"):
        g.matmul_distill_grad(f, A, B, teacher, ids, f)
    for bad in (A[0], A.T, A[None]):
        with pytest.raises(ValueError, match="2-D"):
            g.matmul_cross_entropy(bad, B, t)
        with pytest.raises(ValueError, match="2-D"):
            g.matmul_distill(bad, B, teacher, ids)
    with pytest.raises(TypeError, match="int32 or int64"):
        g.matmul_cross_entropy(A, B, f)
    with pytest.raises(TypeError, match="int32 or int64"):
        g.matmul_distill(A, B, teacher, teacher)
    with pytest.raises(ValueError, match="accumulate"):
        g.matmul_cross_entropy_grad(f, A, B, t, f, accumulate=True)
    with pytest.raises(ValueError, match="accumulate"):
        g.matmul_distill_grad(f, A, B, teacher, ids, f, accumulate=True)
    with pytest.raises(ValueError, match="shape"):
        g.matmul_cross_entropy_grad(f, A, B, t, f, dB=A)
    assert g.MAX_TOP == 1024


@pytest.mark.parametrize("value, name, kind", [
    (torch.zeros(7), "x", ValueError), (torch.zeros(8, 1), "x", ValueError), (torch.zeros(8), "x", ValueError)])
def test_row_values(value, name, kind):
    with pytest.raises(kind):
        g._row_values(value, name, 8)


def test_types_of_indices():
    assert g._index_code(torch.int32) == g.INDEX_I32 and g._index_code(torch.int64) == g.INDEX_I64
    for t in (torch.int16, torch.float32, torch.uint8):
        with pytest.raises(TypeError):
            g._index_code(t)


# --------------------------------------------------------------- reference

@pytest.mark.parametrize("listed", [False, True])
def test_reference_gradients_are_those_of_the_losses(listed):
    """The reference's gradients against automatic differentiation of its losses and against differences."""
    r = torch.Generator().manual_seed(3)
    M, N, K, scale, z_loss = 7, 13, 5, 0.7, 0.0 if listed else 0.03
    A, B = torch.randn(M, K, generator=r).double(), torch.randn(N, K, generator=r).double()
    if listed:
        ids = torch.randint(-2, N, (M, 4), generator=r)
        ids[2] = -1
        teacher = 3.0 * torch.randn(M, 4, generator=r)
        teacher[1, 1] = -INF
        t, entropy, live = ref.teacher_matrix(teacher, ids, N, 1.0 / scale)
        assert not live[2] and live.sum() >= 4
        for i in range(M):   # the definition, entry by entry
            there = [(int(v), float(x) * scale) for v, x in zip(ids[i], teacher[i]) if v >= 0 and x > -INF]
            total = sum(torch.tensor(x, dtype=torch.float64).exp() for _, x in there)
            for v in range(N):
                p = sum(torch.tensor(x, dtype=torch.float64).exp() / total for w, x in there if w == v)
                assert abs(float(t[i, v]) - float(p)) < 1e-7
    else:
        targets = torch.tensor([0, 12, -100, 5, 5, -1, 7])
        t, entropy, live = ref.target_matrix(targets, N, 0.1), torch.zeros(M).double(), targets >= 0
    d = torch.randn(M, generator=r).double()
    a, b = A.clone().requires_grad_(), B.clone().requires_grad_()
    z = scale * a @ b.T
    lse = torch.logsumexp(z, 1)
    loss = torch.where(live, entropy + lse * t.sum(1) - (t * z).sum(1) + z_loss * lse.square(), torch.zeros(M).double())
    want, want_lse = ref.forward(A, B, t, entropy, live, scale, z_loss)
    assert torch.allclose(loss, want, atol=1e-12)
    if not listed:
        plain = torch.nn.functional.cross_entropy(z, targets.clamp(min=0), reduction="none", label_smoothing=0.1)
        assert torch.allclose(torch.where(live, plain + z_loss * lse.square(), torch.zeros(M).double()), want, atol=1e-6)
    (loss * d).sum().backward()
    (ra, _), (rb, _) = ref.gradients(A, B, t, live, d, want_lse, scale, z_loss)
    assert torch.allclose(a.grad, ra, atol=1e-10) and torch.allclose(b.grad, rb, atol=1e-10)
    step = 1e-5
    for which, grad in ((0, ra), (1, rb)):
        x = torch.randn((A, B)[which].shape, generator=r).double()
        up, down = [[A, B], [A, B]]
        up, down = list(up), list(down)
        up[which], down[which] = (A, B)[which] + step * x, (A, B)[which] - step * x
        f = [(ref.forward(*ab, t, entropy, live, scale, z_loss)[0] * d).sum() for ab in (up, down)]
        assert abs((f[0] - f[1]) / (2 * step) - (grad * x).sum()) < 1e-6 * (1.0 + (grad * x).abs().sum())
