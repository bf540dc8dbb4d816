"""Distillation where a row's entries crowd a tile, lie on both sides of its borders, come many times or
are few, over widths of one and of several segments, on single CTAs and on pairs.  Logits of small
integers, exact in fp32, as in test_losses."""
import pytest
import torch

import dense_gemm_blackwell_tcgen05_gb300 as g
from tests import loss_reference as ref
from tests.test_losses import BF16, F32, gen, marked, ok, only_inside, problem, scale_of

pytestmark = pytest.mark.gpu


def crowded(r, M, N, top):
    """ids about one place a row, some of all rows at tiles' and chunks' borders, some far away, many twice."""
    at = torch.randint(0, N, (M, 1), generator=r, device="cuda")
    ids = (at + torch.randint(-20, 21, (M, top), generator=r, device="cuda")).clamp(0, N - 1)
    borders = torch.tensor([0, 31, 32, 63, 64, 95, 96, 127, 128, 129, 255, 256, N - 2, N - 1], device="cuda").clamp(0, N - 1)
    pick = borders[torch.randint(0, len(borders), (M, top), generator=r, device="cuda")]
    ids = torch.where(torch.rand(M, top, generator=r, device="cuda") < 0.3, pick, ids)
    far = torch.randint(0, N, (M, top), generator=r, device="cuda")
    ids = torch.where(torch.rand(M, top, generator=r, device="cuda") < 0.2, far, ids)
    ids[M // 2] = ids[M // 2, 0].clone()                            # one token, `top` times
    ids[torch.rand(M, top, generator=r, device="cuda") < 0.1] = -1
    ids[M // 3] = -1                                             # none
    ids[M - 1, 1:] = -1                                          # one entry
    ids[M - 1, 0] = N - 1
    ids[0] = torch.arange(top, device="cuda") % N                # a run of them
    return ids


# rows, tokens, width, entries; CTAs of the logits' tiles
SIZES = [(5, 300, 520, 3, 1), (5, 300, 1100, 64, 1), (100, 1000, 2056, 17, 1), (128, 129, 1040, 100, 1), (40, 4000, 600, 1024, 1),
         (300, 700, 520, 9, 1), (300, 700, 1040, 8, 1), (300, 600, 1096, 200, 1), (200, 30000, 1040, 5, 2), (700, 20000, 520, 40, 2),
         (700, 20000, 1032, 128, 2), (1500, 9000, 2056, 1, 2), (257, 40000, 1544, 300, 2), (700, 20000, 264, 40, 2),
         (100, 1000, 200, 64, 1)]


@pytest.mark.parametrize("M, N, K, top, ctas", SIZES)
def test_crowded_lists(M, N, K, top, ctas):
    r, A, B = problem(M, N, K, True, seed=21)
    f = 2.0 / scale_of(K, True)
    ids = crowded(r, M, N, top)
    teacher = 2.0 * torch.randn(M, top, generator=r, device="cuda")
    t, entropy, live = ref.teacher_matrix(teacher, ids, N, f)
    assert not live[M // 3]
    loss, lse = g.matmul_distill(A, B, teacher, ids, temperature=f)
    assert g.gemm_last_schedule()["ctas_per_cluster"] == ctas
    ok()
    want, want_lse = ref.forward(A, B, t, entropy, live, 1.0 / f)
    e_loss, e_lse = ref.forward_bounds(A, B, t, 1.0 / f, want_lse, 0.0, True)
    # p is off by 2^-21 (1 + |teacher / T|) of itself, times its terms
    size = teacher.double().abs().max(1)[0] / f + 1.0
    big = ref.logits(A, B, 1.0 / f).abs().max(1)[0] + want_lse.abs()
    ref.check(lse, want_lse, torch.where(live, e_lse, 0.0), "lse")
    ref.check(loss, want, torch.where(live, e_loss + 2.0 ** -20 * size * (big + entropy.abs() + size), 0.0), "loss")
    dloss = torch.randn(M, generator=r, device="cuda")
    (_, dA), (_, dB) = bufs = marked(M, K, F32, 8), marked(N, K, BF16, 8)
    g.matmul_distill_grad(dloss, A, B, teacher, ids, want_lse.float(), temperature=f, dA=dA, dB=dB)
    ok()
    (ra, ta), (rb, tb) = ref.gradients(A, B, t, live, dloss, want_lse.float(), 1.0 / f, 0.0, F32, BF16, True)
    off = 2.0 ** -20 * torch.where(live, dloss.double().abs() / f * size, 0.0)[:, None] * t
    ref.check(dA, ra, ta + off @ B.double().abs(), "dA")
    ref.check(dB, rb, tb + off.T @ torch.where(live[:, None], A.double().abs(), 0.0), "dB")
    for buf, view in bufs:
        only_inside(buf, view)
    # as a whole: no entry of a crowd is lost (dz to bf16, and a bf16 dB: 2^-8 of each element at most)
    for got, ref_ in ((dA, ra), (dB, rb)):
        assert (got.double() - ref_).norm() <= 2.0 ** -7 * ref_.norm()


@pytest.mark.parametrize("K", [64, 520, 1544])
@pytest.mark.parametrize("M", [40, 300, 700])
def test_every_entry_of_the_gradient_in_wide_products(M, K):
    """B selects elements: the logits' gradient itself, entry by entry, for targets and for lists."""
    N, f = 64, 1.0
    r = gen(M + K)
    B = torch.zeros(N, K, dtype=BF16, device="cuda")
    cols = torch.randperm(K, generator=r, device="cuda")[:N]     # (each token has a column of its own)
    B[torch.arange(N, device="cuda"), cols] = 1.0
    A = torch.zeros(M, K, dtype=BF16, device="cuda")
    A[:, cols] = torch.randint(-6, 7, (M, N), generator=r, device="cuda").to(BF16)
    dloss = torch.randn(M, generator=r, device="cuda")
    targets = torch.arange(M, device="cuda") % N
    ids = crowded(r, M, N, 20)
    teacher = 2.0 * torch.randn(M, 20, generator=r, device="cuda")
    zero = torch.zeros(M, device="cuda", dtype=torch.float64)
    for listed in (False, True):
        t, entropy, live = ref.teacher_matrix(teacher, ids, N, f) if listed else \
            (ref.target_matrix(targets, N, 0.1), zero, targets >= 0)
        lse = ref.forward(A, B, t, entropy, live, f)[1].float()
        if listed:
            dA, _ = g.matmul_distill_grad(dloss, A, B, teacher, ids, lse, need_dB=False)
        else:
            dA, _ = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, label_smoothing=0.1, need_dB=False)
        ok()
        dz, size = ref.dlogits(A, B, t, live, dloss, lse, f)
        # one rounding to bf16 of dz, another of dA; a list's p is off by 2^-20 (1 + 12)
        ref.check(dA[:, cols], dz, 2.0 ** -7 * 1.01 * dz.abs() + size * 2.0 ** -15, "dz")
        rest = torch.ones(K, dtype=torch.bool, device="cuda")
        rest[cols] = False
        assert not dA[:, rest].any()
