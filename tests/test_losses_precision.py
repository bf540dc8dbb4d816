"""Losses over a vocabulary where rounding shows: large logits, sure tokens, a
teacher's extreme logits, gradients of sure rows over wide products."""
import pytest
import torch

import dense_gemm_blackwell_tcgen05_gb300 as g
from tests import loss_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def ok():
    assert g.gemm_last_status(torch.cuda.current_stream().cuda_stream) == g.GEMM_OK


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def shifted(M, N, K, shift, seed):
    """A, B of small integers, and `shift` in all of a row's logits: exact in fp32."""
    r = gen(seed + M + N)
    ints = lambda *s: torch.randint(-2, 3, s, generator=r, device="cuda").to(BF16)  # noqa: E731
    A, B = ints(M, K), ints(N, K)
    A[:, 0], B[:, 0] = shift, 1.0
    return r, A, B


def scale_and_temperature(x):
    """About x in fp32, and the temperature for which a call takes it."""
    t = torch.tensor(1.0 / x)
    return float(1.0 / t), float(t)


def spread(z):
    return z.max(1)[0] - z.min(1)[0]


# few rows in place, one block of rows in runs, many rows
SIZES = [(40, 300), (100, 30000), (400, 3000)]


@pytest.mark.parametrize("scale", [0.25, 0.3])
@pytest.mark.parametrize("shift", [-8192.0, 0.0, 8192.0])
@pytest.mark.parametrize("M, N", SIZES)
def test_a_loss_is_as_exact_as_its_logits_differences(M, N, shift, scale):
    """What all of a row's logits share is no part of its loss, nor of the loss's error: 2^-19 of
    the sums of exponentials, and roundings of differences of logits."""
    r, A, B = shifted(M, N, 64, shift, 1)
    f, temperature = scale_and_temperature(scale)
    z = ref.logits(A, B, f)
    targets = torch.randint(0, N, (M,), generator=r, device="cuda")
    live = torch.ones(M, dtype=torch.bool, device="cuda")
    zero = torch.zeros(M, dtype=torch.float64, device="cuda")
    bound = 2.0 ** -19 + 2.0 ** -21 * (spread(z) + 1.0)
    for smoothing in (0.0, 0.1):
        loss, _ = g.matmul_cross_entropy(A, B, targets, scale=f, label_smoothing=smoothing)
        ok()
        # (the mean of the logits is off by what sums of them cost)
        more = smoothing * 2.0 ** -21 * z.abs().mean(1)
        ref.check(loss, ref.forward(A, B, ref.target_matrix(targets, N, smoothing), zero, live, f)[0], bound + more, "loss")
    ids = torch.randint(0, N, (M, 9), generator=r, device="cuda", dtype=torch.int32)
    teacher = torch.randn(M, 9, generator=r, device="cuda")
    t, entropy, live = ref.teacher_matrix(teacher, ids, N, 1.0 / f)
    loss, _ = g.matmul_distill(A, B, teacher, ids, temperature=temperature)
    ok()
    # p is off by 2^-21 size of itself
    size = teacher.double().abs().max(1)[0] * f + 1.0
    ref.check(loss, ref.forward(A, B, t, entropy, live, f)[0],
              bound + 2.0 ** -20 * size * (spread(z) + 20.0 + entropy.abs() + size), "divergence")


@pytest.mark.parametrize("M, N", SIZES)
def test_a_sure_token_loses_what_is_left(M, N):
    """The target's logit stands out by up to 1000 over others of 0: log(1 + (N - 1) exp(-z)), never
    below 0, whatever the logit's size."""
    K = 64
    A, B = torch.zeros(M, K, dtype=BF16, device="cuda"), torch.zeros(N, K, dtype=BF16, device="cuda")
    sure = torch.tensor([8.0, 11.5, 20.25, 61.0, 203.0, 1000.0], device="cuda").to(BF16).repeat(M)[:M]
    A[:, 3] = sure
    for scale in (1.0, 0.7):
        f, temperature = scale_and_temperature(scale)
        for t in (0, N // 2, N - 1):
            B.zero_()
            B[t, 3] = 1.0
            targets = torch.full((M,), t, device="cuda")
            loss, _ = g.matmul_cross_entropy(A, B, targets, scale=f)
            ids = targets[:, None].int()
            kd, _ = g.matmul_distill(A, B, torch.zeros(M, 1, device="cuda"), ids, temperature=temperature)
            ok()
            want = torch.log1p((N - 1) * torch.exp(-f * sure.double()))
            for got in (loss, kd):
                assert (got >= 0).all()
                ref.check(got, want, 2.0 ** -19 + 2.0 ** -21 * want, "loss")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("temperature", [0.25, 0.5, 1.0, 4.0])
@pytest.mark.parametrize("M, top", [(40, 5), (300, 5), (300, 200)])
def test_a_teachers_extreme_logits(M, top, temperature, dtype):
    """Finite logits are entries, the type's lowest value and what leaves fp32 once it is divided by
    the temperature too; only a logit of -Inf is not there."""
    N, K = 500, 64
    r, A, B = shifted(M, N, K, 0.0, 2)
    lowest = torch.finfo(dtype).min
    ids = torch.randint(0, N, (M, top), generator=r, device="cuda", dtype=torch.int32)
    teacher = torch.randn(M, top, generator=r, device="cuda").to(dtype)
    teacher[0::4, 1:] = lowest               # masked entries beside one that is not
    teacher[1::4] = lowest                   # nothing but them: they are alike
    teacher[2::4, 0] = -lowest               # one that is far ahead
    teacher[3::4, :2] = -lowest              # two
    teacher[5, :] = -torch.inf
    teacher[9, 1:] = -torch.inf
    t, entropy, live = ref.teacher_matrix(teacher.double(), ids, N, temperature)
    assert live.sum() == M - 1
    f = 1.0 / temperature
    want, want_lse = ref.forward(A, B, t, entropy, live, f)
    loss, lse = g.matmul_distill(A, B, teacher, ids, temperature=temperature)
    dloss = torch.rand(M, generator=r, device="cuda")
    dA, _ = g.matmul_distill_grad(dloss, A, B, teacher, ids, want_lse.float(), temperature=temperature, out_dtype=F32)
    ok()
    e_loss, e_lse = ref.forward_bounds(A, B, t, f, want_lse, 0.0, True)
    ref.check(lse, want_lse, torch.where(live, e_lse, 0.0), "lse")
    # p is off by 2^-21 (1 + the difference to the largest) of itself: under 2^-18 where it counts
    size = ref.logits(A, B, f).abs().max(1)[0] + want_lse.abs() + entropy.abs() + 1.0
    ref.check(loss, want, torch.where(live, e_loss + 2.0 ** -17 * size, 0.0), "loss")
    (ra, ta), _ = ref.gradients(A, B, t, live, dloss, want_lse.float(), f, dA=F32, dB=F32, exact=True)
    more = 2.0 ** -17 * torch.where(live, dloss.double() * f, 0.0)[:, None] * t
    # what lies below fp32's 2^-126 becomes 0: 500 terms of it, times 2 of B and 4 of dloss / temperature
    ref.check(dA, ra, ta + more @ B.double().abs() + 2.0 ** -114, "dA")


@pytest.mark.parametrize("M", [1, 130, 300])
@pytest.mark.parametrize("K", [504, 1040, 4096, 8192])
def test_a_sure_rows_gradient_over_a_wide_product(M, K):
    """Rows that leave 5e-3 to 1e-5 to the other tokens: 1 - exp(z - lse) is what the logits' error
    must not reach.  dB's row of a target, along the row of A, is that row's dz.

    Logits are added up over 512 terms (1.1e-9 of the result a term, cut off; twice that allowed) and
    then with a rounding a segment; exp takes 2^-21 (1 + |lse|) of its own; dz is rounded to bf16
    (up to 128 rows, twice); the product to dB costs 2^-17 of what it adds up."""
    N = 2000
    r = gen(M + K)
    A = ((torch.rand(M, K, generator=r, device="cuda") + 0.5) * torch.randn(M, K, generator=r, device="cuda").sign()).to(BF16)
    a = A.double()
    length = a.square().sum(1)
    z_want = 16.0 + 1.5 * (torch.arange(M, device="cuda") % 5 - 2)
    B = torch.zeros(N, K, device="cuda")
    B[:M] = (a / length[:, None] * z_want[:, None]).float()
    B = B.to(BF16)
    targets = torch.arange(M, device="cuda")
    z = ref.logits(A, B, 1.0)
    lse = torch.logsumexp(z, 1).float()
    t, live = ref.target_matrix(targets, N, 0.0), targets >= 0
    one = torch.ones(M, device="cuda")
    want, _ = ref.dlogits(A, B, t, live, one, lse, 1.0)
    left = -want[torch.arange(M), targets]
    assert (left > 3e-6).all() and (left < 2e-2).all()
    bound = (2 * 512 * 1.1e-9 + ((K + 511) // 512) * 2.0 ** -24) * z.max(1)[0] + 2.0 ** -21 * (lse.double() + 1.0)
    rounding = 2.0 ** -16 if M <= 128 else 2.0 ** -8
    for own in (False, True):
        at = g.matmul_cross_entropy(A, B, targets)[1] if own else lse
        exact = 1.0 - torch.exp(z[torch.arange(M), targets] - at.double())
        _, dB = g.matmul_cross_entropy_grad(one, A, B, targets, at, out_dtype=F32, need_dA=False)
        ok()
        got = -(dB[:M].double() * a).sum(1) / length
        # (other rows' dz at this target, of 1e-8, along directions that are nearly orthogonal)
        cross = ((torch.where(t[:, :M] > 0, 0.0, want[:, :M].abs())) * (a @ a.T).abs()).sum(0) / length
        ref.check(got, exact, bound + (rounding + 2.0 ** -17) * exact.abs() + 2.0 ** -17 * cross + cross, "1 - p")
