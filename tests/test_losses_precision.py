"""Losses over a vocabulary where rounding shows: large logits, sure tokens."""
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
