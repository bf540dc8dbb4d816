"""Losses over a vocabulary (matmul_cross_entropy, matmul_distill and their
gradients) against plain 64-bit forms.

Where A and B hold small integers the logits are exact in fp32, and what is
left is the rounding of exponentials, sums and results (loss_reference)."""
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


def matrix(r, rows, cols, exact, std=1.0, pad=8):
    """bf16 [rows, cols] whose pitch is a multiple of 8 with large values behind each row."""
    buf = torch.full((rows, (cols + 7) // 8 * 8 + pad), 1000.0, dtype=BF16, device="cuda")
    if exact:
        buf[:, :cols] = torch.randint(-2, 3, (rows, cols), generator=r, device="cuda").to(BF16)
    else:
        buf[:, :cols] = (std * torch.randn(rows, cols, generator=r, device="cuda")).to(BF16)
    return buf[:, :cols]


def scale_of(K, exact):
    return 2.0 ** -(K.bit_length() // 2) if exact else 1.0


def problem(M, N, K, exact, seed=0):
    r = gen(1000 * seed + M + 7 * N + 13 * K)
    A = matrix(r, M, K, exact)
    B = matrix(r, N, K, exact, std=2.0 / K ** 0.5)
    return r, A, B


def some_targets(r, M, N, dtype, left_out):
    t = torch.randint(0, N, (M,), generator=r, device="cuda")
    t[0] = N - 1
    if M > 2:
        t[1] = 0
    if left_out:
        t[torch.rand(M, generator=r, device="cuda") < left_out] = -100
    return t.to(dtype)


def some_entries(r, M, N, top, dtype, logits, left_out):
    """ids in any order, some twice, some absent; rows without any."""
    ids = torch.randint(0, N, (M, top), generator=r, device="cuda")
    ids[0, 0] = N - 1
    if top > 2:
        ids[:, 2] = ids[:, 0]
    teacher = (3.0 * torch.randn(M, top, generator=r, device="cuda") + 10.0).to(logits)
    if left_out:
        ids[torch.rand(M, top, generator=r, device="cuda") < left_out] = -1
        teacher[torch.rand(M, top, generator=r, device="cuda") < left_out / 2] = -torch.inf
        ids[torch.rand(M, generator=r, device="cuda") < left_out] = -5
    return teacher, ids.to(dtype)


def marked(rows, cols, dtype, pad=0, shift=0):
    buf = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
    return buf, buf[shift:].view(rows, cols + pad)[:, :cols]


def only_inside(buf, view):
    """Nothing behind the view's rows was written."""
    assert int((~buf.isnan()).sum()) == view.numel()


# M, N, K: every tile choice, tile edges on each side, K tails, one row, one token
SHAPES = [(1, 1, 8), (1, 300, 64), (3, 65, 24), (31, 64, 200), (128, 129, 72), (129, 130, 520), (127, 1000, 1032),
          (256, 513, 64), (257, 1000, 96), (300, 2049, 1100), (300, 2049, 1104), (513, 777, 40), (700, 5003, 264)]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("M, N, K", SHAPES)
def test_cross_entropy(M, N, K, exact):
    r, A, B = problem(M, N, K, exact)
    scale = scale_of(K, exact)
    for smoothing, z_loss, dtype, left_out in ((0.0, 0.0, torch.int64, 0.0), (0.1, 1e-3, torch.int32, 0.3)):
        targets = some_targets(r, M, N, dtype, left_out)
        live = targets >= 0
        loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale, label_smoothing=smoothing, z_loss=z_loss)
        ok()
        assert loss.dtype is F32 and lse.dtype is F32
        t = ref.target_matrix(targets, N, smoothing)
        want, want_lse = ref.forward(A, B, t, torch.zeros(M, device="cuda", dtype=torch.float64), live, scale, z_loss)
        e_loss, e_lse = ref.forward_bounds(A, B, t, scale, want_lse, z_loss, exact)
        ref.check(lse, want_lse, torch.where(live, e_lse, 0.0), "lse")
        ref.check(loss, want, torch.where(live, e_loss, 0.0), "loss")


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("odd", [True, False])
@pytest.mark.parametrize("M, N, K", SHAPES)
def test_cross_entropy_gradient(M, N, K, odd, exact):
    r, A, B = problem(M, N, K, exact, seed=1)
    scale = scale_of(K, exact)
    dloss = torch.randn(M, generator=r, device="cuda")
    for smoothing, z_loss, dtype, left_out, da, db in ((0.0, 0.0, torch.int64, 0.0, BF16, BF16),
                                                       (0.1, 1e-3, torch.int32, 0.3, F32, F32)):
        targets = some_targets(r, M, N, dtype, left_out)
        live = targets >= 0
        t = ref.target_matrix(targets, N, smoothing)
        lse = ref.forward(A, B, t, torch.zeros(M, device="cuda", dtype=torch.float64), live, scale)[1].float()
        # rows that start on an element, and on 32 bytes
        (_, dA), (_, dB) = bufs = (marked(M, K, da, 3, 1), marked(N, K, db, 5, 1)) if odd else \
            (marked(M, K, da, -K % 16), marked(N, K, db, -K % 16 + 16))
        got = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale, label_smoothing=smoothing, z_loss=z_loss,
                                          dA=dA, dB=dB)
        ok()
        assert got[0] is dA and got[1] is dB
        (ra, ta), (rb, tb) = ref.gradients(A, B, t, live, dloss, lse, scale, z_loss, da, db, exact)
        ref.check(dA, ra, ta, "dA")
        ref.check(dB, rb, tb, "dB")
        for buf, view in bufs:
            only_inside(buf, view)


TOPS = [(1, 1, 8, 1), (2, 40, 64, 3), (33, 100, 24, 40), (128, 129, 72, 64), (257, 1000, 96, 100), (300, 2049, 264, 17),
        (5, 1030, 40, 300), (3, 4000, 16, 1024), (600, 5003, 136, 8)]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("M, N, K, top", TOPS)
def test_distill(M, N, K, top, exact):
    r, A, B = problem(M, N, K, exact, seed=2)
    for temperature, logits, dtype, left_out in ((1.0, F32, torch.int32, 0.0), (2.0 if exact else 0.7, BF16, torch.int64, 0.3)):
        f = temperature / scale_of(K, exact)
        teacher, ids = some_entries(r, M, N, top, dtype, logits, left_out)
        loss, lse = g.matmul_distill(A, B, teacher, ids, temperature=f)
        ok()
        t, entropy, live = ref.teacher_matrix(teacher, ids, N, f)
        want, want_lse = ref.forward(A, B, t, entropy, live, 1.0 / f)
        e_loss, e_lse = ref.forward_bounds(A, B, t, 1.0 / f, want_lse, 0.0, exact)
        # 1 / temperature is rounded; p is off by 2^-21 (1 + |teacher / T|) of itself, times its terms
        big = ref.logits(A, B, 1.0 / f).abs().max(1)[0] + want_lse.abs()
        size = teacher.double().masked_fill(teacher == -torch.inf, 0.0).abs().max(1)[0] / f + 1.0
        e_loss = e_loss + 2.0 ** -20 * size * (big + entropy.abs() + size)
        ref.check(lse, want_lse, torch.where(live, e_lse, 0.0), "lse")
        ref.check(loss, want, torch.where(live, e_loss, 0.0), "loss")


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("M, N, K, top", TOPS)
def test_distill_gradient(M, N, K, top, exact):
    r, A, B = problem(M, N, K, exact, seed=3)
    dloss = torch.randn(M, generator=r, device="cuda")
    for temperature, logits, dtype, left_out, da, db in ((1.0, F32, torch.int32, 0.0, BF16, F32),
                                                         (2.0 if exact else 0.7, BF16, torch.int64, 0.3, F32, BF16)):
        f = temperature / scale_of(K, exact)
        teacher, ids = some_entries(r, M, N, top, dtype, logits, left_out)
        t, entropy, live = ref.teacher_matrix(teacher, ids, N, f)
        lse = ref.forward(A, B, t, entropy, live, 1.0 / f)[1].float()
        (_, dA), (_, dB) = bufs = marked(M, K, da, 1), marked(N, K, db, 2)
        g.matmul_distill_grad(dloss, A, B, teacher, ids, lse, temperature=f, dA=dA, dB=dB)
        ok()
        (ra, ta), (rb, tb) = ref.gradients(A, B, t, live, dloss, lse, 1.0 / f, 0.0, da, db, exact)
        # p is off by 2^-21 (1 + |teacher / T|) of itself
        size = 2.0 ** -20 * (teacher.double().masked_fill(teacher == -torch.inf, 0.0).abs().max(1)[0] / f + 1.0)
        off = torch.where(live, dloss.double().abs() / f * size, 0.0)[:, None] * t
        ref.check(dA, ra, ta + off @ B.double().abs(), "dA")
        ref.check(dB, rb, tb + off.T @ torch.where(live[:, None], A.double().abs(), 0.0), "dB")
        for buf, view in bufs:
            only_inside(buf, view)


@pytest.mark.parametrize("N", [8, 64, 200, 264, 520])
def test_every_element_of_the_logits_gradient(N):
    """With B the identity, dA is the logits' gradient itself, element by element."""
    r = gen(N)
    M, top = 2 * N, 7
    B = torch.eye(N, dtype=BF16, device="cuda")
    A = torch.randint(-6, 7, (M, N), generator=r, device="cuda").to(BF16)
    targets = torch.arange(M, device="cuda") % N
    dloss = torch.randn(M, generator=r, device="cuda")
    for smoothing, z_loss in ((0.0, 0.0), (0.2, 1e-2)):
        t = ref.target_matrix(targets, N, smoothing)
        live = targets >= 0
        zero = torch.zeros(M, device="cuda", dtype=torch.float64)
        lse = ref.forward(A, B, t, zero, live, 1.0)[1].float()
        dA, none = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, label_smoothing=smoothing, z_loss=z_loss, need_dB=False)
        assert none is None
        dz, size = ref.dlogits(A, B, t, live, dloss, lse, 1.0, z_loss)
        # one rounding: a product with the identity is exact, and so is the second rounding of a bf16 value
        ref.check(dA, dz, 2.0 ** -8 * dz.abs() + size * 2.0 ** -16, "dz")
    teacher, ids = some_entries(r, M, N, top, torch.int32, F32, 0.2)
    t, entropy, live = ref.teacher_matrix(teacher, ids, N, 1.0)
    lse = ref.forward(A, B, t, entropy, live, 1.0)[1].float()
    dA, _ = g.matmul_distill_grad(dloss, A, B, teacher, ids, lse)
    dz, size = ref.dlogits(A, B, t, live, dloss, lse, 1.0)
    ref.check(dA, dz, 2.0 ** -8 * dz.abs() + size * 2.0 ** -15, "dz of a list")


@pytest.mark.parametrize("M", [1, 63, 64, 65, 127, 128])
def test_few_rows_gradients_keep_two_halves(M):
    """Up to 128 rows dz is a sum of two bf16 terms, each rounded by 2^-8 of itself: 2^-16 in all.
    B and A select single elements of it, in sums that are exact but for their last rounding."""
    N, K = 257, 264
    r = gen(M)
    B = torch.zeros(N, K, dtype=BF16, device="cuda")
    B[:, :N] = torch.eye(N, dtype=BF16, device="cuda")
    A = torch.zeros(M, K, dtype=BF16, device="cuda")
    A[:, :N] = torch.randint(-6, 7, (M, N), generator=r, device="cuda").to(BF16)
    targets = some_targets(r, M, N, torch.int64, 0.2)
    live = targets >= 0
    dloss = torch.randn(M, generator=r, device="cuda")
    t = ref.target_matrix(targets, N, 0.1)
    lse = ref.forward(A, B, t, torch.zeros(M, device="cuda", dtype=torch.float64), live, 1.0)[1].float()
    dA, dB = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, label_smoothing=0.1, out_dtype=F32)
    dz, size = ref.dlogits(A, B, t, live, dloss, lse, 1.0)
    off = 2.0 ** -16 * dz.abs() + size * 2.0 ** -16
    ref.check(dA[:, :N], dz, off, "dz")
    assert not dA[:, N:].any()
    a = A.double()
    # (a step of the tensor core cuts 17 addends off below 2^-23 of the largest: 2^-18.9 of all)
    want, steps = dz.T @ a, (2 * M + 142) // 16
    ref.check(dB, want, off.T @ a.abs() + steps * 2.0 ** -18.9 * (dz.abs().T @ a.abs()), "dB")


def test_a_sure_row_keeps_its_small_gradient():
    """exp(z - lse) near 1 at the target: the difference is taken before anything is rounded to bf16."""
    N = 64
    B = torch.eye(N, dtype=BF16, device="cuda")
    A = torch.zeros(4, N, dtype=BF16, device="cuda")
    for i, sure in enumerate((4.0, 8.0, 10.0, 12.0)):
        A[i, 5] = sure
    targets = torch.full((4,), 5, device="cuda")
    loss, lse = g.matmul_cross_entropy(A, B, targets)
    dA, _ = g.matmul_cross_entropy_grad(torch.ones(4, device="cuda"), A, B, targets, lse, out_dtype=F32, need_dB=False)
    p = torch.softmax(A.double(), 1)
    want = p.clone()
    want[:, 5] = -(1.0 - p[:, 5])
    # 2^-8 of the value for bf16, and the absolute error of exp(z - lse) <= 1 and of lse (below 16)
    assert ((dA.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * p).all()
    assert (want[:, 5].abs() > 100 * 2.0 ** -19).sum() >= 3


@pytest.mark.parametrize("K", [72, 80, 528])
@pytest.mark.parametrize("top", [0, 9])
@pytest.mark.parametrize("M", [100, 200, 700])
def test_pieces_of_the_vocabulary(M, top, K):
    """A vocabulary of several pieces, entries on both sides of each border."""
    N = 10007
    r, A, B = problem(M, N, K, True, seed=4)
    scale = scale_of(K, True)
    dloss = torch.randn(M, generator=r, device="cuda")
    borders = torch.tensor([0, 3583, 3584, 3585, 7167, 7168, N - 1], device="cuda")
    if top == 0:
        targets = some_targets(r, M, N, torch.int64, 0.2)
        targets[:7] = borders
        live, entropy = targets >= 0, torch.zeros(M, device="cuda", dtype=torch.float64)
        t = ref.target_matrix(targets, N, 0.0)
        loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
        dA, dB = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale)
    else:
        teacher, ids = some_entries(r, M, N, top, torch.int32, F32, 0.2)
        ids[:50, 1:8] = borders.int()
        t, entropy, live = ref.teacher_matrix(teacher, ids, N, 1.0 / scale)
        loss, lse = g.matmul_distill(A, B, teacher, ids, temperature=1.0 / scale)
        dA, dB = g.matmul_distill_grad(dloss, A, B, teacher, ids, lse, temperature=1.0 / scale)
    ok()
    want, want_lse = ref.forward(A, B, t, entropy, live, scale)
    e_loss, e_lse = ref.forward_bounds(A, B, t, scale, want_lse, 0.0, True)
    ref.check(lse, want_lse, torch.where(live, e_lse, 0.0), "lse")
    ref.check(loss, want, torch.where(live, e_loss + 2.0 ** -15, 0.0), "loss")   # 2^-15: a list's p, as in test_distill
    (ra, ta), (rb, tb) = ref.gradients(A, B, t, live, dloss, lse, scale, exact=True)
    more = 2.0 ** -14 * torch.where(live, dloss.double().abs() * scale, 0.0)[:, None] * t if top else torch.zeros_like(t)
    ref.check(dA, ra, ta + more @ B.double().abs(), "dA")
    ref.check(dB, rb, tb + more.T @ A.double().abs(), "dB")


@pytest.mark.parametrize("M, N, K", [(100, 300, 64), (600, 1000, 136)])
def test_rows_left_out_do_not_count_whatever_they_hold(M, N, K):
    r, A, B = problem(M, N, K, True, seed=5)
    scale = scale_of(K, True)
    targets = some_targets(r, M, N, torch.int64, 0.4)
    out = targets < 0
    dloss = torch.randn(M, generator=r, device="cuda")
    loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
    dA, dB = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale)
    for value in (float("nan"), float("inf"), -float("inf")):
        A2, d2, l2 = A.clone(), dloss.clone(), lse.clone()
        A2[out], d2[out], l2[out] = value, value, value
        loss2, lse2 = g.matmul_cross_entropy(A2, B, targets, scale=scale)
        dA2, dB2 = g.matmul_cross_entropy_grad(d2, A2, B, targets, l2, scale=scale)
        ok()
        for x, y in ((loss, loss2), (lse, lse2), (dA, dA2), (dB, dB2)):
            assert torch.equal(x, y)
    assert (dA[out] == 0).all() and (loss[out] == 0).all() and (lse[out] == 0).all()
    # none is left
    targets = torch.full_like(targets, -1)
    loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
    dA, dB = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale)
    ok()
    assert not (loss.any() or lse.any() or dA.any() or dB.any())
    old = torch.randn(N, K, generator=r, device="cuda")
    dB = old.clone()
    g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale, dB=dB, accumulate=True)
    assert torch.equal(dB, old)
    teacher, ids = some_entries(r, M, N, 5, torch.int32, F32, 0.0)
    loss, lse = g.matmul_distill(A, B, teacher, torch.full_like(ids, -1))
    assert not (loss.any() or lse.any())
    loss, lse = g.matmul_distill(A, B, torch.full_like(teacher, -torch.inf), ids)
    assert not (loss.any() or lse.any())


@pytest.mark.parametrize("M", [40, 400])
def test_wrong_tokens_and_values_that_are_not_finite(M):
    N, K = 500, 64
    r, A, B = problem(M, N, K, True, seed=6)
    targets = some_targets(r, M, N, torch.int64, 0.0)
    clean, _ = g.matmul_cross_entropy(A, B, targets)
    targets[3] = N
    targets[5] = 2 ** 40
    A[7, 2] = float("nan")
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[[3, 5, 7]] = True
    loss, lse = g.matmul_cross_entropy(A, B, targets)
    assert loss[bad].isnan().all() and torch.equal(loss[~bad], clean[~bad])
    dA, dB = g.matmul_cross_entropy_grad(torch.ones(M, device="cuda"), A, B, targets, lse)
    ok()
    assert dA[bad].isnan().all() and not dA[~bad].isnan().any()
    teacher, ids = some_entries(r, M, N, 6, torch.int64, F32, 0.0)
    clean, _ = g.matmul_distill(A, B, teacher, ids)
    ids[3, 1] = N
    ids[5, 4] = 2 ** 31
    ids[9, 0] = 2 ** 33
    teacher[11, 0] = float("nan")
    teacher[13, 5] = float("inf")
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[[3, 5, 7, 9, 11, 13]] = True
    loss, lse = g.matmul_distill(A, B, teacher, ids)
    assert loss[bad].isnan().all() and torch.equal(loss[~bad], clean[~bad])
    dA, dB = g.matmul_distill_grad(torch.ones(M, device="cuda"), A, B, teacher, ids, lse)
    ok()
    assert dA[bad].isnan().all() and not dA[~bad].isnan().any()


def test_far_logits():
    """Logits whose exponentials leave fp32, and one that leaves all others behind."""
    N, K = 300, 64
    A = torch.zeros(4, K, dtype=BF16, device="cuda")
    B = torch.zeros(N, K, dtype=BF16, device="cuda")
    B[:, 0] = torch.arange(N, device="cuda").to(BF16)
    B[:, 1] = 1.0
    A[0, 1], A[1, 1], A[2, 0], A[3, 0] = 1e4, -1e4, 1.0, -40.0
    targets = torch.tensor([7, 7, 298, 0], device="cuda")
    loss, lse = g.matmul_cross_entropy(A, B, targets)
    ok()
    t = ref.target_matrix(targets, N, 0.0)
    live = targets >= 0
    want, want_lse = ref.forward(A, B, t, torch.zeros(4, device="cuda", dtype=torch.float64), live, 1.0)
    e_loss, e_lse = ref.forward_bounds(A, B, t, 1.0, want_lse, 0.0, True)
    ref.check(lse, want_lse, e_lse, "lse")
    ref.check(loss, want, e_loss, "loss")


@pytest.mark.parametrize("db", [BF16, F32])
@pytest.mark.parametrize("M, N, K", [(60, 200, 64), (500, 1000, 200), (300, 9001, 96), (300, 9001, 100), (130, 1000, 1040)])
def test_accumulate(M, N, K, db):
    r, A, B = problem(M, N, K, True, seed=7)
    scale = scale_of(K, True)
    targets = some_targets(r, M, N, torch.int64, 0.1)
    dloss = torch.randn(M, generator=r, device="cuda")
    _, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
    old = torch.randn(N, K, generator=r, device="cuda").to(db)
    dB = old.clone()
    g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale, dB=dB, accumulate=True, need_dA=False)
    ok()
    t = ref.target_matrix(targets, N, 0.0)
    _, (rb, tb) = ref.gradients(A, B, t, targets >= 0, dloss, lse, scale, dB=db, exact=True)
    ref.check(dB, rb + old.double(), tb + ref.U[db] * (rb + old.double()).abs() + 2.0 ** -23 * old.double().abs(), "dB")


def test_one_value_for_all_rows_and_strides():
    """An expanded dloss, a strided one, and outputs given by the caller."""
    M, N, K = 300, 1000, 64
    r, A, B = problem(M, N, K, False, seed=8)
    targets = some_targets(r, M, N, torch.int64, 0.1)
    out = torch.full((M,), -1.0, device="cuda"), torch.full((M,), -1.0, device="cuda")
    loss, lse = g.matmul_cross_entropy(A, B, targets, out=out)
    assert loss is out[0] and lse is out[1]
    for d in (torch.tensor(0.25, device="cuda").expand(M), torch.rand(3 * M, generator=r, device="cuda")[::3]):
        got = g.matmul_cross_entropy_grad(d, A, B, targets, lse)
        want = g.matmul_cross_entropy_grad(d.contiguous(), A, B, targets, lse)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    ok()


@pytest.mark.parametrize("M, N, K, top", [(48, 3000, 128, 12), (700, 9001, 200, 30)])
def test_the_same_bits_captured_on_streams_and_with_one_workspace(M, N, K, top):
    """Two graphs that share a workspace, replayed with new inputs, and calls on another stream."""
    r, A, B = problem(M, N, K, False, seed=9)
    targets = some_targets(r, M, N, torch.int64, 0.2)
    teacher, ids = some_entries(r, M, N, top, torch.int32, F32, 0.2)
    dloss = torch.rand(M, generator=r, device="cuda")

    def ce(ws=None, stream=None):
        w = [None, None] if ws is None else ws
        loss, lse = g.matmul_cross_entropy(A, B, targets, workspace=w[0], stream=stream)
        return (loss, lse, *g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, workspace=w[1], stream=stream))

    def kd(ws=None, stream=None):
        w = [None, None] if ws is None else ws
        loss, lse = g.matmul_distill(A, B, teacher, ids, workspace=w[0], stream=stream)
        return (loss, lse, *g.matmul_distill_grad(dloss, A, B, teacher, ids, lse, workspace=w[1], stream=stream))

    first = [t.clone() for t in (*ce(), *kd())]
    again = (*ce(), *kd())
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    shared = [g.distill_workspace(M, N, K, top, grad) for grad in (False, True)]
    assert all(a.numel() >= b.numel() for a, b in zip(shared, [g.cross_entropy_workspace(M, N, K, x) for x in (False, True)]))
    graphs, outs = [], []
    for call in (ce, kd):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(shared))
        graphs.append(graph)
    for ws in shared:
        ws.fill_(0xFF)                      # uninitialised, for all the calls know
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    ok()
    assert all(torch.equal(x, y) for x, y in zip(first, (*outs[0], *outs[1])))
    # other inputs in the same places
    old = A.clone()
    A.copy_(A.flip(0))
    targets.copy_(targets.flip(0))
    ids.copy_(ids.flip(0))
    teacher.copy_(teacher.flip(0))
    want = [t.clone() for t in (*ce(), *kd())]
    for graph in graphs[::-1]:
        graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(want, (*outs[0], *outs[1])))
    A.copy_(old)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    own = [g.distill_workspace(M, N, K, top, grad) for grad in (False, True)]
    got = kd(own, side)
    torch.cuda.current_stream().wait_stream(side)
    here = kd()
    assert all(torch.equal(x, y) for x, y in zip(got, here))
    with pytest.raises(ValueError, match="workspace"):
        kd(None, side)


def test_nothing_to_do():
    B = torch.ones(40, 64, dtype=BF16, device="cuda")
    A = torch.ones(0, 64, dtype=BF16, device="cuda")
    targets = torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse = g.matmul_cross_entropy(A, B, targets)
    assert loss.shape == lse.shape == (0,)
    dA, dB = g.matmul_cross_entropy_grad(loss, A, B, targets, lse)
    assert dA.shape == (0, 64) and not dB.any()
    dB = torch.ones(40, 64, device="cuda")
    g.matmul_cross_entropy_grad(loss, A, B, targets, lse, dB=dB, accumulate=True)
    assert (dB == 1).all()
    # no width: logits of 0
    for M in (3, 300):
        A, B = torch.ones(M, 0, dtype=BF16, device="cuda"), torch.ones(40, 0, dtype=BF16, device="cuda")
        loss, lse = g.matmul_cross_entropy(A, B, torch.zeros(M, dtype=torch.int64, device="cuda"), label_smoothing=0.3)
        want = torch.log(torch.tensor(40.0, dtype=torch.float64))
        assert ((loss.double().cpu() - want).abs() < 2.0 ** -19).all() and ((lse.double().cpu() - want).abs() < 2.0 ** -19).all()
        dA, dB = g.matmul_cross_entropy_grad(loss, A, B, torch.zeros(M, dtype=torch.int64, device="cuda"), lse)
        assert dA.shape == (M, 0) and dB.shape == (40, 0)
    ok()


def test_workspaces_are_not_overrun():
    M, N, K, top = 300, 5000, 96, 20
    r, A, B = problem(M, N, K, False, seed=10)
    teacher, ids = some_entries(r, M, N, top, torch.int32, F32, 0.1)
    for grad in (False, True):
        n = g.gemm_bf16_distill_workspace_bytes(M, N, K, top, int(grad))
        buf = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        ws = buf[256:256 + n]
        if not grad:
            loss, lse = g.matmul_distill(A, B, teacher, ids, workspace=ws)
        else:
            g.matmul_distill_grad(torch.ones(M, device="cuda"), A, B, teacher, ids, lse, workspace=ws)
        ok()
        assert (buf[:256] == 0x5A).all() and (buf[256 + n:] == 0x5A).all()
        with pytest.raises(g.GemmError):
            if not grad:
                g.matmul_distill(A, B, teacher, ids, workspace=ws[:-1])
            else:
                g.matmul_distill_grad(torch.ones(M, device="cuda"), A, B, teacher, ids, lse, workspace=ws[:-1])


def test_a_step_as_it_is_used():
    """Losses, their mean's gradient and both weights' gradients through a layer before the loss."""
    M, N, K, W = 513, 2000, 128, 72
    r = gen(11)
    X = torch.randn(M, W, generator=r, device="cuda").to(BF16)
    W1 = (torch.randn(K, W, generator=r, device="cuda") / W ** 0.5).to(BF16)
    B = (2.0 * torch.randn(N, K, generator=r, device="cuda") / K ** 0.5).to(BF16)
    targets = some_targets(r, M, N, torch.int64, 0.25)
    H = g.matmul_bf16(X, W1)
    loss, lse = g.matmul_cross_entropy(H, B, targets)
    count = (targets >= 0).sum()
    dH, dB = g.matmul_cross_entropy_grad((1.0 / count).float().expand(M), H, B, targets, lse)
    o = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    dW1 = g.matmul_grouped_wgrad(dH, X, o, out_dtype=F32)[0]
    ok()
    h, b = (x.double().requires_grad_() for x in (H, B))
    each = torch.nn.functional.cross_entropy(h @ b.T, targets, reduction="none", ignore_index=-100)
    (each.sum() / count).backward()
    t, live = ref.target_matrix(targets, N, 0.0), targets >= 0
    want_lse = torch.where(live, torch.logsumexp(h @ b.T, 1), 0.0).detach()
    e_loss, e_lse = ref.forward_bounds(H, B, t, 1.0, want_lse)
    ref.check(loss, each.detach(), torch.where(live, e_loss, 0.0), "loss")
    # (lse, from which the gradients go on, is off by e_lse)
    (ra, ta), (rb, tb) = ref.gradients(H, B, t, live, (1.0 / count).float().expand(M), lse, 1.0)
    off = torch.where(live, e_lse / count, 0.0)[:, None] * torch.softmax(h @ b.T, 1).detach()
    ref.check(dH, h.grad, ta + off @ b.abs().detach(), "dH")
    ref.check(dB, b.grad, tb + off.T @ h.abs().detach(), "dB")
    want, S = dH.double().T @ X.double(), dH.double().abs().T @ X.double().abs()
    ref.check(dW1, want, (32 + 2) * 2.0 ** -19 * S + 2.0 ** -24 * want.abs(), "dW1")


def test_refusals():
    M, N, K, top = 40, 300, 64, 6
    r, A, B = problem(M, N, K, True, seed=12)
    t, f = some_targets(r, M, N, torch.int64, 0.0), torch.ones(M, device="cuda")
    teacher, ids = some_entries(r, M, N, top, torch.int32, F32, 0.0)
    bad = [
        (ValueError, "disagree", dict(B=B[:, :56])), (TypeError, "bfloat16", dict(A=A.half())), (TypeError, "bfloat16", dict(B=B.float())),
        (ValueError, "CUDA", dict(B=B.cpu())), (ValueError, "2-D", dict(A=A.T)), (g.GemmError, "alignment", dict(A=A[:, 1:], B=B[:, 1:])),
    ]
    for error, match, change in bad:
        x = {"A": A, "B": B, **change}
        for call in (lambda: g.matmul_cross_entropy(x["A"], x["B"], t), lambda: g.matmul_cross_entropy_grad(f, x["A"], x["B"], t, f),
                     lambda: g.matmul_distill(x["A"], x["B"], teacher, ids),
                     lambda: g.matmul_distill_grad(f, x["A"], x["B"], teacher, ids, f)):
            with pytest.raises(error, match=match):
                call()
    two = torch.zeros(2 * M, dtype=torch.int64, device="cuda")[::2]
    for error, match, call in (
            (ValueError, "targets", lambda: g.matmul_cross_entropy(A, B, t[1:])),
            (ValueError, "contiguous", lambda: g.matmul_cross_entropy(A, B, two)),
            (ValueError, "CUDA", lambda: g.matmul_cross_entropy(A, B, t.cpu())),
            (ValueError, "out", lambda: g.matmul_cross_entropy(A, B, t, out=(f[1:], f))),
            (TypeError, "out", lambda: g.matmul_cross_entropy(A, B, t, out=(f, f.double()))),
            (TypeError, "dloss", lambda: g.matmul_cross_entropy_grad(f.half(), A, B, t, f)),
            (ValueError, "lse", lambda: g.matmul_cross_entropy_grad(f, A, B, t, f[:5])),
            (TypeError, "bfloat16 or float32", lambda: g.matmul_cross_entropy_grad(f, A, B, t, f, out_dtype=torch.float16)),
            (ValueError, "dA", lambda: g.matmul_cross_entropy_grad(f, A, B, t, f, dA=torch.empty(K, M, dtype=BF16, device="cuda").T)),
            (ValueError, "shape", lambda: g.matmul_distill(A, B, teacher, ids[:, 1:])),
            (ValueError, "shape", lambda: g.matmul_distill(A, B, teacher[1:], ids[1:])),
            (ValueError, "2-D", lambda: g.matmul_distill(A, B, teacher[:, 0], ids)),
            (TypeError, "bfloat16 or float32", lambda: g.matmul_distill(A, B, teacher.half(), ids)),
            (g.GemmError, "invalid", lambda: g.matmul_distill(A, B, teacher[:, :0], ids[:, :0])),
            (g.GemmError, "invalid", lambda: g.matmul_distill(A, B, teacher, ids, temperature=0.0)),
            (g.GemmError, "invalid", lambda: g.matmul_cross_entropy(A, B, t, scale=-1.0)),
            (g.GemmError, "invalid", lambda: g.matmul_cross_entropy(A, B, t, label_smoothing=1.5)),
            (g.GemmError, "invalid", lambda: g.matmul_cross_entropy(A, B[:0], t))):
        with pytest.raises(error, match=match):
            call()
    ok()
