"""Losses over a vocabulary at sizes of their own: which kernels a call takes, long
dimensions, calls on several streams, the watchdog.  Logits of small integers,
exact in fp32, as in test_losses."""
import pytest
import torch

import dense_gemm_blackwell_tcgen05_gb300 as g
from tests import loss_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def status():
    return g.gemm_last_status(torch.cuda.current_stream().cuda_stream)


def problem(M, N, K, seed=0):
    r = torch.Generator("cuda").manual_seed(seed + M + 3 * N + 7 * K)
    ints = lambda *s: torch.randint(-2, 3, s, generator=r, device="cuda", dtype=torch.int8).to(BF16)  # noqa: E731
    targets = torch.randint(0, N, (M,), generator=r, device="cuda")
    targets[torch.rand(M, generator=r, device="cuda") < 0.2] = -100
    targets[0], targets[M - 1] = N - 1, 0
    return ints(M, K), ints(N, K), targets, torch.randn(M, generator=r, device="cuda"), 2.0 ** -(K.bit_length() // 2)


def check_rows(A, B, targets, scale, loss, lse, step=1 << 16):
    """Losses and lse, some rows at a time."""
    for lo in range(0, A.shape[0], step):
        a, tg = A[lo:lo + step], targets[lo:lo + step]
        live, t = tg >= 0, ref.target_matrix(tg, B.shape[0], 0.0)
        want, want_lse = ref.forward(a, B, t, torch.zeros(len(a), device="cuda", dtype=torch.float64), live, scale)
        e_loss, e_lse = ref.forward_bounds(a, B, t, scale, want_lse, 0.0, True)
        ref.check(lse[lo:lo + step], want_lse, torch.where(live, e_lse, 0.0), "lse")
        ref.check(loss[lo:lo + step], want, torch.where(live, e_loss, 0.0), "loss")


# M, N, K; CTAs a cluster of the logits' and of the gradients' products
KERNELS = [(20, 3000, 512, 1, 1), (128, 9000, 256, 1, 1), (129, 40000, 1024, 2, 2), (200, 700, 64, 1, 1), (1500, 9000, 512, 2, 2),
           (256, 20000, 2048, 2, 2), (300, 600, 96, 1, 1)]


@pytest.mark.parametrize("M, N, K, forward, backward", KERNELS)
def test_kernels_that_sizes_take(M, N, K, forward, backward):
    A, B, targets, dloss, scale = problem(M, N, K)
    loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
    assert g.gemm_last_schedule()["ctas_per_cluster"] == forward
    check_rows(A, B, targets, scale, loss, lse)
    dA, dB = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale)
    assert g.gemm_last_schedule()["ctas_per_cluster"] == backward
    assert status() == g.GEMM_OK
    t, live = ref.target_matrix(targets, N, 0.0), targets >= 0
    (ra, ta), (rb, tb) = ref.gradients(A, B, t, live, dloss, lse, scale, exact=True)
    # (lse is the kernel's own)
    ref.check(dA, ra, ta, "dA")
    ref.check(dB, rb, tb, "dB")


def test_widths_of_a_tile():
    """Tiles of 32 to 256 columns, whole and ragged, on one CTA and on pairs."""
    for M in (5, 140):
        for N in (31, 32, 33, 64, 95, 96, 97, 127, 128, 159, 160, 161, 4863, 4864, 4865, 9727, 12160, 14593, 17000, 19457):
            A, B, targets, dloss, scale = problem(M, N, 40)
            loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
            check_rows(A, B, targets, scale, loss, lse)
            dA, _ = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale, need_dB=False)
            t, live = ref.target_matrix(targets, N, 0.0), targets >= 0
            (ra, ta), _ = ref.gradients(A, B, t, live, dloss, lse, scale, exact=True)
            ref.check(dA, ra, ta, f"dA at {M}, {N}")
    assert status() == g.GEMM_OK


def test_a_million_rows():
    M, N, K = (1 << 20) + 1, 520, 64
    A, B, targets, dloss, scale = problem(M, N, K)
    loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
    assert status() == g.GEMM_OK
    check_rows(A, B, targets, scale, loss, lse)
    dA, dB = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale, out_dtype=F32)
    assert status() == g.GEMM_OK
    rb, tb = torch.zeros(N, K, device="cuda", dtype=torch.float64), torch.zeros(N, K, device="cuda", dtype=torch.float64)
    step = 1 << 16
    for lo in range(0, M, step):
        s = slice(lo, lo + step)
        t, live = ref.target_matrix(targets[s], N, 0.0), targets[s] >= 0
        (ra, ta), (b, e) = ref.gradients(A[s], B, t, live, dloss[s], lse[s], scale, dA=F32, dB=F32, exact=True)
        ref.check(dA[s], ra, ta, "dA")
        dz, _ = ref.dlogits(A[s], B, t, live, dloss[s], lse[s], scale)
        rb += b
        # the sum's steps are the whole sum's: each cuts off below 2^-19 of what is added up by then
        tb += e + M / 16 * 2.0 ** -19 * (dz.abs().T @ A[s].double().abs())
    ref.check(dB, rb, tb, "dB")


@pytest.mark.parametrize("M", [40, 300])
def test_a_million_tokens(M):
    N, K = (1 << 20) + 3, 64
    A, B, targets, dloss, scale = problem(M, N, K)
    loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
    assert status() == g.GEMM_OK
    for lo in range(0, M, 64):
        s = slice(lo, lo + 64)
        check_rows(A[s], B, targets[s], scale, loss[s], lse[s])
    dA, dB = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale)
    assert status() == g.GEMM_OK
    t, live = ref.target_matrix(targets, N, 0.0), targets >= 0
    (ra, ta), (rb, tb) = ref.gradients(A, B, t, live, dloss, lse, scale, exact=True)
    ref.check(dA, ra, ta, "dA")
    ref.check(dB, rb, tb, "dB")


# M, N, K: pieces of 4096 tokens at least, and of 512 MiB of g at most
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("M, N, K, wide", [(34000, 9000, 72, 4608), (34000, 9000, 74, 4608), (300, 1800000, 24, 600064),
                                           (128, 2200000, 16, 733440), (5, 9000000, 8, 3000064)])
def test_pieces(M, N, K, wide, listed):
    """Gradients by several pieces of the vocabulary, entries on both sides of a border."""
    A, B, targets, dloss, scale = problem(M, N, (K + 7) // 8 * 8)
    A, B = A[:, :K], B[:, :K]
    border = min(M, 60)
    targets[:border] = torch.arange(wide - border // 2, wide - border // 2 + border, device="cuda")
    if listed:
        ids = torch.stack([targets, targets.flip(0), targets], 1).int()
        ids[:, 2] = torch.where(ids[:, 2] < 0, -1, (ids[:, 2] + 1) % N)
        teacher = torch.linspace(-1.0, 1.0, 3 * M, device="cuda").view(M, 3)
        t, entropy, live = ref.teacher_matrix(teacher, ids, N, 1.0 / scale)
        loss, lse = g.matmul_distill(A, B, teacher, ids, temperature=1.0 / scale)
        dA, dB = g.matmul_distill_grad(dloss, A, B, teacher, ids, lse, temperature=1.0 / scale, out_dtype=F32)
    else:
        t, live = ref.target_matrix(targets, N, 0.0), targets >= 0
        loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
        dA, dB = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale, out_dtype=F32)
    assert status() == g.GEMM_OK
    (ra, ta), (rb, tb) = ref.gradients(A, B, t, live, dloss, lse, scale, dA=F32, dB=F32, exact=True)
    # a list's p is off by 2^-20 (1 + |teacher / T|) of itself, and these are below 1
    more = 2.0 ** -19 * torch.where(live, dloss.double().abs() * scale, 0.0)[:, None] * t if listed else torch.zeros_like(t[:, :1])
    ref.check(dA, ra, ta + (more @ B.double().abs() if listed else 0.0), "dA")
    ref.check(dB, rb, tb + (more.T @ A.double().abs() if listed else 0.0), "dB")


@pytest.mark.parametrize("db, accumulate", [(BF16, False), (F32, False), (F32, True)])
@pytest.mark.parametrize("M, N, K", [(4000, 512, 256), (2100, 130, 520), (9000, 600, 72), (2048, 40, 1000), (2500, 1000, 64),
                                     (20000, 300, 136)])
def test_matrices_of_few_tiles(M, N, K, db, accumulate):
    """Many rows, a small matrix: its product is dealt in parts of the rows.  With most rows left
    out it is not."""
    A, B, targets, dloss, scale = problem(M, N, K)
    for some in (targets, torch.where(torch.arange(M, device="cuda") % 50 == 0, targets, -1)):
        t, live = ref.target_matrix(some, N, 0.0), some >= 0
        loss, lse = g.matmul_cross_entropy(A, B, some, scale=scale)
        old = torch.linspace(-1.0, 1.0, N * K, device="cuda").view(N, K).to(db)
        buf = torch.full((N, K + 8), 7.0, dtype=db, device="cuda")
        for need_dA in (True, False):
            dB = buf[:, :K]
            dB.copy_(old)
            dA, got = g.matmul_cross_entropy_grad(dloss, A, B, some, lse, scale=scale, dB=dB, accumulate=accumulate,
                                                  need_dA=need_dA)
            assert got is dB and status() == g.GEMM_OK and (buf[:, K:] == 7.0).all()
            (ra, ta), (rb, tb) = ref.gradients(A, B, t, live, dloss, lse, scale, dB=db, exact=True)
            # up to 152 parts' sums are added up with a rounding each
            steps = 152 * 2.0 ** -24 * (ref.dlogits(A, B, t, live, dloss, lse, scale)[0].abs().T @ A.double().abs())
            if accumulate:
                rb, tb = rb + old.double(), tb + 2.0 ** -23 * (rb.abs() + old.double().abs())
            ref.check(dB, rb, tb + steps, "dB")
            if need_dA:
                ref.check(dA, ra, ta, "dA")
            else:
                assert dA is None


def test_a_long_width():
    M, N, K = 40, 300, 1 << 17
    A, B, targets, dloss, scale = problem(M, N, K)
    loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
    check_rows(A, B, targets, scale, loss, lse)
    dA, dB = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale)
    assert status() == g.GEMM_OK
    t, live = ref.target_matrix(targets, N, 0.0), targets >= 0
    (ra, ta), (rb, tb) = ref.gradients(A, B, t, live, dloss, lse, scale, exact=True)
    ref.check(dA, ra, ta, "dA")
    ref.check(dB, rb, tb, "dB")


def test_two_calls_at_once():
    """On two streams, each with its own workspace and results."""
    a, b = problem(700, 9000, 200, 1), problem(60, 20000, 512, 2)
    want = []
    for A, B, targets, dloss, scale in (a, b):
        loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
        want.append((loss, lse, *g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [[g.cross_entropy_workspace(*A.shape[:1], *B.shape, grad) for grad in (False, True)] for A, B, *_ in (a, b)]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (A, B, targets, dloss, scale) in enumerate((a, b)):
            loss, lse = g.matmul_cross_entropy(A, B, targets, scale=scale, workspace=spaces[i][0], stream=streams[i])
            got[i].append((loss, lse, *g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale, workspace=spaces[i][1],
                                                                   stream=streams[i])))
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for one in many:
            assert all(torch.equal(x, y) for x, y in zip(w, one))
    assert status() == g.GEMM_OK


QUEUED = 20_000_000   # clocks that the current stream is kept busy: about 10 ms


@pytest.mark.parametrize("name", ["cross_entropy", "cross_entropy_grad", "distill", "distill_grad"])
def test_results_made_on_another_stream(name):
    """Their memory is not one that the current stream's queued work still writes."""
    A, B, targets, dloss, scale = problem(300, 2000, 128)
    ids = torch.randint(-1, 2000, (300, 9), device="cuda", dtype=torch.int32)
    teacher = torch.randn(300, 9, device="cuda")
    _, lse = g.matmul_cross_entropy(A, B, targets)
    _, lse_kd = g.matmul_distill(A, B, teacher, ids)
    ws = g.distill_workspace(300, 2000, 128, 9, True), g.distill_workspace(300, 2000, 128, 9)
    call = {
        "cross_entropy": lambda **k: g.matmul_cross_entropy(A, B, targets, workspace=ws[1], **k),
        "cross_entropy_grad": lambda **k: g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, workspace=ws[0], **k),
        "distill": lambda **k: g.matmul_distill(A, B, teacher, ids, workspace=ws[1], **k),
        "distill_grad": lambda **k: g.matmul_distill_grad(dloss, A, B, teacher, ids, lse_kd, workspace=ws[0], **k),
    }[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()              # (calls that share a workspace must not overlap)
    call(stream=side)                     # (first-call set-up)
    torch.cuda.synchronize()
    junk = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(QUEUED)
    for t in junk:
        t.fill_(7)
    del junk, t
    got = call(stream=side)
    torch.cuda.synchronize()
    assert not any(t.isnan().any() for t in want)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_host_memory_is_refused():
    A, B, targets, dloss, scale = problem(40, 300, 64)
    host = torch.zeros(1 << 20, dtype=torch.uint8).pin_memory()
    ws = g.cross_entropy_workspace(40, 300, 64, True)
    loss, lse = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    args = [A.data_ptr(), B.data_ptr(), targets.data_ptr(), loss.data_ptr(), lse.data_ptr()]
    rest = [40, 300, 64, 64, 64, g.INDEX_I64, 1.0, 0.0, 0.0]
    for i in range(5):
        bad = list(args)
        bad[i] = host.data_ptr()
        assert g.gemm_bf16_cross_entropy(*bad, *rest, ws.data_ptr(), ws.nbytes, s) == g.GEMM_ERR_INVALID_ARG
    assert g.gemm_bf16_cross_entropy(*args, *rest, host.data_ptr(), host.nbytes, s) == g.GEMM_ERR_INVALID_ARG
    assert g.gemm_bf16_cross_entropy(*args, *rest, ws.data_ptr(), ws.nbytes, s) == g.GEMM_OK
    assert status() == g.GEMM_OK


@pytest.mark.parametrize("M, N, K", [(40, 3000, 512), (600, 9000, 512)])
@pytest.mark.parametrize("stall", [0, 5])
@pytest.mark.parametrize("grad", [False, True])
def test_a_stage_that_never_fills(M, N, K, stall, grad):
    """The call's waits run out, the status word says so, and the next call is right."""
    A, B, targets, dloss, scale = problem(M, N, K)
    want, lse = g.matmul_cross_entropy(A, B, targets, scale=scale)
    grads = g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale)
    call = (lambda: g.matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale=scale)) if grad else \
        (lambda: g.matmul_cross_entropy(A, B, targets, scale=scale))
    old = g.gemm_set_watchdog_ms(100)
    try:
        assert g.gemm_debug_stall_next_launch(stall) == g.GEMM_OK
        call()
        assert status() == g.GEMM_ERR_TIMEOUT
        assert status() == g.GEMM_OK
        got = call()
        assert status() == g.GEMM_OK
    finally:
        g.gemm_set_watchdog_ms(old)
    assert all(torch.equal(x, y) for x, y in zip(got, grads if grad else (want, lse)))
