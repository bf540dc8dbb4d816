"""Gradients of the losses over several pieces of the vocabulary and over very many rows, by how far
they are from the 64-bit form as a whole: a lost piece, target or row would be most of it.

What a norm may be off, relative to its own: dz's and a bf16 output's roundings, 2^-8 of each element
at most and of either sign, and 1.1e-9 a term that the tensor core cuts off (a million rows: 1.1e-3;
parts of nine million tokens: 3e-4).  Below 2^-7 together."""
import functools

import pytest
import torch

import dense_gemm_blackwell_tcgen05_gb300 as g

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
OFF = 2.0 ** -7


def ok():
    assert g.gemm_last_status(torch.cuda.current_stream().cuda_stream) == g.GEMM_OK


def near(got, want, what):
    assert got.isfinite().all(), what
    err, size = (got.double() - want).norm().item(), want.norm().item()
    assert size > 0.0 and err <= OFF * size, f"{what}: {err / size:.2e} of the norm off"


# rows, tokens, width, a piece's tokens
SIZES = [(34000, 9000, 72, 4608), (34000, 9000, 74, 4608), (300, 1800000, 24, 600064), (128, 2200000, 16, 733440),
         (5, 9000000, 8, 3000064)]


@functools.lru_cache(maxsize=1)
def problem(M, N, K, wide):
    r = torch.Generator("cuda").manual_seed(M + N + K)
    ints = lambda *s: torch.randint(-2, 3, s, generator=r, device="cuda", dtype=torch.int8).to(BF16)  # noqa: E731
    A, B = ints(M, (K + 7) // 8 * 8)[:, :K], ints(N, (K + 7) // 8 * 8)[:, :K]
    targets = torch.randint(0, N, (M,), generator=r, device="cuda")
    border = min(M, 60)                    # targets on both sides of a border
    assert border // 2 <= wide <= N - border
    targets[:border] = torch.arange(wide - border // 2, wide - border // 2 + border, device="cuda")
    targets[border:][torch.rand(M - border, generator=r, device="cuda") < 0.2] = -100
    ids = torch.stack([targets, targets.flip(0), torch.where(targets < 0, targets, (targets + 1) % N)], 1).int()
    teacher = torch.randn(M, 3, generator=r, device="cuda")
    return A, B, targets, ids, teacher, 0.5 + torch.rand(M, generator=r, device="cuda"), 2.0 ** -(K.bit_length() // 2)


def learnt(which, targets, ids, teacher, f, N, smoothing):
    """(rows that count, what they learn [M, N] in fp64, as its terms' places and values)."""
    if which == "ce":
        live = targets >= 0
        return live, targets.clamp(min=0)[:, None], torch.where(live, 1.0 - smoothing, 0.0).double()[:, None]
    live = (ids >= 0).any(1)
    x = (teacher.double() * f).masked_fill(ids < 0, -torch.inf)
    return live, ids.long().clamp(min=0), torch.where(ids >= 0, torch.softmax(torch.where(live[:, None], x, 0.0), 1), 0.0)


@functools.lru_cache(maxsize=1)
def reference(size, which, smoothing, z_loss):
    """(lse, dA, dB) in 64 bits, a share of the rows at a time."""
    M, N, K, _ = size
    A, B, targets, ids, teacher, d, f = problem(*size)
    live, places, values = learnt(which, targets, ids, teacher, f, N, smoothing)
    b = B.double()
    lse, dA, dB = torch.zeros(M, device="cuda"), torch.zeros(M, K, device="cuda", dtype=torch.float64), torch.zeros_like(b)
    for s in torch.arange(M, device="cuda").split(max(1, (1 << 27) // N)):
        z = f * (A[s].double() @ b.T)
        lse[s] = torch.where(live[s], torch.logsumexp(z, 1), 0.0).float()
        at = lse[s].double()[:, None]
        dz = z.sub_(at).exp_().mul_(1.0 + 2.0 * z_loss * at).sub_(smoothing / N)
        dz.scatter_add_(1, places[s], -values[s])
        dz *= torch.where(live[s], d[s] * f, 0.0).double()[:, None]
        dA[s], dB = dz @ b, dB + dz.T @ A[s].double()
    return lse, dA, dB


# loss, label smoothing, penalty, dA and dB (None: not wanted), whether dB is added to
FORMS = [("ce", 0.1, 1e-2, BF16, BF16, False), ("ce", 0.1, 1e-2, BF16, BF16, True), ("ce", 0.1, 1e-2, None, F32, True),
         ("ce", 0.1, 1e-2, None, BF16, False), ("ce", 0.1, 1e-2, F32, None, False), ("ce", 0.1, 1e-2, None, BF16, True),
         ("kd", 0.0, 0.0, F32, F32, False), ("kd", 0.0, 0.0, BF16, F32, True), ("kd", 0.0, 0.0, F32, BF16, True)]


@pytest.mark.parametrize("which, smoothing, z_loss, da, db, accumulate", FORMS)
@pytest.mark.parametrize("size", SIZES)
def test_several_pieces(size, which, smoothing, z_loss, da, db, accumulate):
    M, N, K, wide = size
    A, B, targets, ids, teacher, d, f = problem(*size)
    lse, ra, rb = reference(size, which, smoothing, z_loss)
    dA = None if da is None else torch.full((M, K + 3), float("nan"), dtype=da, device="cuda")[:, :K]
    old = dB = None
    if db is not None:
        # of dB's own size, so that what is added shows
        old = (torch.randn(N, 1, device="cuda") * rb.norm() / (N * K) ** 0.5).float() if accumulate else None
        dB = torch.empty(N, K + 5, dtype=db, device="cuda")[:, :K]
        dB.copy_(old) if accumulate else dB.fill_(float("nan"))
        old = dB.double() if accumulate else None
    more = dict(dA=dA, dB=dB, need_dA=da is not None, need_dB=db is not None, accumulate=accumulate)
    if which == "ce":
        got = g.matmul_cross_entropy_grad(d, A, B, targets, lse, scale=f, label_smoothing=smoothing, z_loss=z_loss, **more)
    else:
        got = g.matmul_distill_grad(d, A, B, teacher, ids, lse, temperature=1.0 / f, **more)
    ok()
    assert got[0] is dA and got[1] is dB
    live = targets >= 0 if which == "ce" else (ids >= 0).any(1)
    pieces = [slice(lo, min(N, lo + wide)) for lo in range(0, N, wide)]
    assert len(pieces) > 1
    if da is not None:
        near(dA, ra, "dA")
        assert not dA[~live].any()
        near(dA[:min(M, 60)], ra[:min(M, 60)], "dA of targets at a border")
    if db is not None:
        want = rb + old if accumulate else rb
        near(dB, want, "dB")
        learnt_rows = torch.zeros(N, dtype=torch.bool, device="cuda")
        learnt_rows[(targets[live] if which == "ce" else ids[live].long()).flatten().clamp(min=0)] = True
        for p in pieces:
            if learnt_rows[p].any():       # (five rows' targets all lie about one border)
                near(dB[p][learnt_rows[p]], want[p][learnt_rows[p]], f"dB of a piece's targets from {p.start}")
            near(dB[p][~learnt_rows[p]], want[p][~learnt_rows[p]], f"dB of a piece's other tokens from {p.start}")


@pytest.mark.parametrize("db, accumulate", [(F32, False), (F32, True), (BF16, False), (BF16, True)])
def test_a_million_rows_as_a_whole(db, accumulate):
    size = ((1 << 20) + 1, 520, 64, 260)
    M, N, K, _ = size
    A, B, targets, ids, teacher, d, f = problem(*size)
    lse, ra, rb = reference(size, "ce", 0.1, 1e-2)
    dB = (torch.randn(N, K, device="cuda") * rb.norm() / (N * K) ** 0.5).to(db) if accumulate else torch.empty(N, K, dtype=db, device="cuda")
    want = rb + dB.double() if accumulate else rb
    dA, _ = g.matmul_cross_entropy_grad(d, A, B, targets, lse, scale=f, label_smoothing=0.1, z_loss=1e-2, dB=dB,
                                        accumulate=accumulate, out_dtype=F32)
    ok()
    near(dA, ra, "dA")
    near(dB, want, "dB")
    for rows in dB.sub(want).norm(dim=1).split(1):   # no token's row is lost either
        assert rows.item() <= 2 * OFF * want.norm() / N ** 0.5
