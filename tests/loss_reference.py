"""Plain 64-bit forms of the losses over a vocabulary and their gradients, and
how far a GPU result may be from them.

Steps of the tensor core: 16 terms a step, 17 addends each cut off below 2^-23 of
the largest, under 2^-19 of S = sum |a b| a step on average; the forward pass adds
up segments of 512 terms (at most 32 steps, and a rounded addition a segment).

exp is within 2^-22 of a value whose argument, a fused multiply-add in base 2 with
a rounded factor, is off by 2^-22 of the largest |z| or |lse| (+ 1); sums of
exponentials add a few dozen roundings, under 2^-19 together."""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def live_targets(targets):
    return targets >= 0


def target_matrix(targets, N, smoothing):
    """[M, N]: what each row learns."""
    t = torch.full((targets.shape[0], N), smoothing / N, dtype=torch.float64, device=targets.device)
    t.scatter_add_(1, targets.long().clamp(0, N - 1)[:, None], torch.full((targets.shape[0], 1), 1.0 - smoothing,
                                                                         dtype=torch.float64, device=targets.device))
    return t


def teacher_matrix(teacher, ids, N, temperature):
    """([M, N], entropy terms [M], which rows have entries)."""
    there = (ids >= 0) & (teacher != -torch.inf)
    live = there.any(1)
    x = (teacher.double() / temperature).masked_fill(~there, -torch.inf)
    x = torch.where(live[:, None], x, torch.zeros_like(x))
    p = torch.where(there, torch.softmax(x, 1), torch.zeros_like(x))
    t = torch.zeros(ids.shape[0], N, dtype=torch.float64, device=ids.device)
    t.scatter_add_(1, ids.long().clamp(0, N - 1), p)
    return t, torch.special.xlogy(p, p).sum(1), live


def logits(A, B, scale):
    return scale * (A.double() @ B.double().T)


def forward(A, B, t, entropy, live, scale, z_loss=0.0):
    """(loss, lse): loss = sum t (log t or 0 - z + lse) + z_loss lse^2, 0 for rows that are not live."""
    z = logits(A, B, scale)
    lse = torch.logsumexp(z, 1)
    loss = entropy + lse * t.sum(1) - (t * z).sum(1) + z_loss * lse.square()
    zero = torch.zeros_like(lse)
    return torch.where(live, loss, zero), torch.where(live, lse, zero)


def z_error(A, B, scale, exact):
    """[M]: how far a row's logits may be off, the largest of them."""
    if exact:
        return torch.zeros(A.shape[0], dtype=torch.float64, device=A.device)
    K = A.shape[1]
    S = (A.double().abs() @ B.double().abs().T).max(1)[0]
    return scale * S * ((min(K, 512) + 15) // 16 * 2.0 ** -19 + (K // 512 + 1) * 2.0 ** -23)


def forward_bounds(A, B, t, scale, lse, z_loss=0.0, exact=False):
    """How far (loss, lse) may be off: lse by its logits' largest error; the loss by lse's, its
    entries' and what is left of the differences' roundings."""
    z = logits(A, B, scale)
    big = z.abs().max(1)[0] + lse.abs() + 1.0
    e = z_error(A, B, scale, exact)
    e_lse = e + 2.0 ** -19 + 2.0 ** -21 * big
    e_loss = e_lse * (1.0 + 2.0 * abs(z_loss) * lse.abs()) + e + 2.0 ** -21 * big + 2.0 ** -21 * abs(z_loss) * lse.square()
    return e_loss, e_lse


def dlogits(A, B, t, live, dloss, lse, scale, z_loss=0.0):
    """(dz, the size of its terms), [M, N]."""
    q = torch.exp(logits(A, B, scale) - lse.double()[:, None])
    f = (1.0 + 2.0 * z_loss * lse.double())[:, None]
    g = torch.where(live, dloss.double() * scale, torch.zeros_like(lse, dtype=torch.float64))[:, None]
    g = torch.where(live[:, None], g, torch.zeros_like(g))
    zero = torch.zeros_like(q)
    return (torch.where(live[:, None], g * (f * q - t), zero),
            torch.where(live[:, None], g.abs() * (f.abs() * q + t), zero))


def gradients(A, B, t, live, dloss, lse, scale, z_loss=0.0, dA=torch.bfloat16, dB=torch.bfloat16, exact=False):
    """((dA, its bound), (dB, its bound)).  dz is rounded to bf16 (2^-8 of itself) from terms each
    within 2^-17 + e of itself, e the logits' error (they are computed without segments)."""
    a, b = torch.where(live[:, None], A.double(), torch.zeros_like(A, dtype=torch.float64)), B.double()
    dz, size = dlogits(A, B, t, live, dloss, lse, scale, z_loss)
    big = torch.where(live, logits(A, B, scale).abs().max(1)[0] + lse.abs().double(), torch.zeros_like(lse, dtype=torch.float64))
    e = z_error(A, B, scale, exact) if exact or A.shape[1] <= 512 else \
        scale * (A.double().abs() @ b.abs().T).max(1)[0] * ((A.shape[1] + 15) // 16 * 2.0 ** -19)
    e = torch.where(live, e, torch.zeros_like(e))
    off = 2.0 ** -8 * dz.abs() * 1.01 + size * (2.0 ** -17 + 2.0 ** -20 * big + 2.0 * e)[:, None]
    steps = lambda n: ((n + 15) // 16 + 1) * 2.0 ** -19  # noqa: E731
    ra, rb = dz @ b, dz.T @ a
    # the pieces' sums are added up with a rounding each
    ta = off @ b.abs() + (steps(B.shape[0]) + 2.0 ** -20) * (dz.abs() @ b.abs()) + U[dA] * ra.abs()
    tb = off.T @ a.abs() + steps(A.shape[0]) * (dz.abs().T @ a.abs()) + U[dB] * rb.abs()
    return (ra, ta), (rb, tb)


def check(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound + 1e-300)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                           f"{got.flatten()[bad.flatten()][0].item()} for {want.flatten()[bad.flatten()][0].item()}, "
                           f"worst {(err / (bound + 1e-300)).nan_to_num(torch.inf).max().item():.3g} of the bound")
