"""Measured cases of the losses over a vocabulary.

Rows A [rows, width] (hidden states) and a vocabulary matrix B [vocab, width],
both bf16, have logits z = scale A B^T, which the library never stores.  Four
operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and as calls of the library:

* ``ce``: softmax cross entropy with a target per row,
  loss = lse(z) - (1 - s) z[target] - s mean(z) + c lse(z)^2, with label
  smoothing s and a penalty c on lse; it returns the losses and lse(z);
* ``ce_grad``: its gradients to A and B, given the losses' own and lse;
* ``kd``: distillation from a teacher's top logits,
  loss = sum_j p_j (log p_j - z[id_j] / T + lse(z / T)), p = softmax(teacher / T)
  over the row's entries; it returns the losses and lse(z / T);
* ``kd_grad``: its gradients to A and B, given the losses' own and lse.

Rows with a negative target, or with no entry of an id that is not negative, are
left out: loss, lse and gradients are zero.
"""
import math

import torch

own = False


def listed():
    return [
        # one generated token's likelihood: a call that is all latency
        {"name": "ce one token", "op": "ce", "rows": 1, "vocab": 16384, "width": 1024, "masked": 0.0, "smoothing": 0.0, "z": 0.0},
        # the likelihoods of a few candidates under a large vocabulary: the matrix is read for a few rows
        {"name": "ce few rows", "op": "ce", "rows": 48, "vocab": 131072, "width": 4096, "masked": 0.0, "smoothing": 0.0, "z": 0.0},
        # a training or evaluation batch
        {"name": "ce batch", "op": "ce", "rows": 8192, "vocab": 131072, "width": 4096, "masked": 0.0, "smoothing": 0.0, "z": 0.0},
        # prompts and padding left out, sizes that fill no tile, smoothed labels and a penalty on lse
        {"name": "ce ragged", "op": "ce", "rows": 4099, "vocab": 50021, "width": 1040, "masked": 0.3, "smoothing": 0.1, "z": 1e-4},
        # a small model's step back
        {"name": "ce_grad small", "op": "ce_grad", "rows": 64, "vocab": 16384, "width": 512, "masked": 0.0, "smoothing": 0.0, "z": 0.0},
        # a training batch on its way back
        {"name": "ce_grad batch", "op": "ce_grad", "rows": 8192, "vocab": 65536, "width": 4096, "masked": 0.0, "smoothing": 0.0, "z": 0.0},
        # the same with prompts and padding left out, sizes that fill no tile, smoothed labels and a penalty on lse
        {"name": "ce_grad ragged", "op": "ce_grad", "rows": 4099, "vocab": 50021, "width": 1040, "masked": 0.3, "smoothing": 0.1, "z": 1e-4},
        # a short sequence scored against its teacher
        {"name": "kd short", "op": "kd", "rows": 129, "vocab": 32768, "width": 2048, "masked": 0.0, "top": 16, "temperature": 1.0},
        # a batch with as many entries as teachers' files keep
        {"name": "kd batch", "op": "kd", "rows": 8192, "vocab": 65536, "width": 4096, "masked": 0.0, "top": 64, "temperature": 2.0},
        {"name": "kd_grad short", "op": "kd_grad", "rows": 129, "vocab": 32768, "width": 2048, "masked": 0.0, "top": 16, "temperature": 1.0},
        {"name": "kd_grad batch", "op": "kd_grad", "rows": 4096, "vocab": 65536, "width": 4096, "masked": 0.0, "top": 64, "temperature": 2.0},
        # lists of uneven length, rows without any, sizes that fill no tile
        {"name": "kd_grad ragged", "op": "kd_grad", "rows": 2053, "vocab": 50021, "width": 1040, "masked": 0.2, "top": 100, "temperature": 0.7},
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["ce", "ce_grad", "kd", "kd_grad"])
    while True:
        # the width is a pitch that TMA reads
        case = {"op": op, "rows": _log_uniform(rng, 1, 8192), "vocab": _log_uniform(rng, 512, 131072),
                "width": max(64, _log_uniform(rng, 64, 8192) // 8 * 8), "masked": rng.choice([0.0, 0.0, 0.1, 0.3, 0.6])}
        if op.startswith("ce"):
            case["smoothing"], case["z"] = rng.choice([0.0, 0.0, 0.05, 0.1]), rng.choice([0.0, 0.0, 1e-4])
        else:
            case["top"], case["temperature"] = _log_uniform(rng, 1, 128), round(rng.uniform(0.5, 4.0), 2)
        products = 3 if op.endswith("grad") else 1
        if case["vocab"] * case["width"] <= 5.4e8 and 2 * products * case["rows"] * case["vocab"] * case["width"] <= 8.7e12:
            return case


def _generator(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _left_out(case):
    return int(case["rows"] * case["masked"])


def prepare(case, seed):
    g = _generator(seed)
    rows, vocab, width = case["rows"], case["vocab"], case["width"]
    u = lambda *s: torch.rand(*s, device="cuda", generator=g)  # noqa: E731
    # logits of standard deviation 2 and, so that some rows are sure of their target and
    # others are not, up to 12 more at it
    b = torch.empty(vocab, width, dtype=torch.bfloat16, device="cuda").normal_(0.0, 2.0 / math.sqrt(width), generator=g)
    a = torch.randn(rows, width, device="cuda", generator=g)
    # frequent tokens have low numbers
    target = (u(rows).square() * vocab).long()
    a += 3.0 * u(rows, 1) * b[target].float()
    state = {"case": case, "a": a.bfloat16(), "b": b}
    out = torch.randperm(rows, device="cuda", generator=g)[:_left_out(case)]
    if case["op"].startswith("ce"):
        target[out] = -100
        state["target"] = target
    else:
        top = case["top"]
        ids = (u(rows, top).square() * vocab).long()
        ids[:, 0] = target
        # a teacher's top logits: falling, over a range of about 10
        teacher = (torch.randn(rows, top, device="cuda", generator=g) * 2.5 + 15.0).sort(1, descending=True)[0]
        if case["masked"] > 0.0:
            # lists of uneven length end in entries of no id
            ids[torch.arange(top, device="cuda")[None, :] >= 1 + (u(rows, 1) * top).long()] = -1
            ids[out] = -1
        state["ids"], state["teacher"] = ids.int(), teacher
    if case["op"].endswith("grad"):
        # the losses are averaged with uneven weights
        state["dloss"] = (0.5 + u(rows)) / rows
        live, scale = _live(state), 1.0 / case.get("temperature", 1.0)
        lse = (state["a"].float() @ b.float().T).mul_(scale).logsumexp(1)
        state["lse"] = torch.where(live, lse, 0.0)
        state["da"], state["db"] = torch.empty_like(state["a"]), torch.empty_like(b)
    return state


def _live(state):
    return state["target"] >= 0 if "target" in state else (state["ids"] >= 0).any(1)


def run(state):
    case = state["case"]
    if own:
        import dense_gemm_blackwell_tcgen05_gb300 as lib
        if case["op"] == "ce":
            return lib.matmul_cross_entropy(state["a"], state["b"], state["target"], label_smoothing=case["smoothing"],
                                            z_loss=case["z"])
        if case["op"] == "ce_grad":
            return lib.matmul_cross_entropy_grad(state["dloss"], state["a"], state["b"], state["target"], state["lse"],
                                                 label_smoothing=case["smoothing"], z_loss=case["z"],
                                                 dA=state["da"], dB=state["db"])
        if case["op"] == "kd":
            return lib.matmul_distill(state["a"], state["b"], state["teacher"], state["ids"], temperature=case["temperature"])
        return lib.matmul_distill_grad(state["dloss"], state["a"], state["b"], state["teacher"], state["ids"], state["lse"],
                                       temperature=case["temperature"], dA=state["da"], dB=state["db"])
    a, b, live = state["a"].float(), state["b"].float(), _live(state)
    z = (a @ b.T).mul_(1.0 / case.get("temperature", 1.0))
    if case["op"] in ("ce", "kd"):
        top = z.max(1, keepdim=True)[0]
        lse = (z - top).exp_().sum(1).log() + top[:, 0]
        if case["op"] == "ce":
            s = case["smoothing"]
            loss = lse - (1.0 - s) * z.gather(1, state["target"].clamp(min=0)[:, None])[:, 0] + case["z"] * lse.square()
            if s > 0.0:
                loss = loss - s * z.double().mean(1).float()
        else:
            p, logp = _teacher(state)
            loss = (p * (logp + (lse[:, None] - z.gather(1, state["ids"].long().clamp(min=0))))).sum(1)
        return torch.where(live, loss, 0.0), torch.where(live, lse, 0.0)
    lse = state["lse"]
    q = z.sub_(lse[:, None]).exp_()
    if case["op"] == "ce_grad":
        s = case["smoothing"]
        if case["z"] > 0.0:
            q.mul_((1.0 + 2.0 * case["z"] * lse)[:, None])
        if s > 0.0:
            q.sub_(s / case["vocab"])
        q.scatter_add_(1, state["target"].clamp(min=0)[:, None], torch.full_like(lse, s - 1.0)[:, None])
    else:
        q.scatter_add_(1, state["ids"].long().clamp(min=0), -_teacher(state)[0])
    q.mul_(torch.where(live, state["dloss"] / case.get("temperature", 1.0), 0.0)[:, None])
    return (q @ b).to(torch.bfloat16), (q.T @ a).to(torch.bfloat16)


def _teacher(state):
    """A teacher's probabilities of its entries and their logarithms, both 0 where there is no entry."""
    there = state["ids"] >= 0
    t = torch.where(there, state["teacher"].float() / state["case"]["temperature"], -math.inf)
    t = t - t.max(1, keepdim=True)[0].clamp(min=-1e30)
    e = t.exp()
    total = e.sum(1, keepdim=True).clamp(min=1e-30)
    return e / total, torch.where(there, t - total.log(), 0.0)


def work(case):
    rows, vocab, width = case["rows"] - _left_out(case), case["vocab"], case["width"]
    read = 2 * (rows + vocab) * width + (8 * case["rows"] if case["op"].startswith("ce") else 8 * case["rows"] * case["top"])
    if case["op"].endswith("grad"):
        # the logits, and from them a product to the rows and one to the matrix
        return {"bytes": read + 8 * case["rows"] + 2 * (case["rows"] + vocab) * width, "flops": 6 * rows * vocab * width}
    return {"bytes": read + 8 * case["rows"], "flops": 2 * rows * vocab * width}


def exact(case, seed):
    state = prepare(case, seed)
    rows, vocab, back = case["rows"], case["vocab"], case["op"].endswith("grad")
    a, b = state["a"].double(), state["b"].double()
    if (6 if back else 2) * rows * vocab * case["width"] > 1.4e13:
        return None
    losses = torch.zeros(rows, dtype=torch.float64, device="cuda")
    lses = torch.zeros_like(losses)
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    step = max(1, (1 << 28) // vocab)
    for lo in range(0, rows, step):
        # the rows that count, by their numbers
        r = torch.arange(lo, min(rows, lo + step), device="cuda")
        t = torch.zeros(len(r), vocab, dtype=torch.float64, device="cuda")   # the distribution that is learnt
        if "target" in state:
            keep = state["target"][r] != -100
            r, t = r[keep], t[keep]
            s = case["smoothing"]
            t += s / vocab
            t[torch.arange(len(r), device="cuda"), state["target"][r]] += 1.0 - s
            temperature, entropy, c = 1.0, 0.0, case["z"]
        else:
            keep = state["ids"][r].max(1)[0] >= 0
            r, t = r[keep], t[keep]
            temperature, c = case["temperature"], 0.0
            ids = state["ids"][r].long()
            w = torch.softmax((state["teacher"][r].double() / temperature).masked_fill(ids < 0, -math.inf), 1)
            t.scatter_add_(1, ids.clamp(min=0), w)
            entropy = torch.special.xlogy(w, w).sum(1)
        if len(r) == 0:
            continue
        z = a[r] @ b.T / temperature
        if back:
            lse = state["lse"][r].double()
            d = torch.exp(z - lse[:, None]) * (1.0 + 2.0 * c * lse[:, None]) - t
            d *= (state["dloss"][r].double() / temperature)[:, None]
            da[r] = d @ b
            db += d.T @ a[r]
        else:
            lse = torch.logsumexp(z, 1)
            losses[r] = lse - (t * z).sum(1) + entropy + c * lse.square()
            lses[r] = lse
    return (da, db) if back else (losses, lses)
