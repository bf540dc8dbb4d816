"""Measured cases of the expert-training operators.

Four operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and as calls of the library:

* ``grouped``: rows sorted by expert times each expert's weights,
  D[r] = A[r] B[e(r)]^T, for the rows offsets[e] <= r < offsets[e + 1];
* ``dgrad``: its gradient to the rows, dA[r] = dD[r] B[e(r)];
* ``wgrad``: its gradient to the weights, dB[e] = sum over e's rows r of
  dD[r]^T A[r];
* ``muon``: each matrix of a batch orthogonalised by Newton-Schulz products
  (quintic, 5 steps).
"""
import math

import numpy as np
import torch

own = False

STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def listed():
    return [
        # one generated token sent to 2 of 8 small experts: a call that is all latency
        {"name": "grouped one token", "op": "grouped", "rows": 2, "groups": 8, "n": 1024, "k": 1024, "skew": 0.0, "out": "bf16"},
        # 32 sequences generate a token each, 8 of 64 experts a token: every expert's weights are read for a few rows
        {"name": "grouped decode batch", "op": "grouped", "rows": 256, "groups": 64, "n": 2048, "k": 4096, "skew": 0.5, "out": "bf16"},
        # a prompt or a training batch, unevenly routed
        {"name": "grouped batch", "op": "grouped", "rows": 16384, "groups": 32, "n": 4096, "k": 2048, "skew": 0.7, "out": "bf16"},
        # sizes that fill no tile, some experts without rows, and sums kept in 32 bits for a reduction over devices or choices
        {"name": "grouped ragged f32", "op": "grouped", "rows": 4099, "groups": 24, "n": 2053, "k": 1040, "skew": 1.5, "out": "f32"},
        # a training batch on its way back, to the activations
        {"name": "dgrad batch", "op": "dgrad", "rows": 8192, "groups": 16, "n": 4096, "k": 2048, "skew": 0.7, "out": "bf16"},
        {"name": "dgrad ragged", "op": "dgrad", "rows": 4099, "groups": 24, "n": 1040, "k": 2056, "skew": 1.5, "out": "bf16"},
        # the same to the weights: kept in 32 bits for an optimiser, or in 16 for a reduction over devices
        {"name": "wgrad batch f32", "op": "wgrad", "rows": 8192, "groups": 16, "n": 4096, "k": 2048, "skew": 0.7, "out": "f32"},
        {"name": "wgrad ragged", "op": "wgrad", "rows": 4099, "groups": 24, "n": 1040, "k": 2056, "skew": 1.5, "out": "bf16"},
        # one small weight matrix's update: a chain of small products
        {"name": "muon small", "op": "muon", "batch": 1, "rows": 256, "cols": 256, "in": "f32"},
        # the experts' updates of one layer, taken together
        {"name": "muon experts", "op": "muon", "batch": 16, "rows": 1024, "cols": 2048, "in": "f32"},
        # a large dense layer, its momentum kept in 16 bits
        {"name": "muon large", "op": "muon", "batch": 1, "rows": 4096, "cols": 4096, "in": "bf16"},
        # a tall matrix of sizes that fill no tile
        {"name": "muon tall ragged", "op": "muon", "batch": 1, "rows": 2053, "cols": 1040, "in": "f32"},
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "dgrad", "wgrad", "muon", "muon"])
    while True:
        if op == "muon":
            case = {"op": op, "batch": _log_uniform(rng, 1, 32), "rows": _log_uniform(rng, 64, 8192),
                    "cols": _log_uniform(rng, 64, 8192), "in": rng.choice(["f32", "bf16"])}
            if work(case)["flops"] <= 1.3e12:
                return case
        else:
            n, k = _log_uniform(rng, 256, 4096), _log_uniform(rng, 256, 4096)
            # k is a pitch that TMA reads, and so is n on the way back
            case = {"op": op, "rows": _log_uniform(rng, 1, 16384), "groups": _log_uniform(rng, 4, 128),
                    "n": n if op == "grouped" else max(8, n // 8 * 8), "k": max(8, k // 8 * 8),
                    "skew": round(rng.uniform(0.0, 1.5), 2), "out": rng.choice(["bf16", "bf16", "f32"])}
            if case["groups"] * case["n"] * case["k"] <= 5.3e8 and 2 * case["rows"] * case["n"] * case["k"] <= 2.7e11:
                return case


def _generator(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _rows_of_groups(case, seed):
    """How many rows each expert gets: a multinomial of uneven expert loads."""
    r = np.random.RandomState(seed % (1 << 32))
    load = np.exp(case["skew"] * r.standard_normal(case["groups"]))
    return r.multinomial(case["rows"], load / load.sum())


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "muon":
        # momentum: a few strong directions over a noise floor, rows of uneven size
        b, m, n = case["batch"], case["rows"], case["cols"]
        rank = max(1, min(m, n) // 8)
        u = torch.randn(b, m, rank, device="cuda", generator=g) / torch.arange(1, rank + 1, device="cuda").sqrt()
        v = torch.randn(b, rank, n, device="cuda", generator=g)
        x = torch.bmm(u, v) + 0.5 * torch.randn(b, m, n, device="cuda", generator=g)
        x *= torch.exp(0.3 * torch.randn(b, m, 1, device="cuda", generator=g)) * 1e-3
        x = x if case["in"] == "f32" else x.bfloat16()
        return {"case": case, "x": x, "out": torch.empty(b, m, n, dtype=torch.bfloat16, device="cuda")}
    rows, e, n, k = case["rows"], case["groups"], case["n"], case["k"]
    per = _rows_of_groups(case, seed)
    offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(per)]).astype(np.int32)).cuda()
    state = {"case": case, "offsets": offsets, "most": int(per.max())}
    out = torch.float32 if case["out"] == "f32" else torch.bfloat16
    if case["op"] != "wgrad":
        w = torch.empty(e, n, k, dtype=torch.bfloat16, device="cuda")
        state["b"] = w.normal_(0.0, 1.0 / math.sqrt(k if case["op"] == "grouped" else n), generator=g)
    if case["op"] != "dgrad":
        state["a"] = torch.randn(rows, k, device="cuda", generator=g).bfloat16()
    if case["op"] != "grouped":
        state["dd"] = (1e-2 * torch.randn(rows, n, device="cuda", generator=g)).bfloat16()
    state["out"] = torch.empty({"grouped": (rows, n), "dgrad": (rows, k), "wgrad": (e, n, k)}[case["op"]], dtype=out, device="cuda")
    return state


def run(state):
    case = state["case"]
    if own:
        import dense_gemm_blackwell_tcgen05_gb300 as lib
        if case["op"] == "grouped":
            return lib.matmul_grouped(state["a"], state["b"], state["offsets"], out=state["out"])
        if case["op"] == "dgrad":
            return lib.matmul_grouped_dgrad(state["dd"], state["b"], state["offsets"], out=state["out"])
        if case["op"] == "wgrad":
            return lib.matmul_grouped_wgrad(state["dd"], state["a"], state["offsets"], out=state["out"])
        return lib.newton_schulz(state["x"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS, out=state["out"])
    if case["op"] == "muon":
        return _plain_newton_schulz(state["x"]).to(torch.bfloat16)
    offsets, most, out = state["offsets"], state["most"], state["out"].dtype
    if case["op"] == "wgrad":
        dd = _by_expert(state["dd"], offsets, most)
        return torch.bmm(dd.transpose(1, 2), _by_expert(state["a"], offsets, most)).to(out)
    x = state["a"] if case["op"] == "grouped" else state["dd"]
    expert = torch.searchsorted(offsets[1:], torch.arange(x.shape[0], device=x.device, dtype=torch.int32), right=True)
    if x.shape[0] <= case["groups"]:
        # fewer rows than experts: each row with the weights of its own
        w = state["b"][expert].float()
        w = w.transpose(1, 2) if case["op"] == "grouped" else w
        return torch.bmm(x.float().unsqueeze(1), w).squeeze(1).to(out)
    w = state["b"].float()
    w = w.transpose(1, 2) if case["op"] == "grouped" else w
    y = torch.bmm(_by_expert(x, offsets, most), w)
    return y[expert, torch.arange(x.shape[0], device=x.device) - offsets[:-1][expert]].to(out)


def _by_expert(x, offsets, most):
    """Rows [experts, most, width] in 32 bits, zero past each expert's own."""
    at = offsets[:-1, None] + torch.arange(most, device=x.device, dtype=torch.int32)
    live = at < offsets[1:, None]
    return torch.where(live[:, :, None], x[at.clamp(max=x.shape[0] - 1)].float(), 0.0)


def _plain_newton_schulz(g):
    a, b, c = COEFFICIENTS
    x = g.float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        p = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * p + c * torch.bmm(p, p), x)
    return x.transpose(1, 2) if tall else x


def work(case):
    if case["op"] == "muon":
        b, m, n = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        size = 4 if case["in"] == "f32" else 2
        # X X^T and its square are symmetric: half of each; then a full m x m by m x n product
        return {"bytes": b * m * n * (size + 2), "flops": b * STEPS * (m * m * n + m * m * m + 2 * m * m * n)}
    rows, e, n, k = case["rows"], case["groups"], case["n"], case["k"]
    size = 4 if case["out"] == "f32" else 2
    if case["op"] == "wgrad":
        return {"bytes": 2 * rows * (n + k) + size * e * n * k + 4 * (e + 1), "flops": 2 * rows * n * k}
    # weights of the experts that rows are sent to: at most as many as there are rows
    read, written = (k, n) if case["op"] == "grouped" else (n, k)
    return {"bytes": 2 * rows * read + 2 * min(e, rows) * n * k + size * rows * written + 4 * (e + 1),
            "flops": 2 * rows * n * k}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "muon":
        a, b, c = COEFFICIENTS
        out = []
        for g in state["x"].double():
            # the iteration on the smaller side, from the definition
            # X <- a X + b (X X^T) X + c (X X^T)^2 X
            x = g.T if g.shape[0] > g.shape[1] else g
            x = x / (torch.linalg.vector_norm(x) + EPS)
            for _ in range(STEPS):
                gram = x @ x.T
                gx = gram @ x
                x = a * x + b * gx + c * (gram @ gx)
            out.append(x.T if g.shape[0] > g.shape[1] else x)
        return torch.stack(out)
    o = state["offsets"].tolist()
    full = torch.zeros(state["out"].shape, dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(zip(o[:-1], o[1:])):
        if case["op"] == "wgrad":
            full[e] = state["dd"][lo:hi].double().T @ state["a"][lo:hi].double()
        elif hi > lo and case["op"] == "grouped":
            full[lo:hi] = state["a"][lo:hi].double() @ state["b"][e].double().T
        elif hi > lo:
            full[lo:hi] = state["dd"][lo:hi].double() @ state["b"][e].double()
    return full
