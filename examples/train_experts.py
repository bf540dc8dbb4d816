"""Trains a small mixture-of-experts layer with the library's expert operators.

Every token goes to its `top` experts; an expert is two matrices with a ReLU
between them.  One step runs

  * the router's logits (gemm_bf16) and its choice, sorted by expert, on the GPU;
  * both expert products on the sorted rows (matmul_grouped);
  * their gradients: to the rows (matmul_grouped_dgrad), and to the weights,
    added straight to the fp32 momentum (matmul_grouped_wgrad, accumulate);
  * the update: every expert's momentum orthogonalised (newton_schulz).

Nothing in a step waits for the GPU: the group offsets stay there.  The router
is left as it is.  Run: python examples/train_experts.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_blackwell_tcgen05_gb300 as g  # noqa: E402


class Experts:
    def __init__(self, experts=8, width=256, hidden=512, top=2, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)
        self.experts, self.top = experts, top
        self.numbers = torch.arange(experts + 1, device="cuda")
        self.router = (rand(experts, width) / width ** 0.5).bfloat16()
        # fp32 masters, the bf16 copies that the products read, fp32 momenta
        self.masters = [rand(experts, hidden, width) / width ** 0.5, rand(experts, width, hidden) / hidden ** 0.5]
        self.weights = [m.bfloat16() for m in self.masters]
        self.momenta = [torch.zeros_like(m) for m in self.masters]
        self.workspaces = [g.newton_schulz_workspace(*m.shape) for m in self.masters]

    def route(self, x):
        """(rows' tokens, rows' weights, offsets): the chosen (token, expert) pairs sorted by expert."""
        weight, expert = torch.softmax(g.matmul_bf16(x, self.router).float(), -1).topk(self.top, -1)
        weight = weight / weight.sum(-1, keepdim=True)
        by_expert, order = expert.flatten().sort(stable=True)
        # (bincount would read the largest expert's number back to the host)
        offsets = torch.searchsorted(by_expert, self.numbers, out_int32=True)
        return order // self.top, weight.flatten()[order], offsets

    def forward(self, x):
        token, weight, offsets = self.route(x)
        rows = x[token]
        up = g.matmul_grouped(rows, self.weights[0], offsets)
        act = torch.relu(up)
        down = g.matmul_grouped(act, self.weights[1], offsets, out_dtype=torch.float32)
        y = torch.zeros(x.shape, dtype=torch.float32, device="cuda").index_add_(0, token, down * weight[:, None])
        return y, (token, weight, offsets, rows, up, act)

    def backward(self, dy, saved, decay=0.9):
        """Adds the weights' gradients to the decayed momenta; returns the rows' own."""
        token, weight, offsets, rows, up, act = saved
        d_down = (dy[token] * weight[:, None]).bfloat16()
        d_up = g.matmul_grouped_dgrad(d_down, self.weights[1], offsets) * (up > 0)
        for momentum, dD, A in ((self.momenta[0], d_up, rows), (self.momenta[1], d_down, act)):
            g.matmul_grouped_wgrad(dD, A, offsets, out=momentum.mul_(decay), accumulate=True)
        return g.matmul_grouped_dgrad(d_up, self.weights[0], offsets)

    def update(self, rate):
        for master, weights, momentum, ws in zip(self.masters, self.weights, self.momenta, self.workspaces):
            step = g.newton_schulz(momentum, workspace=ws)
            rows, cols = master.shape[1:]
            master.sub_(step, alpha=rate * (rows / cols) ** 0.5 if rows > cols else rate)
            weights.copy_(master)


def train(steps=60, tokens=4096, width=256, rate=0.02, seed=0, report=None):
    """Fits the layer to a fixed random function; returns the losses."""
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    layer = Experts(width=width, seed=seed)
    target = Experts(width=width, seed=seed)          # the same router, other experts
    target.weights = [(w.float() + 0.7 * w.float().std() * torch.randn(w.shape, device="cuda", generator=gen)).bfloat16()
                      for w in target.weights]
    losses = []
    for i in range(steps):
        x = torch.randn(tokens, width, device="cuda", generator=gen).bfloat16()
        want, _ = target.forward(x)
        y, saved = layer.forward(x)
        diff = y - want
        layer.backward(diff * (2.0 / diff.numel()), saved)
        layer.update(rate * (1.0 - i / steps))
        losses.append(diff.square().mean())
        if report and (i % 10 == 0 or i + 1 == steps):
            report(f"step {i:4d}  loss {losses[-1].item():.4f}")
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    train(steps=ap.parse_args().steps, report=print)
    rc = g.gemm_last_status(torch.cuda.current_stream().cuda_stream)
    if rc != g.GEMM_OK:
        raise SystemExit(g.gemm_status_string(rc))
