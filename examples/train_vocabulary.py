"""Trains a small token model on targets and on a teacher's top logits.

A token's row of an embedding goes through one matrix to a hidden state H, and
the vocabulary's matrix B gives the logits H B^T, which are never stored.  One
step runs

  * the hidden states (gemm_bf16);
  * the cross entropy of the targets (matmul_cross_entropy) and the divergence
    from a teacher's lists (matmul_distill);
  * their gradients: both add to B's in fp32 (the second with accumulate), the
    rows' go through the matrix to its own gradient (matmul_grouped_wgrad);
  * plain gradient descent on fp32 masters.

Rows of padding have a negative target and empty lists: they cost nothing.
Nothing in a step waits for the GPU.  Run: python examples/train_vocabulary.py
[--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_blackwell_tcgen05_gb300 as g  # noqa: E402


class Model:
    def __init__(self, vocabulary=2000, width=128, hidden=256, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.embedding = rand(vocabulary, width).bfloat16()
        # fp32 masters, the bf16 copies that the products read, fp32 gradients
        self.masters = [rand(hidden, width) / width ** 0.5, rand(vocabulary, hidden) / hidden ** 0.5]
        self.weights = [m.bfloat16() for m in self.masters]
        self.gradients = [torch.empty_like(m) for m in self.masters]

    def hidden(self, tokens):
        x = self.embedding[tokens]
        return x, g.matmul_bf16(x, self.weights[0])

    def top_logits(self, tokens, top):
        """A teacher's (logits, tokens) of its `top` most likely."""
        return g.matmul_bf16(self.hidden(tokens)[1], self.weights[1]).topk(top, -1)

    def step(self, tokens, targets, teacher, ids, temperature=2.0, share=0.5):
        """The mean of (1 - share) cross entropy + share temperature^2 divergence over the rows
        that count; its gradients in self.gradients."""
        x, h = self.hidden(tokens)
        B, (dW, dB) = self.weights[1], self.gradients
        counted = (targets >= 0).sum().clamp(min=1)
        hard, lse = g.matmul_cross_entropy(h, B, targets)
        soft, lse_t = g.matmul_distill(h, B, teacher, ids, temperature=temperature)
        rows = len(tokens)
        d_hard = ((1.0 - share) / counted).expand(rows)
        d_soft = (share * temperature ** 2 / counted).expand(rows)
        dh, _ = g.matmul_cross_entropy_grad(d_hard, h, B, targets, lse, dB=dB, out_dtype=torch.float32)
        dh2, _ = g.matmul_distill_grad(d_soft, h, B, teacher, ids, lse_t, temperature=temperature, dB=dB, accumulate=True,
                                       out_dtype=torch.float32)
        offsets = torch.arange(2, device="cuda", dtype=torch.int32) * rows      # one group of all rows
        g.matmul_grouped_wgrad((dh + dh2).bfloat16(), x, offsets, out=dW[None])
        return (hard * d_hard + soft * d_soft).sum()

    def update(self, rate):
        for master, weights, gradient in zip(self.masters, self.weights, self.gradients):
            master.sub_(gradient, alpha=rate)
            weights.copy_(master)


def train(steps=60, rows=1024, vocabulary=2000, top=16, rate=2.0, seed=0, report=None):
    """Fits a model to another's samples and top logits; returns the losses."""
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    teacher, model = Model(vocabulary, seed=seed), Model(vocabulary, seed=seed + 2)
    model.embedding = teacher.embedding
    teacher.weights[1] = (2.0 * teacher.masters[1]).bfloat16()
    losses = []
    for i in range(steps):
        tokens = torch.randint(0, vocabulary, (rows,), device="cuda", generator=gen)
        logits, ids = teacher.top_logits(tokens, top)
        targets = ids.gather(1, torch.multinomial(torch.softmax(logits.float(), -1), 1, generator=gen))[:, 0]
        padding = torch.rand(rows, device="cuda", generator=gen) < 0.25
        targets = torch.where(padding, -100, targets)
        ids = torch.where(padding[:, None], -1, ids)
        losses.append(model.step(tokens, targets, logits, ids))
        model.update(rate)
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
