"""The expert operators together, as examples/train_experts.py uses them: its
gradients against the chain rule in 64 bits, and that a short training run
brings the loss down."""
import os
import sys

import pytest
import torch

import dense_gemm_blackwell_tcgen05_gb300 as g

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_gradients():
    """The saved activations and the incoming gradient are bf16; each product
    of theirs is rounded to bf16 once (2^-8), twice along the longer path, so
    the momenta and the rows' gradient are within 3 * 2^-8 of 64-bit ones (2-norm)."""
    from train_experts import Experts
    layer = Experts(experts=5, width=64, hidden=136, top=2, seed=3)
    gen = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(300, 64, device="cuda", generator=gen).bfloat16()
    y, saved = layer.forward(x)
    token, weight, offsets, rows, up, act = saved
    dy = torch.randn(y.shape, device="cuda", generator=gen)
    d_rows = layer.backward(dy, saved)
    assert g.gemm_last_status(torch.cuda.current_stream().cuda_stream) == g.GEMM_OK

    w = [t.double().requires_grad_() for t in layer.weights]
    r = rows.double().requires_grad_()
    out = torch.zeros_like(y, dtype=torch.float64)
    o = offsets.tolist()
    for e in range(layer.experts):
        s = slice(o[e], o[e + 1])
        h = torch.relu(r[s] @ w[0][e].T)
        out = out.index_add(0, token[s], (h @ w[1][e].T) * weight[s, None].double())
    assert (y.double() - out).norm() <= 3 * 2.0 ** -8 * out.norm()
    out.backward(dy.double())
    for got, want in ((layer.momenta[0], w[0].grad), (layer.momenta[1], w[1].grad), (d_rows, r.grad)):
        assert (got.double() - want).norm() <= 3 * 2.0 ** -8 * want.norm()


def test_training_reduces_the_loss():
    from train_experts import train
    losses = train(steps=40, tokens=2048)
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5])


def test_a_step_does_not_wait_for_the_gpu():
    """Routing, products, gradients and updates with every read-back an error."""
    from train_experts import Experts
    layer = Experts(experts=6, width=64, hidden=128, top=2, seed=5)
    gen = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(200, 64, device="cuda", generator=gen).bfloat16()

    def step():
        y, saved = layer.forward(x)
        layer.backward(y, saved)
        layer.update(0.01)
        return saved[2]

    offsets = step()   # (the library's first-call set-up)
    torch.cuda.set_sync_debug_mode("error")
    try:
        again = step()
    finally:
        torch.cuda.set_sync_debug_mode("default")
    expert = torch.softmax(g.matmul_bf16(x, layer.router).float(), -1).topk(2, -1)[1].flatten()
    want = [0] + torch.bincount(expert, minlength=6).cumsum(0).tolist()
    assert offsets.tolist() == want and again.tolist() == want and offsets.dtype == torch.int32
