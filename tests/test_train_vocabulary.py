"""The example that trains a token model: it runs, its gradients are the losses'
own, and a step does not wait for the GPU."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_vocabulary
    finally:
        sys.path.pop(0)
    return train_vocabulary


def batch(ex, rows=300, vocabulary=500, top=7, seed=3):
    gen = torch.Generator("cuda").manual_seed(seed)
    teacher, model = ex.Model(vocabulary, 64, 96, seed=1), ex.Model(vocabulary, 64, 96, seed=2)
    tokens = torch.randint(0, vocabulary, (rows,), device="cuda", generator=gen)
    logits, ids = teacher.top_logits(tokens, top)
    targets = torch.where(torch.rand(rows, device="cuda", generator=gen) < 0.3, -100, ids[:, 1])
    return model, tokens, targets, logits, torch.where(targets[:, None] < 0, -1, ids)


def test_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "train_vocabulary.py"), "--steps", "3"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "step    2" in r.stdout


def test_gradients():
    ex = example()
    model, tokens, targets, teacher, ids = batch(ex)
    T, share = 2.0, 0.5
    loss = model.step(tokens, targets, teacher, ids, T, share)
    live = targets >= 0
    W, B = (w.double().requires_grad_() for w in model.weights)
    x = model.embedding[tokens].double()
    h = x @ W.T
    h = h + (model.hidden(tokens)[1].double() - h.detach())    # (the hidden states as they were rounded)
    z = h @ B.T
    hard = torch.nn.functional.cross_entropy(z, targets, reduction="none", ignore_index=-100)
    p = torch.softmax(teacher.double() / T, -1)
    soft = (p * (p.log() - torch.log_softmax(z / T, -1).gather(1, ids.clamp(min=0)))).sum(1)
    want = torch.where(live, (1 - share) * hard + share * T * T * soft, 0.0).sum() / live.sum()
    want.backward()
    assert abs(loss.item() - want.item()) < 1e-4 * abs(want.item())
    # the logits' gradient is rounded to bf16 (2^-8), that of two losses; the rows' gradient once more
    for got, ref in zip(model.gradients, (W.grad, B.grad)):
        assert (got.double() - ref).norm() <= 3 * 2.0 ** -8 * ref.norm()


def test_a_step_does_not_wait_for_the_gpu():
    ex = example()
    args = batch(ex)
    model = args[0]
    model.step(*args[1:])
    torch.cuda.synchronize()
    torch.cuda.set_sync_debug_mode("error")
    try:
        model.step(*args[1:])
        model.update(0.1)
    finally:
        torch.cuda.set_sync_debug_mode("default")
