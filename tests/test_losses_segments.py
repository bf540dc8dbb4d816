"""Losses over widths of several segments: the same bits captured, on streams and at once, rows left out,
and the watchdog."""
import pytest
import torch

import dense_gemm_blackwell_tcgen05_gb300 as g

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def status():
    return g.gemm_last_status(torch.cuda.current_stream().cuda_stream)


class Problem:
    """A loss of either kind on rows of which some are left out, and its gradient."""

    def __init__(self, M, N, K, top, seed=0):
        r = torch.Generator("cuda").manual_seed(seed + M + N + K)
        self.A = torch.randn(M, K, generator=r, device="cuda").to(BF16)
        self.B = (2.0 * torch.randn(N, K, generator=r, device="cuda") / K ** 0.5).to(BF16)
        out = torch.rand(M, generator=r, device="cuda") < 0.2
        out[0] = False
        self.targets = torch.where(out, -100, torch.randint(0, N, (M,), generator=r, device="cuda"))
        self.out, self.top = out, top
        if top:
            self.ids = torch.randint(0, N, (M, top), generator=r, device="cuda").int()
            self.ids[out] = -1
            self.teacher = torch.randn(M, top, generator=r, device="cuda")
        self.dloss = torch.rand(M, generator=r, device="cuda")

    def forward(self, **k):
        if self.top:
            return g.matmul_distill(self.A, self.B, self.teacher, self.ids, **k)
        return g.matmul_cross_entropy(self.A, self.B, self.targets, **k)

    def backward(self, lse, **k):
        if self.top:
            return g.matmul_distill_grad(self.dloss, self.A, self.B, self.teacher, self.ids, lse, **k)
        return g.matmul_cross_entropy_grad(self.dloss, self.A, self.B, self.targets, lse, **k)

    def both(self, ws=(None, None), stream=None):
        loss, lse = self.forward(workspace=ws[0], stream=stream)
        return (loss, lse, *self.backward(lse, workspace=ws[1], stream=stream))

    def workspaces(self):
        M, (N, K) = len(self.A), self.B.shape
        return [g.distill_workspace(M, N, K, self.top, x) if self.top else g.cross_entropy_workspace(M, N, K, x)
                for x in (False, True)]


SIZES = [(48, 3000, 1040, 0), (100, 30000, 2056, 12), (200, 30000, 1040, 0), (700, 9000, 1032, 30), (1500, 9000, 4096, 0)]


@pytest.mark.parametrize("M, N, K, top", SIZES)
def test_the_same_bits(M, N, K, top):
    p = Problem(M, N, K, top)
    first = [t.clone() for t in p.both()]
    assert all(torch.equal(x, y) for x, y in zip(first, p.both()))
    ws = p.workspaces()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = p.both(ws)
    for w in ws:
        w.fill_(0xFF)
    for _ in range(3):
        graph.replay()
    assert status() == g.GEMM_OK
    assert all(torch.equal(x, y) for x, y in zip(first, got))
    # what rows that are left out hold does not matter
    for value in (float("nan"), float("inf")):
        p.A[p.out] = value
        p.dloss[p.out] = value
        assert all(torch.equal(x, y) for x, y in zip(first, p.both()))
    assert status() == g.GEMM_OK
    assert not first[2][p.out].any()


def test_calls_at_once():
    """Four streams, each with its own problem and workspaces."""
    problems = [Problem(*size, seed=5) for size in SIZES[:4]]
    want = [[t.clone() for t in p.both()] for p in problems]
    spaces, streams = [p.workspaces() for p in problems], [torch.cuda.Stream() for _ in problems]
    torch.cuda.synchronize()
    got = [[] for _ in problems]
    for _ in range(6):
        for p, ws, s, o in zip(problems, spaces, streams, got):
            o.append(p.both(ws, s))
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for one in many:
            assert all(torch.equal(x, y) for x, y in zip(w, one))
    assert status() == g.GEMM_OK


@pytest.mark.parametrize("M, N, K, top", [(40, 3000, 1040, 0), (200, 30000, 1040, 4), (600, 9000, 1544, 0)])
@pytest.mark.parametrize("stall", [0, 9, 16])
@pytest.mark.parametrize("grad", [False, True])
def test_a_stage_that_never_fills(M, N, K, top, stall, grad):
    """In the first and in later segments: the waits run out, the status says so, the next call is right."""
    p = Problem(M, N, K, top)
    want, lse = p.forward()
    grads = p.backward(lse)
    call = (lambda: p.backward(lse)) if grad else p.forward
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
