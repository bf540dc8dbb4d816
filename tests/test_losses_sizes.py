"""Workspaces of the losses' calls at the largest sizes: no GPU is needed."""
import pytest

import dense_gemm_blackwell_tcgen05_gb300 as g
from tests.test_losses_abi import INVALID, ce, ce_grad, kd, kd_grad

MOST = (1 << 31) - 1
WIDE = (1 << 31) - 8          # a pitch


@pytest.mark.parametrize("M, N, K", [(MOST, 8, MOST), (MOST, MOST, MOST), (MOST, 8, 1431655704), (1 << 30, 8, MOST), (MOST, 8, WIDE)])
def test_sizes_that_no_memory_holds(M, N, K):
    """Bytes that leave 63 bits, or come round to few."""
    for grad in (0, 1):
        n = g.gemm_bf16_cross_entropy_workspace_bytes(M, N, K, grad)
        assert n == INVALID or 2 * M * K <= n < 1 << 62
        n = g.gemm_bf16_distill_workspace_bytes(M, N, K, 1024, grad)
        assert n == INVALID or 2 * M * K <= n < 1 << 62
    assert g.gemm_bf16_cross_entropy_workspace_bytes(M, N, K, 1) == INVALID


@pytest.mark.parametrize("call", [ce, ce_grad, kd, kd_grad])
def test_calls_of_such_sizes_are_refused(call):
    big = dict(M=MOST, K=WIDE, lda=WIDE, ldb=WIDE, n=(1 << 63) - 1)
    if call in (ce_grad, kd_grad):
        big.update(ld_da=WIDE, ld_db=WIDE)
    assert call(**big) == INVALID


def test_workspaces_grow_with_each_size():
    """From one size to the next in steps of up to 8 times, to the largest that are not refused."""
    for grad in (0, 1):
        for at in range(3):
            last, sizes = 0, [64, 64, 64]
            for x in (1, 8, 64, 512, 4096, 1 << 15, 1 << 18, 1 << 21, 1 << 24, 1 << 27, 1 << 30, MOST):
                sizes[at] = x
                n = g.gemm_bf16_cross_entropy_workspace_bytes(*sizes, grad)
                # (dA's parts get fewer as rows and widths grow: what they take then is at most 128 MiB)
                assert n >= last - (128 << 20) and n > 0
                last = n


def up(n, m):
    return (n + m - 1) // m * m


@pytest.mark.parametrize("M, N, K", [
    (1, 16384, 1024), (1, 1, 1), (5, 9000000, 8), (64, 131072, 4096), (100, 10007, 528), (128, 2200000, 16), (129, 32768, 2048),
    (256, 20000, 2048), (257, 1000, 96), (300, 1800000, 24), (512, 131072, 512), (1024, 262144, 4096), (2053, 50021, 1040),
    (4000, 512, 256), (4096, 65536, 1024), (4099, 50021, 1040), (8192, 131072, 4096), (34000, 9000, 72), (100000, 50021, 1040),
    (1 << 20, 520, 64)])
@pytest.mark.parametrize("top", [0, 1, 64])
def test_workspaces_are_what_the_header_says(M, N, K, top):
    """To the rounding of rows, widths and columns, vectors of 32 bytes a row, and 256 bytes a part."""
    def of(grad):
        return (g.gemm_bf16_distill_workspace_bytes(M, N, K, top, grad) if top else
                g.gemm_bf16_cross_entropy_workspace_bytes(M, N, K, grad))
    K64 = up(K, 64)
    more = 32 * M + 256 * 20 + ((12 * top + 150) * M if top else 0)
    # tiles have 32 columns at least, 256 in large calls; one block of rows needs no more than a slot
    # for each of 152 clusters
    slots = -(-N // (256 if M >= 2048 and N >= 32768 else 32))
    if M <= 128:
        slots = min(slots, 152)
    assert of(0) <= (2 * M * K64 if M > 256 else 0) + 24 * up(M, 32) * slots + 4 * M * max(top, 1) + more
    R = M + up(M, 64) if M <= 128 else M
    sums = 4 * R * K64
    piece = 2 * R * up(N, 256)
    if piece > 1 << 29:
        piece = max(1 << 29, 2 * R * 4096) + 2 * R * 256
    fixed = 2 * R * K64 + piece + (10 << 20 if M > 256 else 0) + more
    assert of(1) <= fixed + max(sums, min(32 * sums, (128 << 20) * K64 // K))
    # and no part of that is left out
    assert of(1) >= 2 * R * K + 4 * R * K + min(2 * R * N, 1 << 28)
