"""The kernels that large sizes take: pairs of CTAs with tiles of 256 x 256, one
CTA's of 128 x 128, and clusters of two that share a reduction.  Each case says
which of them its size goes to and checks that it did (gemm_last_schedule).

Small integers throughout unless said otherwise: every sum is exact, so the
result is the exact one rounded once, bit for bit."""
import pytest
import torch

import dense_gemm_blackwell_tcgen05_gb300 as g
from tests.test_grouped import (DTYPES, ceil_div, dgrad64, equal_bits, forward64, gen, ints, last_schedule, marked,
                                offsets_of, ok, schedule_of, stream, wgrad64)

pytestmark = pytest.mark.gpu

# rows per group, output columns, reduction, rows and columns of the tiles taken
ROWS = [
    ([1, 0, 255, 257, 513, 31, 443], 1300, 904, 256, 256),       # a pair: 1 to 3 tiles a group, 1 to 513 rows
    ([256, 16, 700, 33, 0, 912, 0, 100], 1041, 711, 256, 256),   # odd sides; the last tile holds 17 columns
    ([1024] * 4, 1024, 1024, 256, 256),                          # whole tiles
    ([3000], 999, 1640, 256, 256),
    ([127, 0, 129, 1, 900, 143], 1000, 700, 128, 128),
    ([900, 1100, 49], 521, 1111, 128, 128),
]


def both_ways(r, per, L, red, first=0, hi=3):
    """(name, call, 64-bit result) of a forward product and a row gradient with L
    output columns and a reduction of `red`."""
    o, M, groups = offsets_of(per, first), sum(per) + 2 * first, len(per)
    X = ints(r, M, red, hi=hi)
    B, Bt = ints(r, groups, L, red, hi=hi), ints(r, groups, red, L, hi=hi)
    return o, [("forward", lambda **k: g.matmul_grouped(X, B, o, **k), lambda: forward64(X, B, o)),
               ("dgrad", lambda **k: g.matmul_grouped_dgrad(X, Bt, o, **k), lambda: dgrad64(X, Bt, o))]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("per, L, red, nt, lt", ROWS)
def test_rows_exact(per, L, red, nt, lt, dtype):
    first = 3
    _, forms = both_ways(gen(L), per, L, red, first)
    M = sum(per) + 2 * first
    for name, call, want64 in forms:
        want = want64()
        for pad, shift in ((0, 0), (1, 1)):
            buf, out = marked((M, L), dtype, pad, shift)
            call(out=out)
            ok()
            assert last_schedule() == schedule_of(nt, lt, M, len(per), L), name
            equal_bits(out, want)          # (rows of no group: NaN in both)
            out.fill_(float("nan"))
            assert buf.isnan().all(), "wrote outside the output"


# the reduction of each of 38 < tiles <= 76 is shared by two CTAs
SHARED = [([2, 0, 65, 64, 130, 100, 151, 2], 264, 3264), ([60, 1, 64, 90, 85, 0], 520, 3999), ([300], 1000, 3208),
          ([7] * 12, 600, 4100)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("per, L, red", SHARED)
def test_reduction_shared_by_two_exact(per, L, red, dtype):
    _, forms = both_ways(gen(red), per, L, red, 1, hi=2)
    M = sum(per) + 2
    tiles = schedule_of(64, 128, M, len(per), L)[1]
    for name, call, want64 in forms:
        buf, out = marked((M, L), dtype, 3, 1)
        call(out=out)
        ok()
        s = g.gemm_last_schedule()
        assert (s["ctas_per_cluster"], s["sk_tiles"], s["sk_unit"]) == (2, tiles, ceil_div(ceil_div(red, 64), 2)), name
        equal_bits(out, want64())
        out.fill_(float("nan"))
        assert buf.isnan().all(), "wrote outside the output"


def weight_tiles(groups, N, K):
    """A pair's launch of a weight gradient whose rows hold whole sectors or fp32."""
    return 2, groups * ceil_div(N, 256) * ceil_div(K, 256)


# rows per group (some over 512 and no multiples of 64), N, K
SUMS = [([513, 0, 700, 1, 1786], 1300, 1040), ([0, 2025, 15, 1960], 1000, 1328), ([1024] * 4, 1024, 1024)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("per, N, K", SUMS)
def test_weight_gradient_of_pairs_exact(per, N, K, dtype):
    """Overwriting and added, rows of whole sectors and ones that start anywhere."""
    r = gen(N)
    groups, o, M = len(per), offsets_of(per, 2), sum(per) + 5
    A, dD = ints(r, M, K), ints(r, M, N)
    want = wgrad64(dD, A, o, groups)
    for pad, shift in ((0, 0), (16, 16), (1, 1)):
        buf, dB = marked((groups, N, K), dtype, pad, shift)
        g.matmul_grouped_wgrad(dD, A, o, out=dB)
        ok()
        assert last_schedule() == weight_tiles(groups, N, K)
        equal_bits(dB, want)
        old = torch.randint(-9, 10, (groups, N, K), generator=r, device="cuda").to(dtype)
        dB.copy_(old)
        g.matmul_grouped_wgrad(dD, A, o, out=dB, accumulate=True)
        ok()
        assert last_schedule() == weight_tiles(groups, N, K)
        equal_bits(dB, old.double() + want)
        dB.fill_(float("nan"))
        assert buf.isnan().all(), "wrote outside the output"


@pytest.mark.parametrize("dtype", DTYPES)
def test_other_groups_values_stay_out_of_pairs(dtype):
    """NaN and Inf in rows of other groups and of none, and in their matrices:
    the tail of a ragged reduction is cleared in both CTAs of a pair."""
    per, N, K = [707, 5, 0, 1291], 1200, 1456
    r = gen(9)
    o, M = offsets_of(per, 2), sum(per) + 6
    A, dD, B = ints(r, M, K), ints(r, M, N), ints(r, 4, N, K)
    lo, hi = 2, 2 + per[0]
    cA, cD, cB = A.clone(), dD.clone(), B.clone()
    for t in (A, dD):
        t[:lo] = float("inf")
        t[hi:] = float("nan")
    B[1:] = float("nan")
    D = g.matmul_grouped(A, B, o, out_dtype=dtype)
    assert last_schedule() == schedule_of(256, 256, M, 4, N)
    dA = g.matmul_grouped_dgrad(dD, B, o, out_dtype=dtype)
    assert last_schedule() == schedule_of(256, 256, M, 4, K)
    dB = g.matmul_grouped_wgrad(dD, A, o, out_dtype=dtype)
    assert last_schedule() == weight_tiles(4, N, K)
    ok()
    assert torch.equal(D[lo:hi], (cA[lo:hi].double() @ cB[0].double().T).to(dtype))
    assert torch.equal(dA[lo:hi], (cD[lo:hi].double() @ cB[0].double()).to(dtype))
    assert torch.equal(dB[0], (cD[lo:hi].double().T @ cA[lo:hi].double()).to(dtype))
    assert (dB[2] == 0).all()
    assert D[hi:hi + 5].isnan().all() and dB[1].isnan().all() and dB[3].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_real_values_on_pairs(dtype):
    """Random values within the bound that test_grouped.py derives; the same bits twice."""
    per, N, K = [600, 0, 1101, 302], 1200, 1456
    r = gen(5)
    o, M = offsets_of(per), sum(per)
    A, dD = (torch.randn(M, n, device="cuda", generator=r).bfloat16() for n in (K, N))
    B = torch.randn(4, N, K, device="cuda", generator=r).bfloat16()
    u = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8

    def check(call, ref, S, red):
        got = call()
        assert last_schedule()[0] == 2
        n = 32 + red / 512 if dtype == torch.float32 else ceil_div(red, 16)
        assert ((got.double() - ref).abs() <= u * ref.abs() + n * 2.0 ** -19 * S).all()
        if dtype == torch.float32:
            assert (got.double() - ref).norm() <= 1e-6 * ref.norm()
        assert torch.equal(got, call())

    check(lambda: g.matmul_grouped(A, B, o, out_dtype=dtype), forward64(A, B, o), forward64(A.abs(), B.abs(), o), K)
    check(lambda: g.matmul_grouped_dgrad(dD, B, o, out_dtype=dtype), dgrad64(dD, B, o), dgrad64(dD.abs(), B.abs(), o), N)
    check(lambda: g.matmul_grouped_wgrad(dD, A, o, out_dtype=dtype), wgrad64(dD, A, o, 4),
          wgrad64(dD.abs(), A.abs(), o, 4), max(per))
    ok()


@pytest.mark.parametrize("stall", [0, 3])
def test_stalled_load_of_pairs_times_out_then_recovers(stall):
    per, N, K = [700, 0, 1303], 1200, 1200
    r = gen(13)
    o, M = offsets_of(per), sum(per)
    A, dD, B = ints(r, M, K), ints(r, M, N), ints(r, 3, N, K)
    old = g.gemm_set_watchdog_ms(100)
    try:
        for f, want in ((lambda: g.matmul_grouped(A, B, o), lambda: forward64(A, B, o)),
                        (lambda: g.matmul_grouped_dgrad(dD, B, o), lambda: dgrad64(dD, B, o)),
                        (lambda: g.matmul_grouped_wgrad(dD, A, o, out_dtype=torch.float32),
                         lambda: wgrad64(dD, A, o, 3))):
            assert g.gemm_debug_stall_next_launch(stall) == g.GEMM_OK
            f()
            assert last_schedule()[0] == 2
            assert g.gemm_last_status(stream()) == g.GEMM_ERR_TIMEOUT
            got = f()
            ok()
            equal_bits(got, want())
    finally:
        g.gemm_set_watchdog_ms(old)
