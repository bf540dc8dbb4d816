"""How the products of the losses' gradients are dealt to clusters: every item once, and no cluster
long after the others, whatever the sizes.  The arithmetic is the kernels' own, compiled for the
host: no GPU is needed."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_gemm_blackwell_tcgen05_gb300", "csrc")


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("deal") / "deal.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", f"-I{CSRC}",
                    os.path.join(ROOT, "tests", "loss_deal_shim.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).loss_deal_walk
    f.argtypes = [ctypes.c_uint32] * 13 + [ctypes.POINTER(ctypes.c_uint64)]
    f.restype = None

    def call(*sizes):
        out = (ctypes.c_uint64 * 6)()
        f(*sizes, out)
        return dict(zip(("parts", "parts_db", "missing", "twice", "last", "mean"), out))
    return call


def check(walk, M, count, n, K, width, cg, most, most_db, rows, matrix, db_cost):
    nt = -(-(-(-K // -(-K // (128 * cg)))) // 64) * 64
    lt, G = 128 * cg, 152 // cg
    d = walk(M, count, n, K, width, nt, lt, most, most_db, rows, matrix, db_cost, G)
    assert d["missing"] == d["twice"] == 0, d
    if n < width:
        return d
    # no cluster can end before the mean, nor before the shortest part of Rows; beyond that, an item of
    # either kind more than others have, and what Rows' parts are kept few for, their sums' way
    part = -(-(-(-width // 64)) // most) + 5 if rows and count else 0
    item = max(-(-(-(-count // 64)) // d["parts_db"]) + 3, db_cost) if matrix else 0
    way = min(d["parts"], most) * (count * K * 8 // 1500000) if rows else 0
    each = -(-(-(-width // 64)) // d["parts"]) + 5 if rows and count else 0
    assert d["last"] <= 16 * (max(d["mean"] / 16, part) + item + each / 2 + way + 2) * 1.1, d
    return d


# rows, tokens of a piece, width: pieces are 2^28 / rows tokens wide at most
@pytest.mark.parametrize("matrix", [0, 1])
@pytest.mark.parametrize("rows, width, K", [(129, 1 << 20, 64), (129, (1 << 20) + 64, 64), (65, 3000064, 8), (69, 3000064, 8),
                                            (256, (1 << 20), 64), (65, 4100096, 256), (65, 2200064, 1024)])
@pytest.mark.parametrize("cg", [1, 2])
def test_few_rows_against_millions_of_tokens(walk, rows, width, K, matrix, cg):
    """Rows' few tiles go in parts there most of all: one of a tile would be 16 000 stages and more."""
    d = check(walk, rows, rows, width, K, width, cg, 32, 1, 1, matrix, 6)
    assert d["parts"] > 1


def test_sizes_of_all_kinds(walk):
    rng = random.Random(5)
    log = lambda lo, hi: int(round(2 ** rng.uniform(lo, hi)))  # noqa: E731
    for _ in range(1500):
        M = log(0, 17)
        count = M if rng.random() < 0.5 else rng.randint(0, M)
        width = min(log(0, 22), max(4096, 2 ** 28 // M))
        n = width if rng.random() < 0.7 else rng.randint(1, width)
        K = log(3, 13) // 8 * 8
        cg = rng.choice([1, 2])
        most = max(1, min(32, -(-width // 256), (128 << 20) // (4 * M * K)))
        tiles = -(-width // 128) * -(-K // 128)
        most_db = max(1, min(152 // tiles, -(-M // 64) // 8)) if n == width else 1
        rows, matrix = rng.choice([(1, 1), (1, 1), (0, 1), (1, 0)])
        check(walk, M, count, n, K, width, cg, most, most_db, rows, matrix, rng.choice([6, 10]))


@pytest.mark.parametrize("M, width, K", [(1 << 20, 4096, 8192), (1 << 22, 4096, 64), (1, 1 << 22, 1 << 17)])
def test_times_that_leave_32_bits(walk, M, width, K):
    check(walk, M, M, width, K, width, 2, max(1, min(32, (128 << 20) // (4 * M * K))), 1, 1, 1, 6)
