"""Index arithmetic of the CUDA-core dK/dV pass (csrc/diff_rows.h), compiled for
the host: sizes whose run would take minutes, against Python's integers."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILE = 64


@pytest.fixture(scope="module")
def part_rows(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx, "a C++ compiler builds the library, and this test"
    folder = tmp_path_factory.mktemp("diff_rows")
    src, out = folder / "rows.cpp", folder / "rows.so"
    src.write_text('#include "diff_rows.h"\n'
                   'extern "C" void rows(const int* a, int* r) {\n'
                   "  const fbob::RowRange x = fbob::part_rows(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);\n"
                   "  r[0] = x.first;\n  r[1] = x.end;\n}\n")
    include = os.path.join(ROOT, "exact_second_order_two_gb300", "csrc")
    # sums and products past 31 bits wrap, as on the device
    subprocess.run([cxx, "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I" + include, str(src),
                    "-o", str(out)], check=True)
    fn = ctypes.CDLL(str(out)).rows

    def call(*a):
        r = (ctypes.c_int * 2)()
        fn((ctypes.c_int * 7)(*a), r)
        return r[0], r[1]
    return call


def check(part_rows, N, G, start, split):
    """The parts of a group cover every row of every head once, in tiles."""
    per_head = (N - start + TILE - 1) // TILE
    cuts = [per_head * G * p // split for p in range(split + 1)]
    heads = sorted({0, 1, G // 2, G - 1} & set(range(G)))
    for g in heads:
        at = start
        for t0, t1 in zip(cuts, cuts[1:]):
            if t0 >= t1 or not (t0 // per_head <= g and g * per_head < t1):
                continue
            first, end = part_rows(t0, t1, g, per_head, start, N, TILE)
            lo, hi = max(t0, g * per_head), min(t1, (g + 1) * per_head)
            assert first == start + (lo - g * per_head) * TILE
            assert end == min(N, start + (hi - g * per_head) * TILE)
            assert first == at
            at = end
        assert at == N


# (B H N is at most 2^33, B H at most 32767, N at most 2^30)
@pytest.mark.parametrize("N,G", [(65600, 32767), (1 << 18, 32767), (1 << 30, 8), (1 << 30, 1), (1, 32767)])
@pytest.mark.parametrize("split", [1, 2, 152])
def test_largest_sizes(part_rows, N, G, split):
    for start in {0, N // 2 // TILE * TILE, (N - 1) // TILE * TILE}:
        check(part_rows, N, G, start, split)


def test_small_sizes(part_rows):
    rng = random.Random(1)
    for _ in range(300):
        N = rng.randint(1, 2000)
        check(part_rows, N, rng.randint(1, 9), rng.randrange(0, N) // TILE * TILE, rng.randint(1, 40))
