"""Which kernel a product of the 4-bit expert block takes, from the library's own rule: csrc/ep_w4_rules.hpp is plain host code, compiled
here with a C++ compiler, without the GPU."""
import ctypes
import functools
import os
import subprocess
import tempfile

import pytest

from ffn_rules import CSRC

SHIM = """
#include "ep_w4_rules.hpp"
extern "C" int w4(int T, int K, int E, int El, int N, int up) { return ep::w4_kernel(ep::W4Sizes{T, K, E, El, N, up != 0}); }
"""
STREAM, TILE32, TILE64, TILE128 = range(4)


@functools.lru_cache(maxsize=None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "rules.cpp"), os.path.join(d, "rules.so")
        with open(src, "w") as f:
            f.write(SHIM)
        subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I" + CSRC, src, "-o", lib], check=True)
        return ctypes.CDLL(lib)


def w4(T, K, E, N, up, ranks=1):
    return _lib().w4(T, K, E, E // ranks, N, int(up))


# rows per expert, gate and up, down: the sizes whose times stand beside the rule
@pytest.mark.parametrize("E,H,I,rows,up,down", [
    (8, 1024, 512, 1, STREAM, STREAM), (8, 1024, 512, 40, STREAM, STREAM),
    (16, 2048, 768, 12, STREAM, STREAM), (16, 2048, 768, 128, TILE64, TILE64),
    (8, 7168, 2048, 2, STREAM, STREAM), (8, 7168, 2048, 12, STREAM, TILE32), (8, 7168, 2048, 64, TILE64, TILE64),
    (64, 4096, 1408, 2, TILE32, TILE32), (64, 4096, 1408, 128, TILE64, TILE64),
    (32, 7168, 2048, 16, TILE32, TILE32), (32, 7168, 2048, 24, TILE64, TILE64), (32, 7168, 2048, 1024, TILE128, TILE128),
])
def test_measured_sizes(E, H, I, rows, up, down):
    assert (w4(rows * E, 1, E, I, True), w4(rows * E, 1, E, H, False)) == (up, down)


def test_tiles_grow_with_the_rows():
    for E, N in [(1, 128), (8, 2048), (64, 1408), (1024, 256)]:
        for up in (False, True):
            kernels = [w4(T, 4, E, N, up) for T in [1, 2, 5, 16, 60, 200, 1000, 5000, 40000, 300000]]
            assert kernels[-1] == TILE128
            # streamed first, tiles of 32 rows next, then tiles of 64 and 128
            low = [min(k, TILE64) for k in kernels]
            assert low == sorted(low)


@pytest.mark.parametrize("E,H,I,rows,up,down", [
    (32, 7168, 2048, 40, TILE64, TILE64), (32, 7168, 2048, 56, TILE128, TILE128), (32, 7168, 2048, 96, TILE128, TILE128),
    (32, 7168, 2048, 128, TILE64, TILE64), (32, 7168, 2048, 192, TILE128, TILE128), (16, 2048, 768, 80, TILE64, TILE64),
    (4, 4096, 1408, 256, TILE64, TILE64), (16, 2048, 768, 400, TILE128, TILE128), (8, 1024, 512, 400, TILE64, TILE64),
])
def test_measured_heights(E, H, I, rows, up, down):
    assert (w4(rows * E, 1, E, I, True), w4(rows * E, 1, E, H, False)) == (up, down)


@pytest.mark.parametrize("up", [False, True])
def test_largest_and_smallest_sizes_have_a_kernel(up):
    for T in (1, 2 ** 31 - 1):
        for K in (1, 128):
            for E, ranks in ((1, 1), (32768, 8), (1024, 1024)):
                for N in (32, 32768):
                    assert w4(T, K, E, N, up, ranks) in range(4)
