"""Which kernels the layer for a few tokens takes, from the library's own rules: csrc/ep_few_rules.hpp is plain host code, compiled here with a
C++ compiler, without the GPU."""
import ctypes
import functools
import os
import subprocess
import tempfile

import pytest

from ffn_rules import CSRC

SHIM = """
#include "ep_few_rules.hpp"
extern "C" int by_entry(int T, int K, int E) { return ep::few_by_entry(T, K, E); }
extern "C" int narrow(int H) { return ep::few_narrow(H); }
extern "C" int steps(int T, int K, int E) { const double r = ep::few_rows(T, K, E); return 10 * ep::few_up_steps(r) + ep::few_down_steps(r); }
"""


@functools.lru_cache(maxsize=None)
def rules():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "rules.cpp"), os.path.join(d, "rules.so")
        with open(src, "w") as f:
            f.write(SHIM)
        subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I" + CSRC, src, "-o", lib], check=True)
        return ctypes.CDLL(lib)


# tokens, top-k, experts: sizes whose times stand beside the rule (us with int4, e4m3 and bf16 weights by themselves / together)
@pytest.mark.parametrize("T,K,E,by_entry", [
    (1, 8, 16, True),       # 42 / 45, 68 / 74, 132 / 132
    (2, 4, 8, True),        # 41 / 44, 67 / 74, 132 / 130
    (4, 2, 8, True),        # small experts 11.6 / 15.6
    (2, 8, 32, True),       # 68 / 73, 117 / 121
    (1, 32, 32, True),
    (2, 4, 4, False),       # 36 / 35, 53 / 42, 119 / 70
    (2, 8, 8, False),       # 62 / 45, 112 / 75, 242 / 131
    (4, 4, 4, False),       # 58 / 35, 94 / 43, 212 / 71
    (16, 1, 1, False),      # 53 / 34, 91 / 34, 168 / 40
    (4, 4, 16, False),      # 64 / 58, 110 / 96, 238 / 190
    (3, 4, 12, False),      # 54 / 44, 82 / 74, 170 / 130
    (17, 1, 1024, False),   # more entries than waves
])
def test_entries_by_themselves(T, K, E, by_entry):
    assert bool(rules().by_entry(T, K, E)) == by_entry


@pytest.mark.parametrize("T,K,E,up,down", [
    (32, 8, 32, 1, 1), (48, 8, 32, 1, 1), (64, 8, 32, 2, 2), (96, 8, 32, 2, 2), (128, 8, 32, 4, 2), (64, 8, 16, 4, 2), (128, 8, 8, 4, 2),
])
def test_steps(T, K, E, up, down):
    assert rules().steps(T, K, E) == 10 * up + down


@pytest.mark.parametrize("H,narrow", [(8, True), (2048, True), (4096, True), (4104, False), (4608, False), (6144, False), (7168, False), (32768, False)])
def test_channels(H, narrow):
    assert bool(rules().narrow(H)) == narrow
