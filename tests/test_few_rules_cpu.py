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
    (1, 8, 16, True),       # 41 / 43, 67 / 72, 132 / 131
    (2, 4, 8, True),        # 40 / 43, 67 / 71, 130 / 129
    (4, 2, 8, True),        # small experts 11.3 / 13.8
    (2, 8, 32, True),       # 66 / 71, 117 / 119
    (2, 4, 4, False),       # 35 / 33, 53 / 40, 114 / 69
    (2, 8, 8, False),       # 60 / 44, 110 / 72, 235 / 130
    (4, 4, 4, False),       # 56 / 33, 93 / 41, 206 / 69
    (16, 1, 1, False),      # 51 / 32, 89 / 32, 165 / 34
    (4, 4, 16, False),      # 62 / 57, 109 / 95, 235 / 185
    (3, 4, 12, False),      # 53 / 43, 80 / 71, 168 / 128
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
