"""Which kernels a call of the expert block takes, from the library's own rules: csrc/ep_ffn_rules.hpp is plain host code, so
it is compiled here with a C++ compiler, without the GPU."""
import ctypes
import functools
import os
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_get_dispatch_03_amd", "csrc")

SHIM = """
#include "ep_ffn_rules.hpp"
extern "C" int ffn_path(int T, int K, int E, int El, int hidden, int inter, int fp8) {
    const ep::FfnSizes s{T, K, E, El, hidden, inter, fp8 != 0};
    return (ep::few_rows_up(s) ? 1 : 0) | (ep::few_rows_down(s) ? 2 : 0) | (ep::weights_once(s) ? 4 : 0);
}
"""


@functools.lru_cache(maxsize=None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "rules.cpp"), os.path.join(d, "rules.so")
        with open(src, "w") as f:
            f.write(SHIM)
        subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I" + CSRC, src, "-o", lib], check=True)
        return ctypes.CDLL(lib)


def path(T, K, E, ranks, hidden, inter, fmt):
    """(gate and up projection, down projection): "stream", "tile" or, for weights marked as read once, "tile once"."""
    bits = _lib().ffn_path(T, K, E, E // ranks, hidden, inter, int(fmt == "fp8"))
    return "stream" if bits & 1 else "tile once" if bits & 4 else "tile", "stream" if bits & 2 else "tile"


# A tiled kernel runs on 256 workgroups at most, so with more tiles than that a workgroup hands over from one to another.
BM_UP, BM_DOWN = dict(bf16=256, fp8=192), dict(bf16=256, fp8=160)


def row_tiles(counts, bm):
    return sum(-(-c // bm) for c in counts)


def tiles(counts, hidden, inter, fmt):
    """Tiles of the two forward products and (bf16) of the gradients' row products, dp and dx."""
    up, down = row_tiles(counts, BM_UP[fmt]), row_tiles(counts, BM_DOWN[fmt])
    return dict(up=up * -(-inter // 128), down=down * -(-hidden // 256), dp=up * -(-inter // 256), dx=up * -(-hidden // 256))
