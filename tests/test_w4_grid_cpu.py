"""What the choice of a kernel for the 4-bit block has to hold to over all sizes that the interface takes: streaming only while its grid is
small, tiles of 128 rows for the largest calls, streaming for the smallest."""
import pytest

from test_w4_rules_cpu import STREAM, TILE128, w4

MAX_TOKENS, MAX_TOPK, MAX_EXPERTS, MAX_RANKS, MAX_CHANNELS = 10 ** 9, 32, 1024, 64, 32768
TOKENS = sorted({t for b in range(30) for t in (1 << b, (1 << b) + 1, 3 << b) if t <= MAX_TOKENS} | {MAX_TOKENS})
EXPERTS = [(1, 1), (8, 1), (64, 64), (96, 3), (256, 8), (1024, 1), (MAX_EXPERTS, MAX_RANKS)]


def grid(T, K, E, ranks, N, up):
    """Workgroups of the streamed kernel: 64 rows by 32 channels of gate and up each or by 64, every expert's last tile short."""
    entries = T * K
    busy, channels = min(entries, E // ranks), 32 if up else 64
    return (entries + 63 * busy) // 64 * -(-N // channels)


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("E,ranks", EXPERTS)
def test_streamed_grids_are_small(E, ranks, up):
    streamed = 0
    for N in (32, 96, 512, 2048, 7168, MAX_CHANNELS):
        for K in (1, 8, MAX_TOPK):
            for T in TOKENS:
                if w4(T, K, E, N, up, ranks) == STREAM:
                    streamed += 1
                    # far below 2^32 threads of 256 a workgroup: few rows or few tiles are what streaming is for
                    assert grid(T, K, E, ranks, N, up) < 1 << 18, (T, K, N)
    assert streamed


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("E,ranks", EXPERTS)
def test_largest_and_smallest(E, ranks, up):
    assert w4(1, 1, E, 32, up, ranks) == STREAM
    assert w4(MAX_TOKENS, MAX_TOPK, E, MAX_CHANNELS, up, ranks) == TILE128
