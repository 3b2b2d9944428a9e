"""The layer for a few tokens where each entry stands by itself: up to 16 entries on enough experts, some shared all the same, unused,
invalid, or another rank's; output widths of 16 and of 32 channels a workgroup."""
import pytest
import torch

import expert_reference as R
import w4_reference as Q
from test_few_rules_cpu import rules
from test_gpu_expert_ffn import table
from test_gpu_few import DEV, ep, weights     # noqa: F401  (ep is the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,H,I", [("bf16", 1032, 328), ("bf16", 6152, 40), ("e4m3", 384, 256), ("e4m3", 7168, 128), ("int4_64", 320, 448),
                                     ("e2m1_128", 6272, 128)])
@pytest.mark.parametrize("T,K,E,ranks,rank,how", [
    (1, 16, 64, 1, 0, "uniform"), (1, 3, 8, 2, 1, "uniform"), (2, 4, 8, 1, 0, "one"), (4, 2, 12, 3, 1, "holes"), (8, 1, 8, 1, 0, "none"),
    (16, 1, 40, 1, 0, "zipf"), (2, 8, 32, 2, 0, "uniform"), (5, 3, 30, 1, 0, "holes"),
])
def test_values(ep, T, K, E, ranks, rank, how, fmt, H, I):
    assert rules().by_entry(T, K, E)
    idx = table(T, E, K, how, 5)
    if T > 3 and K > 1:
        idx[0, 0], idx[0, 1] = 2 ** 63 - 1, -2 ** 63
    El = E // ranks
    lo = rank * El
    g = torch.Generator(device=DEV).manual_seed(T * 31 + H)
    call, expert = weights(ep, fmt, g, El, H, I)
    used = sorted({e - lo for e in idx.view(-1).tolist()} & set(range(El)))
    idx = idx.to(DEV)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    w = torch.rand(T, K, generator=g, device=DEV) + 0.1
    w[(idx < lo) | (idx >= lo + El)] = float("nan")          # weights of entries that add nothing
    bias = (torch.randn(T, H, generator=g, device=DEV) * 0.3).bfloat16()
    out = ep.ep_moe_few(x, idx, w, call[0], call[1], w13_scales=call[2], w2_scales=call[3], num_ranks=ranks, rank=rank, bias=bias)
    want, bound = Q.layer(x, idx, w, bias, lo, {e: expert(e) for e in used}, K)
    R.assert_within(out, want, bound, "out")
