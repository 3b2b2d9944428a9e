"""The layer for a few tokens between 4096 and 6144 output channels, where its second kernel goes from 16 channels a workgroup to 32."""
import pytest
import torch

import expert_reference as R
import w4_reference as Q
from test_gpu_expert_ffn import table
from test_gpu_few import DEV, ep, weights     # noqa: F401  (ep is the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,H,I", [("bf16", 4096, 40), ("bf16", 4104, 136), ("bf16", 4120, 264), ("e4m3", 4224, 128), ("int4_32", 4128, 96),
                                     ("e2m1_64", 5632, 192)])
@pytest.mark.parametrize("T,K,E,how", [(1, 8, 16, "uniform"), (13, 3, 6, "holes"), (60, 4, 12, "zipf")])
def test_values(ep, T, K, E, how, fmt, H, I):
    idx = table(T, E, K, how, 17)
    g = torch.Generator(device=DEV).manual_seed(T + H)
    call, expert = weights(ep, fmt, g, E, H, I)
    used = sorted(set(idx.view(-1).tolist()) & set(range(E)))
    idx = idx.to(DEV)
    x, bias = torch.randn(T, H, generator=g, device=DEV).bfloat16(), torch.randn(T, H, generator=g, device=DEV).bfloat16()
    w = torch.rand(T, K, generator=g, device=DEV) + 0.1
    out = ep.ep_moe_few(x, idx, w, call[0], call[1], w13_scales=call[2], w2_scales=call[3], bias=bias)
    want, bound = Q.layer(x, idx, w, bias, 0, {e: expert(e) for e in used}, K)
    R.assert_within(out, want, bound, "out")
