"""The layer for a few tokens at widths from 6144 channels on, where a workgroup of its second kernel takes 32 output channels: widths
that leave its second 16 partly or wholly absent, entries by themselves, in registers and through LDS, the largest call."""
import pytest
import torch

import expert_reference as R
import harness as Hn
import w4_reference as Q
from test_gpu_expert_ffn import table
from test_gpu_few import DEV, ep, weights     # noqa: F401  (ep is the fixture)

pytestmark = pytest.mark.gpu

FORMATS = [("bf16", 6152, 40), ("bf16", 6160, 264), ("bf16", 6168, 136), ("e4m3", 7168, 128), ("int4_32", 6176, 96), ("e2m1_64", 6208, 192),
           ("int4_128", 7168, 256)]
CALLS = [
    # T, K, E, routing: which entries go together in the second kernel
    (1, 8, 16, "uniform"),       # each by itself
    (4, 4, 4, "holes"),          # the same, experts shared
    (9, 7, 8, "uniform"),        # 16 rows an item, found in registers
    (40, 4, 20, "holes"),        # the same through LDS
    (16, 4, 3, "one"),           # 64 rows of one expert, 32 an item, in registers
    (128, 8, 48, "zipf"),        # 32 rows an item, through LDS, as many entries as there may be
    (128, 8, 256, "uniform"),    # as many, 16 rows an item: the most LDS (with 1024 experts)
]


@pytest.mark.parametrize("T,K,E,how,fmt,H,I", [c + f for c in CALLS for f in FORMATS] + [(128, 8, 1024, "uniform", "bf16", 6152, 40)])
def test_values(ep, T, K, E, how, fmt, H, I):
    print("[few wide] %s" % ((T, K, E, how, fmt, H, I),), flush=True)
    idx = table(T, E, K, how, 11) if K <= E else torch.full((T, K), E - 1, dtype=torch.int64)
    g = torch.Generator(device=DEV).manual_seed(T + H)
    call, expert = weights(ep, fmt, g, E, H, I)
    used = sorted(set(idx.view(-1).tolist()) & set(range(E)))
    idx = idx.to(DEV)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    w = torch.rand(T, K, generator=g, device=DEV) + 0.1
    bias = (torch.randn(T, H, generator=g, device=DEV) * 0.3).bfloat16()
    out, go = Hn.guarded_tensor((T, H), torch.bfloat16, DEV, "out")
    ws, gw = Hn.guarded_tensor((ep.ep_moe_few_workspace_bytes(T, K, I),), torch.uint8, DEV, "ws")
    ep.ep_moe_few(x, idx, w, call[0], call[1], w13_scales=call[2], w2_scales=call[3], bias=bias, out=out, workspace=ws)
    torch.cuda.synchronize()
    want, bound = Q.layer(x, idx, w, bias, 0, {e: expert(e) for e in used}, K)
    R.assert_within(out, want, bound, "out")
    Hn.assert_guards(go)
    Hn.assert_guards(gw)
