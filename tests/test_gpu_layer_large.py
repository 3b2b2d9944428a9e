"""The layer for a few tokens, the 4-bit experts and the norms at their largest sizes, where offsets into one expert's weights pass 2^31
bytes, and side by side on two streams."""
import pytest
import torch

import expert_reference as R
import norm_reference as N
import w4_reference as Q
from test_gpu_expert_ffn import table
from test_gpu_few import run, setup, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4_32", "e2m1_128"])
def test_largest_expert(ep, fmt):
    H = I = 32768
    g = torch.Generator(device=DEV).manual_seed(1)
    call, expert = weights(ep, fmt, g, 1, H, I)
    w13, w2 = expert(0)
    for T in (1, 40):
        print("[large] %s T=%d" % (fmt, T), flush=True)
        x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
        idx = torch.zeros(T, 1, dtype=torch.int64, device=DEV)
        w = torch.rand(T, 1, generator=g, device=DEV) + 0.1
        got = ep.ep_moe_few(x, idx, w, call[0], call[1], w13_scales=call[2], w2_scales=call[3])
        want, bound = Q.layer(x, idx, w, None, 0, {0: (w13, w2)}, 1)
        R.assert_within(got, want, bound, "out")
    if isinstance(call[0], ep.W4Weights):
        for T in (20, 300):
            print("[large] %s T=%d, experts" % (fmt, T), flush=True)
            h, _ = ep.ep_get_layout(torch.zeros(T, 1, dtype=torch.int64, device=DEV), 1)
            x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
            y = ep.ep_expert_ffn_w4(h, x, call[0], call[1])
            f = R.ffn_expert(x.double(), w13, w2)
            R.assert_within(y, f["y"], f["ey"], "y")
    del w13, w2, call, expert
    torch.cuda.empty_cache()


def test_norm_rows_far_apart(ep):
    """More than 2^31 channels in all: the first and last rows."""
    T, H, eps = 66000, 32768, 1e-5
    g = torch.Generator(device=DEV).manual_seed(2)
    n = lambda *z: torch.randn(*z, generator=g, device=DEV, dtype=torch.bfloat16)
    y, res, go, gn, post, pre = n(T, H), n(T, H), n(T, H), n(T, H), n(H), n(H)
    out, normed = ep.ep_combine_norm(None, y, residual=res, post_weight=post, pre_weight=pre, eps=eps)
    d = ep.ep_combine_norm_backward(go, gn, y, residual=res, post_weight=post, pre_weight=pre, eps=eps, need_vectors=False)
    for rows in (slice(0, 3), slice(T - 3, T)):
        f = y[rows].double()
        o = N.around(f, torch.zeros_like(f), res[rows], post, None, 1.0, pre, eps)
        R.assert_within(out[rows], o["out"], o["eout"], "out")
        R.assert_within(normed[rows], o["n"], o["en"], "normed")
        want = N.gradients(f, res[rows], post, None, 1.0, pre, eps, go[rows], gn[rows])
        for k in ("grad_f", "grad_residual"):
            R.assert_within(d[k][rows], *want[k], k)
    del y, res, go, gn, out, normed, d
    torch.cuda.empty_cache()


def test_two_at_once(ep):
    """Two streams, each with its own workspaces, give what one after the other gives."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for s in range(2):
        idx, x, w, bias, call, experts, m = setup(ep, (90, 8, 6, 12, 1, 0, 4, "holes"), "int4_64", seed=20 + s)
        g = torch.Generator(device=DEV).manual_seed(s)
        n = lambda *z: torch.randn(*z, generator=g, device=DEV).bfloat16()
        T, H = x.shape
        many = table(700, 12, 4, "zipf", 30 + s).to(DEV)
        h, _ = ep.ep_get_layout(many, 12, expert_alignment=16)
        rows = n(h.recv_capacity, H)
        f, res, go, gn, post, pre = torch.randn(700, H, generator=g, device=DEV), n(700, H), n(700, H), n(700, H), n(H), n(H)
        ws = torch.empty(ep.ep_moe_few_workspace_bytes(T, 4, m["I"]), dtype=torch.uint8, device=DEV)
        ws_ffn = torch.empty(ep.ep_expert_ffn_workspace_bytes(h, H, m["I"]), dtype=torch.uint8, device=DEV)
        ws_norm = torch.empty(ep.ep_combine_norm_workspace_bytes(700, H), dtype=torch.uint8, device=DEV)

        def step(stream, idx=idx, x=x, w=w, call=call, m=m, bias=bias, h=h, rows=rows, f=f, res=res, go=go, gn=gn, post=post, pre=pre,
                 ws=ws, ws_ffn=ws_ffn, ws_norm=ws_norm):
            out = run(ep, idx, x, w, call, m, bias=bias, workspace=ws, stream=stream)
            y = ep.ep_expert_ffn_w4(h, rows, call[0], call[1], y=torch.zeros_like(rows), workspace=ws_ffn, stream=stream)
            r, nrm = ep.ep_combine_norm(h, y, residual=res, post_weight=post, pre_weight=pre, stream=stream)
            d = ep.ep_combine_norm_backward(go, gn, f, residual=res, post_weight=post, pre_weight=pre, workspace=ws_norm, stream=stream)
            return [out, y, r, nrm, d["grad_f"], d["grad_residual"], d["grad_post"], d["grad_pre"]]
        work.append(step)
    torch.cuda.synchronize()
    alone = []
    for step in work:
        alone.append(step(None))
        torch.cuda.synchronize()
    together = []
    for _ in range(6):
        for step, stream in zip(work, streams):
            with torch.cuda.stream(stream):
                together.append(step(stream))
    torch.cuda.synchronize()
    for i, got in enumerate(together):
        for a, b in zip(got, alone[i % 2]):
            assert torch.equal(a, b), i
