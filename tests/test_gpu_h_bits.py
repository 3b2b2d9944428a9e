"""What h, the experts' input of the second product, keeps of its value: outputs are as close to their definition in 64 bits as one
rounding to bf16 can put them.

Rounding what is exact leaves an error of norm r.  h's own rounding, were it to bf16, would leave another of that size (1.4 r together); the
11 bits and more that it keeps leave at most an eighth of it, 1.008 r together.  1.1 r is between the two."""
import pytest
import torch

import expert_reference as R
import w4_reference as Q
from test_gpu_expert_ffn import table
from test_gpu_few import DEV, FORMATS, ep, weights     # noqa: F401  (ep is the fixture)
from test_w4_rules_cpu import STREAM, TILE32, TILE64, TILE128, w4

pytestmark = pytest.mark.gpu


def assert_one_rounding(got, want, what):
    left = float((want.bfloat16().double() - want).norm())
    off = float((got.double() - want).norm())
    assert off <= 1.1 * left, "%s: %.3f of one rounding" % (what, off / left)


def ffn64(x, w13, w2):
    p = x @ w13.t()
    I = w2.shape[1]
    return (p[:, :I] * torch.sigmoid(p[:, :I]) * p[:, I:]) @ w2.t()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K,E,H,I", [
    (1, 8, 16, 2048, 512),       # entries by themselves
    (1, 20, 40, 512, 256),       # more of them than waves
    (1, 2, 4, 512, 8192),        # rows that come to LDS in steps
    (4, 2, 12, 6400, 384),
    (9, 7, 8, 768, 640),         # an expert's together: 16 rows at a time, from registers
    (40, 4, 20, 6400, 256),      # through LDS
    (128, 8, 40, 512, 512),      # 32 rows at a time
    (128, 8, 24, 6400, 128),
])
def test_few(ep, T, K, E, H, I, fmt):
    idx = table(T, E, K, "uniform", 3).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(T + K)
    call, expert = weights(ep, fmt, g, E, H, I)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    w = torch.rand(T, K, generator=g, device=DEV) + 0.1
    want = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in idx.unique().tolist():
        t, k = (idx == e).nonzero(as_tuple=True)
        want.index_add_(0, t, w[t, k].double()[:, None] * ffn64(x[t].double(), *expert(e)))
    got = ep.ep_moe_few(x, idx, w, call[0], call[1], w13_scales=call[2], w2_scales=call[3])
    assert_one_rounding(got, want, "out")


@pytest.mark.parametrize("kind,group", [("int4", 32), ("int4", 64), ("int4", 128), ("e2m1", 32), ("e2m1", 64), ("e2m1", 128)])
@pytest.mark.parametrize("T,K,E,H,I,up,down", [
    (40, 2, 8, 640, 384, STREAM, STREAM),
    (1, 2, 8, 2048, 1152, STREAM, STREAM),
    (24, 4, 8, 7168, 2048, STREAM, TILE32),        # streamed gate and up before tiles
    (16, 8, 64, 512, 7680, TILE32, STREAM),        # and the other way round
    (100, 8, 64, 2048, 768, TILE32, TILE32),
    (320, 8, 64, 2176, 896, TILE64, TILE64),
    (480, 8, 64, 3200, 1664, TILE128, TILE128),
])
def test_w4(ep, T, K, E, H, I, up, down, kind, group):
    assert (w4(T, K, E, I, True), w4(T, K, E, H, False)) == (up, down)
    print("[w4 bits] %s" % ((T, K, E, H, I, kind, group),), flush=True)
    idx = table(T, E, K, "uniform", 3)
    slot, start, count = R.segments(idx, E, 0, E, 1)
    h, _ = ep.ep_get_layout(idx.to(DEV), E, expert_alignment=1)
    g = torch.Generator(device=DEV).manual_seed(T + K)
    (w13, w2, _, _), expert = weights(ep, "%s_%d" % (kind, group), g, E, H, I)
    x = torch.randn(h.recv_capacity, H, generator=g, device=DEV).bfloat16()
    got = ep.ep_expert_ffn_w4(h, x, w13, w2)
    want = torch.cat([ffn64(x[s:s + c].double(), *expert(e)) for e, (s, c) in enumerate(zip(start, count)) if c])
    assert_one_rounding(got[:want.shape[0]], want, "y")


@pytest.mark.parametrize("T,fmt", [(1, "int4_32"), (6, "int4_32"), (1, "bf16"), (6, "bf16"), (30, "e4m3"), (30, "bf16")])
def test_few_of_any_size(ep, T, fmt):
    """Values of h far from one: scaling x by powers of two through a linear gate scales out exactly, and infinities stay."""
    H, I, E, K = 256, 256, 8, 2
    idx = table(T, E, K, "uniform", 3).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(T)
    call, expert = weights(ep, fmt, g, E, H, I)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    run = lambda x: ep.ep_moe_few(x, idx, None, call[0], call[1], w13_scales=call[2], w2_scales=call[3])
    for scale in (2.0 ** 40, 2.0 ** 20, 2.0 ** -40):
        t = (x.double() * scale).bfloat16()
        want = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        for e in idx.unique().tolist():
            i, k = (idx == e).nonzero(as_tuple=True)
            want.index_add_(0, i, ffn64(t[i].double(), *expert(e)))
        assert_one_rounding(run(t), want, "out at %g" % scale)
    x[0, 5] = float("inf")
    assert not run(x)[0].isfinite().any()
    x[0, 5] = float("nan")
    assert run(x)[0].isnan().all()
    x[0] = 0
    assert not run(x)[0].any()


@pytest.mark.parametrize("kind,group", [("int4", 32), ("e2m1", 64), ("int4", 128)])
@pytest.mark.parametrize("T,K,E,H,I", [(1, 2, 4, 256, 640), (20, 2, 4, 256, 640), (60, 8, 64, 2048, 768), (320, 8, 64, 2176, 896), (480, 8, 64, 3200, 1664)])
@pytest.mark.parametrize("by", [9, -9])
def test_channels_of_unlike_size(ep, T, K, E, H, I, kind, group, by):
    """Every other group of channels 2^9 times as large or small as the others, and taken back by the second product's weights: blocks of a row
    differ in size, and all count the same in the result."""
    g = torch.Generator(device=DEV).manual_seed(T)
    w13, s13 = Q.random_w4(g, kind, group, E, 2 * I, H, DEV, H ** -0.5)
    w2, s2 = Q.random_w4(g, kind, group, E, H, I, DEV, I ** -0.5)
    s13[:, I:].view(E, I // group, group, -1)[:, ::2] *= 2.0 ** by
    s2[:, :, ::2] *= 2.0 ** -by
    p13, p2 = ep.ep_w4_pack(w13, s13, kind), ep.ep_w4_pack(w2, s2, kind)
    idx = table(T, E, K, "uniform", 3)
    expert = lambda e: (Q.widen(w13[e], s13[e], kind), Q.widen(w2[e], s2[e], kind))
    if T <= 128:
        x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
        want = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        for e in idx.unique().tolist():
            i, k = (idx == e).nonzero(as_tuple=True)
            i = i.to(DEV)
            want.index_add_(0, i, ffn64(x[i].double(), *expert(e)))
        assert_one_rounding(ep.ep_moe_few(x, idx.to(DEV), None, p13, p2), want, "out")
    slot, start, count = R.segments(idx, E, 0, E, 1)
    h, _ = ep.ep_get_layout(idx.to(DEV), E, expert_alignment=1)
    x = torch.randn(h.recv_capacity, H, generator=g, device=DEV).bfloat16()
    got = ep.ep_expert_ffn_w4(h, x, p13, p2)
    want = torch.cat([ffn64(x[s:s + c].double(), *expert(e)) for e, (s, c) in enumerate(zip(start, count)) if c])
    assert_one_rounding(got[:want.shape[0]], want, "y")


@pytest.mark.parametrize("power", range(-14, 4))
def test_every_scale(ep, power):
    """One step of a block's number from end to end: 16 powers of two of h, with e4m3 and 4-bit weights."""
    H, I, E, K, T = 256, 256, 4, 2, 24
    idx = table(T, E, K, "uniform", 3).to(DEV)
    for fmt in ("e4m3", "int4_32"):
        g = torch.Generator(device=DEV).manual_seed(T)
        call, expert = weights(ep, fmt, g, E, H, I)
        x = (torch.randn(T, H, generator=g, device=DEV) * 2.0 ** (power / 2 if power < 0 else power)).bfloat16()
        want = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        for e in range(E):
            i, k = (idx == e).nonzero(as_tuple=True)
            want.index_add_(0, i, ffn64(x[i].double(), *expert(e)))
        assert_one_rounding(ep.ep_moe_few(x, idx, None, call[0], call[1], w13_scales=call[2], w2_scales=call[3]), want, "%s out" % fmt)


@pytest.mark.parametrize("T,K,E", [(1, 2, 4), (1, 20, 24), (5, 2, 16), (20, 2, 4), (90, 4, 8)])
@pytest.mark.parametrize("by", [9, -9])
def test_single_channels_of_unlike_size(ep, T, K, E, by):
    """The same with every other channel, so that neighbours differ."""
    H, I = 256, 648
    g = torch.Generator(device=DEV).manual_seed(T)
    (w13, w2, _, _), expert = weights(ep, "bf16", g, E, H, I)
    w13[:, I::2] *= 2.0 ** by
    w2[:, :, ::2] *= 2.0 ** -by
    idx = table(T, E, K, "uniform", 3).to(DEV)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    want = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in idx.unique().tolist():
        i, k = (idx == e).nonzero(as_tuple=True)
        want.index_add_(0, i, ffn64(x[i].double(), *expert(e)))
    assert_one_rounding(ep.ep_moe_few(x, idx, None, w13, w2), want, "out")
