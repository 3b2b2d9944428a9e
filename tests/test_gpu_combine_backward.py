"""Gradient of the combine against its definition in 64 bits."""
import pytest
import torch

import expert_reference as R
import harness as Hn
from test_gpu_expert_ffn import table, untouched

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


@pytest.mark.parametrize("T,H,E,ranks,rank,K,A,how", [
    (1, 8, 1, 1, 0, 1, 1, "uniform"),
    (1, 7168, 256, 1, 0, 8, 128, "uniform"),
    (61, 1032, 64, 1, 0, 6, 16, "holes"),
    (130, 520, 40, 4, 3, 32, 1, "holes"),
    (64, 32768, 4, 1, 0, 2, 1, "uniform"),
    (17, 2056, 4, 1, 0, 3, 8, "one"),
    (33, 256, 4, 1, 0, 3, 8, "none"),
    (600, 4096, 16, 1, 0, 9, 1, "uniform"),
])
@pytest.mark.parametrize("weighted", [True, False])
def test_values(ep, T, H, E, ranks, rank, K, A, how, weighted):
    print("[combine grad] T%d H%d K%d %s" % (T, H, K, how), flush=True)
    idx = table(T, E, K, how, 5)
    El = E // ranks
    slot, start, count = R.segments(idx, E, rank * El, El, A)
    slot = slot.to(DEV)
    h, _ = ep.ep_get_layout(idx.to(DEV), E, ranks, rank, A)
    rows = h.recv_capacity + 2
    gen = torch.Generator(device=DEV).manual_seed(T)
    y = torch.randn(rows, H, device=DEV, generator=gen).bfloat16()
    valid = torch.zeros(rows, dtype=torch.bool, device=DEV)
    valid[slot[slot >= 0]] = True
    y[~valid] = float("nan")
    g = torch.randn(T, H, device=DEV, generator=gen).bfloat16()
    w = torch.randn(T, K, device=DEV, generator=gen) if weighted else None
    gy, guard1 = Hn.guarded_tensor((rows, H), torch.bfloat16, DEV, "gy")
    gw, guard2 = Hn.guarded_tensor((T, K), torch.float32, DEV, "gw")
    ep.ep_combine_backward(h, g, y, w, grad_y=gy, grad_topk_weights=gw)
    torch.cuda.synchronize()
    t, k = (slot >= 0).nonzero(as_tuple=True)
    s = slot[t, k]
    scale = w[t, k].double()[:, None] if weighted else 1.0
    want = scale * g[t].double()
    # one product in fp32 (2^-24) and one rounding to bf16 (2^-8)
    R.assert_within(gy[s], want, want.abs() * (R.UBF * 1.001) + R.TINY, "grad_y")
    prod = g[t].double() * y[s].double()
    R.assert_within(gw[t, k], prod.sum(1), H * R.U32 * prod.abs().sum(1) + R.TINY, "grad_topk_weights")
    assert not gw[slot < 0].any()
    untouched(gy, valid)
    Hn.assert_guards(guard1)
    Hn.assert_guards(guard2)
    # each output alone, and again: the same bits
    only_y, none = ep.ep_combine_backward(h, g, None, w, need_grad_topk_weights=False)
    assert none is None and torch.equal(only_y.view(torch.int16)[s], gy.view(torch.int16)[s])
    none, only_w = ep.ep_combine_backward(h, g, y, w, need_grad_y=False)
    assert none is None and torch.equal(only_w, gw)


def test_no_tokens(ep):
    h, _ = ep.ep_get_layout(torch.empty((0, 2), dtype=torch.int64, device=DEV), 4)
    gy, gw = ep.ep_combine_backward(h, torch.empty((0, 64), dtype=torch.bfloat16, device=DEV),
                                    torch.empty((0, 64), dtype=torch.bfloat16, device=DEV))
    torch.cuda.synchronize()
    assert gy.shape == (0, 64) and gw.shape == (0, 2)


def test_graph_replay(ep):
    T, H, E, K = 50, 1040, 8, 3
    idx = table(T, E, K, "holes", 1).to(DEV)
    h, _ = ep.ep_get_layout(idx, E)
    y = torch.randn(h.recv_capacity, H, device=DEV).bfloat16()
    g, w = torch.randn(T, H, device=DEV).bfloat16(), torch.rand(T, K, device=DEV)
    gy, gw = torch.zeros_like(y), torch.zeros_like(w)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    ep.ep_combine_backward(h, g, y, w, grad_y=gy, grad_topk_weights=gw)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ep.ep_combine_backward(h, g, y, w, grad_y=gy, grad_topk_weights=gw, stream=side)
    for _ in range(3):
        g.copy_(torch.randn(T, H, device=DEV))
        gy.zero_(), gw.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ry, rw = ep.ep_combine_backward(h, g, y, w, grad_y=torch.zeros_like(y))
        torch.cuda.synchronize()
        assert torch.equal(ry, gy) and torch.equal(rw, gw)
