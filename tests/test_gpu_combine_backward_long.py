"""Gradient of the combine over more tokens than a launch holds workgroups of 256 threads in one dimension."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_more_tokens_than_one_grid_dimension_holds():
    import combine_get_dispatch_03_amd as ep
    T, H, E = (1 << 24) + 1237, 8, 3                 # 2^24 workgroups of 256 threads are 2^32 threads
    g = torch.Generator(device=DEV).manual_seed(2)
    idx = torch.randint(-1, E, (T, 1), generator=g, device=DEV)
    h, _ = ep.ep_get_layout(idx, E)
    # small whole numbers: products and sums are exact, whatever the order
    go = torch.randint(-8, 9, (T, H), generator=g, device=DEV, dtype=torch.int8).bfloat16()
    w = torch.randint(1, 5, (T, 1), generator=g, device=DEV, dtype=torch.int8).float()
    y = torch.randint(-8, 9, (h.recv_capacity, H), generator=g, device=DEV, dtype=torch.int8).bfloat16()
    gy, gw = ep.ep_combine_backward(h, go, y, w, grad_y=torch.zeros_like(y))
    order = torch.sort(torch.where(idx.view(-1) < 0, E, idx.view(-1)), stable=True).indices
    order = order[:int((idx >= 0).sum())]            # token of each row, expert after expert
    n = order.numel()
    assert torch.equal(gy[:n], go[order] * w[order].bfloat16()) and not gy[n:].any()
    want = torch.zeros(T, device=DEV)
    want[order] = (go[order].float() * y[:n].float()).sum(1)
    assert torch.equal(gw.view(-1), want)
