"""Calls over so many tokens that one grid dimension does not hold their workgroups' threads (2^32): every token is served.
Rows are as narrow as they may be and hold small whole numbers, so values are exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    yield ep
    torch.cuda.empty_cache()


def whole(g, *shape):
    return torch.randint(-8, 9, shape, generator=g, device=DEV, dtype=torch.int8).bfloat16()


def test_adapter(ep):
    T, H, N, r = (1 << 29) + 777, 8, 8, 8            # two workgroups of 256 threads for 64 tokens: 2^32 threads at 2^29
    g = torch.Generator(device=DEV).manual_seed(4)
    idx = torch.randint(-1, 2, (T, 1), generator=g, device=DEV, dtype=torch.int8).long()
    h, _ = ep.ep_get_layout(idx, 2)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).random_(-2, 3, generator=g)
    a, b = whole(g, 2, r, H).clamp(-1, 1), whole(g, 2, N, r).clamp(-1, 1)
    base = torch.empty(T, N, dtype=torch.bfloat16, device=DEV).random_(-2, 3, generator=g)
    out = ep.ep_adapter(h, x, a, b, base=base)
    for at in (0, T // 3, T - 5_000_000):
        s = slice(at, at + 5_000_000)
        # every value is a whole number below 2^8, exact in bf16, but for sums past it: those round once
        v = torch.bmm(x[s].float().expand(2, -1, -1), a.float().transpose(1, 2).contiguous()).bfloat16().float()
        d = torch.bmm(v, b.float().transpose(1, 2).contiguous())
        i = idx[s].view(-1)
        want = base[s].float() + torch.where((i == 0)[:, None], d[0], torch.where((i == 1)[:, None], d[1], 0.0))
        assert torch.equal(out[s], want.bfloat16())
