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


def layout(ep, T, E, g, ranks=1, lo=-1):
    """A layout of one entry per token, and the token of every row of rank 0."""
    idx = torch.randint(lo, E, (T, 1), generator=g, device=DEV, dtype=torch.int32).long()
    h, lay = ep.ep_get_layout(idx, E, ranks)
    mine = E // ranks
    token = [(idx.view(-1) == e).nonzero().view(-1) for e in range(mine)]
    return idx, h, torch.cat(token)


@pytest.mark.parametrize("what", ["bf16", "fp8", "rows"])
def test_dispatch(ep, what):
    T, H = (1 << 26) + 1237, 128 if what == "fp8" else 8      # a wave per token: 2^32 threads at 2^26
    g = torch.Generator(device=DEV).manual_seed(1)
    idx, h, token = layout(ep, T, 3, g)
    if what == "fp8":
        x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
        x[:, 0] = torch.randint(1, 5, (T,), generator=g, device=DEV, dtype=torch.int8).bfloat16() * 7
        out = ep.ep_dispatch(h, x, fp8=True, want_meta=False)
        # the largest of the 128 channels becomes 448, the scale what it was divided by
        assert bool((out["recv_x"][:token.numel(), 0] == 0x7E).all())
        got = out["recv_x_scales"][:token.numel(), 0] * 448
        assert bool(((got - x[token, 0].float()).abs() <= 448 * 28 * 2.0 ** -22).all())
    else:
        x = whole(g, T, H)
        out = ep.ep_dispatch(h, x, fp8=False) if what == "bf16" else ep.ep_dispatch_rows(h, x)
        assert torch.equal(out["recv_x"][:token.numel()], x[token])
        assert torch.equal(out["recv_src_idx"][:token.numel()], token.int())


def test_combine(ep):
    T, H = (1 << 26) + 1237, 8
    g = torch.Generator(device=DEV).manual_seed(2)
    idx, h, token = layout(ep, T, 3, g)
    y, bias = whole(g, h.recv_capacity, H), whole(g, T, H)
    out = ep.ep_combine(h, y, None, bias=bias)
    want = bias.clone()
    want[token] += y[:token.numel()]
    assert torch.equal(out, want)


def test_combine_tokens_and_reduce(ep):
    T, H = (1 << 26) + 1237, 8
    g = torch.Generator(device=DEV).manual_seed(3)
    idx, h, token = layout(ep, T, 4, g, ranks=2)
    e = idx.view(-1)
    here, there = ((e >= 0) & (e < 2)).nonzero().view(-1), (e >= 2).nonzero().view(-1)
    y = whole(g, T, H)
    want = torch.zeros_like(y)
    want[here] = y[:here.numel()]
    assert torch.equal(ep.ep_combine_tokens(h, y), want)
    partials = torch.zeros(2, T, H, dtype=torch.bfloat16, device=DEV)
    partials[1] = y
    want = torch.zeros_like(y)
    want[there] = y[:there.numel()]
    assert torch.equal(ep.ep_combine_reduce(h, partials), want)


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
