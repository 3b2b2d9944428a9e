"""The expert block, the combine's gradient and the adapters through handles that other calls made: the static handle of the
call without allocations, the receiver's layout over rows from other ranks, and layouts that start from nothing."""
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


def weights(E, H, I, g):
    n = lambda *s, std: (torch.randn(*s, generator=g) * std).bfloat16().to(DEV)
    return n(E, 2 * I, H, std=H ** -0.5), n(E, H, I, std=I ** -0.5)


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("T", [3, 300])
def test_static_handle(ep, T):
    """ep_layout_dispatch_noalloc's handle serves every operator as an allocated one does."""
    H, I, E, K, A = 256, 136, 6, 2, 16
    g = torch.Generator().manual_seed(T)
    idx, x, w = W.route_uniform_distinct(T, E, K, g).to(DEV), torch.randn(T, H, generator=g).bfloat16().to(DEV), torch.rand(T, K, generator=g).to(DEV)
    go = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    w13, w2 = weights(E, H, I, g)

    def run(h, rows):
        pre = torch.zeros(rows.shape[0], 2 * I, device=DEV)
        z = lambda: torch.zeros(rows.shape[0], H, dtype=torch.bfloat16, device=DEV)
        y = ep.ep_expert_ffn(h, rows, w13, w2, y=z(), pre=pre)
        gy, gw = ep.ep_combine_backward(h, go, y, w, grad_y=z())
        dx, dw13, dw2 = ep.ep_expert_ffn_backward(h, gy, rows, pre, w13, w2, dx=z())
        return [y, gy, dx, dw13, dw2, gw]

    h, _ = ep.ep_get_layout(idx, E, expert_alignment=A)
    d = ep.ep_dispatch(h, x, w, fp8=False, do_zero_padding=True)
    want = run(h, d["recv_x"])
    out = ep.alloc_dispatch_outputs(h, H, False)
    s, _, ds = ep.ep_layout_dispatch_noalloc(idx, x, E, out, expert_alignment=A, topk_weights=w, fp8=False, do_zero_padding=True)
    got = run(s, ds["recv_x"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    ids = torch.randint(-1, 3, (T, 1), generator=g).to(DEV)
    a, b = torch.randn(3, 16, H, generator=g).bfloat16().to(DEV), torch.randn(3, 40, 16, generator=g).bfloat16().to(DEV)
    h, _ = ep.ep_get_layout(ids, 3)
    want = ep.ep_adapter(h, x, a, b)
    s, _, _ = ep.ep_layout_dispatch_noalloc(ids, x, 3, ep.alloc_dispatch_outputs(h, H, False), fp8=False)
    assert same(ep.ep_adapter(s, x, a, b), want)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_rows_received_from_other_ranks(ep, fmt):
    """Rank 1 of two places the rows that rank 0 sent it and runs its experts on them: the same rows as through one layout of
    both ranks' experts."""
    T, H, I, E, K, A = 150, 256, 128, 8, 3, 16
    g = torch.Generator().manual_seed(4)
    idx, x = W.route_uniform_distinct(T, E, K, g).to(DEV), torch.randn(T, H, generator=g).bfloat16().to(DEV)
    w = torch.rand(T, K, generator=g).to(DEV)
    fp8 = fmt == "fp8"
    if fp8:
        q = lambda *s: (torch.randn(*s, generator=g) * 104).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
        u = lambda *s: (torch.rand(*s, generator=g) / 1000).to(DEV)
        w13, w2, scales = q(E, 2 * I, H), q(E, H, I), (u(E, 2 * I // 128, H // 128), u(E, H // 128, I // 128))
    else:
        (w13, w2), scales = weights(E, H, I, g), None
    run = lambda h, d, e: ep.ep_expert_ffn(h, d["recv_x"], w13[e].contiguous(), w2[e].contiguous(), d["recv_x_scales"],
                                           *((t[e].contiguous() for t in scales) if fp8 else (None, None)))
    whole, _ = ep.ep_get_layout(idx, E, expert_alignment=A)
    d = ep.ep_dispatch(whole, x, w, fp8=fp8)
    y = run(whole, d, slice(0, E))
    out = ep.ep_combine(whole, y, w)

    h0, lay = ep.ep_get_layout(idx, E, 2, 0, A)
    d0 = ep.ep_dispatch(h0, x, w, fp8=fp8)
    n = int(lay["num_tokens_per_rank"][1])
    window = dict(x=d0["send_x"][1], s=d0["send_x_scales"][1] if fp8 else None, i=d0["send_topk_idx"][1].clone(), w=d0["send_topk_weights"][1])
    window["i"][n:] = -1
    h1, _ = ep.ep_get_layout(window["i"], E // 2, expert_alignment=A)
    d1 = ep.ep_dispatch_rows(h1, window["x"], window["s"], window["w"])
    if not fp8:
        d1["recv_x_scales"] = None
    y1 = run(h1, d1, slice(E // 2, E))
    back = torch.zeros(2, T, H, dtype=torch.bfloat16, device=DEV)
    back[1] = ep.ep_combine(h1, y1, window["w"])
    local = ep.ep_combine(h0, run(h0, d0, slice(0, E // 2)), w)
    got = ep.ep_combine_reduce(h0, back, local)
    # each rank's partial sum is rounded to bf16 on its way, and so are both results and the size itself: 2^-8 of the size at
    # most for the partial sums together and for each result
    size = ep.ep_combine(whole, y.abs(), w).float()
    assert bool(((got.float() - out.float()).abs() <= 4 * 2.0 ** -8 * size + 1e-30).all())


def test_parameters_and_views(ep):
    """Weights as a module holds them (parameters), and rows that are views into larger buffers."""
    T, H, I, E = 20, 64, 24, 2
    g = torch.Generator().manual_seed(1)
    idx = torch.randint(0, E, (T, 1), generator=g).to(DEV)
    h, _ = ep.ep_get_layout(idx, E)
    w13, w2 = weights(E, H, I, g)
    big = torch.randn(2 * T, H, generator=g).bfloat16().to(DEV)
    want = ep.ep_expert_ffn(h, big[T:].clone(), w13, w2)
    got = ep.ep_expert_ffn(h, big[T:], torch.nn.Parameter(w13), torch.nn.Parameter(w2))
    assert same(got, want) and not got.requires_grad
    a, b = torch.randn(E, 8, H, generator=g).bfloat16().to(DEV), torch.randn(E, 16, 8, generator=g).bfloat16().to(DEV)
    assert same(ep.ep_adapter(h, big[T:], torch.nn.Parameter(a), torch.nn.Parameter(b)), ep.ep_adapter(h, big[T:].clone(), a, b))
