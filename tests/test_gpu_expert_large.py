"""Offsets past 32 bits, weights larger than the caches, calls side by side: the expert block, the combine's gradient and
the adapters.

The rows of a layout with a large alignment lie gigabytes apart; which kernels run and in which order they add depends on
the sizes of the routing alone, so its results are those of the dense layout bit for bit.
"""
import threading

import pytest
import torch

import expert_reference as R
import test_gpu_adapter as A
import test_gpu_expert_ffn as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


def e4m3(t):
    return (t.float() * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def valid_rows(idx, E, align):
    """Rows of the layout's valid rows, expert after expert."""
    _, start, count = R.segments(idx.cpu(), E, 0, E, align)
    return torch.cat([torch.arange(s, s + c) for s, c in zip(start, count)]).to(DEV)


def spread(t, rows, cap):
    out = torch.zeros(cap, t.shape[1], dtype=t.dtype, device=DEV)
    out[rows] = t
    return out


@pytest.mark.parametrize("T", [10, 400])            # streamed weights, tiles
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_rows_far_apart(ep, T, fmt):
    E, H, I, far = 5, 8192, 128, 65536              # 327,680 rows of 16 KiB: 5.4 GB
    g = torch.Generator(device=DEV).manual_seed(5)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).bfloat16()
    idx = (torch.arange(T, device=DEV) * 7 % E).view(T, 1)
    x, dy, w13, w2 = n(T, H), n(T, H), n(E, 2 * I, H, std=H ** -0.5), n(E, H, I, std=I ** -0.5)
    gout, w = n(T, H), torch.rand(T, 1, generator=g, device=DEV)
    scales = {}
    if fmt == "fp8":
        x, w13, w2 = e4m3(x), e4m3(w13), e4m3(w2)
        u = lambda *s: torch.rand(*s, generator=g, device=DEV) / 100
        xs, scales = u(T, H // 128), dict(w13_scales=u(E, 2 * I // 128, H // 128), w2_scales=u(E, H // 128, I // 128))
    results = []
    for align in (1, far):
        h, _ = ep.ep_get_layout(idx, E, 1, 0, align)
        rows, cap = valid_rows(idx, E, align), h.recv_capacity
        xa = spread(x, rows, cap)
        if fmt == "fp8":
            y = ep.ep_expert_ffn(h, xa, w13, w2, spread(xs, rows, cap), **scales)
            results.append([y[rows]])
        else:
            pre = torch.zeros(cap, 2 * I, device=DEV)
            y = ep.ep_expert_ffn(h, xa, w13, w2, pre=pre)
            got = [y[rows], pre[rows]]
            gy, gw = ep.ep_combine_backward(h, gout, y, w)
            got += [gy[rows], gw]
            del gy, y
            dx, dw13, dw2 = ep.ep_expert_ffn_backward(h, spread(dy, rows, cap), xa, pre, w13, w2)
            results.append(got + [dx[rows], dw13, dw2])
            del dx, pre
        del xa
    for near, away in zip(*results):
        assert torch.isfinite(near.float()).all() and torch.equal(near, away)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("shape", [
    # T, H, I, E, ranks, rank, K, A, routing; w13 holds 151 MB in e4m3: read past the caches, on one row tile each,
    # on several, streamed where a call has too few tiles, and on a rank that owns half the experts
    (60, 2048, 1152, 32, 1, 0, 4, 1, "uniform"),
    (500, 4096, 1152, 16, 1, 0, 2, 16, "zipf"),
    (1, 4096, 1152, 16, 1, 0, 3, 1, "uniform"),
    (90, 2048, 1152, 64, 2, 1, 4, 8, "holes"),
], ids=["tiles", "uneven", "one_token", "second_rank"])
def test_weights_past_the_caches(ep, shape, fmt):
    F.test_forward(ep, shape, fmt)
    if fmt == "bf16":
        F.test_backward(ep, shape)


def test_adapter_tokens_far_apart(ep):
    T, H, N, r, n = 300_000, 8192, 8192, 8, 3       # x and out: 4.9 GB each
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    some = torch.cat([torch.arange(40), torch.arange(T - 40, T)]).to(DEV)
    x[some] = torch.randn(80, H, generator=g, device=DEV).bfloat16()
    a = (torch.randn(n, r, H, generator=g, device=DEV) * H ** -0.5).bfloat16()
    b = torch.randn(n, N, r, generator=g, device=DEV).bfloat16()
    ids = torch.randint(-1, n, (T, 1), generator=g, device=DEV)
    h, _ = ep.ep_get_layout(ids, n)
    out = ep.ep_adapter(h, x, a, b)
    ref, bound = A.reference(x[some], a, b, None, None, ids[some], 0)
    assert ((out[some].double() - ref).abs() <= bound).all()
    assert not out[1000:1100].any()                 # rows of zeros


def test_side_by_side(ep):
    """Three host threads, a stream each: every call gives what it gives alone."""
    wrong = {}

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            g = torch.Generator(device=DEV).manual_seed(8 + i)
            T, H, I, E = 5 + 350 * i, 512, 264, 4
            idx = torch.randint(0, E, (T, 2), generator=g, device=DEV)
            h, _ = ep.ep_get_layout(idx, E, 1, 0, 1)
            x = torch.randn(h.recv_capacity, H, generator=g, device=DEV).bfloat16()
            w13 = (torch.randn(E, 2 * I, H, generator=g, device=DEV) * H ** -0.5).bfloat16()
            w2 = (torch.randn(E, H, I, generator=g, device=DEV) * I ** -0.5).bfloat16()
            first = None
            for _ in range(10):
                pre = torch.zeros(h.recv_capacity, 2 * I, device=DEV)
                y = ep.ep_expert_ffn(h, x, w13, w2, pre=pre)
                got = (y,) + ep.ep_expert_ffn_backward(h, y, x, pre, w13, w2)
                stream.synchronize()
                first = first or got
                wrong[i] = wrong.get(i, 0) + sum(not torch.equal(p, q) for p, q in zip(first, got))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == {0: 0, 1: 0, 2: 0}
