"""The operators as they are used together: a training step of a mixture-of-experts layer through layout, dispatch, the
experts, the combine and back; the same in e4m3 for serving; and a shared projection with adapters as the combine's bias."""
import pytest
import torch

import expert_reference as R
import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


def layer64(x, idx, w, w13, w2):
    """The layer in 64 bits: out[t] = sum_k w[t,k] ffn_e(x[t])."""
    I = w2.shape[2]
    out = torch.zeros_like(x)
    for k in range(idx.shape[1]):
        for e in range(w13.shape[0]):
            t = (idx[:, k] == e).nonzero().view(-1)
            p = x[t] @ w13[e].t()
            h = torch.nn.functional.silu(p[:, :I]) * p[:, I:]
            out = out.index_add(0, t, w[t, k, None] * (h @ w2[e].t()))
    return out


@pytest.mark.parametrize("T,H,I,E,K,A", [(96, 128, 64, 4, 2, 16), (301, 256, 136, 6, 3, 1)])
def test_training_step(ep, T, H, I, E, K, A):
    g = torch.Generator().manual_seed(T)
    idx = W.route_uniform_distinct(T, E, K, g)
    idx[::7, K - 1] = -1
    idx = idx.to(DEV)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DEV)
    x, w = n(T, H).bfloat16(), torch.rand(T, K, generator=g).to(DEV) + 0.1
    w13, w2, go = n(E, 2 * I, H, std=H ** -0.5).bfloat16(), n(E, H, I, std=I ** -0.5).bfloat16(), n(T, H).bfloat16()

    h, _ = ep.ep_get_layout(idx, E, expert_alignment=A)
    rows = ep.ep_dispatch(h, x, w, fp8=False)["recv_x"]
    pre = torch.empty(rows.shape[0], 2 * I, device=DEV)
    y = ep.ep_expert_ffn(h, rows, w13, w2, pre=pre)
    out = ep.ep_combine(h, y, w)
    gy, gw = ep.ep_combine_backward(h, go, y, w)
    dxr, dw13, dw2 = ep.ep_expert_ffn_backward(h, gy, rows, pre, w13, w2)
    dx = ep.ep_combine(h, dxr)                      # the dispatch's gradient: the sum over a token's rows

    leaf = [t.double().requires_grad_() for t in (x, w, w13, w2)]
    ref = layer64(leaf[0], idx, *leaf[1:])
    want = torch.autograd.grad((ref * go.double()).sum(), leaf)
    # a chain of at most four bf16 roundings, each 2^-8 of its value at most and unbiased: the norm of the
    # difference stays under four of them
    for name, a, b in (("out", out, ref.detach()), ("dx", dx, want[0]), ("dw", gw, torch.where(idx >= 0, want[1], 0.0)),
                       ("dw13", dw13, want[2]), ("dw2", dw2, want[3])):
        off = float((a.double() - b).norm() / b.norm())
        assert off < 4 * 2.0 ** -8, "%s is off by %.3g" % (name, off)

    # against differences: the loss moves by the gradient's component along a direction.  The loss itself is evaluated
    # in 64 bits, so the difference quotient is good to O(step^2).
    for i, got in ((0, dx), (1, gw), (2, dw13), (3, dw2)):
        d = torch.randn(leaf[i].shape, generator=g, dtype=torch.float64).to(DEV)
        d /= d.norm()
        d = d + got.double() / got.double().norm()   # a direction along which the loss does move
        step = 1e-4
        moved = [[(t + s * d).detach() if j == i else t.detach() for j, t in enumerate(leaf)] for s in (step, -step)]
        lo = [(layer64(m[0], idx, *m[1:]) * go.double()).sum() for m in moved]
        slope = float((lo[0] - lo[1]) / (2 * step))
        mine = float((got.double() * d).sum())
        assert abs(slope - mine) < 4 * 2.0 ** -8 * float(got.double().norm()) * float(d.norm()), (i, slope, mine)


def test_serving_step_fp8(ep):
    T, H, I, E, K, A = 130, 512, 256, 8, 2, 128
    g = torch.Generator().manual_seed(1)
    idx = W.route_uniform_distinct(T, E, K, g).to(DEV)
    x, w = torch.randn(T, H, generator=g).bfloat16().to(DEV), torch.rand(T, K, generator=g).to(DEV) + 0.1
    q = lambda *s: (torch.randn(*s, generator=g) * 104).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    u = lambda std, *s: (torch.rand(*s, generator=g) * 0.7 + 0.7).mul(std / 104).to(DEV)
    w13, s13, w2, s2 = q(E, 2 * I, H), u(H ** -0.5, E, 2 * I // 128, H // 128), q(E, H, I), u(I ** -0.5, E, H // 128, I // 128)
    h, _, d = ep.ep_layout_dispatch(idx, x, E, expert_alignment=A, topk_weights=w, fp8=True)
    y = ep.ep_expert_ffn(h, d["recv_x"], w13, w2, recv_x_scales=d["recv_x_scales"], w13_scales=s13, w2_scales=s2)
    # the shared expert's down projection, with an adapter for some of the requests, joins as bias
    ids = torch.randint(-1, 3, (T, 1), generator=g).to(DEV)
    ha, _ = ep.ep_get_layout(ids, 3)
    a, b = torch.randn(3, 16, H, generator=g).mul(H ** -0.5).bfloat16().to(DEV), torch.randn(3, H, 16, generator=g).mul(0.25).bfloat16().to(DEV)
    shared = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    bias = ep.ep_adapter(ha, x, a, b, base=shared)
    out = ep.ep_combine(h, y, w, bias=bias)

    wide = lambda qq, ss: torch.stack([R.widen(qq[e], ss[e], 128) for e in range(E)])
    ref = layer64(x.double(), idx, w.double(), wide(w13, s13), wide(w2, s2)) + shared.double()
    for i in range(3):
        t = (ids.view(-1) == i).nonzero().view(-1)
        ref[t] += x[t].double() @ a[i].double().t() @ b[i].double().t()
    # the rows' e4m3 rounding is 2^-4 of an element at most, unbiased, in a sum of H products; the rest is bf16
    off = float((out.double() - ref).norm() / ref.norm())
    assert off < 2.0 ** -4, off
