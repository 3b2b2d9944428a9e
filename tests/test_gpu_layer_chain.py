"""Norms, 4-bit experts and the layer for a few tokens as they are used together: decoding through two layers, eagerly and in a
captured graph; a prefill of the same layers; and a training step of a layer with norms around its experts."""
import pytest
import torch

import expert_reference as R
import norm_reference as N
import w4_reference as Q
import workloads as W
from test_gpu_expert_chain import layer64

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


def make_layers(ep, gen, kind, group, count, H, I, E):
    layers = []
    for _ in range(count):
        w13, s13 = Q.random_w4(gen, kind, group, E, 2 * I, H, DEV, H ** -0.5)
        w2, s2 = Q.random_w4(gen, kind, group, E, H, I, DEV, I ** -0.5)
        vec = lambda mean: (torch.randn(H, generator=gen, device=DEV) * 0.2 + mean).bfloat16()
        layers.append(dict(w13=ep.ep_w4_pack(w13, s13, kind), w2=ep.ep_w4_pack(w2, s2, kind), post=vec(1.0), gate=vec(0.5), pre=vec(1.0),
                           wide=lambda e, a=(w13, s13, w2, s2): (Q.widen(a[0][e], a[1][e], kind), Q.widen(a[2][e], a[3][e], kind))))
    return layers


def inputs(gen, T, H, E, K, count):
    cpu = torch.Generator().manual_seed(T)
    idx = [W.route_uniform_distinct(T, E, K, cpu) for _ in range(count)]
    for i in idx:
        i[::5, K - 1] = -1
    w = [torch.rand(T, K, generator=gen, device=DEV) + 0.1 for _ in range(count)]
    return [i.to(DEV) for i in idx], w, torch.randn(T, H, generator=gen, device=DEV).bfloat16()


def around(l, residual):
    return dict(residual=residual, post_weight=l["post"], gate=l["gate"], pre_weight=l["pre"], residual_scale=0.9, eps=EPS)


def check_norm(l, f, ef, residual, out, normed, name):
    o = N.around(f, ef, residual, l["post"], l["gate"], 0.9, l["pre"], EPS)
    R.assert_within(out, o["out"], o["eout"], name + " out")
    R.assert_within(normed, o["n"], o["en"], name + " normed")


@pytest.mark.parametrize("kind,group", [("int4", 128), ("e2m1", 32)])
@pytest.mark.parametrize("T", [1, 7, 40])
def test_decoding(ep, T, kind, group):
    H, I, E, K, count = 256, 384, 8, 3, 2
    g = torch.Generator(device=DEV).manual_seed(T)
    layers = make_layers(ep, g, kind, group, count, H, I, E)
    idx, w, x = inputs(g, T, H, E, K, count)
    shared = [torch.randn(T, H, generator=g, device=DEV).bfloat16() for _ in range(count)]
    first = torch.ones(H, device=DEV).bfloat16()
    ws = torch.empty(ep.ep_moe_few_workspace_bytes(T, K, I), dtype=torch.uint8, device=DEV)     # one of all layers: they follow each other

    def step(s):
        s["stream"].copy_(s["x"])
        n = ep.ep_combine_norm(None, s["stream"], pre_weight=first, eps=EPS, need_out=False, normed=s["n"][0])
        for i, l in enumerate(layers):
            ep.ep_moe_few(s["n"][i], idx[i], w[i], l["w13"], l["w2"], bias=shared[i], out=s["y"][i], workspace=ws)
            ep.ep_combine_norm(None, s["y"][i], out=s["out"][i], normed=s["n"][i + 1],
                               **around(l, s["stream"] if i == 0 else s["out"][i - 1]))

    new = lambda: torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    s = dict(x=x, stream=new(), n=[new() for _ in range(count + 1)], y=[new() for _ in range(count)], out=[new() for _ in range(count)])
    step(s)
    torch.cuda.synchronize()
    residual = s["stream"]
    o = N.around(x.double(), torch.zeros(T, H, dtype=torch.float64, device=DEV), None, None, None, 1.0, first, EPS)
    R.assert_within(s["n"][0], o["n"], o["en"], "first norm")
    for i, l in enumerate(layers):
        used = sorted(set(idx[i].view(-1).tolist()) - {-1})
        want, bound = Q.layer(s["n"][i], idx[i], w[i], shared[i], 0, {e: l["wide"](e) for e in used}, K)
        R.assert_within(s["y"][i], want, bound, "experts of layer %d" % i)
        check_norm(l, s["y"][i].double(), torch.zeros_like(want), residual, s["out"][i], s["n"][i + 1], "layer %d" % i)
        residual = s["out"][i]

    # the step in a graph, replayed on other tokens with eager steps in between
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(s)
    eager = dict(x=None, stream=new(), n=[new() for _ in range(count + 1)], y=[new() for _ in range(count)], out=[new() for _ in range(count)])
    for i in range(4):
        s["x"].copy_(torch.randn(T, H, generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        eager["x"] = s["x"].clone()
        step(eager)
        torch.cuda.synchronize()
        for k in ("n", "y", "out"):
            for a, b in zip(s[k], eager[k]):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16)), "%s of replay %d" % (k, i)


@pytest.mark.parametrize("kind,group", [("int4", 64), ("e2m1", 128)])
@pytest.mark.parametrize("T,A", [(100, 1), (900, 16)])
def test_prefill(ep, T, A, kind, group):
    H, I, E, K, count = 384, 256, 6, 2, 2
    g = torch.Generator(device=DEV).manual_seed(T)
    layers = make_layers(ep, g, kind, group, count, H, I, E)
    idx, w, x = inputs(g, T, H, E, K, count)
    n, residual = x, torch.randn(T, H, generator=g, device=DEV).bfloat16()
    for i, l in enumerate(layers):
        slot, start, rows_of = R.segments(idx[i].cpu(), E, 0, E, A)
        h, _ = ep.ep_get_layout(idx[i], E, expert_alignment=A)
        rows = ep.ep_dispatch(h, n, w[i], fp8=False)["recv_x"]
        y = ep.ep_expert_ffn_w4(h, rows, l["w13"], l["w2"])
        r = dict(zip(("out", "normed"), ep.ep_combine_norm(h, y, w[i], **around(l, residual))))
        torch.cuda.synchronize()
        for e in range(E):
            at = slice(start[e], start[e] + rows_of[e])
            f = R.ffn_expert(rows[at].double(), *l["wide"](e))
            R.assert_within(y[at], f["y"], f["ey"], "layer %d, expert %d" % (i, e))
        f, ef = N.combined(slot.to(DEV), y, w[i], None)
        check_norm(l, f, ef, residual, r["out"], r["normed"], "layer %d" % i)
        if T <= 128:
            # the layer in two kernels is the same but for the rounding of the experts' outputs and of their sum: two roundings
            few = ep.ep_moe_few(n, idx[i], w[i], l["w13"], l["w2"])
            again = dict(zip(("out", "normed"), ep.ep_combine_norm(None, few, **around(l, residual))))
            for k in ("out", "normed"):
                off = float((again[k].double() - r[k].double()).norm() / r[k].double().norm())
                assert off < 3 * 2.0 ** -8, (k, off)
        n, residual = r["normed"], r["out"]


@pytest.mark.parametrize("T,H,I,E,K,A", [(96, 128, 64, 4, 2, 16), (301, 256, 136, 6, 3, 1)])
def test_training_step(ep, T, H, I, E, K, A):
    g = torch.Generator().manual_seed(T)
    idx = W.route_uniform_distinct(T, E, K, g)
    idx[::7, K - 1] = -1
    idx = idx.to(DEV)
    n = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).to(DEV)
    x, w = n(T, H).bfloat16(), torch.rand(T, K, generator=g).to(DEV) + 0.1
    w13, w2 = n(E, 2 * I, H, std=H ** -0.5).bfloat16(), n(E, H, I, std=I ** -0.5).bfloat16()
    residual, post, pre, gate = n(T, H).bfloat16(), n(H, std=0.2, mean=1.0), n(H, std=0.2, mean=1.0), n(H, std=0.3, mean=0.5)
    go, gn = n(T, H).bfloat16(), n(T, H).bfloat16()

    h, _ = ep.ep_get_layout(idx, E, expert_alignment=A)
    rows = ep.ep_dispatch(h, x, w, fp8=False)["recv_x"]
    before = torch.empty(rows.shape[0], 2 * I, device=DEV)
    y = ep.ep_expert_ffn(h, rows, w13, w2, pre=before)
    f = torch.empty(T, H, device=DEV)
    a = dict(residual=residual, post_weight=post, gate=gate, pre_weight=pre, residual_scale=0.8, eps=EPS)
    out_got, normed_got = ep.ep_combine_norm(h, y, w, kept=f, **a)
    d = ep.ep_combine_norm_backward(go, gn, f, **a)
    gy, gw = ep.ep_combine_backward(h, d["grad_f"], y, w)
    dxr, dw13, dw2 = ep.ep_expert_ffn_backward(h, gy, rows, before, w13, w2)
    got = [ep.ep_combine(h, dxr), gw, dw13, dw2, d["grad_residual"], d["grad_post"], d["grad_pre"], d["grad_gate"]]
    names = ["x", "w", "w13", "w2", "residual", "post", "pre", "gate"]

    def loss(x, w, w13, w2, residual, post, pre, gate):
        norm = lambda v: v * ((v * v).mean(1, keepdim=True) + EPS).rsqrt()
        out = 0.8 * residual + gate * (norm(layer64(x, idx, w, w13, w2)) * post)
        normed = norm(out) * pre
        return (out * go.double()).sum() + (normed * gn.double()).sum(), out, normed

    leaf = [t.double().requires_grad_() for t in (x, w, w13, w2, residual, post, pre, gate)]
    total, out, normed = loss(*leaf)
    want = list(torch.autograd.grad(total, leaf))
    want[1] = torch.where(idx >= 0, want[1], 0.0)
    # Roundings to bf16 on the longest way: h and y forward, then grad_f, the rows of the combine's gradient, dh, dp, the rows of dx and
    # dx, each at most 2^-8 of its value and unbiased: the norm of the difference stays under eight of them.  Forward there are
    # three (h, y, the result).
    for name, a, b, count in [("out", out_got, out.detach(), 3), ("normed", normed_got, normed.detach(), 3)] + [
            ("d" + k, a, b, 8) for k, a, b in zip(names, got, want)]:
        off = float((a.double() - b).norm() / b.norm())
        assert off < count * 2.0 ** -8, "%s is off by %.3g" % (name, off)
    # against differences of the loss in 64 bits, along directions in which it does move
    for i, name in enumerate(names):
        mine = got[i].double()
        way = torch.randn(leaf[i].shape, generator=g, dtype=torch.float64).to(DEV)
        way = way / way.norm() + mine / mine.norm()
        step = 1e-4
        moved = [float(loss(*[(t + s * way if j == i else t).detach() for j, t in enumerate(leaf)])[0]) for s in (step, -step)]
        slope, along = (moved[0] - moved[1]) / (2 * step), float((mine * way).sum())
        assert abs(slope - along) < 8 * 2.0 ** -8 * float(mine.norm()) * float(way.norm()), (name, slope, along)
