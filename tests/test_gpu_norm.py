"""The combine with the norms around a block, and its gradient, against their definition in 64 bits: every part present and
absent, rows of one to four chunks a thread, tokens without entries, padding rows full of NaN, canaries behind every output."""
import pytest
import torch

import expert_reference as R
import harness as Hn
import norm_reference as N
import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


def table(T, E, K, how, seed):
    g = torch.Generator().manual_seed(seed)
    idx = W.route_uniform_distinct(T, E, K, g) if T else torch.empty(0, K, dtype=torch.int64)
    if how == "holes":
        idx[torch.rand(idx.shape, generator=g) < 0.3] = -1
        if T > 3:
            idx[1, 0], idx[2, 0] = E + 5, -9
            idx[3] = -1
    elif how == "none":
        idx[:] = -1
    return idx


CASES = [
    # T, H, E, ranks, rank, K, A, routing; K = 0: a block's output without a handle
    (1, 8, 4, 1, 0, 1, 1, "uniform"),
    (1, 7168, 64, 1, 0, 8, 1, "uniform"),
    (5, 72, 4, 1, 0, 3, 16, "holes"),
    (33, 264, 6, 2, 1, 4, 8, "holes"),
    (7, 512, 8, 1, 0, 2, 1, "none"),
    (64, 4096, 8, 1, 0, 5, 16, "holes"),
    (9, 4104, 32, 1, 0, 15, 1, "uniform"),
    (700, 136, 40, 4, 2, 32, 1, "holes"),
    (6, 8200, 8, 1, 0, 7, 1, "holes"),
    (3, 32768, 8, 1, 0, 2, 128, "uniform"),
    (1, 40, 0, 1, 0, 0, 1, ""),
    (1100, 2112, 0, 1, 0, 0, 1, ""),
    (4, 16392, 0, 1, 0, 0, 1, ""),
]
PARTS = [
    # bias, residual, post, gate, pre, vectors
    (True, True, True, "channel", True, torch.float32),
    (False, True, True, "token", True, torch.bfloat16),
    (False, False, False, "none", True, torch.float32),
    (True, True, False, "channel", False, torch.bfloat16),
    (False, True, True, "none", False, torch.float32),
    (True, False, True, "token", True, torch.float32),
]
ID = lambda c: "T%d_H%d_E%d_R%d_K%d_A%d_%s" % (c[0], c[1], c[2], c[3], c[5], c[6], c[7])
PID = lambda p: "".join(n[0] if v not in (False, "none") else "-" for n, v in zip(("bias", "residual", "post", "gate", "xpre"), p)) + (
    "_t" if p[3] == "token" else "") + ("_16" if p[5] == torch.bfloat16 else "")


def make(ep, case, parts, seed=5):
    T, H, E, ranks, rank, K, A, how = case
    bias, residual, post, gate, pre, kind = parts
    g = torch.Generator(device=DEV).manual_seed(seed + T * 131 + H)
    n = lambda *s, std=1.0, mean=0.0, dtype=torch.bfloat16: (torch.randn(*s, generator=g, device=DEV) * std + mean).to(dtype)
    d = dict(h=None, w=None, slot=None)
    if K:
        idx = table(T, E, K, how, seed)
        El = E // ranks
        d["slot"], start, count = R.segments(idx, E, rank * El, El, A)
        d["slot"] = d["slot"].to(DEV)
        d["h"], _ = ep.ep_get_layout(idx.to(DEV), E, ranks, rank, A)
        d["y"] = n(d["h"].recv_capacity + 2, H)
        valid = torch.zeros(d["y"].shape[0], dtype=torch.bool)
        for s, c in zip(start, count):
            valid[s:s + c] = True
        d["y"][~valid.to(DEV)] = float("nan")
        d["w"] = torch.rand(T, K, generator=g, device=DEV) + 0.1
    else:
        d["y"] = n(T, H)
    d["bias"] = n(T, H, std=0.3) if bias else None
    d["around"] = dict(residual=n(T, H, std=2.0) if residual else None, post_weight=n(H, std=0.2, mean=1.0, dtype=kind) if post else None,
                       gate=None if gate == "none" else n(T, H, std=0.5) if gate == "token" else n(H, std=0.3, mean=0.4, dtype=kind),
                       residual_scale=0.7 if residual else 1.0, pre_weight=n(H, std=0.2, mean=1.0, dtype=kind) if pre else None, eps=EPS)
    return d, n


def reference(d):
    a = d["around"]
    if d["slot"] is None:
        f = d["y"].double() + (0 if d["bias"] is None else d["bias"].double())
        ef = N.U * f.abs() if d["bias"] is not None else torch.zeros_like(f)
    else:
        f, ef = N.combined(d["slot"], d["y"], d["w"], d["bias"])
    o = N.around(f, ef, a["residual"], a["post_weight"], a["gate"], a["residual_scale"], a["pre_weight"], a["eps"])
    return f, ef, o


@pytest.mark.parametrize("parts", PARTS, ids=PID)
@pytest.mark.parametrize("case", CASES, ids=ID)
def test_forward(ep, case, parts):
    print("[norm] %s %s" % (ID(case), PID(parts)), flush=True)
    d, _ = make(ep, case, parts)
    T, H = case[0], case[1]
    out, g1 = Hn.guarded_tensor((T, H), torch.bfloat16, DEV, "out")
    kept, g2 = Hn.guarded_tensor((T, H), torch.float32, DEV, "kept")
    normed, g3 = Hn.guarded_tensor((T, H), torch.bfloat16, DEV, "normed") if parts[4] else (None, None)
    got = ep.ep_combine_norm(d["h"], d["y"], d["w"], bias=d["bias"], out=out, kept=kept, normed=normed, **d["around"])
    torch.cuda.synchronize()
    assert got[0] is out and got[1] is normed
    f, ef, o = reference(d)
    R.assert_within(kept, f, ef + N.TINY, "kept")
    R.assert_within(out, o["out"], o["eout"], "out")
    if normed is not None:
        R.assert_within(normed, o["n"], o["en"], "normed")
    for g in (g1, g2, g3):
        if g is not None:
            Hn.assert_guards(g)
    # each output alone, and out in place of the residual: the same bits
    bits = lambda t: t.view(torch.int16)
    if normed is not None:
        none, n2 = ep.ep_combine_norm(d["h"], d["y"], d["w"], bias=d["bias"], need_out=False, **d["around"])
        assert none is None and torch.equal(bits(n2), bits(normed))
    if parts[1]:
        ref, _ = ep.ep_combine_norm(d["h"], d["y"], d["w"], bias=d["bias"], out=d["around"]["residual"], **d["around"])
        assert ref is d["around"]["residual"] and torch.equal(bits(ref), bits(out))


@pytest.mark.parametrize("parts", PARTS, ids=PID)
@pytest.mark.parametrize("case", CASES, ids=ID)
def test_backward(ep, case, parts):
    print("[norm grad] %s %s" % (ID(case), PID(parts)), flush=True)
    d, n = make(ep, case, parts)
    T, H, K = case[0], case[1], case[5]
    a = d["around"]
    if K or parts[0]:
        f = torch.empty(T, H, device=DEV)
        ep.ep_combine_norm(d["h"], d["y"], d["w"], bias=d["bias"], kept=f, **a)
    else:
        f = d["y"]
    do, dn = n(T, H), n(T, H) if parts[4] else None
    if parts[4] and not parts[1]:
        do = None
    o = {"grad_f": ((T, H), torch.bfloat16)}
    if parts[1]:
        o["grad_residual"] = ((T, H), torch.bfloat16)
    if parts[2]:
        o["grad_post"] = ((H,), torch.float32)
    if dn is not None:
        o["grad_pre"] = ((H,), torch.float32)
    if parts[3] != "none":
        o["grad_gate"] = ((H,), torch.float32) if parts[3] == "channel" else ((T, H), torch.bfloat16)
    made = {k: Hn.guarded_tensor(s, t, DEV, k) for k, (s, t) in o.items()}
    ws, gw = Hn.guarded_tensor((ep.ep_combine_norm_workspace_bytes(T, H),), torch.uint8, DEV, "ws")
    got = ep.ep_combine_norm_backward(do, dn, f, workspace=ws, **{k: v[0] for k, v in made.items()}, **a)
    torch.cuda.synchronize()
    assert {k for k, v in got.items() if v is not None} == set(o)
    want = N.gradients(f, a["residual"], a["post_weight"], a["gate"], a["residual_scale"], a["pre_weight"], a["eps"], do, dn)
    assert set(want) == set(o)
    for k, (v, e) in want.items():
        R.assert_within(got[k], v, e, k)
        Hn.assert_guards(made[k][1])
    Hn.assert_guards(gw)
    # rows alone and vectors alone: the same bits
    bits = lambda t: t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)
    for need in (dict(need_rows=False), dict(need_vectors=False)):
        if need == dict(need_rows=False) and not any(t == torch.float32 for _, t in o.values()):
            continue
        for k, v in ep.ep_combine_norm_backward(do, dn, f, **need, **a).items():
            if v is not None:
                assert torch.equal(bits(v), bits(got[k])), (k, need)


def test_no_tokens(ep):
    y = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    out, normed = ep.ep_combine_norm(None, y, post_weight=w, pre_weight=w)
    assert out.shape == normed.shape == (0, 64)
    got = ep.ep_combine_norm_backward(y, y, y, post_weight=w, pre_weight=w, grad_post=torch.full((64,), 7.0, device=DEV))
    torch.cuda.synchronize()
    assert not got["grad_post"].any() and not got["grad_pre"].any()


def test_inf_and_nan_stay_in_their_rows(ep):
    case, parts = (40, 520, 6, 1, 0, 2, 1, "uniform"), PARTS[0]
    d, n = make(ep, case, parts)
    clean = ep.ep_combine_norm(d["h"], d["y"], d["w"], bias=d["bias"], **d["around"])
    d["y"][d["slot"][3, 1], 100], d["y"][d["slot"][17, 0], 519] = float("inf"), float("nan")
    got = ep.ep_combine_norm(d["h"], d["y"], d["w"], bias=d["bias"], **d["around"])
    others = torch.ones(40, dtype=torch.bool, device=DEV)
    others[[3, 17]] = False
    for a, b in zip(got, clean):
        assert torch.equal(a.view(torch.int16)[others], b.view(torch.int16)[others])
        assert a[17].isnan().all() and a[3].isnan().any()


def test_large_and_small_values(ep):
    """Rows of 1e15 and of 1e-20 with an eps below their squares' mean: the norms are the same as at 1."""
    y = torch.randn(3, 256, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)).bfloat16()
    y[1] = (y[0].float() * 2.0 ** 50).bfloat16()
    y[2] = (y[0].float() * 2.0 ** -50).bfloat16()
    one = torch.ones(256, device=DEV)
    _, normed = ep.ep_combine_norm(None, y, pre_weight=one, eps=1e-37)
    assert torch.equal(normed[0], normed[1]) and torch.equal(normed[0], normed[2])
    _, zero = ep.ep_combine_norm(None, torch.zeros_like(y), pre_weight=one)
    assert not zero.any()


@pytest.mark.parametrize("case", [(3, 1024, 6, 1, 0, 2, 1, "holes"), (600, 264, 6, 1, 0, 2, 1, "uniform")], ids=ID)
def test_graph_replay_and_streams(ep, case):
    """Forward and backward captured on a side stream, replayed with eager work between; every replay equals the eager result on
    the inputs of the moment."""
    d, n = make(ep, case, PARTS[0])
    T, H, a = case[0], case[1], d["around"]
    do, dn = n(T, H), n(T, H)
    ws = torch.empty(ep.ep_combine_norm_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    new = lambda: dict(out=torch.zeros(T, H, dtype=torch.bfloat16, device=DEV), normed=torch.zeros(T, H, dtype=torch.bfloat16, device=DEV),
                       kept=torch.zeros(T, H, device=DEV), grad_f=torch.zeros(T, H, dtype=torch.bfloat16, device=DEV),
                       grad_residual=torch.zeros(T, H, dtype=torch.bfloat16, device=DEV), grad_post=torch.zeros(H, device=DEV),
                       grad_pre=torch.zeros(H, device=DEV), grad_gate=torch.zeros(H, device=DEV))

    def run(o, ws, stream=None):
        fwd = {k: o[k] for k in ("out", "normed", "kept")}
        ep.ep_combine_norm(d["h"], d["y"], d["w"], bias=d["bias"], stream=stream, **fwd, **a)
        ep.ep_combine_norm_backward(do, dn, o["kept"], workspace=ws, stream=stream, **{k: v for k, v in o.items() if k not in fwd}, **a)

    o = new()
    run(o, ws)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(o, ws, stream=side)
    for i in range(3):
        d["y"].normal_()
        do.normal_()
        for t in o.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = new()
        run(ref, torch.empty_like(ws))
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k], ref[k]), "%s, replay %d" % (k, i)


@pytest.mark.parametrize("T,H,K", [(40, 72, 2), (30, 264, 0)])
def test_against_differences(ep, T, H, K):
    """The loss moves by the gradients' component along a direction (the loss in 64 bits, so the quotient is good to O(step^2))."""
    d, n = make(ep, (T, H, 5, 1, 0, K, 1, "uniform"), PARTS[0] if K else (False,) + PARTS[0][1:])
    a = d["around"]
    do, dn = n(T, H), n(T, H)
    f = d["y"]
    if K:
        f = torch.empty(T, H, device=DEV)
        ep.ep_combine_norm(d["h"], d["y"], d["w"], bias=d["bias"], kept=f, **a)
    got = ep.ep_combine_norm_backward(do, dn, f, **a)
    leaf = dict(grad_f=f, grad_residual=a["residual"], grad_post=a["post_weight"], grad_pre=a["pre_weight"], grad_gate=a["gate"])
    leaf = {k: v.double() for k, v in leaf.items()}

    def loss(v):
        z = torch.zeros_like(v["grad_f"])
        o = N.around(v["grad_f"], z, v["grad_residual"], v["grad_post"], v["grad_gate"], a["residual_scale"], v["grad_pre"], EPS)
        return float((o["r"] * do.double()).sum() + (o["n"] * dn.double()).sum())

    for k in leaf:
        g = got[k].double()
        way = torch.randn(g.shape, dtype=torch.float64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(9))
        way = way / way.norm() + g / g.norm()
        step = 1e-4
        up, down = ({**leaf, k: leaf[k] + s * way} for s in (step, -step))
        slope, mine = (loss(up) - loss(down)) / (2 * step), float((g * way).sum())
        # one rounding of the gradient to bf16, and the quotient's own error
        assert abs(slope - mine) < 2 * 2.0 ** -8 * float(g.norm()) * float(way.norm()), (k, slope, mine)
