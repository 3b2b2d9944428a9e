"""The experts' gated feed-forward block and its gradients against their definition in 64 bits, over the sizes, masks and
formats where a ragged product can go wrong, with canaries in every row that no call may write."""
import pytest
import torch

import expert_reference as R
import harness as Hn
import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


def table(T, E, K, how, seed):
    """A routing table: distinct uniform experts with a few unused and invalid entries, or one of the extremes."""
    g = torch.Generator().manual_seed(seed)
    idx = W.route_uniform_distinct(T, E, K, g) if T else torch.empty(0, K, dtype=torch.int64)
    if how == "holes":
        idx[torch.rand(idx.shape, generator=g) < 0.3] = -1
        if T > 3:
            idx[1, 0], idx[2, 0] = E + 5, -9
            idx[3] = -1
    elif how == "one":          # every entry on one expert (the same index several times in a row)
        idx[:] = E - 1
    elif how == "none":
        idx[:] = -1
    elif how == "zipf":
        idx = W.route_zipf(T, E, K, 1.1, g)
    return idx


def rows_and_weights(cap, H, I, El, fmt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std
    if fmt == "bf16":
        return dict(x=n(cap, H).bfloat16(), w13=n(El, 2 * I, H, std=H ** -0.5).bfloat16(),
                    w2=n(El, H, I, std=I ** -0.5).bfloat16(), xs=None, s13=None, s2=None)
    q = lambda *s: (n(*s) * 104).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    u = lambda std, *s: torch.rand(*s, generator=g, device=DEV).mul(0.7).add(0.7).mul(std / 104)
    return dict(x=q(cap, H), w13=q(El, 2 * I, H), w2=q(El, H, I), xs=u(1.0, cap, H // 128),
                s13=u(H ** -0.5, El, 2 * I // 128, H // 128), s2=u(I ** -0.5, El, H // 128, I // 128))


def poison(t, valid):
    """Rows that are not valid rows hold NaN (bf16: quiet NaN; e4m3: its NaN code; fp32 scales and saved values: NaN)."""
    if t is None:
        return
    if t.dtype == torch.uint8:
        t[~valid] = 0x7F
    else:
        t[~valid] = float("nan")


SHAPES = [
    # T, H, I, E, ranks, rank, K, A, routing
    (1, 256, 128, 8, 1, 0, 2, 1, "uniform"),
    (1, 8, 8, 1, 1, 0, 1, 1, "uniform"),
    (5, 72, 136, 4, 1, 0, 3, 16, "holes"),
    (33, 264, 88, 6, 2, 1, 4, 8, "holes"),
    (64, 128, 128, 300, 1, 0, 4, 1, "uniform"),
    (128, 256, 512, 8, 1, 0, 2, 16, "uniform"),
    (200, 520, 328, 3, 1, 0, 1, 128, "zipf"),
    (257, 320, 200, 5, 1, 0, 2, 1, "one"),
    (40, 256, 128, 4, 1, 0, 2, 16, "none"),
    (150, 264, 136, 32, 1, 0, 2, 16, "one"),       # few rows by the average, 300 on one expert
    (100, 640, 384, 8, 1, 0, 2, 1, "zipf"),
    (700, 512, 264, 4, 1, 0, 3, 1, "zipf"),
    (1000, 1032, 520, 20, 4, 2, 8, 128, "holes"),
    (2100, 256, 384, 4, 1, 0, 4, 128, "zipf"),
]
IDS = ["T%d_H%d_I%d_E%d_R%d_K%d_A%d_%s" % (s[0], s[1], s[2], s[3], s[4], s[6], s[7], s[8]) for s in SHAPES]


def setup(ep, shape, fmt, seed=3, extra_rows=3):
    T, H, I, E, ranks, rank, K, A, how = shape
    if fmt == "fp8":
        H, I = -(-H // 128) * 128, -(-I // 128) * 128
    idx = table(T, E, K, how, seed)
    El = E // ranks
    slot, start, count = R.segments(idx, E, rank * El, El, A)
    h, _ = ep.ep_get_layout(idx.to(DEV), E, ranks, rank, A)
    cap = h.recv_capacity + extra_rows
    d = rows_and_weights(cap, H, I, El, fmt, seed)
    valid = torch.zeros(cap, dtype=torch.bool)
    for s, c in zip(start, count):
        valid[s:s + c] = True
    valid = valid.to(DEV)
    poison(d["x"], valid)
    poison(d["xs"], valid)
    return h, d, dict(H=H, I=I, El=El, cap=cap, start=start, count=count, valid=valid)


def expert_values(d, m, e):
    rows = slice(m["start"][e], m["start"][e] + m["count"][e])
    return (rows, R.widen(d["x"][rows], None if d["xs"] is None else d["xs"][rows], 1),
            R.widen(d["w13"][e], None if d["s13"] is None else d["s13"][e], 128),
            R.widen(d["w2"][e], None if d["s2"] is None else d["s2"][e], 128))


def untouched(t, valid):
    ref = torch.empty_like(t)
    Hn._canary_fill(ref, "y")
    v = torch.int32 if t.dtype == torch.float32 else torch.int16
    assert torch.equal(t.view(v)[~valid], ref.view(v)[~valid]), "a row that is no valid row was written"


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(ep, shape, fmt):
    print("[ffn] %s %s" % (shape, fmt), flush=True)
    h, d, m = setup(ep, shape, fmt)
    y, gy = Hn.guarded_tensor((m["cap"], m["H"]), torch.bfloat16, DEV, "y")
    pre = gp = None
    if fmt == "bf16":
        pre, gp = Hn.guarded_tensor((m["cap"], 2 * m["I"]), torch.float32, DEV, "pre")
    ws, gw = Hn.guarded_tensor((ep.ep_expert_ffn_workspace_bytes(h, m["H"], m["I"]),), torch.uint8, DEV, "ws")
    out = ep.ep_expert_ffn(h, d["x"], d["w13"], d["w2"], recv_x_scales=d["xs"], w13_scales=d["s13"], w2_scales=d["s2"],
                           y=y, pre=pre, workspace=ws)
    torch.cuda.synchronize()
    assert out is y
    for e in range(m["El"]):
        rows, x, w13, w2 = expert_values(d, m, e)
        f = R.ffn_expert(x, w13, w2)
        R.assert_within(y[rows], f["y"], f["ey"], "y of expert %d" % e)
        if pre is not None:
            R.assert_within(pre[rows], f["p"], f["ep"], "pre of expert %d" % e)
    untouched(y, m["valid"])
    if pre is not None:
        untouched(pre, m["valid"])
        Hn.assert_guards(gp)
    Hn.assert_guards(gy)
    Hn.assert_guards(gw)
    # the same call again, without pre and with its own outputs: the same bits
    again = ep.ep_expert_ffn(h, d["x"], d["w13"], d["w2"], recv_x_scales=d["xs"], w13_scales=d["s13"], w2_scales=d["s2"])
    assert torch.equal(again.view(torch.int16)[m["valid"]], y.view(torch.int16)[m["valid"]])


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(ep, shape):
    print("[ffn grad] %s" % (shape,), flush=True)
    h, d, m = setup(ep, shape, "bf16")
    H, I, El, cap = m["H"], m["I"], m["El"], m["cap"]
    pre = torch.full((cap, 2 * I), float("nan"), device=DEV)
    ep.ep_expert_ffn(h, d["x"], d["w13"], d["w2"], pre=pre)
    dy = torch.randn(cap, H, device=DEV, generator=torch.Generator(device=DEV).manual_seed(8)).bfloat16()
    poison(dy, m["valid"])
    dx, g1 = Hn.guarded_tensor((cap, H), torch.bfloat16, DEV, "dx")
    dw13, g2 = Hn.guarded_tensor((El, 2 * I, H), torch.bfloat16, DEV, "dw13")
    dw2, g3 = Hn.guarded_tensor((El, H, I), torch.bfloat16, DEV, "dw2")
    ws, g4 = Hn.guarded_tensor((ep.ep_expert_ffn_workspace_bytes(h, H, I, backward=True),), torch.uint8, DEV, "ws")
    ep.ep_expert_ffn_backward(h, dy, d["x"], pre, d["w13"], d["w2"], dx=dx, dw13=dw13, dw2=dw2, workspace=ws)
    torch.cuda.synchronize()
    for e in range(El):
        rows, x, w13, w2 = expert_values(d, m, e)
        f = R.ffn_expert_grads(x, w13, w2, dy[rows].double())
        R.assert_within(dx[rows], f["dx"], f["edx"], "dx of expert %d" % e)
        R.assert_within(dw13[e], f["dw13"], f["edw13"], "dw13 of expert %d" % e)
        R.assert_within(dw2[e], f["dw2"], f["edw2"], "dw2 of expert %d" % e)
        if m["count"][e] == 0:
            assert not dw13[e].any() and not dw2[e].any()
    untouched(dx, m["valid"])
    for g in (g1, g2, g3, g4):
        Hn.assert_guards(g)
    # each gradient on its own is the same, bit for bit
    for need in ("dx", "dw13", "dw2"):
        got = ep.ep_expert_ffn_backward(h, dy, d["x"], pre, d["w13"], d["w2"],
                                        **{"need_" + k: k == need for k in ("dx", "dw13", "dw2")})
        mine = dict(zip(("dx", "dw13", "dw2"), got))
        assert [k for k, v in mine.items() if v is not None] == [need]
        a, b = mine[need].view(torch.int16), dict(dx=dx, dw13=dw13, dw2=dw2)[need].view(torch.int16)
        assert torch.equal(a[m["valid"]], b[m["valid"]]) if need == "dx" else torch.equal(a, b)


def test_no_tokens(ep):
    idx = torch.empty((0, 2), dtype=torch.int64, device=DEV)
    h, _ = ep.ep_get_layout(idx, 4, expert_alignment=1)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    w13 = torch.randn(4, 32, 64, device=DEV).bfloat16()
    w2 = torch.randn(4, 64, 16, device=DEV).bfloat16()
    y = ep.ep_expert_ffn(h, x, w13, w2)
    assert y.shape == (0, 64)
    pre = torch.empty((0, 32), device=DEV)
    dw13 = torch.full_like(w13, 7.0)
    dx, dw13, dw2 = ep.ep_expert_ffn_backward(h, x, x, pre, w13, w2, dw13=dw13)
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and not dw13.any() and not dw2.any()


def test_extreme_values(ep):
    """Gates far out on both sides (silu saturates to the value itself and to zero), zero rows and zero weights: no NaN,
    and the definition's values."""
    T, H, I = 6, 64, 16
    idx = torch.zeros((T, 1), dtype=torch.int64)
    h, _ = ep.ep_get_layout(idx.to(DEV), 1)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = torch.tensor([1.0, -1.0, 100.0, -100.0, 0.0, 1e-3], dtype=torch.bfloat16)
    w13 = torch.zeros(1, 2 * I, H, dtype=torch.bfloat16, device=DEV)
    w13[0, :I, 0], w13[0, I:, 0] = 300.0, 2.0
    w2 = torch.zeros(1, H, I, dtype=torch.bfloat16, device=DEV)
    w2[0, :8] = 1.0
    pre = torch.empty(T, 2 * I, device=DEV)
    y = ep.ep_expert_ffn(h, x, w13, w2, pre=pre)
    f = R.ffn_expert_grads(x.double(), w13[0].double(), w2[0].double(), torch.ones(T, H, dtype=torch.float64, device=DEV))
    R.assert_within(y, f["y"], f["ey"], "y")
    dx, dw13, dw2 = ep.ep_expert_ffn_backward(h, torch.ones_like(x), x, pre, w13, w2)
    R.assert_within(dx, f["dx"], f["edx"], "dx")
    R.assert_within(dw13[0], f["dw13"], f["edw13"], "dw13")
    R.assert_within(dw2[0], f["dw2"], f["edw2"], "dw2")


def test_inf_and_nan_stay_in_their_rows(ep):
    """A row that holds an infinity or a NaN spoils its own output row and no other."""
    shape = (300, 256, 128, 3, 1, 0, 1, 16, "uniform")
    h, d, m = setup(ep, shape, "bf16")
    clean = ep.ep_expert_ffn(h, d["x"], d["w13"], d["w2"])
    rows = m["valid"].nonzero().view(-1)[[0, 5, 131]]
    d["x"][rows[0], 3], d["x"][rows[1], 0], d["x"][rows[2], 255] = float("nan"), float("inf"), float("-inf")
    got = ep.ep_expert_ffn(h, d["x"], d["w13"], d["w2"])
    others = m["valid"].clone()
    others[rows] = False
    assert torch.equal(got.view(torch.int16)[others], clean.view(torch.int16)[others])
    assert got[rows[0]].isnan().all()


@pytest.mark.parametrize("T", [3, 200, 1500])
def test_graph_replay_and_streams(ep, T):
    """Forward and backward captured on a side stream, replayed with eager work between the replays; every replay equals
    the eager result on the inputs of the moment."""
    shape = (T, 384, 264, 6, 1, 0, 2, 16, "zipf")
    h, d, m = setup(ep, shape, "bf16")
    H, I, cap = m["H"], m["I"], m["cap"]
    x, dy = d["x"], torch.randn(cap, H, device=DEV).bfloat16()
    ws = torch.empty(ep.ep_expert_ffn_workspace_bytes(h, H, I, backward=True), dtype=torch.uint8, device=DEV)
    o = dict(y=torch.zeros(cap, H, dtype=torch.bfloat16, device=DEV), pre=torch.zeros(cap, 2 * I, device=DEV),
             dx=torch.zeros(cap, H, dtype=torch.bfloat16, device=DEV), dw13=torch.empty_like(d["w13"]), dw2=torch.empty_like(d["w2"]))

    def run(o, ws, stream=None):
        ep.ep_expert_ffn(h, x, d["w13"], d["w2"], y=o["y"], pre=o["pre"], workspace=ws, stream=stream)
        ep.ep_expert_ffn_backward(h, dy, x, o["pre"], d["w13"], d["w2"], dx=o["dx"], dw13=o["dw13"], dw2=o["dw2"],
                                  workspace=ws, stream=stream)

    run(o, ws)      # attributes that a first call sets are set outside the capture
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(o, ws, stream=side)
    for i in range(3):
        x[m["valid"]] = torch.randn(int(m["valid"].sum()), H, device=DEV).bfloat16()
        for t in o.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = {k: torch.zeros_like(t) for k, t in o.items()}
        run(ref, torch.empty_like(ws))
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k], ref[k]), "%s, replay %d" % (k, i)
