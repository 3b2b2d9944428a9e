"""The tiled kernels of the expert block where they can go wrong: a workgroup that hands over from one tile to the next, weights
marked as read once, sums of a single stage, more than 64 blocks of scales, NaN rows, rows gigabytes apart, graphs.

Every case states which kernels it means and asks the library's rule for them, so that a changed rule cannot move a case off
its kernels unnoticed."""
import pytest
import torch

import expert_reference as R
import ffn_rules as Rules
import test_gpu_expert_ffn as F
from test_gpu_expert_large import e4m3, spread, valid_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


def counts_of(shape, seed=3):
    T, H, I, E, ranks, rank, K, A, how = shape
    El = E // ranks
    return R.segments(F.table(T, E, K, how, seed), E, rank * El, El, A)[2]


# name: (shape (T, H, I, E, ranks, rank, K, A, routing), formats, path, products with more tiles than workgroups).  Sizes are
# multiples of 128, so that both formats take them as they are.
CASES = {
    # two full rounds of short tiles, every expert's weights read by one of them
    "one_short_tile_each": ((60, 1152, 2048, 32, 1, 0, 4, 1, "uniform"), ("bf16", "fp8"), ("tile once", "stream"), ("up",)),
    "one_short_tile_each_second_rank": ((64, 1152, 2048, 64, 2, 1, 8, 16, "holes"), ("bf16", "fp8"), ("tile once", "stream"), ("up",)),
    # uneven counts: hand-overs between tiles of different heights, experts and scales
    "uneven": ((700, 256, 4352, 16, 1, 0, 2, 1, "zipf"), ("bf16", "fp8"), ("tile", "tile"), ("up", "dp")),
    "uneven_wide_out": ((600, 4352, 256, 16, 1, 0, 2, 8, "zipf"), ("bf16", "fp8"), ("stream", "tile"), ("down", "dx")),
    "even": ((1200, 896, 2304, 16, 1, 0, 1, 128, "uniform"), ("bf16", "fp8"), ("tile", "tile"), ("up",)),
    # e4m3 sums of one real stage (the tiles pad to two and four): 128 terms
    "hidden_128": ((1200, 128, 4352, 8, 1, 0, 1, 1, "uniform"), ("bf16", "fp8"), ("tile", "tile"), ("up",)),
    "inter_128": ((1200, 8704, 128, 8, 1, 0, 1, 1, "uniform"), ("bf16", "fp8"), ("stream", "tile"), ("down",)),
    "inter_256": ((1200, 8704, 256, 8, 1, 0, 1, 1, "zipf"), ("bf16", "fp8"), ("stream", "tile"), ("down",)),
    # scale rows of more than 64 and of more than 192 blocks
    "hidden_8320": ((300, 8320, 1536, 4, 1, 0, 1, 1, "uniform"), ("fp8",), ("tile", "tile"), ()),
    "inter_8320": ((400, 256, 8320, 4, 1, 0, 1, 1, "uniform"), ("bf16", "fp8"), ("tile", "tile"), ("up",)),
    "hidden_24704": ((300, 24704, 2048, 2, 1, 0, 1, 1, "uniform"), ("fp8",), ("tile", "tile"), ()),
    "inter_24704": ((300, 256, 24704, 2, 1, 0, 1, 1, "uniform"), ("fp8",), ("tile", "tile"), ("up",)),
}
FORWARD = [(n, f) for n, c in CASES.items() for f in c[1]]
BACKWARD = [n for n, c in CASES.items() if "bf16" in c[1]]


def as_meant(name, fmt):
    (T, H, I, E, ranks, rank, K, A, how), _, path, many = CASES[name]
    assert Rules.path(T, K, E, ranks, H, I, fmt) == path
    n = Rules.tiles(counts_of(CASES[name][0]), H, I, fmt)
    for product in many:
        assert n[product] > 256 or (product in ("dp", "dx") and fmt == "fp8"), (product, n)


@pytest.mark.parametrize("name,fmt", FORWARD, ids=["%s-%s" % c for c in FORWARD])
def test_forward(ep, name, fmt):
    as_meant(name, fmt)
    F.test_forward(ep, CASES[name][0], fmt)


@pytest.mark.parametrize("name", BACKWARD)
def test_backward(ep, name):
    as_meant(name, "bf16")
    F.test_backward(ep, CASES[name][0])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_inf_and_nan_stay_in_their_rows(ep, fmt):
    """On tiles, with hand-overs: a row that holds an infinity or a NaN spoils its own output row and no other."""
    name = "uneven"
    as_meant(name, fmt)
    h, d, m = F.setup(ep, CASES[name][0], fmt)
    call = lambda: ep.ep_expert_ffn(h, d["x"], d["w13"], d["w2"], d["xs"], d["s13"], d["s2"])
    clean = call()
    rows = m["valid"].nonzero().view(-1)[[0, 5, 131, 700]]
    if fmt == "bf16":
        d["x"][rows[0], 3], d["x"][rows[1], 0] = float("nan"), float("inf")
        d["x"][rows[2], 255], d["x"][rows[3], 64] = float("-inf"), float("nan")
    else:
        d["x"][rows[0], 3] = 0x7F
        d["xs"][rows[1], 0], d["xs"][rows[2], 1], d["xs"][rows[3], 1] = float("inf"), float("nan"), float("-inf")
    got = call()
    others = m["valid"].clone()
    others[rows] = False
    assert torch.equal(got.view(torch.int16)[others], clean.view(torch.int16)[others])
    assert got[rows[0]].isnan().all() and not got[rows].isfinite().any()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_rows_far_apart(ep, fmt):
    """All products on tiles with rows gigabytes apart: the dense layout's results bit for bit, and those of the definition."""
    T, E, H, I, far = 400, 5, 8192 if fmt == "bf16" else 16384, 4160 if fmt == "bf16" else 1280, 65536
    assert Rules.path(T, 1, E, 1, H, I, fmt)[0].startswith("tile") and Rules.path(T, 1, E, 1, H, I, fmt)[1] == "tile"
    assert E * (far - 1) * 2 * I * (4 if fmt == "bf16" else 1) > 2 ** 32 or E * (far - 1) * H > 2 ** 32
    g = torch.Generator(device=DEV).manual_seed(15)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).bfloat16()
    idx = (torch.arange(T, device=DEV) * 7 % E).view(T, 1)
    x, dy, w13, w2 = n(T, H), n(T, H), n(E, 2 * I, H, std=H ** -0.5), n(E, H, I, std=I ** -0.5)
    xs, scales = None, {}
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
            results.append([ep.ep_expert_ffn(h, xa, w13, w2, spread(xs, rows, cap), **scales)[rows]])
        else:
            pre = torch.zeros(cap, 2 * I, device=DEV)
            got = [ep.ep_expert_ffn(h, xa, w13, w2, pre=pre)[rows], pre[rows]]
            dx, dw13, dw2 = ep.ep_expert_ffn_backward(h, spread(dy, rows, cap), xa, pre, w13, w2)
            results.append(got + [dx[rows], dw13, dw2])
            del pre, dx
        del xa
    for near, away in zip(*results):
        assert torch.isfinite(near.float()).all() and torch.equal(near, away)
    # one expert against the definition; spread() took the tensors' rows in the layout's order
    e, first = 2, int((idx < 2).sum())
    mine = slice(first, first + int((idx == e).sum()))
    x64 = R.widen(x[mine], None if xs is None else xs[mine], 1)
    w64 = [R.widen(w[e], scales[k][e] if scales else None, 128) for w, k in ((w13, "w13_scales"), (w2, "w2_scales"))]
    if fmt == "fp8":
        f = R.ffn_expert(x64, *w64)
        R.assert_within(results[1][0][mine], f["y"], f["ey"], "y")
    else:
        f = R.ffn_expert_grads(x64, *w64, dy[mine].double())
        for got, key in zip(results[1], ("y", "p", "dx", "dw13", "dw2")):
            R.assert_within(got[e] if key.startswith("dw") else got[mine], f[key], f["e" + key], key)


@pytest.mark.parametrize("name", ["uneven", "one_short_tile_each"])
def test_graph_replay(ep, name):
    """Tiles with hand-overs, captured on a side stream: every replay equals the eager result on the inputs of the moment."""
    as_meant(name, "bf16")
    h, d, m = F.setup(ep, CASES[name][0], "bf16")
    H, I, cap = m["H"], m["I"], m["cap"]
    x, dy = d["x"], torch.randn(cap, H, device=DEV).bfloat16()
    ws = torch.empty(ep.ep_expert_ffn_workspace_bytes(h, H, I, backward=True), dtype=torch.uint8, device=DEV)
    o = dict(y=torch.zeros(cap, H, dtype=torch.bfloat16, device=DEV), pre=torch.zeros(cap, 2 * I, device=DEV),
             dx=torch.zeros(cap, H, dtype=torch.bfloat16, device=DEV), dw13=torch.empty_like(d["w13"]), dw2=torch.empty_like(d["w2"]))

    def run(o, ws, stream=None):
        ep.ep_expert_ffn(h, x, d["w13"], d["w2"], y=o["y"], pre=o["pre"], workspace=ws, stream=stream)
        ep.ep_expert_ffn_backward(h, dy, x, o["pre"], d["w13"], d["w2"], dx=o["dx"], dw13=o["dw13"], dw2=o["dw2"],
                                  workspace=ws, stream=stream)

    run(o, ws)
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


@pytest.mark.parametrize("name", ["hidden_128", "inter_128"])
def test_infinite_block_scale(ep, name):
    """A weight block's scale that has overflowed gives infinities, as the definition does, and no NaN: also in sums of one stage,
    which the tiles pad with stages of zeros.  All values are positive, so no infinities meet with other signs."""
    as_meant(name, "fp8")
    h, d, m = F.setup(ep, CASES[name][0], "fp8")
    for k in ("x", "w13", "w2"):
        d[k].fill_(0x38)                             # 1.0
    call = lambda: ep.ep_expert_ffn(h, d["x"], d["w13"], d["w2"], d["xs"], d["s13"], d["s2"])
    clean = call()
    e, I = 3, m["I"]
    rows = slice(m["start"][e], m["start"][e] + m["count"][e])
    want = clean.clone()
    if name == "hidden_128":
        d["s13"][e, I // 128, 0] = float("inf")      # up projection, first 128 channels: u, h and every y of the expert
        want[rows] = float("inf")
    else:
        d["s2"][e, 5, 0] = float("inf")              # output channels 640 .. 767
        want[rows, 640:768] = float("inf")
    got = call()
    assert bool(clean[m["valid"]].isfinite().all())
    assert torch.equal(got[m["valid"]], want[m["valid"]])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [3, 70])
def test_largest_sizes(ep, T, fmt):
    """hidden and intermediate at their limits: one expert's w13 is 4 GiB in bf16.  Down projection streamed and on tiles."""
    shape = (T, 32768, 32768, 1, 1, 0, 1, 1, "uniform")
    assert Rules.path(T, 1, 1, 1, 32768, 32768, fmt) == (
        "tile" if (T, fmt) == (70, "fp8") else "tile once", "tile" if T == 70 else "stream")
    F.test_forward(ep, shape, fmt)
    if fmt == "bf16" and T == 70:
        F.test_backward(ep, shape)
    torch.cuda.empty_cache()
