"""A whole layer for a few tokens against its definition in 64 bits: every format of weights, one to 128 tokens, one to 1024
entries, ranks, duplicates, entries that add nothing, and the same layer by way of layout, dispatch, experts and combine."""
import pytest
import torch

import expert_reference as R
import harness as Hn
import w4_reference as Q
from test_gpu_expert_ffn import table

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = ["bf16", "e4m3", "int4_32", "int4_64", "int4_128", "e2m1_32", "e2m1_64", "e2m1_128"]


@pytest.fixture(scope="module")
def ep():
    import combine_get_dispatch_03_amd as ep
    return ep


SHAPES = [
    # T, H, I, E, ranks, rank, K, routing; H and I in units of the format (bf16: 8)
    (1, 1, 1, 1, 1, 0, 1, "uniform"),
    (1, 6, 3, 16, 1, 0, 8, "uniform"),
    (2, 5, 9, 4, 2, 1, 3, "uniform"),
    (16, 2, 5, 8, 2, 0, 1, "holes"),
    (4, 20, 13, 9, 1, 0, 4, "holes"),
    (2, 3, 17, 1, 1, 0, 5, "one"),
    (8, 3, 2, 300, 1, 0, 8, "uniform"),
    (13, 9, 5, 6, 1, 0, 4, "holes"),
    (17, 4, 7, 32, 4, 3, 8, "holes"),
    (64, 2, 3, 8, 1, 0, 1, "zipf"),
    (70, 7, 4, 3, 1, 0, 2, "one"),
    (33, 3, 3, 1024, 1, 0, 31, "uniform"),
    (128, 5, 6, 64, 1, 0, 8, "holes"),
    (128, 9, 4, 5, 1, 0, 5, "zipf"),
    (128, 3, 5, 2, 1, 0, 8, "one"),
    (30, 4, 4, 8, 2, 0, 2, "none"),
]
IDS = ["T%d_H%d_I%d_E%d_R%d_K%d_%s" % (s[0], s[1], s[2], s[3], s[4], s[6], s[7]) for s in SHAPES]


def weights(ep, fmt, g, El, H, I):
    """What the call takes (w13, w2, scales) and the experts in 64 bits, made when asked for."""
    if fmt == "bf16":
        n = lambda *s: (torch.randn(*s, generator=g, device=DEV) * s[-1] ** -0.5).bfloat16()
        w13, w2 = n(El, 2 * I, H), n(El, H, I)
        return (w13, w2, None, None), lambda e: (w13[e].double(), w2[e].double())
    if fmt == "e4m3":
        q = lambda *s: (torch.randn(*s, generator=g, device=DEV) * 104).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        u = lambda std, *s: torch.rand(*s, generator=g, device=DEV).mul(0.7).add(0.7).mul(std / 104)
        w13, w2 = q(El, 2 * I, H), q(El, H, I)
        s13, s2 = u(H ** -0.5, El, 2 * I // 128, H // 128), u(I ** -0.5, El, H // 128, I // 128)
        return (w13, w2, s13, s2), lambda e: (R.widen(w13[e], s13[e], 128), R.widen(w2[e], s2[e], 128))
    kind, group = fmt.split("_")
    w13, s13 = Q.random_w4(g, kind, int(group), El, 2 * I, H, DEV, H ** -0.5)
    w2, s2 = Q.random_w4(g, kind, int(group), El, H, I, DEV, I ** -0.5)
    return (ep.ep_w4_pack(w13, s13, kind), ep.ep_w4_pack(w2, s2, kind), None, None), lambda e: (
        Q.widen(w13[e], s13[e], kind), Q.widen(w2[e], s2[e], kind))


def setup(ep, shape, fmt, seed=7):
    T, H, I, E, ranks, rank, K, how = shape
    unit = 8 if fmt == "bf16" else 128 if fmt == "e4m3" else int(fmt.split("_")[1])
    if fmt == "bf16":
        H, I = H * 5, I * 5
    H, I = H * unit, I * unit
    if how == "uniform" and K > E:
        how = "one"
    idx = table(T, E, K, how, seed) if K <= E else torch.full((T, K), E - 1, dtype=torch.int64)
    El = E // ranks
    g = torch.Generator(device=DEV).manual_seed(seed + T)
    call, expert = weights(ep, fmt, g, El, H, I)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    w = torch.rand(T, K, generator=g, device=DEV) + 0.1
    bias = (torch.randn(T, H, generator=g, device=DEV) * 0.3).bfloat16()
    used = sorted(set((idx - rank * El).view(-1).tolist()) & set(range(El)))
    return idx.to(DEV), x, w, bias, call, {e: expert(e) for e in used}, dict(H=H, I=I, El=El, lo=rank * El, ranks=ranks, rank=rank)


def run(ep, idx, x, w, call, m, **kw):
    return ep.ep_moe_few(x, idx, w, call[0], call[1], w13_scales=call[2], w2_scales=call[3], num_ranks=m["ranks"], rank=m["rank"], **kw)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_values(ep, shape, fmt):
    print("[few] %s %s" % (shape, fmt), flush=True)
    T, K = shape[0], shape[6]
    idx, x, w, bias, call, experts, m = setup(ep, shape, fmt)
    out, go = Hn.guarded_tensor((T, m["H"]), torch.bfloat16, DEV, "out")
    ws, gw = Hn.guarded_tensor((ep.ep_moe_few_workspace_bytes(T, K, m["I"]),), torch.uint8, DEV, "ws")
    got = run(ep, idx, x, w, call, m, bias=bias, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert got is out
    want, bound = Q.layer(x, idx, w, bias, m["lo"], experts, K)
    R.assert_within(out, want, bound, "out")
    Hn.assert_guards(go)
    Hn.assert_guards(gw)
    # without weights and bias, and again with the bias in out's place
    plain = run(ep, idx, x, None, call, m)
    want, bound = Q.layer(x, idx, None, None, m["lo"], experts, K)
    R.assert_within(plain, want, bound, "out without weights")
    again = run(ep, idx, x, w, call, m, bias=bias, out=bias)
    assert again is bias and torch.equal(bias.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("fmt", ["bf16", "int4_64"])
def test_same_layer_in_steps(ep, fmt):
    """Layout, dispatch, experts and combine give the same layer but for the rounding of the experts' outputs."""
    T, K, E = 96, 4, 12
    idx, x, w, bias, call, experts, m = setup(ep, (T, 4, 6, E, 1, 0, K, "uniform"), fmt)
    got = run(ep, idx, x, w, call, m, bias=bias)
    h, _ = ep.ep_get_layout(idx, E, expert_alignment=16)
    rows = ep.ep_dispatch(h, x, w, fp8=False)["recv_x"]
    y = ep.ep_expert_ffn(h, rows, call[0], call[1]) if fmt == "bf16" else ep.ep_expert_ffn_w4(h, rows, call[0], call[1])
    steps = ep.ep_combine(h, y, w, bias=bias)
    off = float((got.double() - steps.double()).norm() / steps.double().norm())
    assert off < 2 * 2.0 ** -8, off


@pytest.mark.parametrize("T", [4, 6, 30])      # each entry by itself, in one wave's registers, through LDS
def test_invalid_entries_add_nothing(ep, T):
    shape = (T, 3, 2, 8, 2, 1, 3, "uniform")
    idx, x, w, bias, call, experts, m = setup(ep, shape, "bf16")
    idx[0] = torch.tensor([-1, -2 ** 63, 2 ** 63 - 1])
    idx[1] = torch.tensor([0, 3, 8])             # the other rank's, and past the last expert
    idx[2] = torch.tensor([4, 4, 4])             # one expert three times
    w[0], w[1] = float("nan"), float("inf")      # weights of entries that add nothing
    out = run(ep, idx, x, w, call, m, bias=bias)
    assert torch.equal(out[:2], bias[:2])
    experts = {e: (call[0][e].double(), call[1][e].double()) for e in range(4)}
    want, bound = Q.layer(x[2:], idx[2:], w[2:], bias[2:], 4, experts, 3)
    R.assert_within(out[2:], want, bound, "out")


def test_no_tokens(ep):
    idx, x, w, bias, call, experts, m = setup(ep, (2, 3, 2, 4, 1, 0, 2, "uniform"), "bf16")
    assert run(ep, idx[:0], x[:0], w[:0], call, m).shape == (0, m["H"])


def test_nan_stays_with_its_token(ep):
    idx, x, w, bias, call, experts, m = setup(ep, (40, 6, 4, 4, 1, 0, 2, "uniform"), "e2m1_32")
    clean = run(ep, idx, x, w, call, m)
    x[5, 3] = float("nan")
    x[17, 0] = float("inf")
    got = run(ep, idx, x, w, call, m)
    others = torch.ones(40, dtype=torch.bool, device=DEV)
    others[[5, 17]] = False
    assert torch.equal(got.view(torch.int16)[others], clean.view(torch.int16)[others])
    assert got[5].isnan().all() and not got[17].isfinite().any()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4_128"])
@pytest.mark.parametrize("T", [1, 40])
def test_graph_replay_and_streams(ep, T, fmt):
    """Captured on a side stream and replayed with new tokens and new routing, eager work between."""
    idx, x, w, bias, call, experts, m = setup(ep, (T, 4, 3, 16, 1, 0, 8, "uniform"), fmt)
    out = torch.empty_like(x)
    ws = torch.empty(ep.ep_moe_few_workspace_bytes(T, 8, m["I"]), dtype=torch.uint8, device=DEV)
    run(ep, idx, x, w, call, m, bias=bias, out=out, workspace=ws)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(ep, idx, x, w, call, m, bias=bias, out=out, workspace=ws, stream=side)
    for i in range(3):
        x.normal_()
        idx.copy_(table(T, 16, 8, "holes" if i == 1 else "uniform", 50 + i))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run(ep, idx, x, w, call, m, bias=bias)), i
