"""The rest of a mixture-of-experts layer: what is measured, in plain torch and through the library.

Three operators beside the layout, the dispatch, the experts and the combine:

  w4     the experts' gated feed-forward block over dispatched rows with weights of four bits: w[n, k] = s[n, k / group] *
         v(code[n, k]), v(code) = code - 8 ("int4") or the e2m1 value of the code ("e2m1"), scales in bf16.
  few    the whole layer for a few tokens, from tokens and routing to tokens: out[t] = bias[t] + sum_k w[t,k] ffn_e(x[t]), with
         bf16, e4m3 (a scale per 128 x 128 block) or 4-bit weights.
  norm   the combine with the norms around a block: f = sum_k w[t,k] y[row] + bias;  a = f rsqrt(mean f^2 + eps) post;
         r = residual_scale residual + gate a;  n = r rsqrt(mean r^2 + eps) pre.  `norm_train` is its forward and backward pass.

Where `own` is false everything is computed from elementary torch operations in 32 bits; where it is true, by the
library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128     # channels per scale of the e4m3 weights
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ----------------------------------------------------------------------------------------------------------

def _w4(name, T, H, I, E, K, align, kind, group, routing="uniform", idle=0):
    return {"name": name, "op": "w4", "tokens": T, "hidden": H, "inter": I, "experts": E, "topk": K, "align": align,
            "fmt": kind, "group": group, "routing": routing, "idle": idle}


def _few(name, T, H, I, E, K, fmt, group, routing="uniform", idle=0, bias=False):
    return {"name": name, "op": "few", "tokens": T, "hidden": H, "inter": I, "experts": E, "topk": K, "align": 1, "fmt": fmt,
            "group": group, "routing": routing, "idle": idle, "bias": bias}


def _norm(name, op, T, H, E, K, align, gate, bias=False, idle=0, routing="uniform", vectors="fp32"):
    """K = 0: the block's output as it is (no combine)."""
    return {"name": name, "op": op, "tokens": T, "hidden": H, "experts": E, "topk": K, "align": align, "gate": gate,
            "bias": bias, "idle": idle, "routing": routing, "vectors": vectors}


def listed():
    return [
        # the repository's tiny workload with a block of twice its width: launches and latency are all there is
        _w4("w4_tiny_e2m1", 128, 256, 512, 8, 2, 16, "e2m1", 32),
        # a decode batch on a rank's 32 experts, about 32 rows each: every weight is read
        _w4("w4_decode_int4", 128, 7168, 2048, 32, 8, 128, "int4", 128),
        # a padded batch of odd sizes, experts that few or no rows reach
        _w4("w4_ragged_int4", 777, 2112, 1344, 20, 3, 1, "int4", 64, "zipf", 40),
        # the prefill batch over a rank's 32 experts, about 1024 rows each
        _w4("w4_prefill_e2m1", 4096, 7168, 2048, 32, 8, 128, "e2m1", 32),
        # four requests through the tiny workload's layer: launches and latency
        _few("few_tiny_bf16", 4, 256, 512, 8, 2, "bf16", 0),
        # one request against the decode workload's 256 experts
        _few("few_one_token_int4", 1, 7168, 2048, 256, 8, "int4", 128),
        # a small decode batch of that layer in the format its dispatch would use, with a shared expert's output
        _few("few_decode_e4m3", 32, 7168, 2048, 256, 8, "e4m3", 0, bias=True),
        # an odd batch with unused slots on a rank's 32 experts of skewed popularity
        _few("few_ragged_e2m1", 61, 7168, 2048, 32, 8, "e2m1", 32, "zipf", 5),
        # the end of a layer for one request
        _norm("norm_one_token", "norm", 1, 7168, 256, 8, 1, "channel"),
        # the end of the prefill workload's layer, the shared expert's output as bias
        _norm("norm_prefill", "norm", 4096, 7168, 256, 8, 128, "channel", bias=True, routing="grouped"),
        # a training step of it
        _norm("norm_train", "norm_train", 4096, 7168, 256, 8, 128, "channel", routing="grouped"),
        # the same around a block without experts, odd sizes, a gate for each token, 16-bit vectors
        _norm("norm_train_ragged", "norm_train", 777, 2112, 8, 0, 1, "token", vectors="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4", "w4", "few", "few", "norm", "norm_train"])
    routing = rng.choice(["uniform", "zipf"])
    if op == "norm" or op == "norm_train":
        T = _log(rng, 1, 4096)
        case = _norm("", op, T, 8 * max(1, _log(rng, 64, 7168) // 8), rng.choice([8, 64, 100, 256]), rng.randint(0, 8),
                     rng.choice([1, 16, 128]), rng.choice(["none", "channel", "token"]), rng.choice([False, True]),
                     rng.choice([0, 0, T // 7]), routing, rng.choice(["fp32", "bf16"]))
    else:
        T = _log(rng, 1, 4096 if op == "w4" else 128)
        E = rng.choice([4, 8, 20, 32, 33, 64])
        fmt = rng.choice(["int4", "e2m1"] if op == "w4" else ["int4", "e2m1", "bf16", "e4m3"])
        group = rng.choice([32, 64, 128]) if fmt in ("int4", "e2m1") else 0
        unit = group or (BLOCK if fmt == "e4m3" else 8)
        H = unit * max(1, _log(rng, 256, 7168) // unit)
        I = unit * max(1, _log(rng, 128, 2048) // unit)
        K, idle = rng.randint(1, min(8, E)), rng.choice([0, 0, T // 9])
        if op == "w4":
            case = _w4("", T, H, I, E, K, rng.choice([1, 16, 128]), fmt, group, routing, idle)
        else:
            case = _few("", T, H, I, E, K, fmt, group, routing, idle, rng.choice([False, True]))
    case.pop("name")
    return case


# ---- inputs ---------------------------------------------------------------------------------------------------------

PIECE = 1 << 27


def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    """N(0, std^2) in `dtype`, drawn in pieces so that large weights need no 32-bit copy of themselves."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), PIECE):
        n = min(PIECE, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device=DEV, dtype=torch.float32).mul_(std).to(dtype)
    return out


def _e4m3(gen, *shape):
    """e4m3 values as a block-scaled normal tensor has them: sigma 104, the largest near 448."""
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), PIECE):
        n = min(PIECE, flat.numel() - i)
        v = torch.randn(n, generator=gen, device=DEV, dtype=torch.float32).mul_(104.0).clamp_(-448.0, 448.0)
        flat[i:i + n] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _codes(gen, kind, *shape):
    """4-bit codes of a group-scaled normal tensor, two a byte, the lower half first: [..., k / 2]."""
    out = torch.empty(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, device=DEV)
    flat = out.view(-1)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for i in range(0, flat.numel(), PIECE // 2):
        n = min(PIECE // 2, flat.numel() - i)
        v = torch.randn(2, n, generator=gen, device=DEV, dtype=torch.float32)
        if kind == "int4":
            code = v.mul_(2.8).round_().clamp_(-8.0, 7.0).add_(8.0).to(torch.uint8)
        else:
            v.mul_(2.2)
            code = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) + (v < 0).to(torch.uint8) * 8
        flat[i:i + n] = code[0] + code[1] * 16
    return out


def _scales(gen, std, *shape):
    return torch.empty(shape, device=DEV).uniform_(0.7, 1.4, generator=gen).mul_(std)


def _weights(gen, case, E, N, K):
    """(weights [E, N, K], scales) of deviation K^-1/2 in the case's format."""
    fmt, std = case["fmt"], K ** -0.5
    if fmt == "bf16":
        return _normal(gen, E, N, K, std=std), None
    if fmt == "e4m3":
        return _e4m3(gen, E, N, K), _scales(gen, std / 104.0, E, N // BLOCK, K // BLOCK)
    codes = _codes(gen, fmt, E, N, K)
    return codes, _scales(gen, std / (2.8 if fmt == "int4" else 2.2), E, N, K // case["group"]).to(torch.bfloat16)


def _routing(case, gen):
    """topk_idx int64 [T, K]; the last `idle` tokens are padding of the batch (every entry -1)."""
    T, E, K = case["tokens"], case["experts"], case["topk"]
    logits = torch.randn(T, E, generator=gen, device=DEV, dtype=torch.float64)
    if case["routing"] == "grouped" and E % 8 == 0:      # group-limited gating: the four best of eight groups
        best = logits.view(T, 8, E // 8).amax(2).topk(4, dim=1).indices
        keep = torch.zeros(T, 8, dtype=torch.bool, device=DEV).scatter_(1, best, True)
        logits = logits.masked_fill(~keep.repeat_interleave(E // 8, dim=1), -math.inf)
    elif case["routing"] == "zipf":                      # popularity (i + 1)^-1.1 over a permutation, without replacement
        pop = torch.randperm(E, generator=gen, device=DEV).double() + 1
        u = torch.rand(T, E, generator=gen, device=DEV, dtype=torch.float64).clamp_(1e-300, 1 - 1e-12)
        logits = -1.1 * pop.log() - (-u.log()).log()
    idx = logits.topk(K, dim=1).indices
    if case["idle"]:
        idx[T - case["idle"]:] = -1
    return idx.contiguous()


def _plan(case, idx):
    """The layout of the routing table, by the definition: each entry's row, the experts' starts and counts."""
    E, A = case["experts"], case["align"]
    flat = idx.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    count = torch.zeros(E + 1, dtype=torch.int64, device=DEV).index_add_(0, key, torch.ones_like(flat))[:E]
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), ((count + A - 1) // A * A).cumsum(0)])
    order = torch.sort(key, stable=True).indices
    before = count.cumsum(0) - count
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=DEV)
    safe = flat.clamp(min=0)
    slot = torch.where(flat < 0, -1, start[safe] + place - before[safe])
    most = max(1, int(count.max()))
    used = count.nonzero().view(-1)
    if used.numel() == 0:
        used = torch.zeros(1, dtype=torch.int64, device=DEV)
    return {"slot": slot.view_as(idx), "start": start[:-1].contiguous(), "count": count, "most": most, "used": used,
            "rows": case["tokens"] * case["topk"] + E * (A - 1)}


def _share(gen, T, K):
    w = torch.rand(T, K, generator=gen, device=DEV) + 0.05
    return w / w.sum(1, keepdim=True)


def _prepare_norm(case, gen, s):
    T, H = case["tokens"], case["hidden"]
    if case["topk"]:
        idx = s["idx"] = _routing(case, gen)
        s["plan"] = _plan(case, idx)
        s["y"], s["w"] = _normal(gen, s["plan"]["rows"], H), _share(gen, T, case["topk"])
    else:
        s["y"], s["w"] = _normal(gen, T, H), None
    s["bias"] = _normal(gen, T, H, std=0.1) if case["bias"] else None
    s["residual"] = _normal(gen, T, H, std=2.0)
    kind = torch.float32 if case["vectors"] == "fp32" else torch.bfloat16
    vector = lambda mean, std: torch.randn(H, generator=gen, device=DEV).mul_(std).add_(mean).to(kind)
    s["post"], s["pre"] = vector(1.0, 0.1), vector(1.0, 0.1)
    s["gate"] = None if case["gate"] == "none" else vector(0.5, 0.2) if case["gate"] == "channel" else _normal(gen, T, H, std=0.5)
    s["rs"] = 0.75
    if case["op"] == "norm_train":
        s["do"], s["dn"] = _normal(gen, T, H), _normal(gen, T, H)
    if own:
        import combine_get_dispatch_03_amd as ep
        s["handle"] = ep.ep_get_layout(s["idx"], case["experts"], expert_alignment=case["align"])[0] if case["topk"] else None
        if case["op"] == "norm_train":
            s["ws"] = torch.empty(ep.ep_combine_norm_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
            s["kept"] = torch.empty(T, H, device=DEV) if case["topk"] or case["bias"] else None
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 1000003 + 29)
    s = {"case": case}
    if case["op"] in ("norm", "norm_train"):
        return _prepare_norm(case, gen, s)
    T, H, I, E, K = case["tokens"], case["hidden"], case["inter"], case["experts"], case["topk"]
    idx = s["idx"] = _routing(case, gen)
    s["plan"] = _plan(case, idx)
    s["w13"], s["s13"] = _weights(gen, case, E, 2 * I, H)
    s["w2"], s["s2"] = _weights(gen, case, E, H, I)
    if case["op"] == "w4":
        s["x"] = _normal(gen, s["plan"]["rows"], H)
        s["y"] = torch.zeros(s["plan"]["rows"], H, dtype=torch.bfloat16, device=DEV)     # rows that no entry owns stay zero
    else:
        s["x"], s["w"] = _normal(gen, T, H), _share(gen, T, K)
        s["bias"] = _normal(gen, T, H, std=0.1) if case["bias"] else None
    if own:
        import combine_get_dispatch_03_amd as ep
        if case["group"]:                                # a program packs its weights when it loads them
            s["w13"], s["s13"] = ep.ep_w4_pack(s["w13"], s["s13"], case["fmt"]), None
            s["w2"], s["s2"] = ep.ep_w4_pack(s["w2"], s["s2"], case["fmt"]), None
        if case["op"] == "w4":
            s["handle"] = ep.ep_get_layout(idx, E, expert_alignment=case["align"])[0]
            n = ep.ep_expert_ffn_workspace_bytes(s["handle"], H, I)
        else:
            n = ep.ep_moe_few_workspace_bytes(T, K, I)
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------------

def _segments(plan):
    """Rows of each used expert's segment as [experts, most], and which of them are valid; others point at row 0."""
    at = torch.arange(plan["most"], device=DEV)
    ok = at < plan["count"][plan["used"], None]
    return torch.where(ok, plan["start"][plan["used"], None] + at, 0), ok


def _wide(q, scales, used, fmt):
    """Weights of the used experts in 32 bits."""
    if used.numel() < q.shape[0]:
        q, scales = q[used], None if scales is None else scales[used]
    if fmt == "bf16":
        return q.float()
    if fmt == "e4m3":
        E, N, K = q.shape
        w = q.view(torch.float8_e4m3fn).float().view(E, N // BLOCK, BLOCK, K // BLOCK, BLOCK)
        return w.mul_(scales[:, :, None, :, None]).view(E, N, K)
    E, N, B = q.shape
    values = torch.arange(16, device=DEV).float() - 8.0 if fmt == "int4" else torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    w = torch.empty(E, N, B, 2, device=DEV)
    for e in range(E):
        w[e, :, :, 0] = values[(q[e] & 15).int()]
        w[e, :, :, 1] = values[(q[e] >> 4).int()]
    G = scales.shape[2]
    return w.view(E, N, G, 2 * B // G).mul_(scales.float()[..., None]).view(E, N, 2 * B)


def _plain_ffn(s, x, at):
    """The block over x [used experts, rows, H] -> [used experts, rows, H] in 32 bits."""
    I, fmt, used = s["case"]["inter"], s["case"]["fmt"], s["plan"]["used"]
    w13 = _wide(s["w13"], s["s13"], used, fmt)
    p = torch.bmm(x, w13.transpose(1, 2))
    del w13
    g, u = p[..., :I], p[..., I:]
    h = g / (1.0 + torch.exp(-g)) * u
    return torch.bmm(h, _wide(s["w2"], s["s2"], used, fmt).transpose(1, 2))


def _plain_w4(s):
    at, ok = _segments(s["plan"])
    y = _plain_ffn(s, torch.where(ok[..., None], s["x"][at].float(), 0.0), at)
    full = torch.zeros(s["y"].shape[0] + 1, s["y"].shape[1], dtype=torch.bfloat16, device=DEV)
    full[torch.where(ok, at, s["y"].shape[0])] = y.to(torch.bfloat16)
    return full[:-1]


def _plain_few(s):
    case, plan = s["case"], s["plan"]
    at, ok = _segments(plan)
    K, V = case["topk"], plan["slot"].numel()
    entry = torch.zeros(plan["rows"] + 1, dtype=torch.int64, device=DEV)       # which entry a row belongs to
    slot = plan["slot"].view(-1)
    entry[torch.where(slot < 0, plan["rows"], slot)] = torch.arange(V, device=DEV)
    y = _plain_ffn(s, torch.where(ok[..., None], s["x"][entry[at] // K].float(), 0.0), at)
    flat = torch.zeros(V + 1, case["hidden"], device=DEV)
    flat[torch.where(ok, entry[at], V)] = y
    out = (flat[:V].view(-1, K, case["hidden"]) * torch.where(plan["slot"] < 0, 0.0, s["w"])[..., None]).sum(1)
    return (out if s["bias"] is None else out + s["bias"].float()).to(torch.bfloat16)


def _plain_norm(s):
    train = s["case"]["op"] == "norm_train"
    post, pre, rs = s["post"].float(), s["pre"].float(), s["rs"]
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    if s["w"] is None:
        f = s["y"].float()
    else:
        slot = s["plan"]["slot"]
        f = torch.zeros(slot.shape[0], s["y"].shape[1], device=DEV)
        for k in range(slot.shape[1]):
            f += torch.where(slot[:, k, None] < 0, 0.0, s["w"][:, k, None] * s["y"][slot[:, k].clamp(min=0)].float())
    if s["bias"] is not None:
        f += s["bias"].float()
    rf = 1.0 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)
    fh = f * rf
    a = fh * post
    r = rs * s["residual"].float() + gate * a
    rr = 1.0 / torch.sqrt((r * r).mean(1, keepdim=True) + EPS)
    rh = r * rr
    out = {"out": r.to(torch.bfloat16), "normed": (rh * pre).to(torch.bfloat16)}
    if not train:
        return out
    dn = s["dn"].float()
    dnp = dn * pre
    dr = s["do"].float() + rr * (dnp - rh * (dnp * rh).mean(1, keepdim=True))
    da = gate * dr
    dap = da * post
    out["grad_f"] = (rf * (dap - fh * (dap * fh).mean(1, keepdim=True))).to(torch.bfloat16)
    out["grad_residual"] = (rs * dr).to(torch.bfloat16)
    out["grad_post"], out["grad_pre"] = (da * fh).sum(0), (dn * rh).sum(0)
    if s["gate"] is not None:
        out["grad_gate"] = (dr * a).sum(0) if s["gate"].dim() == 1 else (dr * a).to(torch.bfloat16)
    return out


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return _plain_w4(s) if op == "w4" else _plain_few(s) if op == "few" else _plain_norm(s)
    import combine_get_dispatch_03_amd as ep
    if op == "w4":
        return ep.ep_expert_ffn_w4(s["handle"], s["x"], s["w13"], s["w2"], y=s["y"], workspace=s["ws"])
    if op == "few":
        return ep.ep_moe_few(s["x"], s["idx"], s["w"], s["w13"], s["w2"], w13_scales=s["s13"], w2_scales=s["s2"], bias=s["bias"],
                             workspace=s["ws"])
    around = dict(residual=s["residual"], post_weight=s["post"], gate=s["gate"], residual_scale=s["rs"], pre_weight=s["pre"], eps=EPS)
    if op == "norm":
        out, normed = ep.ep_combine_norm(s["handle"], s["y"], s["w"], bias=s["bias"], **around)
        return {"out": out, "normed": normed}
    out, normed = ep.ep_combine_norm(s["handle"], s["y"], s["w"], bias=s["bias"], kept=s["kept"], **around)
    f = s["y"] if s["kept"] is None else s["kept"]
    grads = ep.ep_combine_norm_backward(s["do"], s["dn"], f, workspace=s["ws"], **around)
    return dict(out=out, normed=normed, **{k: v for k, v in grads.items() if v is not None})


# ---- what a pass cannot do without, and what it gives in 64 bits -----------------------------------------------------

def work(case):
    T, H, K = case["tokens"], case["hidden"], case["topk"]
    live = T - case["idle"]
    if case["op"] in ("norm", "norm_train"):
        V = live * K if K else T
        read = 2 * H * (V + T * (1 + case["bias"] + (case["gate"] == "token"))) + 12 * T * K
        forward = read + 2 * H * 2 * T
        if case["op"] == "norm":
            return {"bytes": forward, "flops": (2 * V + 12 * T) * H}
        return {"bytes": forward + 2 * H * T * (4 + (case["gate"] == "token")), "flops": (2 * V + 45 * T) * H}
    I, E = case["inter"], case["experts"]
    used = E * (1 - (1 - K / E) ** live)                 # experts that some row reaches, were the routing uniform
    wide = {"bf16": 2.0, "e4m3": 1.0}.get(case["fmt"]) or 0.5 + 2.0 / case["group"]
    rows = 4 * live * K * H if case["op"] == "w4" else 2 * H * T * (2 + case["bias"])
    return {"bytes": 3 * H * I * wide * used + rows, "flops": 6 * live * K * H * I}


def _expert64(s, e):
    """One expert's weights in 64 bits."""
    def wide(q, scales):
        fmt = s["case"]["fmt"]
        if fmt == "bf16":
            return q[e].double()
        if fmt == "e4m3":
            return q[e].view(torch.float8_e4m3fn).double() * scales[e].double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
        code = torch.stack([q[e] % 16, q[e] // 16], dim=2).flatten(1).long()
        if fmt == "int4":
            v = code.double() - 8
        else:
            ex, m = code // 2 % 4, code % 2
            v = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (ex.double() - 1)) * (1 - 2 * (code // 8))
        return v * scales[e].double().repeat_interleave(s["case"]["group"], 1)
    return wide(s["w13"], s["s13"]), wide(s["w2"], s["s2"])


def _ffn64(s, e, x):
    w13, w2 = _expert64(s, e)
    I = w2.shape[1]
    p = x @ w13.t()
    return (p[:, :I] * torch.sigmoid(p[:, :I]) * p[:, I:]) @ w2.t()


def _exact_norm(s):
    """The gradients by torch's own differentiation of the definition in 64 bits."""
    train = s["case"]["op"] == "norm_train"
    leaf = {k: s[k].double().requires_grad_(train) for k in ("residual", "post", "pre", "gate") if s[k] is not None}
    if s["w"] is None:
        f = s["y"].double()
    else:
        f = torch.zeros(s["case"]["tokens"], s["case"]["hidden"], dtype=torch.float64, device=DEV)
        for k in range(s["case"]["topk"]):
            t = (s["plan"]["slot"][:, k] >= 0).nonzero().view(-1)
            f[t] += s["w"][t, k].double()[:, None] * s["y"][s["plan"]["slot"][t, k]].double()
    if s["bias"] is not None:
        f = f + s["bias"].double()
    leaf["f"] = f.requires_grad_(train)
    rms = lambda v: v / (v.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    r = leaf["residual"] * s["rs"] + rms(leaf["f"]) * leaf["post"] * leaf.get("gate", 1.0)
    n = rms(r) * leaf["pre"]
    out = {"out": r.detach(), "normed": n.detach()}
    if train:
        grads = torch.autograd.grad([r, n], list(leaf.values()), [s["do"].double(), s["dn"].double()])
        grads = dict(zip(leaf, grads))
        for k in ("f", "residual", "post", "pre", "gate"):
            if k in grads:
                out["grad_" + k] = grads[k]
    return out


def exact(case, seed):
    global own
    kept, own = own, False                               # the inputs alone
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(s)
    plan = s["plan"]
    if case["op"] == "w4":
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
        for e, (at, n) in enumerate(zip(plan["start"].tolist(), plan["count"].tolist())):
            if n:
                y[at:at + n] = _ffn64(s, e, s["x"][at:at + n].double())
        return y
    out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device=DEV)
    for e in plan["used"].tolist():
        t, k = (s["idx"] == e).nonzero(as_tuple=True)
        if t.numel():
            out.index_add_(0, t, s["w"][t, k].double()[:, None] * _ffn64(s, e, s["x"][t].double()))
    return out if s["bias"] is None else out + s["bias"].double()
