"""Plain forms in 64 bits of the expert block, its gradients, the combine's gradient and the adapters, with the error that
fp32 sums and the documented roundings can leave in each output.  They take the routing table and work the layout out
for themselves; nothing here uses the library.

Error bounds.  A sum of n products in fp32, in any order, is off by at most n * 2^-24 * sum |products| (U32 below, with
a factor of 2 for the widening of e4m3 blocks by their scales and for the order inside a matrix instruction); rounding to
bf16 is off by at most 2^-8 of the value (half of bf16's step 2^-7).  exp and the divide of the sigmoid are off by
a few fp32 steps plus the rounding of the exponent's argument, (|g| + 16) * 2^-23 of the value.  A bound of an output is the bounds of
what goes into it, carried through by the triangle inequality:  |d silu/dg| <= 1.1, |d silu'/dg| <= 0.5.
"""
import torch

U32 = 2.0 * 2.0 ** -24
UBF = 2.0 ** -8
TINY = 1e-30


def segments(topk_idx, E, lo, El, A):
    """Rows of every local entry by the layout's definition: (slot [T, K], start [El], count [El]) as host data."""
    idx = topk_idx.cpu()
    T, K = idx.shape
    flat = idx.reshape(-1)
    slot = torch.full((T * K,), -1, dtype=torch.int64)
    start, count, at = [], [], 0
    for e in range(lo, lo + El):
        mine = (flat == e).nonzero().view(-1)
        slot[mine] = at + torch.arange(mine.numel())
        start.append(at)
        count.append(mine.numel())
        at += -(-mine.numel() // A) * A
    return slot.view(T, K), start, count


def widen(q, scales, block):
    """bf16, or e4m3 bytes with a scale per 128 columns and `block` rows, as float64."""
    if q.dtype != torch.uint8:
        return q.double()
    s = scales.double().repeat_interleave(128, dim=1)
    return q.view(torch.float8_e4m3fn).double() * (s.repeat_interleave(block, dim=0) if block > 1 else s)


def ffn_expert(x, w13, w2):
    """One expert's rows: values and bounds of the pre-activations, h and y (all float64)."""
    I = w2.shape[1]
    p = x @ w13.t()
    ep = x.shape[1] * U32 * (x.abs() @ w13.abs().t())
    g, u, eg, eu = p[:, :I], p[:, I:], ep[:, :I], ep[:, I:]
    s = torch.sigmoid(g)
    act = g * s
    h = act * u
    h32 = 1.1 * u.abs() * eg + act.abs() * eu + eg * eu + h.abs() * (g.abs() + 16) * 2.0 ** -23
    eh = h32 + UBF * (h.abs() + h32)
    y = h @ w2.t()
    ey = eh @ w2.abs().t() + I * U32 * ((h.abs() + eh) @ w2.abs().t())
    ey = ey + UBF * (y.abs() + ey) + TINY
    return dict(p=p, ep=ep + TINY, h=h, eh=eh, y=y, ey=ey)


def ffn_expert_grads(x, w13, w2, dy):
    f = ffn_expert(x, w13, w2)
    I, H = w2.shape[1], w2.shape[0]
    n = x.shape[0]
    g, u, eg, eu = f["p"][:, :I], f["p"][:, I:], f["ep"][:, :I], f["ep"][:, I:]
    s = torch.sigmoid(g)
    act, slope = g * s, s * (1 + g * (1 - s))
    dh = dy @ w2
    edh = H * U32 * (dy.abs() @ w2.abs())
    dg, du = dh * u * slope, dh * act
    rel = (g.abs() + 16) * 2.0 ** -22
    edg = 1.1 * u.abs() * edh + (dh.abs() + edh) * (0.5 * u.abs() * eg + 1.1 * eu + 0.5 * eg * eu) + dh.abs() * u.abs() * 1.1 * rel
    edu = act.abs() * edh + (dh.abs() + edh) * 1.1 * eg + du.abs() * rel
    dp, edp = torch.cat([dg, du], 1), torch.cat([edg, edu], 1)
    edp = edp + UBF * (dp.abs() + edp)

    def product(a, ea, b, eb, terms):
        v = a @ b
        e = ea @ b.abs() + (a.abs() + ea) @ eb if eb is not None else ea @ b.abs()
        e = e + terms * U32 * ((a.abs() + ea) @ (b.abs() + (0 if eb is None else eb)))
        return v, e + UBF * (v.abs() + e) + TINY

    dx = product(dp, edp, w13, None, 2 * I)
    dw13 = product(dp.t(), edp.t(), x, None, max(n, 1))
    dw2 = product(dy.t(), torch.zeros_like(dy.t()), f["h"], f["eh"], max(n, 1))
    return dict(f, dx=dx[0], edx=dx[1], dw13=dw13[0], edw13=dw13[1], dw2=dw2[0], edw2=dw2[1], dp=dp)


def assert_within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its bound (|error| %.3g, value %.3g)" % (
        what, int(bad.sum()), bad.numel(), float((err / bound).nan_to_num(nan=float("inf")).max()),
        float(err.nan_to_num(nan=float("inf")).max()), float(want.reshape(-1)[(err / bound).reshape(-1).argmax()]))
