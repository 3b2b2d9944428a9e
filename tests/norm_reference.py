"""The combine with its norms and its gradient in 64 bits, with the error that fp32 arithmetic and the documented roundings can
leave in each output.  Nothing here uses the library.

Error bounds.  U is twice an fp32 rounding (2^-24): every elementary operation is off by at most that, a square root and a
divide included.  A sum over a row is made of at most 32 terms in a thread, 6 steps over the lanes and 16 over the waves, so SUM =
56 roundings of the sum of the terms' magnitudes; a sum over tokens is off by at most one rounding per token.  Rounding to bf16 is off
by at most 2^-8 of the value.  A factor 1 / sqrt(m + eps) is off by half of m's relative error.  The rest is the triangle
inequality.
"""
import torch

U = 2.0 * 2.0 ** -24
UBF = 2.0 ** -8
SUM = 56
TINY = 1e-30


def combined(slot, y, w, bias):
    """f [T, H] and its bound: the weighted sum of a token's rows (slot [T, K], -1 = none) and bias."""
    T, K = slot.shape
    f = torch.zeros(T, y.shape[1], dtype=torch.float64, device=y.device)
    size = f.clone()
    for k in range(K):
        t = (slot[:, k] >= 0).nonzero().view(-1)
        v = y[slot[t, k]].double() * (1.0 if w is None else w[t, k].double()[:, None])
        f[t] += v
        size[t] += v.abs()
    if bias is not None:
        f, size = f + bias.double(), size + bias.double().abs()
    return f, (K + 2) * U * size


def _factor(v, ev, eps):
    """1 / sqrt(mean v^2 + eps) per row and its relative error."""
    m = (v * v).mean(1, keepdim=True) + eps
    return m.rsqrt(), 0.5 * ((SUM + 4) * U + (2 * v.abs() * ev + ev * ev).mean(1, keepdim=True) / m) + 4 * U


def around(f, ef, residual, post, gate, rs, pre, eps):
    """Everything the forward pass computes, with bounds (None where a part is absent)."""
    one = torch.ones((), dtype=torch.float64, device=f.device)
    d = lambda t: one if t is None else t.double()
    rf, df = (one, 0.0 * one) if post is None else _factor(f, ef, eps)
    a = f * rf * d(post)
    ea = (rf * d(post)).abs() * ef + a.abs() * (df + 3 * U)
    res = 0.0 * f if residual is None else residual.double() * rs
    r = res + d(gate) * a
    er = res.abs() * 2 * U + d(gate).abs() * ea + (d(gate) * a).abs() * 4 * U
    o = dict(rf=rf, df=df, a=a, ea=ea, r=r, er=er, out=r, eout=er + UBF * (r.abs() + er) + TINY)
    if pre is not None:
        rr, dr = _factor(r, er, eps)
        n = r * rr * d(pre)
        en = (rr * d(pre)).abs() * er + n.abs() * (dr + 3 * U)
        o.update(rr=rr, dr=dr, n=n, en=en + UBF * (n.abs() + en) + TINY)
    return o


def gradients(f, residual, post, gate, rs, pre, eps, dout, dn):
    """Gradients by the formulas, and bounds, from f exactly as given."""
    f = f.double()
    T = f.shape[0]
    o = around(f, torch.zeros_like(f), residual, post, gate, rs, pre, eps)
    one = torch.ones((), dtype=torch.float64, device=f.device)
    gate_, post_ = (one if t is None else t.double() for t in (gate, post))
    g = {}
    dr = torch.zeros_like(f) if dout is None else dout.double()
    edr = 2 * U * dr.abs()

    def through_norm(d, ed, v, ev, fac, rel):
        """Gradient of v * fac with respect to v, from the gradient d."""
        h = v * fac
        eh = fac * ev + h.abs() * (rel + 2 * U)
        m = (d * h).mean(1, keepdim=True)
        em = (ed * h.abs() + d.abs() * eh + (SUM + 4) * U * (d * h).abs()).mean(1, keepdim=True)
        x = fac * (d - h * m)
        ex = fac * (ed + eh * m.abs() + h.abs() * em + 4 * U * (d.abs() + (h * m).abs())) + x.abs() * (rel + 2 * U)
        return x, ex, h, eh

    if dn is not None:
        d = dn.double() * pre.double()
        x, ex, h, eh = through_norm(d, U * d.abs(), o["r"], o["er"], o["rr"], o["dr"])
        dr, edr = dr + x, edr + ex + 2 * U * x.abs()
        v = dn.double() * h
        g["grad_pre"] = v.sum(0), (dn.double().abs() * eh + (T + 4) * U * v.abs()).sum(0) + TINY
    if residual is not None:
        v, e = rs * dr, abs(rs) * (edr + 2 * U * dr.abs())
        g["grad_residual"] = v, e + UBF * (v.abs() + e) + TINY
    if gate is not None:
        v, e = dr * o["a"], edr * o["a"].abs() + dr.abs() * o["ea"] + 4 * U * (dr * o["a"]).abs()
        g["grad_gate"] = (v, e + UBF * (v.abs() + e) + TINY) if gate.dim() == 2 else (v.sum(0), (e + T * U * v.abs()).sum(0) + TINY)
    da, eda = gate_ * dr, gate_.abs() * edr + U * (gate_ * dr).abs()
    if post is not None:
        h = f * o["rf"]
        v = da * h
        g["grad_post"] = v.sum(0), (eda * h.abs() + v.abs() * (o["df"] + (T + 4) * U)).sum(0) + TINY
        d, ed = da * post_, post_.abs() * eda + U * (da * post_).abs()
        da, eda, _, _ = through_norm(d, ed, f, torch.zeros_like(f), o["rf"], o["df"])
    g["grad_f"] = da, eda + UBF * (da.abs() + eda) + TINY
    return g
