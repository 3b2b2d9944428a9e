"""4-bit weights by their definition, and the whole layer in 64 bits with the error that fp32 sums and the documented roundings can
leave (see expert_reference.py).  Nothing here uses the library."""
import torch

import expert_reference as R

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def random_w4(gen, kind, group, M, N, K, device, std=1.0):
    """codes uint8 [M, N, K / 2] over all sixteen values, and bf16 scales [M, N, K / group]."""
    codes = torch.randint(0, 256, (M, N, K // 2), generator=gen, device=device, dtype=torch.int32).to(torch.uint8)
    scales = (torch.rand(M, N, K // group, generator=gen, device=device) + 0.5) * (std / (4.6 if kind == "int4" else 2.9))
    return codes, scales.bfloat16()


def widen(codes, scales, kind):
    """[N, K / 2] codes and [N, K / group] scales -> float64 [N, K]."""
    low, high = (codes & 15).long(), (codes >> 4).long()
    code = torch.stack([low, high], dim=2).flatten(1)
    table = [float(i - 8) for i in range(16)] if kind == "int4" else E2M1 + [-v for v in E2M1]
    v = torch.tensor(table, dtype=torch.float64, device=codes.device)[code]
    return v * scales.double().repeat_interleave(v.shape[1] // scales.shape[1], dim=1)


def layer(x, idx, w, bias, lo, experts, K):
    """out [T, H] and its bound: experts(e) gives (w13, w2) in 64 bits of the local expert e."""
    T, H = x.shape
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    err, size = out.clone(), out.clone()
    local = idx - lo
    for e, (w13, w2) in experts.items():
        t, k = (local == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        f = R.ffn_expert(x[t].double(), w13, w2)
        ey = f["eh"] @ w2.abs().t() + w2.shape[1] * R.U32 * ((f["h"].abs() + f["eh"]) @ w2.abs().t())
        s = torch.ones(t.numel(), 1, dtype=torch.float64, device=x.device) if w is None else w[t, k].double()[:, None]
        out.index_add_(0, t, s * f["y"])
        err.index_add_(0, t, s.abs() * ey)
        size.index_add_(0, t, s.abs() * (f["y"].abs() + ey))
    if bias is not None:
        out, size = out + bias.double(), size + bias.double().abs()
    err = err + (K + 2) * R.U32 * size
    return out, err + R.UBF * (out.abs() + err) + R.TINY
