"""Packed 4-bit weights put together by hand, for instance from a checkpoint: a W4Weights only holds tensors of the sizes that its kind,
group and shape have, and keeps them (the kernels take its word for how far they may read)."""
import pytest
import torch

import combine_get_dispatch_03_amd as ep

M, N, K, G = 2, 32, 160, 32
U8 = torch.uint8


def parts(M=M, N=N, K=K, group=G):
    return torch.zeros(ep.ep_w4_packed_bytes(M, N, K, group), dtype=U8), torch.zeros(ep.ep_w4_packed_scale_bytes(M, N, K, group), dtype=U8)


def test_fits():
    v, s = parts()
    w = ep.W4Weights(v, s, "e2m1", G, [M, N, K])
    assert w.values is v and w.scales is s and w.kind == "e2m1" and w.group == G and w.shape == (M, N, K) and w.device == v.device


V, S = parts()


@pytest.mark.parametrize("kw,what", [
    (dict(kind="int3"), ValueError), (dict(shape=(M, N)), ValueError), (dict(shape=(M, N, K, 1)), ValueError),
    (dict(group=48), ep.EPError), (dict(group=64), ep.EPError), (dict(shape=(M, 24, K)), ep.EPError), (dict(shape=(0, N, K)), ep.EPError),
    (dict(shape=(M + 1, N, K)), ValueError), (dict(shape=(M, 2 * N, K)), ValueError), (dict(shape=(M, N, 2 * K)), ValueError),
    (dict(values=V[:-16]), ValueError), (dict(values=V.view(torch.int8)), TypeError), (dict(values=None), TypeError),
    (dict(values=torch.zeros(2 * V.numel(), dtype=U8)[::2]), ValueError), (dict(values=V.view(2, -1)), ValueError),
    (dict(scales=S[:-16]), ValueError), (dict(scales=S.view(torch.bfloat16)), TypeError), (dict(scales=None), TypeError),
    (dict(scales=S.to("meta")), ValueError),
])
def test_refusals(kw, what):
    with pytest.raises(what):
        ep.W4Weights(**{**dict(values=V, scales=S, kind="int4", group=G, shape=(M, N, K)), **kw})


@pytest.mark.parametrize("name", ["values", "scales", "kind", "group", "shape", "device"])
def test_parts_stay(name):
    w = ep.W4Weights(V, S, "int4", G, (M, N, K))
    with pytest.raises(AttributeError):
        setattr(w, name, getattr(w, name))
