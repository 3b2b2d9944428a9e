"""Refusals of the 4-bit weights and of the layer for a few tokens: every argument is checked on the host before anything is
enqueued.  The device addresses below are never dereferenced."""
import ctypes

import pytest
import torch

import combine_get_dispatch_03_amd as ep

L = ep._lib
A, B, N = 0x100000, 0x200000, None
INT4, E2M1, E4M3, BF16 = ep.EP_WEIGHTS_INT4, ep.EP_WEIGHTS_E2M1, ep.EP_WEIGHTS_E4M3, ep.EP_WEIGHTS_BF16


def weights(fmt=INT4, group=32, values=A, scales=A):
    return ctypes.byref(ep._Weights(values, scales, fmt, group))


def pack(codes=A, scales=A, fmt=INT4, M=2, rows=32, cols=64, group=32, out=B, out_scales=B):
    return L.ep_w4_pack(codes, scales, fmt, M, rows, cols, group, out, out_scales, None)


@pytest.mark.parametrize("kw,why", [
    (dict(fmt=BF16), b"format"), (dict(fmt=E4M3), b"format"), (dict(fmt=9), b"format"),
    (dict(group=16), b"group"), (dict(group=0), b"group"), (dict(group=256), b"group"),
    (dict(M=0), b"matrices"), (dict(M=1025), b"matrices"), (dict(rows=24), b"rows"), (dict(rows=0), b"rows"), (dict(rows=65552), b"rows"),
    (dict(cols=48), b"columns"), (dict(cols=0), b"columns"), (dict(cols=32800), b"columns"), (dict(cols=64, group=128), b"columns"),
    (dict(codes=N), b"codes"), (dict(codes=A + 8), b"codes"), (dict(scales=N), b"scales"), (dict(scales=A + 2), b"scales"),
    (dict(out=N), b"packed"), (dict(out=B + 8), b"packed"), (dict(out_scales=N), b"packed"), (dict(out_scales=B + 4), b"packed"),
])
def test_pack_refusals(kw, why):
    assert pack(**kw) == 1 and why in L.ep_last_error()


def test_packed_sizes():
    assert L.ep_w4_packed_bytes(2, 32, 128, 32) == 2 * 32 * 64 and L.ep_w4_packed_scale_bytes(2, 32, 128, 32) == 2 * 32 * 4 * 2
    assert L.ep_w4_packed_bytes(1, 16, 160, 32) == 16 * 128 and L.ep_w4_packed_scale_bytes(1, 16, 160, 32) == 16 * 8 * 2
    assert L.ep_w4_packed_scale_bytes(3, 16, 192, 64) == 3 * 16 * 4 * 2 and L.ep_w4_packed_scale_bytes(3, 16, 384, 128) == 3 * 16 * 3 * 2
    assert L.ep_w4_packed_bytes(1024, 65536, 32768, 128) == 1024 * 65536 * 16384
    for bad in ((0, 32, 128, 32), (2, 40, 128, 32), (2, 32, 100, 32), (2, 32, 128, 48)):
        assert L.ep_w4_packed_bytes(*bad) == 0 and L.ep_w4_packed_scale_bytes(*bad) == 0


def few(x=A, idx=A, w=A, T=4, K=2, E=8, R=1, rank=0, H=64, I=32, w13=None, w2=None, bias=N, out=B, ws=B, nws=1 << 20, **kw):
    return L.ep_moe_few(x, idx, w, T, K, E, R, rank, H, I, w13 or weights(**kw), w2 or weights(**kw), bias, out, ws, nws, None)


@pytest.mark.parametrize("kw,why", [
    (dict(T=-1), b"num_tokens"), (dict(T=129), b"num_tokens"), (dict(T=128, K=9), b"1024"), (dict(K=0), b"num_topk"), (dict(K=33), b"num_topk"),
    (dict(E=0), b"num_experts"), (dict(E=1025), b"num_experts"), (dict(E=8, R=3), b"num_ranks"), (dict(rank=1), b"rank"), (dict(rank=-1), b"rank"),
    (dict(fmt=7), b"format"), (dict(fmt=-1), b"format"), (dict(w2=weights(E2M1)), b"same format"), (dict(w2=weights(INT4, 64)), b"same group"),
    (dict(group=48), b"group"), (dict(H=72), b"multiples of the group"), (dict(I=16), b"multiples of the group"),
    (dict(fmt=BF16, H=12), b"hidden"), (dict(fmt=BF16, I=12), b"intermediate"), (dict(fmt=E4M3, H=64, I=128), b"128"),
    (dict(H=32800), b"hidden"), (dict(I=32800), b"intermediate"),
    (dict(x=N), b"x must"), (dict(x=A + 8), b"x must"), (dict(idx=N), b"topk_idx"), (dict(values=N), b"values"), (dict(values=A + 8), b"values"),
    (dict(scales=N), b"scales"), (dict(scales=A + 8), b"scales"), (dict(fmt=E4M3, H=128, I=128, scales=N), b"scales"),
    (dict(bias=A + 2), b"bias"), (dict(out=N), b"out must"), (dict(out=B + 8), b"out must"),
    (dict(ws=N), b"workspace"), (dict(ws=B + 16), b"256-byte"), (dict(nws=8 * 64 * 2 - 1), b"workspace_bytes"),
])
def test_few_refusals(kw, why):
    assert few(**kw) == 1 and why in L.ep_last_error()


def test_few_needs_weights():
    assert L.ep_moe_few(A, A, A, 4, 2, 8, 1, 0, 64, 32, None, weights(), None, B, B, 1 << 20, None) == 1
    assert b"non-NULL" in L.ep_last_error()


def test_few_workspace_bytes():
    f = L.ep_moe_few_workspace_bytes
    assert f(0, 1, 64) == 256 and f(1, 8, 2048) == 8 * 4096 and f(128, 8, 8) == 1024 * 128
    assert f(129, 1, 64) == f(128, 9, 64) == f(-1, 1, 64) == f(1, 0, 64) == f(1, 1, 12) == f(1, 1, 0) == f(1, 1, 32776) == 0


def test_ffn_w4_refuses_a_dead_handle():
    assert L.ep_expert_ffn_w4(0x1234, A, 64, 32, 4, weights(), weights(), B, B, 1 << 20, None) == 1 and b"handle" in L.ep_last_error()


def test_binding_refusals():
    codes, scales = torch.zeros(2, 32, 32, dtype=torch.uint8), torch.ones(2, 32, 2, dtype=torch.bfloat16)
    for a, what in (((codes, scales, "int3"), ValueError), ((codes[0], scales, "int4"), ValueError), ((codes, scales[0], "int4"), ValueError),
                    ((codes.int(), scales, "int4"), TypeError), ((codes, scales.float(), "int4"), TypeError),
                    ((codes, scales[:, :16], "int4"), ValueError), ((codes, scales[:, :, :0], "int4"), ValueError),
                    ((codes, torch.ones(2, 32, 3, dtype=torch.bfloat16), "int4"), ValueError),
                    ((codes, torch.ones(2, 32, 4, dtype=torch.bfloat16), "int4"), ep.EPError), ((codes, scales, "int4"), ValueError)):
        with pytest.raises(what):
            ep.ep_w4_pack(*a)
    x, idx = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int64)
    w13, w2 = torch.zeros(2, 64, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 32, dtype=torch.bfloat16)
    base = dict(x=x, topk_idx=idx, topk_weights=None, w13=w13, w2=w2)
    for kw, what in ((dict(x=x.float()), TypeError), (dict(x=x[0]), ValueError), (dict(topk_idx=idx.int()), TypeError),
                     (dict(topk_idx=idx[:3]), ValueError), (dict(topk_weights=torch.ones(4, 3)), ValueError), (dict(bias=x[:1]), ValueError),
                     (dict(w2=w2[0]), ValueError), (dict(w2=None), ValueError), (dict(w13=None), ValueError), (dict(w13=w13[:, :32]), ValueError),
                     (dict(w2=w2.float()), TypeError), (dict(w13=w13.to(torch.uint8)), TypeError),
                     (dict(w13=w13.to(torch.uint8), w2=w2.to(torch.uint8)), ValueError), (dict(num_experts=3), ValueError),
                     (dict(num_ranks=0), ValueError), (dict(out=x.float()), TypeError), (dict(workspace=torch.zeros(4)), TypeError),
                     (dict(), ValueError)):
        with pytest.raises(what):
            ep.ep_moe_few(**{**base, **kw})
    # the scales of e4m3 weights
    e13, e2 = torch.zeros(2, 256, 128, dtype=torch.uint8), torch.zeros(2, 128, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="w13_scales"):
        ep.ep_moe_few(torch.zeros(4, 128, dtype=torch.bfloat16), idx, None, e13, e2)
