"""CPU checks of what the expert block, its gradients, the combine's gradient and the adapters refuse: the C ABI's host
checks that need no live handle, and the binding's checks of every tensor before any library call (host tensors stand
in for device tensors, a Handle without a library object for a layout)."""
import ctypes

import pytest
import torch

import combine_get_dispatch_03_amd as ep
from combine_get_dispatch_03_amd import _lib

P = ctypes.c_void_p
T, K, E, H, I, A = 10, 2, 4, 256, 128, 16
CAP = T * K + E * (A - 1)
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def handle(topk=K, tokens=T, experts=E):
    return ep.Handle(None, torch.zeros(tokens, topk, dtype=torch.int64), None, tokens, topk, experts, 1, 0, A)


def test_workspace_bytes():
    f = _lib.ep_expert_ffn_workspace_bytes
    assert f(1000, H, I, 0) >= 1000 * I * 2
    assert f(1000, H, I, 1) >= 1000 * I * 6
    assert f(0, H, I, 0) > 0
    for bad in ((-1, H, I), (1 << 31, H, I), (10, 0, I), (10, 12, I), (10, 32776, I), (10, H, 0), (10, H, 4), (10, H, 32776)):
        assert f(*bad, 0) == 0
    f = _lib.ep_adapter_workspace_bytes
    assert f(0, 1, 8, 8) > 0 and f(4096, 1024, 32768, 128) > 0
    for bad in ((-1, 1, 64, 8), (4, 0, 64, 8), (4, 1025, 64, 8), (4, 1, 60, 8), (4, 1, 64, 0), (4, 1, 64, 12), (4, 1, 64, 136)):
        assert f(*bad) == 0


def test_bad_handles_are_refused_before_anything():
    junk = (ctypes.c_uint32 * 64)()
    for h in (None, P(0x10), ctypes.cast(junk, P)):
        for rc in (_lib.ep_expert_ffn(h, None, None, 0, H, I, CAP, None, None, None, None, None, None, None, 0, None),
                   _lib.ep_expert_ffn_backward(h, None, None, None, H, I, CAP, None, None, None, None, None, None, 0, None),
                   _lib.ep_combine_backward(h, None, H, None, CAP, None, None, None, None),
                   _lib.ep_adapter(h, None, H, None, None, 8, 8, None, None, None, None, 0, None)):
            assert rc == 1
            assert b"handle" in _lib.ep_last_error()


def bf(*s):
    return torch.zeros(*s, dtype=BF)


def ffn_args(**over):
    a = dict(recv_x=bf(CAP, H), w13=bf(E, 2 * I, H), w2=bf(E, H, I))
    a.update(over)
    return a


@pytest.mark.parametrize("over,err,match", [
    (dict(recv_x=torch.zeros(CAP, H)), TypeError, "recv_x"),
    (dict(recv_x=None), TypeError, "recv_x"),
    (dict(recv_x=bf(CAP * H)), ValueError, "recv_x"),
    (dict(recv_x=bf(CAP, 2 * H)[:, ::2]), ValueError, "contiguous"),
    (dict(w13=None), ValueError, "w13"),
    (dict(w13=bf(E, I, H)), ValueError, "w13"),
    (dict(w13=bf(E, H, 2 * I).transpose(1, 2)), ValueError, "contiguous"),
    (dict(w13=bf(E - 1, 2 * I, H)), ValueError, "w13"),
    (dict(w13=torch.zeros(E, 2 * I, H)), TypeError, "w13"),
    (dict(w2=bf(E, I, H + 8)), ValueError, "w2"),
    (dict(w2=bf(H, I)), ValueError, "w2"),
    (dict(y=bf(CAP - 1, H)), ValueError, "y must have shape"),
    (dict(y=torch.zeros(CAP, H)), TypeError, "y must be"),
    (dict(pre=bf(CAP, 2 * I)), TypeError, "pre"),
    (dict(pre=torch.zeros(CAP, I)), ValueError, "pre"),
    (dict(workspace=torch.zeros(16)), TypeError, "workspace"),
    (dict(workspace=torch.zeros(4, 4, dtype=U8)), ValueError, "workspace"),
    (dict(recv_x=torch.zeros(CAP, H, dtype=U8)), TypeError, "w2 must be torch.uint8"),
])
def test_ffn_refuses(over, err, match):
    a = ffn_args(**over)
    with pytest.raises(err, match=match):
        ep.ep_expert_ffn(handle(), a.pop("recv_x"), a.pop("w13"), a.pop("w2"), **a)


@pytest.mark.parametrize("missing", ["recv_x_scales", "w13_scales", "w2_scales"])
def test_ffn_fp8_needs_scales(missing):
    q = lambda *s: torch.zeros(*s, dtype=U8)
    s = dict(recv_x_scales=torch.zeros(CAP, H // 128), w13_scales=torch.zeros(E, 2 * I // 128, H // 128),
             w2_scales=torch.zeros(E, H // 128, I // 128))
    with pytest.raises(ValueError, match=missing):
        ep.ep_expert_ffn(handle(), q(CAP, H), q(E, 2 * I, H), q(E, H, I), **dict(s, **{missing: None}))
    short = s[missing].narrow(s[missing].dim() - 1, 0, s[missing].shape[-1] - 1) if s[missing].shape[-1] > 1 else s[missing][:-1]
    with pytest.raises(ValueError, match=missing):
        ep.ep_expert_ffn(handle(), q(CAP, H), q(E, 2 * I, H), q(E, H, I), **dict(s, **{missing: short.contiguous()}))


@pytest.mark.parametrize("over,err,match", [
    (dict(dy=torch.zeros(CAP, H)), TypeError, "dy"),
    (dict(recv_x=None), ValueError, "dw13 needs recv_x"),
    (dict(recv_x=bf(CAP - 1, H)), ValueError, "recv_x"),
    (dict(pre=None), TypeError, "pre"),
    (dict(pre=bf(CAP, 2 * I)), TypeError, "pre"),
    (dict(w13=None), ValueError, "dx needs w13"),
    (dict(w2=bf(E, H + 8, I)), ValueError, "w2"),
    (dict(dx=bf(CAP - 1, H)), ValueError, "dx"),
    (dict(dw13=torch.zeros(E, 2 * I, H)), TypeError, "dw13"),
    (dict(dw2=bf(E, I, H)), ValueError, "dw2"),
])
def test_ffn_backward_refuses(over, err, match):
    a = dict(dy=bf(CAP, H), recv_x=bf(CAP, H), pre=torch.zeros(CAP, 2 * I), w13=bf(E, 2 * I, H), w2=bf(E, H, I))
    a.update(over)
    with pytest.raises(err, match=match):
        ep.ep_expert_ffn_backward(handle(), a.pop("dy"), a.pop("recv_x"), a.pop("pre"), a.pop("w13"), a.pop("w2"), **a)


@pytest.mark.parametrize("over,err,match", [
    (dict(grad_out=bf(T + 1, H)), ValueError, "grad_out"),
    (dict(grad_out=torch.zeros(T, H)), TypeError, "grad_out"),
    (dict(y=None), ValueError, "needs y"),
    (dict(y=bf(CAP, H + 8)), ValueError, "y must be"),
    (dict(topk_weights=torch.zeros(T, K + 1)), ValueError, "topk_weights"),
    (dict(topk_weights=bf(T, K)), TypeError, "topk_weights"),
    (dict(grad_y=bf(CAP - 1, H)), ValueError, "grad_y"),
    (dict(grad_topk_weights=bf(T, K)), TypeError, "grad_topk_weights"),
])
def test_combine_backward_refuses(over, err, match):
    a = dict(grad_out=bf(T, H), y=bf(CAP, H))
    a.update(over)
    with pytest.raises(err, match=match):
        ep.ep_combine_backward(handle(), a.pop("grad_out"), a.pop("y"), **a)


@pytest.mark.parametrize("over,err,match", [
    (dict(x=bf(T - 1, H)), ValueError, "x must have shape"),
    (dict(x=torch.zeros(T, H)), TypeError, "x must be"),
    (dict(a=bf(E, 16, H + 8)), ValueError, "a must"),
    (dict(a=bf(E, 8, H)), ValueError, "a must"),
    (dict(b=bf(E, 16)), ValueError, "b must"),
    (dict(b=bf(E, 16, 40).transpose(1, 2)), ValueError, "contiguous"),
    (dict(scales=bf(E)), TypeError, "scales"),
    (dict(scales=torch.zeros(E + 1)), ValueError, "scales"),
    (dict(base=bf(T, 48)), ValueError, "base"),
    (dict(out=torch.zeros(T, 40)), TypeError, "out"),
    (dict(workspace=torch.zeros(8, dtype=torch.int32)), TypeError, "workspace"),
    (dict(a=bf(E, 12, H), b=bf(E, 40, 12)), ep.EPError, "rank=12"),
])
def test_adapter_refuses(over, err, match):
    a = dict(x=bf(T, H), a=bf(E, 16, H), b=bf(E, 40, 16))
    a.update(over)
    with pytest.raises(err, match=match):
        ep.ep_adapter(handle(topk=1), a.pop("x"), a.pop("a"), a.pop("b"), **a)


def test_tensors_on_another_device_are_refused():
    h = handle()
    h.topk_idx = torch.empty((T, K), dtype=torch.int64, device="meta")
    with pytest.raises(ValueError, match="must be on meta"):
        ep.ep_expert_ffn(h, bf(CAP, H), bf(E, 2 * I, H), bf(E, H, I))
