"""Refusals of ep_combine_norm and its gradient: every argument is checked on the host before anything is enqueued.  The device
addresses below are never dereferenced."""
import ctypes
import math

import pytest
import torch

import combine_get_dispatch_03_amd as ep

L = ep._lib
A, B = 0x100000, 0x200000
N = None


def norm(**kw):
    a = ep._NormArgs(residual=A, post_weight=A, pre_weight=A, gate=A, residual_scale=1.0, eps=1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def forward(h=N, y=A, H=64, rows=4, w=N, bias=N, n=norm, out=B, normed=B, kept=N, **kw):
    return L.ep_combine_norm(h, y, H, rows, w, bias, n(**kw) if callable(n) else n, out, normed, kept, None)


def backward(do=A, dn=A, f=A, kind=0, T=4, H=64, gf=B, gr=B, gpost=B, gpre=B, gg=B, ws=B, nws=1 << 30, n=norm, **kw):
    return L.ep_combine_norm_backward(do, dn, f, kind, T, H, n(**kw) if callable(n) else n, gf, gr, gpost, gpre, gg, ws, nws, None)


@pytest.mark.parametrize("kw,why", [
    (dict(h=0x1234), b"invalid handle"),
    (dict(H=12), b"hidden"), (dict(H=0), b"hidden"), (dict(H=32776), b"hidden"),
    (dict(rows=-1), b"y_rows"), (dict(rows=1000000001), b"y_rows"),
    (dict(w=A), b"handle"),
    (dict(n=N), b"norm is NULL"),
    (dict(eps=0.0), b"eps"), (dict(eps=-1.0), b"eps"), (dict(eps=math.nan), b"eps"), (dict(eps=math.inf), b"eps"),
    (dict(residual_scale=math.inf), b"residual_scale"), (dict(residual_scale=math.nan), b"residual_scale"),
    (dict(residual=A + 8), b"aligned"), (dict(post_weight=A + 4), b"aligned"), (dict(pre_weight=A + 2), b"aligned"), (dict(gate=A + 8), b"aligned"),
    (dict(out=N, normed=N), b"all NULL"), (dict(pre_weight=N), b"pre_weight"),
    (dict(y=N), b"y must"), (dict(y=A + 8), b"y must"), (dict(bias=A + 2), b"bias"),
    (dict(out=B + 8), b"aligned"), (dict(normed=B + 8), b"aligned"), (dict(kept=B + 4), b"aligned"),
])
def test_forward_refusals(kw, why):
    assert forward(**kw) == 1 and why in L.ep_last_error()


@pytest.mark.parametrize("kw,why", [
    (dict(T=-1), b"num_tokens"), (dict(T=1000000001), b"num_tokens"), (dict(H=4), b"hidden"), (dict(kind=2), b"f_type"),
    (dict(n=N), b"norm is NULL"), (dict(eps=0.0), b"eps"),
    (dict(gf=N, gr=N, gpost=N, gpre=N, gg=N), b"no gradient"),
    (dict(pre_weight=N), b"pre_weight"), (dict(dn=N), b"grad_pre"), (dict(post_weight=N), b"grad_post"), (dict(gate=N), b"grad_gate"),
    (dict(residual=N), b"grad_residual"),
    (dict(gf=B + 8), b"aligned"), (dict(gr=B + 8), b"aligned"), (dict(gg=B + 4), b"aligned"),
    (dict(do=N, dn=N, gpre=N), b"both NULL"), (dict(do=A + 8), b"aligned"), (dict(dn=A + 8), b"aligned"),
    (dict(f=N), b"f must"), (dict(f=A + 8), b"f must"),
    (dict(ws=N), b"workspace"), (dict(ws=B + 16), b"256-byte"), (dict(nws=4 * 3 * 64 * 4 - 1), b"workspace_bytes"),
])
def test_backward_refusals(kw, why):
    assert backward(**kw) == 1 and why in L.ep_last_error()


def test_workspace_bytes():
    f = L.ep_combine_norm_workspace_bytes
    assert f(0, 64) == f(1, 64) == 3 * 64 * 4 and f(4, 64) == 4 * 3 * 64 * 4
    assert f(1000000000, 32768) < 1 << 30
    assert f(-1, 64) == f(4, 12) == f(4, 0) == f(4, 32776) == f(1000000001, 64) == 0


def test_binding_refusals():
    y = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    for kw, what in ((dict(y=y.float()), TypeError), (dict(y=y[0]), ValueError), (dict(topk_weights=w), ValueError),
                     (dict(post_weight=w.double()), TypeError), (dict(post_weight=w, pre_weight=w.bfloat16()), TypeError),
                     (dict(gate=torch.ones(4, 64)), TypeError), (dict(gate=torch.ones(3, 64, dtype=torch.bfloat16)), ValueError),
                     (dict(gate="x"), TypeError), (dict(pre_weight=w[:32]), ValueError), (dict(residual=y[:2]), ValueError),
                     (dict(bias=y.float()), TypeError), (dict(out=y[:1]), ValueError)):
        with pytest.raises(what):
            ep.ep_combine_norm(None, **{"y": y, **kw})
    for kw, what in ((dict(f=y.double()), TypeError), (dict(grad_out=y[:2]), ValueError), (dict(grad_normed=y.float()), TypeError)):
        with pytest.raises(what):
            ep.ep_combine_norm_backward(**{"grad_out": y, "grad_normed": None, "f": y, **kw})
