"""What the library refuses for a live handle, with nothing enqueued and no output touched: short or misaligned
buffers, sizes outside the limits, formats without their scales, a handle that routes a token to several adapters."""
import ctypes

import pytest
import torch

import combine_get_dispatch_03_amd as ep
from combine_get_dispatch_03_amd import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
T, K, E, H, I, A = 20, 2, 4, 128, 128, 16


@pytest.fixture(scope="module")
def live():
    idx = torch.randint(0, E, (T, K), device=DEV)
    h, _ = ep.ep_get_layout(idx, E, expert_alignment=A)
    buf = torch.full((1 << 22,), 7.0, device=DEV)      # one block stands in for every buffer
    yield h, buf
    torch.cuda.synchronize()
    assert bool((buf == 7.0).all()), "a refused call wrote something"


def refused(rc, why, status=1):
    assert rc == status, (rc, _lib.ep_last_error())
    assert why in _lib.ep_last_error(), _lib.ep_last_error()


def test_ffn(live):
    h, buf = live
    p, cap, none = buf.data_ptr(), h.recv_capacity, None

    def call(x=p, xs=p, dtype=0, hid=H, inter=I, rows=cap, w13=p, s13=p, w2=p, s2=p, y=p, pre=none, ws=p, n=1 << 24):
        return _lib.ep_expert_ffn(h.ptr, x, xs, dtype, hid, inter, rows, w13, s13, w2, s2, y, pre, ws, n, none)

    refused(call(x=none), b"recv_x")
    refused(call(x=p + 8), b"recv_x")
    refused(call(rows=cap - 1), b"rows")
    refused(call(dtype=2), b"dtype")
    refused(call(hid=100), b"hidden")
    refused(call(hid=0), b"hidden")
    refused(call(hid=32776), b"hidden")
    refused(call(inter=4), b"intermediate")
    refused(call(inter=32776), b"intermediate")
    refused(call(dtype=1, inter=136), b"FP8")
    refused(call(dtype=1, xs=none), b"scales")
    refused(call(dtype=1, s13=none), b"scales")
    refused(call(dtype=1, s2=none), b"scales")
    refused(call(dtype=1, pre=p), b"pre")
    refused(call(pre=p + 4), b"pre")
    refused(call(w13=none), b"w13")
    refused(call(w2=p + 2), b"w2")
    refused(call(y=none), b"y must")
    refused(call(ws=none), b"workspace")
    refused(call(ws=p + 16), b"256-byte")
    refused(call(n=cap * I * 2 - 1), b"workspace_bytes")


def test_ffn_backward(live):
    h, buf = live
    p, cap, none = buf.data_ptr(), h.recv_capacity, None

    def call(dy=p, x=p, pre=p, hid=H, inter=I, rows=cap, w13=p, w2=p, dx=p, dw13=p, dw2=p, ws=p, n=1 << 24):
        return _lib.ep_expert_ffn_backward(h.ptr, dy, x, pre, hid, inter, rows, w13, w2, dx, dw13, dw2, ws, n, none)

    refused(call(dy=none), b"dy")
    refused(call(x=none), b"recv_x")
    refused(call(pre=none), b"pre")
    refused(call(w13=none), b"w13")
    refused(call(w2=none), b"w2")
    refused(call(hid=12), b"hidden")
    refused(call(inter=12), b"intermediate")
    refused(call(rows=cap - 1), b"rows")
    refused(call(dx=none, dw13=none, dw2=none), b"all NULL")
    refused(call(dx=p + 8), b"dx")
    refused(call(ws=none), b"workspace")
    refused(call(n=cap * I * 6 - 1), b"workspace_bytes")


def test_combine_backward(live):
    h, buf = live
    p, cap, none = buf.data_ptr(), h.recv_capacity, None

    def call(g=p, hid=H, y=p, rows=cap, w=p, gy=p, gw=p):
        return _lib.ep_combine_backward(h.ptr, g, hid, y, rows, w, gy, gw, none)

    refused(call(g=none), b"grad_out")
    refused(call(g=p + 2), b"grad_out")
    refused(call(hid=4), b"hidden")
    refused(call(y=none), b"y must")
    refused(call(rows=cap - 1), b"y_rows")
    refused(call(gy=none, gw=none), b"both NULL")
    refused(call(gy=p + 8), b"grad_y")


def test_adapter(live):
    h2, buf = live
    ids = torch.randint(0, E, (T, 1), device=DEV)
    h, _ = ep.ep_get_layout(ids, E)
    p, none = buf.data_ptr(), None

    def call(handle=h, x=p, hid=H, a=p, b=p, r=16, n=64, s=p, base=p, out=p, ws=p, nb=1 << 24):
        return _lib.ep_adapter(handle.ptr, x, hid, a, b, r, n, s, base, out, ws, nb, none)

    refused(call(handle=h2), b"num_topk", status=2)
    refused(call(x=none), b"x must")
    refused(call(hid=12), b"hidden")
    refused(call(r=12), b"rank")
    refused(call(r=0), b"rank")
    refused(call(r=136), b"rank")
    refused(call(n=12), b"out_features")
    refused(call(n=65544), b"out_features")
    refused(call(a=none), b"a and b")
    refused(call(b=p + 8), b"a and b")
    refused(call(base=p + 8), b"base")
    refused(call(out=none), b"out")
    refused(call(ws=none), b"workspace")
    refused(call(ws=p + 128), b"256-byte")
    refused(call(nb=0), b"workspace_bytes")


def test_freed_handle(live):
    h, _ = ep.ep_get_layout(torch.zeros((T, 1), dtype=torch.int64, device=DEV), E)
    ptr = ctypes.c_void_p(h.ptr.value)
    h.free()
    refused(_lib.ep_combine_backward(ptr, None, H, None, 0, None, None, None, None), b"handle")
