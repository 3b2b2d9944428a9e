"""An empty batch through the gradient of ep_combine_norm: whatever is asked for, there is nothing to do for its rows.  (Empty
tensors have no address, so a call for rows alone arrives with every gradient NULL.)  Nothing here reaches the GPU."""
import ctypes

import pytest

import combine_get_dispatch_03_amd as ep

L = ep._lib
A, N = 0x100000, None


def backward(T, **kw):
    a = ep._NormArgs(residual_scale=1.0, eps=1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return L.ep_combine_norm_backward(N, N, N, 0, T, 64, ctypes.byref(a), N, N, N, N, N, A, 1 << 20, N)


@pytest.mark.parametrize("kw", [dict(), dict(post_weight=A, pre_weight=A), dict(gate_per_token=1), dict(gate=A)])
def test_rows_of_an_empty_batch(kw):
    assert backward(0, **kw) == ep.EP_OK, L.ep_last_error()


def test_rows_that_are_there_need_a_gradient():
    assert backward(1) == 1 and b"no gradient" in L.ep_last_error()
