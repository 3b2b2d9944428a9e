"""Sizes past which a kernel's grid would hold more than 2^32 threads are refused on the host."""
import ctypes

from combine_get_dispatch_03_amd import _lib

P = ctypes.c_void_p
MOST = 1_000_000_000       # tokens; the layout's grids take 1024 threads for 256 of them


def test_number_of_tokens():
    h = P()
    layout = lambda T: _lib.ep_get_layout(P(0x10000), T, 1, 2, 1, 0, 1, P(0x100000), 0, None, None, None, None, None, ctypes.byref(h), None)
    for T in (MOST + 1, 1 << 30, (1 << 31) - 1):
        assert layout(T) == 1 and b"num_tokens" in _lib.ep_last_error()
        assert _lib.ep_layout_workspace_bytes(T, 1, 2, 1, 1) == 0
        assert _lib.ep_recv_capacity(T, 1, 2, 1) == -1
        assert _lib.ep_adapter_workspace_bytes(T, 2, 64, 8) == 0
    assert layout(MOST) == 1 and b"workspace_bytes" in _lib.ep_last_error()      # past the size checks
    assert _lib.ep_layout_workspace_bytes(MOST, 1, 2, 1, 1) > 4 * MOST
    assert _lib.ep_recv_capacity(MOST, 1, 2, 1) == MOST
    assert _lib.ep_adapter_workspace_bytes(MOST, 2, 64, 8) > 32 * MOST
