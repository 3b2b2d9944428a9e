"""Python binding of libep_mi355x.so (include/ep.h): MoE expert-parallel layout, dispatch and combine on one
MI355X (gfx950) GPU.

The functions keep the C names (ep_get_layout, ep_dispatch, ep_layout_dispatch, ep_combine, ep_combine_tokens,
ep_dispatch_rows, ep_combine_reduce, ep_expert_ffn, ep_expert_ffn_backward, ep_combine_backward, ep_adapter,
ep_handle_free, ep_recv_capacity and the ep_*_workspace_bytes).  They only marshal arguments: tensors become device pointers, the stream is
torch's current HIP stream, and output tensors are allocated by torch when the caller does not pass them.
Every step of the path runs in the HIP kernels of the library; there is no other implementation, and if
the library is not built or cannot be loaded the import of this binding fails.

    h, lay = ep_get_layout(topk_idx, num_experts=256, expert_alignment=128)
    d = ep_dispatch(h, x, topk_weights, fp8=True, do_zero_padding=True)
    y = ep_expert_ffn(h, d["recv_x"], w13, w2, d["recv_x_scales"], w13_scales, w2_scales)
    out = ep_combine(h, y, topk_weights, bias=None)
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libep_mi355x.so")

EP_OK = 0
EP_DTYPE_BF16 = 0
EP_DTYPE_FP8_E4M3 = 1
EP_WEIGHTS_BF16, EP_WEIGHTS_E4M3, EP_WEIGHTS_INT4, EP_WEIGHTS_E2M1 = 0, 1, 2, 3
_W4_KINDS = {"int4": EP_WEIGHTS_INT4, "e2m1": EP_WEIGHTS_E2M1}


class EPError(RuntimeError):
    pass


class _DispatchOut(ctypes.Structure):
    _fields_ = [
        ("recv_x", ctypes.c_void_p), ("recv_x_scales", ctypes.c_void_p), ("recv_src_idx", ctypes.c_void_p),
        ("recv_topk_weights", ctypes.c_void_p), ("recv_topk_idx", ctypes.c_void_p),
        ("recv_capacity", ctypes.c_int64),
        ("send_x", ctypes.c_void_p), ("send_x_scales", ctypes.c_void_p), ("send_src_idx", ctypes.c_void_p),
        ("send_topk_idx", ctypes.c_void_p), ("send_topk_weights", ctypes.c_void_p),
    ]


class _Weights(ctypes.Structure):
    _fields_ = [("values", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("format", ctypes.c_int), ("group", ctypes.c_int)]


class _NormArgs(ctypes.Structure):
    _fields_ = [
        ("residual", ctypes.c_void_p), ("post_weight", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p),
        ("gate", ctypes.c_void_p), ("gate_per_token", ctypes.c_int), ("vectors_bf16", ctypes.c_int),
        ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float),
    ]


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libep_mi355x.so is not built: run `python -m combine_get_dispatch_03_amd.build` "
                          "(or __graft_entry__.build())")
    # torch is imported first, so the HIP runtime the library links (soname libamdhip64.so.7) resolves to the
    # one torch already loaded: streams and device pointers then belong to the same runtime.
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.ep_recv_capacity.restype = I64
    lib.ep_recv_capacity.argtypes = [I, I, I, I]
    lib.ep_layout_workspace_bytes.restype = SZ
    lib.ep_layout_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.ep_status_string.restype = ctypes.c_char_p
    lib.ep_status_string.argtypes = [I]
    lib.ep_last_error.restype = ctypes.c_char_p
    lib.ep_last_error.argtypes = []
    lib.ep_get_layout.restype = I
    lib.ep_get_layout.argtypes = [P, I, I, I, I, I, I, P, SZ, P, P, P, P, P, ctypes.POINTER(P), P]
    lib.ep_dispatch.restype = I
    lib.ep_dispatch.argtypes = [P, P, I, P, I, I, I, ctypes.POINTER(_DispatchOut), P]
    lib.ep_combine.restype = I
    lib.ep_combine.argtypes = [P, P, I, I64, P, P, P, P]
    lib.ep_handle_free.restype = I
    lib.ep_handle_free.argtypes = [P]
    lib.ep_dispatch_rows.restype = I
    lib.ep_dispatch_rows.argtypes = [P, P, I, P, I, P, I, ctypes.POINTER(_DispatchOut), P]
    lib.ep_combine_reduce.restype = I
    lib.ep_combine_reduce.argtypes = [P, P, I, P, P, P, P]
    lib.ep_combine_tokens.restype = I
    lib.ep_combine_tokens.argtypes = [P, P, I, I64, P, P, P]
    lib.ep_layout_dispatch_noalloc.restype = I
    lib.ep_layout_dispatch_noalloc.argtypes = [P, I, I, I, I, I, I, P, P, P, P, P, P, I, P, I, I, I,
                                               ctypes.POINTER(_DispatchOut), ctypes.POINTER(P), P]
    lib.ep_layout_dispatch.restype = I
    lib.ep_layout_dispatch.argtypes = [P, I, I, I, I, I, I, P, SZ, P, P, P, P, P, P, I, P, I, I, I,
                                       ctypes.POINTER(_DispatchOut), ctypes.POINTER(P), P]
    lib.ep_combine_backward.restype = I
    lib.ep_combine_backward.argtypes = [P, P, I, P, I64, P, P, P, P]
    lib.ep_expert_ffn_workspace_bytes.restype = SZ
    lib.ep_expert_ffn_workspace_bytes.argtypes = [I64, I, I, I]
    lib.ep_expert_ffn.restype = I
    lib.ep_expert_ffn.argtypes = [P, P, P, I, I, I, I64, P, P, P, P, P, P, P, SZ, P]
    lib.ep_expert_ffn_backward.restype = I
    lib.ep_expert_ffn_backward.argtypes = [P, P, P, P, I, I, I64, P, P, P, P, P, P, SZ, P]
    lib.ep_adapter_workspace_bytes.restype = SZ
    lib.ep_adapter_workspace_bytes.argtypes = [I, I, I, I]
    lib.ep_adapter.restype = I
    lib.ep_adapter.argtypes = [P, P, I, P, P, I, I, P, P, P, P, SZ, P]
    W = ctypes.POINTER(_Weights)
    lib.ep_w4_packed_bytes.restype = SZ
    lib.ep_w4_packed_bytes.argtypes = [I, I, I, I]
    lib.ep_w4_packed_scale_bytes.restype = SZ
    lib.ep_w4_packed_scale_bytes.argtypes = [I, I, I, I]
    lib.ep_w4_pack.restype = I
    lib.ep_w4_pack.argtypes = [P, P, I, I, I, I, I, P, P, P]
    lib.ep_expert_ffn_w4.restype = I
    lib.ep_expert_ffn_w4.argtypes = [P, P, I, I, I64, W, W, P, P, SZ, P]
    lib.ep_moe_few_workspace_bytes.restype = SZ
    lib.ep_moe_few_workspace_bytes.argtypes = [I, I, I]
    lib.ep_moe_few.restype = I
    lib.ep_moe_few.argtypes = [P, P, P, I, I, I, I, I, I, I, W, W, P, P, P, SZ, P]
    lib.ep_combine_norm_workspace_bytes.restype = SZ
    lib.ep_combine_norm_workspace_bytes.argtypes = [I, I]
    lib.ep_combine_norm.restype = I
    lib.ep_combine_norm.argtypes = [P, P, I, I64, P, P, ctypes.POINTER(_NormArgs), P, P, P, P]
    lib.ep_combine_norm_backward.restype = I
    lib.ep_combine_norm_backward.argtypes = [P, P, P, I, I, I, ctypes.POINTER(_NormArgs), P, P, P, P, P, P, SZ, P]
    return lib


_lib = _load_library()


def hip_runtimes_loaded() -> list[str]:
    """Paths of the libamdhip64 copies mapped into this process (exactly one is expected)."""
    paths = set()
    with open("/proc/self/maps") as f:
        for line in f:
            if "libamdhip64" in line:
                paths.add(line.split()[-1])
    return sorted(paths)


def _check(status: int, what: str):
    if status != EP_OK:
        msg = _lib.ep_last_error().decode(errors="replace")
        raise EPError("%s failed: %s (%s)" % (what, _lib.ep_status_string(status).decode(), msg))


def _ptr(t):
    # a plain int: the c_void_p argument types convert it (cheaper than building a c_void_p per pointer)
    return None if t is None else t.data_ptr()


# torch's current raw stream without building a Stream object (~0.2 us instead of ~2.5 us per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    """HIP stream handle: the given torch stream's, else torch's current stream on the current device."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _cur_device is not None:
        return _raw_stream(_cur_device())
    return torch.cuda.current_stream().cuda_stream


def _on_stream(stream, fn, *args, **kw):
    """Run an allocating helper with `stream` current, so that the tensors it makes belong to the stream the
    call's kernels write them on: torch's caching allocator hands a freed block to later work of the block's
    own stream only, which then is ordered after those kernels.  stream=None: torch's current stream, where
    the kernels run anyway."""
    if stream is None:
        return fn(*args, **kw)
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _need(t, dtype, name, device=None, shape=None):
    """t must be a contiguous tensor of `dtype` and `shape` (when given) on `device` (when given; else on a GPU).
    The shape is checked before the placement, so the shape rules can be exercised without a GPU."""
    # one expression for the common (valid) case; the checks below only name what is wrong
    if (type(t) is torch.Tensor and t.dtype is dtype and (shape is None or t.shape == shape)
            and (t.device == device if device is not None else t.is_cuda) and t.is_contiguous()):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if device is not None:
        if t.device != device:
            raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    elif not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _opt(out, key, dtype, shape, device):
    """An optional output: absent/None, or exactly dtype/shape on device."""
    t = out.get(key)
    if t is not None:
        _need(t, dtype, key, device, shape)


def check_layout_outputs(outputs, T, E, R, device):
    """Caller-supplied layout outputs (any entry may be None): the sizes the library writes."""
    El = E // R
    _opt(outputs, "num_tokens_per_rank", torch.int32, (R,), device)
    _opt(outputs, "num_tokens_per_expert", torch.int32, (E,), device)
    _opt(outputs, "is_token_in_rank", torch.uint8, (T, R), device)
    _opt(outputs, "psum_num_recv_tokens_per_expert", torch.int32, (El + 1,), device)
    _opt(outputs, "num_invalid_topk", torch.int32, (1,), device)


def check_workspace(workspace, device):
    """A caller's workspace: one contiguous uint8 buffer on the device (its length is checked by the library)."""
    _need(workspace, torch.uint8, "workspace", device)
    if workspace.dim() != 1:
        raise ValueError("workspace must be a 1-D uint8 tensor")


def check_dispatch_outputs(out, T, K, R, hidden, fp8, do_expand, device):
    """Every dispatch output the library will write, against the sizes it writes: recv_x [cap, hidden] (e4m3
    bytes or bf16) with every other recv array on the same cap rows, the send windows [R, T, ...].  Returns cap
    (the recv_capacity passed to the library, which checks it against the layout's bound)."""
    if not isinstance(out, dict) or out.get("recv_x") is None:
        raise ValueError("out must be a dict holding recv_x")
    rx = out["recv_x"]
    xdt = torch.uint8 if fp8 else torch.bfloat16
    if not isinstance(rx, torch.Tensor) or rx.dim() != 2:
        raise ValueError("recv_x must be a 2-D tensor [rows, hidden]")
    cap = rx.shape[0]
    _need(rx, xdt, "recv_x", device, (cap, hidden))
    if fp8:
        if out.get("recv_x_scales") is None:
            raise ValueError("FP8 dispatch needs recv_x_scales")
        _need(out["recv_x_scales"], torch.float32, "recv_x_scales", device, (cap, hidden // 128))
    _opt(out, "recv_src_idx", torch.int32, (cap,), device)
    _opt(out, "recv_topk_weights", torch.float32, (cap,) if do_expand else (T, K), device)
    if not do_expand:
        _opt(out, "recv_topk_idx", torch.int64, (T, K), device)
    if R > 1:
        if out.get("send_x") is None:
            raise ValueError("num_ranks > 1 needs send_x")
        _need(out["send_x"], xdt, "send_x", device, (R, T, hidden))
        if fp8:
            if out.get("send_x_scales") is None:
                raise ValueError("num_ranks > 1 with FP8 needs send_x_scales")
            _need(out["send_x_scales"], torch.float32, "send_x_scales", device, (R, T, hidden // 128))
        _opt(out, "send_src_idx", torch.int32, (R, T), device)
        _opt(out, "send_topk_idx", torch.int64, (R, T, K), device)
        _opt(out, "send_topk_weights", torch.float32, (R, T, K), device)
    return cap


def check_rows_outputs(out, row_dtype, row_elems, G, device):
    """Outputs of ep_dispatch_rows: recv_x [cap, row_elems] of the rows' dtype, scales [cap, G] when G > 0, and
    the optional per-row metadata on the same cap rows.  Returns cap."""
    if not isinstance(out, dict) or out.get("recv_x") is None:
        raise ValueError("out must be a dict holding recv_x")
    rx = out["recv_x"]
    if not isinstance(rx, torch.Tensor) or rx.dim() != 2:
        raise ValueError("recv_x must be a 2-D tensor [rows, row_elements]")
    cap = rx.shape[0]
    _need(rx, row_dtype, "recv_x", device, (cap, row_elems))
    if G > 0:
        if out.get("recv_x_scales") is None:
            raise ValueError("rows with scales need recv_x_scales")
        _need(out["recv_x_scales"], torch.float32, "recv_x_scales", device, (cap, G))
    _opt(out, "recv_src_idx", torch.int32, (cap,), device)
    _opt(out, "recv_topk_weights", torch.float32, (cap,), device)
    return cap


def ep_recv_capacity(num_tokens, num_topk, num_local_experts, expert_alignment) -> int:
    return int(_lib.ep_recv_capacity(num_tokens, num_topk, num_local_experts, expert_alignment))


def ep_layout_workspace_bytes(num_tokens, num_topk, num_experts, num_ranks=1, expert_alignment=1) -> int:
    return int(_lib.ep_layout_workspace_bytes(num_tokens, num_topk, num_experts, num_ranks, expert_alignment))


class Handle:
    """Owns an ep_handle_t plus references to the tensors it points into (topk_idx and the workspace)."""

    def __init__(self, ptr, topk_idx, workspace, num_tokens, num_topk, num_experts, num_ranks, rank,
                 expert_alignment):
        self._ptr = ptr
        self.topk_idx = topk_idx
        self.workspace = workspace
        self.num_tokens, self.num_topk, self.num_experts = num_tokens, num_topk, num_experts
        self.num_ranks, self.rank, self.expert_alignment = num_ranks, rank, expert_alignment
        self.num_local_experts = num_experts // num_ranks
        self._cap = None
        self._device = None

    @property
    def device(self):
        """The device of the layout (its topk_idx)."""
        if self._device is None:
            self._device = self.topk_idx.device
        return self._device

    @property
    def recv_capacity(self):
        """Rows of the expert-major receive buffers (ep_recv_capacity of the handle's sizes)."""
        if self._cap is None:
            self._cap = ep_recv_capacity(self.num_tokens, self.num_topk, self.num_local_experts,
                                         self.expert_alignment)
        return self._cap

    @property
    def ptr(self):
        if self._ptr is None:
            raise EPError("handle already freed")
        return self._ptr

    def free(self):
        if self._ptr is not None and _lib is not None:
            _check(_lib.ep_handle_free(self._ptr), "ep_handle_free")
        self._ptr = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def _layout_prep(topk_idx, num_experts, num_ranks, expert_alignment, workspace, outputs):
    _need(topk_idx, torch.int64, "topk_idx")
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [num_tokens, num_topk]")
    T, K = topk_idx.shape
    dev = topk_idx.device
    if num_ranks < 1 or num_experts < 1 or num_experts % num_ranks != 0:
        raise ValueError("num_experts must be a positive multiple of num_ranks")
    if workspace is not None:   # its length is checked by the library call itself
        check_workspace(workspace, dev)
    else:
        nbytes = ep_layout_workspace_bytes(T, K, num_experts, num_ranks, expert_alignment)
        if nbytes == 0:
            raise EPError("ep_layout_workspace_bytes rejected the sizes (T=%d K=%d E=%d R=%d A=%d)"
                          % (T, K, num_experts, num_ranks, expert_alignment))
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    El = num_experts // num_ranks
    if outputs is not None:
        check_layout_outputs(outputs, T, num_experts, num_ranks, dev)
    else:
        outputs = dict(
            num_tokens_per_rank=torch.empty(num_ranks, dtype=torch.int32, device=dev),
            num_tokens_per_expert=torch.empty(num_experts, dtype=torch.int32, device=dev),
            is_token_in_rank=torch.empty((T, num_ranks), dtype=torch.uint8, device=dev),
            psum_num_recv_tokens_per_expert=torch.empty(El + 1, dtype=torch.int32, device=dev),
            num_invalid_topk=torch.empty(1, dtype=torch.int32, device=dev))
    return T, K, workspace, outputs


_LAYOUT_KEYS = ("num_tokens_per_rank", "num_tokens_per_expert", "is_token_in_rank",
                "psum_num_recv_tokens_per_expert", "num_invalid_topk")


def _layout_ptrs(outputs):
    g = outputs.get
    return tuple(None if t is None else t.data_ptr() for t in (g(k) for k in _LAYOUT_KEYS))


def ep_get_layout(topk_idx, num_experts, num_ranks=1, rank=0, expert_alignment=1, workspace=None, outputs=None,
                  stream=None):
    """Layout of `topk_idx` (int64 [T, K] on the GPU).  Returns (Handle, dict) with the device outputs
    num_tokens_per_rank, num_tokens_per_expert, is_token_in_rank, psum_num_recv_tokens_per_expert and
    num_invalid_topk.  `outputs` may supply any of those tensors (or None entries to skip them)."""
    T, K, workspace, outputs = _on_stream(stream, _layout_prep, topk_idx, num_experts, num_ranks, expert_alignment,
                                          workspace, outputs)
    h = ctypes.c_void_p()
    _check(_lib.ep_get_layout(
        _ptr(topk_idx), T, K, num_experts, num_ranks, rank, expert_alignment, _ptr(workspace), workspace.numel(),
        *_layout_ptrs(outputs), ctypes.byref(h), _stream(stream)), "ep_get_layout")
    return Handle(h, topk_idx, workspace, T, K, num_experts, num_ranks, rank, expert_alignment), outputs


def alloc_dispatch_outputs(handle: Handle, hidden: int, fp8: bool, want_meta=True, want_send_meta=True,
                           device=None, recv_capacity=None, do_expand=True):
    """Allocate (uninitialised) dispatch output tensors for `handle` (token-major shapes when do_expand is
    False: num_tokens rows, recv_topk_weights and recv_topk_idx [T, K])."""
    dev = device if device is not None else handle.topk_idx.device
    T, K, R = handle.num_tokens, handle.num_topk, handle.num_ranks
    if recv_capacity is not None:
        cap = recv_capacity
    else:
        cap = handle.recv_capacity if do_expand else T
    G = hidden // 128
    o = {}
    if fp8:
        o["recv_x"] = torch.empty((cap, hidden), dtype=torch.uint8, device=dev)
        o["recv_x_scales"] = torch.empty((cap, G), dtype=torch.float32, device=dev)
    else:
        o["recv_x"] = torch.empty((cap, hidden), dtype=torch.bfloat16, device=dev)
        o["recv_x_scales"] = None
    o["recv_src_idx"] = torch.empty(cap, dtype=torch.int32, device=dev) if want_meta else None
    wshape = cap if do_expand else (T, K)
    o["recv_topk_weights"] = torch.empty(wshape, dtype=torch.float32, device=dev) if want_meta else None
    o["recv_topk_idx"] = torch.empty((T, K), dtype=torch.int64, device=dev) if (want_meta and not do_expand) else None
    if R > 1:
        o["send_x"] = torch.empty((R, T, hidden), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
        o["send_x_scales"] = torch.empty((R, T, G), dtype=torch.float32, device=dev) if fp8 else None
        o["send_src_idx"] = torch.empty((R, T), dtype=torch.int32, device=dev) if want_send_meta else None
        o["send_topk_idx"] = torch.empty((R, T, K), dtype=torch.int64, device=dev) if want_send_meta else None
        o["send_topk_weights"] = torch.empty((R, T, K), dtype=torch.float32, device=dev) if want_send_meta else None
    else:
        for k in ("send_x", "send_x_scales", "send_src_idx", "send_topk_idx", "send_topk_weights"):
            o[k] = None
    return o


_RECV_KEYS = ("recv_x", "recv_x_scales", "recv_src_idx", "recv_topk_weights", "recv_topk_idx")
_SEND_KEYS = ("send_x", "send_x_scales", "send_src_idx", "send_topk_idx", "send_topk_weights")


def _dispatch_struct(out, cap, keys=_RECV_KEYS + _SEND_KEYS):
    s = _DispatchOut()   # zeroed: absent tensors stay NULL
    for k in keys:
        t = out.get(k)
        if t is not None:
            setattr(s, k, t.data_ptr())
    s.recv_capacity = cap
    return s


def ep_dispatch(handle: Handle, x, topk_weights=None, fp8=True, do_expand=True, do_zero_padding=False, out=None,
                want_meta=True, want_send_meta=True, stream=None):
    """Dispatch `x` (bf16 [T, H]) through `handle`.  Returns the dict of output tensors (allocated here unless
    `out` is given; rows that the call does not write keep whatever the tensors held)."""
    _need(x, torch.bfloat16, "x")
    if x.dim() != 2 or x.shape[0] != handle.num_tokens:
        raise ValueError("x must be [num_tokens, hidden]")
    H = x.shape[1]
    dev = x.device
    if topk_weights is not None:
        _need(topk_weights, torch.float32, "topk_weights", dev, (handle.num_tokens, handle.num_topk))
    if out is None:
        out = _on_stream(stream, alloc_dispatch_outputs, handle, H, fp8, want_meta, want_send_meta,
                         device=dev, do_expand=do_expand)
        cap = out["recv_x"].shape[0]
    else:
        cap = check_dispatch_outputs(out, handle.num_tokens, handle.num_topk, handle.num_ranks, H, fp8,
                                     do_expand, dev)
    s = _dispatch_struct(out, cap)
    _check(_lib.ep_dispatch(handle.ptr, _ptr(x), H, _ptr(topk_weights),
                            EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16, int(bool(do_expand)),
                            int(bool(do_zero_padding)), ctypes.byref(s), _stream(stream)), "ep_dispatch")
    return out


def ep_layout_dispatch(topk_idx, x, num_experts, num_ranks=1, rank=0, expert_alignment=1, topk_weights=None,
                       fp8=True, do_expand=True, do_zero_padding=False, out=None, workspace=None, outputs=None,
                       want_meta=True, want_send_meta=True, stream=None):
    """ep_get_layout + ep_dispatch in one call (one kernel launch for <= 256 tokens).  Returns (Handle, layout
    outputs dict, dispatch outputs dict), the same as the two calls would."""
    T, K, workspace, outputs = _on_stream(stream, _layout_prep, topk_idx, num_experts, num_ranks, expert_alignment,
                                          workspace, outputs)
    dev = topk_idx.device
    _need(x, torch.bfloat16, "x", dev)
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [num_tokens, hidden]")
    H = x.shape[1]
    if topk_weights is not None:
        _need(topk_weights, torch.float32, "topk_weights", dev, (T, K))
    if out is None:
        tmp = Handle(None, topk_idx, workspace, T, K, num_experts, num_ranks, rank, expert_alignment)
        out = _on_stream(stream, alloc_dispatch_outputs, tmp, H, fp8, want_meta, want_send_meta, device=dev,
                         do_expand=do_expand)
        cap = out["recv_x"].shape[0]
    else:
        cap = check_dispatch_outputs(out, T, K, num_ranks, H, fp8, do_expand, dev)
    s = _dispatch_struct(out, cap)
    h = ctypes.c_void_p()
    _check(_lib.ep_layout_dispatch(
        _ptr(topk_idx), T, K, num_experts, num_ranks, rank, expert_alignment, _ptr(workspace), workspace.numel(),
        *_layout_ptrs(outputs), _ptr(x), H, _ptr(topk_weights), EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16,
        int(bool(do_expand)), int(bool(do_zero_padding)), ctypes.byref(s), ctypes.byref(h), _stream(stream)),
        "ep_layout_dispatch")
    return Handle(h, topk_idx, workspace, T, K, num_experts, num_ranks, rank, expert_alignment), outputs, out


def ep_layout_dispatch_noalloc(topk_idx, x, num_experts, out, num_ranks=1, rank=0, expert_alignment=1,
                               topk_weights=None, fp8=True, do_expand=True, do_zero_padding=False, outputs=None,
                               stream=None):
    """ep_layout_dispatch for callers that cannot allocate: no workspace (the library's static per-GPU scratch
    serves as one), caller-supplied dispatch outputs `out`, and optional layout `outputs` (None: not written).
    Nothing is allocated here either.  The returned Handle wraps the GPU's static handle: valid until the next
    call of this function on the same GPU, which overwrites it; freeing it is a no-op.  Returns (Handle,
    outputs, out)."""
    _need(topk_idx, torch.int64, "topk_idx")
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [num_tokens, num_topk]")
    T, K = topk_idx.shape
    dev = topk_idx.device
    if num_ranks < 1 or num_experts < 1 or num_experts % num_ranks != 0:
        raise ValueError("num_experts must be a positive multiple of num_ranks")
    _need(x, torch.bfloat16, "x", dev)
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [num_tokens, hidden]")
    H = x.shape[1]
    if topk_weights is not None:
        _need(topk_weights, torch.float32, "topk_weights", dev, (T, K))
    if out is None:
        raise ValueError("ep_layout_dispatch_noalloc needs caller-allocated dispatch outputs (out)")
    cap = check_dispatch_outputs(out, T, K, num_ranks, H, fp8, do_expand, dev)
    if outputs is None:
        outputs = {}
    else:
        check_layout_outputs(outputs, T, num_experts, num_ranks, dev)
    s = _dispatch_struct(out, cap)
    h = ctypes.c_void_p()
    _check(_lib.ep_layout_dispatch_noalloc(
        _ptr(topk_idx), T, K, num_experts, num_ranks, rank, expert_alignment, *_layout_ptrs(outputs), _ptr(x), H,
        _ptr(topk_weights), EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16, int(bool(do_expand)),
        int(bool(do_zero_padding)), ctypes.byref(s), ctypes.byref(h), _stream(stream)),
        "ep_layout_dispatch_noalloc")
    return Handle(h, topk_idx, None, T, K, num_experts, num_ranks, rank, expert_alignment), outputs, out


def ep_combine(handle: Handle, y, topk_weights=None, bias=None, out=None, stream=None):
    """Combine expert outputs `y` (bf16 [>= recv_capacity, H]) back to token order.  Returns out [T, H] bf16."""
    _need(y, torch.bfloat16, "y")
    if y.dim() != 2:
        raise ValueError("y must be [rows, hidden]")
    H = y.shape[1]
    T = handle.num_tokens
    dev = y.device
    if topk_weights is not None:
        _need(topk_weights, torch.float32, "topk_weights", dev, (T, handle.num_topk))
    if bias is not None:
        _need(bias, torch.bfloat16, "bias", dev, (T, H))
    if out is None:
        out = _on_stream(stream, torch.empty, (T, H), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, torch.bfloat16, "out", dev, (T, H))
    _check(_lib.ep_combine(handle.ptr, _ptr(y), H, y.shape[0], _ptr(topk_weights), _ptr(bias), _ptr(out),
                           _stream(stream)), "ep_combine")
    return out


def ep_combine_tokens(handle: Handle, y, bias=None, out=None, stream=None):
    """Combine for the token-major rows (dispatch with do_expand=False): out[t] = y[row of t] + bias, where
    y (bf16 [>= T, H]) holds one row per token of this rank in dispatch order.  Returns out [T, H] bf16."""
    _need(y, torch.bfloat16, "y")
    if y.dim() != 2:
        raise ValueError("y must be [rows, hidden]")
    H = y.shape[1]
    T = handle.num_tokens
    dev = y.device
    if bias is not None:
        _need(bias, torch.bfloat16, "bias", dev, (T, H))
    if out is None:
        out = _on_stream(stream, torch.empty, (T, H), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, torch.bfloat16, "out", dev, (T, H))
    _check(_lib.ep_combine_tokens(handle.ptr, _ptr(y), H, y.shape[0], _ptr(bias), _ptr(out), _stream(stream)),
           "ep_combine_tokens")
    return out


def ep_dispatch_rows(handle: Handle, rows, scales=None, topk_weights=None, do_zero_padding=False, out=None,
                     stream=None):
    """Place received rows (uint8 [N, row_bytes] or bf16 [N, H]) expert-major through `handle` (a layout over
    the rows' local expert ids).  scales: fp32 [N, G] travelling with the rows.  Returns the output dict."""
    if not isinstance(rows, torch.Tensor) or rows.dtype not in (torch.uint8, torch.bfloat16):
        raise TypeError("rows must be a uint8 or bfloat16 tensor")
    _need(rows, rows.dtype, "rows")
    if rows.dim() != 2 or rows.shape[0] != handle.num_tokens:
        raise ValueError("rows must be [num_received_rows, row_elements]")
    dev = rows.device
    N = handle.num_tokens
    row_bytes = rows.shape[1] * rows.element_size()
    G = 0
    if scales is not None:
        if not isinstance(scales, torch.Tensor) or scales.dim() != 2:
            raise ValueError("scales must be a 2-D tensor [num_received_rows, num_scales]")
        G = scales.shape[1]
        _need(scales, torch.float32, "scales", dev, (N, G))
    if topk_weights is not None:
        _need(topk_weights, torch.float32, "topk_weights", dev, (N, handle.num_topk))
    cap = handle.recv_capacity
    if out is None:
        out = _on_stream(stream, lambda: dict(
            recv_x=torch.empty((cap, rows.shape[1]), dtype=rows.dtype, device=dev),
            recv_x_scales=torch.empty((cap, G), dtype=torch.float32, device=dev) if G else None,
            recv_src_idx=torch.empty(cap, dtype=torch.int32, device=dev),
            recv_topk_weights=torch.empty(cap, dtype=torch.float32, device=dev)))
    cap = check_rows_outputs(out, rows.dtype, rows.shape[1], G, dev)
    s = _dispatch_struct(out, cap, _RECV_KEYS[:4])   # the library reads the recv fields only
    _check(_lib.ep_dispatch_rows(handle.ptr, _ptr(rows), row_bytes, _ptr(scales), G, _ptr(topk_weights),
                                 int(bool(do_zero_padding)), ctypes.byref(s), _stream(stream)), "ep_dispatch_rows")
    return out


def ep_combine_reduce(handle: Handle, partials=None, local=None, bias=None, out=None, hidden=None, stream=None):
    """Sum the combine partials returned by the other ranks (bf16 [R, T, H], window r from rank r) with this
    rank's local combine output and the bias.  Returns out [T, H] bf16."""
    T = handle.num_tokens
    ref = next((t for t in (partials, local, bias, out) if t is not None), None)
    if ref is None:
        raise ValueError("ep_combine_reduce needs at least one of partials, local, bias, out")
    _need(ref, torch.bfloat16, "partials/local/bias/out")
    H = ref.shape[-1] if hidden is None else hidden
    dev = ref.device
    if partials is not None:
        _need(partials, torch.bfloat16, "partials", dev, (handle.num_ranks, T, H))
    if local is not None:
        _need(local, torch.bfloat16, "local", dev, (T, H))
    if bias is not None:
        _need(bias, torch.bfloat16, "bias", dev, (T, H))
    if out is None:
        out = _on_stream(stream, torch.empty, (T, H), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, torch.bfloat16, "out", dev, (T, H))
    _check(_lib.ep_combine_reduce(handle.ptr, _ptr(partials), H, _ptr(local), _ptr(bias), _ptr(out),
                                  _stream(stream)), "ep_combine_reduce")
    return out


def _device(handle):
    """The GPU of a handle, where every tensor of its calls must be; it must be the current one (the stream is its)."""
    device = handle.device
    if device.type == "cuda" and device.index != (_cur_device or torch.cuda.current_device)():
        raise ValueError("the handle's device %s is not the current device" % device)
    return device


def _columns(t, name):
    """Columns of a 2-D tensor [rows, columns] (its type and placement are checked with its shape, by _need)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor" % name)
    return t.shape[1]


def _empty(stream, like, shape, dtype=torch.bfloat16):
    """An output or workspace of a call, on `like`'s device, belonging to the call's stream (see _on_stream)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def ep_combine_backward(handle: Handle, grad_out, y=None, topk_weights=None, grad_y=None, grad_topk_weights=None,
                        need_grad_y=True, need_grad_topk_weights=True, stream=None):
    """Gradient of ep_combine.  grad_out: bf16 [T, H]; y: the rows given to ep_combine (needed for the weights'
    gradient); topk_weights as given to it.  Returns (grad_y bf16 [rows, H], grad_topk_weights fp32 [T, K]), None where
    not needed.  Rows of grad_y that no entry owns keep what the tensor held."""
    dev, T, K = _device(handle), handle.num_tokens, handle.num_topk
    H = _columns(grad_out, "grad_out")
    _need(grad_out, torch.bfloat16, "grad_out", dev, (T, H))
    if topk_weights is not None:
        _need(topk_weights, torch.float32, "topk_weights", dev, (T, K))
    need_w = need_grad_topk_weights or grad_topk_weights is not None
    rows = handle.recv_capacity
    if y is not None:
        if _columns(y, "y") != H:
            raise ValueError("y must be [rows, %d]" % H)
        rows = y.shape[0]
        _need(y, torch.bfloat16, "y", dev, (rows, H))
    elif need_w:
        raise ValueError("the gradient of topk_weights needs y")
    if grad_y is not None:
        if y is None and isinstance(grad_y, torch.Tensor) and grad_y.dim() == 2:
            rows = grad_y.shape[0]
        _need(grad_y, torch.bfloat16, "grad_y", dev, (rows, H))
    elif need_grad_y:
        grad_y = _empty(stream, grad_out, (rows, H))
    if grad_topk_weights is not None:
        _need(grad_topk_weights, torch.float32, "grad_topk_weights", dev, (T, K))
    elif need_w:
        grad_topk_weights = _empty(stream, grad_out, (T, K), torch.float32)
    _check(_lib.ep_combine_backward(handle.ptr, _ptr(grad_out), H, _ptr(y), rows, _ptr(topk_weights), _ptr(grad_y),
                                    _ptr(grad_topk_weights), _stream(stream)), "ep_combine_backward")
    return grad_y, grad_topk_weights


def ep_expert_ffn_workspace_bytes(handle: Handle, hidden, intermediate, backward=False) -> int:
    """Bytes of workspace of ep_expert_ffn and ep_expert_ffn_w4 (or, with backward, of either pass) for the handle's rows."""
    return _ffn_bytes(handle.recv_capacity, hidden, intermediate, bool(backward))


# The sizes follow from the arguments alone; a call into the library costs 0.9 us, a tenth of a small call.
@functools.lru_cache(maxsize=1024)
def _ffn_bytes(recv_capacity, hidden, intermediate, backward):
    return int(_lib.ep_expert_ffn_workspace_bytes(recv_capacity, hidden, intermediate, int(backward)))


@functools.lru_cache(maxsize=1024)
def _adapter_bytes(num_tokens, num_local_experts, hidden, rank):
    return int(_lib.ep_adapter_workspace_bytes(num_tokens, num_local_experts, hidden, rank))


def check_ffn_weights(w13, w2, dtype, El, H, device):
    """w13 [El, 2 I, H] and w2 [El, H, I] of `dtype`; returns I."""
    if not isinstance(w2, torch.Tensor) or w2.dim() != 3:
        raise ValueError("w2 must be [num_local_experts, hidden, intermediate]")
    I = w2.shape[2]
    _need(w2, dtype, "w2", device, (El, H, I))
    if w13 is not None:
        _need(w13, dtype, "w13", device, (El, 2 * I, H))
    return I


def check_ffn_scales(xs, s13, s2, rows, El, H, I, device):
    """The scales of e4m3 rows and weights: per row and 128 channels (xs False: the rows have none), per 128 x 128 block."""
    for t, name, shape in ((xs, "recv_x_scales", (rows, H // 128)), (s13, "w13_scales", (El, 2 * I // 128, H // 128)),
                           (s2, "w2_scales", (El, H // 128, I // 128))):
        if t is False:
            continue
        if t is None:
            raise ValueError("e4m3 %s need %s" % ("rows" if xs is not False else "weights", name))
        _need(t, torch.float32, name, device, shape)


def _ffn_workspace(handle, H, I, backward, workspace, device, stream):
    if workspace is not None:   # its length is checked by the library call itself
        check_workspace(workspace, device)
        return workspace
    n = ep_expert_ffn_workspace_bytes(handle, H, I, backward)
    if n == 0:
        raise EPError("ep_expert_ffn_workspace_bytes rejected the sizes (hidden=%d intermediate=%d)" % (H, I))
    return _empty(stream, handle.topk_idx, n, torch.uint8)


def ep_expert_ffn(handle: Handle, recv_x, w13, w2, recv_x_scales=None, w13_scales=None, w2_scales=None, y=None, pre=None,
                  workspace=None, stream=None):
    """The experts' gated feed-forward block over the rows a dispatch placed: y = (silu(x Wg^T) * (x Wu^T)) Wd^T per
    expert.  recv_x [rows, H], w13 [El, 2 I, H] (gate rows first) and w2 [El, H, I]: all bf16, or all uint8 holding e4m3
    with recv_x_scales [rows, H / 128], w13_scales [El, 2 I / 128, H / 128] and w2_scales [El, H / 128, I / 128].
    pre: fp32 [rows, 2 I] to keep for ep_expert_ffn_backward (bf16 only).  Returns y bf16 [rows, H]; rows that are not
    valid rows of an expert keep what y held."""
    if not isinstance(recv_x, torch.Tensor) or recv_x.dtype not in (torch.bfloat16, torch.uint8):
        raise TypeError("recv_x must be a bfloat16 or uint8 (e4m3) tensor")
    fp8 = recv_x.dtype == torch.uint8
    dev, El = _device(handle), handle.num_local_experts
    H = _columns(recv_x, "recv_x")
    rows = recv_x.shape[0]
    _need(recv_x, recv_x.dtype, "recv_x", dev, (rows, H))
    if w13 is None:
        raise ValueError("w13 is required")
    I = check_ffn_weights(w13, w2, recv_x.dtype, El, H, dev)
    if fp8:
        check_ffn_scales(recv_x_scales, w13_scales, w2_scales, rows, El, H, I, dev)
    if y is None:
        y = _empty(stream, recv_x, (rows, H))
    else:
        _need(y, torch.bfloat16, "y", dev, (rows, H))
    if pre is not None:
        _need(pre, torch.float32, "pre", dev, (rows, 2 * I))
    workspace = _ffn_workspace(handle, H, I, False, workspace, dev, stream)
    _check(_lib.ep_expert_ffn(handle.ptr, _ptr(recv_x), _ptr(recv_x_scales) if fp8 else None,
                              EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16, H, I, rows, _ptr(w13),
                              _ptr(w13_scales) if fp8 else None, _ptr(w2), _ptr(w2_scales) if fp8 else None, _ptr(y),
                              _ptr(pre), _ptr(workspace), workspace.numel(), _stream(stream)), "ep_expert_ffn")
    return y


def ep_expert_ffn_backward(handle: Handle, dy, recv_x, pre, w13, w2, dx=None, dw13=None, dw2=None, workspace=None,
                           need_dx=True, need_dw13=True, need_dw2=True, stream=None):
    """Gradients of ep_expert_ffn (bf16) from dy [rows, H] and the forward pass' pre.  Returns (dx [rows, H], dw13 like
    w13, dw2 like w2), bf16, None where not needed.  Rows of dx that are not valid rows keep what it held; dw13 and dw2
    are written whole."""
    dev, El = _device(handle), handle.num_local_experts
    H = _columns(dy, "dy")
    rows = dy.shape[0]
    _need(dy, torch.bfloat16, "dy", dev, (rows, H))
    need_dx, need_dw13, need_dw2 = need_dx or dx is not None, need_dw13 or dw13 is not None, need_dw2 or dw2 is not None
    if need_dx and w13 is None:
        raise ValueError("dx needs w13")
    I = check_ffn_weights(w13, w2, torch.bfloat16, El, H, dev)
    if recv_x is not None:
        _need(recv_x, torch.bfloat16, "recv_x", dev, (rows, H))
    elif need_dw13:
        raise ValueError("dw13 needs recv_x")
    _need(pre, torch.float32, "pre", dev, (rows, 2 * I))

    def grad(t, name, shape, needed):
        if t is not None:
            return _need(t, torch.bfloat16, name, dev, shape)
        return _empty(stream, dy, shape) if needed else None

    dx = grad(dx, "dx", (rows, H), need_dx)
    dw13 = grad(dw13, "dw13", (El, 2 * I, H), need_dw13)
    dw2 = grad(dw2, "dw2", (El, H, I), need_dw2)
    workspace = _ffn_workspace(handle, H, I, True, workspace, dev, stream)
    _check(_lib.ep_expert_ffn_backward(handle.ptr, _ptr(dy), _ptr(recv_x), _ptr(pre), H, I, rows, _ptr(w13), _ptr(w2),
                                       _ptr(dx), _ptr(dw13), _ptr(dw2), _ptr(workspace), workspace.numel(),
                                       _stream(stream)), "ep_expert_ffn_backward")
    return dx, dw13, dw2


def ep_adapter_workspace_bytes(handle: Handle, hidden, rank) -> int:
    """Bytes of workspace of ep_adapter for the handle's tokens and adapters."""
    return _adapter_bytes(handle.num_tokens, handle.num_local_experts, hidden, rank)


def ep_adapter(handle: Handle, x, a, b, scales=None, base=None, out=None, workspace=None, stream=None):
    """Low-rank adapters beside a shared projection: out[t] = base[t] + scales[i] * b[i] (a[i] x[t]), i the token's
    adapter in the handle (a layout over the adapter ids [T, 1], -1 = none).  x bf16 [T, H], a bf16 [El, r, H], b bf16
    [El, N, r], scales fp32 [El], base bf16 [T, N] (None: zeros).  Returns out bf16 [T, N] (may be base itself)."""
    dev, T, El = _device(handle), handle.num_tokens, handle.num_local_experts
    H = _columns(x, "x")
    _need(x, torch.bfloat16, "x", dev, (T, H))
    if not isinstance(b, torch.Tensor) or b.dim() != 3:
        raise ValueError("b must be [num_local_experts, out_features, rank]")
    N, r = b.shape[1], b.shape[2]
    _need(b, torch.bfloat16, "b", dev, (El, N, r))
    _need(a, torch.bfloat16, "a", dev, (El, r, H))
    if scales is not None:
        _need(scales, torch.float32, "scales", dev, (El,))
    if base is not None:
        _need(base, torch.bfloat16, "base", dev, (T, N))
    if out is None:
        out = _empty(stream, x, (T, N))
    else:
        _need(out, torch.bfloat16, "out", dev, (T, N))
    if workspace is not None:
        check_workspace(workspace, dev)
    else:
        n = ep_adapter_workspace_bytes(handle, H, r)
        if n == 0:
            raise EPError("ep_adapter_workspace_bytes rejected the sizes (hidden=%d rank=%d)" % (H, r))
        workspace = _empty(stream, x, n, torch.uint8)
    _check(_lib.ep_adapter(handle.ptr, _ptr(x), H, _ptr(a), _ptr(b), r, N, _ptr(scales), _ptr(base), _ptr(out),
                           _ptr(workspace), workspace.numel(), _stream(stream)), "ep_adapter")
    return out


class W4Weights:
    """4-bit weights [matrices, rows, columns] as ep_w4_pack lays them out: `values` and `scales` (uint8 tensors, opaque), `kind`
    ("int4" or "e2m1"), `group` and `shape`.  A program may keep these and put them together again; they stay as they are then."""

    def __init__(self, values, scales, kind, group, shape):
        if kind not in _W4_KINDS:
            raise ValueError("kind must be one of %s" % sorted(_W4_KINDS))
        shape = tuple(shape)
        if len(shape) != 3:
            raise ValueError("shape must be (matrices, rows, columns)")
        n = _w4_bytes(*shape, group)
        _need(values, torch.uint8, "values", getattr(values, "device", None), (n[0],))
        _need(scales, torch.uint8, "scales", values.device, (n[1],))
        self._parts = values, scales, kind, group, shape, values.device
        self._args = _Weights(values.data_ptr(), scales.data_ptr(), _W4_KINDS[kind], group)

    values = property(lambda self: self._parts[0])
    scales = property(lambda self: self._parts[1])
    kind = property(lambda self: self._parts[2])
    group = property(lambda self: self._parts[3])
    shape = property(lambda self: self._parts[4])
    device = property(lambda self: self._parts[5])


def _w4_bytes(matrices, rows, columns, group):
    """Sizes of packed values and scales."""
    n = ep_w4_packed_bytes(matrices, rows, columns, group)
    if n == 0:
        raise EPError("ep_w4_pack takes no weights of matrices=%d rows=%d columns=%d group=%d" % (matrices, rows, columns, group))
    return n, ep_w4_packed_scale_bytes(matrices, rows, columns, group)


def ep_w4_packed_bytes(matrices, rows, columns, group) -> int:
    return int(_lib.ep_w4_packed_bytes(matrices, rows, columns, group))


def ep_w4_packed_scale_bytes(matrices, rows, columns, group) -> int:
    return int(_lib.ep_w4_packed_scale_bytes(matrices, rows, columns, group))


def ep_w4_pack(codes, scales, kind, stream=None) -> W4Weights:
    """Lays 4-bit weights out for ep_expert_ffn_w4 and ep_moe_few, once, when they are loaded: w = scales[..., k / group] *
    value(code).  codes: uint8 [matrices, rows, columns / 2], two codes a byte, the even column in the lower half; scales: bf16
    [matrices, rows, columns / group], group 32, 64 or 128; kind "int4" (code - 8) or "e2m1".  codes and scales are not needed
    afterwards."""
    if kind not in _W4_KINDS:
        raise ValueError("kind must be one of %s" % sorted(_W4_KINDS))
    if not isinstance(codes, torch.Tensor) or codes.dim() != 3:
        raise ValueError("codes must be [matrices, rows, columns / 2]")
    if not isinstance(scales, torch.Tensor) or scales.dim() != 3:
        raise ValueError("scales must be [matrices, rows, columns / group]")
    dev = _on_current(codes, "codes")
    M, N, K = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
    _need(codes, torch.uint8, "codes", dev)
    _need(scales, torch.bfloat16, "scales", dev, (M, N, scales.shape[2]))
    if scales.shape[2] == 0 or K % scales.shape[2] != 0:
        raise ValueError("scales must be [matrices, rows, columns / group]")
    group = K // scales.shape[2]
    n, m = _w4_bytes(M, N, K, group)
    _need(codes, torch.uint8, "codes")     # on a GPU, after the rules on shapes
    values, packed = _empty(stream, codes, n, torch.uint8), _empty(stream, codes, m, torch.uint8)
    _check(_lib.ep_w4_pack(_ptr(codes), _ptr(scales), _W4_KINDS[kind], M, N, K, group, _ptr(values), _ptr(packed), _stream(stream)),
           "ep_w4_pack")
    return W4Weights(values, packed, kind, group, (M, N, K))


def check_w4_weights(w13, w2, El, H, device):
    """w13 [El, 2 I, H] and w2 [El, H, I], packed; returns I.  (Formats and groups are checked by the library.)"""
    for w, name in ((w13, "w13"), (w2, "w2")):
        if not isinstance(w, W4Weights):
            raise TypeError("%s must be W4Weights (ep_w4_pack)" % name)
        if w.device != device:
            raise ValueError("%s must be on %s, got %s" % (name, device, w.device))
    I = w2.shape[2]
    for w, name, shape in ((w2, "w2", (El, H, I)), (w13, "w13", (El, 2 * I, H))):
        if w.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, shape, w.shape))
    return I


def ep_expert_ffn_w4(handle: Handle, recv_x, w13: W4Weights, w2: W4Weights, y=None, workspace=None, stream=None):
    """ep_expert_ffn with bf16 rows [rows, H] and 4-bit weights: w13 [El, 2 I, H] (gate rows first) and w2 [El, H, I] from
    ep_w4_pack.  Returns y bf16 [rows, H]; rows that are not valid rows of an expert keep what y held."""
    dev, El = _device(handle), handle.num_local_experts
    H = _columns(recv_x, "recv_x")
    rows = recv_x.shape[0]
    _need(recv_x, torch.bfloat16, "recv_x", dev, (rows, H))
    I = check_w4_weights(w13, w2, El, H, dev)
    if y is None:
        y = _empty(stream, recv_x, (rows, H))
    else:
        _need(y, torch.bfloat16, "y", dev, (rows, H))
    workspace = _ffn_workspace(handle, H, I, False, workspace, dev, stream)
    _check(_lib.ep_expert_ffn_w4(handle.ptr, _ptr(recv_x), H, I, rows, ctypes.byref(w13._args), ctypes.byref(w2._args), _ptr(y),
                                 _ptr(workspace), workspace.numel(), _stream(stream)), "ep_expert_ffn_w4")
    return y


@functools.lru_cache(maxsize=1024)
def ep_moe_few_workspace_bytes(num_tokens, num_topk, intermediate) -> int:
    """Bytes of workspace of ep_moe_few."""
    return int(_lib.ep_moe_few_workspace_bytes(num_tokens, num_topk, intermediate))


def ep_moe_few(x, topk_idx, topk_weights, w13, w2, w13_scales=None, w2_scales=None, num_experts=None, num_ranks=1, rank=0, bias=None,
               out=None, workspace=None, stream=None):
    """This rank's share of a whole mixture-of-experts layer for a few tokens (up to 128, and 1024 entries), in two kernels:
    out[t] = sum_k topk_weights[t,k] * ffn_e(x[t]) + bias[t] over the entries whose expert e = topk_idx[t,k] is this rank's.
    x bf16 [T, H], topk_idx int64 [T, K], topk_weights fp32 [T, K] or None (1).  w13 [El, 2 I, H] (gate rows first) and w2
    [El, H, I]: both bf16, both uint8 holding e4m3 with w13_scales [El, 2 I / 128, H / 128] and w2_scales [El, H / 128, I / 128],
    or both W4Weights (ep_w4_pack).  num_experts defaults to El * num_ranks.  Returns out bf16 [T, H] (may be bias itself)."""
    H = _columns(x, "x")
    dev, T = _on_current(x, "x"), x.shape[0]
    _need(x, torch.bfloat16, "x", dev)
    K = _columns(topk_idx, "topk_idx")
    _need(topk_idx, torch.int64, "topk_idx", dev, (T, K))
    if topk_weights is not None:
        _need(topk_weights, torch.float32, "topk_weights", dev, (T, K))
    if bias is not None:
        _need(bias, torch.bfloat16, "bias", dev, (T, H))
    if not hasattr(w2, "shape") or len(w2.shape) != 3:
        raise ValueError("w2 must be [num_local_experts, hidden, intermediate]")
    El = w2.shape[0]
    if num_ranks < 1 or El < 1:
        raise ValueError("num_experts must be a positive multiple of num_ranks")
    if num_experts is None:
        num_experts = El * num_ranks
    elif num_experts != El * num_ranks:
        raise ValueError("num_experts must be %d (the experts of w2) * num_ranks" % El)
    if isinstance(w2, W4Weights):
        I = check_w4_weights(w13, w2, El, H, dev)
        a13, a2 = w13._args, w2._args
    else:
        if w13 is None:
            raise ValueError("w13 is required")
        if w2.dtype not in (torch.bfloat16, torch.uint8):
            raise TypeError("w2 must be bfloat16, uint8 (e4m3) or W4Weights, got %s" % w2.dtype)
        fp8 = w2.dtype == torch.uint8
        I = check_ffn_weights(w13, w2, w2.dtype, El, H, dev)
        if fp8:
            check_ffn_scales(False, w13_scales, w2_scales, 0, El, H, I, dev)
        kind = EP_WEIGHTS_E4M3 if fp8 else EP_WEIGHTS_BF16
        a13 = _Weights(w13.data_ptr(), w13_scales.data_ptr() if fp8 else None, kind, 0)
        a2 = _Weights(w2.data_ptr(), w2_scales.data_ptr() if fp8 else None, kind, 0)
    if out is None:
        out = _empty(stream, x, (T, H))
    else:
        _need(out, torch.bfloat16, "out", dev, (T, H))
    if workspace is not None:
        check_workspace(workspace, dev)
    else:
        n = ep_moe_few_workspace_bytes(T, K, I)
        if n == 0:
            raise EPError("ep_moe_few takes no calls of T=%d K=%d intermediate=%d" % (T, K, I))
        workspace = _empty(stream, x, n, torch.uint8)
    _need(x, torch.bfloat16, "x")     # on a GPU, after the rules on shapes
    _check(_lib.ep_moe_few(_ptr(x), _ptr(topk_idx), _ptr(topk_weights), T, K, num_experts, num_ranks, rank, H, I, ctypes.byref(a13),
                           ctypes.byref(a2), _ptr(bias), _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)), "ep_moe_few")
    return out


def ep_combine_norm_workspace_bytes(num_tokens, hidden) -> int:
    """Bytes of workspace of ep_combine_norm_backward."""
    return _norm_bytes(num_tokens, hidden)


@functools.lru_cache(maxsize=1024)
def _norm_bytes(num_tokens, hidden):
    return int(_lib.ep_combine_norm_workspace_bytes(num_tokens, hidden))


def _on_current(t, name):
    """The device of a call that has no handle: its first tensor's, which must be the current one (the stream is its)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    device = t.device
    if device.type == "cuda" and device.index != (_cur_device or torch.cuda.current_device)():
        raise ValueError("%s is on %s, which is not the current device" % (name, device))
    return device


def check_norm_args(T, H, device, residual, post_weight, gate, residual_scale, pre_weight, eps):
    """What stands around a block, against the sizes the library reads; returns the library's arguments."""
    a = _NormArgs()
    kind = None
    for t, name in ((post_weight, "post_weight"), (pre_weight, "pre_weight"), (gate, "gate")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if name == "gate" and t.dim() == 2:
            _need(t, torch.bfloat16, name, device, (T, H))
            a.gate_per_token = 1
        else:
            if t.dtype not in (torch.float32, torch.bfloat16):
                raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
            if kind is not None and t.dtype != kind:
                raise TypeError("%s is %s beside %s vectors" % (name, t.dtype, kind))
            kind = t.dtype
            _need(t, kind, name, device, (H,))
        setattr(a, name, t.data_ptr())
    if residual is not None:
        _need(residual, torch.bfloat16, "residual", device, (T, H))
        a.residual = residual.data_ptr()
    a.vectors_bf16 = int(kind is torch.bfloat16)
    a.residual_scale, a.eps = residual_scale, eps
    return a


def ep_combine_norm(handle, y, topk_weights=None, bias=None, residual=None, post_weight=None, gate=None, residual_scale=1.0,
                    pre_weight=None, eps=1e-6, out=None, normed=None, kept=None, need_out=True, stream=None):
    """The combine with the norms, gate and residual around a block: f = combine(y, topk_weights, bias), or y + bias with
    handle None; a = f / sqrt(mean f^2 + eps) * post_weight; r = residual_scale * residual + gate * a; n = r / sqrt(mean r^2
    + eps) * pre_weight.  Returns (out = r, normed = n), bf16 [T, H]; normed is None without pre_weight, out with
    need_out=False.  post_weight, pre_weight and gate [H] are all fp32 or all bf16; gate may be bf16 [T, H].  out may be
    the residual itself.  kept: fp32 [T, H] to keep f for ep_combine_norm_backward."""
    H = _columns(y, "y")
    if handle is not None:
        dev, T = _device(handle), handle.num_tokens
        _need(y, torch.bfloat16, "y", dev)
        if topk_weights is not None:
            _need(topk_weights, torch.float32, "topk_weights", dev, (T, handle.num_topk))
    else:
        dev, T = _on_current(y, "y"), y.shape[0]
        _need(y, torch.bfloat16, "y", dev)
        if topk_weights is not None:
            raise ValueError("topk_weights needs a handle")
    if bias is not None:
        _need(bias, torch.bfloat16, "bias", dev, (T, H))
    a = check_norm_args(T, H, dev, residual, post_weight, gate, residual_scale, pre_weight, eps)
    if out is not None:
        _need(out, torch.bfloat16, "out", dev, (T, H))
    elif need_out:
        out = _empty(stream, y, (T, H))
    if normed is not None:
        _need(normed, torch.bfloat16, "normed", dev, (T, H))
    elif pre_weight is not None:
        normed = _empty(stream, y, (T, H))
    if kept is not None:
        _need(kept, torch.float32, "kept", dev, (T, H))
    _need(y, torch.bfloat16, "y")     # on a GPU, after the rules on shapes
    _check(_lib.ep_combine_norm(None if handle is None else handle.ptr, _ptr(y), H, y.shape[0], _ptr(topk_weights), _ptr(bias),
                                ctypes.byref(a), _ptr(out), _ptr(normed), _ptr(kept), _stream(stream)), "ep_combine_norm")
    return out, normed


def ep_combine_norm_backward(grad_out, grad_normed, f, residual=None, post_weight=None, gate=None, residual_scale=1.0,
                             pre_weight=None, eps=1e-6, grad_f=None, grad_residual=None, grad_post=None, grad_pre=None,
                             grad_gate=None, need_rows=True, need_vectors=True, workspace=None, stream=None):
    """Gradients of ep_combine_norm from grad_out and grad_normed (bf16 [T, H], either may be None) and f: the fp32 [T, H]
    that the forward pass kept, or the bf16 y of a call without handle and bias.  Returns a dict: grad_f and
    grad_residual bf16 [T, H], grad_post and grad_pre fp32 [H], grad_gate fp32 [H] or bf16 [T, H] as the gate; None for what
    the call did not have, and, unless given, for the rows with need_rows=False and the vectors with need_vectors=False.
    grad_f goes on as grad_out of ep_combine_backward."""
    H = _columns(f, "f")
    dev, T = _on_current(f, "f"), f.shape[0]
    if f.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("f must be float32 or bfloat16, got %s" % f.dtype)
    _need(f, f.dtype, "f", dev)
    for t, name in ((grad_out, "grad_out"), (grad_normed, "grad_normed")):
        if t is not None:
            _need(t, torch.bfloat16, name, dev, (T, H))
    a = check_norm_args(T, H, dev, residual, post_weight, gate, residual_scale, pre_weight, eps)
    per_token = bool(a.gate_per_token)

    _need(f, f.dtype, "f")            # on a GPU, after the rules on shapes

    def grad(t, name, dtype, shape, has, needed):
        if t is not None:
            return _need(t, dtype, name, dev, shape)
        return _empty(stream, f, shape, dtype) if has and needed else None

    g = dict(
        grad_f=grad(grad_f, "grad_f", torch.bfloat16, (T, H), True, need_rows),
        grad_residual=grad(grad_residual, "grad_residual", torch.bfloat16, (T, H), residual is not None, need_rows),
        grad_post=grad(grad_post, "grad_post", torch.float32, (H,), post_weight is not None, need_vectors),
        grad_pre=grad(grad_pre, "grad_pre", torch.float32, (H,), pre_weight is not None and grad_normed is not None, need_vectors),
        grad_gate=grad(grad_gate, "grad_gate", torch.bfloat16 if per_token else torch.float32, (T, H) if per_token else (H,),
                       gate is not None, need_rows if per_token else need_vectors))
    if workspace is not None:
        check_workspace(workspace, dev)
    else:
        n = ep_combine_norm_workspace_bytes(T, H)
        if n == 0:
            raise EPError("ep_combine_norm_workspace_bytes rejected the sizes (T=%d hidden=%d)" % (T, H))
        workspace = _empty(stream, f, n, torch.uint8)
    _check(_lib.ep_combine_norm_backward(
        _ptr(grad_out), _ptr(grad_normed), _ptr(f), int(f.dtype is torch.bfloat16), T, H, ctypes.byref(a), _ptr(g["grad_f"]),
        _ptr(g["grad_residual"]), _ptr(g["grad_post"]), _ptr(g["grad_pre"]), _ptr(g["grad_gate"]), _ptr(workspace),
        workspace.numel(), _stream(stream)), "ep_combine_norm_backward")
    return g


def ep_handle_free(handle: Handle):
    handle.free()


__all__ = ["ep_get_layout", "ep_dispatch", "ep_layout_dispatch", "ep_layout_dispatch_noalloc", "ep_combine", "ep_combine_tokens", "ep_handle_free", "ep_recv_capacity",
           "ep_dispatch_rows", "ep_combine_reduce", "ep_combine_backward", "ep_expert_ffn", "ep_expert_ffn_backward",
           "ep_expert_ffn_workspace_bytes", "ep_adapter", "ep_adapter_workspace_bytes",
           "ep_w4_pack", "W4Weights", "ep_w4_packed_bytes", "ep_w4_packed_scale_bytes", "ep_expert_ffn_w4", "ep_moe_few", "ep_moe_few_workspace_bytes",
           "ep_combine_norm", "ep_combine_norm_backward", "ep_combine_norm_workspace_bytes",
           "ep_layout_workspace_bytes", "alloc_dispatch_outputs", "Handle", "EPError", "LIB_PATH",
           "hip_runtimes_loaded"]
