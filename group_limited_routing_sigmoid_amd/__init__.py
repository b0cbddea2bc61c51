"""Python binding of libbeam_moe.so, the MI355X (gfx950) Beam MoE block.

Argument marshalling only: every step of the block runs in the library's HIP
kernels.  torch supplies device memory and the current stream.  The names
follow the C ABI in include/beam_moe.h (beam_moe_route, beam_moe_forward,
beam_moe_permute, beam_moe_quant_e4m3, beam_moe_workspace_bytes,
beam_moe_validate; around the block beam_moe_route_backward,
beam_moe_matmul_e4m3, beam_moe_quant_e4m3_2d, beam_moe_norm_residual and its
_backward).  There is no CPU fallback: without the built library
every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# another build of the same library (e.g. a host-sanitizer build) may be
# named in BEAM_MOE_LIB; there is no fallback when the file is missing
LIB_PATH = os.environ.get("BEAM_MOE_LIB") or os.path.join(_HERE, "libbeam_moe.so")

F32, BF16, FP8_E4M3, MXFP4 = 0, 1, 2, 3
ROUTE_LOGITS_IN, PATH_STREAM, PATH_GROUPED = 1 << 0, 1 << 1, 1 << 2
TILE_128, TILE_256, TILE_160, TILE_64 = 1 << 3, 1 << 4, 1 << 5, 1 << 6
ROUTE_SOFTMAX, ROUTE_UNNORMED = 1 << 7, 1 << 8
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = 0, -1, -2, -3, -4

SYMBOLS = ("beam_status_string", "beam_moe_validate", "beam_moe_workspace_bytes",
           "beam_moe_route", "beam_moe_permute", "beam_moe_quant_e4m3",
           "beam_moe_forward", "beam_moe_timer_create", "beam_moe_timer_destroy",
           "beam_moe_timer_reset", "beam_moe_timer_count", "beam_moe_timer_read",
           "beam_moe_forward_timed", "beam_moe_bias_update", "beam_moe_bias_gamma",
           "beam_moe_forward_residual", "beam_moe_quant_mxfp8",
           "beam_moe_forward_noalloc", "beam_moe_route_backward",
           "beam_moe_norm_residual", "beam_moe_norm_residual_workspace_bytes",
           "beam_moe_norm_residual_backward", "beam_moe_matmul_e4m3",
           "beam_moe_quant_e4m3_2d")
NOALLOC_SCRATCH_BYTES = 64 << 20


class Desc(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("intermediate", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("group_score_topn", ctypes.c_int32),
                ("routed_scale", ctypes.c_float), ("act_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class BeamError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m group_limited_routing_sigmoid_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        D = ctypes.POINTER(Desc)
        L.beam_status_string.argtypes = [ctypes.c_int]
        L.beam_status_string.restype = ctypes.c_char_p
        L.beam_moe_validate.argtypes = [D, i64]
        L.beam_moe_workspace_bytes.argtypes = [D, i64, ctypes.POINTER(sz)]
        L.beam_moe_route.argtypes = [D, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_route_backward.argtypes = [D, i64, vp, vp, vp, vp, vp]
        L.beam_moe_quant_e4m3_2d.argtypes = [i64, i64, i32, i32, vp, vp, vp, vp, vp, vp]
        L.beam_moe_matmul_e4m3.argtypes = [i64, i64, i64, vp, vp, i64, i64, vp, vp, i64, i64, i32,
                                           i32, vp, vp]
        f32 = ctypes.c_float
        L.beam_moe_norm_residual.argtypes = [i64, i64, i32, vp, vp, vp, i64, vp, f32, f32, f32,
                                             vp, vp, vp, vp, vp, vp]
        L.beam_moe_norm_residual_workspace_bytes.argtypes = [i64, i64, ctypes.POINTER(sz)]
        L.beam_moe_norm_residual_backward.argtypes = [i64, i64, i32, vp, vp, vp, i64, vp, f32, f32,
                                                      f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_permute.argtypes = [D, i64, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_quant_e4m3.argtypes = [i64, i64, i32, vp, vp, vp, vp]
        L.beam_moe_quant_mxfp8.argtypes = [i64, i64, i32, vp, vp, vp, vp]
        L.beam_moe_forward.argtypes = [D, i64, vp, vp, vp, vp, vp, vp, vp, vp,
                                       vp, vp, vp, vp, sz, vp]
        L.beam_moe_forward_timed.argtypes = L.beam_moe_forward.argtypes + [vp]
        L.beam_moe_forward_noalloc.argtypes = [D, i64, vp, vp, vp, vp, vp, vp, vp, vp,
                                               vp, vp, vp, vp]
        L.beam_moe_forward_residual.argtypes = [D, i64, vp, vp, vp, vp, vp, vp, vp, vp,
                                                ctypes.c_float, i32, vp, vp, vp, sz, vp]
        L.beam_moe_timer_create.argtypes = [i32, ctypes.POINTER(vp)]
        L.beam_moe_timer_destroy.argtypes = [vp]
        L.beam_moe_timer_destroy.restype = None
        L.beam_moe_timer_reset.argtypes = [vp]
        L.beam_moe_timer_reset.restype = None
        L.beam_moe_timer_count.argtypes = [vp]
        L.beam_moe_timer_read.argtypes = [vp, i32, ctypes.POINTER(ctypes.c_char_p),
                                          ctypes.POINTER(ctypes.c_float)]
        L.beam_moe_bias_update.argtypes = [D, i64, vp, ctypes.c_float, vp, vp]
        L.beam_moe_bias_gamma.argtypes = [i64, i64, ctypes.c_float, ctypes.c_float]
        L.beam_moe_bias_gamma.restype = ctypes.c_float
        for f in SYMBOLS[1:]:
            if getattr(L, f).restype is ctypes.c_int or f in (
                    "beam_moe_timer_destroy", "beam_moe_timer_reset",
                    "beam_moe_bias_gamma"):
                continue
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().beam_status_string(status).decode()


def _check(status: int, what: str):
    if status != OK:
        raise BeamError(status, what)


def make_desc(shape, act_dtype: int, weight_dtype: int, flags: int = 0) -> Desc:
    """Descriptor from any object with the layer-shape fields (hidden,
    intermediate, n_experts, n_groups, topk_groups, top_k, group_score_topn,
    routed_scale)."""
    return Desc(shape.hidden, shape.intermediate, shape.n_experts,
                shape.n_groups, shape.topk_groups, shape.top_k,
                getattr(shape, "group_score_topn", 2),
                getattr(shape, "routed_scale", 2.5), act_dtype, weight_dtype,
                flags)


def with_flags(desc: Desc, flags: int) -> Desc:
    d = Desc.from_buffer_copy(desc)
    d.flags = flags
    return d


def validate(desc: Desc, T: int) -> int:
    return lib().beam_moe_validate(ctypes.byref(desc), T)


def workspace_bytes(desc: Desc, T: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().beam_moe_workspace_bytes(ctypes.byref(desc), T, ctypes.byref(n)),
           "beam_moe_workspace_bytes")
    return n.value


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the HIP library must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the HIP library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _addr(t: Optional[torch.Tensor]):
    """As _p, but a plain integer (ctypes converts it)."""
    if t is None:
        return None
    if t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _p(t)  # raises


def _torch_stream(stream, device):
    return stream if stream is not None else torch.cuda.current_stream(device)


def _stream(stream=None, device=None):
    if stream is None:  # the current stream's handle without a Stream object
        i = device.index if device is not None else None
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(
            torch.cuda.current_device() if i is None else i))
    return ctypes.c_void_p(stream.cuda_stream)


class Workspace:
    """A growable device byte buffer reused across calls.

    Calls that may overlap (calls on different streams) need distinct
    workspaces.  The buffer is allocated on the stream of the call that
    grows it, and marked as used by any other stream a later call runs on,
    so torch's allocator never hands its memory out again while queued
    kernels may still use it."""

    def __init__(self, device="cuda"):
        self.device = torch.device(device)
        self.buf = None
        self.streams = set()

    def get(self, nbytes: int, stream=None) -> Optional[torch.Tensor]:
        if nbytes == 0:
            return None
        s = _torch_stream(stream, self.device)
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = None
            with torch.cuda.stream(s):
                self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            self.streams = {s.cuda_stream}
        elif s.cuda_stream not in self.streams:
            self.buf.record_stream(s)
            self.streams.add(s.cuda_stream)
        return self.buf


# one default workspace per (device, stream): calls on one stream are
# ordered, calls on different streams never share scratch memory
_default_ws = {}


def _capturing(stream, device) -> bool:
    """Whether a call's stream (None: `device`'s current one) is being captured
    into a graph; torch answers for the current device's current stream."""
    if stream is None:
        if device.index == _current_device():
            return torch._C._cuda_isCurrentStreamCapturing()
        stream = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        return torch._C._cuda_isCurrentStreamCapturing()


def _scratch(n: int, workspace: Optional[Workspace], device, stream=None):
    if n == 0:
        return None
    if workspace is not None:
        return workspace.get(n, _torch_stream(stream, device))
    # A call that is being captured takes memory of its graph instead: graphs
    # are captured on one stream and replayed on any.
    if _capturing(stream, device):
        return Workspace(device).get(n, _torch_stream(stream, device))
    key = (device.index, _raw_stream(device.index) if stream is None else stream.cuda_stream)
    workspace = _default_ws.get(key)
    if workspace is None:
        workspace = _default_ws[key] = Workspace(device)
    elif workspace.buf is not None and workspace.buf.numel() >= n:
        return workspace.buf  # allocated on the key's stream, used there only
    return workspace.get(n, _torch_stream(stream, device))


def _ws(desc: Desc, T: int, workspace: Optional[Workspace], device, stream=None):
    n = workspace_bytes(desc, T)
    return _scratch(n, workspace, device, stream), n


def _alloc_on(stream):
    """Context in which the binding allocates a call's outputs: the call's
    stream, so that torch's allocator orders their reuse after its kernels."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _arg(name: str, t: torch.Tensor, dev: int, dtype: torch.dtype, shape: tuple,
         strided: bool = False) -> int:
    """Address of a contiguous (or strided, where a call takes strides) tensor
    on GPU `dev` of the given dtype and shape; raises ValueError otherwise."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0
            and (strided or t.is_contiguous())):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name}: tensors passed to the HIP library must be on the GPU")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on cuda:{t.get_device()}, the other tensors on cuda:{dev}")
    raise ValueError(f"{name}: tensors passed to the HIP library must be contiguous")


def _floats(name: str, t: torch.Tensor, dev: int, shape: tuple, more: bool = False) -> int:
    """As _arg for fp32 values that are read or written in order: a tensor of
    any shape with as many elements (`more`: or with room for more)."""
    n = t.numel() - math.prod(shape)
    if (t.dtype is torch.float32 and (n == 0 or (more and n > 0)) and t.get_device() == dev >= 0
            and t.is_contiguous()):
        return t.data_ptr()
    return _arg(name, t, dev, torch.float32, shape)  # raises


# torch.empty parses its arguments for half of its time (1.3 us): on the current
# device and stream the allocation that torch's compiled graphs call (0.75 us)
# is used where this torch has it
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None),
                         "_empty_strided_cuda", None)


def _on(stream, dev: int):
    """Where a call runs, for _empty and _run: True on the current device's
    current stream, else the stream it was given (None: GPU `dev`'s current
    one)."""
    return True if stream is None and dev >= 0 and dev == _current_device() else stream


def _empty(on, device, dtype: torch.dtype, *shape) -> torch.Tensor:
    """An output of one or two dimensions, allocated on the call's stream."""
    if on is True and _empty_strided is not None:
        return _empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype)
    with _alloc_on(None if on is True else on):
        return torch.empty(*shape, dtype=dtype, device=device)


def _empty_t(on, device, dtype: torch.dtype, rows: int, cols: int) -> torch.Tensor:
    """An output [rows, cols] stored column by column."""
    if on is True and _empty_strided is not None:
        return _empty_strided((rows, cols), (1, rows), dtype)
    return _empty(on, device, dtype, cols, rows).t()


def _run(fn, what: str, on, dev: int, tensors, *args):
    """Call a library entry point whose last argument is the stream on GPU
    `dev`, whichever is current.  Tensors read or written on a stream that is
    not the current one are marked as used there, so torch's allocator keeps
    their memory until the kernels are done."""
    if on is True:
        status = fn(*args, _raw_stream(dev))
        if status != OK:
            raise BeamError(status, what)
        return
    stream = on
    raw = _raw_stream(dev)
    # every GPU's default stream has the same handle
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"{what}: a stream of {stream.device} for tensors on cuda:{dev}")
    if stream is not None and stream.cuda_stream != raw:
        raw = stream.cuda_stream
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    if _current_device() == dev:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != OK:
        raise BeamError(status, what)


def route(desc: Desc, x: Optional[torch.Tensor], w_router: Optional[torch.Tensor],
          bias: Optional[torch.Tensor] = None, logits: Optional[torch.Tensor] = None,
          workspace: Optional[Workspace] = None, stream=None):
    """beam_moe_route.  Returns (topk_idx [T,K] int32, topk_w [T,K] fp32,
    logits [T,E] fp32).  With ROUTE_LOGITS_IN in desc.flags, `logits` is the
    input and x / w_router may be None; without it `logits` may be a buffer for
    them, also one with room for more.  bias and logits are contiguous fp32 on
    x's GPU and may have other shapes of the same size.  ROUTE_SOFTMAX and
    ROUTE_UNNORMED choose the scores and the weights."""
    lin = bool(desc.flags & ROUTE_LOGITS_IN)
    ref = logits if lin else x
    T, E, device, dev = ref.shape[0], desc.n_experts, ref.device, ref.get_device()
    on = _on(stream, dev)
    px, pr = (None, None) if lin else (_addr(x), _addr(w_router))
    pb = None if bias is None else _floats("bias", bias, dev, (E,))
    if logits is None:
        logits = _empty(on, device, torch.float32, T, E)
    pl = _floats("logits", logits, dev, (T, E), not lin)
    idx = _empty(on, device, torch.int32, T, desc.top_k)
    w = _empty(on, device, torch.float32, T, desc.top_k)
    # routing from given logits uses no scratch memory
    buf, n = (None, 0) if lin else _ws(desc, T, workspace, device, stream)
    _run(lib().beam_moe_route, "beam_moe_route", on, dev, (x, w_router, bias, logits, idx, w),
         ctypes.byref(desc), T, px, pr, pb, pl, idx.data_ptr(), w.data_ptr(), _addr(buf), n)
    return idx, w, logits


def route_backward(desc: Desc, logits: torch.Tensor, topk_idx: torch.Tensor,
                   d_topk_w: torch.Tensor, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """beam_moe_route_backward: the gradient [T,E] fp32 of the logits from that
    of the routing weights (the selection and the bias are constants)."""
    T, E, K, dev = logits.shape[0], desc.n_experts, desc.top_k, logits.get_device()
    on = _on(stream, dev)
    pl = _arg("logits", logits, dev, torch.float32, (T, E))
    pi = _arg("topk_idx", topk_idx, dev, torch.int32, (T, K))
    pw = _arg("d_topk_w", d_topk_w, dev, torch.float32, (T, K))
    if out is None:
        out = _empty(on, logits.device, torch.float32, T, E)
        po = out.data_ptr()
    else:
        po = _arg("out", out, dev, torch.float32, (T, E))
    _run(lib().beam_moe_route_backward, "beam_moe_route_backward", on, dev,
         (logits, topk_idx, d_topk_w, out), ctypes.byref(desc), T, pl, pi, pw, po)
    return out


def permute(desc: Desc, topk_idx: torch.Tensor,
            workspace: Optional[Workspace] = None, stream=None):
    """beam_moe_permute.  Returns dict(counts, offsets, slot_token, slot_of)."""
    T, dev = topk_idx.shape[0], topk_idx.device
    E, S = desc.n_experts, T * desc.top_k
    with _alloc_on(stream):
        out = dict(counts=torch.empty(E, dtype=torch.int32, device=dev),
                   offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                   slot_token=torch.empty(max(S, 1), dtype=torch.int32, device=dev),
                   slot_of=torch.empty(max(S, 1), dtype=torch.int32, device=dev))
    buf, n = _ws(desc, T, workspace, dev, stream)
    _check(lib().beam_moe_permute(ctypes.byref(desc), T, _p(topk_idx),
                                  _p(out["counts"]), _p(out["offsets"]),
                                  _p(out["slot_token"]), _p(out["slot_of"]),
                                  _p(buf), n, _stream(stream, dev)), "beam_moe_permute")
    out["slot_token"] = out["slot_token"][:S]
    out["slot_of"] = out["slot_of"][:S].view(T, desc.top_k)
    return out


def forward_residual(desc: Desc, x: torch.Tensor, w_router: Optional[torch.Tensor],
                     bias: Optional[torch.Tensor], w_gate_up: torch.Tensor,
                     w_down: torch.Tensor, norm_weight: torch.Tensor, eps: float,
                     step: int, residual: torch.Tensor,
                     s_gate_up: Optional[torch.Tensor] = None,
                     s_down: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None,
                     workspace: Optional[Workspace] = None, stream=None):
    """beam_moe_forward_residual: the block, then residual (fp32 [T,H], in
    place) = sqrt((k-1)/k) residual + RMSNorm(block output) * norm_weight /
    sqrt(k).  Returns residual (and writes out when given)."""
    T, dev = x.shape[0], x.device
    buf, n = _ws(desc, T, workspace, dev, stream)
    _check(lib().beam_moe_forward_residual(
        ctypes.byref(desc), T, _p(x), _p(w_router), _p(bias), _p(w_gate_up),
        _p(s_gate_up), _p(w_down), _p(s_down), _p(norm_weight), float(eps),
        int(step), _p(residual), _p(out), _p(buf), n, _stream(stream, dev)),
        "beam_moe_forward_residual")
    return residual


def bias_update(desc: Desc, topk_idx: torch.Tensor, gamma: float,
                bias: torch.Tensor, stream=None):
    """beam_moe_bias_update: one balancing step on `bias` (in place)."""
    _check(lib().beam_moe_bias_update(ctypes.byref(desc), topk_idx.shape[0],
                                      _p(topk_idx), float(gamma), _p(bias),
                                      _stream(stream, bias.device)), "beam_moe_bias_update")
    return bias


def bias_gamma(t: int, n: int, g0: float, g1: float) -> float:
    """beam_moe_bias_gamma: cosine-decayed update speed (host only)."""
    return lib().beam_moe_bias_gamma(t, n, g0, g1)


def quant_e4m3(v: torch.Tensor, stream=None):
    """beam_moe_quant_e4m3 of a 2-D fp32/bf16 tensor: (codes uint8, scales)."""
    rows, cols = v.shape
    dt = BF16 if v.dtype == torch.bfloat16 else F32
    if v.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(v.dtype)
    with _alloc_on(stream):
        q = torch.empty(rows, cols, dtype=torch.uint8, device=v.device)
        s = torch.empty(rows, max(cols // 128, 1), dtype=torch.float32, device=v.device)
    _check(lib().beam_moe_quant_e4m3(rows, cols, dt, _p(v), _p(q), _p(s),
                                     _stream(stream, v.device)), "beam_moe_quant_e4m3")
    return q, s[:, :cols // 128]


def quant_mxfp8(v: torch.Tensor, stream=None):
    """beam_moe_quant_mxfp8 of a 2-D fp32/bf16 tensor: (codes uint8, E8M0
    scales uint8 [rows, cols/32])."""
    rows, cols = v.shape
    if v.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(v.dtype)
    dt = BF16 if v.dtype == torch.bfloat16 else F32
    with _alloc_on(stream):
        q = torch.empty(rows, cols, dtype=torch.uint8, device=v.device)
        s = torch.empty(rows, max(cols // 32, 16), dtype=torch.uint8, device=v.device)
    _check(lib().beam_moe_quant_mxfp8(rows, cols, dt, _p(v), _p(q), _p(s),
                                      _stream(stream, v.device)), "beam_moe_quant_mxfp8")
    return q, s[:, :cols // 32]


def quant_e4m3_2d(v: torch.Tensor, block: bool = False, straight: bool = True,
                  transposed: bool = True, stream=None):
    """beam_moe_quant_e4m3_2d of a 2-D fp32/bf16 tensor [R,C]: (codes [R,C'],
    scales, transposed codes [C,R'], their scales), C' and R' the next
    multiples of 128, the added codes zero.  A scale covers 128 values of a
    row (of a column in the transposed codes): [R,C'/128] and [C,R'/128],
    stored block-major (views of transposed tensors); or with block 128 x 128
    values: [R'/128,C'/128] and its transpose.  None for an orientation that
    is not asked for."""
    if v.dim() != 2:
        raise ValueError(f"v: shape {tuple(v.shape)}, expected [rows, cols]")
    if v.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"v: dtype {v.dtype}, expected torch.bfloat16 or torch.float32")
    rows, cols = v.shape
    dev, device = v.get_device(), v.device
    on = _on(stream, dev)
    pv = _arg("v", v, dev, v.dtype, (rows, cols))
    nr, nc = (rows + 127) // 128, (cols + 127) // 128
    q = s = qt = st = None
    if straight:
        q = _empty(on, device, torch.uint8, rows, nc * 128)
        s = (_empty(on, device, torch.float32, nr, nc) if block else
             _empty_t(on, device, torch.float32, rows, nc))
    if transposed:
        qt = _empty(on, device, torch.uint8, cols, nr * 128)
        st = (_empty(on, device, torch.float32, nc, nr) if block else
              _empty_t(on, device, torch.float32, cols, nr))
    _run(lib().beam_moe_quant_e4m3_2d, "beam_moe_quant_e4m3_2d", on, dev, (v, q, s, qt, st),
         rows, cols, BF16 if v.dtype is torch.bfloat16 else F32, 1 if block else 0, pv,
         *(None if t is None else t.data_ptr() for t in (q, s, qt, st)))
    return q, s, qt, st


def matmul_e4m3(a: torch.Tensor, s_a: torch.Tensor, b: torch.Tensor, s_b: torch.Tensor,
                dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """beam_moe_matmul_e4m3: a b^T [M,N] in `dtype` from e4m3 codes a [M,K] and
    b [N,K] (uint8), K a multiple of 128, with scales s_a [M,K/128] and s_b
    [ceil(N/128),K/128] (128 x 128 blocks) or [N,K/128] (rows of b), which may
    have any strides from a 16-byte aligned first element.  The product of two
    scales that meet has to be 0 or a normal fp32 number."""
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)}, expected [M, K] and [N, K]")
    (M, K), N = a.shape, b.shape[0]
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"dtype {dtype}, expected torch.bfloat16 or torch.float32")
    if K % 128:
        raise ValueError(f"K = {K} is not a multiple of 128")
    rows = s_b.dim() == 2 and s_b.shape[0] == N
    dev = a.get_device()
    on = _on(stream, dev)
    pa, pb = _arg("a", a, dev, torch.uint8, (M, K)), _arg("b", b, dev, torch.uint8, (N, K))
    psa = _arg("s_a", s_a, dev, torch.float32, (M, K // 128), True)
    psb = _arg("s_b", s_b, dev, torch.float32, (N if rows else (N + 127) // 128, K // 128), True)
    if out is None:
        out = _empty(on, a.device, dtype, M, N)
        py = out.data_ptr()
    else:
        py = _arg("out", out, dev, dtype, (M, N))
    _run(lib().beam_moe_matmul_e4m3, "beam_moe_matmul_e4m3", on, dev, (a, s_a, b, s_b, out),
         M, N, K, pa, psa, *s_a.stride(), pb, psb, *s_b.stride(), 1 if rows else 0,
         BF16 if dtype is torch.bfloat16 else F32, py)
    return out


def residual_scale(step: int):
    """(alpha, beta) of the depth-scaled residual stream at sublayer step k >= 1:
    sqrt((k-1)/k) and 1/sqrt(k), as forward_residual uses them."""
    if step < 1:
        raise ValueError(f"step {step}: steps count from 1")
    return math.sqrt((step - 1) / step), 1.0 / math.sqrt(step)


def _norm_inputs(residual, o, post_weight, gate, pre_weight, dtype):
    """Checked arguments of a step: (T, H, device index, dtype, addresses of o,
    post_weight and gate, gate_cols, address of pre_weight)."""
    if residual.dim() != 2:
        raise ValueError(f"residual: shape {tuple(residual.shape)}, expected [T, H]")
    T, H = residual.shape
    dev = residual.get_device()
    if o is None:
        if post_weight is not None or gate is not None:
            raise ValueError("post_weight and gate belong to o")
        if dtype is None:
            dtype = torch.bfloat16
    else:
        if dtype is not None and dtype is not o.dtype:
            raise ValueError(f"dtype {dtype} with o in {o.dtype}: o, gate and x share one dtype")
        dtype = o.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"dtype {dtype}, expected torch.bfloat16 or torch.float32")
    po = pw = pg = pp = None
    cols = 0
    if o is not None:
        if post_weight is None:
            raise ValueError("o needs its post_weight")
        po = _arg("o", o, dev, dtype, (T, H))
        pw = _arg("post_weight", post_weight, dev, torch.float32, (H,))
        if gate is not None:
            cols = H if gate.dim() == 2 and gate.shape[1] == H else 1
            pg = _arg("gate", gate, dev, dtype, (T, cols))
    if pre_weight is not None:
        pp = _arg("pre_weight", pre_weight, dev, torch.float32, (H,))
    return T, H, dev, dtype, po, pw, pg, cols, pp


def _norm_residual(residual, o, post_weight, gate, pre_weight, eps, alpha, beta, dtype,
                   residual_out, want_x, codes, stream):
    T, H, dev, dtype, po, pw, pg, cols, pp = _norm_inputs(
        residual, o, post_weight, gate, pre_weight, dtype)
    pr = _arg("residual", residual, dev, torch.float32, (T, H))
    device, on = residual.device, _on(stream, dev)
    x = q = s = p_out = px = pq = ps = None
    if o is None:
        if residual_out is not None:
            raise ValueError("residual_out belongs to o: without it r' is the residual itself")
        residual_out = residual
    else:
        if residual_out is None:
            residual_out = _empty(on, device, torch.float32, T, H)
            p_out = residual_out.data_ptr()
        else:
            p_out = _arg("residual_out", residual_out, dev, torch.float32, (T, H))
    if pp is not None and want_x:
        x = _empty(on, device, dtype, T, H)
        px = x.data_ptr()
    if codes:
        q = _empty(on, device, torch.uint8, T, H)
        s = _empty(on, device, torch.float32, T, H // 128)
        pq, ps = q.data_ptr(), s.data_ptr()
    _run(lib().beam_moe_norm_residual, "beam_moe_norm_residual", on, dev,
         (residual, o, post_weight, gate, pre_weight, residual_out, x, q, s), T, H,
         BF16 if dtype is torch.bfloat16 else F32, po, pw, pg, cols, pp, eps, alpha, beta, pr, p_out,
         px, pq, ps)
    return residual_out, x, q, s


def norm_residual(residual: torch.Tensor, o: Optional[torch.Tensor] = None,
                  post_weight: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None,
                  pre_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  alpha: float = 1.0, beta: float = 1.0, dtype: Optional[torch.dtype] = None,
                  residual_out: Optional[torch.Tensor] = None, stream=None):
    """beam_moe_norm_residual: the step between two blocks.  Returns (r', x):
    r' = alpha residual + beta sigmoid(gate) RMSNorm(o) post_weight, fp32
    (residual itself without o; residual_out may be residual), and x =
    RMSNorm(r') pre_weight in o's dtype (`dtype`, bf16 by default, without o;
    None without pre_weight).  gate is [T,H] or [T,1]."""
    return _norm_residual(residual, o, post_weight, gate, pre_weight, eps, alpha, beta, dtype,
                          residual_out, True, False, stream)[:2]


def norm_residual_e4m3(residual: torch.Tensor, o: Optional[torch.Tensor] = None,
                       post_weight: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None,
                       pre_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                       alpha: float = 1.0, beta: float = 1.0,
                       dtype: Optional[torch.dtype] = None,
                       residual_out: Optional[torch.Tensor] = None, with_x: bool = False,
                       stream=None):
    """norm_residual with x as e4m3 codes [T,H] uint8 and scales [T,H/128], as
    matmul_e4m3 takes them.  Returns (r', codes, scales), and x too with
    with_x."""
    if pre_weight is None:
        raise ValueError("the codes are x's: pre_weight is needed")
    r, x, q, s = _norm_residual(residual, o, post_weight, gate, pre_weight, eps, alpha, beta, dtype,
                                residual_out, with_x, True, stream)
    return (r, q, s, x) if with_x else (r, q, s)


def norm_residual_backward(residual_out: torch.Tensor,
                           d_residual_out: Optional[torch.Tensor] = None,
                           d_x: Optional[torch.Tensor] = None,
                           o: Optional[torch.Tensor] = None,
                           post_weight: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None,
                           pre_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                           alpha: float = 1.0, beta: float = 1.0,
                           workspace: Optional[Workspace] = None, stream=None) -> dict:
    """beam_moe_norm_residual_backward.  residual_out is the forward's r' (its
    residual without o); d_residual_out and d_x are the gradients of r' and x
    (None for zero, not both; d_x is needed without o).  Returns a dict: d_residual [T,H] fp32; with o
    d_o and d_post_weight, with gate d_gate, with d_x d_pre_weight."""
    if d_residual_out is None and d_x is None:
        raise ValueError("one of d_residual_out and d_x is needed")
    if d_x is None and o is None:
        raise ValueError("without o there is only the gradient of x: d_x is needed")
    if d_x is not None and pre_weight is None:
        raise ValueError("d_x needs the pre_weight")
    T, H, dev, dtype, po, pw, pg, cols, pp = _norm_inputs(
        residual_out, o, post_weight, gate, pre_weight,
        d_x.dtype if o is None and d_x is not None else None)
    device, f32, on = residual_out.device, torch.float32, _on(stream, dev)
    pr = _arg("residual_out", residual_out, dev, f32, (T, H))
    p_dr = None if d_residual_out is None else _arg("d_residual_out", d_residual_out, dev, f32, (T, H))
    p_dx = None if d_x is None else _arg("d_x", d_x, dev, dtype, (T, H))
    need = ctypes.c_size_t(0)
    _check(lib().beam_moe_norm_residual_workspace_bytes(T, H, ctypes.byref(need)),
           "beam_moe_norm_residual_workspace_bytes")
    out = {"d_residual": _empty(on, device, f32, T, H)}
    if o is not None:
        out["d_o"] = _empty(on, device, dtype, T, H)
        out["d_post_weight"] = _empty(on, device, f32, H)
        if gate is not None:
            out["d_gate"] = _empty(on, device, dtype, T, cols)
    if d_x is not None:
        out["d_pre_weight"] = _empty(on, device, f32, H)
    buf = _scratch(need.value, workspace, device, stream)
    ptr = {k: v.data_ptr() for k, v in out.items()}
    _run(lib().beam_moe_norm_residual_backward, "beam_moe_norm_residual_backward", on, dev,
         (residual_out, d_residual_out, d_x, o, post_weight, gate, pre_weight, *out.values()),
         T, H, BF16 if dtype is torch.bfloat16 else F32, po, pw, pg, cols, pp, eps, alpha, beta, pr,
         p_dr, p_dx, ptr["d_residual"], ptr.get("d_o"), ptr.get("d_gate"), ptr.get("d_pre_weight"),
         ptr.get("d_post_weight"), None if buf is None else buf.data_ptr(), need.value)
    return out


class Timer:
    """beam_moe_timer: HIP event pairs around each kernel of a timed forward."""

    def __init__(self, capacity: int = 4096):
        h = ctypes.c_void_p()
        _check(lib().beam_moe_timer_create(capacity, ctypes.byref(h)),
               "beam_moe_timer_create")
        self.handle = h

    def reset(self):
        lib().beam_moe_timer_reset(self.handle)

    def records(self):
        """[(kernel name, ms)] in launch order; waits for the events."""
        L = lib()
        out = []
        for i in range(L.beam_moe_timer_count(self.handle)):
            name, ms = ctypes.c_char_p(), ctypes.c_float()
            _check(L.beam_moe_timer_read(self.handle, i, ctypes.byref(name),
                                         ctypes.byref(ms)), "beam_moe_timer_read")
            out.append((name.value.decode(), ms.value))
        return out

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.beam_moe_timer_destroy(self.handle)
            self.handle = None


def forward(desc: Desc, x: torch.Tensor, w_router: Optional[torch.Tensor],
            bias: Optional[torch.Tensor], w_gate_up: torch.Tensor,
            w_down: torch.Tensor, s_gate_up: Optional[torch.Tensor] = None,
            s_down: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, logits: Optional[torch.Tensor] = None,
            return_routing: bool = False, workspace: Optional[Workspace] = None,
            stream=None, timer: Optional[Timer] = None):
    """beam_moe_forward (beam_moe_forward_timed with a timer).  Returns out
    [T,H] (act dtype), or (out, topk_idx, topk_w, logits) with
    return_routing."""
    T, dev = x.shape[0], x.device
    idx = w = None
    with _alloc_on(stream):
        if out is None:
            out = torch.empty(T, desc.hidden, dtype=x.dtype, device=dev)
        if return_routing:
            idx = torch.empty(T, desc.top_k, dtype=torch.int32, device=dev)
            w = torch.empty(T, desc.top_k, dtype=torch.float32, device=dev)
            if logits is None:
                logits = torch.empty(T, desc.n_experts, dtype=torch.float32, device=dev)
    buf, n = _ws(desc, T, workspace, dev, stream)
    args = [ctypes.byref(desc), T, _p(x), _p(w_router), _p(bias), _p(w_gate_up),
            _p(s_gate_up), _p(w_down), _p(s_down), _p(out), _p(idx), _p(w),
            _p(logits), _p(buf), n, _stream(stream, dev)]
    if timer is None:
        _check(lib().beam_moe_forward(*args), "beam_moe_forward")
    else:
        _check(lib().beam_moe_forward_timed(*args, timer.handle),
               "beam_moe_forward_timed")
    if return_routing:
        return out, idx, w, logits
    return out


def forward_noalloc(desc: Desc, x: torch.Tensor, w_router: Optional[torch.Tensor],
                    bias: Optional[torch.Tensor], w_gate_up: torch.Tensor,
                    w_down: torch.Tensor, out: torch.Tensor,
                    s_gate_up: Optional[torch.Tensor] = None,
                    s_down: Optional[torch.Tensor] = None,
                    topk_idx: Optional[torch.Tensor] = None,
                    topk_w: Optional[torch.Tensor] = None,
                    logits: Optional[torch.Tensor] = None, stream=None):
    """beam_moe_forward_noalloc: the block with the library's own per-device
    scratch array as workspace (at most NOALLOC_SCRATCH_BYTES).  Every output
    is the caller's; nothing is allocated.  Calls that may overlap on one GPU
    race on the shared array."""
    T, dev = x.shape[0], x.device
    _check(lib().beam_moe_forward_noalloc(
        ctypes.byref(desc), T, _p(x), _p(w_router), _p(bias), _p(w_gate_up),
        _p(s_gate_up), _p(w_down), _p(s_down), _p(out), _p(topk_idx), _p(topk_w),
        _p(logits), _stream(stream, dev)), "beam_moe_forward_noalloc")
    return out
