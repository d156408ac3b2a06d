"""block_scaled_fp4_topk_amd -- Python binding of libmoefp4 (MI355X / gfx950).

Thin ctypes marshalling over the C ABI declared in ``include/moefp4.h``:
every step of the MoE forward and of the requantisation runs in the HIP
kernels of the library.  PyTorch only provides device memory and the current
stream.  There is no CPU fallback: if ``libmoefp4.so`` is missing or no GPU is
present the calls raise.

Functions mirror the C entry points:
  workspace_bytes(problem)            -> moe_fp4_workspace_bytes
  workspace_offsets(problem)          -> moe_fp4_workspace_offsets
  gate(x, gate_w, top_k, ...)         -> moe_fp4_gate (the router)
  route(problem, topk_ids, ...)       -> moe_fp4_route
  forward(x, topk_ids, topk_w, ...)   -> moe_fp4_forward (fused=True: moe_fp4_forward_fused)
  layer(x, gate_w, top_k, w13, ...)   -> moe_fp4_layer (router and forward)
  forward_static(x, topk_ids, ...)    -> moe_fp4_forward_static (no workspace)
  project(x, w, w_sf, w_gs, ...)      -> moe_fp4_project (FP4 projection with low-rank adapters)
  grouped(x, w, offsets, ...)         -> moe_fp4_grouped (products grouped by expert, bfloat16 or FP4 weights)
  grouped_dx(dy, w, offsets, ...)     -> moe_fp4_grouped_dx (their gradient towards the rows)
  grouped_dw(dy, x, offsets, ...)     -> moe_fp4_grouped_dw (and towards the weights)
  block_norm(h, y, ...)               -> moe_fp4_block_norm (norms around a layer, gate and residual scale)
  block_norm_grad(dh, dn, h, y, ...)  -> moe_fp4_block_norm_grad (their gradient)
  requant_gran_k(src, src_sf, ...)    -> fp4_requant_gran_k
  prepare_gemm_weights(src, src_sf, ...) -> moe_fp4_prepare_gemm_weights
  prepare_gemm_weights_g16(src, src_sf, src_gs, ...) -> moe_fp4_prepare_gemm_weights_g16
  quantize_act(x, ...)                -> moe_fp4_quantize_act
  quantize_act_fp4(x, ...)            -> moe_fp4_quantize_act_fp4

None of them records a graph for autograd: results need no gradient, whatever
the arguments do; gradients are calls of their own (grouped_dx, grouped_dw,
block_norm_grad).
"""

from __future__ import annotations

import ctypes
import functools
import os
import struct

__all__ = ["Problem", "MoeFp4Error", "lib", "workspace_bytes", "workspace_offsets", "gate", "route", "forward",
           "forward_problem", "forward_static", "layer", "project", "grouped", "grouped_dx", "grouped_dw",
           "block_norm", "block_norm_grad",
           "requant_gran_k", "prepare_gemm_weights", "prepare_gemm_weights_g16", "quantize_act", "quantize_act_fp4",
           "dropped_assignments", "abandoned_waits", "LIB_PATH"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoefp4.so")

OK, EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP = range(5)
ACT_BF16, ACT_FP8_UE8M0_K32, ACT_BF16_QUANT_FP8_K32, ACT_FP4_UE8M0_K32, ACT_BF16_QUANT_FP4_K32 = range(5)
GATE_UP, UP_GATE = 0, 1


OUT_BF16, OUT_F32 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GATE_W_BF16, GATE_W_F32 = 0, 1
W_RAW, W_GEMM = 0, 1
_LAYOUTS = {"raw": W_RAW, "gemm": W_GEMM}
_LAYER_ACT = {False: ACT_BF16, None: ACT_BF16, True: ACT_BF16_QUANT_FP8_K32, "fp8": ACT_BF16_QUANT_FP8_K32,
              "fp4": ACT_BF16_QUANT_FP4_K32}


class Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "E", "top_k", "H", "I", "gran_k", "act_fmt", "w13_order", "out_fmt", "w_layout")]


class Gate(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("top_k", "shared", "scoring", "renormalize", "w_fmt")] + \
        [("scale", ctypes.c_float)]


class Linear(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("T", "N", "K")] + \
        [(n, ctypes.c_int32) for n in ("gran_k", "out_fmt", "adapters", "rank")]


class Grouped(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("M", "N", "K")] + \
        [(n, ctypes.c_int32) for n in ("E", "gran_k", "out_fmt")]


class Norm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("T", "H")] + \
        [(n, ctypes.c_int32) for n in ("h_fmt", "post_fmt", "pre_fmt", "gate_fmt", "gate_kind", "gate_sigmoid")] + \
        [(n, ctypes.c_float) for n in ("scale", "h_scale", "eps")]


class MoeFp4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"moefp4 status {status}: {message}")
        self.status = status


_lib = None
_P = ctypes.c_void_p


def lib():
    """Load libmoefp4.so (built in-tree by ``python -m block_scaled_fp4_topk_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run python -m block_scaled_fp4_topk_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        st = ctypes.c_int
        L.moe_fp4_workspace_bytes.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(ctypes.c_size_t)]
        L.moe_fp4_workspace_bytes.restype = st
        L.moe_fp4_workspace_offsets.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(ctypes.c_size_t),
                                                ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
        L.moe_fp4_workspace_offsets.restype = st
        L.moe_fp4_route.argtypes = [ctypes.POINTER(Problem), _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.moe_fp4_route.restype = st
        i64 = ctypes.c_int64
        L.moe_fp4_gate_workspace_bytes.argtypes = [ctypes.POINTER(Gate), i64, i64, i64,
                                                   ctypes.POINTER(ctypes.c_size_t)]
        L.moe_fp4_gate_workspace_bytes.restype = st
        L.moe_fp4_gate.argtypes = [ctypes.POINTER(Gate), i64, i64, i64, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.moe_fp4_gate.restype = st
        gp = ctypes.POINTER(Gate)
        L.moe_fp4_layer_workspace_bytes.argtypes = [ctypes.POINTER(Problem), gp, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_fp4_layer_workspace_bytes.restype = st
        L.moe_fp4_layer.argtypes = [ctypes.POINTER(Problem), gp] + [_P] * 13 + [ctypes.c_size_t, _P]
        L.moe_fp4_layer.restype = st
        lp = ctypes.POINTER(Linear)
        L.moe_fp4_project_workspace_bytes.argtypes = [lp, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_fp4_project_workspace_bytes.restype = st
        L.moe_fp4_project.argtypes = [lp] + [_P] * 10 + [ctypes.c_size_t, _P]
        L.moe_fp4_project.restype = st
        rp = ctypes.POINTER(Grouped)
        L.moe_fp4_grouped_workspace_bytes.argtypes = [rp, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_fp4_grouped_workspace_bytes.restype = st
        L.moe_fp4_grouped.argtypes = [rp] + [_P] * 7 + [ctypes.c_size_t, _P]
        L.moe_fp4_grouped.restype = st
        L.moe_fp4_grouped_dx.argtypes = L.moe_fp4_grouped.argtypes
        L.moe_fp4_grouped_dx.restype = st
        L.moe_fp4_grouped_dw.argtypes = [rp] + [_P] * 4 + [ctypes.c_int32, _P, ctypes.c_size_t, _P]
        L.moe_fp4_grouped_dw.restype = st
        np_ = ctypes.POINTER(Norm)
        L.moe_fp4_block_norm.argtypes = [np_] + [_P] * 8
        L.moe_fp4_block_norm.restype = st
        L.moe_fp4_block_norm_grad_workspace_bytes.argtypes = [np_, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_fp4_block_norm_grad_workspace_bytes.restype = st
        L.moe_fp4_block_norm_grad.argtypes = [np_] + [_P] * 13 + [ctypes.c_size_t, _P]
        L.moe_fp4_block_norm_grad.restype = st
        L.moe_fp4_forward.argtypes = [ctypes.POINTER(Problem), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                      _P, _P, ctypes.c_size_t, _P]
        L.moe_fp4_forward.restype = st
        L.moe_fp4_forward_fused.argtypes = L.moe_fp4_forward.argtypes
        L.moe_fp4_forward_fused.restype = st
        L.moe_fp4_forward_static.argtypes = [ctypes.POINTER(Problem), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                             _P, _P]
        L.moe_fp4_forward_static.restype = st
        L.fp4_requant_gran_k.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _P, _P,
                                         ctypes.c_int32, _P, _P, _P, ctypes.c_int32, _P]
        L.fp4_requant_gran_k.restype = st
        L.moe_fp4_prepare_gemm_weights.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                   ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _P]
        L.moe_fp4_prepare_gemm_weights.restype = st
        L.moe_fp4_prepare_gemm_weights_g16.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                       ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _P, _P]
        L.moe_fp4_prepare_gemm_weights_g16.restype = st
        L.moe_fp4_quantize_act.argtypes = [ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P]
        L.moe_fp4_quantize_act.restype = st
        L.moe_fp4_quantize_act_fp4.argtypes = [ctypes.c_int64, ctypes.c_int64, _P, _P, _P, _P]
        L.moe_fp4_quantize_act_fp4.restype = st
        L.moefp4_last_error.argtypes = []
        L.moefp4_last_error.restype = ctypes.c_char_p
        L.moefp4_mfma_peak_probe.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P,
                                             ctypes.POINTER(ctypes.c_double), _P]
        L.moefp4_mfma_peak_probe.restype = st
        L.moefp4_set_stage_events.argtypes = [_P, ctypes.c_int32]
        L.moefp4_set_stage_events.restype = st
        L.moefp4_set_wait_looks.argtypes = [ctypes.c_int32]
        L.moefp4_set_wait_looks.restype = st
        L.moefp4_version.argtypes = []
        L.moefp4_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(status: int):
    if status != OK:
        raise MoeFp4Error(status, lib().moefp4_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, name, dtypes):
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# gate / layer / project are called for single tokens, where the host's work
# per call shows: one test per tensor argument, workspace sizes remembered per
# problem, raw addresses handed to ctypes.


def _arg(t, name, dtypes, shape, device):
    """A tensor argument of gate / layer / project: its type, shape, layout and device, which must be the first
    argument's and the current one (the library launches on the current device).  Returns its address."""
    if t is None:
        return None
    try:
        if t.dtype in dtypes and t.shape == shape and t.device == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, name, dtypes)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, expected {device}")


def _dims(t, name, dtypes, dims):
    """A tensor whose sizes others are measured by: its type, number of dimensions and layout."""
    if _dev(t, name, dtypes) is None:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    return t.shape


def _current(t, stream):
    """The tensor's device, which must be the current one and the stream's (a kernel is launched on the current
    device)."""
    import torch
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"tensors are on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    if stream is not None and stream.device_index != t.get_device():
        raise ValueError(f"tensors are on {t.device}, but the stream is on cuda:{stream.device_index}")
    return t.device


def _empty(like, shape, dtype, stream):
    """Memory on like's device for work on ``stream`` (allocated on it, so that the allocator does not hand it to
    another one)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _scratch(workspace, need, like, stream):
    import torch
    if workspace is None:
        return _empty(like, max(need, 256), torch.uint8, stream)
    _dev(workspace, "workspace", (torch.uint8,))
    if workspace.device != like.device:
        raise ValueError(f"workspace is on {workspace.device}, expected {like.device}")
    return workspace


def _raw_stream(stream, device):
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _need(fn, *args):
    n = ctypes.c_size_t(0)
    _check(fn(*args, ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=1024)
def _gate_need(top_k, shared, scoring, w_fmt, T, E, H):
    return _need(lib().moe_fp4_gate_workspace_bytes, ctypes.byref(make_gate(top_k, scoring, False, 1.0, shared, w_fmt)),
                 T, E, H)


@functools.lru_cache(maxsize=1024)
def _layer_need(device, top_k, shared, scoring, w_fmt, *problem):
    g = make_gate(top_k, scoring, False, 1.0, shared, w_fmt)
    return _need(lib().moe_fp4_layer_workspace_bytes, ctypes.byref(Problem(*problem)), ctypes.byref(g))


@functools.lru_cache(maxsize=1024)
def _grouped_problem(direction, *problem):
    """(the problem as the library takes it, the workspace it needs)"""
    p = ctypes.byref(Grouped(*problem))
    return p, _need(lib().moe_fp4_grouped_workspace_bytes, p, direction)


def _grouped_need(direction, *problem):
    return _grouped_problem(direction, *problem)[1]


@functools.lru_cache(maxsize=1024)
def _norm_grad_need(T, H):
    return _need(lib().moe_fp4_block_norm_grad_workspace_bytes, ctypes.byref(Norm(T, H, eps=1.0)))


@functools.lru_cache(maxsize=1024)
def _project_need(*linear):
    return _need(lib().moe_fp4_project_workspace_bytes, ctypes.byref(Linear(*linear)))


def _order(w13_order):
    if isinstance(w13_order, str):
        return {"gate_up": GATE_UP, "w31": GATE_UP, "up_gate": UP_GATE, "w13": UP_GATE}[w13_order]
    return w13_order


def make_problem(T, E, top_k, H, I, gran_k, act_fmt=ACT_BF16, w13_order=GATE_UP,
                 out_fmt=OUT_BF16, w_layout=W_RAW) -> Problem:
    if isinstance(w_layout, str):
        w_layout = {"raw": W_RAW, "gemm": W_GEMM}[w_layout]
    return Problem(T, E, top_k, H, I, gran_k, act_fmt, _order(w13_order), out_fmt, w_layout)


def workspace_bytes(problem: Problem) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_fp4_workspace_bytes(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def workspace_offsets(problem: Problem):
    """(h, h_sf, slot_of) byte offsets of the forward's intermediate h, its
    UE8M0 scales (0 if none) and the assignment -> slot map in the workspace
    (moe_fp4_workspace_offsets)."""
    h, hs, so = ctypes.c_size_t(0), ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().moe_fp4_workspace_offsets(ctypes.byref(problem), ctypes.byref(h), ctypes.byref(hs),
                                           ctypes.byref(so)))
    return h.value, hs.value, so.value


def _workspace(problem, workspace, device):
    import torch
    need = workspace_bytes(problem)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    return workspace


def make_gate(top_k, scoring="softmax", renormalize=False, scale=1.0, shared=0, w_fmt=GATE_W_BF16) -> Gate:
    if isinstance(scoring, str):
        if scoring not in ("softmax", "sigmoid"):
            raise ValueError(f"scoring must be 'softmax' or 'sigmoid', got {scoring!r}")
        scoring = SCORE_SIGMOID if scoring == "sigmoid" else SCORE_SOFTMAX
    return Gate(top_k, shared, scoring, 1 if renormalize else 0, w_fmt, scale)


def _router_args(x, gate_w, bias, stream):
    """(T, E, H, w_fmt, device, addresses) of a router's tensors, checked."""
    import torch
    wt = (torch.bfloat16, torch.float32)
    (T, H), (E, _) = _dims(x, "x", (torch.bfloat16,), 2), _dims(gate_w, "gate_w", wt, 2)
    dev = _current(x, stream)
    at = x.data_ptr(), _arg(gate_w, "gate_w", wt, (E, H), dev), _arg(bias, "bias", (torch.float32,), (E,), dev)
    return T, E, H, GATE_W_F32 if gate_w.dtype is torch.float32 else GATE_W_BF16, dev, at


def gate(x, gate_w, top_k, bias=None, scoring="softmax", renormalize=False, scale=1.0, shared=0, topk_ids=None,
         topk_w=None, workspace=None, stream=None):
    """The router: (topk_ids [T, top_k + shared] int32, topk_w float32) for
    forward().  x [T, H] bfloat16; gate_w [E, H] bfloat16 or float32; bias [E]
    float32 or None, added to the scores for the selection only (-inf masks an
    expert); scoring "softmax" or "sigmoid"; renormalize divides the selected
    scores by their sum; scale multiplies the weights; shared appends experts
    E, E + 1, ... with weight 1.  Places without an expert (everything masked,
    or logits that are not finite) hold id -1 and weight 0."""
    import torch
    T, E, H, w_fmt, dev, at = _router_args(x, gate_w, bias, stream)
    g = make_gate(top_k, scoring, renormalize, scale, shared, w_fmt)
    need = _gate_need(top_k, shared, scoring, w_fmt, T, E, H)
    shape = (T, top_k + shared)
    if topk_ids is None:
        topk_ids = _empty(x, shape, torch.int32, stream)
    if topk_w is None:
        topk_w = _empty(x, shape, torch.float32, stream)
    ws = _scratch(workspace, need, x, stream)
    _check(_lib.moe_fp4_gate(ctypes.byref(g), T, E, H, *at, _arg(topk_ids, "topk_ids", (torch.int32,), shape, dev),
                             _arg(topk_w, "topk_w", (torch.float32,), shape, dev), ws.data_ptr(), ws.numel(),
                             _raw_stream(stream, dev)))
    return topk_ids, topk_w


def route(problem: Problem, topk_ids, workspace=None, stream=None):
    """Returns (counts [E], offsets [E+1], sorted_assign [T*k], slot_of [T*k]) int32 tensors."""
    import torch
    _dev(topk_ids, "topk_ids", (torch.int32,))
    dev = topk_ids.device
    A = problem.T * problem.top_k
    counts = torch.empty(problem.E, dtype=torch.int32, device=dev)
    offsets = torch.empty(problem.E + 1, dtype=torch.int32, device=dev)
    sa = torch.empty(max(A, 1), dtype=torch.int32, device=dev)
    so = torch.empty(max(A, 1), dtype=torch.int32, device=dev)
    ws = _workspace(problem, workspace, dev)
    _check(lib().moe_fp4_route(ctypes.byref(problem), _ptr(topk_ids), _ptr(counts), _ptr(offsets),
                               _ptr(sa), _ptr(so), _ptr(ws), ws.numel(), _stream(stream)))
    return counts, offsets, sa[:A], so[:A]


def forward_problem(x, topk_ids, w13, w2, gran_k, x_sf=None, w13_order="gate_up", out_dtype=None,
                    quantize_x=False, w_layout="raw") -> Problem:
    """The problem descriptor forward() passes to moe_fp4_forward for these
    arguments (shapes from the tensors, the activation format from x / x_sf
    / quantize_x)."""
    import torch
    quant = {False: None, None: None, True: "fp8", "fp8": "fp8", "fp4": "fp4"}.get(quantize_x, "?")
    if quant == "?":
        raise ValueError(f"quantize_x must be False, True, 'fp8' or 'fp4', got {quantize_x!r}")
    a8 = x_sf is not None
    E, two_i, _ = w13.shape
    H = w2.shape[1]
    T, xcols = x.shape
    a4 = a8 and xcols * 2 == H
    if xcols != H and not a4:
        raise ValueError(f"x has {xcols} columns; expected H={H} (or H/2 packed FP4 codes with x_sf)")
    k = topk_ids.shape[1]
    if out_dtype is None:
        out_dtype = torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    if quant and a8:
        raise ValueError("quantize_x takes bfloat16 x without x_sf")
    act = (ACT_FP4_UE8M0_K32 if a4 else ACT_FP8_UE8M0_K32 if a8 else
           ACT_BF16_QUANT_FP8_K32 if quant == "fp8" else ACT_BF16_QUANT_FP4_K32 if quant == "fp4" else ACT_BF16)
    return make_problem(T, E, k, H, two_i // 2, gran_k, act, w13_order,
                        OUT_F32 if out_dtype == torch.float32 else OUT_BF16, w_layout)


def forward(x, topk_ids, topk_w, w13, w13_sf, w13_gs, w2, w2_sf, w2_gs, gran_k, x_sf=None,
            w13_order="gate_up", out=None, workspace=None, stream=None, out_dtype=None,
            quantize_x=False, w_layout="raw", fused=False):
    """MoE forward on the GPU.  x: [T, H] bfloat16 (A16); uint8/float8_e4m3fn
    [T, H] with x_sf [T, H/32] uint8 (A8); or uint8 [T, H/2] (two E2M1 codes
    per byte) with x_sf (A4).  quantize_x with bfloat16 x asks the library to
    quantise x first: True or "fp8" -> the A8 format (act_fmt
    BF16_QUANT_FP8_K32), "fp4" -> the A4 format (BF16_QUANT_FP4_K32).
    Weights uint8 as in include/moefp4.h; w_layout="gemm" for weights from
    prepare_gemm_weights.  fused=True runs FC1 and FC2 in one persistent
    launch (moe_fp4_forward_fused; 16-row decode tiles only, same result).
    Returns out [T, H] bfloat16 (default) or float32 (out_dtype=torch.float32)."""
    import torch
    u8 = (torch.uint8,)
    fp8 = (torch.uint8, torch.float8_e4m3fn)
    a8 = x_sf is not None
    _dev(x, "x", fp8 if a8 else (torch.bfloat16, torch.int16, torch.uint16))
    _dev(x_sf, "x_sf", u8)
    _dev(topk_ids, "topk_ids", (torch.int32,))
    _dev(topk_w, "topk_w", (torch.float32,))
    for n, t in (("w13", w13), ("w13_sf", w13_sf), ("w2", w2), ("w2_sf", w2_sf)):
        _dev(t, n, u8)
    _dev(w13_gs, "w13_gs", (torch.float32,))
    _dev(w2_gs, "w2_gs", (torch.float32,))
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    p = forward_problem(x, topk_ids, w13, w2, gran_k, x_sf, w13_order, out_dtype, quantize_x, w_layout)
    if out is None:
        out = torch.empty((p.T, p.H), dtype=out_dtype, device=x.device)
    _dev(out, "out", (out_dtype,))
    ws = _workspace(p, workspace, x.device)
    fn = lib().moe_fp4_forward_fused if fused else lib().moe_fp4_forward
    _check(fn(ctypes.byref(p), _ptr(x), _ptr(x_sf), _ptr(topk_ids), _ptr(topk_w), _ptr(w13), _ptr(w13_sf),
              _ptr(w13_gs), _ptr(w2), _ptr(w2_sf), _ptr(w2_gs), _ptr(out), _ptr(ws), ws.numel(),
              _stream(stream)))
    return out


def forward_static(x, topk_ids, topk_w, w13, w13_sf, w13_gs, w2, w2_sf, w2_gs, gran_k, x_sf=None,
                   w13_order="gate_up", out=None, stream=None, out_dtype=None, quantize_x=False, w_layout="raw"):
    """forward() without a workspace: moe_fp4_forward_static, whose
    workspace is the library's static device scratch (64 MiB per GPU; larger
    problems raise with status EWORKSPACE).  Calls that overlap on one GPU
    race; calls on one stream are ordered."""
    import torch
    u8 = (torch.uint8,)
    a8 = x_sf is not None
    _dev(x, "x", (torch.uint8, torch.float8_e4m3fn) if a8 else (torch.bfloat16, torch.int16, torch.uint16))
    _dev(x_sf, "x_sf", u8)
    _dev(topk_ids, "topk_ids", (torch.int32,))
    _dev(topk_w, "topk_w", (torch.float32,))
    for n, t in (("w13", w13), ("w13_sf", w13_sf), ("w2", w2), ("w2_sf", w2_sf)):
        _dev(t, n, u8)
    _dev(w13_gs, "w13_gs", (torch.float32,))
    _dev(w2_gs, "w2_gs", (torch.float32,))
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    p = forward_problem(x, topk_ids, w13, w2, gran_k, x_sf, w13_order, out_dtype, quantize_x, w_layout)
    if out is None:
        out = torch.empty((p.T, p.H), dtype=out_dtype, device=x.device)
    _dev(out, "out", (out_dtype,))
    _check(lib().moe_fp4_forward_static(ctypes.byref(p), _ptr(x), _ptr(x_sf), _ptr(topk_ids), _ptr(topk_w),
                                        _ptr(w13), _ptr(w13_sf), _ptr(w13_gs), _ptr(w2), _ptr(w2_sf),
                                        _ptr(w2_gs), _ptr(out), _stream(stream)))
    return out


def layer(x, gate_w, top_k, w13, w13_sf, w13_gs, w2, w2_sf, w2_gs, gran_k, bias=None, scoring="softmax",
          renormalize=False, scale=1.0, shared=0, w13_order="gate_up", out=None, workspace=None, stream=None,
          out_dtype=None, quantize_x=False, w_layout="raw", topk_ids=None, topk_w=None):
    """A whole mixture-of-experts layer on bfloat16 x [T, H]: gate() with
    gate_w [E - shared, H], then forward() over the E experts of the weight
    tensors, the last `shared` of which every token takes with weight 1.  Up
    to 8 tokens (2 with group32 weights) run in two launches (moe_fp4_layer).  quantize_x, w_layout,
    w13_order and out_dtype as for forward(); topk_ids / topk_w
    [T, top_k + shared]: optional outputs for the selection.  Returns out
    [T, H]; NaN stands where a wait inside the two-launch form exceeded its
    bound (abandoned_waits counts them)."""
    import torch
    T, routed, H, w_fmt, dev, at = _router_args(x, gate_w, bias, stream)
    act = _LAYER_ACT.get(quantize_x)
    if act is None:
        raise ValueError(f"quantize_x must be False, True, 'fp8' or 'fp4', got {quantize_x!r}")
    if gran_k not in (16, 32):
        raise ValueError(f"gran_k must be 16 or 32, got {gran_k}")
    u8, f32 = (torch.uint8,), (torch.float32,)
    E, kt = routed + shared, top_k + shared
    I = _dims(w13, "w13", u8, 3)[1] // 2
    weights = (_arg(w13, "w13", u8, (E, 2 * I, H // 2), dev), _arg(w13_sf, "w13_sf", u8, (E, 2 * I, H // gran_k), dev),
               _arg(w13_gs, "w13_gs", f32, (E,), dev), _arg(w2, "w2", u8, (E, H, I // 2), dev),
               _arg(w2_sf, "w2_sf", u8, (E, H, I // gran_k), dev), _arg(w2_gs, "w2_gs", f32, (E,), dev))
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    g = make_gate(top_k, scoring, renormalize, scale, shared, w_fmt)
    problem = (T, E, kt, H, I, gran_k, act, _order(w13_order), OUT_F32 if out_dtype is torch.float32 else OUT_BF16,
               _LAYOUTS.get(w_layout, w_layout))
    need = _layer_need(dev, top_k, shared, scoring, w_fmt, *problem)
    if out is None:
        out = _empty(x, (T, H), out_dtype, stream)
    ws = _scratch(workspace, need, x, stream)
    _check(_lib.moe_fp4_layer(ctypes.byref(Problem(*problem)), ctypes.byref(g), *at, *weights,
                              _arg(out, "out", (out_dtype,), (T, H), dev),
                              _arg(topk_ids, "topk_ids", (torch.int32,), (T, kt), dev),
                              _arg(topk_w, "topk_w", f32, (T, kt), dev), ws.data_ptr(), ws.numel(),
                              _raw_stream(stream, dev)))
    return out


def project(x, w, w_sf, w_gs, gran_k, lora_a=None, lora_b=None, lora_id=None, lora_scale=None, out=None,
            workspace=None, stream=None, out_dtype=None):
    """A projection over FP4 weights with low-rank adapters beside it:
    out[t] = W x[t] + lora_scale[l] * B_l (A_l x[t]), l = lora_id[t] (outside
    [0, L), e.g. -1: no adapter).  x [T, K] bfloat16; w [N, K/2] uint8, w_sf
    [N, K/gran_k] uint8, w_gs [1] float32 or None; lora_a [L, R, K] and lora_b
    [L, N, R] bfloat16, lora_id [T] int32, lora_scale [L] float32, or all four
    None.  Returns out [T, N] bfloat16 (default) or float32."""
    import torch
    u8, f32, bf = (torch.uint8,), (torch.float32,), (torch.bfloat16,)
    (T, K), (N, _) = _dims(x, "x", bf, 2), _dims(w, "w", u8, 2)
    dev = _current(x, stream)
    if gran_k not in (16, 32):
        raise ValueError(f"gran_k must be 16 or 32, got {gran_k}")
    at = (x.data_ptr(), _arg(w, "w", u8, (N, K // 2), dev), _arg(w_sf, "w_sf", u8, (N, K // gran_k), dev),
          _arg(w_gs, "w_gs", f32, (1,), dev))
    adapters = rank = 0
    lora = (None, None, None, None)
    if lora_a is not None:
        if lora_b is None or lora_id is None or lora_scale is None:
            raise ValueError("lora_a, lora_b, lora_id and lora_scale go together")
        adapters, rank, _ = _dims(lora_a, "lora_a", bf, 3)
        if adapters < 1:
            raise ValueError("lora_a must be [L, R, K] with L >= 1")
        lora = (_arg(lora_a, "lora_a", bf, (adapters, rank, K), dev), _arg(lora_b, "lora_b", bf, (adapters, N, rank), dev),
                _arg(lora_id, "lora_id", (torch.int32,), (T,), dev),
                _arg(lora_scale, "lora_scale", f32, (adapters,), dev))
    elif lora_b is not None or lora_id is not None or lora_scale is not None:
        raise ValueError("lora_a, lora_b, lora_id and lora_scale go together")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    linear = (T, N, K, gran_k, OUT_F32 if out_dtype is torch.float32 else OUT_BF16, adapters, rank)
    need = _project_need(*linear)
    if out is None:
        out = _empty(x, (T, N), out_dtype, stream)
    ws = _scratch(workspace, need, x, stream)
    _check(_lib.moe_fp4_project(ctypes.byref(Linear(*linear)), *at, *lora, _arg(out, "out", (out_dtype,), (T, N), dev),
                                ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)))
    return out


def _out_dtype(out, out_dtype):
    import torch
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    return out_dtype, OUT_F32 if out_dtype is torch.float32 else OUT_BF16


def _grouped_scratch(need, workspace, like, stream):
    """(the workspace, held until the call is enqueued; its address; its size), None and 0 where none is needed."""
    if need == 0 and workspace is None:
        return None, None, 0
    ws = _scratch(workspace, need, like, stream)
    return ws, ws.data_ptr(), ws.numel()


def _grouped_product(entry, direction, name, x, w, offsets, w_sf, w_gs, gran_k, out, workspace, stream, out_dtype):
    import torch
    u8, bf = (torch.uint8,), (torch.bfloat16,)
    M, cols = _dims(x, name, bf, 2)
    dev = _current(x, stream)
    sf = gs = None
    if gran_k:
        if gran_k not in (16, 32):
            raise ValueError(f"gran_k must be None (bfloat16 weights), 16 or 32, got {gran_k}")
        gran_k = int(gran_k)  # (what the problem is remembered by: a tensor's value can change)
        E, N, K = _dims(w, "w", u8, 3)
        K *= 2
        if w_sf is None:
            raise ValueError("FP4 weights need w_sf")
        sf = _arg(w_sf, "w_sf", u8, (E, N, K // gran_k), dev)
        gs = _arg(w_gs, "w_gs", (torch.float32,), (E,), dev)
    else:
        E, N, K = _dims(w, "w", bf, 3)
        if w_sf is not None or w_gs is not None:
            raise ValueError("w_sf and w_gs go with FP4 weights (gran_k)")
    ins, outs = (K, N) if direction == 0 else (N, K)
    if cols != ins or w.device != dev:  # (what else _arg looks at is known)
        _arg(x, name, bf, (M, ins), dev)
        _arg(w, "w", (w.dtype,), w.shape, dev)
    out_dtype, fmt = _out_dtype(out, out_dtype)
    off = _arg(offsets, "offsets", (torch.int32,), (E + 1,), dev)
    problem, need = _grouped_problem(direction, M, N, K, E, gran_k or 0, fmt)
    if out is None:
        out = _empty(x, (M, outs), out_dtype, stream)
        out_at = out.data_ptr()
    else:
        out_at = _arg(out, "out", (out_dtype,), (M, outs), dev)
    ws, *room = _grouped_scratch(need, workspace, x, stream)
    _check(getattr(_lib, entry)(problem, x.data_ptr(), w.data_ptr(), sf, gs, off, out_at, *room, _raw_stream(stream, dev)))
    return out


def grouped(x, w, offsets, w_sf=None, w_gs=None, gran_k=None, out=None, workspace=None, stream=None, out_dtype=None):
    """Products grouped by expert: out[r] = W_e x[r] for the rows r in
    [offsets[e], offsets[e + 1]).  x [M, K] bfloat16; offsets [E + 1] int32,
    ascending (as route() gives them); w [E, N, K] bfloat16, or [E, N, K/2] uint8
    FP4 codes with w_sf [E, N, K/gran_k] uint8 (and w_gs [E] float32) and gran_k 16
    or 32 (a code times its scale is taken as a bfloat16: exact below 2^128, an
    infinity from there on).  Returns out [M, N] bfloat16 (default) or float32; rows outside
    [offsets[0], offsets[E]) are left as they are (not set, in an out that the call
    allocates).

    No call of this module records a graph for autograd: its results need no gradient,
    whatever its arguments do.  The gradients are calls of their own (grouped_dx,
    grouped_dw, block_norm_grad), for a torch.autograd.Function's backward."""
    return _grouped_product("moe_fp4_grouped", 0, "x", x, w, offsets, w_sf, w_gs, gran_k, out, workspace, stream,
                            out_dtype)


def grouped_dx(dy, w, offsets, w_sf=None, w_gs=None, gran_k=None, out=None, workspace=None, stream=None,
               out_dtype=None):
    """The gradient of grouped() towards its rows: out[r] = W_e^T dy[r], dy [M, N]
    bfloat16, the weights and offsets as grouped() takes them.  Returns out
    [M, K]; rows outside [offsets[0], offsets[E]) as there."""
    return _grouped_product("moe_fp4_grouped_dx", 1, "dy", dy, w, offsets, w_sf, w_gs, gran_k, out, workspace, stream,
                            out_dtype)


def grouped_dw(dy, x, offsets, out=None, accumulate=False, workspace=None, stream=None, out_dtype=None):
    """The gradient of grouped() towards its weights: out[e] = the sum over
    expert e's rows of dy[r] x[r]^T, zeros for an expert without rows.  dy [M, N]
    and x [M, K] bfloat16, offsets [E + 1] int32.  accumulate adds the sums to
    what out holds.  Returns out [E, N, K] bfloat16 (default) or float32."""
    import torch
    bf = (torch.bfloat16,)
    (M, N), (_, K) = _dims(dy, "dy", bf, 2), _dims(x, "x", bf, 2)
    dev = _current(dy, stream)
    E = _dims(offsets, "offsets", (torch.int32,), 1)[0] - 1
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    out_dtype, fmt = _out_dtype(out, out_dtype)
    at = dy.data_ptr(), _arg(x, "x", bf, (M, K), dev), _arg(offsets, "offsets", (torch.int32,), (E + 1,), dev)
    problem, need = _grouped_problem(2, M, N, K, E, 0, fmt)
    if out is None:
        out = _empty(dy, (E, N, K), out_dtype, stream)
        out_at = out.data_ptr()
    else:
        out_at = _arg(out, "out", (out_dtype,), (E, N, K), dev)
    ws, *room = _grouped_scratch(need, workspace, dy, stream)
    _check(_lib.moe_fp4_grouped_dw(problem, *at, out_at, 1 if accumulate else 0, *room, _raw_stream(stream, dev)))
    return out


_numbers = struct.Struct("3d")


@functools.lru_cache(maxsize=1024)
def _norm_problem(*fields):
    """The problem of a block norm as the library takes it; last of the fields: scale, h_scale and eps as _numbers."""
    return ctypes.byref(Norm(*fields[:-1], *_numbers.unpack(fields[-1])))


def _norm_args(first, name, y, post_w, gate, gate_act, pre_w, scale, h_scale, eps, stream):
    """((T, H), gate kind, problem, device, addresses of y, post_w, gate and pre_w) of a block norm whose residual
    stream's type and sizes are those of ``first``."""
    import torch
    bf, f32, some = (torch.bfloat16,), torch.float32, (torch.bfloat16, torch.float32)
    T, H = shape = _dims(first, name, some, 2)
    dev = _current(first, stream)
    if y is None and (post_w is not None or gate is not None):
        raise ValueError("post_w and gate go with y")
    if y is None and pre_w is None:
        raise ValueError("y or pre_w is needed")
    if gate_act is not None and gate_act != "sigmoid":
        raise ValueError(f"gate_act must be None or 'sigmoid', got {gate_act!r}")
    kind, gate_at, gate_fmt = 0, None, OUT_BF16
    if gate is not None:
        _dev(gate, "gate", some)
        # (a gate of T = H elements is one per channel; [T, 1] says per token)
        size = tuple(gate.shape)
        kind = 1 if size == (H,) else 2 if size == (T,) or size == (T, 1) else 3 if size == (T, H) else 0
        if kind == 0:
            raise ValueError(f"gate must have shape {(H,)}, {(T,)}, {(T, 1)} or {(T, H)}, got {size}")
        gate_at, gate_fmt = _arg(gate, "gate", some, gate.shape, dev), OUT_F32 if gate.dtype is f32 else OUT_BF16
    at = (_arg(y, "y", bf, shape, dev), _arg(post_w, "post_w", some, (H,), dev), gate_at,
          _arg(pre_w, "pre_w", some, (H,), dev))
    # (what a problem is remembered by are its numbers' bits, as they are at this call: a tensor's value can change, and
    # -0.0 == 0.0)
    if not (type(scale) is type(h_scale) is type(eps) is float):
        scale, h_scale, eps = (ctypes.c_double(v).value for v in (scale, h_scale, eps))
    problem = _norm_problem(T, H, OUT_F32 if first.dtype is f32 else OUT_BF16,
                            OUT_F32 if post_w is not None and post_w.dtype is f32 else OUT_BF16,
                            OUT_F32 if pre_w is not None and pre_w.dtype is f32 else OUT_BF16, gate_fmt, kind,
                            0 if gate_act is None else 1, _numbers.pack(scale, h_scale, eps))
    return shape, kind, problem, dev, at


def block_norm(h, y=None, post_w=None, gate=None, gate_act=None, scale=1.0, h_scale=1.0, pre_w=None, eps=1e-6,
               h_out=None, n=None, stream=None):
    """The norms before and after a layer with its gate and residual scale:
    h' = h_scale h + scale act(gate) a, a = rms(y) post_w (or y without post_w), and
    n = rms(h') pre_w; rms(v) = v / sqrt(mean(v^2) + eps).  h [T, H] bfloat16 or
    float32 (the residual stream), y [T, H] bfloat16 (the layer's output); gate [H]
    (per channel; also where T = H), [T] or [T, 1] (per token) or [T, H]; gate_act
    None or "sigmoid"; weights and gate bfloat16 or float32; eps from 1e-20 to 1.
    scale, h_scale and eps are numbers; of a tensor with one element the value at the
    call is taken, on the host (one on the device is waited for, and cannot be taken
    while a graph is captured).  h_out may be h (in place).  Returns (h', n): h' of h's
    type, n [T, H] bfloat16.  Without y h' is h itself; without pre_w n is None.  Nothing is
    recorded for autograd: the gradient is block_norm_grad()."""
    import torch
    shape, _, problem, dev, at = _norm_args(h, "h", y, post_w, gate, gate_act, pre_w, scale, h_scale, eps, stream)
    if y is None and h_out is not None:
        raise ValueError("h_out goes with y")
    if pre_w is None and n is not None:
        raise ValueError("n goes with pre_w")
    h_at, n_at = _arg(h_out, "h_out", (h.dtype,), shape, dev), _arg(n, "n", (torch.bfloat16,), shape, dev)
    if y is not None and h_out is None:
        h_out = _empty(h, shape, h.dtype, stream)
        h_at = h_out.data_ptr()
    if pre_w is not None and n is None:
        n = _empty(h, shape, torch.bfloat16, stream)
        n_at = n.data_ptr()
    _check((_lib or lib()).moe_fp4_block_norm(problem, h.data_ptr(), *at, h_at, n_at, _raw_stream(stream, dev)))
    return (h if y is None else h_out), n


def block_norm_grad(dh, dn, h, y=None, post_w=None, gate=None, gate_act=None, scale=1.0, h_scale=1.0, pre_w=None,
                    eps=1e-6, d_h=None, workspace=None, stream=None):
    """The gradient of block_norm(): dh and dn are those of h' and n (dh None: zero;
    dn None without pre_w), h is the h' that block_norm() returned (None without
    pre_w), the rest as block_norm() had it.  d_h may be dh (in place).  Returns
    (d_h, d_y, d_post_w, d_gate, d_pre_w), None for what block_norm() did not have:
    d_h of h's type, d_y bfloat16, the weights' and the gate's float32 (a gate [T, H]:
    of its type)."""
    import torch
    if (pre_w is None) != (dn is None) or (pre_w is None) != (h is None):
        raise ValueError("dn and h go with pre_w")
    first, name = (h, "h") if h is not None else (dh, "dh")
    shape, kind, problem, dev, at = _norm_args(first, name, y, post_w, gate, gate_act, pre_w, scale, h_scale, eps, stream)
    T, H = shape
    need = _norm_grad_need(T, H)
    own = (first.dtype,)
    bf16, f32 = torch.bfloat16, torch.float32
    dh_at, dn_at, h_at = _arg(dh, "dh", own, shape, dev), _arg(dn, "dn", (bf16,), shape, dev), None
    if h is not None:
        h_at = h.data_ptr()
    if d_h is None:
        d_h = _empty(first, shape, first.dtype, stream)
        d_h_at = d_h.data_ptr()
    else:
        d_h_at = _arg(d_h, "d_h", own, shape, dev)
    d_y = d_post = d_gate = d_pre = d_y_at = d_post_at = d_gate_at = d_pre_at = None
    if y is not None:
        d_y = _empty(first, shape, bf16, stream)
        d_y_at = d_y.data_ptr()
    if post_w is not None:
        d_post = _empty(first, (H,), f32, stream)
        d_post_at = d_post.data_ptr()
    if gate is not None:
        d_gate = _empty(first, gate.shape, gate.dtype if kind == 3 else f32, stream)
        d_gate_at = d_gate.data_ptr()
    if pre_w is not None:
        d_pre = _empty(first, (H,), f32, stream)
        d_pre_at = d_pre.data_ptr()
    ws = _scratch(workspace, need, first, stream)
    _check(_lib.moe_fp4_block_norm_grad(problem, dh_at, dn_at, h_at, *at, d_h_at, d_y_at, d_post_at, d_gate_at, d_pre_at,
                                        ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)))
    return d_h, d_y, d_post, d_gate, d_pre


def requant_gran_k(src, src_sf, src_gs=None, src_gran=16, dst_gran=32, dst=None, dst_sf=None,
                   stream=None):
    """Group16 -> group32 requantisation.  src [E, N, K/2] uint8, src_sf
    [E, N, K/16] uint8 (E4M3), src_gs [E] float32 or None.  Returns
    (dst [E, N, K/2], dst_sf [E, N, K/32]); dst may be src (in place)."""
    import torch
    _dev(src, "src", (torch.uint8,))
    _dev(src_sf, "src_sf", (torch.uint8,))
    _dev(src_gs, "src_gs", (torch.float32,))
    E, N, kh = src.shape
    K = 2 * kh
    if dst is None:
        dst = torch.empty_like(src)
    if dst_sf is None:
        dst_sf = torch.empty((E, N, K // dst_gran), dtype=torch.uint8, device=src.device)
    _dev(dst, "dst", (torch.uint8,))
    _dev(dst_sf, "dst_sf", (torch.uint8,))
    _check(lib().fp4_requant_gran_k(E, N, K, _ptr(src), _ptr(src_sf), src_gran, _ptr(src_gs),
                                    _ptr(dst), _ptr(dst_sf), dst_gran, _stream(stream)))
    return dst, dst_sf




def prepare_gemm_weights(src, src_sf, which, w13_order="gate_up", dst=None, dst_sf=None, stream=None):
    """RAW group32 weights (src [E, N, K/2] uint8, src_sf [E, N, K/32] uint8)
    -> (dst, dst_sf) of the same shapes in the prefill GEMM layout
    (moe_fp4_prepare_gemm_weights).  which: "w13" (or 0) / "w2" (or 1)."""
    import torch
    _dev(src, "src", (torch.uint8,))
    _dev(src_sf, "src_sf", (torch.uint8,))
    w = {"w13": 0, "w2": 1}.get(which, which)
    E, N, kh = src.shape
    if dst is None:
        dst = torch.empty_like(src)
    if dst_sf is None:
        dst_sf = torch.empty_like(src_sf)
    _dev(dst, "dst", (torch.uint8,))
    _dev(dst_sf, "dst_sf", (torch.uint8,))
    _check(lib().moe_fp4_prepare_gemm_weights(E, N, 2 * kh, w, _order(w13_order), _ptr(src), _ptr(src_sf),
                                              _ptr(dst), _ptr(dst_sf), _stream(stream)))
    return dst, dst_sf


def prepare_gemm_weights_g16(src, src_sf, src_gs, which, w13_order="gate_up", dst=None, dst_sf=None,
                             stream=None):
    """RAW group16 weights (src [E, N, K/2] uint8, src_sf [E, N, K/16] E4M3
    bytes, src_gs [E] float32 or None) -> (dst [E, N, K/2], dst_sf [E, N,
    K/32]) in the prefill GEMM layout with group32 UE8M0 scales, the global
    scale folded in (moe_fp4_prepare_gemm_weights_g16)."""
    import torch
    _dev(src, "src", (torch.uint8,))
    _dev(src_sf, "src_sf", (torch.uint8,))
    _dev(src_gs, "src_gs", (torch.float32,))
    w = {"w13": 0, "w2": 1}.get(which, which)
    E, N, kh = src.shape
    if dst is None:
        dst = torch.empty_like(src)
    if dst_sf is None:
        dst_sf = torch.empty((E, N, 2 * kh // 32), dtype=torch.uint8, device=src.device)
    _dev(dst, "dst", (torch.uint8,))
    _dev(dst_sf, "dst_sf", (torch.uint8,))
    _check(lib().moe_fp4_prepare_gemm_weights_g16(E, N, 2 * kh, w, _order(w13_order), _ptr(src), _ptr(src_sf),
                                                  _ptr(src_gs), _ptr(dst), _ptr(dst_sf), _stream(stream)))
    return dst, dst_sf


def quantize_act_fp4(x, x_fp4=None, x_sf=None, stream=None):
    """bfloat16 [T, H] -> (E2M1 codes [T, H/2] uint8, two per byte, UE8M0
    scales [T, H/32] uint8), per 32 elements (moe_fp4_quantize_act_fp4)."""
    import torch
    _dev(x, "x", (torch.bfloat16, torch.int16, torch.uint16))
    T, H = x.shape
    if x_fp4 is None:
        x_fp4 = torch.empty((T, H // 2), dtype=torch.uint8, device=x.device)
    if x_sf is None:
        x_sf = torch.empty((T, H // 32), dtype=torch.uint8, device=x.device)
    _dev(x_fp4, "x_fp4", (torch.uint8,))
    _dev(x_sf, "x_sf", (torch.uint8,))
    _check(lib().moe_fp4_quantize_act_fp4(T, H, _ptr(x), _ptr(x_fp4), _ptr(x_sf), _stream(stream)))
    return x_fp4, x_sf


def quantize_act(x, x_fp8=None, x_sf=None, stream=None):
    """bfloat16 [T, H] -> (E4M3 codes [T, H] uint8, UE8M0 scales [T, H/32]
    uint8), per 32 elements (moe_fp4_quantize_act)."""
    import torch
    _dev(x, "x", (torch.bfloat16, torch.int16, torch.uint16))
    T, H = x.shape
    if x_fp8 is None:
        x_fp8 = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    if x_sf is None:
        x_sf = torch.empty((T, H // 32), dtype=torch.uint8, device=x.device)
    _dev(x_fp8, "x_fp8", (torch.uint8,))
    _dev(x_sf, "x_sf", (torch.uint8,))
    _check(lib().moe_fp4_quantize_act(T, H, _ptr(x), _ptr(x_fp8), _ptr(x_sf), _stream(stream)))
    return x_fp8, x_sf


def mfma_peak_probe(a4: bool, iters: int, blocks: int, sink, stream=None) -> float:
    """Enqueue the register-only block-scaled MFMA loop (moefp4_mfma_peak_probe);
    returns the flops it performs.  sink: float32 CUDA tensor of blocks*256."""
    import torch
    _dev(sink, "sink", (torch.float32,))
    f = ctypes.c_double(0)
    _check(lib().moefp4_mfma_peak_probe(1 if a4 else 0, iters, blocks, _ptr(sink), ctypes.byref(f), _stream(stream)))
    return f.value


def set_stage_events(events_array, n: int):
    """Profiling hook (moefp4_set_stage_events): events_array is a ctypes
    array of 6 hipEvent_t handles, or None to stop recording."""
    _check(lib().moefp4_set_stage_events(events_array, n))


def set_wait_looks(looks: int):
    """Test hook (moefp4_set_wait_looks): how often later layer() calls of this
    thread look at FC1's counters before they give a wait up; negative: the
    default."""
    _check(lib().moefp4_set_wait_looks(looks))


def dropped_assignments(workspace) -> int:
    """Number of assignments with an expert id outside [0, E) in the last
    route / forward call that used ``workspace`` (synchronises)."""
    return int(workspace[:4].view(dtype=__import__("torch").int32).item())


def abandoned_waits(workspace) -> int:
    """Number of waits inside the last layer or fused forward call that used
    ``workspace`` that exceeded their bound (synchronises).  A layer's outputs
    behind such a wait are NaN."""
    return int(workspace[4:8].view(dtype=__import__("torch").int32).item())
