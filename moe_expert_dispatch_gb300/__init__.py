"""GB300 MoE expert block: thin Python binding of libmoe_gb300.so.

Every function here marshals torch tensors (device memory) and the current
CUDA stream into the C ABI of include/moe_expert.h and raises on a non-OK
status. All computation runs in the library's CUDA kernels; there is no
fallback: importing this package without the built library raises.
"""
from __future__ import annotations

import array
import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# MOE_GB300_DEBUG=1 loads the MOE_DEBUG build (device-side bounds checks of
# the row indices taken from row maps, reported as MOE_ERR_BOUNDS)
DEBUG = os.environ.get("MOE_GB300_DEBUG", "0") not in ("", "0")
# MOE_GB300_SANITIZE=1 loads the host-sanitizer build (AddressSanitizer and
# UndefinedBehaviorSanitizer on the host code; the process must preload their
# runtimes): it serves the host-side checks on a machine without a GPU
SANITIZE = os.environ.get("MOE_GB300_SANITIZE", "0") not in ("", "0")
LIB_PATH = os.path.join(_HERE, "libmoe_gb300_sanitize.so" if SANITIZE
                        else "libmoe_gb300_debug.so" if DEBUG else "libmoe_gb300.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python moe_expert_dispatch_gb300/build.py` "
        "(the expert block has no CPU or eager fallback)")

_lib = ctypes.CDLL(LIB_PATH)

MOE_OK = 0
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "expert id outside [0, E)",
          4: "workspace missing or too small", 5: "in-kernel wait timed out", 6: "CUDA error",
          7: "row index outside its buffer (debug build)"}
MOE_BF16, MOE_MXFP8 = 0, 1
TILE_M = 128

_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t


class moe_config(ctypes.Structure):
    _fields_ = [("ring_stages", ctypes.c_int), ("save_for_backward", ctypes.c_int),
                ("num_sms", ctypes.c_int), ("fuse_gather", ctypes.c_int),
                ("wait_limit_ns", ctypes.c_longlong),
                ("step_events", ctypes.POINTER(ctypes.c_void_p)),
                ("num_step_events", ctypes.c_int),
                ("mxfp8_tile_n", ctypes.c_int),
                ("cta_pairs", ctypes.c_int),
                ("mx_scales_pretiled", ctypes.c_int)]


class moe_gate_config(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int), ("n_group", ctypes.c_int), ("topk_group", ctypes.c_int),
                ("group_topk", ctypes.c_int), ("renormalise", ctypes.c_int),
                ("scale", ctypes.c_float)]


class moe_norm_config(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("stream_type", ctypes.c_int),
                ("weight_type", ctypes.c_int)]


class moe_dropout_config(ctypes.Structure):
    _fields_ = [("p", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("stream_type", ctypes.c_int),
                ("branch_type", ctypes.c_int)]


STEP_EVENTS = 5       # forward: start, routing, fc1+SwiGLU, fc2, unpermute
BWD_STEP_EVENTS = 7   # backward: start, dO+dprobs, dH, dXp, dX, dW1, dW2
# MXFP8 backward: start, dO + quantise, dH, quantise dA, dXp, dX, quantise x and h, dW1, dW2
MX_BWD_STEP_EVENTS = 9


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("moe_config_init", None, ctypes.POINTER(moe_config))
_sig("moe_status_string", ctypes.c_char_p, _i32)
_sig("moe_get_error", _i32, _vp)
_sig("moe_num_sms", _i32)
_sig("moe_padded_rows", _i64, _i64, _i32, _i32)
_sig("moe_counts_workspace_size", _sz, _i64, _i32)
_sig("moe_counts", _i32, _vp, _i64, _i32, _vp, _vp, _vp, _sz, _vp)
_sig("moe_counts_static", _i32, _vp, _i64, _i32, _vp, _vp, _vp)
_sig("moe_route_topk_workspace_size", _sz, _i64, _i32, _i32)
_sig("moe_route_topk", _i32, _vp, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_sig("moe_permute_workspace_size", _sz, _i64, _i32, _i32)
_sig("moe_permute", _i32, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
     _vp, _vp, _sz, _vp)
_sig("moe_unpermute", _i32, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp)
_sig("moe_quantize_mxfp8", _i32, _vp, _i64, _i32, _vp, _vp, _vp)
_sig("moe_permute_quantize_mxfp8", _i32, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _vp)
_sig("moe_workspace_size", _sz, _i64, _i32, _i32, _i32, _i32, ctypes.POINTER(moe_config), _i32)
_sig("moe_expert_forward", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _vp,
     _vp, _sz, ctypes.POINTER(moe_config), _vp)
_sig("moe_expert_forward_from_logits", _i32, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
     _i32, _vp, _vp, _vp, _vp, _sz, ctypes.POINTER(moe_config), _vp)
_sig("moe_workspace_size_pipelined", _sz, _i64, _i32, _i32, _i32, _i32, _i32)
_sig("moe_expert_forward_pipelined", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
     _i32, _vp, _i32, _vp, _sz, ctypes.POINTER(moe_config), _vp, _vp)
_sig("moe_expert_backward", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
     _i32, _vp, _sz, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _sz, ctypes.POINTER(moe_config), _vp)
_sig("moe_workspace_size_mxfp8", _sz, _i64, _i32, _i32, _i32, _i32, ctypes.POINTER(moe_config))
_sig("moe_workspace_size_mxfp8_backward", _sz, _i64, _i32, _i32, _i32, _i32)
_sig("moe_quantize_mxfp8_t", _i32, _vp, _i64, _i32, _i32, _vp, _vp, _vp)
_sig("moe_quantize_mxfp8_dual", _i32, _vp, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp)
_sig("moe_expert_backward_mxfp8", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
     _i32, _i32, _i32, _i32, _vp, _sz, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _sz,
     ctypes.POINTER(moe_config), _vp)
_sig("moe_expert_forward_mxfp8", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32,
     _i32, _i32, _i32, _vp, _vp, _sz, ctypes.POINTER(moe_config), _vp)
_sig("moe_tile_weight_scales_mxfp8", _i32, _vp, _vp, _vp, _i32, _i32, _i32,
     ctypes.POINTER(moe_config), _vp, _vp, _vp)

_sig("moe_gate_config_init", None, ctypes.POINTER(moe_gate_config))
_sig("moe_route_gate_workspace_size", _sz, _i64, _i32, _i32)
_sig("moe_route_gate", _i32, _vp, _i32, _vp, _i64, _i32, _i32, ctypes.POINTER(moe_gate_config),
     _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_sig("moe_route_gate_backward", _i32, _vp, _vp, _i32, _vp, _vp, _i64, _i32, _i32,
     ctypes.POINTER(moe_gate_config), _vp, _vp)
_sig("moe_norm_config_init", None, ctypes.POINTER(moe_norm_config))
_sig("moe_norm_residual", _i32, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _i32,
     ctypes.POINTER(moe_norm_config), _vp, _vp, _vp, _vp, _vp)
_sig("moe_norm_residual_backward_workspace_size", _sz, _i64, _i32, _i64)
_sig("moe_norm_residual_backward", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _i64,
     _i32, ctypes.POINTER(moe_norm_config), _vp, _vp, _vp, _vp, _vp, _i32, _vp, _sz, _vp)
_sig("moe_clip_grad_norm_workspace_size", _sz)
_sig("moe_clip_grad_norm", _i32, _vp, _vp, _vp, _vp, _i64, ctypes.c_float, _i32, ctypes.c_float,
     _vp, _vp, _sz, _vp)

_sig("moe_gated_ffn_workspace_size", _sz, _i64, _i32, _i32)
_sig("moe_gated_ffn", _i32, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
     _sz, _vp)
_sig("moe_gated_ffn_backward_workspace_size", _sz, _i64, _i32, _i32)
_sig("moe_gated_ffn_backward", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32,
     _i32, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _sz, _vp)
_sig("moe_lora_plan", _i32, _vp, _i64, _i32, _vp, _vp, _vp)
_sig("moe_lora_workspace_size", _sz, _i64, _i32, _i32)
_sig("moe_lora", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _vp,
     _vp, _vp, _sz, _vp)
_sig("moe_lora_backward_workspace_size", _sz, _i64, _i32, _i32)
_sig("moe_lora_backward", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32,
     _i32, _i32, _vp, _vp, _vp, _i32, _vp, _sz, _vp)
_sig("moe_dropout_config_init", None, ctypes.POINTER(moe_dropout_config))
_sig("moe_dropout_residual", _i32, _vp, _vp, _i64, _vp, ctypes.POINTER(moe_dropout_config), _vp,
     _vp)
_sig("moe_dropout_residual_backward", _i32, _vp, _i64, _vp, ctypes.POINTER(moe_dropout_config),
     _vp, _vp, _vp)


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)} (status {status})")
        self.status = status


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None, device=None):
    """The given stream, or the current stream of `device` (the device that
    the call's tensors live on); a given stream must belong to that device."""
    if stream is None:
        s = torch.cuda.current_stream(device)
    else:
        s = stream
        if device is not None and s.device != device:
            raise ValueError(f"stream is on {s.device}, the tensors on {device}")
    return ctypes.c_void_p(s.cuda_stream)


def _cuda(t, name, dtype=None, min_numel=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs at least {min_numel}")


def _device(*named):
    """The one CUDA device of the (name, tensor) pairs given (None tensors
    skipped). Every kernel of a call runs on the device of its tensors, and
    a call whose tensors live on two devices is refused before anything is
    launched."""
    dev, first = None, None
    for name, t in named:
        if t is None:
            continue
        if dev is None:
            dev, first = t.device, name
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device} but {first} is on {dev}: "
                             "all tensors of a call must share one device")
    return dev


def config(ring_stages=0, save_for_backward=False, num_sms=0, fuse_gather=False,
           wait_limit_ns=0, step_events=None, mxfp8_tile_n=0, cta_pairs=0,
           mx_scales_pretiled=False) -> moe_config:
    """A moe_config; step_events: optional list of MOE_STEP_EVENTS torch.cuda.Event
    (already recorded once, so that their CUDA events exist)."""
    c = moe_config()
    _lib.moe_config_init(ctypes.byref(c))
    c.ring_stages = ring_stages
    c.save_for_backward = int(bool(save_for_backward))
    c.num_sms = num_sms
    c.fuse_gather = int(bool(fuse_gather))
    c.mxfp8_tile_n = mxfp8_tile_n
    c.cta_pairs = cta_pairs
    c.mx_scales_pretiled = int(bool(mx_scales_pretiled))
    if wait_limit_ns:
        c.wait_limit_ns = wait_limit_ns
    if step_events is not None:
        n = len(step_events)
        arr = (ctypes.c_void_p * n)(*[ev.cuda_event for ev in step_events])
        c._events_keepalive = arr
        c.step_events = ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))
        c.num_step_events = n
    return c


def moe_get_error(stream=None) -> int:
    """Synchronises the stream (default: the current device's current stream)
    and returns (and clears) the error status of the stream's device."""
    if stream is None:
        return _lib.moe_get_error(_stream(None))
    with torch.cuda.device(stream.device):
        return _lib.moe_get_error(_stream(stream))


def moe_num_sms() -> int:
    return _lib.moe_num_sms()


def moe_padded_rows(n_rows: int, E: int, row_align: int = TILE_M) -> int:
    return _lib.moe_padded_rows(n_rows, E, row_align)


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def moe_counts(expert_ids: torch.Tensor, num_experts: int, counts=None, offsets=None,
               workspace=None, stream=None):
    """(counts int32 [E], offsets int32 [E+1]) of the flattened ids."""
    _cuda(expert_ids, "expert_ids", torch.int32)
    _cuda(counts, "counts", torch.int32, num_experts)
    _cuda(offsets, "offsets", torch.int32, num_experts + 1)
    _cuda(workspace, "workspace")
    dev = _device(("expert_ids", expert_ids), ("counts", counts), ("offsets", offsets),
                  ("workspace", workspace))
    n = expert_ids.numel()
    with torch.cuda.device(dev):
        counts = (torch.empty(num_experts, dtype=torch.int32, device=dev)
                  if counts is None else counts)
        offsets = (torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
                   if offsets is None else offsets)
        need = _lib.moe_counts_workspace_size(n, num_experts)
        ws = _workspace(need, dev) if workspace is None else workspace
        _check(_lib.moe_counts(_p(expert_ids), n, num_experts, _p(counts), _p(offsets), _p(ws),
                               ws.numel(), _stream(stream, dev)), "moe_counts")
    return counts, offsets


def moe_route_topk(logits: torch.Tensor, k: int, expert_ids=None, probs=None, counts=None,
                   offsets=None, workspace=None, stream=None):
    """The top-k softmax gate fused with the counts: (expert_ids int32 [T, k],
    probs float32 [T, k], counts int32 [E], offsets int32 [E+1]) of float32
    router logits [T, E]."""
    _cuda(logits, "logits", torch.float32)
    T, E = logits.shape
    _cuda(expert_ids, "expert_ids", torch.int32, T * k)
    _cuda(probs, "probs", torch.float32, T * k)
    _cuda(counts, "counts", torch.int32, E)
    _cuda(offsets, "offsets", torch.int32, E + 1)
    _cuda(workspace, "workspace")
    dev = _device(("logits", logits), ("expert_ids", expert_ids), ("probs", probs),
                  ("counts", counts), ("offsets", offsets), ("workspace", workspace))
    with torch.cuda.device(dev):
        expert_ids = (torch.empty((T, k), dtype=torch.int32, device=dev)
                      if expert_ids is None else expert_ids)
        probs = torch.empty((T, k), dtype=torch.float32, device=dev) if probs is None else probs
        counts = torch.empty(E, dtype=torch.int32, device=dev) if counts is None else counts
        offsets = (torch.empty(E + 1, dtype=torch.int32, device=dev)
                   if offsets is None else offsets)
        need = _lib.moe_route_topk_workspace_size(T, k, E)
        ws = _workspace(need, dev) if workspace is None else workspace
        _check(_lib.moe_route_topk(_p(logits), T, E, k, _p(expert_ids), _p(probs), _p(counts),
                                   _p(offsets), _p(ws), ws.numel(), _stream(stream, dev)),
               "moe_route_topk")
    return expert_ids, probs, counts, offsets


def moe_counts_static(expert_ids: torch.Tensor, num_experts: int, counts=None, offsets=None,
                      stream=None):
    """moe_counts with the library's fixed scratch instead of a workspace: it
    allocates no device memory (the output tensors are created here only when
    the caller passes none). Calls that overlap on the GPU race on that scratch."""
    _cuda(expert_ids, "expert_ids", torch.int32)
    _cuda(counts, "counts", torch.int32, num_experts)
    _cuda(offsets, "offsets", torch.int32, num_experts + 1)
    dev = _device(("expert_ids", expert_ids), ("counts", counts), ("offsets", offsets))
    with torch.cuda.device(dev):        # the scratch used is the one of this device
        counts = (torch.empty(num_experts, dtype=torch.int32, device=dev)
                  if counts is None else counts)
        offsets = (torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
                   if offsets is None else offsets)
        _check(_lib.moe_counts_static(_p(expert_ids), expert_ids.numel(), num_experts,
                                      _p(counts), _p(offsets), _stream(stream, dev)),
               "moe_counts_static")
    return counts, offsets


def moe_permute(x: torch.Tensor, expert_ids: torch.Tensor, probs, num_experts: int,
                row_align: int = 1, stream=None):
    """Stable permute of token rows into expert-contiguous rows.

    Returns dict(x_perm, row_of, token_of, prob_of, offsets, counts). With
    row_align > 1 every expert segment starts at a multiple of row_align rows
    and the padding rows of x_perm/token_of/prob_of are left uninitialised.
    """
    _cuda(x, "x")
    _cuda(expert_ids, "expert_ids", torch.int32)
    _cuda(probs, "probs", torch.float32)
    T, k = expert_ids.shape
    dev = _device(("x", x), ("expert_ids", expert_ids), ("probs", probs))
    with torch.cuda.device(dev):
        return _moe_permute(x, expert_ids, probs, num_experts, row_align, stream, T, k, dev)


def _moe_permute(x, expert_ids, probs, num_experts, row_align, stream, T, k, dev):
    row_bytes = x[0].numel() * x.element_size() if T else x.element_size()
    cap = _lib.moe_padded_rows(T * k, num_experts, row_align)
    out = dict(
        x_perm=torch.empty((cap,) + tuple(x.shape[1:]), dtype=x.dtype, device=dev),
        row_of=torch.empty((T, k), dtype=torch.int32, device=dev),
        token_of=torch.empty(cap, dtype=torch.int32, device=dev),
        prob_of=torch.empty(cap, dtype=torch.float32, device=dev),
        offsets=torch.empty(num_experts + 1, dtype=torch.int32, device=dev),
        counts=torch.empty(num_experts, dtype=torch.int32, device=dev),
    )
    ws = _workspace(_lib.moe_permute_workspace_size(T, k, num_experts), dev)
    _check(_lib.moe_permute(_p(x), T, row_bytes, _p(expert_ids), _p(probs), k, num_experts,
                            row_align, _p(out["x_perm"]), _p(out["row_of"]), _p(out["token_of"]),
                            _p(out["prob_of"]), _p(out["offsets"]), _p(out["counts"]), _p(ws),
                            ws.numel(), _stream(stream, dev)), "moe_permute")
    return out


def moe_unpermute(o_perm: torch.Tensor, row_of: torch.Tensor, probs=None, y=None, stream=None):
    """y[t] = bf16(sum_j probs[t, j] * o_perm[row_of[t, j]])."""
    _cuda(o_perm, "o_perm", torch.bfloat16)
    _cuda(row_of, "row_of", torch.int32)
    T, k = row_of.shape
    H = o_perm.shape[-1]
    _cuda(probs, "probs", torch.float32, T * k)
    _cuda(y, "y", torch.bfloat16, T * H)
    dev = _device(("o_perm", o_perm), ("row_of", row_of), ("probs", probs), ("y", y))
    with torch.cuda.device(dev):
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if y is None else y
        _check(_lib.moe_unpermute(_p(o_perm), _p(row_of), _p(probs), T, k, H, _p(y),
                                  _stream(stream, dev)), "moe_unpermute")
    return y


def moe_quantize_mxfp8(a: torch.Tensor, stream=None, out=None):
    """(codes uint8 [..., K], scales uint8 [..., K/32]) of a bf16 tensor along
    its last axis, written into out=(codes, scales) when given."""
    _cuda(a, "a", torch.bfloat16)
    K = a.shape[-1]
    rows = a.numel() // K if K else 0
    if out is None:
        q = torch.empty(a.shape, dtype=torch.uint8, device=a.device)
        s = torch.empty(a.shape[:-1] + (K // 32,), dtype=torch.uint8, device=a.device)
    else:
        q, s = out
        _cuda(q, "q", torch.uint8, a.numel())
        _cuda(s, "scales", torch.uint8, a.numel() // 32)
    dev = _device(("a", a), ("q", q), ("scales", s))
    with torch.cuda.device(dev):
        _check(_lib.moe_quantize_mxfp8(_p(a), rows, K, _p(q), _p(s), _stream(stream, dev)),
               "moe_quantize_mxfp8")
    return q, s


def moe_permute_quantize_mxfp8(x: torch.Tensor, row_of: torch.Tensor, n_rows: int | None = None,
                               stream=None, out=None):
    """The MXFP8 dispatch of bf16 x [T, H]: (codes uint8 [n_rows, H] holding
    token t's codes at every row_of[t, j] >= 0, scales uint8 [T, H/32] in
    token order), written into out=(codes, scales) when given. n_rows
    defaults to T * k; rows that row_of does not name stay zero."""
    _cuda(x, "x", torch.bfloat16)
    _cuda(row_of, "row_of", torch.int32)
    T, H = x.shape
    k = row_of.shape[1]
    if out is None:
        rows = T * k if n_rows is None else n_rows
        q = torch.zeros((rows, H), dtype=torch.uint8, device=x.device)
        s = torch.empty((T, H // 32), dtype=torch.uint8, device=x.device)
    else:
        q, s = out
        _cuda(q, "codes", torch.uint8)
        _cuda(s, "scales", torch.uint8, T * H // 32)
    dev = _device(("x", x), ("row_of", row_of), ("codes", q), ("scales", s))
    with torch.cuda.device(dev):
        _check(_lib.moe_permute_quantize_mxfp8(_p(x), T, H, _p(row_of), k, _p(q), _p(s),
                                               _stream(stream, dev)),
               "moe_permute_quantize_mxfp8")
    return q, s


def moe_quantize_mxfp8_t(a: torch.Tensor, stream=None, out=None):
    """MXFP8 along the rows of each matrix of a bf16 [batch, rows, cols] (or
    [rows, cols]) tensor: (codes uint8 [batch, cols, rows], scales uint8
    [batch, cols, rows/32]), written into out=(codes, scales) when given."""
    _cuda(a, "a", torch.bfloat16)
    squeeze = a.dim() == 2
    a3 = a.unsqueeze(0) if squeeze else a
    B, rows, cols = a3.shape
    if out is None:
        q = torch.empty((B, cols, rows), dtype=torch.uint8, device=a.device)
        s = torch.empty((B, cols, rows // 32), dtype=torch.uint8, device=a.device)
    else:
        q, s = out
        _cuda(q, "q", torch.uint8, a.numel())
        _cuda(s, "scales", torch.uint8, a.numel() // 32)
        if squeeze:
            q, s = q.unsqueeze(0), s.unsqueeze(0)
    dev = _device(("a", a), ("q", q), ("scales", s))
    with torch.cuda.device(dev):
        _check(_lib.moe_quantize_mxfp8_t(_p(a3), B, rows, cols, _p(q), _p(s),
                                         _stream(stream, dev)), "moe_quantize_mxfp8_t")
    return (q[0], s[0]) if squeeze else (q, s)


def moe_quantize_mxfp8_dual(a: torch.Tensor, stream=None, out=None):
    """Both orientations of a bf16 [batch, rows, cols] tensor from one read:
    (q [batch, rows, cols], s [batch, rows, cols/32]) as moe_quantize_mxfp8 and
    (qt [batch, cols, rows], st [batch, cols, rows/32]) as moe_quantize_mxfp8_t,
    written into out=(q, s, qt, st) when given."""
    _cuda(a, "a", torch.bfloat16)
    B, rows, cols = a.shape
    if out is None:
        out = (torch.empty((B, rows, cols), dtype=torch.uint8, device=a.device),
               torch.empty((B, rows, cols // 32), dtype=torch.uint8, device=a.device),
               torch.empty((B, cols, rows), dtype=torch.uint8, device=a.device),
               torch.empty((B, cols, rows // 32), dtype=torch.uint8, device=a.device))
    for t, n in zip(out, (a.numel(), a.numel() // 32, a.numel(), a.numel() // 32)):
        _cuda(t, "out", torch.uint8, n)
    dev = _device(("a", a), *(("out", t) for t in out))
    with torch.cuda.device(dev):
        _check(_lib.moe_quantize_mxfp8_dual(_p(a), B, rows, cols, *(_p(t) for t in out),
                                            _stream(stream, dev)), "moe_quantize_mxfp8_dual")
    return out


def moe_workspace_size(T, H, F, E, k, cfg: moe_config | None = None, for_backward=False) -> int:
    c = cfg if cfg is not None else config()
    return _lib.moe_workspace_size(T, H, F, E, k, ctypes.byref(c), int(for_backward))


def moe_expert_forward(x, w_gate, w_up, w_down, expert_ids, probs, y=None, workspace=None,
                       cfg: moe_config | None = None, stream=None):
    """y = the MoE expert block (counts, permute, fc1+SwiGLU, fc2, unpermute).

    Returns (y, workspace); with cfg.save_for_backward the workspace holds
    what moe_expert_backward needs."""
    for t, n in ((x, "x"), (w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down")):
        _cuda(t, n, torch.bfloat16)
    _cuda(expert_ids, "expert_ids", torch.int32)
    _cuda(probs, "probs", torch.float32)
    T, H = x.shape
    E, _, F = w_gate.shape
    k = expert_ids.shape[1]
    _cuda(y, "y", torch.bfloat16, T * H)
    _cuda(workspace, "workspace")
    dev = _device(("x", x), ("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down),
                  ("expert_ids", expert_ids), ("probs", probs), ("y", y),
                  ("workspace", workspace))
    c = cfg if cfg is not None else config()
    need = _lib.moe_workspace_size(T, H, F, E, k, ctypes.byref(c), 0)
    if need == 0 and T > 0:
        raise MoeError(1, "moe_workspace_size")
    with torch.cuda.device(dev):
        ws = _workspace(need, dev) if workspace is None else workspace
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if y is None else y
        _check(_lib.moe_expert_forward(_p(x), _p(w_gate), _p(w_up), _p(w_down), _p(expert_ids),
                                       _p(probs), T, H, F, E, k, _p(y), _p(ws), ws.numel(),
                                       ctypes.byref(c), _stream(stream, dev)),
               "moe_expert_forward")
    return y, ws


def moe_expert_forward_from_logits(x, w_gate, w_up, w_down, router_logits, k, y=None,
                                   expert_ids=None, probs=None, workspace=None,
                                   cfg: moe_config | None = None, stream=None):
    """moe_expert_forward with the fused gate in front: returns
    (y, expert_ids, probs, workspace), the routing as moe_route_topk gives it."""
    for t, n in ((x, "x"), (w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down")):
        _cuda(t, n, torch.bfloat16)
    _cuda(router_logits, "router_logits", torch.float32)
    T, H = x.shape
    E, _, F = w_gate.shape
    _cuda(y, "y", torch.bfloat16, T * H)
    _cuda(expert_ids, "expert_ids", torch.int32, T * k)
    _cuda(probs, "probs", torch.float32, T * k)
    _cuda(workspace, "workspace")
    dev = _device(("x", x), ("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down),
                  ("router_logits", router_logits), ("y", y), ("expert_ids", expert_ids),
                  ("probs", probs), ("workspace", workspace))
    c = cfg if cfg is not None else config()
    need = _lib.moe_workspace_size(T, H, F, E, k, ctypes.byref(c), 0)
    if need == 0 and T > 0:
        raise MoeError(1, "moe_workspace_size")
    with torch.cuda.device(dev):
        ws = _workspace(need, dev) if workspace is None else workspace
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if y is None else y
        expert_ids = (torch.empty((T, k), dtype=torch.int32, device=dev)
                      if expert_ids is None else expert_ids)
        probs = torch.empty((T, k), dtype=torch.float32, device=dev) if probs is None else probs
        _check(_lib.moe_expert_forward_from_logits(_p(x), _p(w_gate), _p(w_up), _p(w_down),
                                                   _p(router_logits), T, H, F, E, k,
                                                   _p(expert_ids), _p(probs), _p(y), _p(ws),
                                                   ws.numel(), ctypes.byref(c),
                                                   _stream(stream, dev)),
               "moe_expert_forward_from_logits")
    return y, expert_ids, probs, ws


_aux_streams = {}


def moe_expert_forward_pipelined(x, w_gate, w_up, w_down, expert_ids, probs, n_chunks, y=None,
                                 workspace=None, cfg: moe_config | None = None, stream=None,
                                 aux_stream=None):
    """moe_expert_forward over n_chunks token chunks, the routing of the next
    chunk and the combine of the last overlapping the GEMMs on a second
    stream (one cached per device unless aux_stream is given). Returns
    (y, workspace)."""
    for t, n in ((x, "x"), (w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down")):
        _cuda(t, n, torch.bfloat16)
    _cuda(expert_ids, "expert_ids", torch.int32)
    _cuda(probs, "probs", torch.float32)
    T, H = x.shape
    E, _, F = w_gate.shape
    k = expert_ids.shape[1]
    _cuda(y, "y", torch.bfloat16, T * H)
    _cuda(workspace, "workspace")
    dev = _device(("x", x), ("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down),
                  ("expert_ids", expert_ids), ("probs", probs), ("y", y),
                  ("workspace", workspace))
    c = cfg if cfg is not None else config()
    need = _lib.moe_workspace_size_pipelined(T, H, F, E, k, n_chunks)
    if need == 0 and T > 0:
        raise MoeError(1, "moe_workspace_size_pipelined")
    with torch.cuda.device(dev):
        ws = _workspace(need, dev) if workspace is None else workspace
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if y is None else y
        if aux_stream is None:
            aux_stream = _aux_streams.get(dev)
            if aux_stream is None:
                aux_stream = _aux_streams[dev] = torch.cuda.Stream(device=dev)
        _check(_lib.moe_expert_forward_pipelined(_p(x), _p(w_gate), _p(w_up), _p(w_down),
                                                 _p(expert_ids), _p(probs), T, H, F, E, k, _p(y),
                                                 n_chunks, _p(ws), ws.numel(), ctypes.byref(c),
                                                 _stream(stream, dev), _stream(aux_stream, dev)),
               "moe_expert_forward_pipelined")
    return y, ws


def moe_expert_backward(dy, x, w_gate, w_up, w_down, expert_ids, probs, fwd_workspace,
                        dx=None, dw_gate=None, dw_up=None, dw_down=None, dprobs=None,
                        accumulate_dw=False, workspace=None, cfg: moe_config | None = None,
                        stream=None):
    """Gradients (dx, dw_gate, dw_up, dw_down, dprobs) of moe_expert_forward."""
    for t, n in ((dy, "dy"), (x, "x"), (w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down")):
        _cuda(t, n, torch.bfloat16)
    _cuda(expert_ids, "expert_ids", torch.int32)
    _cuda(probs, "probs", torch.float32)
    _cuda(fwd_workspace, "fwd_workspace")
    T, H = x.shape
    E, _, F = w_gate.shape
    k = expert_ids.shape[1]
    _cuda(dx, "dx", torch.bfloat16, T * H)
    for t, n in ((dw_gate, "dw_gate"), (dw_up, "dw_up"), (dw_down, "dw_down")):
        _cuda(t, n, torch.float32, E * H * F)
    _cuda(dprobs, "dprobs", torch.float32, T * k)
    _cuda(workspace, "workspace")
    dev = _device(("dy", dy), ("x", x), ("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down),
                  ("expert_ids", expert_ids), ("probs", probs), ("fwd_workspace", fwd_workspace),
                  ("dx", dx), ("dw_gate", dw_gate), ("dw_up", dw_up), ("dw_down", dw_down),
                  ("dprobs", dprobs), ("workspace", workspace))
    c = cfg if cfg is not None else config(save_for_backward=True)
    with torch.cuda.device(dev):
        dx = torch.empty_like(x) if dx is None else dx
        f32 = dict(dtype=torch.float32, device=dev)
        dw_gate = torch.empty((E, H, F), **f32) if dw_gate is None else dw_gate
        dw_up = torch.empty((E, H, F), **f32) if dw_up is None else dw_up
        dw_down = torch.empty((E, F, H), **f32) if dw_down is None else dw_down
        dprobs = torch.empty((T, k), **f32) if dprobs is None else dprobs
        need = _lib.moe_workspace_size(T, H, F, E, k, ctypes.byref(c), 1)
        ws = _workspace(need, dev) if workspace is None else workspace
        _check(_lib.moe_expert_backward(_p(dy), _p(x), _p(w_gate), _p(w_up), _p(w_down),
                                        _p(expert_ids), _p(probs), T, H, F, E, k,
                                        _p(fwd_workspace), fwd_workspace.numel(), _p(dx),
                                        _p(dw_gate), _p(dw_up), _p(dw_down), _p(dprobs),
                                        int(bool(accumulate_dw)), _p(ws), ws.numel(),
                                        ctypes.byref(c), _stream(stream, dev)),
               "moe_expert_backward")
    return dict(dx=dx, dw_gate=dw_gate, dw_up=dw_up, dw_down=dw_down, dprobs=dprobs)


def moe_workspace_size_mxfp8(T, H, F, E, k, cfg: moe_config | None = None) -> int:
    c = cfg if cfg is not None else config()
    return _lib.moe_workspace_size_mxfp8(T, H, F, E, k, ctypes.byref(c))


def moe_workspace_size_mxfp8_backward(T, H, F, E, k) -> int:
    return _lib.moe_workspace_size_mxfp8_backward(T, H, F, E, k)


def moe_tile_weight_scales_mxfp8(wg_s, wu_s, wd_s, cfg: moe_config | None = None, stream=None,
                                 out=None):
    """The weights' scales laid out once for the MXFP8 forward's block-scaled
    MMAs: (wgu_tiled, wd_tiled), to pass as wg_s and wd_s to
    moe_expert_forward_mxfp8 with config(mx_scales_pretiled=True) and the same
    mxfp8_tile_n. wg_s, wu_s [E, F, H/32], wd_s [E, H, F/32] as
    moe_quantize_mxfp8 writes them."""
    for t, n in ((wg_s, "wg_s"), (wu_s, "wu_s"), (wd_s, "wd_s")):
        _cuda(t, n, torch.uint8)
    E, F, H32 = wg_s.shape
    H = 32 * H32
    if tuple(wu_s.shape) != (E, F, H32) or tuple(wd_s.shape) != (E, H, F // 32):
        raise ValueError("wg_s, wu_s [E, F, H/32] and wd_s [E, H, F/32] expected")
    if out is None:
        wgu = torch.empty(E * 2 * F * H32, dtype=torch.uint8, device=wg_s.device)
        wdt = torch.empty(E * H * (F // 32), dtype=torch.uint8, device=wg_s.device)
    else:
        wgu, wdt = out
        _cuda(wgu, "wgu_tiled", torch.uint8, E * 2 * F * H32)
        _cuda(wdt, "wd_tiled", torch.uint8, E * H * (F // 32))
    dev = _device(("wg_s", wg_s), ("wu_s", wu_s), ("wd_s", wd_s), ("wgu_tiled", wgu),
                  ("wd_tiled", wdt))
    c = cfg if cfg is not None else config()
    with torch.cuda.device(dev):
        _check(_lib.moe_tile_weight_scales_mxfp8(_p(wg_s), _p(wu_s), _p(wd_s), H, F, E,
                                                 ctypes.byref(c), _p(wgu), _p(wdt),
                                                 _stream(stream, dev)),
               "moe_tile_weight_scales_mxfp8")
    return wgu, wdt


def moe_expert_forward_mxfp8(x, wg_q, wg_s, wu_q, wu_s, wd_q, wd_s, expert_ids, probs, y=None,
                             workspace=None, cfg: moe_config | None = None, stream=None):
    """The block with MXFP8 operands (x quantised on the fly; weights pre-quantised,
    K-contiguous: wg/wu [E, F, H], wd [E, H, F], scales [..., K/32]). With
    cfg.mx_scales_pretiled, wg_s and wd_s are moe_tile_weight_scales_mxfp8's
    outputs and wu_s may be None."""
    _cuda(x, "x", torch.bfloat16)
    for t, n in ((wg_q, "wg_q"), (wg_s, "wg_s"), (wu_q, "wu_q"), (wu_s, "wu_s"), (wd_q, "wd_q"),
                 (wd_s, "wd_s")):
        _cuda(t, n, torch.uint8)
    _cuda(expert_ids, "expert_ids", torch.int32)
    _cuda(probs, "probs", torch.float32)
    T, H = x.shape
    E, F, _ = wg_q.shape
    k = expert_ids.shape[1]
    _cuda(y, "y", torch.bfloat16, T * H)
    _cuda(workspace, "workspace")
    dev = _device(("x", x), ("wg_q", wg_q), ("wg_s", wg_s), ("wu_q", wu_q), ("wu_s", wu_s),
                  ("wd_q", wd_q), ("wd_s", wd_s), ("expert_ids", expert_ids), ("probs", probs),
                  ("y", y), ("workspace", workspace))
    c = cfg if cfg is not None else config()
    need = _lib.moe_workspace_size_mxfp8(T, H, F, E, k, ctypes.byref(c))
    with torch.cuda.device(dev):
        ws = _workspace(need, dev) if workspace is None else workspace
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if y is None else y
        _check(_lib.moe_expert_forward_mxfp8(_p(x), _p(wg_q), _p(wg_s), _p(wu_q), _p(wu_s),
                                             _p(wd_q), _p(wd_s), _p(expert_ids), _p(probs), T, H,
                                             F, E, k, _p(y), _p(ws), ws.numel(), ctypes.byref(c),
                                             _stream(stream, dev)), "moe_expert_forward_mxfp8")
    return y, ws


def moe_expert_backward_mxfp8(dy, x, w1g_q, w1g_s, w1u_q, w1u_s, w2_q, w2_s, expert_ids, probs,
                              fwd_workspace, dx=None, dw_gate_t=None, dw_up_t=None,
                              dw_down_t=None, dprobs=None, accumulate_dw=False, workspace=None,
                              cfg: moe_config | None = None, stream=None):
    """Gradients of moe_expert_forward_mxfp8 (run with save_for_backward):
    dict(dx, dw_gate_t [E, F, H], dw_up_t [E, F, H], dw_down_t [E, H, F],
    dprobs). The weights come in the backward orientation of
    moe_quantize_mxfp8_t: w1g/w1u [E, H, F], w2 [E, F, H]."""
    for t, n in ((dy, "dy"), (x, "x")):
        _cuda(t, n, torch.bfloat16)
    for t, n in ((w1g_q, "w1g_q"), (w1g_s, "w1g_s"), (w1u_q, "w1u_q"), (w1u_s, "w1u_s"),
                 (w2_q, "w2_q"), (w2_s, "w2_s")):
        _cuda(t, n, torch.uint8)
    _cuda(expert_ids, "expert_ids", torch.int32)
    _cuda(probs, "probs", torch.float32)
    _cuda(fwd_workspace, "fwd_workspace")
    T, H = x.shape
    E, _, F = w1g_q.shape
    k = expert_ids.shape[1]
    _cuda(dx, "dx", torch.bfloat16, T * H)
    for t, n in ((dw_gate_t, "dw_gate_t"), (dw_up_t, "dw_up_t"), (dw_down_t, "dw_down_t")):
        _cuda(t, n, torch.float32, E * H * F)
    _cuda(dprobs, "dprobs", torch.float32, T * k)
    _cuda(workspace, "workspace")
    dev = _device(("dy", dy), ("x", x), ("w1g_q", w1g_q), ("w1g_s", w1g_s), ("w1u_q", w1u_q),
                  ("w1u_s", w1u_s), ("w2_q", w2_q), ("w2_s", w2_s), ("expert_ids", expert_ids),
                  ("probs", probs), ("fwd_workspace", fwd_workspace), ("dx", dx),
                  ("dw_gate_t", dw_gate_t), ("dw_up_t", dw_up_t), ("dw_down_t", dw_down_t),
                  ("dprobs", dprobs), ("workspace", workspace))
    c = cfg if cfg is not None else config(save_for_backward=True)
    with torch.cuda.device(dev):
        dx = torch.empty_like(x) if dx is None else dx
        f32 = dict(dtype=torch.float32, device=dev)
        dw_gate_t = torch.empty((E, F, H), **f32) if dw_gate_t is None else dw_gate_t
        dw_up_t = torch.empty((E, F, H), **f32) if dw_up_t is None else dw_up_t
        dw_down_t = torch.empty((E, H, F), **f32) if dw_down_t is None else dw_down_t
        dprobs = torch.empty((T, k), **f32) if dprobs is None else dprobs
        need = _lib.moe_workspace_size_mxfp8_backward(T, H, F, E, k)
        ws = _workspace(need, dev) if workspace is None else workspace
        _check(_lib.moe_expert_backward_mxfp8(_p(dy), _p(x), _p(w1g_q), _p(w1g_s), _p(w1u_q),
                                              _p(w1u_s), _p(w2_q), _p(w2_s), _p(expert_ids),
                                              _p(probs), T, H, F, E, k, _p(fwd_workspace),
                                              fwd_workspace.numel(), _p(dx), _p(dw_gate_t),
                                              _p(dw_up_t), _p(dw_down_t), _p(dprobs),
                                              int(bool(accumulate_dw)), _p(ws), ws.numel(),
                                              ctypes.byref(c), _stream(stream, dev)),
               "moe_expert_backward_mxfp8")
    return dict(dx=dx, dw_gate_t=dw_gate_t, dw_up_t=dw_up_t, dw_down_t=dw_down_t, dprobs=dprobs)


# ------------------------------------------------------------------ the layer around the block

_TYPES = {torch.float32: 0, torch.bfloat16: 1}
_CLIP_WORKSPACE = _lib.moe_clip_grad_norm_workspace_size()
_SCORES = {"softmax": 0, "sigmoid": 1}
# the current stream of a device as an integer, without a Stream object
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


# the current device: what has a CUDA tensor in hand needs no look at the initialisation
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _fit(dev, *named):
    """Checks (tensor or None, name, dtype, least number of elements) on dev:
    these calls are short, so one pass looks at everything and the messages
    are made only where something is wrong."""
    index = dev.index
    for t, name, dtype, least in named:
        if t is not None and (t.get_device() != index or t.dtype != dtype
                              or not t.is_contiguous() or t.numel() < least):
            _cuda(t, name, dtype, least)
            raise ValueError(f"{name} is on {t.device} but the call's first tensor on {dev}: "
                             "all tensors of a call must share one device")


def _on(dev, fn, *args):
    """fn(*args) with dev current."""
    if dev.index == _current_device():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, dev):
    """_stream as a plain integer."""
    if stream is None:
        return _current_raw_stream(dev.index)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return stream.cuda_stream


def _elsewhere(stream):
    """Whether the call is for another stream than its device's current one."""
    return stream is not None and stream != torch.cuda.current_stream(stream.device)


def _within(stream, fn, args):
    """fn(**args) with stream current, so that what it allocates is stream's: memory
    of another one's pool may still be in use there, and would go back to it
    while the kernels run."""
    with torch.cuda.stream(stream):
        return fn(**args)


def _scratch(workspace, need, dev):
    """(the given workspace or a new one, its bytes); None where none is needed."""
    if workspace is not None:
        _fit(dev, (workspace, "workspace", workspace.dtype, 0))
        return workspace, workspace.nbytes
    if not need:
        return None, 0
    return torch.empty(need, dtype=torch.uint8, device=dev), need


def _typed(t, name):
    """The moe_type of a tensor that may be float32 or bfloat16."""
    code = _TYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    return code


def _shaped(t, name, *shape):
    if t is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _gate_config(score, n_group, topk_group, group_topk, renormalise, scale):
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return moe_gate_config(_SCORES[score], n_group, topk_group, group_topk, bool(renormalise),
                           scale)


def moe_route_gate(logits: torch.Tensor, k: int, bias=None, score="softmax", n_group=1,
                   topk_group=1, group_topk=1, renormalise=True, scale=1.0, expert_ids=None,
                   probs=None, counts=None, offsets=None, workspace=None, stream=None):
    """The top-k gate with softmax or sigmoid scores, a balance bias float32 [E]
    that enters the choice only, groups (the topk_group of n_group groups with
    the largest sum of their group_topk best experts) and weights that are
    renormalised over the chosen and scaled: (expert_ids int32 [T, k], probs
    float32 [T, k], counts int32 [E], offsets int32 [E+1]) of float32 or
    bfloat16 logits [T, E]."""
    if _elsewhere(stream):
        return _within(stream, moe_route_gate, locals())
    lt = _typed(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    _fit(dev, (logits, "logits", logits.dtype, 0), (bias, "bias", torch.float32, 0),
         (expert_ids, "expert_ids", torch.int32, T * k), (probs, "probs", torch.float32, T * k),
         (counts, "counts", torch.int32, E), (offsets, "offsets", torch.int32, E + 1))
    _shaped(bias, "bias", E)
    cfg = _gate_config(score, n_group, topk_group, group_topk, renormalise, scale)
    if expert_ids is None:
        expert_ids = torch.empty((T, max(k, 0)), dtype=torch.int32, device=dev)
    if probs is None:
        probs = torch.empty((T, max(k, 0)), dtype=torch.float32, device=dev)
    if counts is None:
        counts = torch.empty(E, dtype=torch.int32, device=dev)
    if offsets is None:
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    ws, ws_bytes = _scratch(workspace, _lib.moe_route_gate_workspace_size(T, k, E), dev)
    _check(_on(dev, _lib.moe_route_gate, logits.data_ptr(), lt, _ptr(bias), T, E, k, cfg,
               expert_ids.data_ptr(), probs.data_ptr(), counts.data_ptr(), offsets.data_ptr(),
               _ptr(ws), ws_bytes, _raw_stream(stream, dev)), "moe_route_gate")
    return expert_ids, probs, counts, offsets


def moe_route_gate_backward(dprobs, logits, expert_ids, bias=None, score="softmax",
                            renormalise=True, scale=1.0, dlogits=None, stream=None):
    """dlogits [T, E], of the logits' type, of moe_route_gate's weights for the
    choice expert_ids that it made; bias, score, renormalise and scale as there."""
    if _elsewhere(stream):
        return _within(stream, moe_route_gate_backward, locals())
    lt = _typed(logits, "logits")
    T, E = logits.shape
    k = expert_ids.shape[1]
    dev = logits.device
    _fit(dev, (logits, "logits", logits.dtype, 0), (dprobs, "dprobs", torch.float32, 0),
         (expert_ids, "expert_ids", torch.int32, 0), (bias, "bias", torch.float32, 0),
         (dlogits, "dlogits", logits.dtype, T * E))
    _shaped(expert_ids, "expert_ids", T, k)
    _shaped(dprobs, "dprobs", T, k)
    _shaped(bias, "bias", E)
    cfg = _gate_config(score, 1, 1, 1, renormalise, scale)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    _check(_on(dev, _lib.moe_route_gate_backward, dprobs.data_ptr(), logits.data_ptr(), lt,
               _ptr(bias), expert_ids.data_ptr(), T, E, k, cfg, dlogits.data_ptr(),
               _raw_stream(stream, dev)), "moe_route_gate_backward")
    return dlogits


def _norm_weights(dev, H, w_post, gate, w_next):
    """(moe_type of the weights, rows of the gate)."""
    first = w_post if w_post is not None else gate if gate is not None else w_next
    if first is None:
        return 1, 0
    wt = _typed(first, "weights")
    if any(t is not None and t.dtype != first.dtype for t in (gate, w_next)):
        raise ValueError("w_post, gate and w_next share one type: got "
                         f"{[t.dtype for t in (w_post, gate, w_next) if t is not None]}")
    _fit(dev, (w_post, "w_post", first.dtype, 0), (gate, "gate", first.dtype, 0),
         (w_next, "w_next", first.dtype, 0))
    _shaped(w_post, "w_post", H)
    _shaped(w_next, "w_next", H)
    if gate is None:
        return wt, 0
    if gate.dim() not in (1, 2) or gate.shape[-1] != H:
        raise ValueError(f"gate must have shape [{H}] or [rows, {H}], got {list(gate.shape)}")
    return wt, 1 if gate.dim() == 1 else gate.shape[0]


def moe_norm_residual(x, y=None, w_post=None, gate=None, w_next=None, eps=1e-6,
                      residual_scale=1.0, branch_scale=1.0, out=None, n=None, rstd_y=None,
                      rstd_out=None, stream=None):
    """The norm after the block, its gate, the scaled residual and the norm
    before the next block in one pass over x [T, H] (float32 or bfloat16) and
    the block's output y (bfloat16 [T, H]):
      out = residual_scale * x + branch_scale * gate * (w_post * rmsnorm(y))
      n = w_next * rmsnorm(out)
    Without w_post y enters as it is, without gate (of [H], or [rows, H] with T
    / rows consecutive tokens to a row) it is 1, without w_next n is left out.
    Without y it is the norm alone, of x. Returns dict(out, n, rstd_y,
    rstd_out), None where nothing was computed; out may be x itself. All
    tensors of [T, H], [rows, H] and [H] start on 16 bytes."""
    if _elsewhere(stream):
        return _within(stream, moe_norm_residual, locals())
    st = _typed(x, "x")
    T, H = x.shape
    dev = x.device
    _fit(dev, (x, "x", x.dtype, 0), (y, "y", torch.bfloat16, 0), (out, "out", x.dtype, T * H),
         (n, "n", torch.bfloat16, T * H), (rstd_y, "rstd_y", torch.float32, T),
         (rstd_out, "rstd_out", torch.float32, T))
    _shaped(y, "y", T, H)
    wt, rows = _norm_weights(dev, H, w_post, gate, w_next)
    if y is None:
        out = None
    elif out is None:
        out = torch.empty_like(x)
    if w_post is None:
        rstd_y = None
    elif rstd_y is None:
        rstd_y = torch.empty(T, dtype=torch.float32, device=dev)
    if w_next is None:
        n = rstd_out = None
    else:
        if n is None:
            n = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        if rstd_out is None:
            rstd_out = torch.empty(T, dtype=torch.float32, device=dev)
    _check(_on(dev, _lib.moe_norm_residual, x.data_ptr(), _ptr(y), _ptr(w_post), _ptr(gate), rows,
               _ptr(w_next), T, H, moe_norm_config(eps, residual_scale, branch_scale, st, wt),
               _ptr(out), _ptr(n), _ptr(rstd_y), _ptr(rstd_out), _raw_stream(stream, dev)),
           "moe_norm_residual")
    return dict(out=out, n=n, rstd_y=rstd_y, rstd_out=rstd_out)


def moe_norm_residual_backward(d_out, d_n, out, y=None, w_post=None, gate=None, w_next=None,
                               rstd_y=None, rstd_out=None, eps=1e-6, residual_scale=1.0,
                               branch_scale=1.0, dx=None, dy=None, dw_post=None, dgate=None,
                               dw_next=None, accumulate_dw=False, workspace=None, stream=None):
    """Gradients of moe_norm_residual from d_out (of x's type) and d_n
    (bfloat16), either of them None for no gradient. out is the forward's (its
    x where y is None); y, the weights, rstd_y, rstd_out and the scalars are the
    forward's. Returns dict(dx, dy, dw_post, dgate, dw_next), the last three in
    float32 and, with accumulate_dw, added to what the given tensors hold; None
    where there is no such input. dx may be d_out itself. All tensors of [T, H],
    [rows, H] and [H] start on 16 bytes."""
    if _elsewhere(stream):
        return _within(stream, moe_norm_residual_backward, locals())
    st = _typed(out, "out")
    T, H = out.shape
    dev = out.device
    bf16, f32 = torch.bfloat16, torch.float32
    _fit(dev, (out, "out", out.dtype, 0), (d_out, "d_out", out.dtype, 0), (d_n, "d_n", bf16, 0),
         (y, "y", bf16, 0), (rstd_y, "rstd_y", f32, T), (rstd_out, "rstd_out", f32, T),
         (dx, "dx", out.dtype, T * H), (dy, "dy", bf16, T * H))
    _shaped(d_out, "d_out", T, H)
    _shaped(d_n, "d_n", T, H)
    _shaped(y, "y", T, H)
    wt, rows = _norm_weights(dev, H, w_post, gate, w_next)
    _fit(dev, (dw_post, "dw_post", f32, H), (dgate, "dgate", f32, rows * H),
         (dw_next, "dw_next", f32, H))
    if accumulate_dw and any(w is not None and g is None for w, g in (
            (w_post, dw_post), (gate, dgate), (w_next if d_n is not None else None, dw_next))):
        raise ValueError("accumulate_dw adds to dw_post, dgate and dw_next: pass them")
    if dx is None:
        dx = torch.empty_like(out)
    if y is None:
        dy = None
    elif dy is None:
        dy = torch.empty_like(y)
    if w_post is None:
        dw_post = None
    elif dw_post is None:
        dw_post = torch.empty(H, dtype=f32, device=dev)
    if gate is None:
        dgate = None
    elif dgate is None:
        dgate = torch.empty(gate.shape, dtype=f32, device=dev)
    if w_next is None or d_n is None:
        dw_next = None
    elif dw_next is None:
        dw_next = torch.empty(H, dtype=f32, device=dev)
    ws, ws_bytes = _scratch(workspace, _on(
        dev, _lib.moe_norm_residual_backward_workspace_size, T, H, rows), dev)
    _check(_on(dev, _lib.moe_norm_residual_backward, _ptr(d_out), _ptr(d_n), out.data_ptr(),
               _ptr(y), _ptr(w_post), _ptr(gate), rows, _ptr(w_next), _ptr(rstd_y),
               _ptr(rstd_out), T, H, moe_norm_config(eps, residual_scale, branch_scale, st, wt),
               dx.data_ptr(), _ptr(dy), _ptr(dw_post), _ptr(dgate), _ptr(dw_next),
               bool(accumulate_dw), _ptr(ws), ws_bytes, _raw_stream(stream, dev)),
           "moe_norm_residual_backward")
    return dict(dx=dx, dy=dy, dw_post=dw_post, dgate=dgate, dw_next=dw_next)


def moe_clip_grad_norm(grads, max_norm, out=None, norm_type=2.0, eps=1e-6, norm_coef=None,
                       workspace=None, stream=None):
    """One norm over a list of gradients (float32 or bfloat16, contiguous), and
    every one of them scaled by coef = min(1, max_norm / (norm + eps)): in place,
    or into the tensors of the list out (same types and sizes). norm_type is 2.0
    or math.inf; max_norm None computes the norm alone. Returns (norm, coef), two
    float32 tensors of one element; nothing is read back to the host."""
    if _elsewhere(stream):
        return _within(stream, moe_clip_grad_norm, locals())
    grads = list(grads)
    if norm_type not in (2.0, math.inf):
        raise ValueError(f"norm_type must be 2.0 or inf, got {norm_type}")
    if max_norm is not None and not max_norm >= 0:
        raise ValueError(f"max_norm must be None or >= 0, got {max_norm}")
    if max_norm is None and out is not None:
        raise ValueError("out is written when gradients are clipped: max_norm is None")
    if not grads and norm_coef is None:
        raise ValueError("no gradients: pass norm_coef to say where the norm goes")
    dev = grads[0].device if grads else norm_coef.device
    index, n = grads[0].get_device() if grads else dev.index, len(grads)
    # a call may have hundreds of tensors: whole lists at a time, and a loop
    # only to name the one that is wrong
    Tensor = torch.Tensor
    dtypes = [g.dtype for g in grads]
    kinds = set(dtypes)
    sizes = list(map(Tensor.numel, grads))
    if not kinds <= _TYPES.keys() or not all(map(Tensor.is_contiguous, grads)) or \
            set(map(Tensor.get_device, grads)) - {index}:
        for i, g in enumerate(grads):
            if g.dtype not in _TYPES or g.get_device() != index or not g.is_contiguous():
                raise ValueError(f"grads[{i}] must be a contiguous float32 or bfloat16 tensor "
                                 f"on {dev}")
    if dev.type != "cuda":
        raise ValueError("grads must be CUDA tensors")
    outs = None
    if out is not None:
        out = list(out)
        if len(out) != n:
            raise ValueError(f"out holds {len(out)} tensors, grads {n}")
        if [o.dtype for o in out] != dtypes or list(map(Tensor.numel, out)) != sizes or \
                not all(map(Tensor.is_contiguous, out)) or \
                set(map(Tensor.get_device, out)) - {index}:
            for i, o in enumerate(out):
                if o.dtype != dtypes[i] or o.numel() != sizes[i] or not o.is_contiguous() or \
                        o.get_device() != index:
                    raise ValueError(f"out[{i}] must be as grads[{i}]: same type, device and size")
        outs = array.array("Q", list(map(Tensor.data_ptr, out)))
    _fit(dev, (norm_coef, "norm_coef", torch.float32, 2))
    if norm_coef is None and workspace is None:
        # one allocation: the two results, then the workspace
        norm_coef = torch.empty(4 + _CLIP_WORKSPACE // 4, dtype=torch.float32, device=dev)
        result, ws_bytes = norm_coef.data_ptr(), _CLIP_WORKSPACE
        ws_at = result + 16
    else:
        if norm_coef is None:
            norm_coef = torch.empty(2, dtype=torch.float32, device=dev)
        ws, ws_bytes = _scratch(workspace, _CLIP_WORKSPACE, dev)
        result, ws_at = norm_coef.data_ptr(), _ptr(ws)
    ptrs = array.array("Q", list(map(Tensor.data_ptr, grads)))
    numels = array.array("q", sizes)
    codes = array.array("i", [_TYPES[d] for d in (kinds if len(kinds) == 1 else dtypes)])
    if len(kinds) == 1:
        codes *= n
    at = array.array.buffer_info
    _check(_on(dev, _lib.moe_clip_grad_norm, at(ptrs)[0], None if outs is None else at(outs)[0],
               at(numels)[0], at(codes)[0], n, -1.0 if max_norm is None else max_norm,
               norm_type == math.inf, eps, result, ws_at, ws_bytes, _raw_stream(stream, dev)),
           "moe_clip_grad_norm")
    flat = norm_coef.reshape(-1) if norm_coef.dim() != 1 else norm_coef
    return flat[:1], flat[1:2]


def moe_grad_norm(grads, norm_type=2.0, norm_coef=None, workspace=None, stream=None):
    """The norm alone of a list of gradients: a float32 tensor of one element."""
    return moe_clip_grad_norm(grads, None, norm_type=norm_type, norm_coef=norm_coef,
                              workspace=workspace, stream=stream)[0]


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}


def _act(act):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return code


def _all_fit(dev, *named):
    """Checks (tensor or None, name, shape, dtype) on dev; the messages are made
    only where something is wrong."""
    index = dev.index
    for t, name, shape, dtype in named:
        if t is None or (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                         and t.get_device() == index):
            continue
        _cuda(t, name, dtype)
        _shaped(t, name, *shape)
        raise ValueError(f"{name} is on {t.device} but the call's first tensor on {dev}: "
                         "all tensors of a call must share one device")


def _made(t, shape, dtype, dev):
    """The given output, or a new one."""
    return torch.empty(shape, dtype=dtype, device=dev) if t is None else t


def _space(workspace, query, dev, *sizes):
    """(the given workspace or a new one, its bytes); the size may go by the device."""
    if workspace is not None:
        return _scratch(workspace, 0, dev)
    return _scratch(None, _on(dev, query, *sizes), dev)


def _matrix(t, name):
    """The shape of a tensor that has to have two dimensions."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {list(t.shape)}")
    return t.shape


def moe_gated_ffn(x, w_gate, w_up, w_down, act="silu", add=None, save_for_backward=False, y=None,
                  a_gate=None, a_up=None, workspace=None, stream=None):
    """The gated feed-forward block of a dense layer or a shared expert over
    x bf16 [T, H]: y = add + (act(x w_gate) * (x w_up)) w_down, with w_gate and
    w_up bf16 [H, F], w_down bf16 [F, H], act "silu", "gelu", "gelu_tanh" or
    "relu", and add bf16 [T, H] (the routed experts' result) or None. Returns
    dict(y, a_gate, a_up); a_gate = x w_gate and a_up = x w_up (bf16 [T, F]) are
    kept with save_for_backward, else None. y may be add itself. H and F are
    multiples of 8, tensors start on 16 bytes."""
    if stream is not None and _elsewhere(stream):
        return _within(stream, moe_gated_ffn, locals())
    bf16, dev = _BF16, x.device
    T, H = rows = _matrix(x, "x")
    F = _matrix(w_gate, "w_gate")[1]
    if y is None:
        y = torch.empty(rows, dtype=bf16, device=dev)
    if save_for_backward:
        a_gate, a_up = _made(a_gate, (T, F), bf16, dev), _made(a_up, (T, F), bf16, dev)
        _all_fit(dev, (a_gate, "a_gate", (T, F), bf16), (a_up, "a_up", (T, F), bf16))
    else:
        a_gate = a_up = None
    _all_fit(dev, (x, "x", rows, bf16), (w_gate, "w_gate", (H, F), bf16),
             (w_up, "w_up", (H, F), bf16), (w_down, "w_down", (F, H), bf16), (y, "y", rows, bf16))
    if add is not None:
        _all_fit(dev, (add, "add", rows, bf16))
    code = _act(act)
    if workspace is None:
        ws_bytes = _on(dev, _lib.moe_gated_ffn_workspace_size, T, H, F)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    else:
        _, ws_bytes = _scratch(workspace, 0, dev)
    _check(_on(dev, _lib.moe_gated_ffn, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
               w_down.data_ptr(), _ptr(add), T, H, F, code, y.data_ptr(), _ptr(a_gate),
               _ptr(a_up), workspace.data_ptr(), ws_bytes, _raw_stream(stream, dev)),
           "moe_gated_ffn")
    return {"y": y, "a_gate": a_gate, "a_up": a_up}


def moe_gated_ffn_backward(dy, x, w_gate, w_up, w_down, a_gate, a_up, act="silu", add=None,
                           weight_grads=True, dw_dtype=torch.bfloat16, dx=None, dw_gate=None,
                           dw_up=None, dw_down=None, accumulate_dw=False, workspace=None,
                           stream=None):
    """Gradients of moe_gated_ffn from dy bf16 [T, H]; x, the weights, act, a_gate
    and a_up are the forward's, add (bf16 [T, H] or None) what reaches x by other
    ways and joins dx. Returns dict(dx, dw_gate, dw_up, dw_down): the weight
    gradients in the type of those given, else in dw_dtype (torch.bfloat16 or
    torch.float32); in float32 they are added to what is there with accumulate_dw;
    None without weight_grads (frozen weights). dx may be add itself."""
    if stream is not None and _elsewhere(stream):
        return _within(stream, moe_gated_ffn_backward, locals())
    bf16, dev = torch.bfloat16, x.device
    T, H = rows = _matrix(x, "x")
    F = _matrix(w_gate, "w_gate")[1]
    if dx is None:
        dx = torch.empty(rows, dtype=bf16, device=dev)
    dt, wt = bf16, 0
    if weight_grads:
        given = [t for t in (dw_gate, dw_up, dw_down) if t is not None]
        if accumulate_dw and len(given) != 3:
            raise ValueError("accumulate_dw adds to dw_gate, dw_up and dw_down: pass them")
        dt = given[0].dtype if given else dw_dtype
        if dt not in _TYPES:
            raise ValueError(f"weight gradients must be torch.float32 or torch.bfloat16, got {dt}")
        wt = _TYPES[dt]
        dw_gate, dw_up = _made(dw_gate, (H, F), dt, dev), _made(dw_up, (H, F), dt, dev)
        dw_down = _made(dw_down, (F, H), dt, dev)
    else:
        dw_gate = dw_up = dw_down = None
    _all_fit(dev, (x, "x", rows, bf16), (dy, "dy", rows, bf16), (w_gate, "w_gate", (H, F), bf16),
             (w_up, "w_up", (H, F), bf16), (w_down, "w_down", (F, H), bf16),
             (a_gate, "a_gate", (T, F), bf16), (a_up, "a_up", (T, F), bf16),
             (add, "add", rows, bf16), (dx, "dx", rows, bf16), (dw_gate, "dw_gate", (H, F), dt),
             (dw_up, "dw_up", (H, F), dt), (dw_down, "dw_down", (F, H), dt))
    ws, ws_bytes = _space(workspace, _lib.moe_gated_ffn_backward_workspace_size, dev, T, H, F)
    _check(_on(dev, _lib.moe_gated_ffn_backward, dy.data_ptr(), x.data_ptr(), w_gate.data_ptr(),
               w_up.data_ptr(), w_down.data_ptr(), a_gate.data_ptr(), a_up.data_ptr(), _ptr(add),
               T, H, F, _act(act), dx.data_ptr(), _ptr(dw_gate), _ptr(dw_up), _ptr(dw_down), wt,
               bool(accumulate_dw), _ptr(ws), ws_bytes, _raw_stream(stream, dev)),
           "moe_gated_ffn_backward")
    return dict(dx=dx, dw_gate=dw_gate, dw_up=dw_up, dw_down=dw_down)


def moe_lora_plan(adapter_ids, n, order=None, offsets=None, stream=None):
    """The rows of a batch by adapter: (order int32 [T], offsets int32 [n + 1]) of
    adapter_ids int32 [T], -1 for a row without one. Adapter a has the rows
    order[offsets[a]:offsets[a + 1]] in their own order; those without one come
    last. One plan serves every projection and layer of the batch."""
    if stream is not None and _elsewhere(stream):
        return _within(stream, moe_lora_plan, locals())
    dev = adapter_ids.device
    if adapter_ids.dim() != 1:
        raise ValueError(f"adapter_ids must have shape [T], got {list(adapter_ids.shape)}")
    T, i32 = adapter_ids.shape[0], torch.int32
    order = _made(order, (T,), i32, dev)
    offsets = _made(offsets, (max(n, 0) + 1,), i32, dev)
    _all_fit(dev, (adapter_ids, "adapter_ids", (T,), i32), (order, "order", (T,), i32),
             (offsets, "offsets", (max(n, 0) + 1,), i32))
    _check(_on(dev, _lib.moe_lora_plan, adapter_ids.data_ptr(), T, n, order.data_ptr(),
               offsets.data_ptr(), _raw_stream(stream, dev)), "moe_lora_plan")
    return order, offsets


def _lora_shapes(x, a, b):
    """(T, H, N, n, r) of x [T, H], a [n, r, H] and b [n, r, N]."""
    T, H = _matrix(x, "x")
    if a.dim() == 3 and b.dim() == 3:
        n, r, N = b.shape
        if a.shape == (n, r, H):
            return T, H, N, n, r
    raise ValueError(f"a and b must have shapes [n, r, {H}] and [n, r, N], got "
                     f"{list(a.shape)} and {list(b.shape)}")


def moe_lora(x, a, b, adapter_ids, plan=None, scales=None, base=None, out=None, v=None,
             workspace=None, stream=None):
    """Low-rank adapters beside a shared projection: for row t with adapter i =
    adapter_ids[t], v_t = a[i] x_t and out_t = base_t + scales[i] * b[i]^T v_t. x
    bf16 [T, H], a bf16 [n, r, H], b bf16 [n, r, N] (rank first in both),
    adapter_ids int32 [T] with -1 for a row without one, plan what moe_lora_plan
    gives for them (made here when None), scales float32 [n] or None (1), base
    bf16 [T, N] (the projection's result) or None (0). Returns dict(out bf16 [T,
    N], v float32 [T, r]), v for the backward. out may be base itself. r is 1 to
    128, H and N are multiples of 8, tensors start on 16 bytes."""
    if stream is not None and _elsewhere(stream):
        return _within(stream, moe_lora, locals())
    bf16, f32, i32, dev = _BF16, _F32, _I32, x.device
    T, H, N, n, r = _lora_shapes(x, a, b)
    if out is None:
        out = torch.empty((T, N), dtype=bf16, device=dev)
    if v is None:
        v = torch.empty((T, r), dtype=f32, device=dev)
    _all_fit(dev, (x, "x", (T, H), bf16), (a, "a", (n, r, H), bf16), (b, "b", (n, r, N), bf16),
             (adapter_ids, "adapter_ids", (T,), i32), (scales, "scales", (n,), f32),
             (base, "base", (T, N), bf16), (out, "out", (T, N), bf16), (v, "v", (T, r), f32))
    order, offsets = moe_lora_plan(adapter_ids, n) if plan is None else plan
    _all_fit(dev, (order, "order", (T,), i32), (offsets, "offsets", (n + 1,), i32))
    ws, ws_bytes = _scratch(workspace, _lib.moe_lora_workspace_size(T, n, r), dev)
    _check(_on(dev, _lib.moe_lora, x.data_ptr(), a.data_ptr(), b.data_ptr(),
               adapter_ids.data_ptr(), order.data_ptr(), offsets.data_ptr(), _ptr(scales),
               _ptr(base), T, H, N, n, r, out.data_ptr(), v.data_ptr(), _ptr(ws), ws_bytes,
               _raw_stream(stream, dev)), "moe_lora")
    return {"out": out, "v": v}


def moe_lora_backward(dy, x, v, a, b, adapter_ids, plan=None, scales=None, base=None, dx=None,
                      da=None, db=None, accumulate=False, workspace=None, stream=None):
    """Gradients of moe_lora from dy bf16 [T, N]: dict(dx bf16 [T, H], da float32
    [n, r, H], db float32 [n, r, N]). x, v, a, b, adapter_ids, plan and scales are
    the forward's; base (bf16 [T, H] or None) is what reaches x by the projection
    and joins dx. With accumulate da and db are added to what the given tensors
    hold. dx may be base itself. base's own gradient in the forward is dy."""
    if stream is not None and _elsewhere(stream):
        return _within(stream, moe_lora_backward, locals())
    bf16, f32, dev = torch.bfloat16, torch.float32, x.device
    T, H, N, n, r = _lora_shapes(x, a, b)
    if accumulate and (da is None or db is None):
        raise ValueError("accumulate adds to da and db: pass them")
    dx = _made(dx, (T, H), bf16, dev)
    da, db = _made(da, (n, r, H), f32, dev), _made(db, (n, r, N), f32, dev)
    _all_fit(dev, (x, "x", (T, H), bf16), (a, "a", (n, r, H), bf16), (b, "b", (n, r, N), bf16),
             (adapter_ids, "adapter_ids", (T,), _I32), (scales, "scales", (n,), f32),
             (dy, "dy", (T, N), bf16), (v, "v", (T, r), f32), (base, "base", (T, H), bf16),
             (dx, "dx", (T, H), bf16), (da, "da", (n, r, H), f32), (db, "db", (n, r, N), f32))
    order, offsets = moe_lora_plan(adapter_ids, n) if plan is None else plan
    _all_fit(dev, (order, "order", (T,), _I32), (offsets, "offsets", (n + 1,), _I32))
    ws, ws_bytes = _space(workspace, _lib.moe_lora_backward_workspace_size, dev, T, n, r)
    _check(_on(dev, _lib.moe_lora_backward, dy.data_ptr(), x.data_ptr(), v.data_ptr(),
               a.data_ptr(), b.data_ptr(), order.data_ptr(), offsets.data_ptr(), _ptr(scales),
               _ptr(base), T, H, N, n, r, dx.data_ptr(), da.data_ptr(), db.data_ptr(),
               bool(accumulate), _ptr(ws), ws_bytes, _raw_stream(stream, dev)),
           "moe_lora_backward")
    return dict(dx=dx, da=da, db=db)


def moe_dropout_residual(y, rng, p, x=None, residual_scale=1.0, branch_scale=1.0, out=None,
                         stream=None):
    """Dropout of a branch and the scaled residual it joins: out = residual_scale
    * x + branch_scale / (1 - p) * mask * y, the mask made anew wherever it is
    needed from rng, an int64 [2] CUDA tensor of seed and draw that the kernel
    reads (add to rng[1] between steps: a captured graph then drops others at
    every replay). y is float32 or bfloat16 of any shape; x has that shape and
    the result's type, without x there is no residual and the result has y's
    type (or out's). p, in [0, 1), is taken to the nearest 1/65536 and the factor
    is that one's. out may be x itself."""
    if stream is not None and _elsewhere(stream):
        return _within(stream, moe_dropout_residual, locals())
    bt, dev, shape = _typed(y, "y"), y.device, y.shape
    if out is None:
        out = torch.empty(shape, dtype=(y if x is None else x).dtype, device=dev)
    st = _typed(out, "out")
    _all_fit(dev, (y, "y", shape, y.dtype), (x, "x", shape, out.dtype),
             (out, "out", shape, out.dtype), (rng, "rng", (2,), torch.int64))
    _check(_on(dev, _lib.moe_dropout_residual, y.data_ptr(), _ptr(x), y.numel(), rng.data_ptr(),
               moe_dropout_config(p, residual_scale, branch_scale, st, bt), out.data_ptr(),
               _raw_stream(stream, dev)), "moe_dropout_residual")
    return out


def moe_dropout_residual_backward(d_out, rng, p, residual=True, residual_scale=1.0,
                                  branch_scale=1.0, dx=None, dy=None, branch_dtype=torch.bfloat16,
                                  stream=None):
    """Gradients of moe_dropout_residual by the same rng, p and scales: dict(dx,
    dy), dy of dy's type or branch_dtype, dx of d_out's type, or None without a
    residual. dx may be d_out itself."""
    if stream is not None and _elsewhere(stream):
        return _within(stream, moe_dropout_residual_backward, locals())
    st, dev, shape = _typed(d_out, "d_out"), d_out.device, d_out.shape
    if dy is None:
        dy = torch.empty(shape, dtype=branch_dtype, device=dev)
    bt = _typed(dy, "dy")
    if not residual:
        dx = None
    elif dx is None:
        dx = torch.empty(shape, dtype=d_out.dtype, device=dev)
    _all_fit(dev, (d_out, "d_out", shape, d_out.dtype), (dx, "dx", shape, d_out.dtype),
             (dy, "dy", shape, dy.dtype), (rng, "rng", (2,), torch.int64))
    _check(_on(dev, _lib.moe_dropout_residual_backward, d_out.data_ptr(), d_out.numel(),
               rng.data_ptr(), moe_dropout_config(p, residual_scale, branch_scale, st, bt),
               _ptr(dx), dy.data_ptr(), _raw_stream(stream, dev)), "moe_dropout_residual_backward")
    return dict(dx=dx, dy=dy)
