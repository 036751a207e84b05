"""MI355X (gfx950) quantized Mixture-of-Experts FFN layer.

A thin ctypes binding over ``libqmoe.so`` (C ABI declared in
``include/qmoe.h``).  This module only marshals arguments: it checks torch
tensors' device, dtype, contiguity and shape against the sizes it passes, and
hands raw device pointers plus the current HIP stream to the library.  Every
step of the layer runs in the library's HIP kernels; there is no fallback.
PyTorch provides device memory and streams.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmoe.so")

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_HIP = -4
DTYPE_F16 = 1
DTYPE_BF16 = 2
DTYPE_F32 = 3
MX_BLOCK = 32
ACT_SWIGLU = 0
ACT_GEGLU = 1
DECODE_MAX_ROUTES = 80
STAGE_ROUTE, STAGE_GROUP, STAGE_FC1, STAGE_FC2, STAGE_COMBINE = range(5)
RAW_SINGLE_BASE = 0
RAW_MULTI_BASE = 1

EXPORTED = ("qmoe_last_error", "qmoe_route", "qmoe_router", "qmoe_worklist_capacity", "qmoe_group",
            "qmoe_workspace_size", "qmoe_forward", "qmoe_forward_ex", "qmoe_forward_noalloc",
            "qmoe_shared_workspace_size", "qmoe_forward_shared", "qmoe_dequantize",
            "qmoe_raw_codes", "qmoe_permute_workspace_size", "qmoe_permute", "qmoe_unpermute",
            "qmoe_unpermute_backward", "qmoe_mx_quantize", "qmoe_mx_quantize_columns",
            "qmoe_mx_dequantize", "qmoe_mx_matmul",
            "qmoe_timer_start", "qmoe_timer_stop")


class QMoEError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"[{code}] {message}")
        self.code = code


class _Proj(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zero_points", ctypes.c_void_p), ("bits", ctypes.c_int32)]


class _LayerOpts(ctypes.Structure):
    _fields_ = [("fc1_bias", ctypes.c_void_p), ("fc2_bias", ctypes.c_void_p),
                ("fc3", ctypes.POINTER(_Proj)), ("fc3_bias", ctypes.c_void_p),
                ("router_weights", ctypes.c_void_p), ("swiglu_fusion", ctypes.c_int32),
                ("activation_alpha", ctypes.c_float), ("activation_beta", ctypes.c_float),
                ("swiglu_limit", ctypes.c_float)]


SWIGLU_SEPARATE, SWIGLU_INTERLEAVED, SWIGLU_HALVES = 0, 1, 2


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libqmoe.so and declare its signatures (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() or "
                           "python quantized_mixture_experts_route_amd/build.py")
    lib = ctypes.CDLL(path)
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    sz = ctypes.c_size_t
    lib.qmoe_last_error.restype = ctypes.c_char_p
    lib.qmoe_last_error.argtypes = []
    lib.qmoe_route.argtypes = [P, i64, i32, i32, i32, P, P, P]
    lib.qmoe_router.argtypes = [P, P, i64, i32, i32, i32, i32, i32, P, P, P, P]
    lib.qmoe_worklist_capacity.argtypes = [i64, i32, i32, i32, i32, i32]
    lib.qmoe_worklist_capacity.restype = i64
    lib.qmoe_group.argtypes = [P, i64, i32, i32, i32, i32, i32, P, P, P, i64, P, P]
    lib.qmoe_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32]
    lib.qmoe_workspace_size.restype = sz
    lib.qmoe_forward.argtypes = [P, P, i64, i32, i32, i32, ctypes.POINTER(_Proj),
                                 ctypes.POINTER(_Proj), f32, i32, i32, i32, i32, i32, P, P, P, P,
                                 sz, P]
    lib.qmoe_forward_ex.argtypes = [P, P, i64, i32, i32, i32, ctypes.POINTER(_Proj),
                                    ctypes.POINTER(_Proj), f32, i32, i32, i32, i32, i32, P, P, P,
                                    ctypes.POINTER(_LayerOpts), P, sz, P]
    lib.qmoe_forward_noalloc.argtypes = [P, P, i64, i32, i32, i32, ctypes.POINTER(_Proj),
                                         ctypes.POINTER(_Proj), f32, i32, i32, i32, i32, i32, P,
                                         P, P, P]
    lib.qmoe_shared_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32, i32]
    lib.qmoe_shared_workspace_size.restype = sz
    lib.qmoe_forward_shared.argtypes = [P, P, i64, i32, i32, i32, ctypes.POINTER(_Proj),
                                        ctypes.POINTER(_Proj), i32, ctypes.POINTER(_Proj),
                                        ctypes.POINTER(_Proj), P, f32, i32, i32, i32, i32, i32,
                                        P, P, P, P, sz, P]
    lib.qmoe_dequantize.argtypes = [ctypes.POINTER(_Proj), i32, i32, i32, i32, f32, i32, P, P, P]
    lib.qmoe_raw_codes.argtypes = [ctypes.POINTER(_Proj), i32, i32, i32, i32, i32, P, P]
    lib.qmoe_permute_workspace_size.argtypes = [i64, i32, i32]
    lib.qmoe_permute_workspace_size.restype = sz
    lib.qmoe_permute.argtypes = [P, i64, i64, i32, i32, P, i32, i32, P, P, P, P, P, sz, P]
    lib.qmoe_unpermute.argtypes = [P, i64, P, P, i64, i32, i32, i32, P, P]
    lib.qmoe_unpermute_backward.argtypes = [P, i64, P, i64, P, P, i64, i32, i32, i32, P, P, P]
    lib.qmoe_mx_quantize.argtypes = [P, i64, i64, i32, i32, P, P, P]
    lib.qmoe_mx_quantize_columns.argtypes = [P, i32, i32, i32, i32, P, P, P]
    lib.qmoe_mx_dequantize.argtypes = [P, P, i64, i32, i32, P, P]
    lib.qmoe_mx_matmul.argtypes = [P, P, i64, P, P, i32, i32, i32, P, P, i32, i64, i32, P, P]
    lib.qmoe_timer_start.argtypes = [i32]
    lib.qmoe_timer_stop.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64)]
    for name in ("qmoe_route", "qmoe_router", "qmoe_group", "qmoe_forward", "qmoe_forward_ex",
                 "qmoe_forward_noalloc",
                 "qmoe_forward_shared",
                 "qmoe_dequantize", "qmoe_raw_codes", "qmoe_permute", "qmoe_unpermute",
                 "qmoe_unpermute_backward", "qmoe_mx_quantize", "qmoe_mx_quantize_columns",
                 "qmoe_mx_dequantize", "qmoe_mx_matmul",
                 "qmoe_timer_start", "qmoe_timer_stop"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def last_error() -> str:
    return load_library().qmoe_last_error().decode()


def _check(rc: int):
    if rc != OK:
        raise QMoEError(rc, last_error())


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float16:
        return DTYPE_F16
    if dt == torch.bfloat16:
        return DTYPE_BF16
    raise ValueError(f"activation dtype must be float16 or bfloat16, got {dt}")


def zp_row_bytes(n_blocks: int, bits: int) -> int:
    return n_blocks if bits == 3 else -(-n_blocks // (8 // bits))


@dataclass
class Projection:
    """One quantized projection of all experts (device tensors).

    codes: uint8 [E, N, K*bits/8]; scales: fp16/bf16 [E, N, K/block_size];
    zero_points: None or uint8 [E, N, zp_row_bytes(K/block_size, bits)]."""
    codes: torch.Tensor
    scales: torch.Tensor
    zero_points: Optional[torch.Tensor]
    bits: int

    def _struct(self, E, N, K, block_size, name) -> _Proj:
        _dev(self.codes, f"{name}.codes", torch.uint8, (E, N, K * self.bits // 8))
        _dev(self.scales, f"{name}.scales", (torch.float16, torch.bfloat16),
             (E, N, K // block_size))
        if self.zero_points is not None:
            _dev(self.zero_points, f"{name}.zero_points", torch.uint8,
                 (E, N, zp_row_bytes(K // block_size, self.bits)))
        return _Proj(_ptr(self.codes), _ptr(self.scales), _ptr(self.zero_points), int(self.bits))


def route(logits: torch.Tensor, top_k: int, normalize: int = 1, stream=None):
    """Top-k expert ids (int32 [T, k]) and weights (float32 [T, k]) on the device."""
    _dev(logits, "logits", torch.float32)
    T, E = logits.shape
    ids = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    _check(load_library().qmoe_route(_ptr(logits), T, E, top_k, normalize, _ptr(ids), _ptr(w),
                                     _stream(stream)))
    return ids, w


def router(hidden: torch.Tensor, gate_weight: torch.Tensor, top_k: int, normalize: int = 1,
           want_logits: bool = True, stream=None):
    """Router projection + top-k in one launch: (logits float32 [T, E] or None,
    ids int32 [T, k], weights float32 [T, k]); gate_weight is [E, H] in hidden's dtype."""
    dt = dtype_code(hidden.dtype)
    _dev(hidden, "hidden")
    T, H = hidden.shape
    E = gate_weight.shape[0]
    _dev(gate_weight, "gate_weight", hidden.dtype, (E, H))
    dev = hidden.device
    logits = torch.empty((T, E), dtype=torch.float32, device=dev) if want_logits else None
    ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    _check(load_library().qmoe_router(_ptr(hidden), _ptr(gate_weight), T, H, E, dt, top_k,
                                      normalize, _ptr(logits), _ptr(ids), _ptr(w),
                                      _stream(stream)))
    return logits, ids, w


def worklist_capacity(T, top_k, E, m_tile, n_tile, N) -> int:
    return int(load_library().qmoe_worklist_capacity(T, top_k, E, m_tile, n_tile, N))


def group(topk_ids: torch.Tensor, E: int, m_tile: int, n_tile: int, N: int, stream=None,
          capacity: Optional[int] = None):
    """Expert offsets [E+1], sorted route ids [R], work-list [cap, 3], item count [1] (device)."""
    _dev(topk_ids, "topk_ids", torch.int32)
    T, top_k = topk_ids.shape if topk_ids.dim() == 2 else (topk_ids.numel(), 1)
    R = T * top_k
    cap = worklist_capacity(T, top_k, E, m_tile, n_tile, N) if capacity is None else capacity
    dev = topk_ids.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sorted_routes = torch.full((max(R, 1),), -1, dtype=torch.int32, device=dev)
    worklist = torch.zeros((max(cap, 1), 3), dtype=torch.int32, device=dev)
    n_items = torch.zeros(1, dtype=torch.int32, device=dev)
    _check(load_library().qmoe_group(_ptr(topk_ids), T, top_k, E, m_tile, n_tile, N,
                                     _ptr(offsets), _ptr(sorted_routes), _ptr(worklist), cap,
                                     _ptr(n_items), _stream(stream)))
    return offsets, sorted_routes[:R], worklist, n_items


def workspace_size(T, H, I, E, top_k, dtype) -> int:
    return int(load_library().qmoe_workspace_size(T, H, I, E, top_k, dtype))


def alloc_workspace(T, H, I, E, top_k, dtype, device="cuda") -> torch.Tensor:
    n = workspace_size(T, H, I, E, top_k, dtype)
    if n == 0:
        raise ValueError("invalid sizes for the workspace")
    return torch.empty(n, dtype=torch.uint8, device=device)  # torch blocks are 512-byte aligned


def forward(hidden: torch.Tensor, logits: torch.Tensor, fc1: Projection, fc2: Projection, *,
            top_k: int, block_size: int, normalize: int = 1, activation: int = ACT_SWIGLU,
            zero_point_offset: float = math.nan, out: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, return_routing: bool = False,
            stream=None, fc1_bias: Optional[torch.Tensor] = None,
            fc2_bias: Optional[torch.Tensor] = None, fc3: Optional[Projection] = None,
            fc3_bias: Optional[torch.Tensor] = None,
            router_weights: Optional[torch.Tensor] = None,
            swiglu_fusion: int = SWIGLU_INTERLEAVED, activation_alpha: float = 1.0,
            activation_beta: float = 0.0, swiglu_limit: float = math.inf):
    """The QMoE layer: out [T, H] in hidden's dtype (plus routing if asked).

    The keyword options after ``stream`` are the operator's optional inputs and
    attributes (qmoe_forward_ex): expert biases (float32), a separate up
    projection fc3 with swiglu_fusion = SWIGLU_SEPARATE, the gate/up halves
    layout SWIGLU_HALVES, router_weights (float32 [T, E]) and the SwiGLU
    parameters."""
    dt = dtype_code(hidden.dtype)
    _dev(hidden, "hidden")
    T, H = hidden.shape
    _dev(logits, "logits", torch.float32)
    if logits.shape[0] != T:
        raise ValueError("logits rows must equal hidden rows")
    E = logits.shape[1]
    for name, proj in (("fc1", fc1), ("fc2", fc2)):
        # the library reads scales as the layer's dtype; another dtype's bits would be misread
        if proj.scales.dtype != hidden.dtype:
            raise ValueError(f"{name}.scales has dtype {proj.scales.dtype}, expected {hidden.dtype}")
    I = fc2.codes.shape[2] * 8 // fc2.bits
    n1 = I if swiglu_fusion == SWIGLU_SEPARATE else 2 * I
    p1 = fc1._struct(E, n1, H, block_size, "fc1")
    p2 = fc2._struct(E, H, I, block_size, "fc2")
    if out is None:
        out = torch.empty_like(hidden)
    _dev(out, "out", hidden.dtype, (T, H))
    if workspace is None:
        workspace = alloc_workspace(T, H, I, E, top_k, dt, hidden.device)
    _dev(workspace, "workspace", torch.uint8)
    ids = w = None
    if return_routing:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=hidden.device)
        w = torch.empty((T, top_k), dtype=torch.float32, device=hidden.device)
    p3 = None
    if fc3 is not None:
        if fc3.scales.dtype != hidden.dtype:
            raise ValueError(f"fc3.scales has dtype {fc3.scales.dtype}, expected {hidden.dtype}")
        p3 = fc3._struct(E, I, H, block_size, "fc3")
    for name, b, shape in (("fc1_bias", fc1_bias, (E, n1)), ("fc2_bias", fc2_bias, (E, H)),
                           ("fc3_bias", fc3_bias, (E, I)), ("router_weights", router_weights, (T, E))):
        if b is not None:
            _dev(b, name, torch.float32, shape)
    opts = _LayerOpts(_ptr(fc1_bias), _ptr(fc2_bias), ctypes.pointer(p3) if p3 is not None else None,
                      _ptr(fc3_bias), _ptr(router_weights), int(swiglu_fusion),
                      float(activation_alpha), float(activation_beta), float(swiglu_limit))
    _check(load_library().qmoe_forward_ex(
        _ptr(hidden), _ptr(logits), T, H, I, E, ctypes.byref(p1), ctypes.byref(p2),
        float(zero_point_offset), block_size, top_k, normalize, activation, dt, _ptr(out),
        _ptr(ids), _ptr(w), ctypes.byref(opts), _ptr(workspace), workspace.numel(),
        _stream(stream)))
    return (out, ids, w) if return_routing else out


def forward_shared(hidden: torch.Tensor, logits: torch.Tensor, fc1: Projection, fc2: Projection,
                   shared_fc1: Projection, shared_fc2: Projection, shared_gate: torch.Tensor, *,
                   top_k: int, block_size: int, normalize: int = 1, activation: int = ACT_SWIGLU,
                   zero_point_offset: float = math.nan, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, return_routing: bool = False,
                   stream=None):
    """The layer with a shared expert: routed output + sigmoid(x . shared_gate) * shared FFN."""
    dt = dtype_code(hidden.dtype)
    _dev(hidden, "hidden")
    T, H = hidden.shape
    _dev(logits, "logits", torch.float32)
    E = logits.shape[1]
    for name, proj in (("fc1", fc1), ("fc2", fc2), ("shared_fc1", shared_fc1),
                       ("shared_fc2", shared_fc2)):
        if proj.scales.dtype != hidden.dtype:
            raise ValueError(f"{name}.scales has dtype {proj.scales.dtype}, expected {hidden.dtype}")
    I = fc2.codes.shape[2] * 8 // fc2.bits
    Is = shared_fc2.codes.shape[2] * 8 // shared_fc2.bits
    p1 = fc1._struct(E, 2 * I, H, block_size, "fc1")
    p2 = fc2._struct(E, H, I, block_size, "fc2")
    s1 = shared_fc1._struct(1, 2 * Is, H, block_size, "shared_fc1")
    s2 = shared_fc2._struct(1, H, Is, block_size, "shared_fc2")
    _dev(shared_gate, "shared_gate", hidden.dtype, (H,))
    if out is None:
        out = torch.empty_like(hidden)
    _dev(out, "out", hidden.dtype, (T, H))
    if workspace is None:
        n = int(load_library().qmoe_shared_workspace_size(T, H, I, E, top_k, Is, dt))
        if n == 0:
            raise ValueError("invalid sizes for the shared-expert workspace")
        workspace = torch.empty(n, dtype=torch.uint8, device=hidden.device)
    _dev(workspace, "workspace", torch.uint8)
    ids = w = None
    if return_routing:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=hidden.device)
        w = torch.empty((T, top_k), dtype=torch.float32, device=hidden.device)
    _check(load_library().qmoe_forward_shared(
        _ptr(hidden), _ptr(logits), T, H, I, E, ctypes.byref(p1), ctypes.byref(p2), Is,
        ctypes.byref(s1), ctypes.byref(s2), _ptr(shared_gate), float(zero_point_offset),
        block_size, top_k, normalize, activation, dt, _ptr(out), _ptr(ids), _ptr(w),
        _ptr(workspace), workspace.numel(), _stream(stream)))
    return (out, ids, w) if return_routing else out


NOALLOC_SCRATCH_BYTES = 64 << 20


def forward_noalloc(hidden: torch.Tensor, logits: torch.Tensor, fc1: Projection,
                    fc2: Projection, *, top_k: int, block_size: int, normalize: int = 1,
                    activation: int = ACT_SWIGLU, zero_point_offset: float = math.nan,
                    out: torch.Tensor, return_routing: bool = False, stream=None):
    """The QMoE layer through qmoe_forward_noalloc: the library's fixed scratch
    array serves as workspace and the call allocates nothing on the device
    (``out`` and, with return_routing, the routing outputs are the caller's)."""
    dt = dtype_code(hidden.dtype)
    _dev(hidden, "hidden")
    T, H = hidden.shape
    _dev(logits, "logits", torch.float32)
    if logits.shape[0] != T:
        raise ValueError("logits rows must equal hidden rows")
    E = logits.shape[1]
    for name, proj in (("fc1", fc1), ("fc2", fc2)):
        if proj.scales.dtype != hidden.dtype:
            raise ValueError(f"{name}.scales has dtype {proj.scales.dtype}, expected {hidden.dtype}")
    I = fc2.codes.shape[2] * 8 // fc2.bits
    p1 = fc1._struct(E, 2 * I, H, block_size, "fc1")
    p2 = fc2._struct(E, H, I, block_size, "fc2")
    _dev(out, "out", hidden.dtype, (T, H))
    ids = w = None
    if return_routing:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=hidden.device)
        w = torch.empty((T, top_k), dtype=torch.float32, device=hidden.device)
    _check(load_library().qmoe_forward_noalloc(
        _ptr(hidden), _ptr(logits), T, H, I, E, ctypes.byref(p1), ctypes.byref(p2),
        float(zero_point_offset), block_size, top_k, normalize, activation, dt, _ptr(out),
        _ptr(ids), _ptr(w), _stream(stream)))
    return (out, ids, w) if return_routing else out


def dequantize(proj: Projection, E: int, N: int, K: int, block_size: int, dtype: torch.dtype,
               zero_point_offset: float = math.nan, want_codes: bool = True, stream=None):
    """Unpacked codes (int32 [E, N, K] or None) and dequantized weights (dtype [E, N, K])."""
    if proj.scales.dtype != dtype:
        raise ValueError(f"scales have dtype {proj.scales.dtype}, expected {dtype}")
    p = proj._struct(E, N, K, block_size, "projection")
    dev = proj.codes.device
    w = torch.empty((E, N, K), dtype=dtype, device=dev)
    q = torch.empty((E, N, K), dtype=torch.int32, device=dev) if want_codes else None
    _check(load_library().qmoe_dequantize(ctypes.byref(p), E, N, K, block_size,
                                          float(zero_point_offset), dtype_code(dtype), _ptr(q),
                                          _ptr(w), _stream(stream)))
    return q, w


def raw_codes(proj: Projection, E: int, N: int, K: int, block_size: int, dtype: torch.dtype,
              variant: int = RAW_SINGLE_BASE, stream=None):
    """int32 [E, N, K]: the codes the decode kernels' raw-code MFMA operands carry."""
    p = proj._struct(E, N, K, block_size, "projection")
    q = torch.empty((E, N, K), dtype=torch.int32, device=proj.codes.device)
    _check(load_library().qmoe_raw_codes(ctypes.byref(p), E, N, K, dtype_code(dtype), variant,
                                         _ptr(q), _stream(stream)))
    return q


# ------------------------------------------------ sorted by expert and back, MXFP4
# None of these is recorded by autograd: the gradients are calls of their own.  One call takes a few
# microseconds on the GPU, so the binding's own time counts: a tensor that is right passes one
# comparison, and the message is worked out only for one that is not.
_ROW_DTYPES = {torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


def _row_dtype(dt: torch.dtype, name: str) -> int:
    code = _ROW_DTYPES.get(dt)
    if code is None:
        raise ValueError(f"{name} must be float16, bfloat16 or float32, got {dt}")
    return code


def _index(t, name: str, dim: int) -> int:
    """The device index of a call's leading tensor, which must have `dim` dimensions."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    return t.get_device()


def _tensor(t, name: str, index: int, dtype, shape) -> int:
    """Checks a contiguous tensor on device `index`; its address."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        _dev(t, name, dtype, shape)
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    return t.data_ptr()


def _rows(t, name: str, index: int, n: int) -> int:
    """Checks a matrix of n rows (any row stride, neighbouring elements); its row stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dim() != 2 or t.shape[0] != n:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {n} rows")
    h = t.shape[1]
    if h < 1:
        raise ValueError(f"{name} has no columns")
    if t.is_contiguous():
        return h
    stride, step = t.stride()
    if h > 1 and step != 1 or n > 1 and stride < h:
        raise ValueError(f"{name} must have contiguous, non-overlapping rows")
    return stride if n > 1 else h


def _end(t: torch.Tensor) -> int:
    """The address behind a tensor's last element."""
    return t.data_ptr() + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))


def _apart(out: torch.Tensor, **inputs) -> None:
    """Checks that a given output shares no memory with what its kernel reads meanwhile."""
    lo = out.data_ptr()
    hi = lo + out.numel() * out.element_size()
    for name, t in inputs.items():
        if t is not None and t.numel() and lo < _end(t) and t.data_ptr() < hi:
            raise ValueError(f"out overlaps {name}")


_I32_MAX = (1 << 31) - 1


def _fit(*sizes: int):
    """Checks sizes that the library takes as 32-bit integers: ctypes would pass their low bits."""
    for n in sizes:
        if not -_I32_MAX <= n <= _I32_MAX:
            raise QMoEError(ERR_UNSUPPORTED, f"qmoe: size {n} does not fit 32 bits")


def _elsewhere(index: int, stream) -> bool:
    """Whether a call must be made under _on(): on a given stream or not on the current device."""
    return stream is not None or index != _current_device()


def _on(index: int, stream):
    """Makes the device and the stream current, so that outputs are allocated for the stream that
    fills them and the launch goes to the tensors' device."""
    if stream is None:
        stream = torch.cuda.current_stream(index)
    elif stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, tensors are on cuda:{index}")
    return torch.cuda.stream(stream)


# what torch.cuda's own functions call, without the objects and checks around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _current(index: int) -> int:
    """The handle of the current stream."""
    if _raw_stream is None:
        return torch.cuda.current_stream(index).cuda_stream
    return _raw_stream(index)


@functools.lru_cache(maxsize=256)
def permute_workspace_size(T: int, top_k: int, E: int) -> int:
    _fit(top_k, E)
    return int(load_library().qmoe_permute_workspace_size(T, top_k, E))


def permute(hidden: Optional[torch.Tensor], topk_ids: torch.Tensor, E: int, *,
            workspace: Optional[torch.Tensor] = None, stream=None):
    """Tokens sorted by expert: (rows [T*k, H], expert_offsets int32 [E+1], sorted_routes int32
    [T*k], route_rows int32 [T, k]).

    hidden: float16, bfloat16 or float32 [T, H], any row stride; None: rows is None and only the
    maps are made.  Ids outside [0, E) drop their route: its row, behind the last expert's, is zero
    and its route_rows entry is -1 - row.  Autograd does not record the call: rows are detached from
    hidden, and permute_backward is its gradient."""
    dev = _index(topk_ids, "topk_ids", 2)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return permute(hidden, topk_ids, E, workspace=workspace)
    T, top_k = topk_ids.shape
    R = T * top_k
    ids = _tensor(topk_ids, "topk_ids", dev, torch.int32, (T, top_k))
    stride, H, dt, rows = 0, 0, DTYPE_F16, None
    if hidden is not None:
        stride, H, dt = _rows(hidden, "hidden", dev, T), hidden.shape[1], _row_dtype(hidden.dtype, "hidden")
        if H > _I32_MAX:
            _fit(H)
        rows = hidden.new_empty((R, H))
    lib = load_library()
    need = permute_workspace_size(T, top_k, E)  # refuses a top_k or E of more than 32 bits
    if workspace is not None:
        _tensor(workspace, "workspace", dev, torch.uint8, workspace.shape)
    elif need:
        workspace = topk_ids.new_empty((need,), dtype=torch.uint8)
    offsets = topk_ids.new_empty((max(E, 0) + 1,))
    order = topk_ids.new_empty((R,))
    route_rows = torch.empty_like(topk_ids)
    _check(lib.qmoe_permute(_ptr(hidden), stride, T, H, dt, ids, top_k, E, _ptr(rows), offsets.data_ptr(),
                            order.data_ptr(), route_rows.data_ptr(), _ptr(workspace),
                            0 if workspace is None else workspace.numel(), _current(dev)))
    return rows, offsets, order, route_rows


def unpermute(rows: torch.Tensor, route_rows: torch.Tensor, weights: Optional[torch.Tensor] = None, *,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows back to their tokens: out[t] = sum over slots of weights[t, s] * rows[route_rows[t, s]]
    (float32 sums, rounded once; no weights: 1); dropped routes add nothing.  out must not overlap
    rows.  Autograd does not record the call: unpermute_backward is its gradient."""
    dev = _index(route_rows, "route_rows", 2)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return unpermute(rows, route_rows, weights, out=out)
    shape = route_rows.shape
    T, top_k = shape
    at = _tensor(route_rows, "route_rows", dev, torch.int32, shape)
    stride, dt = _rows(rows, "rows", dev, T * top_k), _row_dtype(rows.dtype, "rows")
    H = rows.shape[1]
    if H > _I32_MAX or top_k > _I32_MAX:
        _fit(H, top_k)
    w = None if weights is None else _tensor(weights, "weights", dev, torch.float32, shape)
    if out is None:
        out = rows.new_empty((T, H))
        to = out.data_ptr()
    else:
        to = _tensor(out, "out", dev, rows.dtype, (T, H))
        _apart(out, rows=rows, route_rows=route_rows, weights=weights)
    _check(load_library().qmoe_unpermute(rows.data_ptr(), stride, at, w, T, top_k, H, dt, to, _current(dev)))
    return out


def permute_backward(grad_rows: torch.Tensor, route_rows: torch.Tensor, *,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of permute with respect to hidden: the sum of a token's rows' gradients."""
    return unpermute(grad_rows, route_rows, None, out=out, stream=stream)


def unpermute_backward(grad_out: torch.Tensor, rows: Optional[torch.Tensor], route_rows: torch.Tensor,
                       weights: Optional[torch.Tensor] = None, *, stream=None):
    """The gradient of unpermute: (grad_rows [T*k, H], grad_weights float32 [T, k]).  rows None:
    grad_weights is not computed (None), as for an unpermute without weights.  route_rows has to be
    permute's, which names every row once: of a table of one's own, rows that no entry names come back
    undefined, and -1 stands for a dropped route at row 0, which it clears.  Autograd does not record
    the call."""
    dev = _index(route_rows, "route_rows", 2)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return unpermute_backward(grad_out, rows, route_rows, weights)
    shape = route_rows.shape
    T, top_k = shape
    at = _tensor(route_rows, "route_rows", dev, torch.int32, shape)
    gstride, dt = _rows(grad_out, "grad_out", dev, T), _row_dtype(grad_out.dtype, "grad_out")
    H = grad_out.shape[1]
    if H > _I32_MAX or top_k > _I32_MAX:
        _fit(H, top_k)
    stride, grad_weights = 0, None
    if rows is not None:
        stride = _rows(rows, "rows", dev, T * top_k)
        if rows.dtype is not grad_out.dtype or rows.shape[1] != H:
            raise ValueError(f"rows is {rows.dtype} {tuple(rows.shape)}, expected {grad_out.dtype} "
                             f"{(T * top_k, H)}")
        grad_weights = route_rows.new_empty(shape, dtype=torch.float32)
    w = None if weights is None else _tensor(weights, "weights", dev, torch.float32, shape)
    grad_rows = grad_out.new_empty((T * top_k, H))
    _check(load_library().qmoe_unpermute_backward(
        grad_out.data_ptr(), gstride, _ptr(rows), stride, at, w, T, top_k, H, dt, grad_rows.data_ptr(),
        _ptr(grad_weights), _current(dev)))
    return grad_rows, grad_weights


def mx_quantize(x: torch.Tensor, *, transpose: bool = False, stream=None):
    """MXFP4 codes (uint8 [..., K/2]) and scales (uint8 [..., K/32]) of x [..., K], blocks of 32 along
    K (a matrix may have any row stride).  transpose: x [E, rows, K] or [rows, K] is quantised along
    its rows, giving codes [E, K, rows/2] and scales [E, K, rows/32] of the transposed matrices.
    Autograd does not record the call (the usual gradient passes straight through)."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("x must be a CUDA (HIP) tensor")
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return mx_quantize(x, transpose=transpose)
    dt = _row_dtype(x.dtype, "x")
    lib = load_library()
    if transpose:
        if x.dim() not in (2, 3):
            raise ValueError("x must have 2 or 3 dimensions to be quantised along its rows")
        _dev(x, "x")
        *lead, rows, K = x.shape
        _fit(*lead, rows, K)
        codes = x.new_empty((*lead, K, rows // 2), dtype=torch.uint8)
        scales = x.new_empty((*lead, K, rows // MX_BLOCK), dtype=torch.uint8)
        _check(lib.qmoe_mx_quantize_columns(x.data_ptr(), lead[0] if lead else 1, rows, K, dt,
                                            codes.data_ptr(), scales.data_ptr(), _current(dev)))
        return codes, scales
    if x.dim() < 1:
        raise ValueError("x must have at least 1 dimension")
    *lead, K = x.shape
    if K > _I32_MAX:
        _fit(K)
    if x.dim() == 2:
        rows = lead[0]
        stride = _rows(x, "x", dev, rows)
    else:
        _dev(x, "x")
        rows, stride = math.prod(lead), K
    codes = x.new_empty((*lead, K // 2), dtype=torch.uint8)
    scales = x.new_empty((*lead, K // MX_BLOCK), dtype=torch.uint8)
    _check(lib.qmoe_mx_quantize(x.data_ptr(), stride, rows, K, dt, codes.data_ptr(), scales.data_ptr(),
                                _current(dev)))
    return codes, scales


def _mx(codes, scales, name: str, index: int) -> int:
    """Checks a pair of codes [..., K/2] and scales [..., K/32]; K."""
    if (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor) and codes.get_device() == index
            and scales.get_device() == index and codes.dtype is torch.uint8 and scales.dtype is torch.uint8
            and codes.is_contiguous() and scales.is_contiguous()):
        *lead, half = codes.shape or (0,)
        if half % 16 == 0 and scales.shape == (*lead, half // 16):
            return half * 2
    _dev(codes, f"{name}_codes", torch.uint8)
    _dev(scales, f"{name}_scales", torch.uint8)
    if codes.get_device() != index or scales.get_device() != index:
        raise ValueError(f"{name}_codes is on {codes.device}, {name}_scales on {scales.device}, expected cuda:{index}")
    raise ValueError(f"{name}_codes {tuple(codes.shape)} (two values a byte) and {name}_scales "
                     f"{tuple(scales.shape)} (one byte for {MX_BLOCK} values) do not belong together")


def mx_dequantize(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype, *,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """What MXFP4 codes [..., K/2] with scales [..., K/32] stand for, [..., K] in dtype."""
    dt = _row_dtype(dtype, "dtype")
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda:
        raise ValueError("codes must be a CUDA (HIP) tensor")
    dev = codes.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return mx_dequantize(codes, scales, dtype, out=out)
    K = _mx(codes, scales, "mx", dev)
    if K > _I32_MAX:
        _fit(K)
    shape = (*codes.shape[:-1], K)
    if out is None:
        out = codes.new_empty(shape, dtype=dtype)
        to = out.data_ptr()
    else:
        to = _tensor(out, "out", dev, dtype, shape)
        _apart(out, codes=codes, scales=scales)
    _check(load_library().qmoe_mx_dequantize(codes.data_ptr(), scales.data_ptr(), math.prod(shape[:-1]), K, dt,
                                             to, _current(dev)))
    return out


def mx_matmul(a_codes: torch.Tensor, a_scales: torch.Tensor, w_codes: torch.Tensor,
              w_scales: torch.Tensor, expert_offsets: Optional[torch.Tensor] = None, *,
              sorted_routes: Optional[torch.Tensor] = None, top_k: Optional[int] = None,
              dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Grouped product of MXFP4 rows with MXFP4 expert weights: out [rows, N] in dtype.

    a: [A, K] rows; w: [E, N, K] (or [N, K], one expert); expert_offsets int32 [E+1]: the rows of each
    expert (may be omitted for one expert).  sorted_routes int32 [rows], only together with top_k: row r
    takes a's row sorted_routes[r] // top_k (top_k 1: sorted_routes names a's rows); without it row r
    takes a's row r.  Rows behind the last expert's are zero.  out must not overlap an operand.  Autograd
    does not record the call: the gradient of the rows is the same product on w quantised with
    transpose=True (sorted rows then go through permute_backward to their tokens)."""
    if top_k is None:
        if sorted_routes is not None:  # permute's routes without their top_k would read other tokens
            raise ValueError("sorted_routes needs top_k")
        top_k = 1
    dt = _row_dtype(dtype, "dtype")
    dev = _index(a_codes, "a_codes", 2)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return mx_matmul(a_codes, a_scales, w_codes, w_scales, expert_offsets, sorted_routes=sorted_routes,
                             top_k=top_k, dtype=dtype, out=out)
    K = _mx(a_codes, a_scales, "a", dev)
    if _mx(w_codes, w_scales, "w", dev) != K:
        raise ValueError(f"a has {K} values a row, w {w_codes.shape[-1] * 2}")
    if w_codes.dim() not in (2, 3):
        raise ValueError(f"w_codes must have 2 or 3 dimensions, got {w_codes.dim()}")
    E, N = (1, w_codes.shape[0]) if w_codes.dim() == 2 else w_codes.shape[:2]
    if max(E, N, K, top_k) > _I32_MAX or top_k < 0:
        _fit(E, N, K, top_k)
    offsets = routes = None
    if expert_offsets is not None:
        offsets = _tensor(expert_offsets, "expert_offsets", dev, torch.int32, (E + 1,))
    A = rows = a_codes.shape[0]
    if sorted_routes is not None:
        _index(sorted_routes, "sorted_routes", 1)
        rows = sorted_routes.shape[0]
        routes = _tensor(sorted_routes, "sorted_routes", dev, torch.int32, (rows,))
    if out is None:
        out = a_codes.new_empty((rows, N), dtype=dtype)
        to = out.data_ptr()
    else:
        to = _tensor(out, "out", dev, dtype, (rows, N))
        _apart(out, a_codes=a_codes, a_scales=a_scales, w_codes=w_codes, w_scales=w_scales,
               expert_offsets=expert_offsets, sorted_routes=sorted_routes)
    _check(load_library().qmoe_mx_matmul(
        a_codes.data_ptr(), a_scales.data_ptr(), A, w_codes.data_ptr(), w_scales.data_ptr(), E, N, K, offsets,
        routes, top_k, rows, dt, to, _current(dev)))
    return out


def timer_start(stage: int):
    _check(load_library().qmoe_timer_start(stage))


def timer_stop():
    """(summed milliseconds, number of launches timed) since timer_start."""
    ms = ctypes.c_double(0.0)
    n = ctypes.c_int64(0)
    _check(load_library().qmoe_timer_stop(ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value
