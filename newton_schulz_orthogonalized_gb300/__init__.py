"""Python binding of libnsmuon.so, the GB300 owner-side Muon optimizer step.

This module only marshals arguments: it turns torch tensors into device pointers and
host tables into C arrays and calls the C ABI declared in ``include/nsmuon.h``.  Every
step of the optimizer runs in the library's CUDA kernels; there is no CPU fallback, and
importing the binding fails loudly when the library has not been built.

Names follow the pages ("DeepSpeed 集成 Muon 优化器实战"): ``ns_method`` is
``"standard"`` or ``"gram"`` (default ``"gram"``), ``muon_lr`` / ``adam_lr`` override a
group's ``lr``, the Muon group defaults are lr 0.02 and momentum 0.95, and the Adam group
defaults are lr 3e-4, betas (0.9, 0.95) and eps 1e-10.
"""

from __future__ import annotations

import ctypes
import os
from typing import Dict, Iterable, List, Optional, Sequence, Tuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_REGULAR = os.path.join(_HERE, "libnsmuon.so")
# the bounds-checked build: every kernel tests each access to a matrix's elements before
# making it, records a failure (NSM_ERR_BOUNDS) and skips the access
LIB_CHECKED = os.path.join(_HERE, "libnsmuon_checked.so")
# NSM_CHECKED=1 in the environment makes this process load the checked build
LIB_PATH = LIB_CHECKED if os.environ.get("NSM_CHECKED") == "1" else LIB_REGULAR

NSM_OK = 0
NSM_ERR_NULL = -1
NSM_ERR_SHAPE = -2
NSM_ERR_OFFSET = -3
NSM_ERR_ALIGN = -4
NSM_ERR_METHOD = -5
NSM_ERR_WORKSPACE = -6
NSM_ERR_CUDA = -7
NSM_ERR_TIMEOUT = -8
NSM_ERR_ARG = -9
NSM_ERR_BOUNDS = -10

NS_METHODS = {"standard": 0, "gram": 1, "standard_bf16": 2}
NS_METHOD_DEFAULT = "gram"
NS_STEPS_DEFAULT = 5
MUON_LR_DEFAULT = 0.02
MUON_MOMENTUM_DEFAULT = 0.95
ADAM_LR_DEFAULT = 3e-4
ADAM_BETAS_DEFAULT = (0.9, 0.95)
ADAM_EPS_DEFAULT = 1e-10
# an exponent that no matrix's entries fit: the step chooses one, as it does where none was left
EXPONENT_NONE = 120

_c_i32p = ctypes.POINTER(ctypes.c_int32)
_c_i64p = ctypes.POINTER(ctypes.c_int64)
_vp = ctypes.c_void_p

_lib: Optional[ctypes.CDLL] = None


class NsmError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"nsmuon error {code}: {message}")
        self.code = code


def lib() -> ctypes.CDLL:
    """Loads libnsmuon.so, or libnsmuon_checked.so when NSM_CHECKED=1 (both built in-tree
    by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`")
    L = ctypes.CDLL(LIB_PATH)
    L.nsm_version.restype = ctypes.c_int
    L.nsm_last_error.restype = ctypes.c_char_p
    L.nsm_last_launch_count.restype = ctypes.c_int
    L.nsm_route.argtypes = [ctypes.c_char_p, ctypes.c_int]
    L.nsm_route.restype = ctypes.c_int
    L.nsm_pack.argtypes = [_c_i32p, ctypes.c_int, ctypes.c_int64, _c_i64p, _c_i64p]
    L.nsm_pack.restype = ctypes.c_int
    _c_ip = ctypes.POINTER(ctypes.c_int)
    L.nsm_input_exponent.argtypes = [ctypes.c_float, ctypes.c_int, ctypes.c_int, _c_ip, _c_ip, _c_ip]
    L.nsm_input_exponent.restype = ctypes.c_int
    L.nsm_assign_owners.argtypes = [_c_i32p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                    ctypes.c_int, _c_i32p, _c_i64p]
    L.nsm_assign_owners.restype = ctypes.c_int
    L.nsm_workspace_iterate.argtypes = [_c_i32p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.POINTER(ctypes.c_size_t),
                                        ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
    L.nsm_workspace_iterate.restype = ctypes.c_int
    L.muon_workspace_bytes.argtypes = [_c_i32p, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    L.muon_workspace_bytes.restype = ctypes.c_size_t
    L.muon_step.argtypes = [_vp, _vp, _vp, _c_i64p, _c_i32p, ctypes.c_int, ctypes.c_float,
                            ctypes.c_float, ctypes.c_float, ctypes.c_int, ctypes.c_int,
                            ctypes.c_int, _vp, ctypes.c_size_t, _vp]
    L.muon_step.restype = ctypes.c_int
    L.muon_step_with_copy.argtypes = [_vp, _vp, _vp, _vp, _c_i64p, _c_i32p, ctypes.c_int,
                                      ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_int,
                                      ctypes.c_int, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
    L.muon_step_with_copy.restype = ctypes.c_int
    L.muon_orthogonalize.argtypes = [_vp, _vp, _c_i64p, _c_i32p, ctypes.c_int, ctypes.c_int,
                                     ctypes.c_int, _vp, ctypes.c_size_t, _vp]
    L.muon_orthogonalize.restype = ctypes.c_int
    L.muon_orthogonalize_noalloc.argtypes = [_vp, _vp, _c_i64p, _c_i32p, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_int, _vp]
    L.muon_orthogonalize_noalloc.restype = ctypes.c_int
    L.adamw_step.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int64, ctypes.c_float, ctypes.c_float,
                             ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_int, _vp]
    L.adamw_step.restype = ctypes.c_int
    L.nsm_gemm.argtypes = [_vp, ctypes.c_int, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp,
                           ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                           ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_float,
                           ctypes.c_float, _vp, ctypes.c_size_t, _vp]
    L.nsm_gemm.restype = ctypes.c_int
    L.nsm_gemm_scratch_bytes.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int]
    L.nsm_gemm_scratch_bytes.restype = ctypes.c_size_t
    _i64, _int, _f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_float
    rows_of_logits = [_vp, _int, _i64, _i64, _i64]
    tokens_and_t = [_vp, _int, _f32]
    entries = [_vp, _int, _i64, _vp, _int, _i64, _int, _f32, _int]
    L.nsm_logprobs.argtypes = rows_of_logits + tokens_and_t + [_int, _vp, _vp, _vp, _vp, _vp, _vp]
    L.nsm_logprobs_grad.argtypes = rows_of_logits + tokens_and_t + [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp]
    L.nsm_logprobs_backward.argtypes = rows_of_logits + tokens_and_t + [_vp, _vp, _vp, _vp, _vp, _i64, _vp]
    L.nsm_distill.argtypes = rows_of_logits + entries + [_vp, _vp, _vp, _vp]
    L.nsm_distill_grad.argtypes = rows_of_logits + entries + [_vp, _vp, _i64, _vp, _vp, _vp, _vp]
    L.nsm_distill_backward.argtypes = rows_of_logits + entries + [_vp, _vp, _vp, _vp, _i64, _vp]
    history = [_vp, _int, _i64, _i64, _i64, _vp, _vp]
    mask = [_vp, _i64, _i64, _vp]
    L.nsm_adjust_logits.argtypes = rows_of_logits + history + [_vp, _vp, _vp, _vp, _int, _i64, _vp, _i64, _int] + mask \
        + [_vp, _int, _i64, _vp]
    L.nsm_adjust_logits_backward.argtypes = rows_of_logits + history + [_vp] + mask + [_vp, _int, _i64, _vp, _i64, _vp]
    L.nsm_embedding.argtypes = [_vp, _int, _i64, _i64, _i64, _vp, _int, _i64, _f32, _vp, _int, _i64, _vp]
    L.nsm_embedding_backward.argtypes = [_vp, _int, _i64, _i64, _i64, _vp, _int, _i64, _f32, _int, _vp, _int, _i64, _vp,
                                         ctypes.c_size_t, _vp]
    L.nsm_embedding_workspace_bytes.argtypes = [_i64, _i64, _i64]
    L.nsm_embedding_workspace_bytes.restype = ctypes.c_size_t
    L.nsm_grad_norm.argtypes = [_vp, _vp, _vp, _int, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    L.nsm_clip_grads.argtypes = [_vp, _vp, _vp, _int, _vp, _vp, _f32, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    L.nsm_grad_workspace_bytes.argtypes = [_vp, _int]
    L.nsm_grad_workspace_bytes.restype = ctypes.c_size_t
    for f in (L.nsm_logprobs, L.nsm_logprobs_grad, L.nsm_logprobs_backward, L.nsm_distill, L.nsm_distill_grad,
              L.nsm_distill_backward, L.nsm_adjust_logits, L.nsm_adjust_logits_backward, L.nsm_embedding,
              L.nsm_embedding_backward, L.nsm_grad_norm, L.nsm_clip_grads):
        f.restype = ctypes.c_int
    L.nsm_device_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_int)]
    L.nsm_device_status.restype = ctypes.c_int
    _ip = ctypes.POINTER(ctypes.c_int)
    L.nsm_device_status_detail.argtypes = [_vp, _ip, _ip, _ip, _ip]
    L.nsm_device_status_detail.restype = ctypes.c_int
    L.nsm_set_option.argtypes = [ctypes.c_int, ctypes.c_int]
    L.nsm_set_option.restype = ctypes.c_int
    L.nsm_get_option.argtypes = [ctypes.c_int]
    L.nsm_get_option.restype = ctypes.c_int
    L.nsm_status_selftest.argtypes = [ctypes.c_int, _vp]
    L.nsm_status_selftest.restype = ctypes.c_int
    L.nsm_bounds_selftest.argtypes = [_vp]
    L.nsm_bounds_selftest.restype = ctypes.c_int
    L.nsm_copy_to_device.argtypes = [_vp, _vp, ctypes.c_size_t, ctypes.c_int, _vp]
    L.nsm_copy_to_device.restype = ctypes.c_int
    L.nsm_timing_enable.argtypes = [ctypes.c_int]
    L.nsm_timing_read.argtypes = [ctypes.POINTER(ctypes.c_double), _c_i64p,
                                  ctypes.POINTER(ctypes.c_double)]
    L.nsm_timing_read_kind.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_double), _c_i64p,
                                       ctypes.POINTER(ctypes.c_double)]
    _lib = L
    return L


def _check(rc: int) -> int:
    if rc < 0:
        raise NsmError(rc, last_error())
    return rc


def last_error() -> str:
    return lib().nsm_last_error().decode("utf-8", "replace")


def version() -> int:
    return lib().nsm_version()


def last_launch_count() -> int:
    return lib().nsm_last_launch_count()


def route(name: str, ndim: int) -> bool:
    """Muon (True) or AdamW (False) for a named parameter of ``ndim`` dimensions."""
    return bool(_check(lib().nsm_route(name.encode("utf-8"), int(ndim))))


def input_exponent(max_abs: float, hint=None) -> Tuple[int, int, bool]:
    """(k, next hint, store again) of the stored input's exponent rule for a matrix whose
    largest |U| is ``max_abs`` (a float32 value), with the step's hint or without one."""
    k, nxt, store = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().nsm_input_exponent(float(max_abs), 0 if hint is None else 1, 0 if hint is None else int(hint),
                                    ctypes.byref(k), ctypes.byref(nxt), ctypes.byref(store)))
    return k.value, nxt.value, bool(store.value)


def _shapes_array(shapes: Sequence[Tuple[int, int]]) -> np.ndarray:
    arr = np.ascontiguousarray(np.asarray(shapes, dtype=np.int32).reshape(-1, 2))
    return arr


def _i32p(a: np.ndarray):
    return a.ctypes.data_as(_c_i32p)


def _i64p(a: np.ndarray):
    return a.ctypes.data_as(_c_i64p)


def pack(shapes: Sequence[Tuple[int, int]], align: int = 64) -> Tuple[np.ndarray, int]:
    """Offsets (int64 elements) and total length of the packed buffer for ``shapes``."""
    s = _shapes_array(shapes)
    n = s.shape[0]
    offs = np.zeros(n, dtype=np.int64)
    total = np.zeros(1, dtype=np.int64)
    _check(lib().nsm_pack(_i32p(s), n, int(align), _i64p(offs), _i64p(total)))
    return offs, int(total[0])


def assign_owners(shapes: Sequence[Tuple[int, int]], world: int, ns_method=NS_METHOD_DEFAULT,
                  ns_steps: int = NS_STEPS_DEFAULT) -> Tuple[np.ndarray, np.ndarray]:
    """Owner rank of every matrix (LPT on Newton-Schulz flops) and the flops per owner."""
    s = _shapes_array(shapes)
    owner = np.zeros(s.shape[0], dtype=np.int32)
    load = np.zeros(int(world), dtype=np.int64)
    _check(lib().nsm_assign_owners(_i32p(s), s.shape[0], int(world), method_code(ns_method),
                                   int(ns_steps), _i32p(owner), _i64p(load)))
    return owner, load


def owner_table(shapes: Sequence[Tuple[int, int]], owner: Sequence[int], rank: int,
                align: int = 64):
    """The packed table of one owner: (indices of its matrices, their shapes, offsets in its
    own packed buffer, that buffer's length)."""
    idx = [i for i, o in enumerate(owner) if int(o) == int(rank)]
    sub = [tuple(shapes[i]) for i in idx]
    if not sub:
        return idx, sub, np.zeros(0, dtype=np.int64), 0
    offs, total = pack(sub, align)
    return idx, sub, offs, total


# "Z2 与 Z3 模式" §每步通信字节数 and §显存开销: communication per step on a shard group of
# N ranks, in elements of the Muon-target parameters P_M, and the steady-state memory of
# the packed buffers.
DMUON_COMM_FACTORS = {"naive_z2": 3, "dmuon_z2": 2, "naive_z3": 4, "dmuon_z3": 3}


def dmuon_comm_elements(mode: str, world: int, p_m: float) -> float:
    """Elements each step moves on the shard group: k (N-1)/N P_M (k per mode)."""
    return DMUON_COMM_FACTORS[mode] * (world - 1) / world * p_m


def dmuon_packed_memory_elements(mode: str, world: int, p_m: float,
                                 max_layer_p_m: float = 0.0) -> float:
    """Steady-state elements of owned packed buffers per rank: P_M / N under Z2 (all
    resident), one layer's buffer (max_layer_P_M) under Z3."""
    if mode == "dmuon_z2":
        return p_m / world
    if mode == "dmuon_z3":
        return max_layer_p_m
    raise ValueError(mode)


def method_code(ns_method) -> int:
    if isinstance(ns_method, str):
        if ns_method not in NS_METHODS:
            raise ValueError(f"ns_method must be one of {sorted(NS_METHODS)}")
        return NS_METHODS[ns_method]
    return int(ns_method)


def workspace_bytes(shapes: Sequence[Tuple[int, int]], ns_method=NS_METHOD_DEFAULT,
                    ns_steps: int = NS_STEPS_DEFAULT) -> int:
    s = _shapes_array(shapes)
    b = lib().muon_workspace_bytes(_i32p(s), s.shape[0], method_code(ns_method), int(ns_steps))
    if b == 0:
        raise NsmError(NSM_ERR_ARG, last_error())
    return int(b)


def workspace_iterate(shapes: Sequence[Tuple[int, int]], i: int, buf: int, ns_method=NS_METHOD_DEFAULT,
                      ns_steps: int = NS_STEPS_DEFAULT) -> Tuple[int, int, int]:
    """(byte offset, m, row stride) of matrix i's m x m buffer `buf` in the workspace;
    m = 0 when its chain runs in the small-matrix kernel."""
    s = _shapes_array(shapes)
    off = ctypes.c_size_t(0)
    m = ctypes.c_int(0)
    ld = ctypes.c_int(0)
    _check(lib().nsm_workspace_iterate(_i32p(s), s.shape[0], method_code(ns_method), int(ns_steps), int(i),
                                       int(buf), ctypes.byref(off), ctypes.byref(m), ctypes.byref(ld)))
    return off.value, m.value, ld.value


def mm_buffers(ns_method=NS_METHOD_DEFAULT) -> int:
    """Number of m x m workspace buffers of a method (2 standard forms, 4 gram)."""
    return 4 if method_code(ns_method) == NS_METHODS["gram"] else 2


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream_ptr(stream) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def muon_step(grads, params, momentum, offsets, shapes, lr: float = MUON_LR_DEFAULT,
              wd: float = 0.0, mu: float = MUON_MOMENTUM_DEFAULT,
              ns_method=NS_METHOD_DEFAULT, ns_steps: int = NS_STEPS_DEFAULT,
              nesterov: bool = True, workspace=None, stream=None, params_bf16=None) -> None:
    """One owner-side Muon step on packed buffers (bf16 grads, fp32 params/momentum).

    With ``params_bf16`` (a bf16 buffer of the same length) the step also writes the bf16
    copy of the updated parameters, the buffer an owner broadcasts."""
    s = _shapes_array(shapes)
    o = np.ascontiguousarray(np.asarray(offsets, dtype=np.int64))
    ws_size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().muon_step_with_copy(_ptr(grads), _ptr(params), _ptr(momentum), _ptr(params_bf16),
                                     _i64p(o), _i32p(s), s.shape[0], float(lr), float(wd), float(mu),
                                     method_code(ns_method), int(ns_steps), 1 if nesterov else 0,
                                     _ptr(workspace), ws_size, _stream_ptr(stream)))


def muon_orthogonalize(inp, out, offsets, shapes, ns_method=NS_METHOD_DEFAULT,
                       ns_steps: int = NS_STEPS_DEFAULT, workspace=None, stream=None) -> None:
    """Newton-Schulz orthogonalisation of every matrix of a packed bf16 buffer."""
    s = _shapes_array(shapes)
    o = np.ascontiguousarray(np.asarray(offsets, dtype=np.int64))
    ws_size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().muon_orthogonalize(_ptr(inp), _ptr(out), _i64p(o), _i32p(s), s.shape[0],
                                    method_code(ns_method), int(ns_steps), _ptr(workspace),
                                    ws_size, _stream_ptr(stream)))


def muon_orthogonalize_noalloc(inp, out, offsets, shapes, ns_method=NS_METHOD_DEFAULT,
                               ns_steps: int = NS_STEPS_DEFAULT, stream=None) -> None:
    """muon_orthogonalize without a workspace, for callers that cannot allocate device
    memory (a framework pool that owns all of it, a loop that cannot take an allocation's
    synchronisation).  Uses a 64 MiB array of device memory the library itself holds;
    tables that do not fit raise NsmError(NSM_ERR_WORKSPACE).  Calls that overlap on the
    GPU race on that array: keep them on one stream."""
    s = _shapes_array(shapes)
    o = np.ascontiguousarray(np.asarray(offsets, dtype=np.int64))
    _check(lib().muon_orthogonalize_noalloc(_ptr(inp), _ptr(out), _i64p(o), _i32p(s), s.shape[0],
                                            method_code(ns_method), int(ns_steps),
                                            _stream_ptr(stream)))


def adamw_step(grads, params, exp_avg, exp_avg_sq, lr: float = ADAM_LR_DEFAULT,
               beta1: float = ADAM_BETAS_DEFAULT[0], beta2: float = ADAM_BETAS_DEFAULT[1],
               eps: float = ADAM_EPS_DEFAULT, wd: float = 0.0, step: int = 1,
               stream=None) -> None:
    """Fused AdamW on one flat group (bf16 grads, fp32 params and moments)."""
    numel = 0 if params is None else params.numel()
    _check(lib().adamw_step(_ptr(grads), _ptr(params), _ptr(exp_avg), _ptr(exp_avg_sq), numel,
                            float(lr), float(beta1), float(beta2), float(eps), float(wd),
                            int(step), _stream_ptr(stream)))


GEMM_SYMMETRIC = 1
GEMM_PAIR = 2


def gemm(a, b, out, aux=None, b_mn_major: bool = False, alpha: float = 1.0, beta: float = 0.0,
         diag: float = 0.0, symmetric: bool = False, pair: bool = False, scratch=None,
         stream=None) -> None:
    """out = alpha * a @ op(b) + beta * aux + diag * I on the tensor-core engine.

    ``a`` is M x K; ``b`` is N x K (op = transpose) or, with ``b_mn_major``, K x N.  All
    tensors are 2D bf16 or all fp16, with unit column stride.  ``symmetric`` declares the
    result symmetric: the upper triangle is computed and mirrored.  ``pair`` runs the 2-SM
    kernel (256 x 256 tiles on clusters of two CTAs)."""
    import torch
    M, K = a.shape
    N = b.shape[1] if b_mn_major else b.shape[0]
    fp16 = 1 if a.dtype == torch.float16 else 0
    flags = (GEMM_SYMMETRIC if symmetric else 0) | (GEMM_PAIR if pair else 0)
    if scratch is None:
        need = lib().nsm_gemm_scratch_bytes(M, N, flags)
        scratch = torch.empty(max(int(need), 1024), dtype=torch.uint8, device=a.device)
    _check(lib().nsm_gemm(_ptr(a), a.stride(0), _ptr(b), b.stride(0), _ptr(out), out.stride(0),
                          _ptr(aux), 0 if aux is None else aux.stride(0), M, N, K,
                          1 if b_mn_major else 0, fp16, flags, float(alpha), float(beta),
                          float(diag), _ptr(scratch), scratch.numel(), _stream_ptr(stream)))


# ---------------------------------------------------------------- losses over a vocabulary

TOP_MAX_K = 128
DISTILL_MAX_K = 128
_LOGITS_TYPES: dict = {}
_INDEX_TYPES: dict = {}
_WORD_TYPES: dict = {}
_FLOAT_TYPES: dict = {}
_FLOAT32 = _INT32 = None
_raw_stream = _current_device = _increment_version = None


def _torch_types() -> None:
    """torch's types as the library's codes, once torch is there."""
    global _FLOAT32, _INT32, _raw_stream, _current_device, _increment_version
    import torch
    _LOGITS_TYPES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    _INDEX_TYPES.update({torch.int32: 0, torch.int64: 1})
    _WORD_TYPES.update({torch.int32: 0})
    _FLOAT_TYPES.update({torch.float32: 2})
    _FLOAT32, _INT32 = torch.float32, torch.int32
    # what torch's public functions call: the current stream's handle without a Stream object is a
    # third of a short call's time, the other two save a fifth
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _increment_version = getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version


def _loss_stream(stream, device: int) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream_ptr(stream)


def _matrix(name: str, t, codes, rows: int, cols: int, device: int) -> Tuple[int, int, int]:
    """(pointer, type code, row stride) of a rows x cols tensor with unit column stride."""
    if t is None:
        raise ValueError(f"{name} is missing")
    code = codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} has type {t.dtype}: one of {[str(c) for c in codes]} is wanted")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}: ({rows}, {cols}) is wanted")
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} has column stride {step}: 1 is wanted")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on the logits' device")
    return t.data_ptr(), code, (ld if rows > 1 else max(ld, cols))


def _numbers(name: str, t, shape: Tuple[int, ...], device: int, dtype) -> int:
    """Pointer of a contiguous tensor of that shape and type; 0 for None."""
    if t is None:
        return 0
    if t.dtype != dtype:
        raise ValueError(f"{name} has type {t.dtype}: {dtype} is wanted")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} is not a contiguous tensor of shape {shape}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on the logits' device")
    return t.data_ptr()


def _written(*tensors) -> None:
    """Tells torch that these were written in place, so that a backward pass that saved one of
    them raises in place of using what is there now."""
    _increment_version([t for t in tensors if t is not None])


def _logits(logits) -> Tuple[int, int, int, int, int, int]:
    """(pointer, type code, rows, vocab, row stride, device)."""
    if _FLOAT32 is None:
        _torch_types()
    device = logits.get_device()  # -1: host memory
    shape = logits.shape
    if len(shape) != 2 or device < 0:
        raise ValueError("logits is not a matrix of rows x vocab in device memory")
    if device != _current_device():  # the kernels run there, whatever the logits' device is
        raise ValueError(f"logits is on {logits.device}, not on the current device")
    rows, vocab = shape
    code = _LOGITS_TYPES.get(logits.dtype)
    if code is None:
        raise ValueError(f"logits has type {logits.dtype}: one of {[str(c) for c in _LOGITS_TYPES]} is wanted")
    ld, step = logits.stride()
    if vocab > 1 and step != 1:
        raise ValueError(f"logits has column stride {step}: 1 is wanted")
    return logits.data_ptr(), code, rows, vocab, (ld if rows > 1 else max(ld, vocab)), device


def _tokens(tokens, rows: int, device: int) -> Tuple[int, int]:
    if tokens is None:
        return 0, 0
    code = _INDEX_TYPES.get(tokens.dtype)
    if code is None:
        raise ValueError(f"tokens has type {tokens.dtype}: torch.int32 or torch.int64 is wanted")
    return _numbers("tokens", tokens, (rows,), device, tokens.dtype), code


def _gradient(t, code: int, rows: int, vocab: int, device: int) -> Tuple[int, int]:
    ptr, own_code, ldd = _matrix("d_logits", t, _LOGITS_TYPES, rows, vocab, device)
    if own_code != code:
        raise ValueError(f"d_logits has type {t.dtype}: the logits' is wanted")
    return ptr, ldd


def _entries(teacher, index, rows: int, device: int) -> Tuple[int, int, int, int, int, int, int]:
    shape = () if teacher is None else teacher.shape
    if len(shape) != 2:
        raise ValueError("teacher is not a matrix of rows x k")
    k = shape[1]
    t_ptr, t_code, ldt = _matrix("teacher", teacher, _LOGITS_TYPES, rows, k, device)
    i_ptr, wide, ldi = _matrix("index", index, _INDEX_TYPES, rows, k, device)
    return t_ptr, t_code, ldt, i_ptr, wide, ldi, k


def logprobs(logits, tokens, logprob=None, entropy=None, lse=None, top_logprob=None, top_index=None,
             temperature: float = 1.0, stream=None) -> None:
    """Log probabilities of given tokens, with entropy and top alternatives.

    ``logits`` is rows x vocab (bf16, fp16 or fp32, unit column stride, any row stride);
    ``tokens`` one int32 or int64 index per row (an index outside the vocabulary, such as
    -100: no token) or None.  Writes the outputs that are given: ``logprob``, ``entropy``
    and ``lse`` (float32, one per row), and the k largest logits as log probabilities
    ``top_logprob`` (float32, rows x k) with their indexes ``top_index`` (int32, rows x k),
    ties by ascending index.  The tensors are on the current device, here and in the calls
    below."""
    ptr, code, rows, vocab, ld, dev = _logits(logits)
    row = (rows,)
    t_ptr, wide = _tokens(tokens, rows, dev)
    k = 0
    if top_logprob is not None or top_index is not None:
        shape = () if top_logprob is None or top_index is None else top_logprob.shape
        if len(shape) != 2:
            raise ValueError("top_logprob and top_index go together, as matrices of rows x k")
        k = shape[1]
        top_l = _numbers("top_logprob", top_logprob, (rows, k), dev, _FLOAT32)
        top_i = _numbers("top_index", top_index, (rows, k), dev, _INT32)
    else:
        top_l = top_i = 0
    _check(lib().nsm_logprobs(ptr, code, rows, vocab, ld, t_ptr, wide, float(temperature), k,
                              _numbers("logprob", logprob, row, dev, _FLOAT32), _numbers("entropy", entropy, row, dev, _FLOAT32),
                              _numbers("lse", lse, row, dev, _FLOAT32), top_l, top_i, _loss_stream(stream, dev)))
    _written(logprob, entropy, lse, top_logprob, top_index)


def logprobs_grad(logits, tokens, d_logprob, d_entropy, d_logits, logprob=None, entropy=None, lse=None,
                  temperature: float = 1.0, stream=None) -> None:
    """:func:`logprobs` with the gradient in the same pass, for weights known beforehand:
    writes ``d_logits``, the gradient of sum(d_logprob * logprob + d_entropy * entropy)
    (one of the two weights may be None), in the logits' type; it may be ``logits`` itself."""
    ptr, code, rows, vocab, ld, dev = _logits(logits)
    row = (rows,)
    t_ptr, wide = _tokens(tokens, rows, dev)
    g_ptr, ldd = _gradient(d_logits, code, rows, vocab, dev)
    _check(lib().nsm_logprobs_grad(ptr, code, rows, vocab, ld, t_ptr, wide, float(temperature),
                                   _numbers("d_logprob", d_logprob, row, dev, _FLOAT32),
                                   _numbers("d_entropy", d_entropy, row, dev, _FLOAT32), g_ptr, ldd,
                                   _numbers("logprob", logprob, row, dev, _FLOAT32),
                                   _numbers("entropy", entropy, row, dev, _FLOAT32), _numbers("lse", lse, row, dev, _FLOAT32),
                                   _loss_stream(stream, dev)))
    _written(d_logits, logprob, entropy, lse)


def logprobs_backward(logits, tokens, lse, entropy, d_logprob, d_entropy, d_logits, temperature: float = 1.0,
                      stream=None) -> None:
    """The backward pass of :func:`logprobs` alone, from its ``lse`` (and ``entropy``, needed
    with ``d_entropy``)."""
    ptr, code, rows, vocab, ld, dev = _logits(logits)
    row = (rows,)
    t_ptr, wide = _tokens(tokens, rows, dev)
    g_ptr, ldd = _gradient(d_logits, code, rows, vocab, dev)
    _check(lib().nsm_logprobs_backward(ptr, code, rows, vocab, ld, t_ptr, wide, float(temperature),
                                       _numbers("lse", lse, row, dev, _FLOAT32), _numbers("entropy", entropy, row, dev, _FLOAT32),
                                       _numbers("d_logprob", d_logprob, row, dev, _FLOAT32),
                                       _numbers("d_entropy", d_entropy, row, dev, _FLOAT32), g_ptr, ldd,
                                       _loss_stream(stream, dev)))
    _written(d_logits)


def distill(logits, teacher, index, loss, lse=None, rest=None, temperature: float = 1.0, tail: bool = False,
            stream=None) -> None:
    """Distillation from a teacher's top logits: per row, the divergence of the student's
    softmax from the teacher's k entries (``teacher`` scores, ``index`` int32 or int64).

    Without ``tail`` the teacher is the softmax over its entries at ``temperature``; with
    it ``teacher`` holds log probabilities at that temperature (``top_logprob`` of
    :func:`logprobs`) and the rest of the row is one bucket.  An index outside the
    vocabulary, or given before in its row, does not count.  Writes ``loss`` and, where
    given, the student's ``lse`` and ``rest`` (log of its mass outside the entries)."""
    ptr, code, rows, vocab, ld, dev = _logits(logits)
    row = (rows,)
    e = _entries(teacher, index, rows, dev)
    _check(lib().nsm_distill(ptr, code, rows, vocab, ld, *e, float(temperature), 1 if tail else 0,
                             _numbers("loss", loss, row, dev, _FLOAT32), _numbers("lse", lse, row, dev, _FLOAT32),
                             _numbers("rest", rest, row, dev, _FLOAT32), _loss_stream(stream, dev)))
    _written(loss, lse, rest)


def distill_grad(logits, teacher, index, d_loss, d_logits, loss=None, lse=None, rest=None,
                 temperature: float = 1.0, tail: bool = False, stream=None) -> None:
    """:func:`distill` with the gradient of sum(d_loss * loss) in the same pass (``d_loss``
    None: weights 1); ``d_logits`` has the logits' type and may be ``logits`` itself."""
    ptr, code, rows, vocab, ld, dev = _logits(logits)
    row = (rows,)
    e = _entries(teacher, index, rows, dev)
    g_ptr, ldd = _gradient(d_logits, code, rows, vocab, dev)
    _check(lib().nsm_distill_grad(ptr, code, rows, vocab, ld, *e, float(temperature), 1 if tail else 0,
                                  _numbers("d_loss", d_loss, row, dev, _FLOAT32), g_ptr, ldd,
                                  _numbers("loss", loss, row, dev, _FLOAT32), _numbers("lse", lse, row, dev, _FLOAT32),
                                  _numbers("rest", rest, row, dev, _FLOAT32), _loss_stream(stream, dev)))
    _written(d_logits, loss, lse, rest)


def distill_backward(logits, teacher, index, lse, rest, d_loss, d_logits, temperature: float = 1.0,
                     tail: bool = False, stream=None) -> None:
    """The backward pass of :func:`distill` alone, from its ``lse`` and (with ``tail``) ``rest``."""
    ptr, code, rows, vocab, ld, dev = _logits(logits)
    row = (rows,)
    e = _entries(teacher, index, rows, dev)
    g_ptr, ldd = _gradient(d_logits, code, rows, vocab, dev)
    _check(lib().nsm_distill_backward(ptr, code, rows, vocab, ld, *e, float(temperature), 1 if tail else 0,
                                      _numbers("lse", lse, row, dev, _FLOAT32), _numbers("rest", rest, row, dev, _FLOAT32),
                                      _numbers("d_loss", d_loss, row, dev, _FLOAT32), g_ptr, ldd, _loss_stream(stream, dev)))
    _written(d_logits)


# ---------------------------------------------------------------- penalties, biases and masks on logits

ADJUST_MAX_K = 1024


def _history(history, length, history_row, rows: int, device: int) -> Tuple[int, int, int, int, int, int, int]:
    if history is None:
        return 0, 0, 0, 0, 0, _numbers("length", length, (rows,), device, _INT32), \
            _numbers("history_row", history_row, (rows,), device, _INT32)
    shape = history.shape
    if len(shape) != 2:
        raise ValueError("history is not a matrix of tokens")
    ptr, wide, ld = _matrix("history", history, _INDEX_TYPES, shape[0], shape[1], device)
    return ptr, wide, shape[0], shape[1], ld, _numbers("length", length, (rows,), device, _INT32), \
        _numbers("history_row", history_row, (rows,), device, _INT32)


def _mask(mask, mask_row, rows: int, vocab: int, device: int) -> Tuple[int, int, int, int]:
    row = _numbers("mask_row", mask_row, (rows,), device, _INT32)
    if mask is None:
        return 0, 0, 0, row
    if len(mask.shape) != 2:
        raise ValueError("mask is not a matrix of words")
    ptr, _, ld = _matrix("mask", mask, _WORD_TYPES, mask.shape[0], (vocab + 31) // 32, device)
    return ptr, mask.shape[0], ld, row


def _logits_like(name: str, t, code: int, rows: int, vocab: int, device: int) -> Tuple[int, int, int]:
    """(pointer, type code, row stride) of a rows x vocab tensor of the logits' type or float32."""
    ptr, own_code, ld = _matrix(name, t, _LOGITS_TYPES, rows, vocab, device)
    if own_code != code and own_code != 2:
        raise ValueError(f"{name} has type {t.dtype}: the logits' or torch.float32 is wanted")
    return ptr, own_code, ld


def adjust_logits(logits, out, history=None, length=None, history_row=None, repetition=None, frequency=None,
                  presence=None, bias_index=None, bias=None, mask=None, mask_row=None, stream=None) -> None:
    """Penalties for repeated tokens, biases and a grammar's mask on rows of logits.

    ``out`` (rows x vocab, the logits' type or float32; it may be ``logits`` itself) receives
    each logit, where the row's history holds token v c times: x / ``repetition`` (x *
    ``repetition`` where x <= 0), less ``frequency`` * c + ``presence``; with the biases that
    ``bias_index`` gives for v added; and -inf where the row's mask has bit v clear, which is a
    masked token to :func:`logprobs` and the other losses.

    ``history`` (int32 or int64, history rows x tokens): row r's is the first ``length[r]``
    (int32, None: all) tokens of row ``history_row[r]`` (int32, None: r).  ``repetition``,
    ``frequency`` and ``presence`` are float32, one per row.  ``bias_index`` (int32 or int64) and
    ``bias`` (float32) are rows x k, k <= 1024.  All penalties count over the one history.  ``mask`` (int32, mask rows x ceil(vocab / 32)) has
    bit v % 32 of word v // 32 set where v is allowed; row r's is ``mask_row[r]`` (int32, None: r;
    -1: everything is allowed).  Indexes outside the vocabulary do not count."""
    ptr, code, rows, vocab, ld, dev = _logits(logits)
    row = (rows,)
    o_ptr, o_code, ldo = _logits_like("out", out, code, rows, vocab, dev)
    k, bi_ptr, b_wide, ldbi, b_ptr, ldb = 0, 0, 0, 0, 0, 0
    if bias_index is not None or bias is not None:
        shape = () if bias_index is None or bias is None else bias_index.shape
        if len(shape) != 2:
            raise ValueError("bias_index and bias go together, as matrices of rows x k")
        k = shape[1]
        bi_ptr, b_wide, ldbi = _matrix("bias_index", bias_index, _INDEX_TYPES, rows, k, dev)
        b_ptr, _, ldb = _matrix("bias", bias, _FLOAT_TYPES, rows, k, dev)
    _check(lib().nsm_adjust_logits(ptr, code, rows, vocab, ld, *_history(history, length, history_row, rows, dev),
                                   _numbers("repetition", repetition, row, dev, _FLOAT32),
                                   _numbers("frequency", frequency, row, dev, _FLOAT32),
                                   _numbers("presence", presence, row, dev, _FLOAT32), bi_ptr, b_wide, ldbi, b_ptr, ldb, k,
                                   *_mask(mask, mask_row, rows, vocab, dev), o_ptr, o_code, ldo, _loss_stream(stream, dev)))
    _written(out)


def adjust_logits_backward(logits, d_out, d_logits, history=None, length=None, history_row=None, repetition=None,
                           mask=None, mask_row=None, stream=None) -> None:
    """The backward pass of :func:`adjust_logits`: writes ``d_logits`` (the logits' type) from
    ``d_out`` (that type or float32; of the logits' type it may be ``d_logits`` itself).  ``logits``
    are the forward call's input, as they were before it; only ``repetition`` needs them, and
    without it they may be None.  Frequency, presence and biases change no gradient."""
    if logits is None and repetition is not None:
        raise ValueError("repetition needs the logits")
    like = d_logits if logits is None else logits
    ptr, code, rows, vocab, ld, dev = _logits(like)
    g_ptr, ldd = _gradient(d_logits, code, rows, vocab, dev)
    o_ptr, o_code, ldo = _logits_like("d_out", d_out, code, rows, vocab, dev)
    _check(lib().nsm_adjust_logits_backward(0 if logits is None else ptr, code, rows, vocab, ld,
                                            *_history(history, length, history_row, rows, dev),
                                            _numbers("repetition", repetition, (rows,), dev, _FLOAT32),
                                            *_mask(mask, mask_row, rows, vocab, dev), o_ptr, o_code, ldo, g_ptr, ldd,
                                            _loss_stream(stream, dev)))
    _written(d_logits)


# ---------------------------------------------------------------- the embedding lookup and its gradient


def _rows_of(name: str, t) -> Tuple[int, int, int, int, int, int]:
    """(pointer, type code, rows, columns, row stride, device) of a matrix on the current device."""
    if _FLOAT32 is None:
        _torch_types()
    device = t.get_device()
    shape = t.shape
    if len(shape) != 2 or device < 0:
        raise ValueError(f"{name} is not a matrix in device memory")
    if device != _current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    ptr, code, ld = _matrix(name, t, _LOGITS_TYPES, shape[0], shape[1], device)
    return ptr, code, shape[0], shape[1], ld, device


def embedding(weight, tokens, out, scale: float = 1.0, stream=None) -> None:
    """out[r] = scale * weight[tokens[r]], zeros where the token (int32 or int64) is outside the
    vocabulary.  ``weight`` (vocab x cols) and ``out`` (rows x cols) have any of the three types
    each: an optimizer's fp32 master weights can give bf16 activations."""
    w_ptr, w_code, vocab, cols, ldw, dev = _rows_of("weight", weight)
    rows = len(tokens)
    t_ptr, wide = _tokens(tokens, rows, dev)
    o_ptr, o_code, ldo = _matrix("out", out, _LOGITS_TYPES, rows, cols, dev)
    _check(lib().nsm_embedding(w_ptr, w_code, vocab, cols, ldw, t_ptr, wide, rows, float(scale), o_ptr, o_code, ldo,
                               _loss_stream(stream, dev)))
    _written(out)


def embedding_workspace_bytes(rows: int, vocab: int, cols: int) -> int:
    """Bytes of :func:`embedding_backward`'s workspace; one for the largest batch serves smaller ones."""
    b = lib().nsm_embedding_workspace_bytes(int(rows), int(vocab), int(cols))
    if b == 0:
        raise NsmError(NSM_ERR_SHAPE, last_error())
    return int(b)


def embedding_backward(d_out, tokens, d_weight, workspace, scale: float = 1.0, accumulate: bool = False,
                       stream=None) -> None:
    """The gradient of :func:`embedding`: d_weight[v] = scale * the sum of d_out's rows of token
    v, zeros in rows without one; with ``accumulate`` the sums are added to what ``d_weight``
    holds (a weight that is the output layer's too).  ``d_weight`` and ``d_out`` have any of the
    three types each; ``MuonAdamW.grad(name)`` is such a ``d_weight``.  The order of every sum is set
    by the sizes and the tokens."""
    w_ptr, w_code, vocab, cols, ldw, dev = _rows_of("d_weight", d_weight)
    rows = len(tokens)
    t_ptr, wide = _tokens(tokens, rows, dev)
    g_ptr, g_code, ldg = _matrix("d_out", d_out, _LOGITS_TYPES, rows, cols, dev)
    ws_ptr, ws_size = _workspace(workspace, dev)
    _check(lib().nsm_embedding_backward(g_ptr, g_code, rows, cols, ldg, t_ptr, wide, vocab, float(scale),
                                        1 if accumulate else 0, w_ptr, w_code, ldw, ws_ptr, ws_size,
                                        _loss_stream(stream, dev)))
    _written(d_weight)


def _workspace(workspace, device: int) -> Tuple[int, int]:
    """(pointer, bytes) of a contiguous tensor of any type."""
    if workspace is None:
        return 0, 0
    if workspace.get_device() != device:
        raise ValueError(f"workspace is on {workspace.device}, not on the current device")
    if not workspace.is_contiguous():
        raise ValueError("workspace is not contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------- the norm of many gradients, and clipping

class GradTable:
    """The places of many gradients and, for :func:`clip_grads`, of where the clipped ones go
    (``out``, None: in place).  A program whose gradients stay where they are keeps one from step to
    step; it holds the tensors, and the places that their memory had when it was made: one whose
    memory is changed (``.data``, ``set_``) wants a new table.  Each is contiguous, bf16, fp16 or fp32,
    all on one device."""

    def __init__(self, grads: Sequence, out: Optional[Sequence] = None):
        if _FLOAT32 is None:
            _torch_types()
        self.grads = list(grads)
        self.out = None if out is None else list(out)
        n = len(self.grads)
        if n == 0:
            raise ValueError("no gradients are given")
        if self.out is not None and len(self.out) != n:
            raise ValueError(f"{n} gradients and {len(self.out)} places for them")
        self.device = self.grads[0].get_device()
        self.numels = np.zeros(n, dtype=np.int64)
        self._places, self._types = self._table("gradient", self.grads)
        for i, t in enumerate(self.grads):
            self.numels[i] = t.numel()
        self._out_places = self._out_types = None
        if self.out is not None:
            self._out_places, self._out_types = self._table("out", self.out)
            for i, t in enumerate(self.out):
                if t.numel() != self.numels[i]:
                    raise ValueError(f"out {i} has {t.numel()} elements, its gradient {self.numels[i]}")
        b = lib().nsm_grad_workspace_bytes(self.numels.ctypes.data, n)
        if b == 0:
            raise NsmError(NSM_ERR_SHAPE, last_error())
        self.workspace_bytes = int(b)
        # for the calls: arrays as the library takes them
        self._in_args = (self._places.ctypes.data, self.numels.ctypes.data, self._types.ctypes.data, n)
        self._out_args = (0, 0) if self.out is None else (self._out_places.ctypes.data, self._out_types.ctypes.data)

    def __len__(self) -> int:
        return len(self.grads)

    def _table(self, name: str, tensors) -> Tuple[np.ndarray, np.ndarray]:
        places = np.zeros(len(tensors), dtype=np.uint64)
        types = np.zeros(len(tensors), dtype=np.int32)
        for i, t in enumerate(tensors):
            code = _LOGITS_TYPES.get(t.dtype)
            if code is None:
                raise ValueError(f"{name} {i} has type {t.dtype}: one of {[str(c) for c in _LOGITS_TYPES]} is wanted")
            device = t.get_device()
            if device < 0 or device != self.device:
                raise ValueError(f"{name} {i} is on {t.device}: all are wanted on one device")
            if not t.is_contiguous():
                raise ValueError(f"{name} {i} is not contiguous")
            places[i], types[i] = t.data_ptr(), code
        return places, types

    def _checked(self, norm, norms, workspace, stream):
        """What both calls check; (norm, norms, workspace, its bytes, stream) as the library takes them."""
        device = self.device
        if device != _current_device():
            raise ValueError("the gradients are not on the current device")
        if norm is not None and norm.shape != ():
            norm_ptr = _numbers("norm", norm, (1,), device, _FLOAT32)
        else:
            norm_ptr = _numbers("norm", norm, (), device, _FLOAT32)
        norms_ptr = _numbers("norms", norms, (len(self.grads),), device, _FLOAT32)
        return (norm_ptr, norms_ptr, *_workspace(workspace, device), _loss_stream(stream, device))


def grad_norm(grads, norm, norms=None, workspace=None, stream=None) -> None:
    """Writes the norm of all gradients together to ``norm`` (float32, one element) and each
    one's to ``norms`` (float32, one per gradient, or None).  ``grads`` is a :class:`GradTable` or a
    list of tensors; ``workspace``, which the call cannot do without, has the table's
    ``workspace_bytes``."""
    table = grads if isinstance(grads, GradTable) else GradTable(grads)
    _check(lib().nsm_grad_norm(*table._in_args, *table._checked(norm, norms, workspace, stream)))
    _written(norm, norms)


def clip_grads(grads, max_norm: float, norm=None, norms=None, workspace=None, stream=None) -> None:
    """Scales the gradients by min(1, max_norm / norm), in place or to the table's ``out``
    (converted to its types), and writes the norms before clipping as :func:`grad_norm` does, with
    the same ``workspace``.  An infinity or a NaN in some gradient leaves all as they are; finite ones
    whose norm is past float32's range (written as infinity) are clipped."""
    table = grads if isinstance(grads, GradTable) else GradTable(grads)
    _check(lib().nsm_clip_grads(*table._in_args, *table._out_args, float(max_norm),
                                *table._checked(norm, norms, workspace, stream)))
    _written(norm, norms, *(table.grads if table.out is None else table.out))


def device_status(stream=None) -> int:
    """Synchronises the stream; returns NSM_OK, NSM_ERR_TIMEOUT or (checked build)
    NSM_ERR_BOUNDS, and clears the record."""
    v = ctypes.c_int(0)
    _check(lib().nsm_device_status(_stream_ptr(stream), ctypes.byref(v)))
    return v.value


def device_status_detail(stream=None) -> Tuple[int, int, int, int]:
    """Synchronises the stream; returns (status, kernel, role, site) of the first bounded
    wait that expired, or (checked build) bounds test that failed, since the last read
    (status NSM_OK and zeros when none), and clears the record.  kernel/role/site are the
    NSM_KERNEL_* / NSM_ROLE_* / NSM_SITE_* codes of the C header."""
    v = [ctypes.c_int(0) for _ in range(4)]
    _check(lib().nsm_device_status_detail(_stream_ptr(stream), *[ctypes.byref(x) for x in v]))
    return tuple(x.value for x in v)


NSM_KERNEL_GEMM, NSM_KERNEL_GEMM_PAIR, NSM_KERNEL_SMALL, NSM_KERNEL_SELFTEST = 1, 2, 3, 4
NSM_SITE_SELFTEST = 11
NSM_SITE_SELFTEST_BOUNDS = 23

OPT_PAIR_KERNELS, OPT_SMALL_KERNEL, OPT_PDL, OPT_BOUNDS_CHECKS, OPT_SYM_STORAGE = 1, 2, 3, 4, 5


def set_option(option: int, value: int) -> None:
    """Process-wide choice between the library's equivalent paths (for comparisons):
    OPT_PAIR_KERNELS, OPT_SMALL_KERNEL, OPT_SYM_STORAGE (default 1: symmetric iterates
    kept as their upper 256 x 256 tiles where every launch is on the 2-SM kernel) and
    OPT_PDL (0 off, 1 on, default 2: on for tables of at most 2^25 elements)."""
    _check(lib().nsm_set_option(int(option), int(value)))


def get_option(option: int) -> int:
    return _check(lib().nsm_get_option(int(option)))


def status_selftest(wait_us: int = 20000, stream=None) -> None:
    """Launches one CTA whose bounded wait expires after wait_us and records a timeout in
    the device status word (read it with device_status)."""
    _check(lib().nsm_status_selftest(int(wait_us), _stream_ptr(stream)))


def bounds_selftest(stream=None) -> None:
    """Launches one thread that runs the kernels' bounds test on an index past its range
    and makes no access: the checked build records NSM_ERR_BOUNDS (read it with
    device_status_detail), the regular build nothing."""
    _check(lib().nsm_bounds_selftest(_stream_ptr(stream)))


def copy_to_device(dst, src, stream=None, ctas: int = 0) -> None:
    """dst (device tensor) <- src (pinned host tensor of the same byte size) by SM loads
    over the host link (nsm_copy_to_device); asynchronous on `stream`."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("dst and src differ in size")
    _check(lib().nsm_copy_to_device(_ptr(dst), _ptr(src), nbytes, int(ctas), _stream_ptr(stream)))


def checked_build() -> bool:
    """Whether the loaded library is the bounds-checked build."""
    return get_option(OPT_BOUNDS_CHECKS) == 1


def timing_enable(on: bool = True) -> None:
    lib().nsm_timing_enable(1 if on else 0)


def timing_reset() -> None:
    lib().nsm_timing_reset()


KIND_GEMM, KIND_MOMENTUM, KIND_NORM, KIND_LAYOUT, KIND_APPLY, KIND_ADAMW, KIND_SMALL, KIND_GRAD_NORM, \
    KIND_LOGPROBS, KIND_DISTILL = range(10)
KIND_ADJUST, KIND_EMBEDDING, KIND_GRADS = 11, 12, 13
KIND_NAMES = {KIND_GEMM: "k_ns_gemm", KIND_MOMENTUM: "k_momentum_class", KIND_NORM: "k_scale_finalize",
              KIND_LAYOUT: "k_to_class", KIND_APPLY: "k_from_class", KIND_ADAMW: "k_adamw",
              KIND_SMALL: "k_ns_small", KIND_GRAD_NORM: "k_grad_norm",
              KIND_LOGPROBS: "k_logprobs", KIND_DISTILL: "k_distill", KIND_ADJUST: "k_adjust",
              KIND_EMBEDDING: "k_embed", KIND_GRADS: "k_grad_clip"}


def timing_read(kind: int = KIND_GEMM) -> Tuple[float, int, float]:
    """(device ms, launches, algorithmic work) of one kernel kind since the last reset."""
    ms = ctypes.c_double(0)
    n = ctypes.c_int64(0)
    w = ctypes.c_double(0)
    _check(lib().nsm_timing_read_kind(int(kind), ctypes.byref(ms), ctypes.byref(n), ctypes.byref(w)))
    return ms.value, n.value, w.value


# ---------------------------------------------------------------- optimizer wrapper

class MuonAdamW:
    """Hybrid optimizer state over named parameters, on one GPU.

    Parameters tagged by :func:`route` go to one packed Muon group (fp32 master params,
    fp32 momentum, a bf16 gradient buffer); the rest go to one flat AdamW group (fp32
    master params and moments, bf16 gradients).  The config keys mirror the pages:
    ``muon_lr`` / ``adam_lr`` override ``lr``, ``momentum``, ``weight_decay``, ``betas``,
    ``eps`` and ``ns_method``.  The optimizer owns the fp32 master weights: callers write
    initial weights and each step's gradients through :meth:`param` / :meth:`grad`, and
    :meth:`state_dict` carries the master weights with the moments, so that a checkpoint
    restores the whole state.
    """

    def __init__(self, named_shapes: Iterable[Tuple[str, Tuple[int, ...]]], device="cuda",
                 lr: Optional[float] = None, muon_lr: Optional[float] = None,
                 adam_lr: Optional[float] = None, momentum: float = MUON_MOMENTUM_DEFAULT,
                 weight_decay: float = 0.0, betas=ADAM_BETAS_DEFAULT,
                 eps: float = ADAM_EPS_DEFAULT, ns_method: str = NS_METHOD_DEFAULT,
                 ns_steps: int = NS_STEPS_DEFAULT, nesterov: bool = True):
        import torch
        named = list(named_shapes)
        self.muon_names: List[str] = []
        self.muon_shapes: List[Tuple[int, int]] = []
        self.adam_names: List[str] = []
        self.adam_sizes: List[int] = []
        self._shape_of: Dict[str, Tuple[int, ...]] = {}
        for name, shape in named:
            shape = tuple(int(d) for d in shape)
            if name in self._shape_of:
                raise ValueError(f"parameter {name!r} is listed twice")
            self._shape_of[name] = shape
            if route(name, len(shape)):
                cols = 1
                for d in shape[1:]:
                    cols *= d
                self.muon_names.append(name)
                self.muon_shapes.append((shape[0], cols))
            else:
                size = 1
                for d in shape:
                    size *= d
                self.adam_names.append(name)
                self.adam_sizes.append(size)
        base_lr = lr
        self.muon_lr = muon_lr if muon_lr is not None else (base_lr if base_lr is not None else MUON_LR_DEFAULT)
        self.adam_lr = adam_lr if adam_lr is not None else (base_lr if base_lr is not None else ADAM_LR_DEFAULT)
        self.momentum = momentum
        self.weight_decay = weight_decay
        self.betas = tuple(betas)
        self.eps = eps
        self.ns_method = ns_method
        self.ns_steps = ns_steps
        self.nesterov = nesterov
        self.step_count = 0
        dev = torch.device(device)
        self._muon_index = {n: i for i, n in enumerate(self.muon_names)}
        self._adam_offset: Dict[str, int] = {}
        off = 0
        for n, size in zip(self.adam_names, self.adam_sizes):
            self._adam_offset[n] = off
            off += size
        if self.muon_shapes:
            self.offsets, total = pack(self.muon_shapes)
            self.muon_params = torch.zeros(total, dtype=torch.float32, device=dev)
            self.muon_momentum = torch.zeros(total, dtype=torch.float32, device=dev)
            self.muon_grads = torch.zeros(total, dtype=torch.bfloat16, device=dev)
            self.workspace = torch.empty(workspace_bytes(self.muon_shapes, ns_method, ns_steps),
                                         dtype=torch.uint8, device=dev)
            # the step's exponents (its first 4 bytes per matrix): none yet, where whatever the memory held
            # could be taken for one and change the last bits of the first step
            self._exponents().fill_(EXPONENT_NONE)
        n_adam = sum(self.adam_sizes)
        self.adam_params = torch.zeros(n_adam, dtype=torch.float32, device=dev)
        self.adam_exp_avg = torch.zeros(n_adam, dtype=torch.float32, device=dev)
        self.adam_exp_avg_sq = torch.zeros(n_adam, dtype=torch.float32, device=dev)
        self.adam_grads = torch.zeros(n_adam, dtype=torch.bfloat16, device=dev)
        # clip's outputs and workspace: made here, so that a first clip on a stream of its own finds them ready
        self._clip = None  # the slots' table, made by the first clip
        numels = np.array([m * n for m, n in self.muon_shapes] + self.adam_sizes, dtype=np.int64)
        self._clip_norm = torch.zeros(1, dtype=torch.float32, device=dev)
        self.grad_norms = torch.zeros(len(numels), dtype=torch.float32, device=dev)
        self._clip_workspace = torch.empty(lib().nsm_grad_workspace_bytes(numels.ctypes.data, len(numels)),
                                           dtype=torch.uint8, device=dev)

    def _exponents(self):
        """The exponents that the step keeps in its workspace, one int32 per Muon matrix."""
        import torch
        return self.workspace[:4 * len(self.muon_shapes)].view(torch.int32)

    def _view(self, name: str, muon_buf, adam_buf):
        shape = self._shape_of[name]
        if name in self._muon_index:
            i = self._muon_index[name]
            r, c = self.muon_shapes[i]
            o = int(self.offsets[i])
            return muon_buf[o:o + r * c].view(shape)
        o = self._adam_offset[name]
        size = 1
        for d in shape:
            size *= d
        return adam_buf[o:o + size].view(shape)

    def param(self, name: str):
        """The fp32 master weight of a parameter (a view into its group's buffer)."""
        return self._view(name, getattr(self, "muon_params", None), self.adam_params)

    def grad(self, name: str):
        """The bf16 gradient slot of a parameter (a view; write each step's gradient here)."""
        return self._view(name, getattr(self, "muon_grads", None), self.adam_grads)

    def clip(self, max_norm: float, grads=None, stream=None):
        """Scales all gradient slots together by min(1, max_norm / their norm); with ``grads`` (a
        mapping of every parameter's name to its gradient, bf16, fp16 or fp32) those are clipped
        into the slots, which takes the place of copying them there.  Returns the norm before
        clipping (float32, one element on the device, the same tensor at every call);
        ``grad_norms`` then holds each parameter's, Muon's first, in the order of
        ``muon_names`` and ``adam_names``.  The norm is that of this optimizer's parameters: one owner
        among several clips by its own."""
        names = self.muon_names + self.adam_names
        if not names:  # an owner that got none: its norm stays 0
            if grads:
                raise ValueError("grads names parameters, and the optimizer has none")
            if not 0.0 < max_norm < float("inf"):
                raise NsmError(NSM_ERR_ARG, "max_norm must be positive and finite")
            return self._clip_norm
        places = [b.data_ptr() for b in (getattr(self, "muon_grads", None), self.adam_grads) if b is not None]
        if self._clip is None or self._clip[2] != places:  # its views hold the memory that its places are in
            slots = [self.grad(n) for n in names]
            self._clip = (slots, GradTable(slots), places)
        slots, table, _ = self._clip
        if grads is not None:
            lacking = [n for n in names if grads.get(n) is None]
            if lacking or len(grads) != len(names):
                raise ValueError(f"grads names other parameters than the optimizer's (without {lacking})")
            for n in names:
                if tuple(grads[n].shape) != self._shape_of[n]:
                    raise ValueError(f"the gradient of {n!r} has shape {tuple(grads[n].shape)}: {self._shape_of[n]} is wanted")
            table = GradTable([grads[n] for n in names], slots)
        clip_grads(table, max_norm, self._clip_norm, self.grad_norms, workspace=self._clip_workspace, stream=stream)
        return self._clip_norm

    def step(self, stream=None, max_norm: Optional[float] = None) -> None:
        """One step of both groups on the slots' gradients, clipped to ``max_norm`` together
        first where it is given."""
        if max_norm is not None:
            self.clip(max_norm, stream=stream)
        self.step_count += 1
        if self.muon_shapes:
            muon_step(self.muon_grads, self.muon_params, self.muon_momentum, self.offsets,
                      self.muon_shapes, self.muon_lr, self.weight_decay, self.momentum,
                      self.ns_method, self.ns_steps, self.nesterov, self.workspace, stream)
        if self.adam_params.numel():
            adamw_step(self.adam_grads, self.adam_params, self.adam_exp_avg, self.adam_exp_avg_sq,
                       self.adam_lr, self.betas[0], self.betas[1], self.eps, self.weight_decay,
                       self.step_count, stream)

    def state_dict(self) -> Dict[str, object]:
        """The whole optimizer state as plain tensors (the caller saves and restores them):
        the step count, both groups' fp32 master weights, the Muon momentum and the AdamW
        moments, with the names and shapes they were packed from, and the exponents that the
        next step stores its input with (a copy of their own, made on the current stream: a view
        would save the whole workspace with them)."""
        d: Dict[str, object] = {"step": self.step_count,
                                "muon_names": list(self.muon_names),
                                "muon_shapes": list(self.muon_shapes),
                                "adam_names": list(self.adam_names),
                                "adam_sizes": list(self.adam_sizes),
                                "adam_params": self.adam_params,
                                "adam_exp_avg": self.adam_exp_avg,
                                "adam_exp_avg_sq": self.adam_exp_avg_sq}
        if self.muon_shapes:
            d["muon_params"] = self.muon_params
            d["muon_momentum"] = self.muon_momentum
            d["muon_exponents"] = self._exponents().clone()
        return d

    def load_state_dict(self, d: Dict[str, object]) -> None:
        if (list(d["muon_names"]) != self.muon_names or list(d["adam_names"]) != self.adam_names
                or [tuple(s) for s in d["muon_shapes"]] != self.muon_shapes
                or list(d["adam_sizes"]) != self.adam_sizes):
            raise ValueError("state_dict was saved for other parameters")
        self.step_count = int(d["step"])
        self.adam_params.copy_(d["adam_params"])
        self.adam_exp_avg.copy_(d["adam_exp_avg"])
        self.adam_exp_avg_sq.copy_(d["adam_exp_avg_sq"])
        if self.muon_shapes:
            self.muon_params.copy_(d["muon_params"])
            self.muon_momentum.copy_(d["muon_momentum"])
            if d.get("muon_exponents") is None:  # a checkpoint from before they were carried
                self._exponents().fill_(EXPONENT_NONE)
            else:
                self._exponents().copy_(d["muon_exponents"])
