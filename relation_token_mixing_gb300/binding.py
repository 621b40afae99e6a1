"""Thin Python binding of the Relation C ABI (include/relation.h).

The functions named like the C entry points (``relation_fwd``,
``relation_bwd``, ...) marshal torch CUDA tensors into pointers and call the
library; every step of the computation runs in the library's CUDA kernels.
PyTorch provides device memory and streams only.  There is no fallback: if the
library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import torch

from . import build as _build

RELATION_F32 = 0
RELATION_BF16 = 1
RELATION_LAYOUT_BHTD = 0  # operands [B, H, T, d_h]
RELATION_LAYOUT_BTHD = 1  # operands [B, T, H, d_h]

STATUS = {
    0: "RELATION_OK",
    1: "RELATION_ERR_INVALID_ARGUMENT",
    2: "RELATION_ERR_UNSUPPORTED",
    3: "RELATION_ERR_MISALIGNED",
    4: "RELATION_ERR_WORKSPACE_TOO_SMALL",
    5: "RELATION_ERR_CUDA",
    6: "RELATION_ERR_DEVICE_TIMEOUT",
    7: "RELATION_ERR_DEVICE_UNSAFE",
}


class RelationError(RuntimeError):
    def __init__(self, code: int, what: str, message: str):
        super().__init__(f"{what}: {STATUS.get(code, code)} ({message})")
        self.code = code


class Problem(ctypes.Structure):
    """Mirror of relation_problem_t."""

    _fields_ = [
        ("B", ctypes.c_int64),
        ("H", ctypes.c_int64),
        ("T", ctypes.c_int64),
        ("d_h", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("tau_S", ctypes.c_float),
        ("lam", ctypes.c_float),
        ("causal", ctypes.c_int32),
        ("layout", ctypes.c_int32),
    ]


class Paged(ctypes.Structure):
    """Mirror of relation_paged_t."""

    _fields_ = [
        ("R", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("H", ctypes.c_int64),
        ("G", ctypes.c_int64),
        ("d_h", ctypes.c_int64),
        ("pages", ctypes.c_int64),
        ("page_size", ctypes.c_int64),
        ("table_width", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("tau_S", ctypes.c_float),
        ("lam", ctypes.c_float),
        ("layout", ctypes.c_int32),
    ]


class LinearPacked(ctypes.Structure):
    """Mirror of relation_linear_packed_t."""

    _fields_ = [
        ("R", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("H", ctypes.c_int64),
        ("d_h", ctypes.c_int64),
        ("states", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("tau_S", ctypes.c_float),
    ]


_lock = threading.Lock()
_lib = None

_VP = ctypes.c_void_p
_BWD_ARGTYPES = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Loads the in-tree library (building it first when missing or stale)."""
    global _lib
    if _lib is not None:  # set once, when every entry point has its types
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if build_if_missing and not _build.up_to_date():
            _build.build()
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"Relation CUDA library not built at {_build.LIB}")
        lib = ctypes.CDLL(_build.LIB)
        lib.relation_fwd.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, _VP]
        lib.relation_fwd.restype = ctypes.c_int
        lib.relation_fwd_workspace_bytes.argtypes = [ctypes.POINTER(Problem)]
        lib.relation_fwd_workspace_bytes.restype = ctypes.c_size_t
        lib.relation_fwd_ws.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]
        lib.relation_fwd_ws.restype = ctypes.c_int
        for name in ("relation_bwd", "relation_bwd_prepare", "relation_bwd_main", "relation_bwd_finish"):
            getattr(lib, name).argtypes = _BWD_ARGTYPES
            getattr(lib, name).restype = ctypes.c_int
        lib.relation_bwd_noalloc.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                             _VP]
        lib.relation_bwd_noalloc.restype = ctypes.c_int
        lib.relation_step_host_device_bytes.argtypes = [ctypes.POINTER(Problem), ctypes.c_int]
        lib.relation_step_host_device_bytes.restype = ctypes.c_size_t
        lib.relation_step_host.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                           ctypes.c_int, _VP, ctypes.c_size_t, _VP]
        lib.relation_step_host.restype = ctypes.c_int
        lib.relation_bwd_workspace_bytes.argtypes = [ctypes.POINTER(Problem)]
        lib.relation_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.relation_prologue_fwd.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, ctypes.c_int,
                                              ctypes.c_float, _VP, _VP, _VP, _VP, _VP]
        lib.relation_prologue_fwd.restype = ctypes.c_int
        lib.relation_prologue_bwd.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, ctypes.c_int,
                                              ctypes.c_float, _VP, _VP, _VP, _VP, _VP, _VP]
        lib.relation_prologue_bwd.restype = ctypes.c_int
        lib.relation_fwd_prologue.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, ctypes.c_int,
                                              ctypes.c_float, _VP, _VP, _VP, _VP]
        lib.relation_fwd_prologue.restype = ctypes.c_int
        lib.relation_bwd_prologue_workspace_bytes.argtypes = [ctypes.POINTER(Problem)]
        lib.relation_bwd_prologue_workspace_bytes.restype = ctypes.c_size_t
        lib.relation_bwd_prologue.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, ctypes.c_int,
                                              ctypes.c_float, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                              ctypes.c_size_t, _VP]
        lib.relation_bwd_prologue.restype = ctypes.c_int
        lib.relation_linear_fwd_gate.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                                 _VP, ctypes.c_size_t, _VP]
        lib.relation_linear_fwd_gate.restype = ctypes.c_int
        lib.relation_linear_bwd_gate.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                                 _VP, _VP, _VP, _VP, _VP, ctypes.c_int, _VP, ctypes.c_size_t, _VP]
        lib.relation_linear_bwd_gate.restype = ctypes.c_int
        lib.relation_decode_workspace_bytes.argtypes = [ctypes.POINTER(Problem)]
        lib.relation_decode_workspace_bytes.restype = ctypes.c_size_t
        lib.relation_decode.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP,
                                        _VP, ctypes.c_size_t, _VP]
        lib.relation_decode.restype = ctypes.c_int
        lib.relation_linear_workspace_bytes.argtypes = [ctypes.POINTER(Problem)]
        lib.relation_linear_workspace_bytes.restype = ctypes.c_size_t
        lib.relation_linear_fwd.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                            ctypes.c_size_t, _VP]
        lib.relation_linear_fwd.restype = ctypes.c_int
        lib.relation_linear_bwd.argtypes = [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                            ctypes.c_int, _VP, ctypes.c_size_t, _VP]
        lib.relation_linear_bwd.restype = ctypes.c_int
        _LP = ctypes.POINTER(LinearPacked)
        lib.relation_linear_step.argtypes = [_LP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]
        lib.relation_linear_step.restype = ctypes.c_int
        lib.relation_linear_packed_workspace_bytes.argtypes = [_LP, ctypes.c_int]
        lib.relation_linear_packed_workspace_bytes.restype = ctypes.c_size_t
        lib.relation_linear_packed_fwd.argtypes = [_LP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP,
                                                   _VP, _VP, ctypes.c_size_t, _VP]
        lib.relation_linear_packed_fwd.restype = ctypes.c_int
        _PP = ctypes.POINTER(Paged)
        lib.relation_paged_plan.argtypes = [_PP, _VP, _VP, _VP, ctypes.c_size_t, _VP, _VP, _VP, _VP, _VP, _VP]
        lib.relation_paged_plan.restype = ctypes.c_int
        lib.relation_paged_store.argtypes = [_PP, _VP, _VP, _VP, _VP, ctypes.c_int, ctypes.c_float, _VP, _VP, _VP, _VP,
                                             _VP, _VP]
        lib.relation_paged_store.restype = ctypes.c_int
        lib.relation_paged_workspace_bytes.argtypes = [_PP, ctypes.c_int]
        lib.relation_paged_workspace_bytes.restype = ctypes.c_size_t
        lib.relation_paged_fwd.argtypes = [_PP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP,
                                           ctypes.c_size_t, _VP]
        lib.relation_paged_fwd.restype = ctypes.c_int
        lib.relation_paged_store_q8.argtypes = [_PP, _VP, _VP, _VP, _VP, ctypes.c_int, ctypes.c_float, _VP, _VP, _VP, _VP,
                                                _VP, _VP, _VP]
        lib.relation_paged_store_q8.restype = ctypes.c_int
        lib.relation_paged_read_q8.argtypes = [_PP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]
        lib.relation_paged_read_q8.restype = ctypes.c_int
        lib.relation_paged_q8_workspace_bytes.argtypes = [_PP, ctypes.c_int]
        lib.relation_paged_q8_workspace_bytes.restype = ctypes.c_size_t
        lib.relation_paged_fwd_q8.argtypes = [_PP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP,
                                              ctypes.c_size_t, _VP]
        lib.relation_paged_fwd_q8.restype = ctypes.c_int
        lib.relation_selftest_wait_timeout.argtypes = [ctypes.c_uint32, _VP]
        lib.relation_selftest_wait_timeout.restype = ctypes.c_int
        lib.relation_check_device_status.argtypes = []
        lib.relation_check_device_status.restype = ctypes.c_int
        lib.relation_last_launch_count.argtypes = []
        lib.relation_last_launch_count.restype = ctypes.c_int
        lib.relation_status_string.argtypes = [ctypes.c_int]
        lib.relation_status_string.restype = ctypes.c_char_p
        lib.relation_abi_version.argtypes = []
        lib.relation_abi_version.restype = ctypes.c_int
        _lib = lib
        return lib


def declared_symbols() -> list[str]:
    """Entry points declared in include/*.h."""
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    names = []
    for fn in sorted(os.listdir(inc)):
        if fn.endswith(".h"):
            text = open(os.path.join(inc, fn)).read()
            names += re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*(relation_[a-z0-9_]+)\s*\(", text, re.M)
    return sorted(set(names))


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("Relation tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("Relation tensors must be contiguous [B, H, T, d_h]")
    return t.data_ptr()


def _host_ptr(t) -> int | None:
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError("relation_step_host takes host tensors")
    if not t.is_contiguous():
        raise ValueError("Relation tensors must be contiguous")
    return t.data_ptr()


def _stream_ptr(stream) -> int | None:
    if stream is None:  # the handle alone: a Stream object costs 2.5 us more on the host
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) or None
    return stream.cuda_stream or None


def _check(code: int, what: str) -> None:
    if code != 0:
        msg = load().relation_status_string(code).decode()
        raise RelationError(code, what, msg)


def problem_for(t: torch.Tensor, tau_S: float, lam: float, causal: bool, layout: int = RELATION_LAYOUT_BHTD) -> Problem:
    """Problem for operand tensors shaped [B, H, T, d_h] (BHTD) or [B, T, H, d_h] (BTHD)."""
    if t.dim() != 4:
        raise ValueError("expected 4-D operand tensors")
    if t.dtype == torch.bfloat16:
        dt = RELATION_BF16
    elif t.dtype == torch.float32:
        dt = RELATION_F32
    else:
        raise ValueError(f"unsupported dtype {t.dtype}")
    if layout == RELATION_LAYOUT_BHTD:
        B, H, T, d = t.shape
    elif layout == RELATION_LAYOUT_BTHD:
        B, T, H, d = t.shape
    else:
        raise ValueError(f"unknown layout {layout}")
    return Problem(B, H, T, d, dt, float(tau_S), float(lam), 1 if causal else 0, int(layout))


# ------------------------------------------------------------------ C-ABI calls
def relation_fwd(prob: Problem, P1, P2, V, Y, L=None, stream=None) -> None:
    _check(load().relation_fwd(ctypes.byref(prob), _ptr(P1), _ptr(P2), _ptr(V), _ptr(Y), _ptr(L),
                               _stream_ptr(stream)), "relation_fwd")


def relation_selftest_wait_timeout(limit_ms: int, stream=None) -> None:
    _check(load().relation_selftest_wait_timeout(int(limit_ms), _stream_ptr(stream)), "relation_selftest_wait_timeout")


def relation_fwd_workspace_bytes(prob: Problem) -> int:
    return int(load().relation_fwd_workspace_bytes(ctypes.byref(prob)))


def relation_fwd_ws(prob: Problem, P1, P2, V, Y, L=None, workspace=None, stream=None) -> None:
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().relation_fwd_ws(ctypes.byref(prob), _ptr(P1), _ptr(P2), _ptr(V), _ptr(Y), _ptr(L), _ptr(workspace),
                                  nbytes, _stream_ptr(stream)), "relation_fwd_ws")


def relation_bwd_workspace_bytes(prob: Problem) -> int:
    return int(load().relation_bwd_workspace_bytes(ctypes.byref(prob)))


def _bwd_call(name, prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlambda, workspace, stream):
    fn = getattr(load(), name)
    _check(fn(ctypes.byref(prob), _ptr(P1), _ptr(P2), _ptr(V), _ptr(Y), _ptr(L), _ptr(dY), _ptr(dP1), _ptr(dP2),
              _ptr(dV), _ptr(dlambda), _ptr(workspace), workspace.numel() * workspace.element_size(),
              _stream_ptr(stream)), name)


def relation_bwd(prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlambda, workspace, stream=None) -> None:
    _bwd_call("relation_bwd", prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlambda, workspace, stream)


def relation_bwd_prepare(prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlambda, workspace, stream=None) -> None:
    _bwd_call("relation_bwd_prepare", prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlambda, workspace, stream)


def relation_bwd_main(prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlambda, workspace, stream=None) -> None:
    _bwd_call("relation_bwd_main", prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlambda, workspace, stream)


def relation_bwd_finish(prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlambda, workspace, stream=None) -> None:
    _bwd_call("relation_bwd_finish", prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlambda, workspace, stream)


def relation_bwd_noalloc(prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlambda, stream=None) -> None:
    """relation_bwd with the library's built-in scratch array as workspace (no allocation)."""
    _check(load().relation_bwd_noalloc(ctypes.byref(prob), _ptr(P1), _ptr(P2), _ptr(V), _ptr(Y), _ptr(L), _ptr(dY),
                                       _ptr(dP1), _ptr(dP2), _ptr(dV), _ptr(dlambda), _stream_ptr(stream)),
           "relation_bwd_noalloc")


def relation_step_host_device_bytes(prob: Problem, chunks: int) -> int:
    return int(load().relation_step_host_device_bytes(ctypes.byref(prob), int(chunks)))


def relation_step_host(prob, P1, P2, V, dY, Y, L, dP1, dP2, dV, dlambda, chunks, device_buffer, stream=None) -> None:
    """Host tensors in and out (pinned for overlap); device_buffer a CUDA tensor of
    relation_step_host_device_bytes(prob, chunks) bytes."""
    _check(load().relation_step_host(ctypes.byref(prob), _host_ptr(P1), _host_ptr(P2), _host_ptr(V), _host_ptr(dY),
                                     _host_ptr(Y), _host_ptr(L), _host_ptr(dP1), _host_ptr(dP2), _host_ptr(dV),
                                     _host_ptr(dlambda), int(chunks), _ptr(device_buffer),
                                     device_buffer.numel() * device_buffer.element_size(), _stream_ptr(stream)),
           "relation_step_host")


def relation_decode_workspace_bytes(prob: Problem) -> int:
    return int(load().relation_decode_workspace_bytes(ctypes.byref(prob)))


def relation_decode(prob, P1_new, P2_new, V_new, P2_cache, V_cache, positions, append, Y, L, workspace,
                    stream=None) -> None:
    _check(load().relation_decode(ctypes.byref(prob), _ptr(P1_new), _ptr(P2_new), _ptr(V_new), _ptr(P2_cache),
                                  _ptr(V_cache), _ptr(positions), int(append), _ptr(Y), _ptr(L), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
           "relation_decode")


def relation_prologue_fwd(prob, X1, X2, I, theta, pairing, rope_base, pos0, P1, P2, I_mixed, stream=None) -> None:
    _check(load().relation_prologue_fwd(ctypes.byref(prob), _ptr(X1), _ptr(X2), _ptr(I), _ptr(theta), int(pairing),
                                        float(rope_base), _ptr(pos0), _ptr(P1), _ptr(P2), _ptr(I_mixed),
                                        _stream_ptr(stream)), "relation_prologue_fwd")


def relation_prologue_bwd(prob, dP1, dP2, dI_mixed, I_mixed, theta, pairing, rope_base, pos0, dX1, dX2, dI, dtheta,
                          stream=None) -> None:
    _check(load().relation_prologue_bwd(ctypes.byref(prob), _ptr(dP1), _ptr(dP2), _ptr(dI_mixed), _ptr(I_mixed),
                                        _ptr(theta), int(pairing), float(rope_base), _ptr(pos0), _ptr(dX1),
                                        _ptr(dX2), _ptr(dI), _ptr(dtheta), _stream_ptr(stream)),
           "relation_prologue_bwd")


def relation_fwd_prologue(prob, X1, X2, I, theta, pairing, rope_base, pos0, Y, L=None, stream=None) -> None:
    _check(load().relation_fwd_prologue(ctypes.byref(prob), _ptr(X1), _ptr(X2), _ptr(I), _ptr(theta), int(pairing),
                                        float(rope_base), _ptr(pos0), _ptr(Y), _ptr(L), _stream_ptr(stream)),
           "relation_fwd_prologue")


def relation_bwd_prologue_workspace_bytes(prob: Problem) -> int:
    return int(load().relation_bwd_prologue_workspace_bytes(ctypes.byref(prob)))


def relation_bwd_prologue(prob, X1, X2, I, theta, pairing, rope_base, pos0, Y, L, dY, dX1, dX2, dI, dtheta, dlambda,
                          workspace, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().relation_bwd_prologue(ctypes.byref(prob), _ptr(X1), _ptr(X2), _ptr(I), _ptr(theta), int(pairing),
                                        float(rope_base), _ptr(pos0), _ptr(Y), _ptr(L), _ptr(dY), _ptr(dX1),
                                        _ptr(dX2), _ptr(dI), _ptr(dtheta), _ptr(dlambda), _ptr(workspace), nbytes,
                                        _stream_ptr(stream)), "relation_bwd_prologue")


def fused_prologue_step(X1, X2, I, theta, pairing: int, rope_base: float, tau_S: float, lam: float, dY,
                        causal: bool = True, pos0=None, layout: int = RELATION_LAYOUT_BHTD, workspace=None,
                        stream=None):
    """Forward and backward of the operator with its input prologue fused into the kernels'
    loads; allocates the outputs (and the workspace unless given) and returns
    (Y, L, dX1, dX2, dI, dtheta, dlambda)."""
    prob = problem_for(X1, tau_S, lam, causal, layout)
    Y = torch.empty_like(I)
    L = torch.empty((prob.B, prob.H, prob.T), dtype=torch.float32, device=X1.device)
    relation_fwd_prologue(prob, X1, X2, I, theta, pairing, rope_base, pos0, Y, L, stream)
    dX1, dX2, dI = torch.empty_like(X1), torch.empty_like(X2), torch.empty_like(I)
    dtheta = torch.empty(prob.H // 2, dtype=torch.float32, device=X1.device)
    dlam = torch.empty(1, dtype=torch.float32, device=X1.device)
    if workspace is None:
        n = relation_bwd_prologue_workspace_bytes(prob)
        workspace = torch.empty((n + 3) // 4, dtype=torch.float32, device=X1.device)
    relation_bwd_prologue(prob, X1, X2, I, theta, pairing, rope_base, pos0, Y, L, dY, dX1, dX2, dI, dtheta, dlam,
                          workspace, stream)
    return Y, L, dX1, dX2, dI, dtheta, dlam


def relation_linear_workspace_bytes(prob: Problem) -> int:
    return int(load().relation_linear_workspace_bytes(ctypes.byref(prob)))


def relation_linear_fwd(prob, P1, P2, I, G, Y, state, workspace, stream=None) -> None:
    _check(load().relation_linear_fwd(ctypes.byref(prob), _ptr(P1), _ptr(P2), _ptr(I), _ptr(G), _ptr(Y),
                                      _ptr(state), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream_ptr(stream)), "relation_linear_fwd")


def relation_linear_bwd(prob, P1, P2, I, G, dY, dP1, dP2, dI, dG, states_from_forward, workspace,
                        stream=None) -> None:
    _check(load().relation_linear_bwd(ctypes.byref(prob), _ptr(P1), _ptr(P2), _ptr(I), _ptr(G), _ptr(dY), _ptr(dP1),
                                      _ptr(dP2), _ptr(dI), _ptr(dG), int(states_from_forward), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
           "relation_linear_bwd")


def relation_linear_fwd_gate(prob, P1, P2, I, R, A_log, dt_bias, Y, state, workspace, stream=None) -> None:
    _check(load().relation_linear_fwd_gate(ctypes.byref(prob), _ptr(P1), _ptr(P2), _ptr(I), _ptr(R), _ptr(A_log),
                                           _ptr(dt_bias), _ptr(Y), _ptr(state), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
           "relation_linear_fwd_gate")


def relation_linear_bwd_gate(prob, P1, P2, I, R, A_log, dt_bias, dY, dP1, dP2, dI, dR, dA_log, d_dt_bias,
                             states_from_forward, workspace, stream=None) -> None:
    _check(load().relation_linear_bwd_gate(ctypes.byref(prob), _ptr(P1), _ptr(P2), _ptr(I), _ptr(R), _ptr(A_log),
                                           _ptr(dt_bias), _ptr(dY), _ptr(dP1), _ptr(dP2), _ptr(dI), _ptr(dR),
                                           _ptr(dA_log), _ptr(d_dt_bias), int(states_from_forward), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
           "relation_linear_bwd_gate")


def linear_gate_fwd_bwd(P1, P2, I, R, A_log, dt_bias, dY, tau_S: float, layout: int = RELATION_LAYOUT_BHTD,
                        stream=None):
    """Gated Linear Relation forward and backward (states reused); returns
    (Y, dP1, dP2, dI, dR, dA_log, d_dt_bias)."""
    prob = problem_for(P1, tau_S, 0.0, True, layout)
    ws = linear_workspace(prob, P1.device)
    Y = torch.empty_like(I)
    relation_linear_fwd_gate(prob, P1, P2, I, R, A_log, dt_bias, Y, None, ws, stream)
    dP1, dP2, dI, dR = torch.empty_like(P1), torch.empty_like(P2), torch.empty_like(I), torch.empty_like(R)
    dA, dB = torch.empty_like(A_log), torch.empty_like(dt_bias)
    relation_linear_bwd_gate(prob, P1, P2, I, R, A_log, dt_bias, dY, dP1, dP2, dI, dR, dA, dB, True, ws, stream)
    return Y, dP1, dP2, dI, dR, dA, dB


def relation_linear_step(prob: LinearPacked, P1, P2, I, G, A_log, dt_bias, states, slots_in, slots_out, Y,
                         stream=None) -> None:
    _check(load().relation_linear_step(ctypes.byref(prob), _ptr(P1), _ptr(P2), _ptr(I), _ptr(G), _ptr(A_log),
                                       _ptr(dt_bias), _ptr(states), _ptr(slots_in), _ptr(slots_out), _ptr(Y),
                                       _stream_ptr(stream)), "relation_linear_step")


def relation_linear_packed_workspace_bytes(prob: LinearPacked, max_fresh: int) -> int:
    return int(load().relation_linear_packed_workspace_bytes(ctypes.byref(prob), int(max_fresh)))


def relation_linear_packed_fwd(prob: LinearPacked, P1, P2, I, G, A_log, dt_bias, starts, max_fresh, states, slots_in,
                               slots_out, Y, workspace, stream=None) -> None:
    _check(load().relation_linear_packed_fwd(ctypes.byref(prob), _ptr(P1), _ptr(P2), _ptr(I), _ptr(G), _ptr(A_log),
                                             _ptr(dt_bias), _ptr(starts), max_fresh, _ptr(states), _ptr(slots_in),
                                             _ptr(slots_out), _ptr(Y), _ptr(workspace),
                                             0 if workspace is None else workspace.nbytes, _stream_ptr(stream)),
           "relation_linear_packed_fwd")


def relation_paged_plan(prob: Paged, cached, fresh, free_pages, block_table, starts, slots, positions, used,
                        stream=None) -> None:
    _check(load().relation_paged_plan(ctypes.byref(prob), _ptr(cached), _ptr(fresh), _ptr(free_pages),
                                      0 if free_pages is None else free_pages.numel(), _ptr(block_table),
                                      _ptr(starts), _ptr(slots), _ptr(positions), _ptr(used), _stream_ptr(stream)),
           "relation_paged_plan")


def relation_paged_store(prob: Paged, X1, X2, I, theta, pairing, rope_base, positions, slots, P1, P2_pages, I_pages,
                         stream=None) -> None:
    _check(load().relation_paged_store(ctypes.byref(prob), _ptr(X1), _ptr(X2), _ptr(I), _ptr(theta), pairing,
                                       rope_base, _ptr(positions), _ptr(slots), _ptr(P1), _ptr(P2_pages),
                                       _ptr(I_pages), _stream_ptr(stream)), "relation_paged_store")


def relation_paged_workspace_bytes(prob: Paged, max_fresh: int) -> int:
    return int(load().relation_paged_workspace_bytes(ctypes.byref(prob), int(max_fresh)))


def relation_paged_fwd(prob: Paged, P1, P2_pages, I_pages, block_table, starts, cached, max_fresh, Y, L, workspace,
                       stream=None) -> None:
    _check(load().relation_paged_fwd(ctypes.byref(prob), _ptr(P1), _ptr(P2_pages), _ptr(I_pages), _ptr(block_table),
                                     _ptr(starts), _ptr(cached), max_fresh, _ptr(Y), _ptr(L), _ptr(workspace),
                                     workspace.nbytes, _stream_ptr(stream)), "relation_paged_fwd")


def relation_paged_store_q8(prob: Paged, X1, X2, I, theta, pairing, rope_base, positions, slots, P1, P2_pages, I_pages,
                            scales, stream=None) -> None:
    _check(load().relation_paged_store_q8(ctypes.byref(prob), _ptr(X1), _ptr(X2), _ptr(I), _ptr(theta), pairing,
                                          rope_base, _ptr(positions), _ptr(slots), _ptr(P1), _ptr(P2_pages),
                                          _ptr(I_pages), _ptr(scales), _stream_ptr(stream)), "relation_paged_store_q8")


def relation_paged_read_q8(prob: Paged, slots, P2_pages, I_pages, scales, P2, I, stream=None) -> None:
    _check(load().relation_paged_read_q8(ctypes.byref(prob), _ptr(slots), _ptr(P2_pages), _ptr(I_pages), _ptr(scales),
                                         _ptr(P2), _ptr(I), _stream_ptr(stream)), "relation_paged_read_q8")


def relation_paged_q8_workspace_bytes(prob: Paged, max_fresh: int) -> int:
    return int(load().relation_paged_q8_workspace_bytes(ctypes.byref(prob), int(max_fresh)))


def relation_paged_fwd_q8(prob: Paged, P1, P2_pages, I_pages, scales, block_table, starts, cached, max_fresh, Y, L,
                          workspace, stream=None) -> None:
    _check(load().relation_paged_fwd_q8(ctypes.byref(prob), _ptr(P1), _ptr(P2_pages), _ptr(I_pages), _ptr(scales),
                                        _ptr(block_table), _ptr(starts), _ptr(cached), max_fresh, _ptr(Y), _ptr(L),
                                        _ptr(workspace), workspace.nbytes, _stream_ptr(stream)), "relation_paged_fwd_q8")


def relation_check_device_status() -> int:
    return int(load().relation_check_device_status())


def relation_last_launch_count() -> int:
    return int(load().relation_last_launch_count())


def relation_status_string(code: int) -> str:
    return load().relation_status_string(code).decode()


def relation_abi_version() -> int:
    return int(load().relation_abi_version())


# ------------------------------------------------------- tensor-level helpers
def fwd_workspace(prob: Problem, device):
    """Workspace tensor for relation_fwd_ws, or None when the problem needs none."""
    n = relation_fwd_workspace_bytes(prob)
    return torch.empty((n + 3) // 4, dtype=torch.float32, device=device) if n else None


def fwd(P1, P2, V, tau_S: float, lam: float, causal: bool = True, stream=None, want_L: bool = True,
        layout: int = RELATION_LAYOUT_BHTD, workspace=None, use_workspace: bool = True):
    """Allocates Y (and L [B, H, T]) and runs the forward; returns (Y, L).  Head widths that
    need a workspace (bf16 d_h = 60) get one (allocated here unless given) and run through
    relation_fwd_ws; use_workspace=False runs relation_fwd instead."""
    prob = problem_for(P1, tau_S, lam, causal, layout)
    Y = torch.empty_like(V)
    L = torch.empty((prob.B, prob.H, prob.T), dtype=torch.float32, device=P1.device) if want_L else None
    if use_workspace and relation_fwd_workspace_bytes(prob):
        if workspace is None:
            workspace = fwd_workspace(prob, P1.device)
        relation_fwd_ws(prob, P1, P2, V, Y, L, workspace, stream)
    else:
        relation_fwd(prob, P1, P2, V, Y, L, stream)
    return Y, L


def linear_workspace(prob: Problem, device) -> torch.Tensor:
    """Workspace tensor for relation_linear_fwd / relation_linear_bwd."""
    n = relation_linear_workspace_bytes(prob)
    return torch.empty(max(1, (n + 3) // 4), dtype=torch.float32, device=device)


def linear_fwd(P1, P2, I, G, tau_S: float, layout: int = RELATION_LAYOUT_BHTD, want_state: bool = False,
               stream=None, workspace=None):
    """Linear Relation forward; allocates Y (and the final state [B, H, d, d]); returns (Y, state)."""
    prob = problem_for(P1, tau_S, 0.0, True, layout)
    Y = torch.empty_like(I)
    state = (torch.empty((prob.B, prob.H, prob.d_h, prob.d_h), dtype=torch.float32, device=P1.device)
             if want_state else None)
    if workspace is None:
        workspace = linear_workspace(prob, P1.device)
    relation_linear_fwd(prob, P1, P2, I, G, Y, state, workspace, stream)
    return Y, state


def linear_bwd(P1, P2, I, G, dY, tau_S: float, layout: int = RELATION_LAYOUT_BHTD, stream=None, workspace=None,
               states_from_forward: bool = False):
    """Linear Relation backward; allocates and returns (dP1, dP2, dI, dG).  states_from_forward:
    ``workspace`` still holds what linear_fwd left in it for the same inputs."""
    prob = problem_for(P1, tau_S, 0.0, True, layout)
    dP1, dP2, dI, dG = torch.empty_like(P1), torch.empty_like(P2), torch.empty_like(I), torch.empty_like(G)
    if workspace is None:
        if states_from_forward:
            raise ValueError("states_from_forward needs the forward's workspace")
        workspace = linear_workspace(prob, P1.device)
    relation_linear_bwd(prob, P1, P2, I, G, dY, dP1, dP2, dI, dG, states_from_forward, workspace, stream)
    return dP1, dP2, dI, dG


def decode(P1_new, P2_new, V_new, P2_cache, V_cache, positions, tau_S: float, lam: float, append: bool = True,
           layout: int = RELATION_LAYOUT_BHTD, stream=None, workspace=None):
    """One Relation Cache step; allocates Y [B, H, d_h] and L [B, H]; returns (Y, L)."""
    B, H, d = P1_new.shape
    T = P2_cache.shape[2] if layout == RELATION_LAYOUT_BHTD else P2_cache.shape[1]
    dt = RELATION_BF16 if P1_new.dtype == torch.bfloat16 else RELATION_F32
    prob = Problem(B, H, T, d, dt, float(tau_S), float(lam), 1, int(layout))
    Y = torch.empty_like(P1_new)
    L = torch.empty((B, H), dtype=torch.float32, device=P1_new.device)
    if workspace is None:
        workspace = torch.empty((relation_decode_workspace_bytes(prob) + 3) // 4, dtype=torch.float32,
                                device=P1_new.device)
    relation_decode(prob, P1_new, P2_new, V_new, P2_cache, V_cache, positions, append, Y, L, workspace, stream)
    return Y, L


def step_host(P1, P2, V, dY, tau_S: float, lam: float, causal: bool = True, chunks: int = 1, out=None,
              device_buffer=None, want_L: bool = False, stream=None, layout: int = RELATION_LAYOUT_BHTD):
    """relation_step_host on host tensors; allocates what is not given (pinned host outputs,
    the device buffer).  Returns (Y, L or None, dP1, dP2, dV, dlambda) as host tensors."""
    prob = problem_for(P1, tau_S, lam, causal, layout)
    if out is None:
        out = tuple(torch.empty(P1.shape, dtype=P1.dtype).pin_memory() for _ in range(4))
    Y, dP1, dP2, dV = out
    L = torch.empty((prob.B, prob.H, prob.T), dtype=torch.float32).pin_memory() if want_L else None
    dlam = torch.empty(1, dtype=torch.float32).pin_memory()
    if device_buffer is None:
        nbytes = relation_step_host_device_bytes(prob, chunks)
        device_buffer = torch.empty((nbytes + 3) // 4, dtype=torch.float32, device="cuda")
    relation_step_host(prob, P1, P2, V, dY, Y, L, dP1, dP2, dV, dlam, chunks, device_buffer, stream)
    return Y, L, dP1, dP2, dV, dlam


def bwd(P1, P2, V, Y, L, dY, tau_S: float, lam: float, causal: bool = True, stream=None, workspace=None,
        layout: int = RELATION_LAYOUT_BHTD):
    """Allocates the gradients and workspace and runs relation_bwd; returns (dP1, dP2, dV, dlambda)."""
    prob = problem_for(P1, tau_S, lam, causal, layout)
    dP1, dP2, dV = torch.empty_like(P1), torch.empty_like(P2), torch.empty_like(V)
    dlam = torch.empty(1, dtype=torch.float32, device=P1.device)
    if workspace is None:
        nbytes = relation_bwd_workspace_bytes(prob)
        workspace = torch.empty((nbytes + 3) // 4, dtype=torch.float32, device=P1.device)
    relation_bwd(prob, P1, P2, V, Y, L, dY, dP1, dP2, dV, dlam, workspace, stream)
    return dP1, dP2, dV, dlam


# ------------------------------------------- Linear Relation over a pool of states
def linear_states(states: int, H: int, d_h: int, device="cuda") -> torch.Tensor:
    """A pool of states [states, H, d_h, d_h] float32, zeroed."""
    return torch.zeros(states, H, d_h, d_h, dtype=torch.float32, device=device)


def linear_packed_for(P1, states, R: int, tau_S: float) -> LinearPacked:
    """Problem for packed tensors [N, H, d_h] (P1: one of them) and a pool of states."""
    N, H, d = P1.shape
    if P1.dtype not in _DTYPE_CODES:
        raise ValueError(f"unsupported dtype {P1.dtype}")
    if states.dtype is not torch.float32 or states.shape[1:] != (H, d, d):
        raise ValueError("states are [states, H, d_h, d_h] of torch.float32")
    return LinearPacked(R, N, H, d, states.shape[0], _DTYPE_CODES[P1.dtype], tau_S)


def _on_current_device(*tensors) -> None:
    """The library launches on the current device: tensors of another are refused (-1: host tensors, which _ptr refuses).
    By number: a device object a tensor costs 2 us a call more."""
    device = tensors[0].get_device()
    for x in tensors:
        if x is not None and x.get_device() != device:
            raise ValueError("Relation tensors must be on one device")
    if device >= 0 and device != torch._C._cuda_getDevice():
        raise ValueError("Relation tensors must be on the current device")


def _linear_packed_check(prob, P1, P2, I, G, states, slots_in, slots_out, A_log, dt_bias, *others):
    _on_current_device(P1, P2, I, G, states, slots_in, slots_out, A_log, dt_bias, *others)
    shape, dtype = P1.shape, P1.dtype
    if P2.shape != shape or I.shape != shape or G.shape != shape:
        raise ValueError("P1, P2, I and G are [N, H, d_h]")
    if P2.dtype is not dtype or I.dtype is not dtype or G.dtype is not torch.float32:
        raise ValueError(f"P2 and I are {dtype}, as P1, and G is torch.float32")
    if not (slots_in.dtype is slots_out.dtype is _I32) or slots_in.numel() != prob.R or slots_out.numel() != prob.R:
        raise ValueError("slots_in and slots_out are [R] of torch.int32")
    if (A_log is None) != (dt_bias is None):
        raise ValueError("A_log and dt_bias are given both or neither")
    for x in (A_log, dt_bias):
        if x is not None and (x.dtype is not torch.float32 or x.shape != (prob.H, prob.d_h)):
            raise ValueError("A_log and dt_bias are [H, d_h] of torch.float32")


def _like_on(x, Y, stream):
    """Y, or a tensor like x from the stream that the kernels run on, marked as used by the caller's stream."""
    if Y is None:
        if stream is None:  # the current one
            return torch.empty_like(x)
        with torch.cuda.stream(stream):
            Y = torch.empty_like(x)
        Y.record_stream(torch.cuda.current_stream())
    elif Y.shape != x.shape or Y.dtype is not x.dtype:
        raise ValueError("Y is like P1")
    return Y


def linear_step(P1, P2, I, G, states, slots_in, slots_out, tau_S: float, A_log=None, dt_bias=None, Y=None, stream=None):
    """Linear Relation of one new token per request, rows [R, H, d_h], from and to slots of a pool of states
    (slots_in, slots_out [R] int32; negative: no state yet, not kept); returns Y.  With A_log and dt_bias [H, d_h] G
    holds the retention gate's input."""
    prob = linear_packed_for(P1, states, slots_in.numel(), tau_S)
    _linear_packed_check(prob, P1, P2, I, G, states, slots_in, slots_out, A_log, dt_bias, Y)
    Y = _like_on(P1, Y, stream)
    relation_linear_step(prob, P1, P2, I, G, A_log, dt_bias, states, slots_in, slots_out, Y, stream)
    return Y


def linear_packed_fwd(P1, P2, I, G, starts, states, slots_in, slots_out, max_fresh: int, tau_S: float, A_log=None,
                      dt_bias=None, Y=None, workspace=None, stream=None):
    """Linear Relation of packed requests of any lengths (starts [R + 1] int32) from and to slots of a pool of states;
    returns Y.  max_fresh: a bound of any request's new tokens (0: none known).  Y and workspace are allocated when not
    given, from the stream that the kernels run on."""
    prob = linear_packed_for(P1, states, slots_in.numel(), tau_S)
    _linear_packed_check(prob, P1, P2, I, G, states, slots_in, slots_out, A_log, dt_bias, starts, Y, workspace)
    if starts.dtype is not _I32 or starts.numel() != prob.R + 1:
        raise ValueError("starts is [R + 1] of torch.int32")
    Y = _like_on(P1, Y, stream)
    if workspace is None:
        n = relation_linear_packed_workspace_bytes(prob, max_fresh)
        if n:  # freed on return: the stream's own memory goes to its next work only, which runs after the kernels
            with torch.cuda.stream(stream):
                workspace = torch.empty(n, dtype=torch.uint8, device=P1.device)
    relation_linear_packed_fwd(prob, P1, P2, I, G, A_log, dt_bias, starts, max_fresh, states, slots_in, slots_out, Y,
                               workspace, stream)
    return Y


# ------------------------------------------------------- paged Relation Cache
_DTYPE_CODES = {torch.bfloat16: RELATION_BF16, torch.float32: RELATION_F32}
_I32, _I64 = torch.int32, torch.int64


def paged_row(d_h: int, dtype) -> int:
    """Elements from one cached row to the next (rows start on 16 bytes: bf16 d_h = 60 takes 64)."""
    return -(-d_h // 8) * 8 if dtype == torch.bfloat16 else d_h


def paged_pages(pages: int, G: int, page_size: int, d_h: int, dtype, layout: int = RELATION_LAYOUT_BHTD,
                device="cuda"):
    """A pair of page pools (P2_pages, I_pages), zeroed."""
    shape = (pages, G, page_size) if layout == RELATION_LAYOUT_BHTD else (pages, page_size, G)
    return tuple(torch.zeros(*shape, paged_row(d_h, dtype), dtype=dtype, device=device) for _ in range(2))


def paged_for(heads, pages, R: int, table_width: int, tau_S: float, lam: float, layout: int) -> Paged:
    """Problem for packed tensors [N, H, d_h] (heads: the P1 / X1 tensor) over a page pool."""
    N, H, d = heads.shape
    if pages.dim() != 4 or pages.dtype is not heads.dtype or heads.dtype not in _DTYPE_CODES:
        raise ValueError("pages are 4-D and of the packed tensors' dtype (bfloat16 or float32)")
    if layout == RELATION_LAYOUT_BHTD:
        P, G, page, row = pages.shape
    elif layout == RELATION_LAYOUT_BTHD:
        P, page, G, row = pages.shape
    else:
        raise ValueError(f"unknown layout {layout}")
    if row != paged_row(d, heads.dtype):
        raise ValueError(f"pages hold rows of {row}, heads of {d} need {paged_row(d, heads.dtype)}")
    return Paged(R, N, H, G, d, P, page, table_width, _DTYPE_CODES[heads.dtype], tau_S, lam, layout)


def paged_plan(cached, fresh, free_pages, block_table, pages: int, page_size: int, starts, slots, positions, used,
               stream=None) -> None:
    """Block tables and slot maps of a step: fills block_table (new entries), starts [R + 1], slots [N],
    positions [N] and used [1] from the requests' lengths (all int32, slots int64)."""
    if not (cached.dtype is fresh.dtype is block_table.dtype is starts.dtype is positions.dtype is used.dtype is _I32):
        raise ValueError("cached, fresh, block_table, starts, positions and used are torch.int32")
    if slots.dtype is not _I64 or (free_pages is not None and free_pages.dtype is not _I32):
        raise ValueError("slots are torch.int64, free_pages torch.int32")
    R, width = block_table.shape
    N = slots.numel()
    if cached.numel() != R or fresh.numel() != R or starts.numel() != R + 1 or positions.numel() != N:
        raise ValueError("cached and fresh are [R], starts [R + 1], positions and slots [N]")
    # The plan reads sizes only: heads, width and dtype are stand-ins.
    relation_paged_plan(Paged(R, N, 1, 1, 64, pages, page_size, width, RELATION_BF16, 1.0, 0.0, RELATION_LAYOUT_BHTD),
                        cached, fresh, free_pages, block_table, starts, slots, positions, used, stream)


def paged_store(X1, X2, I, theta, pairing: int, rope_base: float, positions, slots, P1, P2_pages, I_pages,
                layout: int = RELATION_LAYOUT_BHTD, stream=None) -> None:
    """RoPE and Givens mixing of packed new tokens, P1 [N, H, d_h] written in place of a copy and the cached rows
    into their pages; theta None stores the states unmixed."""
    if positions.dtype is not _I32 or slots.dtype is not _I64:
        raise ValueError("positions are torch.int32, slots torch.int64")
    prob = paged_for(X1, P2_pages, 1, 1, 1.0, 0.0, layout)
    N = prob.N
    if X2.shape != (N, prob.G, prob.d_h) or I.shape != X2.shape or P1.shape != X1.shape or \
            I_pages.shape != P2_pages.shape or positions.numel() != N or slots.numel() != N:
        raise ValueError("X1, P1 are [N, H, d_h], X2, I [N, G, d_h], positions, slots [N], both page pools alike")
    if not (X2.dtype is I.dtype is P1.dtype is I_pages.dtype is X1.dtype):
        raise ValueError(f"X2, I, P1 and the pages must be {X1.dtype}, as X1")
    if theta is not None and (theta.dtype is not torch.float32 or theta.numel() != prob.G // 2):
        raise ValueError("theta is [G / 2] of torch.float32")
    relation_paged_store(prob, X1, X2, I, theta, pairing, rope_base, positions, slots, P1, P2_pages, I_pages, stream)


def paged_workspace(prob: Paged, max_fresh: int, device="cuda") -> torch.Tensor:
    """Workspace tensor for relation_paged_fwd."""
    n = relation_paged_workspace_bytes(prob, max_fresh)
    if n == 0:
        raise ValueError("relation_paged_fwd has no workspace for this problem")
    return torch.empty(n, dtype=torch.uint8, device=device)


def paged_fwd(P1, P2_pages, I_pages, block_table, starts, cached, max_fresh: int, tau_S: float, lam: float, Y=None,
              L=None, workspace=None, layout: int = RELATION_LAYOUT_BHTD, stream=None):
    """Relation of packed new tokens P1 [N, H, d_h] over the pages; returns (Y, L).  Y and workspace are allocated
    when not given, from the stream that the kernels run on; L [N, H] float32 is filled when given.  Tensors passed in
    for another stream than their own are the caller's to order and to keep."""
    R, width = block_table.shape
    prob = paged_for(P1, P2_pages, R, width, tau_S, lam, layout)
    if not (block_table.dtype is starts.dtype is cached.dtype is _I32):
        raise ValueError("block_table, starts and cached are torch.int32")
    if starts.numel() != R + 1 or cached.numel() != R or I_pages.shape != P2_pages.shape or \
            I_pages.dtype is not P1.dtype:
        raise ValueError("starts is [R + 1], cached [R], both page pools alike")
    if Y is None:
        with torch.cuda.stream(stream):  # None: the current one
            Y = torch.empty_like(P1)
        if stream is not None:
            Y.record_stream(torch.cuda.current_stream())  # where the caller reads it
    elif Y.shape != P1.shape or Y.dtype is not P1.dtype:
        raise ValueError("Y is like P1")
    if L is not None:
        if L.dtype is not torch.float32 or L.shape != (prob.N, prob.H):
            raise ValueError("L is [N, H] of torch.float32")
    if workspace is None:
        # Freed on return: the stream's own memory goes to its next work only, which runs after the kernels.
        with torch.cuda.stream(stream):
            workspace = paged_workspace(prob, max_fresh, P1.device)
    relation_paged_fwd(prob, P1, P2_pages, I_pages, block_table, starts, cached, max_fresh, Y, L, workspace, stream)
    return Y, L


# ------------------------------------------------------- paged Relation Cache in 8 bits
def paged_row_q8(d_h: int) -> int:
    """Bytes from one cached row to the next (rows start on 16)."""
    return -(-d_h // 16) * 16


def paged_pages_q8(pages: int, G: int, page_size: int, d_h: int, layout: int = RELATION_LAYOUT_BHTD, device="cuda"):
    """8-bit page pools and their scales (P2_pages, I_pages, scales), zeroed."""
    shape = (pages, G, page_size) if layout == RELATION_LAYOUT_BHTD else (pages, page_size, G)
    P2, I = (torch.zeros(*shape, paged_row_q8(d_h), dtype=torch.int8, device=device) for _ in range(2))
    return P2, I, torch.zeros(*shape, 2, dtype=torch.bfloat16, device=device)


def paged_q8_for(N: int, H: int, d_h: int, P2_pages, I_pages, scales, R: int, table_width: int, tau_S: float,
                 lam: float, layout: int) -> Paged:
    """Problem for N packed rows of H heads over 8-bit pages."""
    if not (P2_pages.dtype is I_pages.dtype is torch.int8) or scales.dtype is not torch.bfloat16:
        raise ValueError("8-bit pages are torch.int8, their scales torch.bfloat16")
    if P2_pages.dim() != 4 or I_pages.shape != P2_pages.shape or scales.shape != (*P2_pages.shape[:3], 2):
        raise ValueError("both page pools are alike, 4-D, and scales have two values for each of their rows")
    if layout == RELATION_LAYOUT_BHTD:
        P, G, page, row = P2_pages.shape
    elif layout == RELATION_LAYOUT_BTHD:
        P, page, G, row = P2_pages.shape
    else:
        raise ValueError(f"unknown layout {layout}")
    if row != paged_row_q8(d_h):
        raise ValueError(f"pages hold rows of {row}, heads of {d_h} need {paged_row_q8(d_h)}")
    return Paged(R, N, H, G, d_h, P, page, table_width, RELATION_BF16, tau_S, lam, layout)


def paged_store_q8(X1, X2, I, theta, pairing: int, rope_base: float, positions, slots, P1, P2_pages, I_pages, scales,
                   layout: int = RELATION_LAYOUT_BHTD, stream=None) -> None:
    """paged_store into 8-bit pages: RoPE and Givens mixing of packed new tokens, the cached rows quantised as they are
    written, with one power of two a row (scales)."""
    _on_current_device(X1, X2, I, theta, positions, slots, P1, P2_pages, I_pages, scales)
    if positions.dtype is not _I32 or slots.dtype is not _I64:
        raise ValueError("positions are torch.int32, slots torch.int64")
    N, H, d = X1.shape
    prob = paged_q8_for(N, H, d, P2_pages, I_pages, scales, 1, 1, 1.0, 0.0, layout)
    if X2.shape != (N, prob.G, d) or I.shape != X2.shape or P1.shape != X1.shape or positions.numel() != N or \
            slots.numel() != N:
        raise ValueError("X1, P1 are [N, H, d_h], X2, I [N, G, d_h], positions, slots [N]")
    if not (X1.dtype is X2.dtype is I.dtype is P1.dtype is torch.bfloat16):
        raise ValueError("X1, X2, I and P1 are torch.bfloat16")
    if theta is not None and (theta.dtype is not torch.float32 or theta.numel() != prob.G // 2):
        raise ValueError("theta is [G / 2] of torch.float32")
    relation_paged_store_q8(prob, X1, X2, I, theta, pairing, rope_base, positions, slots, P1, P2_pages, I_pages, scales,
                            stream)


def paged_read_q8(slots, P2_pages, I_pages, scales, d_h: int, P2=None, I=None, layout: int = RELATION_LAYOUT_BHTD,
                  stream=None):
    """The rows (P2, I) [N, G, d_h] bf16 that 8-bit pages hold in some slots [N] int64 (negative: zeros); allocated when
    not given."""
    _on_current_device(slots, P2_pages, I_pages, scales, P2, I)
    N = slots.numel()
    if slots.dtype is not _I64:
        raise ValueError("slots are torch.int64")
    prob = paged_q8_for(N, 1, d_h, P2_pages, I_pages, scales, 1, 1, 1.0, 0.0, layout)
    prob.H = prob.G
    rows = []
    for x in (P2, I):
        if x is None:
            with torch.cuda.stream(stream):  # None: the current one
                x = torch.empty(N, prob.G, d_h, dtype=torch.bfloat16, device=slots.device)
            if stream is not None:
                x.record_stream(torch.cuda.current_stream())
        elif x.shape != (N, prob.G, d_h) or x.dtype is not torch.bfloat16:
            raise ValueError("P2 and I are [N, G, d_h] of torch.bfloat16")
        rows.append(x)
    relation_paged_read_q8(prob, slots, P2_pages, I_pages, scales, *rows, stream)
    return tuple(rows)


def paged_q8_workspace(prob: Paged, max_fresh: int, device="cuda") -> torch.Tensor:
    """Workspace tensor for relation_paged_fwd_q8."""
    n = relation_paged_q8_workspace_bytes(prob, max_fresh)
    if n == 0:
        raise ValueError("relation_paged_fwd_q8 has no workspace for this problem")
    return torch.empty(n, dtype=torch.uint8, device=device)


def paged_fwd_q8(P1, P2_pages, I_pages, scales, block_table, starts, cached, max_fresh: int, tau_S: float, lam: float,
                 Y=None, L=None, workspace=None, layout: int = RELATION_LAYOUT_BHTD, stream=None):
    """paged_fwd over 8-bit pages and their scales; returns (Y, L).  Y and workspace are allocated when not given, from
    the stream that the kernels run on; L [N, H] float32 is filled when given."""
    _on_current_device(P1, P2_pages, I_pages, scales, block_table, starts, cached, Y, L, workspace)
    R, width = block_table.shape
    N, H, d = P1.shape
    if P1.dtype is not torch.bfloat16:
        raise ValueError("P1 is torch.bfloat16")
    prob = paged_q8_for(N, H, d, P2_pages, I_pages, scales, R, width, tau_S, lam, layout)
    if not (block_table.dtype is starts.dtype is cached.dtype is _I32):
        raise ValueError("block_table, starts and cached are torch.int32")
    if starts.numel() != R + 1 or cached.numel() != R:
        raise ValueError("starts is [R + 1], cached [R]")
    if L is not None and (L.dtype is not torch.float32 or L.shape != (N, H)):
        raise ValueError("L is [N, H] of torch.float32")
    Y = _like_on(P1, Y, stream)
    if workspace is None:
        # Freed on return: the stream's own memory goes to its next work only, which runs after the kernels.
        with torch.cuda.stream(stream):
            workspace = paged_q8_workspace(prob, max_fresh, P1.device)
    relation_paged_fwd_q8(prob, P1, P2_pages, I_pages, scales, block_table, starts, cached, max_fresh, Y, L, workspace,
                          stream)
    return Y, L
