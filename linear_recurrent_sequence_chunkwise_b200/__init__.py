"""Multi-scale retention on B200: Python binding of the C ABI in
``include/retention.h``.

The functions below carry the C entry points' names and do argument
marshalling only (torch tensors -> device pointers, sizes, dtypes, the
current CUDA stream); every step of the computation runs in the CUDA library
``libretention.so`` built from ``csrc/``.  There is no fallback: importing
this package fails if the library or the binding of the short calls is missing,
and every call raises
``RetentionError`` when the library returns an error status.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional, Sequence

import torch

__all__ = [
    "RetentionError", "lib", "ret_xpos_rotate", "ret_forward_chunkwise", "ret_forward_chunkwise_ws",
    "ret_chunkwise_workspace_bytes", "ret_chunkwise_prepare_workspace_bytes", "ret_chunkwise_prepare",
    "ret_forward_chunkwise_prepared",
    "ret_backward_chunkwise", "ret_backward_workspace_bytes",
    "ret_forward_chunkwise_noalloc", "ret_chunkwise_noalloc_max_bytes",
    "ret_decode_step", "ret_msr_forward", "ret_msr_workspace_bytes",
    "ret_forward_chunkwise_normalized", "ret_normalized_workspace_bytes", "ret_decode_step_normalized",
    "ret_decode_step_positions", "ret_selftest_bounded_wait",
    "NORM_DECAY", "NORM_SCORE",
    "ret_linear_bf16", "ret_retnet_block_forward", "ret_retnet_block_workspace_bytes",
    "ret_forward_parallel", "ret_forward_recurrent", "ret_check_device_error", "ret_last_error_string",
    "ret_rotary", "ret_rotary_frequencies", "ret_layernorm_forward", "ret_layernorm_backward",
    "ret_layernorm_backward_workspace_bytes",
    "ret_delta_forward_chunkwise", "ret_delta_workspace_bytes", "ret_delta_decode_step",
    "ret_delta_backward_chunkwise", "ret_delta_backward_workspace_bytes",
    "RET_OK", "RET_ERR_INVALID_ARG", "RET_ERR_UNSUPPORTED", "RET_ERR_CUDA", "RET_ERR_TIMEOUT",
    "RET_F32", "RET_BF16",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libretention.so")

RET_OK, RET_ERR_INVALID_ARG, RET_ERR_UNSUPPORTED, RET_ERR_CUDA, RET_ERR_TIMEOUT = 0, 1, 2, 3, 4
RET_F32, RET_BF16 = 0, 1
_STATUS = {0: "RET_OK", 1: "RET_ERR_INVALID_ARG", 2: "RET_ERR_UNSUPPORTED", 3: "RET_ERR_CUDA",
           4: "RET_ERR_TIMEOUT"}


class RetentionError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python linear_recurrent_sequence_chunkwise_b200/build.py` (nvcc, sm_100a)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, d, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_int64
    dp = ctypes.POINTER(ctypes.c_double)
    L.ret_xpos_rotate.argtypes = [vp, i, i, i, i, i, i64, d, vp]
    L.ret_forward_chunkwise.argtypes = [vp, vp, vp, dp, i, i, i, i, i, i, vp, vp, vp, i, i, i, i64, d]
    L.ret_forward_chunkwise_ws.argtypes = [vp, vp, vp, dp, i, i, i, i, i, i, vp, vp, vp, i, i, i, i64, d, vp,
                                           ctypes.c_size_t]
    L.ret_forward_chunkwise_noalloc.argtypes = [vp, vp, vp, dp, i, i, i, i, i, i, vp, vp, vp, i, i, i, i64, d]
    L.ret_backward_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    L.ret_backward_workspace_bytes.restype = ctypes.c_size_t
    L.ret_backward_chunkwise.argtypes = [vp, vp, vp, vp, dp, i, i, i, i, i, i, vp, vp, vp, vp, i, i, i64, d, vp,
                                         ctypes.c_size_t]
    L.ret_chunkwise_prepare.argtypes = [vp, vp, dp, i, i, i, i, i, i, vp, i, i, i64, d, vp, ctypes.c_size_t]
    L.ret_forward_chunkwise_prepared.argtypes = [vp, vp, vp, dp, i, i, i, i, i, i, vp, vp, vp, vp, i, i, i, i64, d,
                                                 vp, ctypes.c_size_t]
    L.ret_chunkwise_noalloc_max_bytes.argtypes = []
    L.ret_chunkwise_noalloc_max_bytes.restype = ctypes.c_size_t
    L.ret_chunkwise_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    L.ret_chunkwise_workspace_bytes.restype = ctypes.c_size_t
    L.ret_chunkwise_prepare_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    L.ret_chunkwise_prepare_workspace_bytes.restype = ctypes.c_size_t
    L.ret_decode_step.argtypes = [vp, vp, vp, dp, vp, vp, vp, i, i, i, i, i, i]
    L.ret_normalized_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    L.ret_normalized_workspace_bytes.restype = ctypes.c_size_t
    L.ret_forward_chunkwise_normalized.argtypes = [vp, vp, vp, dp, i, i, i, i, i, i, i, vp, vp, vp, vp, vp, vp, i,
                                                   i, i, i64, d, vp, ctypes.c_size_t]
    L.ret_decode_step_normalized.argtypes = [vp, vp, vp, dp, vp, vp, vp, i64, i, vp, i, i, i, i, i, i]
    L.ret_selftest_bounded_wait.argtypes = [ctypes.c_uint32, vp]
    L.ret_decode_step_positions.argtypes = [vp, vp, vp, dp, vp, vp, vp, vp, i, d, i, vp, i, i, i, i, i, i]
    L.ret_forward_parallel.argtypes = [vp, vp, vp, dp, i, i, i, i, i, vp, vp, i, i, i, i64, d]
    L.ret_forward_recurrent.argtypes = [vp, vp, vp, dp, i, i, i, i, i, vp, vp, vp, i, i, i, i64, d]
    L.ret_msr_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.ret_msr_workspace_bytes.restype = ctypes.c_size_t
    L.ret_msr_forward.argtypes = [vp, vp, vp, vp, vp, vp, dp, i, i, i, i, i, i, i, d, d, i, i64, d, vp, i, vp,
                                  ctypes.c_size_t, vp]
    L.ret_linear_bf16.argtypes = [vp, vp, vp, i, i, i, i, vp]
    L.ret_retnet_block_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    L.ret_retnet_block_workspace_bytes.restype = ctypes.c_size_t
    L.ret_retnet_block_forward.argtypes = [vp] * 12 + [dp, i, i, i, i, i, i, i, i, d, d, d, i, i64, d, vp, i, vp,
                                                       ctypes.c_size_t, vp]
    L.ret_rotary_frequencies.argtypes = [i, d, i, d, d, d, d, vp, dp]
    L.ret_rotary.argtypes = [vp] * 8 + [vp, d, vp, i64, i, i, i, i, i, i, i, i, i, vp]
    L.ret_layernorm_forward.argtypes = [vp, vp, vp, d, i64, i, vp, vp, vp, i, i, vp]
    L.ret_layernorm_backward_workspace_bytes.argtypes = [i64, i]
    L.ret_layernorm_backward_workspace_bytes.restype = ctypes.c_size_t
    L.ret_layernorm_backward.argtypes = [vp, vp, vp, vp, vp, i64, i, vp, vp, vp, i, i, vp, ctypes.c_size_t, vp]
    L.ret_delta_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    L.ret_delta_workspace_bytes.restype = ctypes.c_size_t
    L.ret_delta_forward_chunkwise.argtypes = [vp] * 7 + [i] * 6 + [vp, vp, vp, i, i, vp, ctypes.c_size_t]
    L.ret_delta_backward_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    L.ret_delta_backward_workspace_bytes.restype = ctypes.c_size_t
    L.ret_delta_backward_chunkwise.argtypes = [vp] * 9 + [i] * 6 + [vp] * 7 + [i, i, vp, ctypes.c_size_t]
    L.ret_delta_decode_step.argtypes = [vp] * 8 + [i] * 7
    L.ret_check_device_error.argtypes = [vp]
    L.ret_last_error_string.restype = ctypes.c_char_p
    L.ret_last_error_string.argtypes = []
    for name in ("ret_xpos_rotate", "ret_forward_chunkwise", "ret_forward_chunkwise_ws",
                 "ret_forward_chunkwise_noalloc", "ret_chunkwise_prepare", "ret_forward_chunkwise_prepared",
                 "ret_backward_chunkwise", "ret_decode_step",
                 "ret_forward_parallel",
                 "ret_forward_recurrent", "ret_check_device_error", "ret_msr_forward", "ret_linear_bf16"):
        getattr(L, name).restype = ctypes.c_int
    return L


lib = _load_library()


def _load_binding(path: str):
    """The short calls without Python on the way: a module built with the library,
    against one torch (its version is in the file's name)."""
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing (torch {torch.__version__}): build it with "
            "`python linear_recurrent_sequence_chunkwise_b200/build.py` (g++)")
    spec = importlib.util.spec_from_file_location(__name__ + "._binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


_binding = _load_binding(os.path.join(_HERE, f"_binding-torch{torch.__version__}.so"))


def ret_last_error_string() -> str:
    return lib.ret_last_error_string().decode(errors="replace")


def _check(status: int):
    if status != RET_OK:
        raise RetentionError(status, ret_last_error_string())


def _dt(t: torch.dtype) -> int:
    if t == torch.float32:
        return RET_F32
    if t == torch.bfloat16:
        return RET_BF16
    raise TypeError(f"unsupported dtype {t}; expected float32 or bfloat16")


def _ptr(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


F32 = (torch.float32,)
FLOATS = (torch.float32, torch.bfloat16)


def _buf(t: Optional[torch.Tensor], name: str, shape, dtypes, like: torch.Tensor):
    """A caller-provided buffer must have the shape and dtype the call reads or
    writes and sit on the inputs' device: the C ABI takes plain pointers and
    cannot check either."""
    if t is None:
        return
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)} (got {list(t.shape)})")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the inputs on {like.device}")


def _same_device(like: torch.Tensor, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != like.device:
            raise ValueError(f"{name} is on {t.device}, the inputs on {like.device}")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _gammas(gammas: Sequence[float], H: int):
    g = [float(x) for x in gammas]
    if len(g) != H:
        raise ValueError(f"gammas has {len(g)} entries, expected H={H}")
    return (ctypes.c_double * H)(*g)


def ret_xpos_rotate(x: torch.Tensor, pos_offset: int = 0, theta_base: float = 10000.0, stream=None) -> torch.Tensor:
    """Rotate x [B, N, H, d] in place (xPos / rotary, consecutive pairs)."""
    B, N, H, d = x.shape
    _check(lib.ret_xpos_rotate(_ptr(x, "x"), _dt(x.dtype), B, N, H, d, int(pos_offset), float(theta_base),
                               _stream(stream)))
    return x


def _seq_shapes(q, k, v):
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("expected q, k [B, N, H, dk] and v [B, N, H, dv]")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k and v must share a dtype")
    _same_device(q, k=k, v=v)
    B, N, H, dk = q.shape
    return B, N, H, dk, v.shape[3]


def _seq_outputs(q, out, final_state, B, N, H, dk, dv, initial_state=None):
    _buf(out, "out", (B, N, H, dv), FLOATS, q)
    _buf(final_state, "final_state", (B, H, dk, dv), F32, q)
    _buf(initial_state, "initial_state", (B, H, dk, dv), F32, q)


def ret_forward_chunkwise(q, k, v, gammas, chunk: int, out=None, final_state=None, out_dtype=None,
                          xpos: bool = False, pos_offset: int = 0, theta_base: float = 10000.0,
                          want_final_state: bool = False, stream=None):
    """Chunkwise retention forward.  Returns ``out`` [B, N, H, dv], or
    ``(out, final_state)`` when a final state is requested (passed in or
    ``want_final_state``)."""
    B, N, H, dk, dv = _seq_shapes(q, k, v)
    if out is None:
        out = torch.empty((B, N, H, dv), dtype=out_dtype or q.dtype, device=q.device)
    if final_state is None and want_final_state:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _seq_outputs(q, out, final_state, B, N, H, dk, dv)
    _check(lib.ret_forward_chunkwise(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _gammas(gammas, H), B, N, H, dk,
                                     dv, int(chunk), _ptr(out, "out"), _ptr(final_state, "final_state"),
                                     _stream(stream), _dt(q.dtype), _dt(out.dtype), int(bool(xpos)),
                                     int(pos_offset), float(theta_base)))
    return (out, final_state) if final_state is not None else out


def ret_chunkwise_workspace_bytes(B, N, H, dk, dv, chunk, dtype=torch.bfloat16, xpos: bool = False) -> int:
    """Workspace bytes ret_forward_chunkwise_ws needs for this shape (0: the
    shape does not take the workspace path)."""
    return int(lib.ret_chunkwise_workspace_bytes(B, N, H, dk, dv, int(chunk), _dt(dtype), int(bool(xpos))))


def ret_forward_chunkwise_ws(q, k, v, gammas, chunk: int, workspace, out=None, final_state=None, out_dtype=None,
                             xpos: bool = False, pos_offset: int = 0, theta_base: float = 10000.0,
                             want_final_state: bool = False, stream=None):
    """Chunkwise forward with a caller-provided workspace (a CUDA uint8 tensor
    of at least ret_chunkwise_workspace_bytes bytes)."""
    B, N, H, dk, dv = _seq_shapes(q, k, v)
    if out is None:
        out = torch.empty((B, N, H, dv), dtype=out_dtype or q.dtype, device=q.device)
    if final_state is None and want_final_state:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _seq_outputs(q, out, final_state, B, N, H, dk, dv)
    _same_device(q, workspace=workspace)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib.ret_forward_chunkwise_ws(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _gammas(gammas, H), B, N, H, dk,
                                        dv, int(chunk), _ptr(out, "out"), _ptr(final_state, "final_state"),
                                        _stream(stream), _dt(q.dtype), _dt(out.dtype), int(bool(xpos)),
                                        int(pos_offset), float(theta_base), _ptr(workspace, "workspace"), nbytes))
    return (out, final_state) if final_state is not None else out


def ret_chunkwise_prepare_workspace_bytes(B, N, H, dk, dv, chunk, dtype=torch.bfloat16, xpos: bool = False) -> int:
    """Workspace bytes of ret_chunkwise_prepare / ret_forward_chunkwise_prepared (0: shape not on that path)."""
    return int(lib.ret_chunkwise_prepare_workspace_bytes(B, N, H, dk, dv, chunk, _dt(dtype), int(bool(xpos))))


def ret_chunkwise_prepare(q, k, gammas, chunk: int, workspace, dv: int, xpos: bool = False, pos_offset: int = 0,
                          theta_base: float = 10000.0, stream=None):
    """First pass of the workspace path: rotated queries (xpos) and rotated,
    zeta-scaled keys into ``workspace``."""
    if q.shape != k.shape or q.dim() != 4:
        raise ValueError("q and k must both be [B, N, H, dk]")
    B, N, H, dk = q.shape
    _same_device(q, k=k, workspace=workspace)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib.ret_chunkwise_prepare(_ptr(q, "q"), _ptr(k, "k"), _gammas(gammas, H), B, N, H, dk, int(dv),
                                     int(chunk), _stream(stream), _dt(q.dtype), int(bool(xpos)), int(pos_offset),
                                     float(theta_base), _ptr(workspace, "workspace"), nbytes))


def ret_forward_chunkwise_prepared(q, k, v, gammas, chunk: int, workspace, out=None, final_state=None,
                                   initial_state=None, out_dtype=None, xpos: bool = False, pos_offset: int = 0,
                                   theta_base: float = 10000.0, want_final_state: bool = False, stream=None):
    """Second pass of the workspace path on a workspace filled by
    ret_chunkwise_prepare with the same arguments; ``initial_state`` (fp32
    [B, H, dk, dv], or None for zero) continues a sequence."""
    B, N, H, dk, dv = _seq_shapes(q, k, v)
    if out is None:
        out = torch.empty((B, N, H, dv), dtype=out_dtype or q.dtype, device=q.device)
    if final_state is None and want_final_state:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _seq_outputs(q, out, final_state, B, N, H, dk, dv, initial_state)
    _same_device(q, workspace=workspace)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib.ret_forward_chunkwise_prepared(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _gammas(gammas, H), B, N,
                                              H, dk, dv, int(chunk), _ptr(out, "out"),
                                              _ptr(final_state, "final_state"),
                                              _ptr(initial_state, "initial_state"), _stream(stream), _dt(q.dtype),
                                              _dt(out.dtype), int(bool(xpos)), int(pos_offset), float(theta_base),
                                              _ptr(workspace, "workspace"), nbytes))
    return (out, final_state) if final_state is not None else out


def ret_backward_workspace_bytes(B, N, H, dk, dv, chunk, in_dtype=torch.bfloat16, xpos: bool = False) -> int:
    """Workspace bytes of ret_backward_chunkwise (0: shape not supported)."""
    return int(lib.ret_backward_workspace_bytes(B, N, H, dk, dv, int(chunk), _dt(in_dtype), int(bool(xpos))))


def ret_backward_chunkwise(q, k, v, dout, gammas, chunk: int, workspace=None, dq=None, dk=None, dv=None,
                           xpos: bool = False, pos_offset: int = 0, theta_base: float = 10000.0, stream=None):
    """Gradients (dq, dk, dv) in fp32 of sum(out * dout) for the chunkwise
    forward of the same arguments."""
    B, N, H, dk_, dv_ = _seq_shapes(q, k, v)
    _buf(dout, "dout", (B, N, H, dv_), (q.dtype,), q)
    dq = torch.empty((B, N, H, dk_), dtype=torch.float32, device=q.device) if dq is None else dq
    dk = torch.empty((B, N, H, dk_), dtype=torch.float32, device=q.device) if dk is None else dk
    dv = torch.empty((B, N, H, dv_), dtype=torch.float32, device=q.device) if dv is None else dv
    if workspace is None:
        nb = ret_backward_workspace_bytes(B, N, H, dk_, dv_, chunk, q.dtype, xpos)
        workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=q.device)
    _buf(dq, "dq", (B, N, H, dk_), F32, q)
    _buf(dk, "dk", (B, N, H, dk_), F32, q)
    _buf(dv, "dv", (B, N, H, dv_), F32, q)
    _same_device(q, workspace=workspace)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib.ret_backward_chunkwise(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _ptr(dout, "dout"),
                                      _gammas(gammas, H), B, N, H, dk_, dv_, int(chunk), _ptr(dq, "dq"),
                                      _ptr(dk, "dk"), _ptr(dv, "dv"), _stream(stream), _dt(q.dtype),
                                      int(bool(xpos)), int(pos_offset), float(theta_base),
                                      _ptr(workspace, "workspace"), nbytes))
    return dq, dk, dv


def ret_chunkwise_noalloc_max_bytes() -> int:
    """Bytes of the library's fixed scratch array used by
    ret_forward_chunkwise_noalloc."""
    return int(lib.ret_chunkwise_noalloc_max_bytes())


def ret_forward_chunkwise_noalloc(q, k, v, gammas, chunk: int, out=None, final_state=None, out_dtype=None,
                                  xpos: bool = False, pos_offset: int = 0, theta_base: float = 10000.0,
                                  want_final_state: bool = False, stream=None):
    """Chunkwise forward whose scratch is a fixed device array inside the
    library: for callers that cannot allocate device memory at call time.
    Pass ``out`` / ``final_state`` to avoid the allocations this wrapper would
    otherwise make for them."""
    B, N, H, dk, dv = _seq_shapes(q, k, v)
    if out is None:
        out = torch.empty((B, N, H, dv), dtype=out_dtype or q.dtype, device=q.device)
    if final_state is None and want_final_state:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _seq_outputs(q, out, final_state, B, N, H, dk, dv)
    _check(lib.ret_forward_chunkwise_noalloc(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _gammas(gammas, H), B, N,
                                             H, dk, dv, int(chunk), _ptr(out, "out"),
                                             _ptr(final_state, "final_state"), _stream(stream), _dt(q.dtype),
                                             _dt(out.dtype), int(bool(xpos)), int(pos_offset), float(theta_base)))
    return (out, final_state) if final_state is not None else out


def ret_forward_parallel(q, k, v, gammas, out=None, out_dtype=None, xpos: bool = False, pos_offset: int = 0,
                         theta_base: float = 10000.0, stream=None):
    """Parallel form (Q K^T (.) D) V, for cross-checks.  Returns ``out``."""
    B, N, H, dk, dv = _seq_shapes(q, k, v)
    if out is None:
        out = torch.empty((B, N, H, dv), dtype=out_dtype or q.dtype, device=q.device)
    _seq_outputs(q, out, None, B, N, H, dk, dv)
    _check(lib.ret_forward_parallel(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _gammas(gammas, H), B, N, H, dk,
                                    dv, _ptr(out, "out"), _stream(stream), _dt(q.dtype), _dt(out.dtype),
                                    int(bool(xpos)), int(pos_offset), float(theta_base)))
    return out


def ret_forward_recurrent(q, k, v, gammas, out=None, final_state=None, out_dtype=None, xpos: bool = False,
                          pos_offset: int = 0, theta_base: float = 10000.0, want_final_state: bool = False,
                          stream=None):
    """Recurrent form token by token, for cross-checks."""
    B, N, H, dk, dv = _seq_shapes(q, k, v)
    if out is None:
        out = torch.empty((B, N, H, dv), dtype=out_dtype or q.dtype, device=q.device)
    if final_state is None and want_final_state:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _seq_outputs(q, out, final_state, B, N, H, dk, dv)
    _check(lib.ret_forward_recurrent(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _gammas(gammas, H), B, N, H, dk,
                                     dv, _ptr(out, "out"), _ptr(final_state, "final_state"), _stream(stream),
                                     _dt(q.dtype), _dt(out.dtype), int(bool(xpos)), int(pos_offset),
                                     float(theta_base)))
    return (out, final_state) if final_state is not None else out


def _step_shapes(q, k, v, state):
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise ValueError("expected q, k [B, H, dk] and v [B, H, dv]")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k and v must share a dtype")
    _same_device(q, k=k, v=v)
    B, H, dk = q.shape
    dv = v.shape[2]
    if state is None:
        raise ValueError("state must be float32 [B, H, dk, dv]")
    _buf(state, "state", (B, H, dk, dv), F32, q)
    return B, H, dk, dv


def ret_decode_step(q, k, v, gammas, state, out=None, out_dtype=None, stream=None):
    """One decode step: state [B, H, dk, dv] fp32 updated in place; returns
    out [B, H, dv]."""
    B, H, dk, dv = _step_shapes(q, k, v, state)
    if out is None:
        out = torch.empty((B, H, dv), dtype=out_dtype or torch.float32, device=q.device)
    _buf(out, "out", (B, H, dv), FLOATS, q)
    _check(lib.ret_decode_step(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _gammas(gammas, H),
                               _ptr(state, "state"), _ptr(out, "out"), _stream(stream), B, H, dk, dv,
                               _dt(q.dtype), _dt(out.dtype)))
    return out


NORM_DECAY = 1  # RET_NORM_DECAY
NORM_SCORE = 2  # RET_NORM_SCORE


def ret_normalized_workspace_bytes(B, N, H, dk, dv, chunk, in_dtype=torch.bfloat16, xpos: bool = False) -> int:
    """Workspace bytes of ret_forward_chunkwise_normalized (0: shape not supported)."""
    return int(lib.ret_normalized_workspace_bytes(B, N, H, dk, dv, int(chunk), _dt(in_dtype), int(bool(xpos))))


def ret_forward_chunkwise_normalized(q, k, v, gammas, chunk: int, norm_flags: int = NORM_DECAY | NORM_SCORE,
                                     workspace=None, out=None, out_dtype=None, initial_state=None,
                                     final_state=None, initial_z=None, final_z=None, xpos: bool = False,
                                     pos_offset: int = 0, theta_base: float = 10000.0, stream=None):
    """Chunkwise forward with the score normalizations (norm_flags: NORM_DECAY,
    NORM_SCORE); states S [B, H, dk, dv] and z [B, H, dk] fp32, optional."""
    B, N, H, dk, dv = _seq_shapes(q, k, v)
    if out is None:
        out = torch.empty((B, N, H, dv), dtype=out_dtype or q.dtype, device=q.device)
    _seq_outputs(q, out, final_state, B, N, H, dk, dv, initial_state)
    _buf(initial_z, "initial_z", (B, H, dk), F32, q)
    _buf(final_z, "final_z", (B, H, dk), F32, q)
    if workspace is None:
        nb = ret_normalized_workspace_bytes(B, N, H, dk, dv, chunk, q.dtype, xpos)
        workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=q.device)
    _same_device(q, workspace=workspace)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib.ret_forward_chunkwise_normalized(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _gammas(gammas, H), B, N,
                                                H, dk, dv, int(chunk), int(norm_flags), _ptr(out, "out"),
                                                _ptr(initial_state, "initial_state"), _ptr(final_state, "final_state"),
                                                _ptr(initial_z, "initial_z"), _ptr(final_z, "final_z"),
                                                _stream(stream), _dt(q.dtype), _dt(out.dtype), int(bool(xpos)),
                                                int(pos_offset), float(theta_base), _ptr(workspace, "workspace"),
                                                nbytes))
    return out


def ret_decode_step_normalized(q, k, v, gammas, state, z, position: int, norm_flags: int = NORM_DECAY | NORM_SCORE,
                               out=None, out_dtype=None, stream=None):
    """One decode step with the score normalizations at 0-based ``position``:
    state [B, H, dk, dv] and z [B, H, dk] (fp32) updated in place."""
    B, H, dk, dv = _step_shapes(q, k, v, state)
    _buf(z, "z", (B, H, dk), F32, q)
    if out is None:
        out = torch.empty((B, H, dv), dtype=out_dtype or torch.float32, device=q.device)
    _buf(out, "out", (B, H, dv), FLOATS, q)
    _check(lib.ret_decode_step_normalized(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _gammas(gammas, H),
                                          _ptr(state, "state"), _ptr(z, "z"), _ptr(out, "out"), int(position),
                                          int(norm_flags), _stream(stream), B, H, dk, dv, _dt(q.dtype),
                                          _dt(out.dtype)))
    return out


def ret_decode_step_positions(q, k, v, gammas, state, positions, z=None, xpos: bool = True,
                              theta_base: float = 10000.0, norm_flags: int = 0, out=None, out_dtype=None,
                              stream=None):
    """One decode step with each sequence at its own position: positions int64
    [B] on the device; xPos rotation of q, k inside the step; optional score
    normalizations with z [B, H, dk] fp32 (in place)."""
    B, H, dk, dv = _step_shapes(q, k, v, state)
    _buf(positions, "positions", (B,), (torch.int64,), q)
    _buf(z, "z", (B, H, dk), F32, q)
    if out is None:
        out = torch.empty((B, H, dv), dtype=out_dtype or torch.float32, device=q.device)
    _buf(out, "out", (B, H, dv), FLOATS, q)
    _check(lib.ret_decode_step_positions(_ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _gammas(gammas, H),
                                         _ptr(state, "state"), _ptr(z, "z"), _ptr(out, "out"),
                                         _ptr(positions, "positions"), int(bool(xpos)), float(theta_base),
                                         int(norm_flags), _stream(stream), B, H, dk, dv, _dt(q.dtype),
                                         _dt(out.dtype)))
    return out


def ret_selftest_bounded_wait(polls: int = 1 << 12, stream=None):
    """Run the bounded-wait self-test: the next ret_check_device_error raises
    with RET_ERR_TIMEOUT."""
    _check(lib.ret_selftest_bounded_wait(int(polls), _stream(stream)))


def ret_check_device_error(stream=None):
    """Synchronise the stream and raise if a kernel gave up a bounded wait."""
    _check(lib.ret_check_device_error(_stream(stream)))


BF16 = (torch.bfloat16,)


def _msr_shapes(x, wq, wk, wv, wg, wo, H: int):
    """B, N, d_model, dk, dv of an MSR layer from x [B, N, d_model] and the
    (input, output) weights W_Q, W_K [d_model, H dk], W_V, W_G [d_model, H dv],
    W_O [H dv, d_model], all bf16 on x's device."""
    if x.dim() != 3 or x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16 [B, N, d_model]")
    B, N, dm = x.shape
    if H < 1 or wq.dim() != 2 or wv.dim() != 2 or wq.shape[1] % H or wv.shape[1] % H:
        raise ValueError("W_Q and W_V must be [d_model, H * d] with H dividing their widths")
    dk, dv = wq.shape[1] // H, wv.shape[1] // H
    _buf(wq, "wq", (dm, H * dk), BF16, x)
    _buf(wk, "wk", (dm, H * dk), BF16, x)
    _buf(wv, "wv", (dm, H * dv), BF16, x)
    _buf(wg, "wg", (dm, H * dv), BF16, x)
    _buf(wo, "wo", (H * dv, dm), BF16, x)
    return B, N, dm, dk, dv


def ret_retnet_block_workspace_bytes(B, N, dmodel, H, dk, dv, dff) -> int:
    return int(lib.ret_retnet_block_workspace_bytes(B, N, dmodel, H, dk, dv, dff))


def ret_retnet_block_forward(x, wq, wk, wv, wg, wo, w1, w2, gammas, H: int, ln1_gain=None, ln1_bias=None,
                             ln2_gain=None, ln2_bias=None, chunk: int = 128, k_scale: float = 1.0,
                             gn_eps: float = 1e-5, ln_eps: float = 1e-5, xpos: bool = True, pos_offset: int = 0,
                             theta_base: float = 10000.0, out=None, out_dtype=torch.bfloat16, workspace=None,
                             stream=None):
    """One pre-LayerNorm RetNet block: Y = MSR(LN1(x)) + x, out = gelu(LN2(Y) W1) W2 + Y.
    x [B, N, d_model] bf16; weights bf16 [in, out]; LayerNorm gains/biases bf16
    [d_model] or None (1 / 0)."""
    B, N, dm, dk, dv = _msr_shapes(x, wq, wk, wv, wg, wo, H)
    dff = w1.shape[1]
    _buf(w1, "w1", (dm, dff), BF16, x)
    _buf(w2, "w2", (dff, dm), BF16, x)
    for name, t in (("ln1_gain", ln1_gain), ("ln1_bias", ln1_bias), ("ln2_gain", ln2_gain), ("ln2_bias", ln2_bias)):
        _buf(t, name, (dm,), BF16, x)
    if out is None:
        out = torch.empty((B, N, dm), dtype=out_dtype, device=x.device)
    _buf(out, "out", (B, N, dm), FLOATS, x)
    if workspace is None:
        workspace = torch.empty(ret_retnet_block_workspace_bytes(B, N, dm, H, dk, dv, dff), dtype=torch.uint8,
                                device=x.device)
    _same_device(x, workspace=workspace)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib.ret_retnet_block_forward(_ptr(x, "x"), _ptr(ln1_gain, "ln1_gain"), _ptr(ln1_bias, "ln1_bias"),
                                        _ptr(wq, "wq"), _ptr(wk, "wk"), _ptr(wv, "wv"), _ptr(wg, "wg"),
                                        _ptr(wo, "wo"), _ptr(ln2_gain, "ln2_gain"), _ptr(ln2_bias, "ln2_bias"),
                                        _ptr(w1, "w1"), _ptr(w2, "w2"), _gammas(gammas, H), B, N, dm, H, dk, dv,
                                        dff, int(chunk), float(k_scale), float(gn_eps), float(ln_eps),
                                        int(bool(xpos)), int(pos_offset), float(theta_base), _ptr(out, "out"),
                                        _dt(out.dtype), _ptr(workspace, "workspace"), nbytes, _stream(stream)))
    return out


def ret_linear_bf16(x, w, out=None, out_dtype=torch.bfloat16, stream=None):
    """Y = X W on the tensor cores; x [..., K] bf16, w [K, N] bf16."""
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("x and w must be bfloat16")
    K = x.shape[-1]
    if w.dim() != 2 or w.shape[0] != K:
        raise ValueError("w must be [K, N]")
    N = w.shape[1]
    M = x.numel() // K
    _same_device(x, w=w)
    if out is None:
        out = torch.empty((*x.shape[:-1], N), dtype=out_dtype, device=x.device)
    _buf(out, "out", (*x.shape[:-1], N), FLOATS, x)
    _check(lib.ret_linear_bf16(_ptr(x, "x"), _ptr(w, "w"), _ptr(out, "out"), M, N, K, _dt(out.dtype),
                               _stream(stream)))
    return out


def ret_msr_workspace_bytes(B, N, dmodel, H, dk, dv) -> int:
    return int(lib.ret_msr_workspace_bytes(B, N, dmodel, H, dk, dv))


def ret_msr_forward(x, wq, wk, wv, wg, wo, gammas, H: int, chunk: int = 128, k_scale: float = 1.0,
                    eps: float = 1e-5, xpos: bool = True, pos_offset: int = 0, theta_base: float = 10000.0,
                    out=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """MultiScaleRetention layer forward.  x [B, N, d_model] bf16; weights
    bf16 [in, out]; returns out [B, N, d_model]."""
    B, N, dm, dk, dv = _msr_shapes(x, wq, wk, wv, wg, wo, H)
    if out is None:
        out = torch.empty((B, N, dm), dtype=out_dtype, device=x.device)
    _buf(out, "out", (B, N, dm), FLOATS, x)
    need = ret_msr_workspace_bytes(B, N, dm, H, dk, dv)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _same_device(x, workspace=workspace)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib.ret_msr_forward(_ptr(x, "x"), _ptr(wq, "wq"), _ptr(wk, "wk"), _ptr(wv, "wv"), _ptr(wg, "wg"),
                               _ptr(wo, "wo"), _gammas(gammas, H), B, N, dm, H, dk, dv, int(chunk), float(k_scale),
                               float(eps), int(bool(xpos)), int(pos_offset), float(theta_base), _ptr(out, "out"),
                               _dt(out.dtype), _ptr(workspace, "workspace"), nbytes, _stream(stream)))
    return out


# ------------------------------------------------- rotary, layer norm, delta rule

def _call(like: torch.Tensor, stream, fn, *args):
    """Call ``fn(*args)`` with ``like``'s device current; the argument
    ``_STREAM`` stands for the stream (default: that device's current one)."""
    if not like.is_cuda:
        raise ValueError("the inputs must be CUDA tensors")
    dev = like.get_device()
    # the plain handle: making a Stream object costs as much as a launch
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    args = [s if a is _STREAM else a for a in args]
    if dev == torch._C._cuda_getDevice():
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status != RET_OK:
        _check(status)


def _new(like: torch.Tensor, shape, dtype, stream):
    """An output or workspace that a call makes itself, on ``like``'s device.  It
    belongs to the call's stream: on another stream its memory could still be in use
    by work before it, and be free again (a workspace: when the call returns) before
    the call's kernels have run."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _workspace(workspace, need: int, like: torch.Tensor, stream):
    """(pointer, bytes) of the caller's workspace, or of a new one, and the
    tensor that holds it."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = _new(like, (need,), torch.uint8, stream)
    else:
        _same_device(like, workspace=workspace)
    return _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(), workspace


_STREAM = object()
_CODES = {torch.float32: RET_F32, torch.bfloat16: RET_BF16}
_Strides = ctypes.c_int64 * 3

_ROTARY_LAYOUTS = {"interleaved": 0, "half": 1}
_ROTARY_SCALINGS = {"none": 0, "linear": 1, "yarn": 2}


def ret_rotary_frequencies(rotary_dim: int, theta_base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                           original_length: float = 4096.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(freqs, scale) for ret_rotary: the angle per position of each pair
    (float64 [rotary_dim / 2] on the CPU) and the factor on cos and sin, plain
    or stretched for longer contexts (``scaling`` "none", "linear", "yarn")."""
    if scaling not in _ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_ROTARY_SCALINGS)} (got {scaling!r})")
    freqs = torch.empty(max(int(rotary_dim), 2) // 2, dtype=torch.float64)
    scale = ctypes.c_double()
    _check(lib.ret_rotary_frequencies(int(rotary_dim), float(theta_base), _ROTARY_SCALINGS[scaling], float(factor),
                                      float(original_length), float(beta_fast), float(beta_slow),
                                      ctypes.c_void_p(freqs.data_ptr()), ctypes.byref(scale)))
    return freqs, scale.value


def _rotary_view(t: Optional[torch.Tensor], name: str):
    """(pointer, strides) of a [B, N, heads, d] view with consecutive components."""
    if t is None:
        return None, None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.is_contiguous():
        return t.data_ptr(), None
    if t.stride(3) != 1 and t.shape[3] > 1:
        raise ValueError(f"the components of {name} must be consecutive (stride {t.stride(3)})")
    return t.data_ptr(), _Strides(*t.stride()[:3])


def ret_rotary(q, k=None, freqs=None, positions=None, pos_offset: int = 0, layout: str = "interleaved",
               scale: float = 1.0, rotary_dim: Optional[int] = None, theta_base: float = 10000.0, inverse: bool = False,
               q_out=None, k_out=None, stream=None):
    """Rotary positions on q [B, N, H, d] and k [B, N, Hk, d] (or None):
    ``freqs`` from ret_rotary_frequencies (its length sets the turned part of
    the head), or None for the plain ones of ``rotary_dim`` (default d) and
    ``theta_base``; ``positions`` int64 [B, N] on the device, or token n at
    pos_offset + n; layout "interleaved" or "half".  Views with consecutive
    components are taken as they are; pass ``q_out=q`` to work in place.
    ``inverse=True`` is the transpose (the gradient).  Returns the output, or
    the pair of them."""
    if q_out is k_out is stream is None and freqs is not None and rotary_dim is None and layout in _ROTARY_LAYOUTS:
        r = _binding.rotary(q, k, freqs, positions, pos_offset, layout == "half", scale, inverse)
        if r is not None:
            return r if r.__class__ is not int else _check(r)
    if layout not in _ROTARY_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_ROTARY_LAYOUTS)} (got {layout!r})")
    if q.dim() != 4 or (k is not None and (k.dim() != 4 or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3])):
        raise ValueError("expected q [B, N, H, d] and k [B, N, Hk, d]")
    if k is not None and k.dtype != q.dtype:
        raise TypeError("q and k must share a dtype")
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    B, N, H, d = q.shape
    Hk = k.shape[2] if k is not None else 0
    if freqs is None:
        freqs, _ = ret_rotary_frequencies(d if rotary_dim is None else rotary_dim, theta_base)
    elif not isinstance(freqs, torch.Tensor):
        freqs = torch.tensor([float(f) for f in freqs], dtype=torch.float64)
    if freqs.dim() != 1 or freqs.dtype != torch.float64 or freqs.is_cuda or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 vector on the CPU")
    if rotary_dim is not None and 2 * freqs.numel() != rotary_dim:
        raise ValueError(f"freqs has {freqs.numel()} entries, expected {rotary_dim // 2}")
    if q_out is None:
        q_out = _new(q, (B, N, H, d), q.dtype, stream)
    else:
        _buf(q_out, "q_out", (B, N, H, d), (q.dtype,), q)
    if k is not None:
        _same_device(q, k=k)
        if k_out is None:
            k_out = _new(q, (B, N, Hk, d), q.dtype, stream)
        else:
            _buf(k_out, "k_out", (B, N, Hk, d), (q.dtype,), q)
    _buf(positions, "positions", (B, N), (torch.int64,), q)
    (qp, qs), (kp, ks) = _rotary_view(q, "q"), _rotary_view(k, "k")
    (qop, qos), (kop, kos) = _rotary_view(q_out, "q_out"), _rotary_view(k_out, "k_out")
    _call(q, stream, lib.ret_rotary, qp, kp, qop, kop, qs, ks, qos, kos, freqs.data_ptr(),
          float(scale), _ptr(positions, "positions"), int(pos_offset), int(bool(inverse)), _ROTARY_LAYOUTS[layout],
          B, N, H, Hk, d, 2 * freqs.numel(), _dt(q.dtype), _STREAM)
    return q_out if k is None else (q_out, k_out)


def _weight_dt(x, d, gain, bias=None):
    """dtype code of the layer norm's weights (fp32 or bf16, the same for both)."""
    _buf(gain, "gain", (d,), FLOATS, x)
    _buf(bias, "bias", (d,), FLOATS, x)
    if gain is not None and bias is not None and gain.dtype != bias.dtype:
        raise TypeError("gain and bias must share a dtype")
    given = bias if gain is None else gain
    return RET_F32 if given is None else _CODES[given.dtype]


def ret_layernorm_forward(x, gain=None, bias=None, eps: float = 1e-5, out=None, mean=None, rstd=None,
                          want_stats: bool = False, stream=None):
    """Layer norm over the last dimension of x [..., d]; gain, bias [d] or None.
    Returns the output, or (out, mean, rstd) (fp32, one per row) when the
    statistics are passed in or wanted."""
    if out is mean is rstd is stream is None:
        r = _binding.layernorm_forward(x, gain, bias, eps, want_stats)
        if r is not None:
            return r if r.__class__ is not int else _check(r)
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError("x must be [..., d] with at least one row")
    d, lead = x.shape[-1], x.shape[:-1]
    rows = x.numel() // d
    w = _weight_dt(x, d, gain, bias)
    if out is None:
        out = _new(x, x.shape, x.dtype, stream)
    else:
        _buf(out, "out", x.shape, (x.dtype,), x)
    _buf(mean, "mean", lead, F32, x)
    _buf(rstd, "rstd", lead, F32, x)
    if want_stats:
        mean = _new(x, lead, torch.float32, stream) if mean is None else mean
        rstd = _new(x, lead, torch.float32, stream) if rstd is None else rstd
    _call(x, stream, lib.ret_layernorm_forward, _ptr(x, "x"), _ptr(gain, "gain"), _ptr(bias, "bias"), float(eps), rows,
          d, _ptr(out, "out"), _ptr(mean, "mean"), _ptr(rstd, "rstd"), _dt(x.dtype), w, _STREAM)
    return (out, mean, rstd) if mean is not None or rstd is not None else out


def ret_layernorm_backward_workspace_bytes(rows: int, d: int) -> int:
    """Workspace bytes of ret_layernorm_backward's weight gradients."""
    return int(lib.ret_layernorm_backward_workspace_bytes(int(rows), int(d)))


def ret_layernorm_backward(dout, x, mean, rstd, gain=None, dx=None, dgain=None, dbias=None, want_weights: bool = True,
                           workspace=None, stream=None):
    """Gradients (dx, dgain, dbias) of ret_layernorm_forward for dout = dL/dout
    and its mean and rstd; dgain and dbias fp32 [d] (None without
    ``want_weights``, unless passed in)."""
    if dx is dgain is dbias is workspace is stream is None and want_weights:
        r = _binding.layernorm_backward(dout, x, mean, rstd, gain)
        if r is not None:
            return r if r.__class__ is not int else _check(r)
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError("x must be [..., d] with at least one row")
    d, lead = x.shape[-1], x.shape[:-1]
    rows = x.numel() // d
    w = _weight_dt(x, d, gain)
    _buf(dout, "dout", x.shape, (x.dtype,), x)
    _buf(mean, "mean", lead, F32, x)
    _buf(rstd, "rstd", lead, F32, x)
    _buf(dgain, "dgain", (d,), F32, x)
    _buf(dbias, "dbias", (d,), F32, x)
    if dx is None:
        dx = _new(x, x.shape, x.dtype, stream)
    else:
        _buf(dx, "dx", x.shape, (x.dtype,), x)
    if want_weights:
        dgain = _new(x, (d,), torch.float32, stream) if dgain is None else dgain
        dbias = _new(x, (d,), torch.float32, stream) if dbias is None else dbias
    wanted = workspace is None and (dgain is not None or dbias is not None)
    need = lib.ret_layernorm_backward_workspace_bytes(rows, d) if wanted else 0
    wp, nbytes, workspace = _workspace(workspace, need, x, stream)
    _call(x, stream, lib.ret_layernorm_backward, _ptr(dout, "dout"), _ptr(x, "x"), _ptr(mean, "mean"),
          _ptr(rstd, "rstd"), _ptr(gain, "gain"), rows, d, _ptr(dx, "dx"), _ptr(dgain, "dgain"), _ptr(dbias, "dbias"),
          _dt(x.dtype), w, wp, nbytes, _STREAM)
    return dx, dgain, dbias


def _delta_shapes(q, k, v, g, beta, n_lead: int):
    """Sizes of a delta-rule call; q, k [*lead, Hk, dk], v [*lead, H, dv], g and beta [*lead, H] fp32."""
    lead = q.shape[:n_lead]
    if q.dim() != n_lead + 2 or k.shape != q.shape or v.dim() != n_lead + 2 or v.shape[:n_lead] != lead:
        raise ValueError("expected q, k [B, N, Hk, dk] and v [B, N, H, dv]" if n_lead == 2 else
                         "expected q, k [B, Hk, dk] and v [B, H, dv]")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k and v must share a dtype")
    _same_device(q, k=k, v=v)
    H, dv = v.shape[n_lead:]
    gates = (*lead, H)
    _buf(g, "g", gates, F32, q)
    _buf(beta, "beta", gates, F32, q)
    Hk, dk = q.shape[n_lead:]
    return lead, Hk, H, dk, dv


def ret_delta_workspace_bytes(B, N, Hk, H, dk, dv, dtype=torch.bfloat16) -> int:
    """Workspace bytes of ret_delta_forward_chunkwise (0: none needed)."""
    return int(lib.ret_delta_workspace_bytes(B, N, Hk, H, dk, dv, _dt(dtype)))


def ret_delta_forward_chunkwise(q, k, v, g, beta, lengths=None, initial_state=None, out=None, final_state=None,
                                out_dtype=None, want_final_state: bool = False, workspace=None, stream=None):
    """Gated delta rule over a (padded) batch of sequences: q, k [B, N, Hk, dk],
    v [B, N, H, dv], g (log decay) and beta [B, N, H] fp32, lengths int32 [B] on
    the device or None, states [B, H, dk, dv] fp32.  Returns ``out`` [B, N, H, dv]
    (rows behind a sequence's end are not written), or ``(out, final_state)``
    when a final state is requested (passed in or ``want_final_state``)."""
    if final_state is workspace is stream is None and (out_dtype is None or out_dtype in FLOATS):
        r = _binding.delta_forward(q, k, v, g, beta, lengths, initial_state, out,
                                   (out_dtype or q.dtype) is torch.bfloat16, want_final_state)
        if r is not None:
            return r if r.__class__ is not int else _check(r)
    (B, N), Hk, H, dk, dv = _delta_shapes(q, k, v, g, beta, 2)
    _seq_outputs(q, out, final_state, B, N, H, dk, dv, initial_state)
    _buf(lengths, "lengths", (B,), (torch.int32,), q)
    if out is None:
        out = _new(q, (B, N, H, dv), out_dtype or q.dtype, stream)
    if final_state is None and want_final_state:
        final_state = _new(q, (B, H, dk, dv), torch.float32, stream)
    need = lib.ret_delta_workspace_bytes(B, N, Hk, H, dk, dv, _dt(q.dtype)) if workspace is None else 0
    wp, nbytes, workspace = _workspace(workspace, need, q, stream)
    _call(q, stream, lib.ret_delta_forward_chunkwise, _ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _ptr(g, "g"),
          _ptr(beta, "beta"), _ptr(lengths, "lengths"), _ptr(initial_state, "initial_state"), B, N, Hk, H, dk, dv,
          _ptr(out, "out"), _ptr(final_state, "final_state"), _STREAM, _dt(q.dtype), _dt(out.dtype), wp, nbytes)
    return (out, final_state) if final_state is not None else out


def ret_delta_decode_step(q, k, v, g, beta, state, out=None, out_dtype=None, stream=None):
    """One token of the gated delta rule: q, k [B, Hk, dk], v [B, H, dv], g and
    beta [B, H] fp32, state [B, H, dk, dv] fp32 updated in place; returns out
    [B, H, dv]."""
    if out is stream is None and (out_dtype is None or out_dtype in FLOATS):
        r = _binding.delta_decode_step(q, k, v, g, beta, state, out_dtype is torch.bfloat16)
        if r is not None:
            return r if r.__class__ is not int else _check(r)
    (B,), Hk, H, dk, dv = _delta_shapes(q, k, v, g, beta, 1)
    if state is None:
        raise ValueError("state must be float32 [B, H, dk, dv]")
    _buf(state, "state", (B, H, dk, dv), F32, q)
    if out is None:
        out = _new(q, (B, H, dv), out_dtype or torch.float32, stream)
    else:
        _buf(out, "out", (B, H, dv), FLOATS, q)
    _call(q, stream, lib.ret_delta_decode_step, _ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _ptr(g, "g"),
          _ptr(beta, "beta"), _ptr(state, "state"), _ptr(out, "out"), _STREAM, B, Hk, H, dk, dv, _dt(q.dtype),
          _dt(out.dtype))
    return out


def ret_delta_backward_workspace_bytes(B, N, Hk, H, dk, dv, dtype=torch.bfloat16) -> int:
    """Workspace bytes of ret_delta_backward_chunkwise (0: shape not supported)."""
    return int(lib.ret_delta_backward_workspace_bytes(B, N, Hk, H, dk, dv, _dt(dtype)))


def ret_delta_backward_chunkwise(q, k, v, g, beta, dout, lengths=None, initial_state=None, dfinal_state=None, dq=None,
                                 dk=None, dv=None, dg=None, dbeta=None, dinitial_state=None, grad_dtype=torch.float32,
                                 want_dinitial_state: Optional[bool] = None, workspace=None, stream=None):
    """Gradients of ret_delta_forward_chunkwise for dout = dL/dout and
    dfinal_state = dL/dfinal_state (or None): (dq, dk, dv, dg, dbeta,
    dinitial_state); dq, dk, dv of ``grad_dtype``, the others fp32.
    dinitial_state is None unless an initial state is given, it is passed in
    or wanted."""
    if dq is dk is dv is dg is dbeta is dinitial_state is workspace is stream is None and grad_dtype in FLOATS:
        r = _binding.delta_backward(q, k, v, g, beta, lengths, initial_state, dout, dfinal_state, grad_dtype is torch.bfloat16,
                                    initial_state is not None if want_dinitial_state is None else want_dinitial_state)
        if r is not None:
            return r if r.__class__ is not int else _check(r)
    (B, N), Hk, H, dk_, dv_ = _delta_shapes(q, k, v, g, beta, 2)
    _buf(dout, "dout", (B, N, H, dv_), (q.dtype,), q)
    _buf(initial_state, "initial_state", (B, H, dk_, dv_), F32, q)
    _buf(dfinal_state, "dfinal_state", (B, H, dk_, dv_), F32, q)
    _buf(lengths, "lengths", (B,), (torch.int32,), q)
    dq = _new(q, (B, N, Hk, dk_), grad_dtype, stream) if dq is None else dq
    _buf(dq, "dq", (B, N, Hk, dk_), FLOATS, q)
    _buf(dk, "dk", (B, N, Hk, dk_), (dq.dtype,), q)
    _buf(dv, "dv", (B, N, H, dv_), (dq.dtype,), q)
    _buf(dg, "dg", (B, N, H), F32, q)
    _buf(dbeta, "dbeta", (B, N, H), F32, q)
    _buf(dinitial_state, "dinitial_state", (B, H, dk_, dv_), F32, q)
    dk = _new(q, (B, N, Hk, dk_), dq.dtype, stream) if dk is None else dk
    dv = _new(q, (B, N, H, dv_), dq.dtype, stream) if dv is None else dv
    dg = _new(q, (B, N, H), torch.float32, stream) if dg is None else dg
    dbeta = _new(q, (B, N, H), torch.float32, stream) if dbeta is None else dbeta
    if dinitial_state is None and (initial_state is not None if want_dinitial_state is None else want_dinitial_state):
        dinitial_state = _new(q, (B, H, dk_, dv_), torch.float32, stream)
    need = lib.ret_delta_backward_workspace_bytes(B, N, Hk, H, dk_, dv_, _dt(q.dtype)) if workspace is None else 0
    wp, nbytes, workspace = _workspace(workspace, need, q, stream)
    _call(q, stream, lib.ret_delta_backward_chunkwise, _ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v"), _ptr(g, "g"),
          _ptr(beta, "beta"), _ptr(dout, "dout"), _ptr(lengths, "lengths"), _ptr(initial_state, "initial_state"),
          _ptr(dfinal_state, "dfinal_state"), B, N, Hk, H, dk_, dv_, _ptr(dq, "dq"), _ptr(dk, "dk"), _ptr(dv, "dv"),
          _ptr(dg, "dg"), _ptr(dbeta, "dbeta"), _ptr(dinitial_state, "dinitial_state"), _STREAM, _dt(q.dtype),
          _dt(dq.dtype), wp, nbytes)
    return dq, dk, dv, dg, dbeta, dinitial_state
