"""Python binding of libtps.so (include/tps.h), through ctypes; the short calls
(norm, dropout, linear product) through the extension of csrc/binding.cpp.

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  Tensors must be CUDA tensors on the current device;
outputs and workspace are allocated with torch on that device and the work
is enqueued on torch's current stream.  There is no CPU path: without the
built library or a GPU these functions raise.  Tensors given by `out` are
written in place, and autograd is told so (their version counters move on).
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import struct
from array import array
from typing import Optional, Sequence

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# TPS_LIBRARY selects another build of the library (the debug build,
# libtps_debug.so, whose kernels bounds-check every store).
LIB_PATH = os.environ.get("TPS_LIBRARY") or os.path.join(_PKG, "libtps.so")

F32, BF16, I32, I64, E4M3 = 0, 1, 2, 3, 4
(OK, ERR_SHAPE, ERR_PARTITION, ERR_DTYPE, ERR_LAYOUT, ERR_LABEL, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_ARG,
 ERR_BOUNDS) = range(11)
BUILD_DEBUG = 1  # bit of tps_build_flags()
AXES = {"rows": 0, "columns": 1, "inner": 2}
ACTS = {"gelu": 0, "gelu_erf": 0, "gelu_tanh": 1, "tanh": 2, "silu": 3}
LINEAR_ACTS = {**ACTS, None: -1}
LAYOUTS = {"in_out": 0, "out_in": 1}

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.int32: I32, torch.int64: I64}
_STATE_DTYPES = {torch.float32: F32, torch.float8_e4m3fn: E4M3}


class TpsTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class TpsCeOptions(ctypes.Structure):
    """tps_ce_options of include/tps.h."""
    _fields_ = [("ignore_index", ctypes.c_int64), ("vocab_size", ctypes.c_int64), ("reduction", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("denominator", ctypes.c_double)]


ROPE_MAX_PAIRS = 256
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
ADAMW_BLOCK = 256  # elements that share a scale of the e4m3 moments


class TpsRopeOptions(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_context", ctypes.c_double), ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("attention_factor", ctypes.c_double)]


class RopePlan(ctypes.Structure):
    """tps_rope_plan: what rope_fwd and rope_bwd need of the frequencies."""
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * ROPE_MAX_PAIRS)]


class TpsAdamwHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64),
                ("seed", ctypes.c_uint32), ("stochastic", ctypes.c_int32)]


class TpsAdamwScalars(ctypes.Structure):
    _fields_ = [("step_size", ctypes.c_float), ("root_scale", ctypes.c_float), ("decay", ctypes.c_float),
                ("seed", ctypes.c_uint32)]


# tps_adamw_tensor and tps_span as rows of a table
_ADAMW_ROW = np.dtype([(n, np.uint64) for n in ("param", "grad", "master", "m", "v", "m_scale", "v_scale")] +
                      [("numel", np.int64), ("place", np.int64), ("param_dtype", np.int32), ("grad_dtype", np.int32),
                       ("state_dtype", np.int32), ("reserved", np.int32)])
_SPAN_ROW = np.dtype([("data", np.uint64), ("numel", np.int64), ("dtype", np.int32), ("reserved", np.int32)])

NO_IGNORE = -(2 ** 63)
REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}


class TpsError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what} (code {code})")
        self.code = code


_lib = None


def library():
    """Load libtps.so once.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libtps.so is not built ({LIB_PATH}); run "
                           "`python -m backward_tcgen05_tma_gemms_gb300.build` first")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(TpsTensor)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.tps_plan_shards.argtypes = [i64, i32, ctypes.POINTER(i64)]
    lib.tps_matmul_fwd_bwd.argtypes = [P, P, P, i32, i32, P, P, P, vp]
    lib.tps_mlp_fwd_bwd.argtypes = [P, P, P, P, i32, i32, i32, P, P, P, P, vp, sz, vp]
    lib.tps_mlp_fwd_bwd_noalloc.argtypes = [P, P, P, P, i32, i32, i32, P, P, P, P, vp]
    lib.tps_glu_mlp_fwd_bwd.argtypes = [P, P, P, P, P, i32, i32, i32, P, P, P, P, P, vp, sz, vp]
    lib.tps_glu_mlp_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    lib.tps_glu_mlp_workspace_bytes.restype = sz
    lib.tps_plan_heads.argtypes = [i32, i32, i32, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i32),
                                   ctypes.POINTER(i32)]
    lib.tps_attn_qkv_fwd.argtypes = [P, P, P, P, i32, i32, i32, i32, P, P, P, vp]
    lib.tps_attn_qkv_bwd.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, P, P, P, P, vp]
    lib.tps_attn_out_fwd_bwd.argtypes = [P, P, P, i32, i32, i32, P, P, P, vp]
    lib.tps_mlp_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    lib.tps_mlp_workspace_bytes.restype = sz
    lib.tps_vocab_ce_fwd_bwd.argtypes = [P, P, P, i32, i32, P, P, P, P, vp, sz, vp]
    lib.tps_vocab_ce_fwd_bwd_ex.argtypes = [P, P, P, i32, i32, ctypes.POINTER(TpsCeOptions), P, P, P, P, P, P, vp,
                                            sz, vp]
    lib.tps_ce_workspace_bytes.argtypes = [i64, i64, i32]
    lib.tps_ce_workspace_bytes.restype = sz
    lib.tps_ce_workspace_bytes_ex.argtypes = [i64, i64, i32, i32]
    lib.tps_ce_workspace_bytes_ex.restype = sz
    V = ctypes.c_char_p  # a tps_tensor packed by _view
    lib.tps_linear_ce_fwd.argtypes = [V, V, V, i32, ctypes.POINTER(TpsCeOptions), V, V, V, vp, sz, vp]
    lib.tps_linear_ce_bwd.argtypes = [V, V, V, V, V, i32, ctypes.POINTER(TpsCeOptions), V, V, vp, sz, vp]
    lib.tps_linear_ce_workspace_bytes.argtypes = [i64, i64, i64, i32, i32, i64]
    lib.tps_linear_ce_workspace_bytes.restype = sz
    lib.tps_rope_plan_init.argtypes = [ctypes.POINTER(TpsRopeOptions), ctypes.POINTER(RopePlan)]
    lib.tps_rope_fwd.argtypes = [ctypes.POINTER(RopePlan), V, V, V, V, V, vp]
    lib.tps_rope_bwd.argtypes = [ctypes.POINTER(RopePlan), V, V, V, V, V, vp]
    lib.tps_adamw_prepare.argtypes = [ctypes.POINTER(TpsAdamwHyper), ctypes.POINTER(TpsAdamwScalars)]
    lib.tps_adamw_step.argtypes = [vp, i32, ctypes.POINTER(TpsAdamwHyper), vp, vp, vp]
    lib.tps_grad_norm.argtypes = [vp, i32, ctypes.c_double, vp, vp, sz, vp]
    lib.tps_grad_norm_workspace_bytes.argtypes = [i32]
    lib.tps_grad_norm_workspace_bytes.restype = sz
    D = ctypes.c_char_p  # a tps_dropout as bytes
    lib.tps_rmsnorm_fwd.argtypes = [V, V, V, ctypes.c_double, D, V, V, V, V, vp]
    lib.tps_rmsnorm_bwd.argtypes = [V, V, V, V, V, D, V, V, V, vp, sz, vp]
    lib.tps_dropout_fwd.argtypes = [V, V, D, V, vp]
    lib.tps_dropout_bwd.argtypes = [V, D, V, vp]
    lib.tps_quantize_e4m3.argtypes = [V, V, V, vp]
    lib.tps_linear_fwd.argtypes = [V, V, V, V, i32, i32, V, V, V, V, vp, sz, vp]
    lib.tps_linear_bwd.argtypes = [V, V, V, V, i32, i32, V, V, V, vp, sz, vp]
    lib.tps_rmsnorm_workspace_bytes.argtypes = [i64, i64]
    lib.tps_rmsnorm_workspace_bytes.restype = sz
    lib.tps_linear_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    lib.tps_linear_workspace_bytes.restype = sz
    lib.tps_last_device_error.argtypes = [vp]
    lib.tps_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
    lib.tps_strerror.argtypes = [ctypes.c_int]
    lib.tps_strerror.restype = ctypes.c_char_p
    lib.tps_last_error_detail.restype = ctypes.c_char_p
    lib.tps_profile_reset.argtypes = [ctypes.c_int]
    lib.tps_profile_summary.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(i64),
                                        ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_double)]
    lib.tps_launch_count.restype = i64
    _lib = lib
    return lib


_fast = None
_FAST_ENTRIES = ("tps_rmsnorm_fwd", "tps_rmsnorm_bwd", "tps_rmsnorm_workspace_bytes", "tps_dropout_fwd",
                 "tps_dropout_bwd", "tps_quantize_e4m3", "tps_linear_fwd", "tps_linear_bwd",
                 "tps_linear_workspace_bytes")  # in the order of Entries in csrc/binding.cpp


def _native():
    """The extension behind norm, dropout and the linear product, calling the
    library that is loaded."""
    global _fast
    if _fast is None:
        lib = library()
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError(f"_binding.so is not built or does not fit the installed torch ({e}); run "
                               "`python -m backward_tcgen05_tma_gemms_gb300.build` first") from e
        _binding.init(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _FAST_ENTRIES))
        _fast = _binding
    return _fast


# --------------------------------------------------------------------- helpers

def _tt(t: Optional[torch.Tensor]):
    """tps_tensor view of a CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU (no CPU path)")
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    if t.dim() > 4 or t.dim() < 1:
        raise ValueError("shape")
    s = TpsTensor()
    s.data = t.data_ptr()
    s.dtype = _DTYPES[t.dtype]
    s.ndim = t.dim()
    for i in range(t.dim()):
        s.shape[i] = t.shape[i]
        s.stride[i] = t.stride(i)
    return ctypes.byref(s), s  # keep the struct alive with the reference


def _ref(x):
    return None if x is None else x[0]


_VIEW = struct.Struct("=Qii8q")  # tps_tensor
_PAD = (0, 0, 0, 0)


def _view(t: Optional[torch.Tensor]):
    """tps_tensor view of a CUDA tensor as bytes (None -> NULL): the same
    checks as _tt, packed in one step for the short calls."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU (no CPU path)")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    n = t.dim()
    if n > 4 or n < 1:
        raise ValueError("shape")
    return _VIEW.pack(t.data_ptr(), code, n, *t.shape, *_PAD[n:], *t.stride(), *_PAD[n:])


def _check(rc: int):
    if rc == OK:
        return
    lib = library()
    detail = lib.tps_last_error_detail().decode()
    if rc == ERR_SHAPE:
        raise ValueError("shape")
    if rc == ERR_PARTITION:
        raise ValueError("partition")
    raise TpsError(rc, f"{lib.tps_strerror(rc).decode()}: {detail}")


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _raw_stream(t: torch.Tensor) -> int:
    """The current stream of t's GPU, without building a Stream object."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _counts_writes(fn):
    """The tensors that a call is given by `out` hold something else afterwards:
    what autograd saved of them is not what it computed with."""
    at = list(inspect.signature(fn).parameters).index("out")

    @functools.wraps(fn)
    def call(*args, **kw):
        r = fn(*args, **kw)
        out = kw.get("out") if len(args) <= at else args[at]
        if out is not None:
            given = (out,) if isinstance(out, torch.Tensor) else out
            torch.autograd.graph.increment_version([t for t in given if t is not None and not t.is_inference()])
        return r
    return call


def _parts(v, name="parts") -> int:
    if type(v) is not int or v < 1:
        raise ValueError("partition")
    return v


# --------------------------------------------------------------------- API

def plan_shards(dim: int, parts: int) -> list:
    """array_split offsets (parts + 1 entries) computed by the library."""
    _parts(parts)
    off = (ctypes.c_int64 * (parts + 1))()
    _check(library().tps_plan_shards(int(dim), parts, off))
    return list(off)


@_counts_writes
def matmul_fwd_bwd(A: torch.Tensor, B: torch.Tensor, G: torch.Tensor, parts: int, axis: str,
                   out: Optional[Sequence[torch.Tensor]] = None):
    """(Y, dA, dB) of L = <G, AB> split over `parts` ranks along `axis`.
    Results are fp32; `out` may supply (Y, dA, dB) to write into."""
    _parts(parts)
    if axis not in AXES:
        raise ValueError("partition")
    if A.dim() != 2 or B.dim() != 2 or G.dim() != 2 or A.shape[1] != B.shape[0] or tuple(G.shape) != (A.shape[0], B.shape[1]):
        raise ValueError("shape")
    M, K = A.shape
    N = B.shape[1]
    if out is None:
        kw = dict(device=A.device, dtype=torch.float32)
        out = (torch.empty(M, N, **kw), torch.empty(M, K, **kw), torch.empty(K, N, **kw))
    Y, dA, dB = out
    a, b, g, y, da, db = (_tt(t) for t in (A, B, G, Y, dA, dB))
    _check(library().tps_matmul_fwd_bwd(_ref(a), _ref(b), _ref(g), parts, AXES[axis], _ref(y), _ref(da), _ref(db),
                                        _stream(A.device)))
    return Y, dA, dB


def mlp_workspace_bytes(T: int, d: int, F: int, tp: int, dtype: torch.dtype) -> int:
    return int(library().tps_mlp_workspace_bytes(T, d, F, tp, _DTYPES[dtype]))


@_counts_writes
def mlp_fwd_bwd(X: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, GY: torch.Tensor, tp: int,
                act: str = "gelu_tanh", weight_layout: str = "in_out", workspace: Optional[torch.Tensor] = None,
                out: Optional[Sequence[torch.Tensor]] = None):
    """Column-then-row TP MLP forward + backward.  Returns (Y, dX, dW1, dW2)
    in fp32 (Y, dX shaped like X; dW1, dW2 like W1, W2)."""
    _parts(tp, "tp")
    if act not in ACTS or weight_layout not in LAYOUTS:
        raise ValueError("argument")
    d = X.shape[-1]
    T = X.numel() // d if d else 0
    F = W1.shape[1] if weight_layout == "in_out" else W1.shape[0]
    if out is None:
        kw = dict(device=X.device, dtype=torch.float32)
        out = (torch.empty(X.shape, **kw), torch.empty(X.shape, **kw), torch.empty(W1.shape, **kw),
               torch.empty(W2.shape, **kw))
    Y, dX, dW1, dW2 = out
    need = mlp_workspace_bytes(T, d, F, tp, X.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=X.device)
    args = [_tt(t) for t in (X, W1, W2, GY, Y, dX, dW1, dW2)]
    _check(library().tps_mlp_fwd_bwd(*[_ref(a) for a in args[:4]], tp, ACTS[act], LAYOUTS[weight_layout],
                                     *[_ref(a) for a in args[4:]], ctypes.c_void_p(workspace.data_ptr()),
                                     workspace.numel() * workspace.element_size(), _stream(X.device)))
    return Y, dX, dW1, dW2


# Size of the static scratch of tps_mlp_fwd_bwd_noalloc (TPS_MLP_NOALLOC_SCRATCH_BYTES).
MLP_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


@_counts_writes
def mlp_fwd_bwd_noalloc(X: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, GY: torch.Tensor, tp: int,
                        act: str = "gelu_tanh", weight_layout: str = "in_out",
                        out: Optional[Sequence[torch.Tensor]] = None):
    """mlp_fwd_bwd without a workspace, for callers that cannot allocate
    device memory (an allocator owned by a hosting framework, or a path that
    must not call cudaMalloc): the library's static 32 MiB device scratch is
    used instead.  Larger problems are rejected; calls that overlap on the
    GPU race on the shared scratch.  Outputs still come from `out` (or are
    allocated here by torch when `out` is None)."""
    _parts(tp, "tp")
    if act not in ACTS or weight_layout not in LAYOUTS:
        raise ValueError("argument")
    if out is None:
        kw = dict(device=X.device, dtype=torch.float32)
        out = (torch.empty(X.shape, **kw), torch.empty(X.shape, **kw), torch.empty(W1.shape, **kw),
               torch.empty(W2.shape, **kw))
    args = [_tt(t) for t in (X, W1, W2, GY, *out)]
    _check(library().tps_mlp_fwd_bwd_noalloc(*[_ref(a) for a in args[:4]], tp, ACTS[act], LAYOUTS[weight_layout],
                                             *[_ref(a) for a in args[4:]], _stream(X.device)))
    return tuple(out)


def ce_workspace_bytes(T: int, V: int, tp: int, dtype: Optional[torch.dtype] = None) -> int:
    """Workspace bytes of the CE entry points: enough for every path when
    `dtype` is None, else for operands of `dtype` on the tensor-core path
    (bf16 logits)."""
    if dtype is None:
        return int(library().tps_ce_workspace_bytes(T, V, tp))
    return int(library().tps_ce_workspace_bytes_ex(T, V, tp, _DTYPES[dtype]))


def _ce_call(fn, T, V, tp, dtype, workspace, device):
    """Run fn(workspace) with the given workspace, or with one sized for
    the tensor-core path; operands that take the fp32 path instead are
    refused before any launch (TPS_ERR_WORKSPACE) and run again with the
    full size."""
    if workspace is not None:
        _check(fn(workspace))
        return
    small = ce_workspace_bytes(T, V, tp, dtype)
    ws = torch.empty(max(small, 1), dtype=torch.uint8, device=device)
    rc = fn(ws)
    full = ce_workspace_bytes(T, V, tp)
    if rc == ERR_WORKSPACE and full > small:
        del ws
        rc = fn(torch.empty(max(full, 1), dtype=torch.uint8, device=device))
    _check(rc)


def glu_mlp_workspace_bytes(T: int, d: int, F: int, tp: int, dtype: torch.dtype) -> int:
    return int(library().tps_glu_mlp_workspace_bytes(T, d, F, tp, _DTYPES[dtype]))


@_counts_writes
def glu_mlp_fwd_bwd(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, W2: torch.Tensor, GY: torch.Tensor,
                    tp: int, act: str = "silu", weight_layout: str = "in_out",
                    workspace: Optional[torch.Tensor] = None, out: Optional[Sequence[torch.Tensor]] = None):
    """Gated tensor-parallel MLP (SwiGLU for act="silu") forward + backward.
    Returns fp32 (Y, dX, dWg, dWu, dW2)."""
    _parts(tp, "tp")
    if act not in ACTS or weight_layout not in LAYOUTS:
        raise ValueError("argument")
    d = X.shape[-1]
    T = X.numel() // d if d else 0
    F = Wg.shape[1] if weight_layout == "in_out" else Wg.shape[0]
    dev = X.device
    if out is None:
        out = (torch.empty(X.shape, device=dev, dtype=torch.float32),
               torch.empty(X.shape, device=dev, dtype=torch.float32),
               torch.empty(Wg.shape, device=dev, dtype=torch.float32),
               torch.empty(Wu.shape, device=dev, dtype=torch.float32),
               torch.empty(W2.shape, device=dev, dtype=torch.float32))
    if workspace is None:
        need = glu_mlp_workspace_bytes(T, d, F, tp, X.dtype)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    args = [_tt(t) for t in (X, Wg, Wu, W2, GY, *out)]
    _check(library().tps_glu_mlp_fwd_bwd(*[_ref(a) for a in args[:5]], tp, ACTS[act], LAYOUTS[weight_layout],
                                         *[_ref(a) for a in args[5:]], ctypes.c_void_p(workspace.data_ptr()),
                                         workspace.numel() * workspace.element_size(), _stream(dev)))
    return tuple(out)


def plan_heads(n_heads: int, n_kv_heads: int, tp: int):
    """Head-aligned plan: (q_off [tp+1], kv_first [tp], kv_count, kv_replicas)."""
    _parts(tp, "tp")
    q_off = (ctypes.c_int64 * (tp + 1))()
    kv_first = (ctypes.c_int64 * tp)()
    cnt, rep = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(library().tps_plan_heads(n_heads, n_kv_heads, tp, q_off, kv_first, ctypes.byref(cnt), ctypes.byref(rep)))
    return list(q_off), list(kv_first), int(cnt.value), int(rep.value)


@_counts_writes
def attn_qkv_fwd(X, Wq, Wk, Wv, n_heads: int, n_kv_heads: int, tp: int, weight_layout: str = "in_out",
                 out_dtype: Optional[torch.dtype] = None, out: Optional[Sequence[torch.Tensor]] = None):
    """(Q, K, V) of the head-split column-parallel projections."""
    _parts(tp, "tp")
    if weight_layout not in LAYOUTS:
        raise ValueError("argument")
    d = X.shape[-1]
    T = X.numel() // d if d else 0
    nq = Wq.shape[1] if weight_layout == "in_out" else Wq.shape[0]
    nkv = Wk.shape[1] if weight_layout == "in_out" else Wk.shape[0]
    dt = out_dtype or X.dtype
    if out is None:
        out = tuple(torch.empty(T, n, device=X.device, dtype=dt) for n in (nq, nkv, nkv))
    args = [_tt(t) for t in (X, Wq, Wk, Wv, *out)]
    _check(library().tps_attn_qkv_fwd(*[_ref(a) for a in args[:4]], n_heads, n_kv_heads, tp, LAYOUTS[weight_layout],
                                      *[_ref(a) for a in args[4:]], _stream(X.device)))
    return tuple(out)


@_counts_writes
def attn_qkv_bwd(X, Wq, Wk, Wv, dQ, dK, dV, n_heads: int, n_kv_heads: int, tp: int, weight_layout: str = "in_out",
                 out: Optional[Sequence[torch.Tensor]] = None):
    """fp32 (dX, dWq, dWk, dWv)."""
    _parts(tp, "tp")
    if weight_layout not in LAYOUTS:
        raise ValueError("argument")
    dev = X.device
    if out is None:
        out = (torch.empty(X.shape, device=dev, dtype=torch.float32),
               *(torch.empty(w.shape, device=dev, dtype=torch.float32) for w in (Wq, Wk, Wv)))
    args = [_tt(t) for t in (X, Wq, Wk, Wv, dQ, dK, dV, *out)]
    _check(library().tps_attn_qkv_bwd(*[_ref(a) for a in args[:7]], n_heads, n_kv_heads, tp, LAYOUTS[weight_layout],
                                      *[_ref(a) for a in args[7:]], _stream(dev)))
    return tuple(out)


@_counts_writes
def attn_out_fwd_bwd(C, Wo, GY, n_heads: int, tp: int, weight_layout: str = "in_out",
                     dC_dtype: Optional[torch.dtype] = None, out: Optional[Sequence[torch.Tensor]] = None):
    """(Y fp32, dC, dWo fp32) of the row-parallel output projection."""
    _parts(tp, "tp")
    if weight_layout not in LAYOUTS:
        raise ValueError("argument")
    dev = C.device
    if out is None:
        out = (torch.empty(GY.shape, device=dev, dtype=torch.float32),
               torch.empty(C.shape, device=dev, dtype=dC_dtype or C.dtype),
               torch.empty(Wo.shape, device=dev, dtype=torch.float32))
    args = [_tt(t) for t in (C, Wo, GY, *out)]
    _check(library().tps_attn_out_fwd_bwd(*[_ref(a) for a in args[:3]], n_heads, tp, LAYOUTS[weight_layout],
                                          *[_ref(a) for a in args[3:]], _stream(dev)))
    return tuple(out)


@_counts_writes
def vocab_ce_fwd_bwd(h: torch.Tensor, Whead: torch.Tensor, labels: torch.Tensor, tp: int,
                     weight_layout: str = "in_out", workspace: Optional[torch.Tensor] = None,
                     out: Optional[Sequence[torch.Tensor]] = None):
    """Vocabulary-sharded cross-entropy forward + backward.  Returns
    (loss fp32 [T], dlogits [T, V] in h's dtype, dHidden fp32 like h,
    owner int32 [T])."""
    _parts(tp, "tp")
    if weight_layout not in LAYOUTS:
        raise ValueError("argument")
    d = h.shape[-1]
    T = h.numel() // d if d else 0
    V = Whead.shape[1] if weight_layout == "in_out" else Whead.shape[0]
    if out is None:
        out = (torch.empty(T, device=h.device, dtype=torch.float32),
               torch.empty(T, V, device=h.device, dtype=h.dtype),
               torch.empty(h.shape, device=h.device, dtype=torch.float32),
               torch.empty(T, device=h.device, dtype=torch.int32))
    loss, dlog, dh, owner = out
    args = [_tt(t) for t in (h, Whead, labels, loss, dlog, dh, owner)]
    _ce_call(lambda ws: library().tps_vocab_ce_fwd_bwd(
        _ref(args[0]), _ref(args[1]), _ref(args[2]), tp, LAYOUTS[weight_layout], *[_ref(a) for a in args[3:]],
        ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size(), _stream(h.device)),
        T, V, tp, h.dtype, workspace, h.device)
    return loss, dlog, dh, owner


@_counts_writes
def vocab_ce_fwd_bwd_ex(h: torch.Tensor, Whead: torch.Tensor, labels: torch.Tensor, tp: int,
                        weight_layout: str = "in_out", ignore_index: Optional[int] = None, vocab_size: int = 0,
                        reduction: str = "none", denominator: float = 0.0, want_dwhead: bool = False,
                        workspace: Optional[torch.Tensor] = None, out: Optional[Sequence] = None):
    """Cross-entropy with vocabulary padding (the first `vocab_size` columns
    of the head are real, 0 = all), `ignore_index`, a "sum" or "mean"
    reduction (the mean divides by `denominator` when > 0, e.g. the
    job-wide count of supervised tokens, else by this call's count), and
    optionally the head's gradient.  Returns (loss [T], loss_reduced (0-d)
    or None, dlogits, dHidden, dWhead or None, owner); `out` may supply
    those six to write into (loss_reduced and dWhead may be None)."""
    _parts(tp, "tp")
    if weight_layout not in LAYOUTS or reduction not in REDUCTIONS:
        raise ValueError("argument")
    d = h.shape[-1]
    T = h.numel() // d if d else 0
    V = Whead.shape[1] if weight_layout == "in_out" else Whead.shape[0]
    dev = h.device
    if out is not None:
        loss, red, dlog, dh, dw, owner = out
    else:
        loss = torch.empty(T, device=dev, dtype=torch.float32)
        red = torch.zeros((), device=dev, dtype=torch.float32) if reduction != "none" else None
        dlog = torch.empty(T, V, device=dev, dtype=h.dtype)
        dh = torch.empty(h.shape, device=dev, dtype=torch.float32)
        dw = torch.empty(Whead.shape, device=dev, dtype=torch.float32) if want_dwhead else None
        owner = torch.empty(T, device=dev, dtype=torch.int32)
    opts = TpsCeOptions(NO_IGNORE if ignore_index is None else int(ignore_index), int(vocab_size),
                        REDUCTIONS[reduction], 0, float(denominator))
    red_t = _tt(red.reshape(1)) if red is not None else None
    head = [_tt(t) for t in (h, Whead, labels, loss)]
    tail = [_tt(t) for t in (dlog, dh, dw, owner)]
    _ce_call(lambda ws: library().tps_vocab_ce_fwd_bwd_ex(
        _ref(head[0]), _ref(head[1]), _ref(head[2]), tp, LAYOUTS[weight_layout], ctypes.byref(opts), _ref(head[3]),
        _ref(red_t), *[_ref(a) for a in tail], ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size(),
        _stream(dev)), T, V, tp, h.dtype, workspace, dev)
    return loss, red, dlog, dh, dw, owner


def linear_ce_workspace_bytes(T: int, d: int, V: int, dtype: torch.dtype, backward: bool, piece: int = 0) -> int:
    """Workspace bytes of linear_ce_fwd / linear_ce_bwd for pieces of `piece`
    vocabulary columns (0: the library's choice)."""
    return int(library().tps_linear_ce_workspace_bytes(T, d, V, _DTYPES[dtype], 1 if backward else 0, piece))


def _room(workspace: torch.Tensor):
    """Address and bytes of a workspace that the kernels may write."""
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not workspace.is_cuda:
        raise ValueError("tensors must live on the GPU (no CPU path)")
    if not workspace.is_contiguous():
        raise TpsError(ERR_LAYOUT, "workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _linear_ce_call(fn, T, d, V, dtype, backward, workspace, device):
    """Run fn(workspace pointer, bytes) with the given workspace, or with one
    for the tensor-core path; operands that do not qualify for it are refused
    before any launch and run again with the other path's size."""
    if workspace is not None:
        _check(fn(*_room(workspace)))
        return
    for dt in (dtype, torch.float32):
        n = max(linear_ce_workspace_bytes(T, d, V, dt, backward), 1)
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        rc = fn(ws.data_ptr(), n)
        if rc != ERR_WORKSPACE:
            break
    _check(rc)


def _linear_ce_args(h, Whead, weight_layout, ignore_index, vocab_size, reduction, denominator):
    if weight_layout not in LAYOUTS or reduction not in REDUCTIONS:
        raise ValueError("argument")
    if Whead.dim() != 2:
        raise ValueError("shape")
    d = h.shape[-1]
    V = Whead.shape[1] if weight_layout == "in_out" else Whead.shape[0]
    opts = TpsCeOptions(NO_IGNORE if ignore_index is None else int(ignore_index), int(vocab_size),
                        REDUCTIONS[reduction], 0, float(denominator))
    return (h.numel() // d if d else 0), d, V, opts


@_counts_writes
def linear_ce_fwd(h: torch.Tensor, Whead: torch.Tensor, labels: torch.Tensor, weight_layout: str = "in_out",
                  ignore_index: Optional[int] = None, vocab_size: int = 0, reduction: str = "none",
                  denominator: float = 0.0, workspace: Optional[torch.Tensor] = None,
                  out: Optional[Sequence] = None):
    """Cross entropy of the head in pieces of the vocabulary, without the
    logits.  Returns (loss [T], loss_reduced (0-d) or None, lse [T]), all
    fp32; lse is what linear_ce_bwd needs.  Options as vocab_ce_fwd_bwd_ex."""
    T, d, V, opts = _linear_ce_args(h, Whead, weight_layout, ignore_index, vocab_size, reduction, denominator)
    if out is not None:
        loss, red, lse = out
    else:
        loss = torch.empty(T, device=h.device, dtype=torch.float32)
        lse = torch.empty(T, device=h.device, dtype=torch.float32)
        red = torch.empty((), device=h.device, dtype=torch.float32) if reduction != "none" else None
    a = [_view(t) for t in (h, Whead, labels, loss, red.reshape(1) if red is not None else None, lse)]
    stream = _raw_stream(h)
    _linear_ce_call(lambda ws, n: library().tps_linear_ce_fwd(
        a[0], a[1], a[2], LAYOUTS[weight_layout], ctypes.byref(opts), a[3], a[4], a[5], ws, n, stream),
        T, d, V, h.dtype, False, workspace, h.device)
    return loss, red, lse


@_counts_writes
def linear_ce_bwd(h: torch.Tensor, Whead: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor,
                  grad_loss: Optional[torch.Tensor] = None, weight_layout: str = "in_out",
                  ignore_index: Optional[int] = None, vocab_size: int = 0, reduction: str = "none",
                  denominator: float = 0.0, want_dhidden: bool = True, want_dwhead: bool = True,
                  grad_dtype: torch.dtype = torch.float32, workspace: Optional[torch.Tensor] = None,
                  out: Optional[Sequence] = None):
    """Backward of linear_ce_fwd from its lse: (dHidden like h, dWhead like
    Whead) in `grad_dtype` (fp32 or bf16), None for one that is not wanted.
    grad_loss: the upstream gradient (T values for reduction "none", else
    one; default ones)."""
    T, d, V, opts = _linear_ce_args(h, Whead, weight_layout, ignore_index, vocab_size, reduction, denominator)
    if out is not None:
        dh, dw = out
    else:
        dh = torch.empty(h.shape, device=h.device, dtype=grad_dtype) if want_dhidden else None
        dw = torch.empty(Whead.shape, device=h.device, dtype=grad_dtype) if want_dwhead else None
    if grad_loss is not None and grad_loss.dim() == 0:
        grad_loss = grad_loss.reshape(1)
    a = [_view(t) for t in (h, Whead, labels, lse, grad_loss, dh, dw)]
    stream = _raw_stream(h)
    _linear_ce_call(lambda ws, n: library().tps_linear_ce_bwd(
        *a[:5], LAYOUTS[weight_layout], ctypes.byref(opts), a[5], a[6], ws, n, stream),
        T, d, V, h.dtype, True, workspace, h.device)
    return dh, dw


# --------------------------------------------------------------------- rotary positions

def rope_plan(rotary_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
              factor: float = 1.0, original_context: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
              attention_factor: float = 0.0) -> RopePlan:
    """Plan of a rotary embedding of the first `rotary_dim` elements of each
    head: halves (default) or interleaved pairs, scaled for long contexts by
    "linear", "ntk" or "yarn" (host only)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("argument")
    plan = RopePlan()
    opts = TpsRopeOptions(int(rotary_dim), 1 if interleaved else 0, ROPE_SCALINGS[scaling], 0, float(base),
                          float(factor), float(original_context), float(beta_fast), float(beta_slow),
                          float(attention_factor))
    _check(library().tps_rope_plan_init(ctypes.byref(opts), ctypes.byref(plan)))
    return plan


def _rope(fn, plan, q, k, positions, head_dim, out):
    def heads(t):
        if t is None or t.dim() != 2:
            return t
        if head_dim is None or head_dim < 1 or t.shape[1] % head_dim:
            raise ValueError("shape")
        return t.unflatten(1, (t.shape[1] // head_dim, head_dim))
    if out is None:
        out = (torch.empty_like(q), None if k is None else torch.empty_like(k))
    _check(fn(plan, _view(heads(q)), _view(heads(k)), _view(positions), _view(heads(out[0])), _view(heads(out[1])),
              _raw_stream(q)))
    return tuple(out)


@_counts_writes
def rope_fwd(plan: RopePlan, q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
             head_dim: Optional[int] = None, out: Optional[Sequence[torch.Tensor]] = None):
    """(q', k'): the heads turned by their positions.  q and k are (T, H, D)
    or (B, S, H, D), or T x H*D as attn_qkv_fwd leaves them (with head_dim);
    out=(q, k) works in place; k may be None."""
    return _rope(library().tps_rope_fwd, plan, q, k, positions, head_dim, out)


@_counts_writes
def rope_bwd(plan: RopePlan, dq: torch.Tensor, dk: Optional[torch.Tensor], positions: torch.Tensor,
             head_dim: Optional[int] = None, out: Optional[Sequence[torch.Tensor]] = None):
    """Gradients of q and k from those of rope_fwd's results."""
    return _rope(library().tps_rope_bwd, plan, dq, dk, positions, head_dim, out)


# --------------------------------------------------------------------- norm and dropout

def rmsnorm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                eps: float = 1e-6, dropout: float = 0.0, seed=0, site: int = 0,
                out_dtype: Optional[torch.dtype] = None, out: Optional[Sequence] = None):
    """Residual addition and root-mean-square norm of rows (..., d):
    h = residual + dropout(x), y = h weight / sqrt(mean h^2 + eps).  Returns
    (y, scale, h, rstd): y in out_dtype (x's by default), with one scale for
    each row when that is torch.float8_e4m3fn (else None); h in the residual's
    type, None where it is x (no residual, no dropout); rstd for rmsnorm_bwd.
    seed: a number, or one int64 on the GPU, which a captured CUDA graph reads
    at every replay; site: which dropout of the model this is.  `out` may
    supply the four; h may be the residual and y may be x."""
    r = (_fast or _native()).rmsnorm_fwd(x, weight, residual, eps, dropout, seed, site, out_dtype, out)
    return r if type(r) is tuple else _check(r)


def rmsnorm_workspace_bytes(T: int, d: int) -> int:
    return int(library().tps_rmsnorm_workspace_bytes(T, d))


def rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: Optional[torch.Tensor], rstd: torch.Tensor,
                dh: Optional[torch.Tensor] = None, dropout: float = 0.0, seed=0, site: int = 0,
                x_dtype: Optional[torch.dtype] = None, want_dweight: bool = True,
                workspace: Optional[torch.Tensor] = None, out: Optional[Sequence] = None):
    """Backward of rmsnorm_fwd from its h (x where it gave none) and rstd:
    (dx, dresidual, dweight).  dh: the gradient that reaches h past the norm.
    dx has x_dtype (h's by default), dresidual h's type; without dropout and
    with one type the two are one tensor.  dweight is fp32.  dropout, seed and
    site as in the forward call.  `out` may supply the three; one tensor for
    the first two only without dropout."""
    r = (_fast or _native()).rmsnorm_bwd(dy, h, weight, rstd, dh, dropout, seed, site, x_dtype, want_dweight, workspace,
                                         out)
    return r if type(r) is tuple else _check(r)


def dropout_fwd(x: torch.Tensor, p: float, seed, site: int = 0, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x with each element dropped with probability p (in steps of 2^-16) and
    multiplied by 1 / (1 - p) otherwise, plus the residual.  The mask is a
    function of seed, site and the element's place, and is not stored."""
    r = (_fast or _native()).dropout(x, p, seed, site, residual, out, False)
    return _check(r) if type(r) is int else r


def dropout_bwd(dy: torch.Tensor, p: float, seed, site: int = 0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of dropout_fwd's x from that of its result (which is the
    residual's too)."""
    r = (_fast or _native()).dropout(dy, p, seed, site, None, out, True)
    return _check(r) if type(r) is int else r


def quantize_e4m3(x: torch.Tensor, out: Optional[Sequence] = None):
    """(q, scale): the rows of x (..., d) as e4m3 numbers, the largest
    magnitude of each row being 448, and one fp32 scale for each row:
    x = q scale."""
    r = (_fast or _native()).quantize_e4m3(x, out)
    return r if type(r) is tuple else _check(r)


# --------------------------------------------------------------------- product with its epilogue

def linear_workspace_bytes(T: int, K: int, N: int, dtype: torch.dtype, backward: bool) -> int:
    """Workspace bytes of linear_fwd / linear_bwd for operands of `dtype`; bf16
    operands that are not 16-byte aligned need those of fp32."""
    code = E4M3 if dtype == torch.float8_e4m3fn else _DTYPES[dtype]
    return int(library().tps_linear_workspace_bytes(T, K, N, code, 1 if backward else 0))


def _linear_codes(act, weight_layout):
    if act not in LINEAR_ACTS or weight_layout not in LAYOUTS:
        raise ValueError("argument")
    return LINEAR_ACTS[act], LAYOUTS[weight_layout]


def linear_fwd(x: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, act: Optional[str] = None, weight_layout: str = "in_out",
               x_scale: Optional[torch.Tensor] = None, w_scale: Optional[torch.Tensor] = None,
               want_pre: bool = False, out_dtype: Optional[torch.dtype] = None,
               workspace: Optional[torch.Tensor] = None, out: Optional[Sequence] = None):
    """(y, z): z = x W + bias and y = act(z) + residual of x (..., K), in
    out_dtype (x's by default, bf16 for e4m3); z, the pre-activation that
    linear_bwd needs, only with want_pre.  x and W are fp32, bf16, or e4m3 with
    x_scale and w_scale, one for each row of x and of W (quantize_e4m3), W then
    being (out, in).  `out` may supply (y, z); y may be the residual."""
    a, layout = _linear_codes(act, weight_layout)
    r = (_fast or _native()).linear_fwd(x, W, bias, residual, a, layout, x_scale, w_scale, want_pre, out_dtype, workspace,
                                        out)
    return r if type(r) is tuple else _check(r)


def linear_bwd(x: torch.Tensor, W: torch.Tensor, dy: torch.Tensor, pre: Optional[torch.Tensor] = None,
               act: Optional[str] = None, weight_layout: str = "in_out", want_dx: bool = True, want_dw: bool = True,
               want_dbias: bool = True, grad_dtype: torch.dtype = torch.float32,
               workspace: Optional[torch.Tensor] = None, out: Optional[Sequence] = None):
    """Gradients of linear_fwd's x, W and bias from that of its y (which is the
    residual's too): (dx, dW, dbias) in `grad_dtype` (fp32 or bf16), None for
    one that is not wanted.  pre: the pre-activation, with an activation."""
    a, layout = _linear_codes(act, weight_layout)
    r = (_fast or _native()).linear_bwd(x, W, dy, pre, a, layout, want_dx, want_dw, want_dbias, grad_dtype, workspace, out)
    return r if type(r) is tuple else _check(r)


# --------------------------------------------------------------------- optimizer step

class AdamWPlan:
    """The tensors an optimizer updates and their moments (adamw_plan).  A
    step updates the storage that each of them has by then: where it is another
    one than the step before (p.data = ..., module.to(), a moved state), the
    tensors are checked and their addresses taken again.  (Operations captured
    into a CUDA graph keep those of the capture.)"""

    def __init__(self, params, master, m, v, m_scale, v_scale):
        self.params, self.master, self.m, self.v, self.m_scale, self.v_scale = params, master, m, v, m_scale, v_scale
        self.numels = array("q", (p.numel() for p in params))
        self.device = params[0].get_device() if params else 0
        self._seen = None

    def _columns(self):
        """(field of the table, tensors, elements of a weight for each of theirs, dtypes) of what there is."""
        state = {self.m[0].dtype} if self.m else set()
        for name, ts, per, dtypes in (("param", self.params, 1, {torch.float32, torch.bfloat16}), ("m", self.m, 1, state),
                                      ("v", self.v, 1, state), ("m_scale", self.m_scale, ADAMW_BLOCK, {torch.float32}),
                                      ("v_scale", self.v_scale, ADAMW_BLOCK, {torch.float32}),
                                      ("master", self.master, 1, {torch.float32})):
            if ts is not None:
                yield name, ts, per, dtypes

    def _check(self, addresses):
        if self.m and self.m[0].dtype not in _STATE_DTYPES:
            raise TypeError(f"unsupported dtype {self.m[0].dtype}")
        scaled = bool(self.m) and self.m[0].dtype == torch.float8_e4m3fn
        if self.params and (scaled != (self.m_scale is not None) or scaled != (self.v_scale is not None)):
            raise ValueError("argument")
        cls, spans = torch.Tensor, []
        for (name, ts, per, dtypes), at in zip(self._columns(), addresses):
            if len(ts) != len(self.numels):
                raise ValueError("shape")
            numels = self.numels if per == 1 else [-(-n // per) for n in self.numels]
            if name == "master":  # None: no copy
                if any(t is not None and p.dtype != torch.bfloat16 for t, p in zip(ts, self.params)):
                    raise TypeError("a master copy is for bf16 weights")
                numels = [n for n, t in zip(numels, ts) if t is not None]
                at = [x for x, t in zip(at, ts) if t is not None]
                ts = [t for t in ts if t is not None]
            if list(map(cls.numel, ts)) != list(numels):
                raise ValueError("shape")
            if not {t.dtype for t in ts} <= dtypes:
                raise TypeError(f"unsupported dtype among {[t.dtype for t in ts]}")
            devices = set(map(cls.get_device, ts))
            if not devices <= {self.device}:
                raise ValueError("tensors must live on the GPU (no CPU path)" if -1 in devices else
                                 "weights and state on different GPUs")
            if not all(map(cls.is_contiguous, ts)):
                raise TpsError(ERR_LAYOUT, "weights and state must be contiguous")
            spans += [(x, x + t.nbytes) for x, t in zip(at, ts) if x]
        spans.sort()
        if any(end > first for (_, end), (first, _) in zip(spans, spans[1:])):
            raise ValueError("weights or state given twice, or overlapping")

    def rows(self):
        """The tensors as rows of tps_adamw_tensor, without gradients."""
        address = torch.Tensor.data_ptr
        addresses = [list(map(address, ts)) for ts in (self.params, self.m, self.v, self.m_scale, self.v_scale) if ts is not None]
        if self.master is not None:
            addresses.append([0 if x is None else address(x) for x in self.master])
        if addresses != self._seen:
            self._check(addresses)
            n = len(self.params)
            t = np.zeros(n, _ADAMW_ROW)
            for (name, _, _, _), at in zip(self._columns(), addresses):
                t[name] = at
            t["numel"] = self.numels
            blocks = [-(-x // ADAMW_BLOCK) for x in self.numels]
            t["place"] = ADAMW_BLOCK * np.concatenate(([0], np.cumsum(blocks)[:-1])) if n else []
            t["param_dtype"] = [_DTYPES[p.dtype] for p in self.params]
            t["state_dtype"] = [_STATE_DTYPES[x.dtype] for x in self.m]
            # These share the storages, so that none is freed (and its address given
            # to another tensor) while the table names it.
            self._kept = [x.detach() for c in self._columns() for x in c[1] if x is not None]
            self._table, self._seen = t, addresses
        return self._table.copy()


def adamw_plan(params: Sequence[torch.Tensor], state_dtype: torch.dtype = torch.float32, master=None,
               m: Optional[Sequence[torch.Tensor]] = None, v: Optional[Sequence[torch.Tensor]] = None,
               m_scale: Optional[Sequence[torch.Tensor]] = None,
               v_scale: Optional[Sequence[torch.Tensor]] = None) -> AdamWPlan:
    """What adamw_step updates: contiguous fp32 or bf16 weights on one GPU
    and their moments, fp32 or (state_dtype=torch.float8_e4m3fn) e4m3 numbers
    with a scale for every 256 elements, where v holds sqrt(v).  Moments are
    made here (zeros) unless given, as from a checkpoint.  master: True keeps
    fp32 copies of the bf16 weights; or the copies themselves, one for each
    weight, None for those without one (fp32 weights are their own)."""
    params = list(params)
    for p in params:
        if not isinstance(p, torch.Tensor) or not p.is_cuda:
            raise ValueError("tensors must live on the GPU (no CPU path)")
        if p.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"unsupported dtype {p.dtype}")
    if m is not None:
        m, v = list(m), list(v)
        state_dtype = m[0].dtype if m else state_dtype
    if state_dtype not in _STATE_DTYPES:
        raise TypeError(f"unsupported dtype {state_dtype}")
    scaled = state_dtype == torch.float8_e4m3fn

    def zeros(dtype, per=1):  # byte by byte: e4m3 zeros are zero bytes
        return [torch.zeros(-(-p.numel() // per) * dtype.itemsize, dtype=torch.uint8, device=p.device).view(dtype)
                for p in params]
    if m is None:
        m, v = zeros(state_dtype), zeros(state_dtype)
        m_scale = zeros(torch.float32, ADAMW_BLOCK) if scaled else None
        v_scale = zeros(torch.float32, ADAMW_BLOCK) if scaled else None
    if master is True:
        master = [p.detach().to(torch.float32).contiguous() if p.dtype == torch.bfloat16 else None for p in params]
    master = list(master) if master else None
    m_scale, v_scale = (list(x) if x is not None else None for x in (m_scale, v_scale))
    plan = AdamWPlan(params, master, m, v, m_scale, v_scale)
    plan.rows()
    return plan


def _grad_list(grads):
    """The gradients as a list (they may come one by one), pointers and sizes (as
    arrays), dtype codes of contiguous gradients, and the GPUs they are on."""
    cls = torch.Tensor
    if not isinstance(grads, (list, tuple)):
        grads = list(grads)
    if not all(map(cls.is_contiguous, grads)):
        raise TpsError(ERR_LAYOUT, "gradients must be contiguous")
    devices = set(map(cls.get_device, grads))
    if len(devices) > 1 or -1 in devices:
        raise ValueError("tensors must live on the GPU (no CPU path)" if -1 in devices else "gradients on different GPUs")
    dtypes = [g.dtype for g in grads]
    kinds = set(dtypes)
    if not kinds <= {torch.float32, torch.bfloat16}:
        raise TypeError("gradients must be fp32 or bf16")
    codes = _DTYPES[dtypes[0]] if len(kinds) == 1 else [_DTYPES[d] for d in dtypes]
    return grads, array("Q", list(map(cls.data_ptr, grads))), array("q", list(map(cls.numel, grads))), codes, devices


@_counts_writes
def grad_norm(grads: Sequence[torch.Tensor], max_norm: float = 0.0, workspace: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """fp32 tensor (norm, coefficient): the 2-norm of all gradients together
    and what brings it to max_norm (1 if it is below, or max_norm is 0; NaN
    for a norm that is not finite), both on the device."""
    grads, ptrs, numels, codes, devices = _grad_list(grads)
    index = next(iter(devices)) if devices else torch.cuda.current_device()
    t = np.zeros(len(ptrs), _SPAN_ROW)
    if len(ptrs):
        t["data"], t["numel"], t["dtype"] = np.frombuffer(ptrs, np.uint64), np.frombuffer(numels, np.int64), codes
    lib = library()
    need = int(lib.tps_grad_norm_workspace_bytes(len(ptrs)))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=index)
    if out is None:
        out = torch.empty(2, dtype=torch.float32, device=index)
    elif out.numel() != 2 or out.dtype != torch.float32 or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("shape")
    _check(lib.tps_grad_norm(t.ctypes.data, len(ptrs), float(max_norm), out.data_ptr(), *_room(workspace),
                             _raw_stream(out)))
    return out


def adamw_scalars(lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, weight_decay: float = 0.0,
                  seed: int = 0) -> torch.Tensor:
    """The numbers of an adamw_step that change from step to step, as four
    int32 words on the host: copied into a device tensor that was given as
    `scalars` when a CUDA graph was captured, they are what its replay uses."""
    h, s = TpsAdamwHyper(lr, beta1, beta2, 0.0, weight_decay, step, seed & 0xffffffff, 0), TpsAdamwScalars()
    _check(library().tps_adamw_prepare(ctypes.byref(h), ctypes.byref(s)))
    return torch.from_numpy(np.frombuffer(bytes(s), dtype=np.int32).copy())


def adamw_step(plan: AdamWPlan, grads: Sequence[torch.Tensor], lr: float, step: int, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
               grad_scale: Optional[torch.Tensor] = None, seed: Optional[int] = None,
               scalars: Optional[torch.Tensor] = None) -> None:
    """One AdamW step of every tensor of `plan`, in place.  step counts from
    1.  grad_scale: a device float that multiplies the gradients (grad_norm's
    coefficient); nothing changes if it is not finite.  seed: rounds e4m3
    moments, and bf16 weights without a master copy, at random (another seed
    each step); None rounds to nearest.  scalars: see adamw_scalars."""
    grads, ptrs, numels, codes, devices = _grad_list(grads)
    if numels != plan.numels:
        raise ValueError("shape")
    if not ptrs:
        return
    if devices != {plan.device}:
        raise ValueError("gradients on another GPU than the weights")
    for t, n, dtype in ((grad_scale, 1, torch.float32), (scalars, 4, torch.int32)):
        if t is not None and (not t.is_cuda or t.numel() != n or t.dtype != dtype or not t.is_contiguous()):
            raise ValueError("shape")
    t = plan.rows()
    t["grad"], t["grad_dtype"] = np.frombuffer(ptrs, np.uint64), codes
    h = TpsAdamwHyper(lr, beta1, beta2, eps, weight_decay, step, 0 if seed is None else seed & 0xffffffff,
                      0 if seed is None else 1)
    _check(library().tps_adamw_step(t.ctypes.data, len(ptrs), ctypes.byref(h),
                                    None if grad_scale is None else grad_scale.data_ptr(),
                                    None if scalars is None else scalars.data_ptr(), _raw_stream(grads[0])))
    # what autograd saved of the weights is not what they are now
    torch.autograd.graph.increment_version(plan.params)


def selftest_wait_timeout(limit_ns: int = 50_000_000) -> None:
    """Enqueue the bounded-wait self test (a wait nothing satisfies, given up
    after `limit_ns`); read the outcome with last_device_error()."""
    _check(library().tps_selftest_wait_timeout(int(limit_ns), _stream(None)))


def last_device_error(device=None) -> int:
    """Synchronize the current stream and read + clear the device error word."""
    return int(library().tps_last_device_error(_stream(device)))


class profile:
    """Context manager recording per-launch CUDA events inside the library.

        with profile() as p:
            ...
        p.summary  ->  {"gemm_tc:mlp_dX": dict(launches, ms, flops, bytes), ...}
    """

    def __enter__(self):
        library().tps_profile_reset(1)
        self.summary = {}
        return self

    def __exit__(self, *exc):
        lib = library()
        lib.tps_profile_stop()
        cap = 64
        names = (ctypes.c_char_p * cap)()
        launches = (ctypes.c_int64 * cap)()
        ms, fl, by = (ctypes.c_double * cap)(), (ctypes.c_double * cap)(), (ctypes.c_double * cap)()
        n = lib.tps_profile_summary(cap, names, launches, ms, fl, by)
        if n < 0:
            raise TpsError(-n, "profile summary failed")
        self.summary = {names[i].decode(): dict(launches=int(launches[i]), ms=float(ms[i]), flops=float(fl[i]),
                                                bytes=float(by[i])) for i in range(min(n, cap))}
        self.launches = int(lib.tps_launch_count())
        return False


def launch_count() -> int:
    return int(library().tps_launch_count())


def reset_launch_count():
    library().tps_profile_reset(0)
