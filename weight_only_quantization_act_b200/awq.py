"""Python binding of libawq (ctypes): argument marshalling only.

Every step of the computation runs in the CUDA kernels of ``lib/libawq.so``; this module turns torch
tensors into device pointers, allocates the caller-owned outputs and workspaces with torch, and passes
the current torch stream. It raises ``RuntimeError`` when the library is missing or a call fails; there
is no fallback path.

Tensors: X is a CUDA bfloat16 [N, K] matrix (tokens x in-features), W a CUDA bfloat16 [O, K] matrix
(torch ``nn.Linear.weight`` layout) or a list of such matrices that read the same X (stacked once).
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libawq.so")

AWQ_OK = 0
STATUS_NAMES = {0: "AWQ_OK", 1: "AWQ_ERR_INVALID_ARG", 2: "AWQ_ERR_UNSUPPORTED", 3: "AWQ_ERR_WORKSPACE",
                4: "AWQ_ERR_CUDA", 5: "AWQ_ERR_TIMEOUT"}
FLAG_EXACT_DIVISION = 0x1
FLAG_EXACT_POW = 0x2
FLAG_INJECT_STALL = 0x100
FLAG_SCALES_WEIGHT_AWARE = 0x10
FLAG_SCALES_RMS = 0x20
FLAG_QUANT_INT8 = 0x40
MAX_N_GRID = 64
GEMV_MAX_TOKENS = 8
MAX_EXPERTS = 1024

# name -> (restype, argtypes)
_P, _I64, _I, _U, _SZ, _D = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t,
                            ctypes.c_double)
SIGNATURES = {
    "awq_last_error": (ctypes.c_char_p, []),
    "awq_version": (_I, []),
    "awq_set_wait_limit_ns": (None, [ctypes.c_uint64]),
    "awq_set_experts_stall": (None, [_I]),
    "awq_set_profile_events": (None, [_P, _P]),
    "awq_act_stats_workspace_size": (_SZ, [_I64, _I64]),
    "awq_act_stats": (_I, [_P, _I64, _I64, _I64, _P, _SZ, _P, _P]),
    "awq_act_stats_noalloc": (_I, [_P, _I64, _I64, _I64, _P, _P]),
    "awq_scale_table_workspace_size": (_SZ, [_I64, _I]),
    "awq_scale_table": (_I, [_P, _I64, _I, _U, _P, _SZ, _P, _P]),
    "awq_scale_table_ex": (_I, [_P, _P, _I64, _I, _U, _P, _SZ, _P, _P]),
    "awq_search_workspace_size": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "awq_search": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _I, _I, _P, _SZ, _P, _P, _P, _P]),
    "awq_search_ex": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _I, _I, _U, _P, _SZ, _P, _P, _P, _P]),
    "awq_search_status": (_I, [_P, _SZ, _P]),
    "awq_search_get_layout": (_I, [_I64, _I64, _I64, _I, _I, _P]),
    "awq_quantize_pack": (_I, [_P, _I64, _I64, _I64, _P, _I, _P, _P, _P, _P]),
    "awq_quantize_pack_ex": (_I, [_P, _I64, _I64, _I64, _P, _I, _U, _P, _P, _P, _P]),
    "awq_quantize_pack_int8": (_I, [_P, _I64, _I64, _I64, _P, _U, _P, _P, _P]),
    "awq_scale_columns": (_I, [_P, _I64, _I64, _I64, _P, _I, _P, _I64, _P]),
    "awq_scale_rows": (_I, [_P, _I64, _I64, _I64, _P, _I, _P, _I64, _P]),
    "awq_w4a16_workspace_size": (_SZ, [_I64, _I64]),
    "awq_w4a16_gemm": (_I, [_P, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _I64, _P, _SZ, _P]),
    "awq_w4a16_gemv": (_I, [_P, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _I, _P, _I64, _P]),
    "awq_expert_sort_workspace_size": (_SZ, [_I64, _I64]),
    "awq_expert_sort": (_I, [_P, _I, _I64, _I64, _P, _SZ, _P, _P, _P, _P]),
    "awq_expert_gather": (_I, [_P, _I64, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _I64, _P]),
    "awq_expert_gather_backward": (_I, [_P, _I64, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _I64, _P]),
    "awq_expert_combine": (_I, [_P, _I64, _I64, _I64, _I64, _P, _P, _P, _I64, _P]),
    "awq_expert_combine_backward": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _I64, _P, _P]),
    "awq_w4a16_experts_workspace_size": (_SZ, [_I64, _I64, _I64, _I64]),
    "awq_w4a16_experts": (_I, [_P, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _I64, _I, _P, _I64, _P, _SZ, _P]),
}


class SearchLayout(ctypes.Structure):
    _fields_ = [("tile_n", ctypes.c_int64), ("tile_o", ctypes.c_int64), ("tiles_n", ctypes.c_int64),
                ("tiles_o", ctypes.c_int64), ("partials_per_tile", ctypes.c_int64), ("partials_offset", ctypes.c_size_t),
                ("workspace_bytes", ctypes.c_size_t)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libawq.so (once) and declare its C signatures. Fails loudly if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libawq.so not found at {path}; build it with "
                           "`python -m weight_only_quantization_act_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class AwqError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn} -> {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def _check(fn: str, status: int) -> None:
    if status != AWQ_OK:
        msg = load_library().awq_last_error().decode(errors="replace")
        raise AwqError(fn, status, msg)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t: torch.Tensor) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _bf16_matrix(name: str, t: torch.Tensor) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 2:
        raise TypeError(f"{name} must be a CUDA bfloat16 matrix")
    if t.stride(1) != 1:
        t = t.contiguous()
    return t


def _float_vector_out(name: str, out: torch.Tensor, n: int, device) -> torch.Tensor:
    """A caller-given float32 output of at least n elements, contiguous, on `device`: the kernels write n
    floats from its first element."""
    if (not isinstance(out, torch.Tensor) or out.dtype != torch.float32 or not out.is_cuda
            or out.device != device or out.numel() < n or not out.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA float32 tensor of at least {n} elements on {device}")
    return out


def _on_first_device(fn):
    """Run an entry point with its first tensor argument's device current, so that the library launches
    there and the stream passed is that device's current stream."""

    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        first = args[0] if args else next(iter(kwargs.values()))
        if isinstance(first, (list, tuple)):
            first = first[0]
        if isinstance(first, torch.Tensor) and first.is_cuda:
            with torch.cuda.device(first.device):
                return fn(*args, **kwargs)
        return fn(*args, **kwargs)

    return wrapper


def _workspace(nbytes: int, device, workspace: torch.Tensor | None) -> torch.Tensor:
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace too small: need {nbytes} bytes")
        return workspace
    # torch's caching allocator returns 512-byte aligned blocks; over-allocate to align to 1024
    raw = torch.empty(nbytes + 1024, dtype=torch.uint8, device=device)
    off = (-raw.data_ptr()) % 1024
    return raw[off:off + nbytes]


def set_wait_limit_ns(ns: int) -> None:
    load_library().awq_set_wait_limit_ns(int(ns))


def set_experts_stall(tile: int) -> None:
    """Test hook: later calls of w4a16_experts wait at this tile for what nobody signals (-1: nowhere)."""
    load_library().awq_set_experts_stall(int(tile))


def set_profile_events(before, after) -> None:
    """Record two torch.cuda.Event objects around the loss GEMM of later searches (None, None stops)."""
    lib = load_library()
    if before is None or after is None:
        lib.awq_set_profile_events(None, None)
        return
    for ev in (before, after):
        if not ev.cuda_event:
            ev.record()  # torch creates the underlying event lazily
    lib.awq_set_profile_events(ctypes.c_void_p(before.cuda_event), ctypes.c_void_p(after.cuda_event))


def version() -> int:
    return load_library().awq_version()


# --------------------------------------------------------------------------------------------- (1)
def act_stats_workspace_size(N: int, K: int) -> int:
    return load_library().awq_act_stats_workspace_size(N, K)


@_on_first_device
def act_stats(X: torch.Tensor, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """act_mean[k] = mean_i |X[i,k]| (fixed-order fp64 sum, rounded to fp32)."""
    lib = load_library()
    X = _bf16_matrix("X", X)
    N, K = X.shape
    if out is None:
        out = torch.empty(K, dtype=torch.float32, device=X.device)
    _float_vector_out("out", out, K, X.device)
    ws = _workspace(lib.awq_act_stats_workspace_size(N, K), X.device, workspace)
    _check("awq_act_stats", lib.awq_act_stats(_ptr(X), N, K, X.stride(0), _ptr(ws), ws.numel(), _ptr(out),
                                              _stream(stream)))
    return out


@_on_first_device
def act_stats_noalloc(X: torch.Tensor, out: torch.Tensor, stream=None) -> torch.Tensor:
    """Same statistic with no workspace, for callers that cannot allocate device memory at call time
    (the scratch is a fixed 16 MiB array inside the library; ceil(N/256)*K <= 2**21). ``out`` must be
    preallocated; calls that overlap on the GPU race on the shared scratch. Nothing is allocated here
    either: X must already have unit column stride (no contiguous copy is made)."""
    lib = load_library()
    if not isinstance(X, torch.Tensor) or X.dtype != torch.bfloat16 or not X.is_cuda or X.dim() != 2:
        raise TypeError("X must be a CUDA bfloat16 matrix")
    if X.stride(1) != 1:
        raise ValueError("X must have unit column stride (this entry point makes no copy)")
    N, K = X.shape
    _float_vector_out("out", out, K, X.device)
    _check("awq_act_stats_noalloc", lib.awq_act_stats_noalloc(_ptr(X), N, K, X.stride(0), _ptr(out),
                                                              _stream(stream)))
    return out


# --------------------------------------------------------------------------------------------- (2)
@_on_first_device
def scale_table(act_mean: torch.Tensor, n_grid: int = 20, exact_pow: bool = False, rule: str = "p4",
                weight_mean: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """float32 [n_grid, K] table of candidate scales; rule "p4" (default), "weight_aware" (needs
    weight_mean) or "rms"."""
    lib = load_library()
    K = act_mean.shape[0]
    table = torch.empty((n_grid, K), dtype=torch.float32, device=act_mean.device)
    ws = _workspace(lib.awq_scale_table_workspace_size(K, n_grid), act_mean.device, None)
    flags = (FLAG_EXACT_POW if exact_pow else 0) | RULE_FLAGS[rule]
    wm = _ptr(weight_mean) if weight_mean is not None else None
    _check("awq_scale_table_ex", lib.awq_scale_table_ex(_ptr(act_mean), wm, K, n_grid, flags, _ptr(ws), ws.numel(),
                                                        _ptr(table), _stream(stream)))
    return table


RULE_FLAGS = {"p4": 0, "weight_aware": FLAG_SCALES_WEIGHT_AWARE, "rms": FLAG_SCALES_RMS}


# --------------------------------------------------------------------------------------------- (3)-(4)
@dataclass
class SearchResult:
    losses: torch.Tensor      # float64 [n_grid] (device)
    best_j: torch.Tensor      # int32 [1] (device)
    scales: torch.Tensor      # float32 [K] (device)
    workspace: torch.Tensor   # uint8 (device), holds the scale table and the per-tile partial sums

    def ratio(self, n_grid: int) -> float:
        return int(self.best_j.item()) / n_grid


def stack_weights(W: torch.Tensor | Sequence[torch.Tensor]) -> torch.Tensor:
    """Linears that read the same X share one scale vector: stack their rows once."""
    if isinstance(W, torch.Tensor):
        return _bf16_matrix("W", W)
    mats = [_bf16_matrix("W", w) for w in W]
    return mats[0] if len(mats) == 1 else torch.cat(mats, dim=0)


def search_workspace_size(N: int, K: int, O: int, n_grid: int = 20, group: int = 128) -> int:
    return load_library().awq_search_workspace_size(N, K, O, group, n_grid)


def search_layout(N: int, K: int, O: int, n_grid: int = 20, group: int = 128) -> SearchLayout:
    lib = load_library()
    lay = SearchLayout()
    _check("awq_search_get_layout", lib.awq_search_get_layout(N, K, O, group, n_grid, ctypes.byref(lay)))
    return lay


@_on_first_device
def search(X: torch.Tensor, W, act_mean: torch.Tensor, n_grid: int = 20, group: int = 128, flags: int = 0,
           workspace: torch.Tensor | None = None, out: SearchResult | None = None, rule: str = "p4",
           quant: str = "int4", stream=None) -> SearchResult:
    """Grid search of the AWQ scale ratio for one linear (or stacked linears sharing X); rule selects the
    candidate scales ("p4" default, "weight_aware", "rms"); quant the weight quantizer ("int4" in groups
    of `group`, or "int8" symmetric per output channel, for which group is ignored)."""
    lib = load_library()
    flags |= RULE_FLAGS[rule]
    if quant == "int8":
        flags |= FLAG_QUANT_INT8
        group = 0
    elif quant != "int4":
        raise ValueError(f"quant must be 'int4' or 'int8', not {quant!r}")
    X = _bf16_matrix("X", X)
    W = stack_weights(W)
    N, K = X.shape
    O = W.shape[0]
    ws = _workspace(lib.awq_search_workspace_size(N, K, O, group, n_grid), X.device, workspace)
    if out is None:
        out = SearchResult(torch.empty(n_grid, dtype=torch.float64, device=X.device),
                           torch.empty(1, dtype=torch.int32, device=X.device),
                           torch.empty(K, dtype=torch.float32, device=X.device), ws)
    else:
        out.workspace = ws
    _check("awq_search_ex", lib.awq_search_ex(
        _ptr(X), N, K, X.stride(0), _ptr(W), O, W.stride(0), _ptr(act_mean), group, n_grid, flags, _ptr(ws),
        ws.numel(), _ptr(out.losses), _ptr(out.best_j), _ptr(out.scales), _stream(stream)))
    return out


def search_status(result: SearchResult, stream=None) -> int:
    """Synchronise and return the device status of the last search on this workspace (0 = ok)."""
    lib = load_library()
    return lib.awq_search_status(_ptr(result.workspace), result.workspace.numel(), _stream(stream))


def tile_partials(result: SearchResult, N: int, K: int, O: int, n_grid: int = 20) -> torch.Tensor:
    """View of the per-tile partial sums: float64 [n_grid, tiles_o, tiles_n, partials_per_tile]; entry e of
    a tile covers tile_n / partials_per_tile consecutive token rows."""
    lay = search_layout(N, K, O, n_grid)
    count = n_grid * lay.tiles_o * lay.tiles_n * lay.partials_per_tile
    raw = result.workspace[lay.partials_offset: lay.partials_offset + 8 * count]
    return raw.view(torch.float64).view(n_grid, lay.tiles_o, lay.tiles_n, lay.partials_per_tile)


# --------------------------------------------------------------------------------------------- (5)
@_on_first_device
def quantize_pack(W: torch.Tensor, scales: torch.Tensor, group: int = 128, flags: int = 0, stream=None):
    """(codes uint32 [O, K/8] as int32 storage, steps float32 [O, K/g], zeros float32 [O, K/g])."""
    lib = load_library()
    W = stack_weights(W)
    O, K = W.shape
    codes = torch.empty((O, K // 8), dtype=torch.int32, device=W.device)
    steps = torch.empty((O, K // group), dtype=torch.float32, device=W.device)
    zeros = torch.empty((O, K // group), dtype=torch.float32, device=W.device)
    _check("awq_quantize_pack_ex", lib.awq_quantize_pack_ex(
        _ptr(W), O, K, W.stride(0), _ptr(scales), group, flags, _ptr(codes), _ptr(steps), _ptr(zeros),
        _stream(stream)))
    return codes, steps, zeros


@_on_first_device
def quantize_pack_int8(W: torch.Tensor, scales: torch.Tensor, flags: int = 0, stream=None):
    """(codes int8 [O, K], steps float32 [O]): symmetric INT8, one step per output channel."""
    lib = load_library()
    W = stack_weights(W)
    O, K = W.shape
    codes = torch.empty((O, K), dtype=torch.int8, device=W.device)
    steps = torch.empty(O, dtype=torch.float32, device=W.device)
    _check("awq_quantize_pack_int8", lib.awq_quantize_pack_int8(
        _ptr(W), O, K, W.stride(0), _ptr(scales), flags, _ptr(codes), _ptr(steps), _stream(stream)))
    return codes, steps


@_on_first_device
def quantize_layer(X: torch.Tensor, W, n_grid: int = 20, group: int = 128, stream=None):
    """The whole path for one layer: statistic, search, and the packed artefact at the best scales."""
    act = act_stats(X, stream=stream)
    res = search(X, W, act, n_grid=n_grid, group=group, stream=stream)
    codes, steps, zeros = quantize_pack(W, res.scales, group=group, stream=stream)
    return dict(act_mean=act, losses=res.losses, best_j=res.best_j, scales=res.scales, codes=codes,
                steps=steps, zeros=zeros)


# --------------------------------------------------------------------------------------------- (6)
SCALE_MULTIPLY = 0
SCALE_DIVIDE = 1


def _as_matrix(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError("expected a CUDA bfloat16 tensor")
    return t.view(1, -1) if t.dim() == 1 else t


@_on_first_device
def scale_columns(A: torch.Tensor, s: torch.Tensor, divide: bool = False, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """out[r, c] = bf16(A[r, c] * s[c]) (or / s[c]); a 1-D tensor is one row. ``out=A`` works in place."""
    lib = load_library()
    A2 = _as_matrix(A)
    if out is None:
        out = torch.empty_like(A)
    O2 = _as_matrix(out)
    R, C = A2.shape
    _check("awq_scale_columns", lib.awq_scale_columns(_ptr(A2), R, C, A2.stride(0), _ptr(s),
                                                      SCALE_DIVIDE if divide else SCALE_MULTIPLY, _ptr(O2),
                                                      O2.stride(0), _stream(stream)))
    return out


@_on_first_device
def scale_rows(A: torch.Tensor, s: torch.Tensor, divide: bool = False, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """out[r, c] = bf16(A[r, c] * s[r]) (or / s[r]); a 1-D tensor is scaled element-wise."""
    lib = load_library()
    one_d = A.dim() == 1
    A2 = A.view(-1, 1) if one_d else A
    if one_d:
        # a vector scaled element-wise by s is a 1 x C column scaling
        return scale_columns(A, s, divide=divide, out=out, stream=stream)
    if out is None:
        out = torch.empty_like(A)
    R, C = A2.shape
    _check("awq_scale_rows", lib.awq_scale_rows(_ptr(A2), R, C, A2.stride(0), _ptr(s),
                                                SCALE_DIVIDE if divide else SCALE_MULTIPLY, _ptr(out),
                                                out.stride(0), _stream(stream)))
    return out


def fold_norm_linear(norm_weight: torch.Tensor, linears: Sequence[torch.Tensor], s: torch.Tensor, stream=None):
    """NormLinearSubgraph: gamma / s for the norm, W diag(s) for every linear reading its output (in place)."""
    scale_columns(norm_weight, s, divide=True, out=norm_weight, stream=stream)
    for w in linears:
        scale_columns(w, s, out=w, stream=stream)


def fold_linear_linear(w1: torch.Tensor, b1: torch.Tensor | None, w2: torch.Tensor, s: torch.Tensor, stream=None):
    """LinearLinearSubgraph / OVSubgraph (multi-head) / UpDownSubgraph: rows (and bias) of the source linear
    divided by s, columns of the target linear multiplied by s (in place)."""
    scale_rows(w1, s, divide=True, out=w1, stream=stream)
    if b1 is not None:
        scale_columns(b1, s, divide=True, out=b1, stream=stream)
    scale_columns(w2, s, out=w2, stream=stream)


# --------------------------------------------------------------------------------------------- (7)
@_on_first_device
def w4a16_gemm(X: torch.Tensor, codes: torch.Tensor, steps: torch.Tensor, zeros: torch.Tensor,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X' deq(W)^T (bf16 [M, O]) from packed codes [O, K/8], steps and zeros [O, K/128]."""
    lib = load_library()
    X = _bf16_matrix("X", X)
    M, K = X.shape
    O = codes.shape[0]
    if out is None:
        out = torch.empty((M, O), dtype=torch.bfloat16, device=X.device)
    if workspace is None:  # zero-filled once; the library keeps its counters zero from call to call
        workspace = torch.zeros(lib.awq_w4a16_workspace_size(K, O), dtype=torch.uint8, device=X.device)
    _check("awq_w4a16_gemm", lib.awq_w4a16_gemm(_ptr(X), M, K, X.stride(0), _ptr(codes), _ptr(steps), _ptr(zeros),
                                                O, _ptr(out), out.stride(0), _ptr(workspace), workspace.numel(),
                                                _stream(stream)))
    return out


# --------------------------------------------------------------------------------------------- (8)
def _on_stream(fn):
    """Run an entry point on its first tensor argument's device, and on `stream` where one is given: what it
    allocates then belongs to that stream, so a workspace is not handed to other work while the stream uses it. The caller's
    tensors are recorded with the stream, so one that is freed after the call is not reused before the stream has read it."""

    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kwargs):
        first = args[0] if args else None
        if not isinstance(first, torch.Tensor):  # arguments given by name, in any order
            first = next((t for t in (*args, *kwargs.values()) if isinstance(t, torch.Tensor)), None)
        on_cuda = first is not None and first.is_cuda
        if stream is not None:
            if on_cuda and stream.device != first.device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {first.device}")
            with torch.cuda.stream(stream):
                result = fn(*args, **kwargs)
            _record(stream, (*args, *kwargs.values()))
            return result
        if not on_cuda or first.get_device() == torch.cuda.current_device():
            return fn(*args, **kwargs)
        with torch.cuda.device(first.device):
            return fn(*args, **kwargs)

    return wrapper


def _record(stream, values) -> None:
    for v in values:
        if isinstance(v, torch.Tensor):
            if v.is_cuda:
                v.record_stream(stream)
        elif isinstance(v, ExpertSort):
            _record(stream, (v.offsets, v.order, v.pos))
        elif isinstance(v, (list, tuple)):
            _record(stream, v)


def _current_stream() -> int:
    """Handle of the current stream of the current device (torch.cuda.current_stream builds an object around it, which
    takes as long as the rest of a call)."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _rows(name: str, t: torch.Tensor, device=None) -> torch.Tensor:
    """A bf16 matrix argument on `device`, with unit column stride."""
    t = _bf16_matrix(name, t)
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t


def _ld(t: torch.Tensor) -> int:
    """Row stride in elements; a single row's stride does not matter and torch may give any number for it."""
    rows, cols = t.shape
    return t.stride(0) if rows > 1 else -(-cols // 8) * 8


def _tensor(name: str, t: torch.Tensor, dtype, shape, device) -> int:
    """The address of a contiguous argument of this type and shape on `device`."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a tensor of {dtype}")
    if t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be contiguous, of shape {list(shape)} and on {device}")
    return t.data_ptr()


def _on_device(name: str, t: torch.Tensor, device) -> None:
    """A caller's workspace: its bytes from its first element on are the library's."""
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {device}")


def _rows_out(name: str, out: torch.Tensor | None, rows: int, cols: int, like: torch.Tensor) -> torch.Tensor:
    """A bf16 output matrix: a new one, or the caller's."""
    if out is None:
        return like.new_empty((rows, cols))
    if not isinstance(out, torch.Tensor) or out.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be a bfloat16 tensor")
    if out.shape != (rows, cols) or out.device != like.device or (cols > 1 and out.stride(1) != 1):
        raise ValueError(f"{name} must be [{rows}, {cols}] with unit column stride on {like.device}")
    return out


def _packed(codes, steps, zeros, lead: tuple, K: int, device) -> tuple:
    """O of packed weights [*lead, O, ...] and their addresses, after checking them against X's K in-features."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != len(lead) + 2:
        raise TypeError(f"codes must be a {len(lead) + 2}-dimensional int32 tensor, as quantize_pack gives it")
    O = codes.shape[-2]
    groups = (*lead, O, K // 128)
    return (O, _tensor("codes", codes, torch.int32, (*lead, O, K // 8), device),
            _tensor("steps", steps, torch.float32, groups, device), _tensor("zeros", zeros, torch.float32, groups, device))


@_on_stream
def w4a16_gemv(X: torch.Tensor, codes: torch.Tensor, steps: torch.Tensor, zeros: torch.Tensor,
               bias: torch.Tensor | None = None, gated: bool = False, out: torch.Tensor | None = None,
               *, stream=None) -> torch.Tensor:
    """Y = X' deq(W)^T (+ bias) for 1 to 8 tokens in one launch (bf16 [M, O]). With ``gated`` the rows of W are a
    gate projection's, then an up projection's, and Y = silu(gate) * up (bf16 [M, O / 2])."""
    lib = load_library()
    X = _rows("X", X)
    M, K = X.shape
    device = X.device
    O, c, s, z = _packed(codes, steps, zeros, (), K, device)
    bias = None if bias is None else _tensor("bias", bias, torch.bfloat16, (O,), device)
    out = _rows_out("out", out, M, O // 2 if gated else O, X)
    _check("awq_w4a16_gemv", lib.awq_w4a16_gemv(X.data_ptr(), M, K, _ld(X), c, s, z, O, bias, bool(gated), out.data_ptr(),
                                                out.stride(0), _current_stream()))
    return out


# --------------------------------------------------------------------------------------------- (9)
@dataclass
class ExpertSort:
    """Where a router's picks ids [T, k] stand in expert order: offsets int32 [E + 1] (first row of each expert),
    order int32 [T * k] (slot t * k + j of each row, -1 behind the last), pos int32 [T, k] (row of each slot, -1 where
    an id names no expert)."""
    offsets: torch.Tensor
    order: torch.Tensor
    pos: torch.Tensor

    def checked(self, device) -> tuple:
        """(T, k, E) and the addresses of offsets, order and pos, after checking the three against each other."""
        if not isinstance(self.pos, torch.Tensor) or self.pos.dim() != 2 or self.offsets.dim() != 1:
            raise TypeError("an ExpertSort holds offsets [E + 1], order [T * k] and pos [T, k]")
        T, k = self.pos.shape
        E = self.offsets.shape[0] - 1
        return (T, k, E, _tensor("offsets", self.offsets, torch.int32, (E + 1,), device),
                _tensor("order", self.order, torch.int32, (T * k,), device),
                _tensor("pos", self.pos, torch.int32, (T, k), device))


@_on_stream
def expert_sort(ids: torch.Tensor, n_experts: int, workspace: torch.Tensor | None = None, *, stream=None) -> ExpertSort:
    """Rows in order of (expert, token, pick) for a router's picks ids [T, k] (int32 or int64). Ids outside
    [0, n_experts) name no expert."""
    lib = load_library()
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64) or not ids.is_cuda or ids.dim() != 2:
        raise TypeError("ids must be a CUDA int32 or int64 matrix [tokens, picks]")
    ids = ids.contiguous()
    n = ids.numel()
    offsets = ids.new_empty(max(n_experts, 0) + 1, dtype=torch.int32)
    order = ids.new_empty(n, dtype=torch.int32)
    pos = ids.new_empty(ids.shape, dtype=torch.int32)
    need = lib.awq_expert_sort_workspace_size(n, n_experts)
    ws = _workspace(need, ids.device, workspace) if need else None
    if need:
        _on_device("workspace", ws, ids.device)
    _check("awq_expert_sort", lib.awq_expert_sort(
        ids.data_ptr(), ids.element_size(), n, n_experts, ws.data_ptr() if need else None, need, offsets.data_ptr(),
        order.data_ptr(), pos.data_ptr(), _current_stream()))
    return ExpertSort(offsets, order, pos)


def _scales(scales, E: int, K: int, device):
    return None if scales is None else _tensor("scales", scales, torch.float32, (E, K), device)


@_on_stream
def expert_gather(X: torch.Tensor, sort: ExpertSort, scales: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  *, stream=None) -> torch.Tensor:
    """Token rows in expert order, bf16 [T * k, K]; with ``scales`` (float32 [E, K]) each divided by its expert's AWQ
    scales, as scale_columns(divide=True) does. Rows behind the last routed one are not written."""
    lib = load_library()
    X = _rows("X", X)
    T, k, E, offsets, order, _ = sort.checked(X.device)
    K = X.shape[1]
    if X.shape[0] != T:
        raise ValueError(f"X has {X.shape[0]} rows, the sort {T} tokens")
    out = _rows_out("out", out, T * k, K, X)
    _check("awq_expert_gather", lib.awq_expert_gather(
        X.data_ptr(), T, K, _ld(X), k, offsets, E, order, _scales(scales, E, K, X.device), out.data_ptr(), _ld(out),
        _current_stream()))
    return out


@_on_stream
def expert_gather_backward(dXs: torch.Tensor, sort: ExpertSort, scales: torch.Tensor | None = None,
                           out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    """Gradient of expert_gather: dX[t] = the sum of its rows of dXs (each divided by its expert's scales)."""
    lib = load_library()
    dXs = _rows("dXs", dXs)
    T, k, E, offsets, _, pos = sort.checked(dXs.device)
    K = dXs.shape[1]
    if dXs.shape[0] != T * k:
        raise ValueError(f"dXs has {dXs.shape[0]} rows, the sort {T * k}")
    out = _rows_out("out", out, T, K, dXs)
    _check("awq_expert_gather_backward", lib.awq_expert_gather_backward(
        dXs.data_ptr(), T, K, _ld(dXs), k, offsets, E, pos, _scales(scales, E, K, dXs.device), out.data_ptr(), _ld(out),
        _current_stream()))
    return out


@_on_stream
def expert_combine(Ys: torch.Tensor, sort: ExpertSort, weights: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    """Y[t] = sum_j weights[t, j] * Ys[pos[t, j]] (bf16 [T, O], fp32 sums; weights float32 [T, k], ones if None)."""
    lib = load_library()
    Ys = _rows("Ys", Ys)
    T, k, _, _, _, pos = sort.checked(Ys.device)
    O = Ys.shape[1]
    if Ys.shape[0] != T * k:
        raise ValueError(f"Ys has {Ys.shape[0]} rows, the sort {T * k}")
    w = None if weights is None else _tensor("weights", weights, torch.float32, (T, k), Ys.device)
    out = _rows_out("out", out, T, O, Ys)
    _check("awq_expert_combine", lib.awq_expert_combine(
        Ys.data_ptr(), T, O, _ld(Ys), k, pos, w, out.data_ptr(), _ld(out), _current_stream()))
    return out


@_on_stream
def expert_combine_backward(dY: torch.Tensor, Ys: torch.Tensor, sort: ExpertSort, weights: torch.Tensor,
                            out: torch.Tensor | None = None, *, stream=None):
    """Gradients of expert_combine: (dYs bf16 [T * k, O], dweights float32 [T, k]). ``out`` takes dYs; its rows behind
    the last routed one are not written."""
    lib = load_library()
    dY = _rows("dY", dY)
    Ys = _rows("Ys", Ys, dY.device)
    T, k, _, _, _, pos = sort.checked(dY.device)
    O = dY.shape[1]
    if dY.shape[0] != T or tuple(Ys.shape) != (T * k, O):
        raise ValueError(f"dY {list(dY.shape)} and Ys {list(Ys.shape)} do not fit a sort of {T} tokens, {k} picks")
    w = _tensor("weights", weights, torch.float32, (T, k), dY.device)
    out = _rows_out("out", out, T * k, O, dY)
    dweights = weights.new_empty((T, k))
    _check("awq_expert_combine_backward", lib.awq_expert_combine_backward(
        dY.data_ptr(), T, O, _ld(dY), Ys.data_ptr(), _ld(Ys), k, pos, w, out.data_ptr(), _ld(out), dweights.data_ptr(),
        _current_stream()))
    return out, dweights


# --------------------------------------------------------------------------------------------- (10)
@_on_stream
def w4a16_experts_workspace(codes: torch.Tensor, rows: int) -> torch.Tensor:
    """A zero-filled workspace for w4a16_experts with these codes [E, O, K / 8] and up to `rows` sorted rows."""
    E, O, words = codes.shape
    nbytes = load_library().awq_w4a16_experts_workspace_size(rows, E, words * 8, O)
    return torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=codes.device)


@_on_stream
def w4a16_status(workspace: torch.Tensor, *, stream=None) -> int:
    """Synchronise and return the device status of the calls of w4a16_experts or w4a16_gemm on this workspace (0 = ok, 5 = a
    device wait gave up; STATUS_NAMES). After a timeout zero the workspace before its next use."""
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise TypeError("workspace must be a CUDA tensor")
    _on_device("workspace", workspace, workspace.device)
    return load_library().awq_search_status(workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                            _current_stream())


@_on_stream
def w4a16_experts(Xs: torch.Tensor, offsets: torch.Tensor, codes: torch.Tensor, steps: torch.Tensor, zeros: torch.Tensor,
                  gated: bool = False, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  *, stream=None) -> torch.Tensor:
    """Products of sorted rows with their experts' packed weights: Y[r] = Xs[r] deq(W_e)^T for offsets[e] <= r <
    offsets[e + 1] (codes [E, O, K/8], steps and whole-numbered zeros [E, O, K/128]); ``gated`` as in w4a16_gemv. Rows behind the last
    routed one are not written.

    A device wait that gives up (set_wait_limit_ns) leaves rows of experts with more than 8 rows as they were and its status in the
    workspace, where w4a16_status finds it; until the workspace is zeroed, later calls on it leave such rows alone too.
    Without a workspace of the caller's a timeout is not reported."""
    lib = load_library()
    Xs = _rows("Xs", Xs)
    R, K = Xs.shape
    E = codes.shape[0] if isinstance(codes, torch.Tensor) and codes.dim() == 3 else 0  # _packed refuses the others
    O, c, s, z = _packed(codes, steps, zeros, (E,), K, Xs.device)
    first = _tensor("offsets", offsets, torch.int32, (E + 1,), Xs.device)
    out = _rows_out("out", out, R, O // 2 if gated else O, Xs)
    if workspace is None:
        workspace = w4a16_experts_workspace(codes, R)
    _on_device("workspace", workspace, Xs.device)
    _check("awq_w4a16_experts", lib.awq_w4a16_experts(
        Xs.data_ptr(), R, K, _ld(Xs), first, E, c, s, z, O, bool(gated), out.data_ptr(), out.stride(0), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _current_stream()))
    return out


@_on_stream
def w4a16_moe(X: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate_up, down, scales: torch.Tensor | None = None,
              workspaces=(None, None), out: torch.Tensor | None = None, *, down_scales: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """A feed-forward block of quantized experts: tokens X [T, K] sorted by their picks ids [T, k], divided by each
    expert's scales, through silu(gate) * up and the down projection of their experts, and back, weighted. gate_up and
    down are (codes, steps, zeros) of all experts, as quantize_experts gives them; scales [E, K] and down_scales [E, I] the
    scales that it gave with each, None where they are folded into what comes before (the down projection's into the up
    rows: fold_linear_linear before packing those). workspaces: one of w4a16_experts_workspace
    for each of the two products, whose w4a16_status then tells of a device timeout (without them it is not reported)."""
    sort = expert_sort(ids, gate_up[0].shape[0])
    Xs = expert_gather(X, sort, scales=scales)
    H = w4a16_experts(Xs, sort.offsets, *gate_up, gated=True, workspace=workspaces[0])
    if down_scales is not None:  # sorted rows stay where they are: each row is its own token
        rows = torch.arange(H.shape[0], dtype=torch.int32, device=H.device)
        H = expert_gather(H, ExpertSort(sort.offsets, rows, rows[:, None]), scales=down_scales)
    Ys = w4a16_experts(H, sort.offsets, *down, workspace=workspaces[1])
    return expert_combine(Ys, sort, weights=weights, out=out)


@_on_stream
def quantize_experts(X: torch.Tensor, ids: torch.Tensor, W: Sequence[torch.Tensor], n_grid: int = 20, group: int = 128,
                     *, stream=None):
    """quantize_layer for every expert of a block, each on the calibration tokens that its router sends there: tokens
    X [N, K] with picks ids [N, k], W one [O, K] weight (or stacked weights) per expert. Returns scales [E, K] and codes, steps,
    zeros [E, O, ...], and losses, best_j per expert. An expert without a token is quantized at scales of one (losses NaN,
    best_j 0). Reads the experts' row counts on the host (one synchronisation)."""
    E = len(W)
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise TypeError("X must be a CUDA bfloat16 matrix")
    rows = set()
    for e, w in enumerate(W):  # a weight wider than X would be read with scales that are not there
        parts = [w] if isinstance(w, torch.Tensor) else list(w)
        for part in parts:
            if part.dim() != 2 or part.shape[1] != X.shape[1] or part.device != X.device:
                raise ValueError(f"expert {e}: a weight must be [O, {X.shape[1]}] on {X.device}")
        rows.add(sum(part.shape[0] for part in parts))
    if len(rows) != 1:
        raise ValueError(f"every expert needs as many weight rows as the others, not {sorted(rows)}")
    mats = [stack_weights(w) for w in W]
    sort = expert_sort(ids, E)
    Xs = expert_gather(X, sort)
    edges = sort.offsets.tolist()
    parts = []
    for e, w in enumerate(mats):
        if edges[e + 1] > edges[e]:
            parts.append(quantize_layer(Xs[edges[e]:edges[e + 1]], w, n_grid=n_grid, group=group))
            continue
        scales = torch.ones(X.shape[1], dtype=torch.float32, device=X.device)
        codes, steps, zeros = quantize_pack(w, scales, group=group)
        parts.append(dict(scales=scales, codes=codes, steps=steps, zeros=zeros,
                          losses=torch.full((n_grid,), float("nan"), dtype=torch.float64, device=X.device),
                          best_j=torch.zeros(1, dtype=torch.int32, device=X.device)))
    return {name: torch.stack([p[name] for p in parts])
            for name in ("scales", "codes", "steps", "zeros", "losses", "best_j")}
