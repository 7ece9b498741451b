"""Python binding of libtpfuse (ctypes).

Argument marshalling only: every step of the fused path runs in the HIP
kernels of ``libtpfuse.so``.  PyTorch supplies device memory (tensors) and
the stream (``torch.cuda.current_stream()``).  If the library is not built
the import of a call fails loudly; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libtpfuse.so")
ARGS_PATH = os.path.join(_HERE, "lib", "_args.so")

# Status codes, dtypes, schedulers, semantics and op ids (include/tpfuse.h).
OK = 0
ERR_INVALID_ARG, ERR_SHAPE, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_UNSUPPORTED, ERR_HIP, ERR_TIMEOUT = range(-1, -8, -1)
BF16, F32 = 0, 1
(SCHED_AUTO, SCHED_PERSISTENT, SCHED_TWO_STREAM, SCHED_UNFUSED, SCHED_GEMM_ONLY, SCHED_REDUCE_ONLY, SCHED_TILE,
 SCHED_FOLD, SCHED_STATIONARY) = range(9)
ALLREDUCE, REDUCESCATTER = 0, 1
OP_MATMUL_ALLREDUCE, OP_MATMUL_REDUCESCATTER, OP_ALLGATHER_MATMUL, OP_MATMUL_DX, OP_MLP_SP = range(5)
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2
NORM_MAX_H = 32768
MAX_SHARDS = 16
MAX_CHUNKS = 64
NOALLOC_SCRATCH_BYTES = 64 << 20

SCHEDS = {"auto": SCHED_AUTO, "persistent": SCHED_PERSISTENT, "two_stream": SCHED_TWO_STREAM,
          "unfused": SCHED_UNFUSED, "gemm_only": SCHED_GEMM_ONLY, "reduce_only": SCHED_REDUCE_ONLY,
          "tile": SCHED_TILE, "fold": SCHED_FOLD, "stationary": SCHED_STATIONARY}

_VP = ctypes.c_void_p
_PP = ctypes.c_void_p      # an array of addresses: a ctypes array, or bytes from `_operands`
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float

# name -> (restype, argtypes); the set of exported functions of include/tpfuse.h
SIGNATURES = {
    "tpf_create": (_I, [ctypes.POINTER(_VP), _I]),
    "tpf_destroy": (_I, [_VP]),
    "tpf_workspace_size": (_SZ, [_I, _I, _I64, _I64, _I64, _I, _I]),
    "tpf_matmul_allreduce": (_I, [_VP, _I, _I64, _I64, _I64, _PP, _PP, _VP, _I, _I, _I, _VP, _SZ, _VP]),
    "tpf_matmul_allreduce_noalloc": (_I, [_VP, _I, _I64, _I64, _I64, _PP, _PP, _VP, _I, _I, _I, _VP]),
    "tpf_matmul_reducescatter": (_I, [_VP, _I, _I64, _I64, _I64, _PP, _PP, _PP, _I, _I, _I, _VP, _SZ, _VP]),
    "tpf_allgather_matmul": (_I, [_VP, _I, _I64, _I64, _I64, _PP, _VP, _VP, _VP, _I, _I, _I, _VP, _SZ, _VP]),
    "tpf_matmul_dx": (_I, [_VP, _I, _I, _I64, _I64, _I64, _PP, _PP, _PP, _I, _I, _I, _VP, _SZ, _VP]),
    "tpf_weight_grad": (_I, [_VP, _I, _I64, _I64, _I64, _PP, _PP, _PP, _I, _VP]),
    "tpf_mlp_sp": (_I, [_VP, _I, _I64, _I64, _I64, _PP, _PP, _PP, _VP, _PP, _PP, _I, _I, _I, _VP, _SZ, _VP]),
    "tpf_block_norm": (_I, [_VP, _I, _I64, _I64, _VP, _I, _PP, _I, _VP, _VP, _VP, _I, _I, _F, _F, _F, _I, _VP, _VP,
                            _VP, _VP]),
    "tpf_block_norm_backward_ws": (_SZ, [_I64, _I64]),
    "tpf_block_norm_backward": (_I, [_VP, _I, _I64, _I64, _VP, _VP, _VP, _I, _PP, _I, _VP, _VP, _VP, _VP, _I, _I, _F,
                                     _F, _I, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "tpf_stash_pack": (_I, [_VP, _I, _I64, _I64, _PP, _I, _PP, _PP, _PP, _VP]),
    "tpf_stash_backward": (_I, [_VP, _I, _I64, _I64, _PP, _PP, _PP, _PP, _PP, _VP]),
    "tpf_stash_weight_grad_ws": (_SZ, [_I, _I64, _I64, _I64]),
    "tpf_stash_weight_grad": (_I, [_VP, _I, _I64, _I64, _I64, _PP, _PP, _PP, _PP, _I, _VP, _SZ, _VP]),
    "tpf_qweight_matmul_ws": (_SZ, [_I, _I64, _I64, _I64, _I]),
    "tpf_qweight_matmul": (_I, [_VP, _I, _I64, _I64, _I64, _I, _PP, _PP, _PP, _PP, _I, _VP, _I, _VP, _SZ, _VP]),
    "tpf_sync_status": (_I, [_VP, _VP]),
    "tpf_debug_set_wait": (_I, [_VP, _I64, _I]),
    "tpf_debug_set_delay": (_I, [_VP, ctypes.c_uint32, _I, _I]),
    "tpf_debug_set_timeline": (_I, [_VP, _VP, _I]),
    "tpf_debug_set_kernel_timing": (_I, [_VP, _I]),
    "tpf_debug_kernel_times": (_I, [_VP, ctypes.POINTER(ctypes.c_float), _I]),
    "tpf_debug_last_sched": (_I, [_VP]),
    "tpf_rowpar_dx": (_I, [_VP, _I, _I64, _I64, _I64, _VP, _VP, _VP, _I, _VP]),
    "tpf_status_string": (ctypes.c_char_p, [_I]),
    "tpf_last_error": (ctypes.c_char_p, []),
    "tpf_version": (_I, []),
}

_lib: Optional[ctypes.CDLL] = None
_args = None                # the MLP block calls' native argument checks (csrc/tpf_args.cpp)
_args_error = ""            # why they could not be loaded


class TpfError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libtpfuse error {code}: {msg}")
        self.code = code


def load() -> ctypes.CDLL:
    """Load the in-tree libtpfuse.so (raises if it has not been built)."""
    global _lib, _args, _args_error
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m tensor_gemm_reduction_amd.build`")
    # Before the library: loaded after it, a 4-bit product over 8 shards takes 25.4 us of host time instead of 23.5.
    spec = importlib.util.spec_from_file_location(
        "_args", ARGS_PATH, loader=importlib.machinery.ExtensionFileLoader("_args", ARGS_PATH))
    try:
        native = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(native)
        _args = native
    except ImportError as e:     # not built, or against another torch: only the MLP block's calls need it
        _args, _args_error = None, str(e)
    lib = ctypes.CDLL(LIB_PATH, mode=ctypes.RTLD_GLOBAL)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _native():
    """The native argument checks of the MLP block's calls."""
    if _args is None:
        load()
        if _args is None:
            raise RuntimeError(f"{ARGS_PATH} cannot be loaded ({_args_error}): build it with "
                               "`python -m tensor_gemm_reduction_amd.build`")
    return _args


def check(code: int) -> None:
    if code != OK:
        msg = load().tpf_last_error().decode(errors="replace")
        raise TpfError(code, msg)


def ptr_array(ptrs: Sequence[int]):
    arr = (ctypes.c_void_p * max(1, len(ptrs)))()
    for i, p in enumerate(ptrs):
        arr[i] = p
    return arr


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return BF16
    if dt == torch.float32:
        return F32
    raise ValueError(f"output dtype must be bfloat16 or float32, got {dt}")


MSG_BF16 = 0x100           # TPF_MSG_BF16: shard partials ("messages") kept as bf16
MESSAGES = {"fp32": 0, "bf16": MSG_BF16}


def _sched(s, message: str = "fp32") -> int:
    return (SCHEDS[s] if isinstance(s, str) else int(s)) | MESSAGES[message]


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _on(stream):
    """Allocation context for buffers the library writes on `stream`.

    torch's caching allocator ties a block to the stream that was current
    when it was allocated and may hand it out again as soon as the tensor is
    freed, ordered only against that stream.  Buffers the binding allocates
    for a call (outputs, workspace) are therefore allocated with the call's
    stream current, so a freed workspace cannot be reused while the library's
    kernels on that stream still write it."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


class Handle:
    """A libtpfuse handle bound to one device (owns a side stream, events, counters)."""

    def __init__(self, device: int = 0):
        lib = load()
        h = ctypes.c_void_p()
        check(lib.tpf_create(ctypes.byref(h), int(device)))
        self._h = h
        self.device = device

    @property
    def ptr(self):
        return self._h

    def close(self):
        if self._h is not None and self._h.value:
            load().tpf_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def sync_status(self, stream=None) -> int:
        return load().tpf_sync_status(self._h, _stream_ptr(stream))

    def debug_set_wait(self, spins: int, unreachable: bool) -> None:
        check(load().tpf_debug_set_wait(self._h, int(spins), 1 if unreachable else 0))

    def set_delay(self, seed: int, period: int, sleeps: int) -> None:
        """Perturb producer timing (a seeded subset of tasks sleeps before
        publishing); period = 0 turns it off."""
        check(load().tpf_debug_set_delay(self._h, int(seed) & 0xFFFFFFFF, int(period), int(sleeps)))

    def set_timeline(self, events: Optional[torch.Tensor]) -> None:
        """Record persistent-kernel task events into `events` (uint8 device tensor, 32 B per event)."""
        if events is None:
            check(load().tpf_debug_set_timeline(self._h, None, 0))
        else:
            check(load().tpf_debug_set_timeline(self._h, events.data_ptr(), events.numel() // 32))

    def set_kernel_timing(self, enable: bool) -> None:
        """Record timing events around each later call's dominant kernel launch."""
        check(load().tpf_debug_set_kernel_timing(self._h, 1 if enable else 0))

    def last_sched(self) -> str:
        """Name of the scheduler the last reducing or AllGather call on this
        handle ran (AUTO resolved), or "" before the first."""
        v = load().tpf_debug_last_sched(self._h)
        if v < -1:
            check(v)
        names = {code: name for name, code in SCHEDS.items()}
        return names.get(v, "")

    def kernel_times(self, max_records: int = 256) -> List[float]:
        """Durations (ms) of the recorded launches, oldest first; clears the record."""
        buf = (ctypes.c_float * max_records)()
        n = load().tpf_debug_kernel_times(self._h, buf, max_records)
        if n < 0:
            check(n)
        return [float(buf[i]) for i in range(n)]


TIMELINE_DTYPE = [("ticket", "<u4"), ("kind", "<u2"), ("chunk", "<u2"), ("block", "<u2"), ("xcd", "<u2"),
                  ("mid", "<u4"), ("t_start", "<u8"), ("t_end", "<u8")]


def timeline_events(events: torch.Tensor, count: int):
    """Decode the first `count` timeline records into a numpy structured array."""
    import numpy as np
    raw = events[: count * 32].cpu().numpy()
    return raw.view(np.dtype(TIMELINE_DTYPE))


_default_handles = {}


def default_handle(device: Optional[int] = None, stream=None) -> Handle:
    """The binding's handle for (device, stream).

    A handle runs one call at a time (its persistent and tile schedulers keep
    work-queue and readiness counters in the handle), and calls on different
    streams may run at the same time, so every stream gets its own default
    handle."""
    dev = torch.cuda.current_device() if device is None else device
    key = (int(dev), _stream_ptr(stream) if stream is not None else _stream_ptr(torch.cuda.current_stream(dev)))
    h = _default_handles.get(key)
    if h is None:
        h = Handle(dev)
        _default_handles[key] = h
    return h


OUT_DTYPES = (torch.bfloat16, torch.float32)


def _need(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _check(name: str, ts, shape, dtypes=(torch.bfloat16,), device=None) -> torch.device:
    """Refuse, before any library call, tensors the library cannot be handed.

    The library reads and writes through raw device pointers whose extents it
    derives from the shape arguments alone, so a tensor on the host, on
    another device, of another shape or strided would be accessed out of
    bounds on the GPU.  Every tensor in `ts` must be a contiguous GPU tensor
    on `device` (default: the first one's), of shape `shape` and one of
    `dtypes`.  Returns the device."""
    _need(len(ts) >= 1, f"{name}: no tensors given")
    dev = device if device is not None else getattr(ts[0], "device", None)
    shape = tuple(shape)
    ok = getattr(dev, "type", None) == "cuda"
    for t in ts:        # one combined test per tensor; the message is built only on failure
        if not (ok and isinstance(t, torch.Tensor) and t.device == dev and t.dtype in dtypes
                and t.shape == shape and t.is_contiguous()):
            ok = False
            break
    if not ok:
        for i, t in enumerate(ts):
            lab = f"{name}[{i}]" if len(ts) > 1 else name
            _need(isinstance(t, torch.Tensor), f"{lab} is not a tensor")
            _need(t.device.type == "cuda", f"{lab} is on {t.device}, not on a GPU")
            _need(t.device == dev, f"{lab} is on {t.device}, expected {dev}")
            _need(t.dtype in dtypes, f"{lab} has dtype {t.dtype}, expected one of {[str(d) for d in dtypes]}")
            _need(tuple(t.shape) == shape, f"{lab} has shape {tuple(t.shape)}, expected {shape}")
            _need(t.is_contiguous(), f"{lab} is not contiguous")
        _need(False, f"{name}: the device {dev} is not a GPU")
    return dev


def _check_shards(name: str, ts, p: int) -> None:
    _need(len(ts) == p, f"{name}: {len(ts)} tensors given, expected one per shard ({p})")


def _check_ws(ws, dev) -> None:
    if ws is not None:
        _check("ws", [ws], tuple(ws.shape), (ws.dtype,), dev)


def _handle(handle, dev, stream=None) -> "Handle":
    h = handle or default_handle(dev.index, stream)
    _need(h.device == dev.index, f"handle is bound to device {h.device}, tensors are on {dev}")
    return h


def workspace_size(op: int, p: int, M: int, N: int, K: int, n_chunks: int = 1, sched=SCHED_AUTO,
                   message: str = "fp32") -> int:
    return int(load().tpf_workspace_size(op, p, M, N, K, n_chunks, _sched(sched, message)))


def _ws(op, p, M, N, K, n_chunks, sched, ws, device, message="fp32", stream=None):
    need = workspace_size(op, p, M, N, K, n_chunks, sched, message)
    if need == 0:
        return ws, 0 if ws is None else ws.numel() * ws.element_size()
    if ws is None:
        with _on(stream):
            ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def matmul_allreduce(X: List[torch.Tensor], W: List[torch.Tensor], out_dtype=torch.bfloat16, n_chunks: int = 1,
                     sched="auto", Y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                     handle: Optional[Handle] = None, stream=None, message: str = "fp32") -> torch.Tensor:
    """Y = sum_k X[k] @ W[k] (row-parallel Linear, AllReduce layout)."""
    p = len(X)
    _need(p >= 1, "X: no shards given")
    M, K = X[0].shape
    N = W[0].shape[1]
    _check_shards("W", W, p)
    dev = _check("X", X, (M, K))
    _check("W", W, (K, N), device=dev)
    if Y is None:
        with _on(stream):
            Y = torch.empty((M, N), dtype=out_dtype, device=dev)
    _check("Y", [Y], (M, N), OUT_DTYPES, dev)
    _check_ws(ws, dev)
    h = _handle(handle, dev, stream)
    ws, ws_bytes = _ws(OP_MATMUL_ALLREDUCE, p, M, N, K, n_chunks, sched, ws, dev, message, stream)
    check(load().tpf_matmul_allreduce(h.ptr, p, M, N, K, ptr_array([x.data_ptr() for x in X]),
                                      ptr_array([w.data_ptr() for w in W]), Y.data_ptr(), _dtype_code(Y.dtype),
                                      n_chunks, _sched(sched, message), ws.data_ptr() if ws is not None else None, ws_bytes,
                                      _stream_ptr(stream)))
    return Y


def matmul_allreduce_noalloc(X: List[torch.Tensor], W: List[torch.Tensor], Y: torch.Tensor, n_chunks: int = 1,
                             sched="auto", handle: Optional[Handle] = None, stream=None,
                             message: str = "fp32") -> torch.Tensor:
    """Y = sum_k X[k] @ W[k] into the caller's Y with no allocation anywhere:
    the library keeps the partials in its static per-device workspace
    (NOALLOC_SCRATCH_BYTES); calls that overlap on one device race."""
    p = len(X)
    _need(p >= 1, "X: no shards given")
    M, K = X[0].shape
    N = W[0].shape[1]
    _check_shards("W", W, p)
    dev = _check("X", X, (M, K))
    _check("W", W, (K, N), device=dev)
    _check("Y", [Y], (M, N), OUT_DTYPES, dev)
    h = _handle(handle, dev, stream)
    check(load().tpf_matmul_allreduce_noalloc(h.ptr, p, M, N, K, ptr_array([x.data_ptr() for x in X]),
                                              ptr_array([w.data_ptr() for w in W]), Y.data_ptr(),
                                              _dtype_code(Y.dtype), n_chunks, _sched(sched, message),
                                              _stream_ptr(stream)))
    return Y


def matmul_reducescatter(X: List[torch.Tensor], W: List[torch.Tensor], out_dtype=torch.bfloat16, n_chunks: int = 1,
                         sched="auto", Y: Optional[List[torch.Tensor]] = None, ws: Optional[torch.Tensor] = None,
                         handle: Optional[Handle] = None, stream=None, message: str = "fp32") -> List[torch.Tensor]:
    """Slice r = rows [r*M/p, (r+1)*M/p) of sum_k X[k] @ W[k] (ReduceScatter layout)."""
    p = len(X)
    _need(p >= 1, "X: no shards given")
    M, K = X[0].shape
    N = W[0].shape[1]
    _check_shards("W", W, p)
    dev = _check("X", X, (M, K))
    _check("W", W, (K, N), device=dev)
    if Y is None:
        with _on(stream):
            Y = [torch.empty((M // p, N), dtype=out_dtype, device=dev) for _ in range(p)]
    _check_shards("Y", Y, p)
    _check("Y", Y, (M // p, N), OUT_DTYPES, dev)
    _need(len({y.dtype for y in Y}) == 1, "Y: the slices differ in dtype")
    _check_ws(ws, dev)
    h = _handle(handle, dev, stream)
    ws, ws_bytes = _ws(OP_MATMUL_REDUCESCATTER, p, M, N, K, n_chunks, sched, ws, dev, message, stream)
    check(load().tpf_matmul_reducescatter(h.ptr, p, M, N, K, ptr_array([x.data_ptr() for x in X]),
                                          ptr_array([w.data_ptr() for w in W]), ptr_array([y.data_ptr() for y in Y]),
                                          _dtype_code(Y[0].dtype), n_chunks, _sched(sched, message),
                                          ws.data_ptr() if ws is not None else None, ws_bytes, _stream_ptr(stream)))
    return Y


def allgather_matmul(X_slices: List[torch.Tensor], W: torch.Tensor, out_dtype=torch.bfloat16, n_chunks: int = 1,
                     sched="auto", X_gathered: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                     handle: Optional[Handle] = None, stream=None):
    """(X_gathered, Y): slices concatenated in rank order, then Y = X_gathered @ W."""
    p = len(X_slices)
    _need(p >= 1, "X_slices: no slices given")
    Ms, K = X_slices[0].shape
    M = Ms * p
    N = W.shape[1]
    dev = _check("W", [W], (K, N))
    _check("X_slices", X_slices, (Ms, K), device=dev)
    with _on(stream):
        if X_gathered is None:
            X_gathered = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
        if Y is None:
            Y = torch.empty((M, N), dtype=out_dtype, device=dev)
    _check("X_gathered", [X_gathered], (M, K), device=dev)
    _check("Y", [Y], (M, N), OUT_DTYPES, dev)
    h = _handle(handle, dev, stream)
    check(load().tpf_allgather_matmul(h.ptr, p, M, N, K, ptr_array([x.data_ptr() for x in X_slices]), W.data_ptr(),
                                      X_gathered.data_ptr(), Y.data_ptr(), _dtype_code(Y.dtype), n_chunks,
                                      _sched(sched), None, 0, _stream_ptr(stream)))
    return X_gathered, Y


def matmul_dx(dY: List[torch.Tensor], W: List[torch.Tensor], semantic: int = ALLREDUCE, out_dtype=torch.bfloat16,
              n_chunks: int = 1, sched="auto", dX=None, ws: Optional[torch.Tensor] = None,
              handle: Optional[Handle] = None, stream=None, message: str = "fp32"):
    """dX = sum_k dY[k] @ W[k]^T; one tensor (ALLREDUCE) or p row slices (REDUCESCATTER)."""
    p = len(dY)
    _need(p >= 1, "dY: no shards given")
    M, Ns = dY[0].shape
    Kin = W[0].shape[0]
    _check_shards("W", W, p)
    dev = _check("dY", dY, (M, Ns))
    _check("W", W, (Kin, Ns), device=dev)
    if dX is None:
        with _on(stream):
            if semantic == ALLREDUCE:
                dX = torch.empty((M, Kin), dtype=out_dtype, device=dev)
            else:
                dX = [torch.empty((M // p, Kin), dtype=out_dtype, device=dev) for _ in range(p)]
    outs = [dX] if semantic == ALLREDUCE else list(dX)
    if semantic == ALLREDUCE:
        _check("dX", outs, (M, Kin), OUT_DTYPES, dev)
    else:
        _check_shards("dX", outs, p)
        _check("dX", outs, (M // p, Kin), OUT_DTYPES, dev)
        _need(len({o.dtype for o in outs}) == 1, "dX: the slices differ in dtype")
    _check_ws(ws, dev)
    h = _handle(handle, dev, stream)
    ws, ws_bytes = _ws(OP_MATMUL_DX, p, M, Kin, Ns, n_chunks, sched, ws, dev, message, stream)
    check(load().tpf_matmul_dx(h.ptr, semantic, p, M, Kin, Ns, ptr_array([d.data_ptr() for d in dY]),
                               ptr_array([w.data_ptr() for w in W]), ptr_array([o.data_ptr() for o in outs]),
                               _dtype_code(outs[0].dtype), n_chunks, _sched(sched, message),
                               ws.data_ptr() if ws is not None else None, ws_bytes, _stream_ptr(stream)))
    return dX


def weight_grad(A: List[torch.Tensor], B: List[torch.Tensor], out_dtype=torch.float32, dW=None,
                handle: Optional[Handle] = None, stream=None) -> List[torch.Tensor]:
    """dW[k] = A[k]^T @ B[k] for every shard k (A[k] [M, R], B[k] [M, C]).

    Row-parallel: A = X_k per shard, B = [dY] * p.  Column-parallel:
    A = [X_gathered] * p, B = dY_k per shard."""
    p = len(A)
    _need(p >= 1, "A: no shards given")
    M, R = A[0].shape
    C = B[0].shape[1]
    _check_shards("B", B, p)
    dev = _check("A", A, (M, R))
    _check("B", B, (M, C), device=dev)
    if dW is None:
        with _on(stream):
            dW = [torch.empty((R, C), dtype=out_dtype, device=dev) for _ in range(p)]
    _check_shards("dW", dW, p)
    _check("dW", dW, (R, C), OUT_DTYPES, dev)
    _need(len({d.dtype for d in dW}) == 1, "dW: the shards differ in dtype")
    h = _handle(handle, dev, stream)
    check(load().tpf_weight_grad(h.ptr, p, M, R, C, ptr_array([a.data_ptr() for a in A]),
                                 ptr_array([b.data_ptr() for b in B]), ptr_array([d.data_ptr() for d in dW]),
                                 _dtype_code(dW[0].dtype), _stream_ptr(stream)))
    return dW


def rowpar_dx(dY: torch.Tensor, W: List[torch.Tensor], out_dtype=torch.bfloat16, dX=None,
              handle: Optional[Handle] = None, stream=None) -> List[torch.Tensor]:
    """dX[k] = dY @ W[k]^T for every shard k: the input gradient of a
    row-parallel Linear (dY [M, N] whole on every rank, W[k] [K_shard, N])."""
    p = len(W)
    _need(p >= 1, "W: no shards given")
    M, N = dY.shape
    Ks = W[0].shape[0]
    dev = _check("dY", [dY], (M, N))
    _check("W", W, (Ks, N), device=dev)
    if dX is None:
        with _on(stream):
            dX = [torch.empty((M, Ks), dtype=out_dtype, device=dev) for _ in range(p)]
    _check_shards("dX", dX, p)
    _check("dX", dX, (M, Ks), OUT_DTYPES, dev)
    _need(len({d.dtype for d in dX}) == 1, "dX: the shards differ in dtype")
    h = _handle(handle, dev, stream)
    check(load().tpf_rowpar_dx(h.ptr, p, M, Ks, N, dY.data_ptr(), ptr_array([w.data_ptr() for w in W]),
                               ptr_array([d.data_ptr() for d in dX]), _dtype_code(dX[0].dtype),
                               _stream_ptr(stream)))
    return dX


def mlp_sp(X_slices: List[torch.Tensor], W1: List[torch.Tensor], W2: List[torch.Tensor], out_dtype=torch.bfloat16,
           n_chunks: int = 1, sched="auto", X_gathered: Optional[torch.Tensor] = None,
           H: Optional[List[torch.Tensor]] = None, Y: Optional[List[torch.Tensor]] = None,
           ws: Optional[torch.Tensor] = None, handle: Optional[Handle] = None, stream=None,
           message: str = "fp32"):
    """MLP block under sequence parallelism: AllGather -> FC1 (column shards) + GeLU
    -> FC2 (row shards) -> ReduceScatter.  Returns (X_gathered, H, Y_slices)."""
    p = len(X_slices)
    _need(p >= 1, "X_slices: no slices given")
    Sp, Hd = X_slices[0].shape
    S = Sp * p
    F = W1[0].shape[1]
    _check_shards("W1", W1, p)
    _check_shards("W2", W2, p)
    dev = _check("X_slices", X_slices, (Sp, Hd))
    _check("W1", W1, (Hd, F), device=dev)
    _check("W2", W2, (F, Hd), device=dev)
    with _on(stream):
        if X_gathered is None:
            X_gathered = torch.empty((S, Hd), dtype=torch.bfloat16, device=dev)
        if H is None:
            H = [torch.empty((S, F), dtype=torch.bfloat16, device=dev) for _ in range(p)]
        if Y is None:
            Y = [torch.empty((Sp, Hd), dtype=out_dtype, device=dev) for _ in range(p)]
    _check("X_gathered", [X_gathered], (S, Hd), device=dev)
    _check_shards("H", H, p)
    _check("H", H, (S, F), device=dev)
    _check_shards("Y", Y, p)
    _check("Y", Y, (Sp, Hd), OUT_DTYPES, dev)
    _need(len({y.dtype for y in Y}) == 1, "Y: the slices differ in dtype")
    _check_ws(ws, dev)
    h = _handle(handle, dev, stream)
    ws, ws_bytes = _ws(OP_MLP_SP, p, S, Hd, F, n_chunks, sched, ws, dev, message, stream)
    check(load().tpf_mlp_sp(h.ptr, p, S, Hd, F, ptr_array([x.data_ptr() for x in X_slices]),
                            ptr_array([w.data_ptr() for w in W1]), ptr_array([w.data_ptr() for w in W2]),
                            X_gathered.data_ptr(), ptr_array([t.data_ptr() for t in H]),
                            ptr_array([y.data_ptr() for y in Y]), _dtype_code(Y[0].dtype), n_chunks,
                            _sched(sched, message), ws.data_ptr() if ws is not None else None, ws_bytes,
                            _stream_ptr(stream)))
    return X_gathered, H, Y


# ---------------------------------------------------------------------------
# The MLP block around its matrix products.
# ---------------------------------------------------------------------------

STASH_BLOCK = 32
CODE_DTYPES = (torch.float8_e4m3fn, torch.uint8)


def _ptrs(ts):
    return (_VP * len(ts))(*[t.data_ptr() for t in ts])


def _operands(idx: int, *groups):
    """Addresses of each group's tensors (tensors, dtype, shape, ...), or None
    where one is not a contiguous tensor on GPU `idx` of that dtype and shape.

    Decode-sized calls run for a few microseconds on the GPU, so the checks of
    good arguments are this one native pass; `_check` names what is wrong."""
    return (_args or _native()).operands(idx, *groups)


def _ctx(handle: Optional[Handle], dev, stream):
    """(handle, raw stream) of a call; the current stream is asked for once."""
    idx = dev.index
    sp = torch._C._cuda_getCurrentRawStream(idx) if stream is None else int(stream.cuda_stream)
    h = handle or _default_handles.get((idx, sp)) or default_handle(idx, stream)
    _need(h.device == idx, f"handle is bound to device {h.device}, tensors are on {dev}")
    return h._h, sp


def _empty(dev, *groups):
    """New tensors (dtype, shape, ...) on GPU `dev`; None for a shape of None."""
    return (_args or _native()).empty(dev.index, *groups)


def _shards(dev, p: int, *groups):
    """p new tensors and their addresses for each (dtype, shape): (tensors, addresses, ...)."""
    return (_args or _native()).shards(dev.index, p, *groups)


def _matrix(name: str, t, sizes: str):
    """The two sizes of a matrix, the first thing that is asked of an operand."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:      # the message is built only on failure
        _need(isinstance(t, torch.Tensor), f"{name} is not a tensor")
        _need(False, f"{name} has {t.dim()} dimensions, expected {sizes}")
    return t.shape


def _norm_operands(x, blocks, w_pre, w_post, gate):
    """Checks shared by the norm's two directions; returns (device, M, H, gate kind, the
    blocks' addresses)."""
    p = len(blocks)
    _need(p >= 1, "blocks: no tensors given")
    M, H = _matrix("x", x, "[M, H]")
    dev, idx = x.device, x.get_device()
    vec, rows = (H,), (M, H)
    try:
        kind = GATE_NONE if gate is None else GATE_TOKEN if gate.dim() == 2 else GATE_CHANNEL
        b, w = blocks[0].dtype, w_pre.dtype
    except AttributeError:       # no tensors: named below
        kind, b, w = GATE_CHANNEL, None, None
    if x.dtype in OUT_DTYPES and b in OUT_DTYPES and w in OUT_DTYPES:
        got = _operands(idx, blocks, b, rows, (x,), x.dtype, rows, (w_pre, w_post), w, vec,
                        () if gate is None else (gate,), w, (M, 1) if kind == GATE_TOKEN else vec)
        if got is not None:
            return dev, M, H, kind, got[0]
    _check("x", [x], (M, H), OUT_DTYPES)
    _check("blocks", blocks, (M, H), OUT_DTYPES, dev)
    _need(all(b.dtype == blocks[0].dtype for b in blocks), "blocks: the tensors differ in dtype")
    _check("w_pre", [w_pre], (H,), OUT_DTYPES, dev)
    _check("w_post", [w_post], (H,), (w_pre.dtype,), dev)
    if gate is not None:
        _check("gate", [gate], (M, 1) if kind == GATE_TOKEN else (H,), (w_pre.dtype,), dev)
    return dev, M, H, kind, _ptrs(blocks)


def block_norm(x: torch.Tensor, blocks: Sequence[torch.Tensor], w_pre: torch.Tensor, w_post: torch.Tensor,
               gate: Optional[torch.Tensor] = None, alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6,
               unit_offset: bool = False, want_stats: bool = False, x_out: Optional[torch.Tensor] = None,
               y: Optional[torch.Tensor] = None, handle: Optional[Handle] = None, stream=None):
    """(x_out, y, stats): the norm after a block with its gate, residual scale
    and residual add, and the norm before the next block, in one pass.

        b     = blocks[0] + ... + blocks[p-1]
        x_out = alpha x + beta gate rms_norm(b) w_post        (x's dtype; may be x itself)
        y     = rms_norm(x_out) w_pre                         (bf16)

    `gate` is None, [H] (one factor a channel) or [M, 1] (one a token); weights
    are stored as offsets from 1 with `unit_offset`.  `stats` ([2, M] fp32, for
    `block_norm_backward`) is None unless `want_stats`."""
    dev, M, H, kind, at = _norm_operands(x, blocks, w_pre, w_post, gate)
    if x_out is not None:
        _check("x_out", [x_out], (M, H), (x.dtype,), dev)
    if y is not None:
        _check("y", [y], (M, H), (torch.bfloat16,), dev)
    with _on(stream):
        new_x, new_y, stats = _empty(dev, x.dtype, (M, H) if x_out is None else None, torch.bfloat16,
                                     (M, H) if y is None else None, torch.float32, (2, M) if want_stats else None)
        x_out, y = new_x if x_out is None else x_out, new_y if y is None else y
    h, sp = _ctx(handle, dev, stream)
    check(load().tpf_block_norm(h, len(blocks), M, H, x.data_ptr(), _dtype_code(x.dtype), at,
                                _dtype_code(blocks[0].dtype), w_pre.data_ptr(), w_post.data_ptr(),
                                gate.data_ptr() if gate is not None else None, kind, _dtype_code(w_pre.dtype), alpha,
                                beta, eps, 1 if unit_offset else 0, x_out.data_ptr(), y.data_ptr(),
                                stats.data_ptr() if stats is not None else None, sp))
    return x_out, y, stats


def block_norm_backward(dy: torch.Tensor, dx_out: Optional[torch.Tensor], x: torch.Tensor,
                        blocks: Sequence[torch.Tensor], stats: torch.Tensor, w_pre: torch.Tensor,
                        w_post: torch.Tensor, gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
                        beta: float = 1.0, unit_offset: bool = False, ws: Optional[torch.Tensor] = None,
                        handle: Optional[Handle] = None, stream=None):
    """(dx, db, dw_pre, dw_post, dgate) of `block_norm`.

    `dy` is the gradient of y, `dx_out` that of x_out from what else reads it
    (None: nothing), `x` the forward's x_out, `stats` its statistics.  `db` is
    the gradient of every tensor of `blocks`; `dgate` has the gate's shape."""
    dev, M, H, kind, at = _norm_operands(x, blocks, w_pre, w_post, gate)
    if _operands(dev.index, (dy,), torch.bfloat16, (M, H), () if dx_out is None else (dx_out,), x.dtype, (M, H),
                 (stats,), torch.float32, (2, M)) is None:
        _check("dy", [dy], (M, H), (torch.bfloat16,), dev)
        if dx_out is not None:
            _check("dx_out", [dx_out], (M, H), (x.dtype,), dev)
        _check("stats", [stats], (2, M), (torch.float32,), dev)
    _check_ws(ws, dev)
    need = load().tpf_block_norm_backward_ws(M, H)
    with _on(stream):
        dx, db, dw_pre, dw_post, dgate, new_ws = _empty(
            dev, x.dtype, (M, H), torch.bfloat16, (M, H), torch.float32, (H,), torch.float32, (H,), torch.float32,
            None if gate is None else tuple(gate.shape), torch.uint8, (max(need, 16),) if ws is None else None)
        ws = new_ws if ws is None else ws
    h, sp = _ctx(handle, dev, stream)
    check(load().tpf_block_norm_backward(
        h, len(blocks), M, H, dy.data_ptr(), dx_out.data_ptr() if dx_out is not None else None, x.data_ptr(),
        _dtype_code(x.dtype), at, _dtype_code(blocks[0].dtype), stats.data_ptr(), w_pre.data_ptr(),
        w_post.data_ptr(), gate.data_ptr() if gate is not None else None, kind, _dtype_code(w_pre.dtype), alpha, beta,
        1 if unit_offset else 0, dx.data_ptr(), db.data_ptr(), dw_pre.data_ptr(), dw_post.data_ptr(),
        dgate.data_ptr() if dgate is not None else None, ws.data_ptr(), ws.numel() * ws.element_size(),
        sp))
    return dx, db, dw_pre, dw_post, dgate


def _stash_shape(M: int, F: int):
    return -(-M // STASH_BLOCK), -(-F // STASH_BLOCK)


def stash_pack(u: Sequence[torch.Tensor], gelu: bool = True, handle: Optional[Handle] = None, stream=None):
    """(h, codes, scales): the activations u[k] ([M, F] bf16) in 8 bits, and
    h[k] = GeLU(u[k]) (bf16) from the same pass (None without `gelu`).

    Every 32 x 32 block shares one power of two, 2^(scales - 127); codes are
    e4m3, so that u ~ codes * 2^(scales - 127)."""
    p = len(u)
    _need(p >= 1, "u: no shards given")
    M, F = _matrix("u[0]", u[0], "[M, F]")
    dev = u[0].device
    at = _operands(u[0].get_device(), u, torch.bfloat16, (M, F))
    if at is None:
        _check("u", u, (M, F))
        at = (_ptrs(u),)
    with _on(stream):
        codes, cat, scales, sat = _shards(dev, p, torch.float8_e4m3fn, (M, F), torch.uint8, _stash_shape(M, F))
        h, hat = _shards(dev, p, torch.bfloat16, (M, F)) if gelu else (None, None)
    hd, sp = _ctx(handle, dev, stream)
    check(load().tpf_stash_pack(hd, p, M, F, at[0], 1 if gelu else 0, hat, cat, sat, sp))
    return h, codes, scales


def _check_stash(codes, scales):
    p = len(codes)
    _need(p >= 1, "codes: no shards given")
    M, F = _matrix("codes[0]", codes[0], "[M, F]")
    _check_shards("scales", scales, p)
    dev = codes[0].device
    at = None
    if codes[0].dtype in CODE_DTYPES:
        at = _operands(codes[0].get_device(), codes, codes[0].dtype, (M, F), scales, torch.uint8, _stash_shape(M, F))
    if at is None:
        _check("codes", codes, (M, F), CODE_DTYPES)
        _check("scales", scales, _stash_shape(M, F), (torch.uint8,), dev)
        at = _ptrs(codes), _ptrs(scales)
    return dev, p, M, F, at


def stash_backward(codes: Sequence[torch.Tensor], scales: Sequence[torch.Tensor], dh: Sequence[torch.Tensor],
                   handle: Optional[Handle] = None, stream=None):
    """(du, h): GeLU's gradient du[k] = dh[k] GeLU'(u) and its value h[k] =
    GeLU(u), u the 8-bit activations of `stash_pack`."""
    dev, p, M, F, at = _check_stash(codes, scales)
    _check_shards("dh", dh, p)
    dat = _operands(dev.index, dh, torch.bfloat16, (M, F))
    if dat is None:
        _check("dh", dh, (M, F), device=dev)
        dat = (_ptrs(dh),)
    with _on(stream):
        du, uat, h, hat = _shards(dev, p, torch.bfloat16, (M, F), torch.bfloat16, (M, F))
    hd, sp = _ctx(handle, dev, stream)
    check(load().tpf_stash_backward(hd, p, M, F, *at, dat[0], uat, hat, sp))
    return du, h


def stash_weight_grad(codes: Sequence[torch.Tensor], scales: Sequence[torch.Tensor], dY: Sequence[torch.Tensor],
                      out_dtype=torch.float32, dW=None, ws: Optional[torch.Tensor] = None,
                      handle: Optional[Handle] = None, stream=None) -> List[torch.Tensor]:
    """dW[k] = U_k^T dY[k], U_k [M, R] the 8-bit activations of `stash_pack`:
    `weight_grad` of an input kept in 8 bits."""
    _need(len(dY) >= 1, "dY: no shards given")
    _, C = _matrix("dY[0]", dY[0], "[M, C]")
    dev, p, M, R, at = _check_stash(codes, scales)
    _check_shards("dY", dY, p)
    yat = _operands(dev.index, dY, torch.bfloat16, (M, C))
    if yat is None:
        _check("dY", dY, (M, C), device=dev)
        yat = (_ptrs(dY),)
    if dW is None:
        _need(out_dtype in OUT_DTYPES, f"output dtype must be bfloat16 or float32, got {out_dtype}")
        with _on(stream):
            dW, wat = _shards(dev, p, out_dtype, (R, C))
            dW = list(dW)
    else:
        _check_shards("dW", dW, p)
        _check("dW", dW, (R, C), OUT_DTYPES, dev)
        _need(all(d.dtype == dW[0].dtype for d in dW), "dW: the shards differ in dtype")
        wat = _ptrs(dW)
    _check_ws(ws, dev)
    need = load().tpf_stash_weight_grad_ws(p, M, R, C)
    if ws is None and need:
        with _on(stream):
            ws, = _empty(dev, torch.uint8, (need,))
    hd, sp = _ctx(handle, dev, stream)
    check(load().tpf_stash_weight_grad(hd, p, M, R, C, *at, yat[0], wat,
                                       _dtype_code(dW[0].dtype), ws.data_ptr() if ws is not None else None,
                                       ws.numel() * ws.element_size() if ws is not None else 0, sp))
    return dW


def qweight_matmul(X: Sequence[torch.Tensor], codes: Sequence[torch.Tensor], scales: Sequence[torch.Tensor],
                   zeros: Optional[Sequence[torch.Tensor]] = None, group: int = 128, gelu: bool = False,
                   out_dtype=torch.bfloat16, Y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                   handle: Optional[Handle] = None, stream=None) -> torch.Tensor:
    """Y = sum_k X[k] W_k^T with 4-bit weights (row-parallel over the shards;
    p = 1: any Linear), GeLU of it with `gelu`.

    X[k] [M, K] bf16; codes[k] [N, K/2] uint8, byte j of every four holding
    code j (low half) and code j + 4 (high half) of a run of eight; scales[k]
    [N, K/group] bf16; zeros[k] [N, K/group] uint8 (None: 8).
    W_k = (code - zero) * scale; group is 32, 64 or 128."""
    p = len(X)
    _need(p >= 1, "X: no shards given")
    M, K = _matrix("X[0]", X[0], "[M, K]")
    _need(group in (32, 64, 128) and K % group == 0, f"group {group} is not 32, 64 or 128 or does not divide K = {K}")
    _check_shards("codes", codes, p)
    _check_shards("scales", scales, p)
    if zeros is not None:
        _check_shards("zeros", zeros, p)
    N, _ = _matrix("codes[0]", codes[0], "[N, K/2]")
    per_group = N, K // group
    dev = X[0].device
    at = _operands(X[0].get_device(), X, torch.bfloat16, (M, K), codes, torch.uint8, (N, K // 2), scales, torch.bfloat16,
                   per_group, () if zeros is None else zeros, torch.uint8, per_group)
    if at is None:
        _check("X", X, (M, K))
        _check("codes", codes, (N, K // 2), (torch.uint8,), dev)
        _check("scales", scales, per_group, (torch.bfloat16,), dev)
        if zeros is not None:
            _check("zeros", zeros, per_group, (torch.uint8,), dev)
        at = _ptrs(X), _ptrs(codes), _ptrs(scales), None if zeros is None else _ptrs(zeros)
    if Y is None:
        _need(out_dtype in OUT_DTYPES, f"output dtype must be bfloat16 or float32, got {out_dtype}")
        with _on(stream):
            Y, = _empty(dev, out_dtype, (M, N))
    else:
        _check("Y", [Y], (M, N), OUT_DTYPES, dev)
    _check_ws(ws, dev)
    need = load().tpf_qweight_matmul_ws(p, M, K, N, group)
    if ws is None and need:
        with _on(stream):
            ws, = _empty(dev, torch.uint8, (need,))
    hd, sp = _ctx(handle, dev, stream)
    check(load().tpf_qweight_matmul(hd, p, M, K, N, group, at[0], at[1], at[2],
                                    None if zeros is None else at[3], 1 if gelu else 0, Y.data_ptr(),
                                    _dtype_code(Y.dtype), ws.data_ptr() if ws is not None else None,
                                    ws.numel() * ws.element_size() if ws is not None else 0, sp))
    return Y
