"""Python binding of libmr, the MI355X W-way sum-reduce and param-contiguous gather library, with the operators of
a training step around them (layer norm, gradient norm, AdamW).

A thin ctypes layer over the C ABI declared in include/mr.h: it turns torch tensors into device
pointers, sizes and the current HIP stream, calls the entry point of the same name and raises on a
non-zero status.  Every step of the computation runs in the HIP kernels of libmr.so; there is no
fallback.  If libmr.so has not been built, loading it raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Any, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmr.so")

MR_OK = 0
STATUS = {
    0: "MR_OK",
    -1: "MR_ERR_INVALID_ARG",
    -2: "MR_ERR_DTYPE",
    -3: "MR_ERR_ALIAS",
    -4: "MR_ERR_WORKSPACE",
    -5: "MR_ERR_HIP",
    -6: "MR_ERR_ENGINE",
}
DTYPE_CODE = {"bf16": 0, "fp16": 1, "fp32": 2, "int32": 3}
STATE_FORMAT = {32: 0, 8: 1}
MODE_CODE = {"oneshot": 0, "twoshot": 1}
OPTION_CODE = {"twoshot_sync": 0, "spin_limit": 1, "tile_shape": 2, "sdma_cu_below": 3}
TWOSHOT_SYNC = {"tile": 0, "chunk": 1, "grid": 2, "last": 3, "auto": 4}
TILE_SHAPE = {"auto": 0, "wide": 1, "medium": 2, "narrow": 3, "wide_pair": 4}
MAX_W = 16
MAX_PARAMS_PER_LAUNCH = 128
MAX_TABLE_W = 64

ADAMW_BLOCK = 32


class _AdamWStateC(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("m", "v", "m_scale", "v_scale", "master")]


class _AdamWHyperC(ctypes.Structure):
    _fields_ = [(k, ctypes.c_double) for k in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_uint64), ("seed", ctypes.c_uint64)]


# Exported symbols of include/mr.h, with ctypes signatures.
_SIGS = {
    "mr_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "mr_last_hip_error": (ctypes.c_int, []),
    "mr_version": (ctypes.c_int, []),
    "mr_allreduce_sum": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_size_t,
                                        ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "mr_allreduce_sum_noalloc": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_size_t,
                                                ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "mr_allgather_param_contig": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                                 ctypes.POINTER(ctypes.c_uint64), ctypes.c_int, ctypes.c_int,
                                                 ctypes.c_void_p, ctypes.c_void_p]),
    "mr_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_size_t, ctypes.c_int]),
    "mr_set_workspace": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t]),
    "mr_workspace_check": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]),
    "mr_reduce_scatter_chunk": (ctypes.c_int, [ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                               ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]),
    "mr_reduce_scatter_sum": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_size_t,
                                             ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "mr_allgather_into_tensor": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_size_t,
                                                ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "mr_allgather_list": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_size_t,
                                         ctypes.c_int, ctypes.POINTER(ctypes.c_void_p), ctypes.c_void_p]),
    "mr_allgather_param_contig_shards": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_int,
                                                        ctypes.POINTER(ctypes.c_uint64), ctypes.c_int, ctypes.c_int,
                                                        ctypes.c_void_p, ctypes.c_void_p]),
    "mr_allgather_param_contig_sdma": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                                      ctypes.POINTER(ctypes.c_uint64), ctypes.c_int, ctypes.c_int,
                                                      ctypes.c_void_p, ctypes.c_void_p]),
    "mr_sdma_engines": (ctypes.c_int, []),
    "mr_layer_norm_forward": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int] + [ctypes.c_void_p] * 3 +
                              [ctypes.c_size_t] * 2 + [ctypes.c_int] * 2 + [ctypes.c_double] + [ctypes.c_void_p] * 5),
    "mr_layer_norm_backward": (ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_size_t] * 2 + [ctypes.c_int] * 2 +
                               [ctypes.c_void_p] * 4),
    "mr_grad_norm": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_uint64), ctypes.c_int,
                                    ctypes.c_int, ctypes.c_double, ctypes.c_double, ctypes.c_void_p, ctypes.c_void_p]),
    "mr_adamw_state_elems": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint64), ctypes.c_int,
                                            ctypes.POINTER(ctypes.c_uint64)]),
    "mr_adamw_step": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_void_p),
                                     ctypes.POINTER(ctypes.c_uint64)] + [ctypes.c_int] * 4 +
                      [ctypes.POINTER(_AdamWStateC), ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(_AdamWStateC),
                       ctypes.POINTER(_AdamWHyperC), ctypes.c_void_p, ctypes.c_void_p]),
    "mr_set_option": (ctypes.c_int, [ctypes.c_int, ctypes.c_int64]),
    "mr_get_option": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]),
}
EXPORTS = tuple(_SIGS)

_lib = None


class MRError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


def lib() -> ctypes.CDLL:
    """Load libmr.so (once).  Raises if it is missing: the product path has no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int, what: str) -> None:
    if status != MR_OK:
        raise MRError(status, what)


_torch_mod = None
_dtype_names: dict = {}


def _torch():
    global _torch_mod
    if _torch_mod is None:
        import torch

        _dtype_names.update({torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32", torch.int32: "int32"})
        _torch_mod = torch
    return _torch_mod


def dtype_name(t) -> str:
    _torch()
    return _dtype_names[t.dtype]


def _stream_handle(stream) -> int | None:
    if stream is not None:
        return stream.cuda_stream or None
    # the handle alone: building a torch.cuda.Stream for it takes 2.8 us of a call, this 0.3
    torch = _torch()
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) or None


def _dev_tensor(t, what: str):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous device tensor")


def _splits_array(splits: Sequence[int]):
    sp = [int(x) for x in splits]
    if not sp or min(sp) < 0:
        raise ValueError("splits must be a non-empty list of non-negative element counts")
    return (ctypes.c_uint64 * len(sp))(*sp), sum(sp)


def _same(tensors, ref, what: str, numel: int) -> None:
    """Every tensor is a contiguous device tensor of ref's dtype holding exactly ``numel`` elements."""
    for t in tensors:
        _dev_tensor(t, what)
        if t.dtype != ref.dtype or t.numel() != numel:
            raise ValueError(f"{what} must hold {numel} elements of {ref.dtype}")


def _prepared(name: str, f, args, keep):
    def call() -> None:
        st = f(*args)
        if st != MR_OK:
            raise MRError(st, name)

    call.keepalive = keep
    return call


# Each prepare_* checks that every tensor is a contiguous device tensor of the sizes the call implies
# (the library takes raw pointers and cannot check extents) and marshals the arguments once; the
# returned no-argument callable enqueues that same call (tight timing loops, graph capture).  The
# stream is marshalled too: without a ``stream`` it is the one that is current at preparation, not at
# the call.  The plain functions are one prepared call.

def prepare_allreduce(bufs: Sequence, out, mode: str = "oneshot", stream=None):
    """Pre-marshalled mr_allreduce_sum: out = elementwise fp32 sum (rank order) of the tensors ``bufs``."""
    _dev_tensor(out, "out")
    _same(bufs, out, "rank buffer", out.numel())
    ptrs = (ctypes.c_void_p * max(len(bufs), 1))(*[b.data_ptr() for b in bufs])
    args = (ptrs, len(bufs), out.numel(), DTYPE_CODE[dtype_name(out)], out.data_ptr(), MODE_CODE[mode],
            _stream_handle(stream))
    return _prepared("mr_allreduce_sum", lib().mr_allreduce_sum, args, (ptrs, list(bufs), out))


def allreduce_sum(bufs: Sequence, out, mode: str = "oneshot", stream=None):
    """out = elementwise fp32 sum (rank order 0..W-1) of the W same-shape, same-dtype tensors ``bufs``."""
    prepare_allreduce(bufs, out, mode, stream)()
    return out


NOALLOC_MAX_BYTES = 32 << 20


def prepare_allreduce_noalloc(bufs: Sequence, out, mode: str = "oneshot", stream=None):
    """Pre-marshalled mr_allreduce_sum_noalloc (two-shot workspace inside the library; never allocates)."""
    _dev_tensor(out, "out")
    _same(bufs, out, "rank buffer", out.numel())
    ptrs = (ctypes.c_void_p * max(len(bufs), 1))(*[b.data_ptr() for b in bufs])
    args = (ptrs, len(bufs), out.numel(), DTYPE_CODE[dtype_name(out)], out.data_ptr(), MODE_CODE[mode],
            _stream_handle(stream))
    return _prepared("mr_allreduce_sum_noalloc", lib().mr_allreduce_sum_noalloc, args, (ptrs, list(bufs), out))


def allreduce_sum_noalloc(bufs: Sequence, out, mode: str = "oneshot", stream=None):
    """allreduce_sum without any device allocation (rank buffers up to NOALLOC_MAX_BYTES)."""
    prepare_allreduce_noalloc(bufs, out, mode, stream)()
    return out


def reduce_scatter_chunk(n: int, W: int, dtype: str, rank: int) -> tuple[int, int]:
    """(offset, count) of rank ``rank``'s chunk of an n-element reduce-scatter."""
    off, cnt = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().mr_reduce_scatter_chunk(n, W, DTYPE_CODE[dtype], rank, ctypes.byref(off), ctypes.byref(cnt)),
           "mr_reduce_scatter_chunk")
    return int(off.value), int(cnt.value)


def prepare_reduce_scatter(bufs: Sequence, rank: int, out, stream=None):
    """Pre-marshalled mr_reduce_scatter_sum: out = rank ``rank``'s chunk of the sum of ``bufs``."""
    _dev_tensor(out, "out")
    n = bufs[0].numel() if len(bufs) else 0
    _same(bufs, out, "rank buffer", n)
    _, cnt = reduce_scatter_chunk(n, len(bufs), dtype_name(out), rank)
    if out.numel() != cnt:
        raise ValueError(f"out must hold the chunk's {cnt} elements")
    ptrs = (ctypes.c_void_p * max(len(bufs), 1))(*[b.data_ptr() for b in bufs])
    args = (ptrs, len(bufs), n, DTYPE_CODE[dtype_name(out)], rank, out.data_ptr(), _stream_handle(stream))
    return _prepared("mr_reduce_scatter_sum", lib().mr_reduce_scatter_sum, args, (ptrs, list(bufs), out))


def reduce_scatter_sum(bufs: Sequence, rank: int, out, stream=None):
    """out = rank ``rank``'s chunk of the elementwise sum of the W same-shape tensors ``bufs``."""
    prepare_reduce_scatter(bufs, rank, out, stream)()
    return out


def prepare_allgather_param_contig(src, W: int, G: int, splits: Sequence[int], out, stream=None):
    """Pre-marshalled mr_allgather_param_contig (src rank-major [W][T], T = sum(splits))."""
    _dev_tensor(src, "src")
    sp, T = _splits_array(splits)
    if W < 1 or src.numel() != W * T:
        raise ValueError(f"src must hold W*sum(splits) = {max(W, 0) * T} elements")
    _same([out], src, "out", src.numel())
    args = (src.data_ptr(), W, G, sp, len(sp), DTYPE_CODE[dtype_name(src)], out.data_ptr(), _stream_handle(stream))
    return _prepared("mr_allgather_param_contig", lib().mr_allgather_param_contig, args, (sp, src, out))


def allgather_param_contig(src, W: int, G: int, splits: Sequence[int], out, stream=None):
    """Scatter the rank-major ``src`` ([W][T], T = sum(splits)) into [param][rank] order in ``out``."""
    prepare_allgather_param_contig(src, W, G, splits, out, stream)()
    return out


def prepare_allgather_param_contig_sdma(src, W: int, G: int, splits: Sequence[int], out, stream=None):
    """Pre-marshalled mr_allgather_param_contig_sdma: the same placement on the SDMA copy engines (a
    synchronous call: it waits for ``stream``, copies, and returns when the copies are complete)."""
    _dev_tensor(src, "src")
    sp, T = _splits_array(splits)
    if W < 1 or src.numel() != W * T:
        raise ValueError(f"src must hold W*sum(splits) = {max(W, 0) * T} elements")
    _same([out], src, "out", src.numel())
    args = (src.data_ptr(), W, G, sp, len(sp), DTYPE_CODE[dtype_name(src)], out.data_ptr(), _stream_handle(stream))
    return _prepared("mr_allgather_param_contig_sdma", lib().mr_allgather_param_contig_sdma, args, (sp, src, out))


def allgather_param_contig_sdma(src, W: int, G: int, splits: Sequence[int], out, stream=None):
    """mr_allgather_param_contig's placement copied by the SDMA engines (synchronous)."""
    prepare_allgather_param_contig_sdma(src, W, G, splits, out, stream)()
    return out


def sdma_engines() -> int:
    """SDMA engines the current device offers for copies within its own memory."""
    return int(lib().mr_sdma_engines())


def _shard_ptrs(shards):
    if not len(shards):
        raise ValueError("at least one shard")
    _same(shards, shards[0], "shard", shards[0].numel())
    return (ctypes.c_void_p * len(shards))(*[t.data_ptr() for t in shards])


def prepare_allgather_shards(shards: Sequence, out, G: int | None = None, splits: Sequence[int] | None = None,
                             stream=None):
    """Pre-marshalled gather from W shards: rank-major into ``out`` (``splits`` None, mr_allgather_into_tensor)
    or param-contiguous (mr_allgather_param_contig_shards, each shard sum(splits) elements)."""
    ptrs = _shard_ptrs(shards)
    W, T = len(shards), shards[0].numel()
    _same([out], shards[0], "out", W * T)
    dt = DTYPE_CODE[dtype_name(out)]
    if splits is None:
        name, args = "mr_allgather_into_tensor", (ptrs, W, T, dt, out.data_ptr(), _stream_handle(stream))
    else:
        sp, ST = _splits_array(splits)
        if ST != T:
            raise ValueError(f"each shard must hold sum(splits) = {ST} elements")
        name = "mr_allgather_param_contig_shards"
        args = (ptrs, W, W if G is None else G, sp, len(sp), dt, out.data_ptr(), _stream_handle(stream))
    return _prepared(name, getattr(lib(), name), args, (args, list(shards), out))


def allgather_into_tensor(shards: Sequence, out, stream=None):
    """out[r*T:(r+1)*T] = shards[r] (rank-major all-gather of W shards of T elements)."""
    prepare_allgather_shards(shards, out, stream=stream)()
    return out


def allgather_param_contig_shards(shards: Sequence, G: int, splits: Sequence[int], out, stream=None):
    """[param][rank] all-gather written straight from W shards (each sum(splits) elements)."""
    prepare_allgather_shards(shards, out, G, splits, stream)()
    return out


def allgather_list(shards: Sequence, outs: Sequence, stream=None):
    """outs[r] = shards[r] for every rank (list-output all-gather), one launch."""
    ptrs = _shard_ptrs(shards)
    if len(outs) != len(shards):
        raise ValueError("one output per shard")
    _same(outs, shards[0], "output", shards[0].numel())
    optrs = (ctypes.c_void_p * len(outs))(*[o.data_ptr() for o in outs])
    _check(lib().mr_allgather_list(ptrs, len(shards), shards[0].numel(), DTYPE_CODE[dtype_name(shards[0])], optrs,
                                   _stream_handle(stream)), "mr_allgather_list")
    return outs


# ------------------------------------------------------------- the training step around the exchange

def _opt(t, what: str, ref_dtype, numel: int):
    """Pointer of an optional tensor of ``numel`` elements of one of the dtypes ``ref_dtype``; None stays None."""
    if t is None:
        return None
    if not (t.is_cuda and t.is_contiguous() and t.numel() == numel and t.dtype in ref_dtype):
        raise ValueError(f"{what} must be a contiguous device tensor of {numel} elements of {' or '.join(map(str, ref_dtype))}")
    return t.data_ptr()


def _weights_dtype(ref, *weights):
    """The dtype of the weights that are given (ref's or fp32, all alike; ref's if none is)."""
    wdt = None
    for w in weights:
        if w is not None:
            if wdt is None:
                wdt = w.dtype
            elif w.dtype != wdt:
                raise ValueError("weights and their gradients must be of one dtype")
    if wdt is not None and wdt != ref.dtype and wdt != _torch().float32:
        raise ValueError(f"weights must be {ref.dtype} or torch.float32")
    return ref.dtype if wdt is None else wdt


_ptr_arrays: dict = {}


def _ptr_array(ptrs):
    n = len(ptrs) or 1
    t = _ptr_arrays.get(n)
    if t is None:
        t = _ptr_arrays[n] = ctypes.c_void_p * n
    return t(*ptrs)


def _layer_norm_forward_args(bufs, gamma, beta, y, eps, residual, x_out, mean, rstd, stream):
    _dev_tensor(y, "y")
    n, cols = y.numel(), y.shape[-1] if y.dim() else 1
    rows, f32 = n // cols if cols else 0, (_torch().float32,)
    same, wdt = (y.dtype,), _weights_dtype(y, gamma, beta)
    dt = DTYPE_CODE[dtype_name(y)]
    return (_ptr_array([_opt(b, "rank buffer", same, n) for b in bufs]), len(bufs), _opt(residual, "residual", same, n),
            _opt(gamma, "gamma", (wdt,), cols), _opt(beta, "beta", (wdt,), cols), rows, cols, dt,
            dt if wdt == y.dtype else DTYPE_CODE["fp32"], eps, _opt(x_out, "x_out", same, n), y.data_ptr(),
            _opt(mean, "mean", f32, rows), _opt(rstd, "rstd", f32, rows), _stream_handle(stream))


def prepare_layer_norm_forward(bufs: Sequence, gamma, beta, y, eps: float = 1e-5, residual=None, x_out=None, mean=None,
                               rstd=None, stream=None):
    """Pre-marshalled mr_layer_norm_forward over the last dimension of ``y``, on ``stream`` or the one current now."""
    args = _layer_norm_forward_args(bufs, gamma, beta, y, eps, residual, x_out, mean, rstd, stream)
    return _prepared("mr_layer_norm_forward", lib().mr_layer_norm_forward, args,
                     (list(bufs), gamma, beta, y, residual, x_out, mean, rstd))


def layer_norm_forward(bufs: Sequence, gamma, beta, y, eps: float = 1e-5, residual=None, x_out=None, mean=None, rstd=None,
                       stream=None):
    """y = layer norm, over the last dimension, of x = the fp32 sum of the tensors ``bufs`` (rank order) and ``residual``.

    ``bufs`` with one tensor and no residual is a plain layer norm; with W tensors it is what follows a
    tensor-parallel all-reduce.  ``gamma`` / ``beta`` may be None (ones / zeros).  ``x_out`` receives x (the residual
    stream, and the backward pass's input); ``mean`` and ``rstd`` (fp32, one per row) the statistics."""
    _check(lib().mr_layer_norm_forward(*_layer_norm_forward_args(bufs, gamma, beta, y, eps, residual, x_out, mean, rstd, stream)),
           "mr_layer_norm_forward")
    return y


def _layer_norm_backward_args(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, dres, stream):
    _dev_tensor(dy, "dy")
    n, cols = dy.numel(), dy.shape[-1] if dy.dim() else 1
    rows, f32 = n // cols if cols else 0, (_torch().float32,)
    same, wdt = (dy.dtype,), _weights_dtype(dy, gamma, dgamma, dbeta)
    if x is None or mean is None or rstd is None:
        raise ValueError("x, mean and rstd are needed")
    dt = DTYPE_CODE[dtype_name(dy)]
    return (dy.data_ptr(), _opt(x, "x", same, n), _opt(gamma, "gamma", (wdt,), cols), _opt(mean, "mean", f32, rows),
            _opt(rstd, "rstd", f32, rows), _opt(dres, "dres", same, n), rows, cols, dt,
            dt if wdt == dy.dtype else DTYPE_CODE["fp32"], _opt(dx, "dx", same, n), _opt(dgamma, "dgamma", (wdt,), cols),
            _opt(dbeta, "dbeta", (wdt,), cols), _stream_handle(stream))


def prepare_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma=None, dbeta=None, dres=None, stream=None):
    """Pre-marshalled mr_layer_norm_backward, on ``stream`` or the one current now."""
    args = _layer_norm_backward_args(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, dres, stream)
    return _prepared("mr_layer_norm_backward", lib().mr_layer_norm_backward, args,
                     (dy, x, gamma, mean, rstd, dx, dgamma, dbeta, dres))


def layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma=None, dbeta=None, dres=None, stream=None):
    """Gradients of layer_norm_forward: ``dx`` (of every rank buffer and the residual alike; plus ``dres``, the gradient
    that reaches x beside the norm), ``dgamma`` and ``dbeta`` (sums over the rows).  Any of the three may be None."""
    _check(lib().mr_layer_norm_backward(*_layer_norm_backward_args(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, dres, stream)),
           "mr_layer_norm_backward")
    return dx


def _tensor_list(tensors, what: str, counts=None):
    """Pointers of contiguous device tensors of one dtype (and of the given element counts)."""
    for i, t in enumerate(tensors):
        if not (t.is_cuda and t.is_contiguous()) or t.dtype != tensors[0].dtype:
            raise ValueError(f"{what} must be contiguous device tensors of one dtype")
        if counts is not None and t.numel() != counts[i]:
            raise ValueError(f"{what}[{i}] must hold {counts[i]} elements")
    if counts is not None and len(tensors) != len(counts):
        raise ValueError(f"{what}: {len(counts)} tensors are needed")
    return _ptr_array([t.data_ptr() or None for t in tensors])


def prepare_grad_norm(grads: Sequence, out, max_norm: float = 0.0, scale: float = 1.0, stream=None):
    """Pre-marshalled mr_grad_norm for gradients that stay where they are, on ``stream`` or the one current now.  ``max_norm``
    and ``scale`` are fixed with it: a loss scale that changes takes grad_norm, or another preparation."""
    grads = list(grads)
    _opt(out, "out", (_torch().float32,), 3)
    _dev_tensor(out, "out")
    ptrs = _tensor_list(grads, "grads")
    counts = (ctypes.c_uint64 * max(len(grads), 1))(*[t.numel() for t in grads])
    dt = DTYPE_CODE[dtype_name(grads[0])] if grads else DTYPE_CODE["fp32"]
    args = (ptrs, counts, len(grads), dt, scale, max_norm, out.data_ptr(), _stream_handle(stream))
    return _prepared("mr_grad_norm", lib().mr_grad_norm, args, (grads, out))


def grad_norm(grads: Sequence, out, max_norm: float = 0.0, scale: float = 1.0, stream=None):
    """out (3 floats) = [N, factor, finite]: N = scale * the 2-norm of all ``grads`` together, factor = scale * min(1,
    max_norm / (N + 1e-6)) (scale alone without a max_norm), finite = 1 if every element is finite, else 0 (and factor
    0).  adamw_step takes it as ``clip``."""
    prepare_grad_norm(grads, out, max_norm, scale, stream)()
    return out


@dataclasses.dataclass
class AdamWState:
    """The flat optimizer state of a list of tensors (mr_adamw_step's layout: each tensor's part starts on a multiple of
    32 elements).  32-bit moments: ``m`` and ``v`` fp32.  8-bit (MXFP8): ``m`` and ``v`` (the second moment's square
    root) torch.float8_e4m3fn with one torch.float8_e8m0fnu scale per 32 elements in ``m_scale`` and ``v_scale``.
    ``master``: fp32 copies of 16-bit parameters, or None."""

    m: Any
    v: Any
    m_scale: Any = None
    v_scale: Any = None
    master: Any = None

    @property
    def bits(self) -> int:
        return 32 if self.m_scale is None else 8

    def moments(self):
        """(m, v) as fp32: what the state stands for, for inspection and checkpoints."""
        if self.bits == 32:
            return self.m, self.v
        m, r = (q.float().view(-1, ADAMW_BLOCK).mul(s.float().view(-1, 1)).view(-1)
                for q, s in ((self.m, self.m_scale), (self.v, self.v_scale)))
        return m, r * r


def adamw_offsets(counts: Sequence[int]) -> tuple[list[int], int]:
    """(first element of each tensor in the flat state, its total length)."""
    c = (ctypes.c_uint64 * max(len(counts), 1))(*counts)
    total = ctypes.c_uint64(0)
    _check(lib().mr_adamw_state_elems(c, len(counts), ctypes.byref(total)), "mr_adamw_state_elems")
    at, n = [], 0
    for k in counts:
        at.append(n)
        n += -(-k // ADAMW_BLOCK) * ADAMW_BLOCK
    return at, int(total.value)


def adamw_init(params: Sequence, bits: int = 32, master: bool = False) -> AdamWState:
    """A zero state for ``params``; with ``master``, fp32 copies of them."""
    torch = _torch()
    if bits not in STATE_FORMAT:
        raise ValueError("bits must be 32 or 8")
    counts = [p.numel() for p in params]
    at, n = adamw_offsets(counts)
    dev = params[0].device
    st = AdamWState(torch.zeros(n, device=dev), torch.zeros(n, device=dev)) if bits == 32 else AdamWState(
        *(torch.zeros(n, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)),
        *(torch.zeros(n // ADAMW_BLOCK, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu) for _ in range(2)))
    if master:
        st.master = torch.zeros(n, device=dev)
        for p, a, k in zip(params, at, counts):
            st.master[a:a + k].copy_(p.detach().reshape(-1))
    return st


def _state_c(st: AdamWState, n: int) -> _AdamWStateC:
    torch = _torch()
    if st.m is None or st.v is None:
        raise ValueError("the state needs m and v")
    if st.bits == 32:
        want, scales = (torch.float32,), (None, None)
        if st.v_scale is not None:
            raise ValueError("v_scale without m_scale")
    else:
        want, f8 = (torch.float8_e4m3fn, torch.uint8), (torch.float8_e8m0fnu, torch.uint8)
        scales = (_opt(st.m_scale, "m_scale", f8, n // ADAMW_BLOCK), _opt(st.v_scale, "v_scale", f8, n // ADAMW_BLOCK))
    return _AdamWStateC(_opt(st.m, "m", want, n), _opt(st.v, "v", want, n), *scales,
                        _opt(st.master, "master", (torch.float32,), n))


def prepare_adamw(params: Sequence, grads: Sequence, state: AdamWState, params_out=None, state_out: AdamWState | None = None,
                  betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01, clip=None, seed: int = 0, stream=None):
    """Pre-marshalled mr_adamw_step for tensors that stay where they are: the returned ``call(lr, step)`` takes step
    ``step`` (from 1), on ``stream`` or the one that is current at preparation.  Results go in place, or to ``params_out`` /
    ``state_out``.  A HIP graph that captures the call repeats its ``lr`` and ``step``, and with them the bias corrections and
    the 8-bit state's random bits: capture each step anew, or keep the call outside."""
    params, grads = list(params), list(grads)
    counts = [p.numel() for p in params]
    _, n = adamw_offsets(counts)
    pp, gp = _tensor_list(params, "params"), _tensor_list(grads, "grads", counts)
    po = None if params_out is None else _tensor_list(list(params_out), "params_out", counts)
    if params_out is not None and params and params_out[0].dtype != params[0].dtype:
        raise ValueError("params_out must be of the params' dtype")
    if params and dtype_name(grads[0]) not in (dtype_name(params[0]), "fp32"):
        raise ValueError("grads must be of the params' dtype or torch.float32")
    sin = _state_c(state, n)
    if state_out is not None and state_out.bits != state.bits:
        raise ValueError("state_out must be in the state's format")
    sout = None if state_out is None else _state_c(state_out, n)
    _opt(clip, "clip", (_torch().float32,), 3)
    hyper = _AdamWHyperC(0.0, betas[0], betas[1], eps, weight_decay, 0, seed)
    args = (pp, gp, (ctypes.c_uint64 * max(len(counts), 1))(*counts), len(counts),
            DTYPE_CODE[dtype_name(params[0])] if params else 2, DTYPE_CODE[dtype_name(grads[0])] if grads else 2,
            STATE_FORMAT[state.bits], ctypes.byref(sin), po, None if sout is None else ctypes.byref(sout), ctypes.byref(hyper),
            None if clip is None else clip.data_ptr(), _stream_handle(stream))
    f = lib().mr_adamw_step

    def call(lr: float, step: int) -> None:
        if not 0 < step < 1 << 64:
            raise ValueError("step must count from 1")
        hyper.lr, hyper.step = lr, step
        st = f(*args)
        if st != MR_OK:
            raise MRError(st, "mr_adamw_step")

    call.keepalive = (params, grads, state, params_out, state_out, clip, sin, sout, hyper)
    return call


def adamw_step(params: Sequence, grads: Sequence, state: AdamWState, lr: float, step: int, params_out=None,
               state_out: AdamWState | None = None, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
               clip=None, seed: int = 0, stream=None) -> None:
    """One AdamW step (decoupled weight decay) over all ``params`` in one launch per 80 tensors, in place or into
    ``params_out`` / ``state_out``.  ``clip``: grad_norm's record, whose factor multiplies the gradients and which leaves the
    step out where a gradient is not finite.  ``seed``: of the 8-bit state's stochastic rounding."""
    prepare_adamw(params, grads, state, params_out, state_out, betas, eps, weight_decay, clip, seed, stream)(lr, step)


def workspace_bytes(W: int, n: int, dtype: str) -> int:
    return int(lib().mr_workspace_bytes(W, n, DTYPE_CODE[dtype]))


def set_workspace(buf=None, stream=None) -> None:
    """Bind a caller-owned uint8 device tensor as the two-shot workspace of ``stream`` (None unbinds)."""
    ptr, nbytes = (None, 0) if buf is None else (buf.data_ptr(), buf.numel() * buf.element_size())
    _check(lib().mr_set_workspace(_stream_handle(stream), ptr, nbytes), "mr_set_workspace")


def workspace_check(stream=None) -> int:
    """Synchronise ``stream`` and return (and clear) its two-shot barrier error word."""
    flags = ctypes.c_uint32(0)
    _check(lib().mr_workspace_check(_stream_handle(stream), ctypes.byref(flags)), "mr_workspace_check")
    return int(flags.value)


def set_option(name: str, value) -> None:
    """Set a process-wide option: ``twoshot_sync`` ("auto", "tile", "chunk", "grid", "last"), ``spin_limit`` (int),
    ``tile_shape`` ("auto", "wide", "medium", "narrow", "wide_pair") or ``sdma_cu_below`` (bytes)."""
    if name == "twoshot_sync" and isinstance(value, str):
        value = TWOSHOT_SYNC[value]
    if name == "tile_shape" and isinstance(value, str):
        value = TILE_SHAPE[value]
    _check(lib().mr_set_option(OPTION_CODE[name], int(value)), "mr_set_option")


def get_option(name: str):
    v = ctypes.c_int64(0)
    _check(lib().mr_get_option(OPTION_CODE[name], ctypes.byref(v)), "mr_get_option")
    if name == "twoshot_sync":
        return {c: k for k, c in TWOSHOT_SYNC.items()}[v.value]
    if name == "tile_shape":
        return {c: k for k, c in TILE_SHAPE.items()}[v.value]
    return int(v.value)
