"""Thin ctypes binding over the C ABI of include/vc.h.

Argument marshalling only: tensors become device pointers, counts and enum
codes; every step of every collective runs in libvcoll.so.  The functions
keep the C names.  There is no fallback: if the library is not built, or a
call fails, an exception is raised.

The C ABI takes bare pointers and counts and cannot see a buffer's size, so
before each call every tensor is checked to hold at least the elements the
call reads or writes there, contiguous, of the call's dtype, on one CUDA
device; anything else raises VCError(VC_ERR_INVALID_ARG) before the library
is called.  The checks cost about 5 us of host time for 16 tensors;
VC_CHECK_TENSORS=0 in the environment skips them.
"""
from __future__ import annotations

import ctypes
import itertools
import operator
import os
import struct
from typing import Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvcoll.so")

VC_SUCCESS, VC_ERR_INVALID_ARG, VC_ERR_UNSUPPORTED, VC_ERR_CUDA, VC_ERR_NOMEM, VC_ERR_TIMEOUT = range(6)
DTYPES = {"f32": 0, "bf16": 1, "i32": 2, "f16": 3, "i8": 4}
OPS = {"sum": 0, "max": 1, "min": 2}
ALGOS = {"fused": 0, "ring": 1, "rhd": 2, "dbt": 3, "binomial": 4, "scatter_allgather": 5,
         "pairwise": 6, "bruck": 7, "auto": 8, "pipe_chain": 9, "pipe_tree": 10, "mesh": 11, "ring_hop": 12}
ALGO_NAMES = {v: k for k, v in ALGOS.items()}
COST_POLICIES = {"hbm": 0, "link": 1}
COLLS = {"allreduce": 0, "reduce_scatter": 1, "allgather": 2, "broadcast": 3, "scatter": 4,
         "alltoall": 5, "gather": 6, "reduce": 7}
SCORES = {"softmax": 0, "sigmoid": 1}


class VCError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class TraceRecord(ctypes.Structure):
    _fields_ = [("coll", ctypes.c_int32), ("algo", ctypes.c_int32), ("step", ctypes.c_int32),
                ("kernel", ctypes.c_int32), ("bytes", ctypes.c_int64), ("nops", ctypes.c_int32),
                ("ms", ctypes.c_float)]


KERNEL_MODES = {0: "copy", 1: "f32", 2: "i32", 3: "bf16", 4: "bf16_pure", 5: "f16", 6: "f16_pure"}
KERNEL_OPS = {0: "sum", 1: "max", 2: "min"}


LAYER_KERNELS = ("norm", "norm_backward", "norm_weight", "route", "route_backward", "dispatch_plan", "dispatch",
                 "combine", "combine_backward", "expert_product", "expert_weight", "expert_product_fp8", "quantize",
                 "grad_norm", "clip", "pad")


def kernel_name(code: int) -> str:
    if code & 512:  # a layer operator
        return LAYER_KERNELS[code & 15]
    mode = KERNEL_MODES[code & 7]
    name = mode if mode == "copy" else f"{KERNEL_OPS[(code >> 3) & 3]}_{mode}"
    if code & 256:  # one launch over the whole GPU, each thread carrying its group through every step
        return name + "_sliced"
    if code & 128:  # one cluster launch for the whole plan
        return name + "_single_launch"
    extra = ("_tma" if mode == "copy" else "_batched") if code & 64 else ""
    return name + ("_large" if code & 32 else "") + extra


class PlanEntry(ctypes.Structure):
    _fields_ = [("step", ctypes.c_int32), ("op", ctypes.c_int32), ("role", ctypes.c_int32),
                ("pos", ctypes.c_int32), ("buf", ctypes.c_int32), ("owner", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("reduce", ctypes.c_int32), ("byte_off", ctypes.c_int64),
                ("n", ctypes.c_int64), ("nb", ctypes.c_int64), ("stride_bytes", ctypes.c_int64),
                ("elem0", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (loaded once); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z, V = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
        PP = ctypes.POINTER(ctypes.c_void_p)
        for name, args in {
            "vc_allreduce": [PP, PP, I, Z, I, I, I, V],
            "vc_reduce_scatter": [PP, PP, I, Z, I, I, I, V],
            "vc_allgather": [PP, PP, I, Z, I, I, V],
            "vc_broadcast": [P, PP, I, Z, I, I, I, V],
            "vc_scatter": [P, PP, I, Z, I, I, I, V],
            "vc_alltoall": [PP, PP, I, Z, I, I, V],
            "vc_broadcast_pipelined": [P, PP, I, Z, I, I, I, I, V],
            "vc_gather": [PP, P, I, Z, I, I, I, V],
            "vc_reduce": [PP, P, I, Z, I, I, I, I, V],
            # pointer arrays as packed bytes
            "vc_reduce_scatter_norm": [V, V, V, V, V, V, V, I, Z, Z, ctypes.c_double, I, I, V],
            "vc_reduce_scatter_norm_backward": [V, V, V, V, V, V, V, V, I, Z, Z, I, V],
            "vc_route": [V, V, V, V, I, Z, I, V, I, V],
            "vc_route_backward": [V, V, V, V, I, Z, I, V, I, V],
            "vc_dispatch_plan": [V, V, V, I, Z, I, I, Z, V],
            "vc_dispatch": [V, V, V, V, V, I, Z, Z, I, Z, I, V],
            "vc_combine": [V, V, V, V, I, Z, Z, I, Z, I, V],
            "vc_combine_backward": [V, V, V, V, V, V, I, Z, Z, I, Z, I, V],
            "vc_expert_product_fp8": [V, V, V, V, V, V, I, I, Z, Z, Z, I, V],
            "vc_quantize_fp8": [V, V, V, V, I, Z, Z, Z, I, I, V],
            "vc_clip_grad_norm": [V, V, V, V, I, Z, V, ctypes.c_double, I, V],
            "vc_expert_product": [V, V, V, V, I, I, Z, Z, Z, I, I, V],
            "vc_expert_product_backward": [V, V, V, V, V, V, I, I, Z, Z, Z, I, I, I, V],
        }.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = I
        L.vc_status_string.argtypes = [I]
        L.vc_status_string.restype = ctypes.c_char_p
        L.vc_last_error.argtypes = []
        L.vc_last_error.restype = ctypes.c_char_p
        L.vc_busbw_factor.argtypes = [I, I]
        L.vc_busbw_factor.restype = ctypes.c_double
        L.vc_plan_describe.argtypes = [I, I, I, Z, I, I, I, I, I, ctypes.POINTER(PlanEntry), Z,
                                       ctypes.POINTER(Z), ctypes.POINTER(Z), ctypes.POINTER(I)]
        L.vc_plan_describe.restype = I
        U32P, U8P = ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(ctypes.c_uint8)
        L.vc_plan_exec_order.argtypes = [I, I, I, Z, I, I, I, I, I, U32P, U8P, Z, U8P, Z, ctypes.POINTER(Z),
                                         ctypes.POINTER(I)]
        L.vc_plan_exec_order.restype = I
        L.vc_plan_form.argtypes = [I, I, I, Z, I, I, I, I, I, ctypes.POINTER(I), ctypes.POINTER(I),
                                   ctypes.POINTER(I)]
        L.vc_plan_form.restype = I
        L.vc_trace_enable.argtypes = [I]
        L.vc_trace_enable.restype = I
        L.vc_trace_read.argtypes = [ctypes.POINTER(TraceRecord), Z, ctypes.POINTER(Z)]
        L.vc_trace_read.restype = I
        L.vc_set_cost_model.argtypes = [I, ctypes.c_double, ctypes.c_double]
        L.vc_set_cost_model.restype = I
        L.vc_get_cost_model.argtypes = [ctypes.POINTER(I), ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]
        L.vc_get_cost_model.restype = I
        L.vc_select_algo.argtypes = [I, I, Z, I, I, ctypes.POINTER(I), ctypes.POINTER(ctypes.c_double)]
        L.vc_select_algo.restype = I
        L.vc_device_errors.argtypes = [V, ctypes.POINTER(ctypes.c_uint32)]
        L.vc_device_errors.restype = I
        L.vc_copy_selftest.argtypes = [V, ctypes.POINTER(ctypes.c_uint32)]
        L.vc_copy_selftest.restype = I
        L.vc_product_selftest.argtypes = [V, ctypes.POINTER(ctypes.c_uint32)]
        L.vc_product_selftest.restype = I
        L.vc_set_single_launch.argtypes = [Z]
        L.vc_set_single_launch.restype = I
        L.vc_get_single_launch.argtypes = [ctypes.POINTER(Z)]
        L.vc_get_single_launch.restype = I
        L.vc_set_merge_steps.argtypes = [I]
        L.vc_set_merge_steps.restype = I
        L.vc_get_merge_steps.argtypes = [ctypes.POINTER(I)]
        L.vc_get_merge_steps.restype = I
        L.vc_set_slice_limit.argtypes = [Z]
        L.vc_set_slice_limit.restype = I
        L.vc_get_slice_limit.argtypes = [ctypes.POINTER(Z)]
        L.vc_get_slice_limit.restype = I
        L.vc_set_reuse_order.argtypes = [Z]
        L.vc_set_reuse_order.restype = I
        L.vc_get_reuse_order.argtypes = [ctypes.POINTER(Z)]
        L.vc_get_reuse_order.restype = I
        L.vc_set_copy_pipeline.argtypes = [Z]
        L.vc_set_copy_pipeline.restype = I
        L.vc_get_copy_pipeline.argtypes = [ctypes.POINTER(Z)]
        L.vc_get_copy_pipeline.restype = I
        L.vc_version.argtypes = []
        L.vc_version.restype = I
        _lib = L
    return _lib


def check(status: int) -> None:
    if status != VC_SUCCESS:
        L = lib()
        raise VCError(status, f"{L.vc_status_string(status).decode()}: {L.vc_last_error().decode()}")


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

_ARRAY_TYPES: dict = {}


def _ptr_array(ptrs: Sequence[int]):
    n = len(ptrs)
    typ = _ARRAY_TYPES.get(n)
    if typ is None:
        typ = _ARRAY_TYPES[n] = ctypes.c_void_p * n
    return typ(*ptrs)


_TORCH_DTYPES: dict = {}


def _dtype_code(t) -> int:
    if not _TORCH_DTYPES:
        import torch

        _TORCH_DTYPES.update({torch.float32: 0, torch.bfloat16: 1, torch.int32: 2, torch.float16: 3})
    code = _TORCH_DTYPES.get(t.dtype)
    if code is None:
        raise VCError(VC_ERR_INVALID_ARG, f"unsupported dtype {t.dtype}")
    return code


_raw_stream = None


def _stream_handle(stream, like) -> int:
    """The cudaStream_t to enqueue on: `stream` (a torch stream or a raw
    handle), else the current stream of `like`'s device."""
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            import torch

            # the raw handle without building a Stream object (measured ~3 us per call)
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
                (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        return int(_raw_stream(like.get_device()))
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


CHECK_TENSORS = os.environ.get("VC_CHECK_TENSORS", "1") != "0"


def _checked(ts, need: int, like) -> list[int]:
    """Pointers of `ts`, each tensor checked to hold at least `need`
    contiguous elements of `like`'s dtype on `like`'s CUDA device."""
    if not CHECK_TENSORS:
        return [t.data_ptr() for t in ts]
    dt, dev = like.dtype, like.get_device()
    if dev < 0:
        raise VCError(VC_ERR_INVALID_ARG, f"tensors must be on a CUDA device, not {like.device}")
    out = []
    for t in ts:
        if t.numel() < need or t.dtype is not dt or t.get_device() != dev or not t.is_contiguous():
            raise VCError(VC_ERR_INVALID_ARG,
                          f"each tensor must be contiguous {dt} on cuda:{dev} with at least {need} elements, "
                          f"not {tuple(t.shape)} {t.dtype} on {t.device}"
                          + ("" if t.is_contiguous() else " (not contiguous)"))
        out.append(t.data_ptr())
    return out


def _ranks(ts, N: int, what: str):
    if len(ts) != N:
        raise VCError(VC_ERR_INVALID_ARG, f"{what}: {len(ts)} tensors for {N} ranks")
    return ts


def _code(table: dict, key) -> int:
    return table[key] if isinstance(key, str) else int(key)


# ---------------------------------------------------------------------------
# collectives (tensor arguments; one tensor per virtual rank)
# ---------------------------------------------------------------------------

def vc_allreduce(send, recv, algo="fused", op="sum", stream=None) -> None:
    """recv[r] = sum over ranks of send[q]; ``send[r] is recv[r]`` allowed."""
    N = len(send)
    n = send[0].numel()
    sp, rp = _checked(send, n, send[0]), _checked(_ranks(recv, N, "recv"), n, send[0])
    check(lib().vc_allreduce(_ptr_array(sp), _ptr_array(rp), N, n, _dtype_code(send[0]), _code(OPS, op),
                             _code(ALGOS, algo), _stream_handle(stream, send[0])))


def vc_reduce_scatter(send, recv, algo="fused", op="sum", stream=None) -> None:
    """recv[r] = block r of the sum; send[q] holds N blocks of recv[r].numel()."""
    N = len(send)
    rc = recv[0].numel()
    sp, rp = _checked(send, N * rc, send[0]), _checked(_ranks(recv, N, "recv"), rc, send[0])
    check(lib().vc_reduce_scatter(_ptr_array(sp), _ptr_array(rp), N, rc, _dtype_code(send[0]), _code(OPS, op),
                                  _code(ALGOS, algo), _stream_handle(stream, send[0])))


def vc_allgather(send, recv, algo="fused", stream=None) -> None:
    """recv[r] = concatenation of send[0..N-1]."""
    N = len(send)
    sc = send[0].numel()
    sp, rp = _checked(send, sc, send[0]), _checked(_ranks(recv, N, "recv"), N * sc, send[0])
    check(lib().vc_allgather(_ptr_array(sp), _ptr_array(rp), N, sc, _dtype_code(send[0]), _code(ALGOS, algo),
                             _stream_handle(stream, send[0])))


def vc_broadcast(send_root, recv, root=0, algo="fused", stream=None) -> None:
    """recv[r] = send_root for every rank; ``send_root is recv[root]`` allowed."""
    N = len(recv)
    n = recv[0].numel()
    (sp,), rp = _checked([send_root], n, send_root), _checked(recv, n, send_root)
    check(lib().vc_broadcast(ctypes.c_void_p(sp), _ptr_array(rp), N, n, _dtype_code(send_root), int(root),
                             _code(ALGOS, algo), _stream_handle(stream, send_root)))


def vc_scatter(send_root, recv, root=0, algo="fused", stream=None) -> None:
    """recv[r] = block r of send_root."""
    N = len(recv)
    rc = recv[0].numel()
    (sp,), rp = _checked([send_root], N * rc, send_root), _checked(recv, rc, send_root)
    check(lib().vc_scatter(ctypes.c_void_p(sp), _ptr_array(rp), N, rc, _dtype_code(send_root), int(root),
                           _code(ALGOS, algo), _stream_handle(stream, send_root)))


def vc_alltoall(send, recv, algo="fused", stream=None) -> None:
    """recv[j] block i = send[i] block j; every buffer holds N blocks."""
    N = len(send)
    blk = send[0].numel() // N
    sp, rp = _checked(send, N * blk, send[0]), _checked(_ranks(recv, N, "recv"), N * blk, send[0])
    check(lib().vc_alltoall(_ptr_array(sp), _ptr_array(rp), N, blk, _dtype_code(send[0]), _code(ALGOS, algo),
                            _stream_handle(stream, send[0])))


def vc_broadcast_pipelined(send_root, recv, root=0, algo="pipe_tree", nchunks=0, stream=None) -> None:
    """Chunked Broadcast; nchunks=0 takes the cost model's optimum."""
    N = len(recv)
    n = recv[0].numel()
    (sp,), rp = _checked([send_root], n, send_root), _checked(recv, n, send_root)
    check(lib().vc_broadcast_pipelined(ctypes.c_void_p(sp), _ptr_array(rp), N, n, _dtype_code(send_root),
                                       int(root), _code(ALGOS, algo), int(nchunks),
                                       _stream_handle(stream, send_root)))


def vc_gather(send, recv_root, root=0, algo="fused", stream=None) -> None:
    """recv_root = concatenation of send[0..N-1] (on the root only)."""
    N = len(send)
    sc = send[0].numel()
    sp, (rp,) = _checked(send, sc, send[0]), _checked([recv_root], N * sc, send[0])
    check(lib().vc_gather(_ptr_array(sp), ctypes.c_void_p(rp), N, sc, _dtype_code(send[0]), int(root),
                          _code(ALGOS, algo), _stream_handle(stream, send[0])))


def vc_reduce(send, recv_root, root=0, algo="fused", op="sum", stream=None) -> None:
    """recv_root = sum over ranks of send[q]; ``recv_root is send[root]`` allowed."""
    N = len(send)
    n = send[0].numel()
    sp, (rp,) = _checked(send, n, send[0]), _checked([recv_root], n, send[0])
    check(lib().vc_reduce(_ptr_array(sp), ctypes.c_void_p(rp), N, n, _dtype_code(send[0]), _code(OPS, op),
                          int(root), _code(ALGOS, algo), _stream_handle(stream, send[0])))


# ---------------------------------------------------------------------------
# layer operators
# ---------------------------------------------------------------------------
# Each per-rank argument is a sequence of one tensor per virtual rank, or one
# contiguous tensor whose first dimension is the ranks (rank r's buffer is its
# slice r).  Sizes come from the tensors' shapes.

# Pointer arrays go to the library as packed bytes, and the checks compare
# attributes in place: the smallest calls spend most of their time here, and a
# ctypes array per argument took twice as long.  N pointers p, p + s, ... are
# one whole number, p * ones + s * steps in 64-bit digits (lowest first, as the
# machine stores them).

_DIGITS: dict = {}
_SEQUENCES = (list, tuple)


def _digits(N: int):
    d = _DIGITS.get(N)
    if d is None:
        d = _DIGITS[N] = sum(1 << 64 * i for i in range(N)), sum(i << 64 * i for i in range(N))
    return d


def _invalid(msg: str):
    return VCError(VC_ERR_INVALID_ARG, msg)


def _refuse(x, what: str, shape: tuple, dtype, dev: int):
    raise _invalid(f"{what}: want contiguous {tuple(shape)} {dtype} on cuda:{dev}, not {tuple(x.shape)} {x.dtype} on "
                   f"{x.device}" + ("" if x.is_contiguous() else " (not contiguous)"))


def _bad(x, shape, dtype, dev) -> bool:
    return x.shape != shape or x.dtype is not dtype or x.get_device() != dev or not x.is_contiguous()


def _first(a, what: str):
    if not a:
        raise _invalid(f"{what}: none, want one for each rank")
    return a[0]


def _shape(a, n: int, what: str) -> tuple:
    """(ranks, the n dimensions of each rank's tensor) of a per-rank argument."""
    shape = (len(a), *_first(a, what).shape) if a.__class__ in _SEQUENCES else a.shape
    if len(shape) != n + 1:
        raise _invalid(f"{what}: want {n} dimensions for each rank, not {tuple(shape[1:])}")
    return shape


def _start(a):
    """What a call's checks go by: a tensor of the per-rank argument, its
    dtype, element size and CUDA device."""
    x = _first(a, "tensors") if a.__class__ in _SEQUENCES else a
    dev = x.get_device()
    if dev < 0:
        raise _invalid(f"tensors must be on a CUDA device, not {x.device}")
    dt = x.dtype
    return x, dt, dt.itemsize, dev


def _ptrs(a, what: str, full: tuple, size: int, dtype, dev: int):
    """The pointer array of a per-rank argument (None stays None): `full` is
    the shape of all ranks' tensors stacked, `size` the bytes of each rank's."""
    if a is None:
        return None
    N = full[0]
    if a.__class__ in _SEQUENCES:
        if len(a) != N:
            raise _invalid(f"{what}: {len(a)} tensors for {N} ranks")
        if CHECK_TENSORS:
            for x in a:
                if _bad(x, full[1:], dtype, dev):
                    _refuse(x, what, full[1:], dtype, dev)
        return struct.pack(f"={N}Q", *[x.data_ptr() for x in a])
    if CHECK_TENSORS and (a.shape != full or a.dtype is not dtype or a.get_device() != dev or not a.is_contiguous()):
        _refuse(a, what, full, dtype, dev)
    ones, steps = _DIGITS.get(N) or _digits(N)
    return (a.data_ptr() * ones + size * steps).to_bytes(8 * N, "little")


def _shared(a, what: str, full: tuple, size: int, dtype, dev: int):
    """As _ptrs, or one tensor that stands for every rank."""
    if a is None or a.__class__ in _SEQUENCES or len(a.shape) == len(full):
        return _ptrs(a, what, full, size, dtype, dev)
    if CHECK_TENSORS and _bad(a, full[1:], dtype, dev):
        _refuse(a, what, full[1:], dtype, dev)
    return a.data_ptr().to_bytes(8, "little") * full[0]


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


_pack_how = struct.Struct("=6if").pack  # vc_route_t: score, topk, ngroups, topk_groups, group_top, renormalize, scale


def _how(*fields) -> bytes:
    try:
        return _pack_how(*fields)
    except (struct.error, OverflowError) as e:
        raise _invalid(f"route description {fields}: {e}") from None


def vc_reduce_scatter_norm(send, weight, out, residual=None, residual_out=None, scale=None, rstd=None,
                           eps: float = 1e-6, stream=None) -> None:
    """ReduceScatter of the ranks' partial sums, residual and RMS norm in one pass.

    ``send[q]`` is (N * rows, hidden), ``out[r]`` (rows, hidden) in the data
    type, or int8 with ``scale[r]`` (rows,) fp32.  ``weight`` is (hidden,) for
    each rank or one for all.  ``residual[r]`` is added, the sum goes to
    ``residual_out[r]`` (which may be the residual), 1/rms to ``rstd[r]``
    (rows,) fp32."""
    torch = _torch()
    x, dt, es, dev = _start(send)
    N, rows, hidden = row = _shape(out, 2, "out")
    odt = (out[0] if out.__class__ in _SEQUENCES else out).dtype
    code, i8, f32 = _dtype_code(x), odt is torch.int8, torch.float32
    if i8 and scale is None:
        raise _invalid("an int8 output wants a scale")
    size, one = rows * hidden * es, (N, rows)
    check(lib().vc_reduce_scatter_norm(
        _ptrs(send, "send", (N, N * rows, hidden), N * size, dt, dev),
        _ptrs(residual, "residual", row, size, dt, dev),
        _shared(weight, "weight", (N, hidden), hidden * es, dt, dev),
        _ptrs(residual_out, "residual_out", row, size, dt, dev),
        _ptrs(out, "out", row, rows * hidden if i8 else size, torch.int8 if i8 else dt, dev),
        _ptrs(scale, "scale", one, rows * 4, f32, dev) if i8 else None,
        _ptrs(rstd, "rstd", one, rows * 4, f32, dev),
        N, rows, hidden, eps, code, DTYPES["i8"] if i8 else code, _stream_handle(stream, x)))


def vc_reduce_scatter_norm_backward(dout, h, weight, rstd, dsend=None, dresidual=None, dweight=None,
                                    dresidual_out=None, stream=None) -> None:
    """Gradients of vc_reduce_scatter_norm; ``h`` is its residual_out.

    ``dsend[q]`` (N * rows, hidden), ``dresidual[r]`` (rows, hidden) and
    ``dweight[r]`` (hidden,) fp32, this rank's part, are written where given;
    ``dresidual_out`` is the gradient that reaches the sum itself."""
    x, dt, es, dev = _start(dout)
    f32 = _torch().float32
    N, rows, hidden = row = _shape(dout, 2, "dout")
    size = rows * hidden * es
    check(lib().vc_reduce_scatter_norm_backward(
        _ptrs(dout, "dout", row, size, dt, dev),
        _ptrs(dresidual_out, "dresidual_out", row, size, dt, dev),
        _ptrs(h, "h", row, size, dt, dev),
        _shared(weight, "weight", (N, hidden), hidden * es, dt, dev),
        _ptrs(rstd, "rstd", (N, rows), rows * 4, f32, dev),
        _ptrs(dsend, "dsend", (N, N * rows, hidden), N * size, dt, dev),
        _ptrs(dresidual, "dresidual", row, size, dt, dev),
        _ptrs(dweight, "dweight", (N, hidden), hidden * 4, f32, dev),
        N, rows, hidden, _dtype_code(x), _stream_handle(stream, x)))


def vc_route(logits, ids, weights, bias=None, score="softmax", ngroups: int = 1, topk_groups: int = 1,
             group_top: int = 1, renormalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """Choice of experts: ``ids[r]`` (rows, topk) int32 and ``weights[r]``
    (rows, topk) fp32 from ``logits[r]`` (rows, experts).

    ``bias`` is (experts,) fp32 for each rank or one for all."""
    torch = _torch()
    x, dt, es, dev = _start(logits)
    N, rows, experts = every = _shape(logits, 2, "logits")
    topk = _shape(ids, 2, "ids")[2]
    chosen, size = (N, rows, topk), rows * topk * 4
    how = _how(_code(SCORES, score), topk, ngroups, topk_groups, group_top, bool(renormalize), scale)
    check(lib().vc_route(
        _ptrs(logits, "logits", every, rows * experts * es, dt, dev),
        _shared(bias, "bias", (N, experts), experts * 4, torch.float32, dev),
        _ptrs(ids, "ids", chosen, size, torch.int32, dev),
        _ptrs(weights, "weights", chosen, size, torch.float32, dev),
        N, rows, experts, how, _dtype_code(x), _stream_handle(stream, x)))


def vc_route_backward(dweights, logits, ids, dlogits, score="softmax", renormalize: bool = True, scale: float = 1.0,
                      stream=None) -> None:
    """``dlogits[r]`` (rows, experts) from ``dweights[r]`` (rows, topk) fp32,
    with vc_route's logits and ids."""
    torch = _torch()
    x, dt, es, dev = _start(logits)
    N, rows, experts = every = _shape(logits, 2, "logits")
    topk = _shape(ids, 2, "ids")[2]
    chosen, size = (N, rows, topk), rows * topk * 4
    how = _how(_code(SCORES, score), topk, 1, 1, 1, bool(renormalize), scale)
    check(lib().vc_route_backward(
        _ptrs(dweights, "dweights", chosen, size, torch.float32, dev),
        _ptrs(logits, "logits", every, rows * experts * es, dt, dev),
        _ptrs(ids, "ids", chosen, size, torch.int32, dev),
        _ptrs(dlogits, "dlogits", every, rows * experts * es, dt, dev),
        N, rows, experts, how, _dtype_code(x), _stream_handle(stream, x)))


def vc_dispatch_plan(ids, slots, offsets, capacity: int, stream=None) -> None:
    """Where every (token, choice) goes: ``slots[r]`` (rows, topk) int32, and
    ``offsets[d]`` (experts of a rank + 1,) int32, where rank d's experts'
    rows begin, from ``ids[r]`` (rows, topk) int32.  ``capacity`` rows a rank
    at most."""
    i32 = _torch().int32
    x, _, _, dev = _start(ids)
    N, rows, topk = chosen = _shape(ids, 2, "ids")
    ends = _shape(offsets, 1, "offsets")[1]
    if capacity < 1 or ends < 1:
        raise _invalid("capacity and the offsets' length must be at least 1")
    check(lib().vc_dispatch_plan(
        _ptrs(ids, "ids", chosen, rows * topk * 4, i32, dev),
        _ptrs(slots, "slots", chosen, rows * topk * 4, i32, dev),
        _ptrs(offsets, "offsets", (N, ends), ends * 4, i32, dev),
        N, rows, topk, (ends - 1) * N, capacity, _stream_handle(stream, x)))


def vc_dispatch(send, slots, recv, scale=None, recv_scale=None, stream=None) -> None:
    """``send[r]``'s rows (rows, hidden) to the slots' rows of ``recv[d]``
    (capacity, hidden), and ``scale[r]`` (rows,) fp32 to ``recv_scale[d]``
    (capacity,) where given.  fp32, bf16, fp16, int8 or float8_e4m3fn rows."""
    torch = _torch()
    x, dt, es, dev = _start(send)
    N, rows, hidden = row = _shape(send, 2, "send")
    topk, cap = _shape(slots, 2, "slots")[2], _shape(recv, 2, "recv")[1]
    check(lib().vc_dispatch(
        _ptrs(send, "send", row, rows * hidden * es, dt, dev),
        _ptrs(scale, "scale", (N, rows), rows * 4, torch.float32, dev),
        _ptrs(slots, "slots", (N, rows, topk), rows * topk * 4, torch.int32, dev),
        _ptrs(recv, "recv", (N, cap, hidden), cap * hidden * es, dt, dev),
        _ptrs(recv_scale, "recv_scale", (N, cap), cap * 4, torch.float32, dev),
        N, rows, hidden, topk, cap, DTYPES["i8"] if dt in (torch.int8, torch.float8_e4m3fn) else _dtype_code(x),
        _stream_handle(stream, x)))


def vc_combine(recv, slots, out, weights=None, stream=None) -> None:
    """``out[r]`` (rows, hidden): each token's rows of ``recv[d]`` (capacity,
    hidden), weighted by ``weights[r]`` (rows, topk) fp32 (1 where None) and
    summed.  With the gradient of recv and no weights: dispatch's gradient."""
    torch = _torch()
    x, dt, es, dev = _start(out)
    N, rows, hidden = row = _shape(out, 2, "out")
    topk, cap = _shape(slots, 2, "slots")[2], _shape(recv, 2, "recv")[1]
    chosen, size = (N, rows, topk), rows * topk * 4
    check(lib().vc_combine(
        _ptrs(recv, "recv", (N, cap, hidden), cap * hidden * es, dt, dev),
        _ptrs(slots, "slots", chosen, size, torch.int32, dev),
        _ptrs(weights, "weights", chosen, size, torch.float32, dev),
        _ptrs(out, "out", row, rows * hidden * es, dt, dev),
        N, rows, hidden, topk, cap, _dtype_code(x), _stream_handle(stream, x)))


def vc_combine_backward(dout, recv, slots, weights=None, drecv=None, dweights=None, stream=None) -> None:
    """Gradients of vc_combine: ``drecv[d]`` (capacity, hidden) and
    ``dweights[r]`` (rows, topk) fp32, where given.  ``recv`` may be None
    without dweights."""
    torch = _torch()
    x, dt, es, dev = _start(dout)
    N, rows, hidden = row = _shape(dout, 2, "dout")
    if recv is None and drecv is None:
        raise _invalid("no gradient is asked for")
    topk, cap = _shape(slots, 2, "slots")[2], _shape(recv if recv is not None else drecv, 2, "recv")[1]
    chosen, size = (N, rows, topk), rows * topk * 4
    there, bulk = (N, cap, hidden), cap * hidden * es
    check(lib().vc_combine_backward(
        _ptrs(dout, "dout", row, rows * hidden * es, dt, dev),
        _ptrs(recv, "recv", there, bulk, dt, dev),
        _ptrs(slots, "slots", chosen, size, torch.int32, dev),
        _ptrs(weights, "weights", chosen, size, torch.float32, dev),
        _ptrs(drecv, "drecv", there, bulk, dt, dev),
        _ptrs(dweights, "dweights", chosen, size, torch.float32, dev),
        N, rows, hidden, topk, cap, _dtype_code(x), _stream_handle(stream, x)))


def _experts(offsets, N: int, what) -> int:
    """Experts of each rank, from the offsets (experts + 1,) of each."""
    ends = _shape(offsets, 1, "offsets")[1]
    if ends < 2:
        raise _invalid(f"offsets: want {what} + 1 for each rank, not {ends}")
    return ends - 1


def vc_expert_product(rows, weight, offsets, out, transposed: bool = False, stream=None) -> None:
    """Each expert's product with the rows that its rank has received.

    ``rows[d]`` (capacity, in) and ``offsets[d]`` (experts of a rank + 1,)
    int32, as vc_dispatch and vc_dispatch_plan write them; ``weight[d]``
    (experts of a rank, in, out), or (experts of a rank, out, in) with
    ``transposed``; ``out[d]`` (capacity, out).  Rows of no expert keep what
    out holds."""
    i32 = _torch().int32
    x, dt, es, dev = _start(rows)
    N, cap, win = row = _shape(rows, 2, "rows")
    width, each = _shape(out, 2, "out")[2], _experts(offsets, N, "experts")
    check(lib().vc_expert_product(
        _ptrs(rows, "rows", row, cap * win * es, dt, dev),
        _ptrs(weight, "weight", (N, each, width, win) if transposed else (N, each, win, width), each * win * width * es, dt, dev),
        _ptrs(offsets, "offsets", (N, each + 1), (each + 1) * 4, i32, dev),
        _ptrs(out, "out", (N, cap, width), cap * width * es, dt, dev),
        N, each * N, cap, win, width, bool(transposed), _dtype_code(x), _stream_handle(stream, x)))


def vc_expert_product_backward(dout, rows, weight, offsets, drows=None, dweight=None, transposed: bool = False,
                               stream=None) -> None:
    """Gradients of vc_expert_product: ``drows[d]`` (capacity, in) and
    ``dweight[d]``, shaped as the weights, in their type or fp32, where given.
    ``weight`` may be None without drows, ``rows`` without dweight."""
    torch = _torch()
    x, dt, es, dev = _start(dout)
    N, cap, width = row = _shape(dout, 2, "dout")
    if drows is None and dweight is None:
        raise _invalid("no gradient is asked for")
    if rows is None and (drows is None or dweight is not None):
        raise _invalid("dweight wants rows")
    win = _shape(rows if rows is not None else drows, 2, "rows")[2]
    each = _experts(offsets, N, "experts")
    every, n = (N, each, width, win) if transposed else (N, each, win, width), each * win * width
    wdt = dt
    if dweight is not None and (_first(dweight, "dweight") if dweight.__class__ in _SEQUENCES else dweight).dtype is torch.float32:
        wdt = torch.float32
    check(lib().vc_expert_product_backward(
        _ptrs(dout, "dout", row, cap * width * es, dt, dev),
        _ptrs(rows, "rows", (N, cap, win), cap * win * es, dt, dev),
        _ptrs(weight, "weight", every, n * es, dt, dev),
        _ptrs(offsets, "offsets", (N, each + 1), (each + 1) * 4, torch.int32, dev),
        _ptrs(drows, "drows", (N, cap, win), cap * win * es, dt, dev),
        _ptrs(dweight, "dweight", every, n * wdt.itemsize, wdt, dev),
        N, each * N, cap, win, width, bool(transposed), _dtype_code(x),
        DTYPES["f32"] if wdt is torch.float32 else _dtype_code(x), _stream_handle(stream, x)))


FP8_BLOCK = 128  # VC_FP8_BLOCK
_dtype_of = operator.attrgetter("dtype")


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def vc_quantize_fp8(x, out, scale, offsets=None, block_rows: int = 1, stream=None) -> None:
    """Rounds ``x[r]`` (rows, width) or (matrices, rows, width) to
    ``out[r]``, float8_e4m3fn of the same shape, with ``scale[r]`` fp32: one for
    each 128 of a row (``block_rows`` 1), shape (.., rows, ceil(width / 128)),
    or for each 128 rows by 128 (``block_rows`` 128).  ``offsets[d]`` (experts
    of a rank + 1,) int32: only the rows that the rank's experts have."""
    torch = _torch()
    t, dt, es, dev = _start(x)
    shape = (len(x), *x[0].shape) if x.__class__ in _SEQUENCES else tuple(x.shape)
    if len(shape) not in (3, 4):
        raise _invalid(f"x: want (rows, width) or (matrices, rows, width) for each rank, not {tuple(shape[1:])}")
    N, rows, width = shape[0], shape[-2], shape[-1]
    mats = shape[1] if len(shape) == 4 else 1
    if block_rows not in (1, FP8_BLOCK):
        raise _invalid(f"block_rows is 1 or {FP8_BLOCK}, not {block_rows}")
    n, down = mats * rows * width, -(-rows // block_rows)
    count = None
    if offsets is not None:
        ends = _experts(offsets, N, "experts") + 1
        first = _ptrs(offsets, "offsets", (N, ends), ends * 4, torch.int32, dev)
        count = struct.pack(f"={N}Q", *(a + 4 * (ends - 1) for a in struct.unpack(f"={N}Q", first)))
    check(lib().vc_quantize_fp8(
        _ptrs(x, "x", shape, n * es, dt, dev),
        _ptrs(out, "out", shape, n, torch.float8_e4m3fn, dev),
        _ptrs(scale, "scale", (*shape[:-2], down, _blocks(width)), mats * down * _blocks(width) * 4, torch.float32, dev),
        count, N, mats, rows, width, block_rows, _dtype_code(t), _stream_handle(stream, t)))


def vc_expert_product_fp8(rows, row_scale, weight, weight_scale, offsets, out, stream=None) -> None:
    """vc_expert_product of float8_e4m3fn ``rows[d]`` (capacity, in) and
    ``weight[d]`` (experts of a rank, out, in), with the scales that
    vc_quantize_fp8 gives them: ``row_scale[d]`` (capacity, ceil(in / 128)) and
    ``weight_scale[d]`` (experts of a rank, ceil(out / 128), ceil(in / 128)).
    ``out[d]`` (capacity, out) in fp32, bf16 or fp16."""
    torch = _torch()
    x, dt, es, dev = _start(out)
    f8, f32 = torch.float8_e4m3fn, torch.float32
    N, cap, win = row = _shape(rows, 2, "rows")
    width, each = _shape(out, 2, "out")[2], _experts(offsets, N, "experts")
    across, down = _blocks(win), _blocks(width)
    check(lib().vc_expert_product_fp8(
        _ptrs(rows, "rows", row, cap * win, f8, dev),
        _ptrs(row_scale, "row_scale", (N, cap, across), cap * across * 4, f32, dev),
        _ptrs(weight, "weight", (N, each, width, win), each * win * width, f8, dev),
        _ptrs(weight_scale, "weight_scale", (N, each, down, across), each * down * across * 4, f32, dev),
        _ptrs(offsets, "offsets", (N, each + 1), (each + 1) * 4, torch.int32, dev),
        _ptrs(out, "out", (N, cap, width), cap * width * es, dt, dev),
        N, each * N, cap, win, width, _dtype_code(x), _stream_handle(stream, x)))


def vc_clip_grad_norm(grads, norm, max_norm=None, out=None, across: bool = True, stream=None) -> None:
    """The norm of the ranks' gradients, and their clipping by it.

    ``grads[r]``: rank r's tensors, the same types in the same order on every
    rank, any sizes; ``norm`` (ranks,) fp32, or one scalar tensor for each
    rank.  With ``across`` the norm is over all ranks (each holds shards of one
    model), without over each rank's own.  ``max_norm`` None: the norm alone;
    else gradients above it are scaled to it, in place or into ``out[r]``."""
    torch = _torch()
    if grads.__class__ not in _SEQUENCES:
        raise _invalid("grads: want a list of each rank's tensors")
    try:
        N, T = len(grads), len(_first(grads, "grads"))
    except TypeError:
        raise _invalid("grads: want a list of each rank's tensors") from None
    like = _first(norm, "norm") if norm.__class__ in _SEQUENCES else norm
    dev = like.get_device()
    if dev < 0:
        raise _invalid(f"tensors must be on a CUDA device, not {like.device}")
    if max_norm is None and out is not None:
        raise _invalid("out wants a max_norm")
    ptrs, outs, sizes, codes = _lists().pack(grads, out, dev) or _gradients(grads, out, N, T, dev)
    check(lib().vc_clip_grad_norm(
        ptrs, None if max_norm is None else ptrs if out is None else outs, sizes, codes, N, T,
        _ptrs(norm, "norm", (N,), 4, torch.float32, dev), 0.0 if max_norm is None else max_norm, bool(across),
        _stream_handle(stream, like)))


_lists_module = None


def _lists():
    """The compiled part of this binding (csrc/lists.cpp)."""
    global _lists_module
    if _lists_module is None:
        version = str(_torch().__version__).split("+")[0]
        try:
            from . import _lists as module
        except ImportError as e:
            raise RuntimeError(f"_lists.so is not built; run __graft_entry__.build() ({e})") from None
        if module.torch != version:
            raise RuntimeError(f"_lists.so is built for PyTorch {module.torch}, not {version}; build again")
        _lists_module = module
    return _lists_module


def _gradients(grads, out, N: int, T: int, dev: int) -> tuple:
    """What _lists.pack returns, for lists that it left alone: sequences and
    tensors that are not plain ones, or that the call refuses."""
    Tensor = _torch().Tensor
    try:
        mine = list(itertools.chain.from_iterable(grads))
        to = mine if out is None else list(itertools.chain.from_iterable(out))
        same = set(map(len, grads)) == {T} and (out is None or (len(out) == N and set(map(len, out)) == {T}))
    except TypeError:
        raise _invalid("grads, out: want a list of each rank's tensors") from None
    if not same:
        raise _invalid("grads, out: want the same number of tensors on every rank")
    for t in mine if out is None else mine + to:
        if not isinstance(t, Tensor):
            raise _invalid(f"grads, out: want tensors, not {type(t).__name__}")
    sizes = list(map(Tensor.numel, mine))
    types = list(map(_dtype_of, mine[:T]))
    if CHECK_TENSORS:
        for ts in (mine, to)[:1 if to is mine else 2]:
            for t, dt, n in zip(ts, types * N, sizes):
                if t.dtype is not dt or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
                    raise _invalid(f"gradients: want contiguous {n} of {dt} on cuda:{dev}, not {tuple(t.shape)} {t.dtype} on "
                                   f"{t.device}" + ("" if t.is_contiguous() else " (not contiguous)"))
    code = {dt: _dtype_code(t) for dt, t in zip(types, mine)}
    pack = struct.Struct(f"={N * T}Q").pack
    return (pack(*map(Tensor.data_ptr, mine)), None if out is None else pack(*map(Tensor.data_ptr, to)), pack(*sizes),
            struct.pack(f"={T}i", *[code[dt] for dt in types]))


def vc_busbw_factor(coll, nranks: int) -> float:
    return lib().vc_busbw_factor(_code(COLLS, coll), int(nranks))


def vc_status_string(status: int) -> str:
    return lib().vc_status_string(int(status)).decode()


def vc_last_error() -> str:
    return lib().vc_last_error().decode()


def vc_version() -> int:
    return lib().vc_version()


def vc_set_cost_model(policy="hbm", alpha_s: float = 0.0, beta_bytes_per_s: float = 0.0) -> None:
    """Cost model behind algo="auto" (0 keeps the policy's default constant)."""
    check(lib().vc_set_cost_model(_code(COST_POLICIES, policy), float(alpha_s), float(beta_bytes_per_s)))


def vc_get_cost_model():
    p, a, b = ctypes.c_int(0), ctypes.c_double(0), ctypes.c_double(0)
    check(lib().vc_get_cost_model(ctypes.byref(p), ctypes.byref(a), ctypes.byref(b)))
    return {0: "hbm", 1: "link"}[p.value], a.value, b.value


def vc_select_algo(coll, nranks: int, count: int, dtype="f32", root: int = 0):
    """(algorithm name, predicted seconds) that algo="auto" would use."""
    a, t = ctypes.c_int(0), ctypes.c_double(0)
    check(lib().vc_select_algo(_code(COLLS, coll), int(nranks), int(count), _code(DTYPES, dtype), int(root),
                               ctypes.byref(a), ctypes.byref(t)))
    return ALGO_NAMES[a.value], t.value


def vc_set_single_launch(max_step_bytes: int) -> None:
    """Run schedules whose steps each move at most this many bytes in one
    launch (0: never; SINGLE_LAUNCH_ALWAYS: whenever eligible)."""
    check(lib().vc_set_single_launch(int(max_step_bytes)))


def vc_get_single_launch() -> int:
    v = ctypes.c_size_t(0)
    check(lib().vc_get_single_launch(ctypes.byref(v)))
    return v.value


SINGLE_LAUNCH_ALWAYS = (1 << 64) - 1
VC_SINGLE_LAUNCH_DEFAULT = 768 << 10  # VC_SINGLE_LAUNCH_DEFAULT


def vc_set_slice_limit(max_bytes_per_rank: int) -> None:
    """Run eligible schedules (fp32 / int32 AllReduce and the like) whose
    message per rank is at most this many bytes in the sliced form (0: never;
    SLICE_ALWAYS: whenever eligible)."""
    check(lib().vc_set_slice_limit(int(max_bytes_per_rank)))


def vc_get_slice_limit() -> int:
    v = ctypes.c_size_t(0)
    check(lib().vc_get_slice_limit(ctypes.byref(v)))
    return v.value


def vc_set_merge_steps(on: bool) -> None:
    """Run consecutive steps that depend on nothing among themselves as one
    launch (default on).  Clears the plan cache."""
    check(lib().vc_set_merge_steps(int(bool(on))))


def vc_get_merge_steps() -> bool:
    v = ctypes.c_int(0)
    check(lib().vc_get_merge_steps(ctypes.byref(v)))
    return bool(v.value)


SLICE_ALWAYS = (1 << 64) - 1
VC_SLICE_DEFAULT = 16 << 20  # VC_SLICE_LIMIT_DEFAULT


def vc_set_reuse_order(min_step_bytes: int) -> None:
    """Steps after one writing at least this many bytes are ordered for L2 reuse
    (0: every step; REUSE_ORDER_NEVER: none).  Clears the plan cache."""
    check(lib().vc_set_reuse_order(int(min_step_bytes)))


def vc_get_reuse_order() -> int:
    v = ctypes.c_size_t(0)
    check(lib().vc_get_reuse_order(ctypes.byref(v)))
    return v.value


REUSE_ORDER_NEVER = (1 << 64) - 1


def vc_set_copy_pipeline(min_bytes: int) -> None:
    """Copy launches of whole 16-byte groups that write at least this many
    bytes take the bulk-copy pipeline (0: every one; COPY_PIPELINE_NEVER: none)."""
    check(lib().vc_set_copy_pipeline(int(min_bytes)))


def vc_get_copy_pipeline() -> int:
    v = ctypes.c_size_t(0)
    check(lib().vc_get_copy_pipeline(ctypes.byref(v)))
    return v.value


COPY_PIPELINE_NEVER = (1 << 64) - 1


def vc_device_errors(stream=None) -> int:
    """Waits for the stream, then reads and clears the device error word."""
    v = ctypes.c_uint32(0)
    s = None if stream is None else (stream if isinstance(stream, int) else int(stream.cuda_stream))
    check(lib().vc_device_errors(s, ctypes.byref(v)))
    return v.value


def vc_copy_selftest(stream=None) -> int:
    """Error word left by a bulk-copy launch whose first wait is made to run out."""
    v = ctypes.c_uint32(0)
    s = None if stream is None else (stream if isinstance(stream, int) else int(stream.cuda_stream))
    check(lib().vc_copy_selftest(s, ctypes.byref(v)))
    return v.value


def vc_product_selftest(stream=None) -> int:
    """Error word left by a launch in which a wait as the expert products' runs out."""
    v = ctypes.c_uint32(0)
    s = None if stream is None else (stream if isinstance(stream, int) else int(stream.cuda_stream))
    check(lib().vc_product_selftest(s, ctypes.byref(v)))
    return v.value


def vc_trace_enable(on: bool = True) -> None:
    """Start (clearing old records) or stop the launch trace."""
    check(lib().vc_trace_enable(int(bool(on))))


def vc_trace_read(capacity: int = 1 << 20) -> list:
    """Wait for the traced launches and return their records (dicts)."""
    buf = (TraceRecord * capacity)()
    n = ctypes.c_size_t(0)
    check(lib().vc_trace_read(buf, capacity, ctypes.byref(n)))
    out = []
    for r in buf[:n.value]:
        out.append({"coll": r.coll, "algo": r.algo, "step": r.step, "kernel": kernel_name(r.kernel),
                    "bytes": r.bytes, "nops": r.nops, "ms": r.ms})
    return out


def vc_plan_describe(coll, algo, nranks: int, count: int, dtype="f32", root: int = 0, inplace: bool = False,
                     nchunks: int = 0, op="sum"):
    """The step plan the library would run, as (entries, scratch_bytes, n_steps);
    host only, needs no GPU."""
    L = lib()
    need, scratch = ctypes.c_size_t(0), ctypes.c_size_t(0)
    steps = ctypes.c_int(0)
    args = (_code(COLLS, coll), _code(ALGOS, algo), int(nranks), int(count), _code(DTYPES, dtype),
            _code(OPS, op), int(root), int(bool(inplace)), int(nchunks))
    check(L.vc_plan_describe(*args, None, 0, ctypes.byref(need), ctypes.byref(scratch), ctypes.byref(steps)))
    buf = (PlanEntry * max(1, need.value))()
    check(L.vc_plan_describe(*args, buf, need.value, ctypes.byref(need), ctypes.byref(scratch),
                             ctypes.byref(steps)))
    return list(buf[:need.value]), scratch.value, steps.value


FORMS = {0: "steps", 1: "cluster", 2: "sliced"}


def vc_plan_form(coll, algo, nranks: int, count: int, dtype="f32", root: int = 0, inplace: bool = False,
                 nchunks: int = 0, op="sum"):
    """The execution form a call takes under the current settings, on aligned
    buffers: ("sliced" | "cluster" | "steps", launches, host_ranges); host
    only, needs no GPU."""
    L = lib()
    form, launches, hr = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    check(L.vc_plan_form(_code(COLLS, coll), _code(ALGOS, algo), int(nranks), int(count), _code(DTYPES, dtype),
                         _code(OPS, op), int(root), int(bool(inplace)), int(nchunks), ctypes.byref(form),
                         ctypes.byref(launches), ctypes.byref(hr)))
    return FORMS[form.value], launches.value, bool(hr.value)


def vc_plan_exec_order(coll, algo, nranks: int, count: int, dtype="f32", root: int = 0, inplace: bool = False,
                       nchunks: int = 0, op="sum"):
    """The order the library executes the plan in (the L2 reuse order): per
    step, the operations' indices as vc_plan_describe numbers them, their keep
    flags, and whether the step walks its tiles backwards.  Returns
    (order, keep, reverse) with order and keep lists of lists per step; host
    only, needs no GPU."""
    L = lib()
    nops, steps = ctypes.c_size_t(0), ctypes.c_int(0)
    args = (_code(COLLS, coll), _code(ALGOS, algo), int(nranks), int(count), _code(DTYPES, dtype),
            _code(OPS, op), int(root), int(bool(inplace)), int(nchunks))
    check(L.vc_plan_exec_order(*args, None, None, 0, None, 0, ctypes.byref(nops), ctypes.byref(steps)))
    order = (ctypes.c_uint32 * max(1, nops.value))()
    keep = (ctypes.c_uint8 * max(1, nops.value))()
    rev = (ctypes.c_uint8 * max(1, steps.value))()
    check(L.vc_plan_exec_order(*args, order, keep, nops.value, rev, steps.value, ctypes.byref(nops),
                               ctypes.byref(steps)))
    entries, _, _ = vc_plan_describe(coll, algo, nranks, count, dtype, root, inplace, nchunks, op)
    per_step = [0] * steps.value
    for e in entries:
        per_step[e.step] = max(per_step[e.step], e.op + 1)
    out_order, out_keep, k = [], [], 0
    for n in per_step:
        out_order.append(list(order[k:k + n]))
        out_keep.append(list(keep[k:k + n]))
        k += n
    return out_order, out_keep, list(rev[:steps.value])
