"""Python binding of libhoc.so (ctypes).  Argument marshalling only.

Every collective runs in the library's CUDA kernels and copy-engine copies;
this module converts tensors (or raw device pointers) and streams into the
C ABI declared in include/hoc.h and turns result codes into exceptions.  If
the library is missing it raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass, field
from typing import Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhoc.so")

SUCCESS, ERR_INVALID_ARG, ERR_CUDA, ERR_OOM, ERR_NOT_INITIALIZED, ERR_UNSUPPORTED, ERR_TIMEOUT, ERR_NO_DEVICE = range(8)
INT32, FLOAT32, BFLOAT16, UINT8 = 0, 1, 2, 3
SUM = 0
PATH_AUTO, PATH_CE, PATH_TMA, PATH_FUSED = 0, 1, 2, 3
KERNEL_REDUCE, KERNEL_FUSED, KERNEL_TMA = 0, 1, 2
OP_ALLREDUCE, OP_REDUCE_SCATTER, OP_ALLGATHER, OP_ALLTOALL, OP_SENDRECV = range(5)
ITEM_REDUCE, ITEM_FUSED, ITEM_COPY, ITEM_TMA, ITEM_JOIN = range(5)
BUF_SEND, BUF_RECV = 0, 1
MAX_RANKS = 16
PATHS = {"auto": PATH_AUTO, "ce": PATH_CE, "tma": PATH_TMA, "fused": PATH_FUSED}
REDUCE_AUTO, REDUCE_LSU, REDUCE_TMA = 0, 1, 2
ENGINES = {"auto": REDUCE_AUTO, "lsu": REDUCE_LSU, "tma": REDUCE_TMA}


class HocError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str):
        self.code = code
        super().__init__(f"{where}: {error_string(code)} ({code}): {detail}")


class _Config(C.Structure):
    _fields_ = [("path", C.c_int), ("chunk_bytes", C.c_size_t), ("n_copy_streams", C.c_int),
                ("pipeline_depth", C.c_int), ("reduce_max_sms", C.c_int), ("copy_max_sms", C.c_int),
                ("use_graphs", C.c_int), ("a2a_interleave", C.c_int), ("a2a_stage_sync", C.c_int),
                ("ring_order", C.POINTER(C.c_int)), ("reduce_engine", C.c_int)]


class _Stats(C.Structure):
    _fields_ = [("path", C.c_int), ("kernels", C.c_int), ("copies", C.c_int), ("max_ctas", C.c_int),
                ("sms_used", C.c_int), ("graph_replayed", C.c_int), ("bytes_exec", C.c_size_t),
                ("bytes_min", C.c_size_t)]


class _PlanItem(C.Structure):
    _fields_ = [("kind", C.c_int), ("step", C.c_int), ("stream", C.c_int), ("stage", C.c_int),
                ("src_rank", C.c_int), ("dst_rank", C.c_int), ("src_buf", C.c_int), ("dst_buf", C.c_int),
                ("src_off", C.c_size_t), ("dst_off", C.c_size_t), ("bytes", C.c_size_t),
                ("n_waits", C.c_int), ("wait0", C.c_int)]


class _StepTime(C.Structure):
    _fields_ = [("kind", C.c_int), ("stream", C.c_int), ("stage", C.c_int), ("start_ms", C.c_float),
                ("end_ms", C.c_float)]


_lib = None

# Exported symbol -> (restype, argtypes)
_SIGS = {
    "hoc_config_default": (C.c_int, [C.POINTER(_Config)]),
    "hoc_init": (C.c_int, [C.POINTER(C.c_void_p), C.c_int, C.c_int, C.POINTER(_Config)]),
    "hoc_destroy": (C.c_int, [C.c_void_p]),
    "hoc_allreduce": (C.c_int, [C.c_void_p, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.c_size_t, C.c_int,
                                C.c_int, C.c_void_p]),
    "hoc_reduce_scatter": (C.c_int, [C.c_void_p, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.c_size_t,
                                     C.c_int, C.c_int, C.c_void_p]),
    "hoc_allgather": (C.c_int, [C.c_void_p, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.c_size_t, C.c_int,
                                C.c_void_p]),
    "hoc_alltoall": (C.c_int, [C.c_void_p, C.POINTER(C.c_void_p), C.POINTER(C.c_size_t), C.POINTER(C.c_size_t),
                               C.POINTER(C.c_void_p), C.POINTER(C.c_size_t), C.c_size_t, C.c_int, C.c_void_p]),
    "hoc_sendrecv": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_size_t, C.c_int,
                               C.c_void_p]),
    "hoc_sendrecv_async": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_size_t, C.c_int,
                                     C.c_void_p, C.c_void_p]),
    "hoc_wait": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int]),
    "hoc_last_stats": (C.c_int, [C.c_void_p, C.POINTER(_Stats)]),
    "hoc_profile_enable": (C.c_int, [C.c_void_p, C.c_int]),
    "hoc_profile_read": (C.c_int, [C.c_void_p, C.c_int, C.POINTER(C.c_int), C.POINTER(C.c_double)]),
    "hoc_error_string": (C.c_char_p, [C.c_int]),
    "hoc_last_error_detail": (C.c_char_p, []),
    "hoc_plan_query": (C.c_int, [C.c_int, C.POINTER(_Config), C.c_int, C.c_size_t, C.c_int, C.POINTER(C.c_size_t),
                                 C.POINTER(_PlanItem), C.c_size_t, C.POINTER(C.c_size_t)]),
    "hoc_probe_launch": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p]),
    "hoc_xor16_launch": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_uint16]),
    "hoc_device_sm_count": (C.c_int, [C.c_int, C.POINTER(C.c_int)]),
    "hoc_tma_moves_noalloc": (C.c_int, [C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.POINTER(C.c_size_t),
                                        C.c_int, C.c_int, C.c_void_p, C.c_int]),
}
NOALLOC_MAX_MOVES = 192
_SIGS["hoc_alltoall_device_counts"] = (C.c_int, [C.c_void_p, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p),
                                                 C.c_void_p, C.c_int, C.POINTER(C.c_size_t), C.POINTER(C.c_size_t),
                                                 C.c_int, C.c_void_p])
_SIGS["hoc_ep_pack"] = (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p,
                                  C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p])
_SIGS["hoc_ep_pack_workspace"] = (C.c_int, [C.c_int, C.c_int, C.c_int, C.POINTER(C.c_size_t)])
_SIGS["hoc_ep_combine"] = (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p,
                                     C.c_void_p])
_SIGS["hoc_ep_dispatch_fused"] = (C.c_int, [C.c_int, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.c_int, C.c_int,
                                            C.c_int, C.c_int, C.POINTER(C.c_void_p), C.POINTER(C.c_size_t),
                                            C.POINTER(C.c_void_p), C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p,
                                            C.c_void_p])
_SIGS["hoc_ep_combine_fused"] = (C.c_int, [C.c_int, C.POINTER(C.c_void_p), C.POINTER(C.c_size_t),
                                           C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.c_void_p,
                                           C.POINTER(C.c_void_p), C.c_int, C.c_int, C.c_int, C.c_int,
                                           C.POINTER(C.c_void_p), C.c_void_p, C.c_void_p])
_SIGS["hoc_ep_pack_all"] = _SIGS["hoc_ep_dispatch_fused"]
_SIGS["hoc_ep_combine_all"] = (C.c_int, [C.c_int, C.POINTER(C.c_void_p), C.POINTER(C.c_size_t), C.POINTER(C.c_void_p),
                                         C.POINTER(C.c_void_p), C.c_int, C.c_int, C.c_int, C.POINTER(C.c_void_p),
                                         C.c_void_p, C.c_void_p])
_SIGS["hoc_ep_combine_grad"] = (C.c_int, [C.c_int, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.POINTER(C.c_size_t),
                                          C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.c_void_p,
                                          C.POINTER(C.c_void_p), C.c_int, C.c_int, C.c_int, C.c_int,
                                          C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.c_void_p, C.c_void_p])
_SIGS["hoc_ep_combine_grad_all"] = (C.c_int, [C.c_int, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p),
                                              C.POINTER(C.c_size_t), C.POINTER(C.c_void_p), C.POINTER(C.c_void_p),
                                              C.c_int, C.c_int, C.c_int, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p),
                                              C.c_void_p, C.c_void_p])


class _RowGroups(C.Structure):
    _fields_ = [("nranks", C.c_int), ("experts", C.c_int), ("sources", C.c_int), ("seg", C.c_void_p),
                ("capacity", C.POINTER(C.c_size_t))]


_SIGS["hoc_ep_segments"] = (C.c_int, [C.c_int, C.POINTER(C.c_void_p), C.c_int, C.c_int, C.c_int, C.c_void_p,
                                      C.c_void_p])
_SIGS["hoc_expert_mm"] = (C.c_int, [C.POINTER(_RowGroups), C.POINTER(C.c_void_p), C.POINTER(C.c_void_p),
                                    C.POINTER(C.c_void_p), C.c_int, C.c_int, C.c_int, C.POINTER(C.c_void_p),
                                    C.POINTER(C.c_void_p), C.c_void_p, C.c_void_p])
_SIGS["hoc_expert_mm_dgrad"] = (C.c_int, [C.POINTER(_RowGroups), C.POINTER(C.c_void_p), C.POINTER(C.c_void_p),
                                          C.c_int, C.c_int, C.c_int, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p),
                                          C.c_void_p, C.c_void_p])
_SIGS["hoc_expert_mm_wgrad"] = (C.c_int, [C.POINTER(_RowGroups), C.POINTER(C.c_void_p), C.POINTER(C.c_void_p),
                                          C.c_int, C.c_int, C.c_int, C.c_int, C.POINTER(C.c_void_p),
                                          C.POINTER(C.c_void_p), C.c_void_p, C.c_void_p])
_SIGS["hoc_linear"] = (C.c_int, [C.c_int, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t,
                                 C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p,
                                 C.c_void_p])
_SIGS["hoc_linear_dgrad"] = (C.c_int, [C.c_int, C.c_void_p, C.c_size_t, C.c_void_p, C.c_int, C.c_int, C.c_int,
                                       C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p])
_SIGS["hoc_linear_wgrad"] = (C.c_int, [C.c_int, C.c_void_p, C.c_size_t, C.c_void_p, C.c_size_t, C.c_int, C.c_int,
                                       C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p])
_SIGS["hoc_act_grad"] = (C.c_int, [C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p])
_SIGS["hoc_layer_trim"] = (C.c_int, [C.c_size_t])
_SIGS["hoc_tensor_list_create"] = (C.c_int, [C.POINTER(C.c_void_p), C.c_int, C.POINTER(C.c_void_p),
                                             C.POINTER(C.c_size_t), C.c_int])
_SIGS["hoc_tensor_list_destroy"] = (C.c_int, [C.c_void_p])
_SIGS["hoc_grad_workspace"] = (C.c_int, [C.c_void_p, C.POINTER(C.c_size_t)])
_SIGS["hoc_grad_norm"] = (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p])
_SIGS["hoc_grad_clip"] = (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(C.c_float), C.c_void_p, C.c_void_p, C.c_size_t,
                                    C.c_void_p])
_ROWS = [C.c_void_p, C.c_size_t]  # rows and their stride
_SIGS["hoc_wire8_row"] = (C.c_int, [C.c_int, C.POINTER(C.c_size_t), C.POINTER(C.c_size_t)])
_SIGS["hoc_rms_norm"] = (C.c_int, [C.c_int, C.c_int, C.c_int] + 2 * _ROWS + [C.c_void_p, C.c_int, C.POINTER(C.c_float)] + 2 * _ROWS
                         + [C.c_void_p, C.c_void_p])
_SIGS["hoc_rms_norm_workspace"] = (C.c_int, [C.c_int, C.c_int, C.POINTER(C.c_size_t)])
_SIGS["hoc_rms_norm_grad"] = (C.c_int, [C.c_int, C.c_int, C.c_int] + 3 * _ROWS + [C.c_void_p, C.c_int, C.POINTER(C.c_float)]
                              + 2 * _ROWS + [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_size_t, C.c_void_p])
_SIGS["hoc_expert_widen"] = (C.c_int, [C.POINTER(_RowGroups), C.POINTER(C.c_void_p), C.c_int, C.POINTER(C.c_void_p),
                                       C.c_void_p, C.c_void_p])
_SIGS["hoc_ep_route"] = (C.c_int, [C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_size_t, C.c_int, C.c_void_p,
                                   C.c_int, C.c_int, C.c_int, C.POINTER(C.c_float), C.c_void_p, C.c_void_p, C.c_void_p])
_SIGS["hoc_ep_route_grad"] = (C.c_int, [C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_size_t, C.c_int, C.c_int,
                                        C.POINTER(C.c_float), C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p])
_SIGS["hoc_dropout"] = (C.c_int, [C.c_size_t, C.c_int, C.c_int] + 2 * _ROWS + [C.POINTER(C.c_double), C.c_void_p] + _ROWS + [C.c_void_p])
_SIGS["hoc_allreduce_host"] = (C.c_int, [C.c_void_p, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.c_size_t,
                                         C.c_int, C.c_int, C.c_void_p])
_SIGS["hoc_proxy_status"] = (C.c_int, [C.c_void_p, C.POINTER(C.c_uint64), C.POINTER(C.c_uint64),
                                       C.POINTER(C.c_int)])
_SIGS["hoc_profile_stream_finish"] = (C.c_int, [C.c_void_p, C.POINTER(C.c_float), C.c_int, C.POINTER(C.c_int)])
_SIGS["hoc_profile_timeline"] = (C.c_int, [C.c_void_p, C.POINTER(_StepTime), C.c_size_t, C.POINTER(C.c_size_t)])
_SIGS["hoc_topo_schedule"] = (C.c_int, [C.c_int, C.POINTER(C.c_int), C.POINTER(C.c_int), C.POINTER(C.c_uint64),
                                        C.c_uint64, C.c_uint64, C.POINTER(C.c_uint64), C.POINTER(C.c_uint64),
                                        C.POINTER(C.c_double), C.c_int, C.POINTER(C.c_int),
                                        C.POINTER(C.c_double)])


def lib():
    """Load libhoc.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m collective_communication_schedules_gb300.build`")
        h = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


def error_string(code: int) -> str:
    return lib().hoc_error_string(code).decode()


def last_error_detail() -> str:
    return lib().hoc_last_error_detail().decode()


def _check(code: int, where: str):
    if code != SUCCESS:
        raise HocError(code, where, last_error_detail())


# ----------------------------------------------------------------- marshalling
def _dtype_code(x) -> int:
    import torch
    m = {torch.int32: INT32, torch.float32: FLOAT32, torch.bfloat16: BFLOAT16, torch.uint8: UINT8}
    if x.dtype not in m:
        raise TypeError(f"unsupported tensor dtype {x.dtype}")
    return m[x.dtype]


DTYPE_BYTES = {INT32: 4, FLOAT32: 4, BFLOAT16: 2, UINT8: 1}


def _ptr(x, nbytes: int = 0, what: str = "buffer", device: bool = True) -> int:
    """Address of `x`.  A tensor must be contiguous, hold at least `nbytes`
    bytes (the span the call touches) and live on the GPU (`device`) or the
    host; an int is taken as a raw address, unchecked."""
    if isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    have = x.numel() * x.element_size()
    if have < nbytes:
        raise ValueError(f"{what}: tensor holds {have} bytes, the call touches {nbytes}")
    if device and not x.is_cuda:
        raise ValueError(f"{what}: rank buffers must be CUDA tensors")
    if not device and x.is_cuda:
        raise ValueError(f"{what}: host buffers must be CPU tensors")
    return x.data_ptr()


def _ptr_array(xs: Sequence, nbytes=0, what: str = "buffer", device: bool = True) -> C.Array:
    """Addresses of the rank buffers; `nbytes` is one span for all ranks or a list, one per rank."""
    one = not isinstance(nbytes, (list, tuple))
    if not one and len(nbytes) != len(xs):
        raise ValueError(f"{what}: expected {len(nbytes)} rank buffers, got {len(xs)}")
    out = []
    for r, x in enumerate(xs):
        n = nbytes if one else nbytes[r]
        # the checks of _ptr, which names the buffer if one fails
        if isinstance(x, int) or x.numel() * x.element_size() < n or x.is_cuda != device or not x.is_contiguous():
            out.append(_ptr(x, n, f"{what}[{r}]", device))
        else:
            out.append(x.data_ptr())
    return (C.c_void_p * len(out))(*out)


def _stream(stream) -> int:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the same handle without building a Stream object
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _sizes(vals, n) -> Optional[C.Array]:
    if vals is None:
        return None
    flat = [int(v) for row in vals for v in (row if hasattr(row, "__len__") else [row])]
    if len(flat) != n:
        raise ValueError(f"expected {n} values, got {len(flat)}")
    return (C.c_size_t * n)(*flat)


@dataclass
class Config:
    path: str = "auto"
    chunk_bytes: int = 0  # 0: picked by the scheduler (allreduce: by move path and rank count)
    n_copy_streams: int = 0  # 0: the scheduler picks per call (8 queues for copies of at most 2 MiB, else 4)
    pipeline_depth: int = 0
    reduce_max_sms: int = 0
    copy_max_sms: int = 0
    use_graphs: bool = True
    a2a_interleave: bool = True
    a2a_stage_sync: bool = False
    ring_order: Optional[Sequence[int]] = None
    reduce_engine: str = "auto"
    _keep: list = field(default_factory=list, repr=False)

    def to_c(self) -> _Config:
        c = _Config()
        c.path = PATHS[self.path] if isinstance(self.path, str) else int(self.path)
        c.chunk_bytes = int(self.chunk_bytes)
        c.n_copy_streams = int(self.n_copy_streams)
        c.pipeline_depth = int(self.pipeline_depth)
        c.reduce_max_sms = int(self.reduce_max_sms)
        c.copy_max_sms = int(self.copy_max_sms)
        c.use_graphs = int(bool(self.use_graphs))
        c.a2a_interleave = int(bool(self.a2a_interleave))
        c.a2a_stage_sync = int(bool(self.a2a_stage_sync))
        c.reduce_engine = ENGINES[self.reduce_engine] if isinstance(self.reduce_engine, str) else int(self.reduce_engine)
        if self.ring_order is not None:
            arr = (C.c_int * len(self.ring_order))(*[int(v) for v in self.ring_order])
            self._keep = [arr]
            c.ring_order = C.cast(arr, C.POINTER(C.c_int))
        else:
            c.ring_order = None
        return c


class Comm:
    """A communicator over `nranks` simulated ranks on one CUDA device."""

    def __init__(self, nranks: int, device: int = 0, config: Optional[Config] = None):
        self.k = nranks
        self.device = device
        self.config = config or Config()
        h = C.c_void_p()
        cfg = self.config.to_c()
        _check(lib().hoc_init(C.byref(h), nranks, device, C.byref(cfg)), "hoc_init")
        self._h = h

    def _ranks(self, xs, nbytes, what, device=True):
        if len(xs) != self.k:
            raise ValueError(f"{what}: expected {self.k} rank buffers, got {len(xs)}")
        return _ptr_array(xs, nbytes, what, device)

    def close(self):
        if getattr(self, "_h", None):
            _check(lib().hoc_destroy(self._h), "hoc_destroy")
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------ collectives
    def allreduce(self, send, recv, count=None, dtype=None, stream=None):
        count = send[0].numel() if count is None else count
        dtype = _dtype_code(send[0]) if dtype is None else dtype
        n = int(count) * DTYPE_BYTES[dtype]
        _check(lib().hoc_allreduce(self._h, self._ranks(send, n, "send"), self._ranks(recv, n, "recv"), count, dtype,
                                   SUM, _stream(stream)), "hoc_allreduce")

    def allreduce_host(self, h_send, h_recv, count=None, dtype=None, stream=None):
        """AllReduce of host (CPU) tensors: one fused launch on host memory the GPU can address (path AUTO/FUSED),
        else the copy-engine pipeline through device staging slots (path CE/TMA)."""
        count = h_send[0].numel() if count is None else count
        dtype = _dtype_code(h_send[0]) if dtype is None else dtype
        n = int(count) * DTYPE_BYTES[dtype]
        _check(lib().hoc_allreduce_host(self._h, self._ranks(h_send, n, "h_send", device=False),
                                        self._ranks(h_recv, n, "h_recv", device=False), count, dtype, SUM,
                                        _stream(stream)), "hoc_allreduce_host")

    def reduce_scatter(self, send, recv, recvcount=None, dtype=None, stream=None):
        recvcount = recv[0].numel() if recvcount is None else recvcount
        dtype = _dtype_code(send[0]) if dtype is None else dtype
        n = int(recvcount) * DTYPE_BYTES[dtype]
        _check(lib().hoc_reduce_scatter(self._h, self._ranks(send, self.k * n, "send"), self._ranks(recv, n, "recv"),
                                        recvcount, dtype, SUM, _stream(stream)), "hoc_reduce_scatter")

    def allgather(self, send, recv, sendcount=None, dtype=None, stream=None):
        sendcount = send[0].numel() if sendcount is None else sendcount
        dtype = _dtype_code(send[0]) if dtype is None else dtype
        n = int(sendcount) * DTYPE_BYTES[dtype]
        _check(lib().hoc_allgather(self._h, self._ranks(send, n, "send"), self._ranks(recv, self.k * n, "recv"),
                                   sendcount, dtype, _stream(stream)), "hoc_allgather")

    def alltoall(self, send, recv, sendcounts=None, sdispls=None, rdispls=None, count=0, dtype=None,
                 stream=None):
        """sendcounts: k x k (row = source) in elements; None = uniform `count`."""
        dtype = _dtype_code(send[0]) if dtype is None else dtype
        k, kk, b = self.k, self.k * self.k, DTYPE_BYTES[dtype]
        cnt = _sizes(sendcounts, kk)
        sd, rd = _sizes(sdispls, kk), _sizes(rdispls, kk)
        c = [cnt[i] for i in range(kk)] if cnt is not None else [int(count)] * kk
        # the span of each rank's buffer: the end of its furthest segment
        s_end = [max((sd[a * k + d] if sd is not None else sum(c[a * k: a * k + d])) + c[a * k + d]
                     for d in range(k)) * b for a in range(k)]
        r_end = [max((rd[d * k + a] if rd is not None else sum(c[x * k + d] for x in range(a))) + c[a * k + d]
                     for a in range(k)) * b for d in range(k)]
        _check(lib().hoc_alltoall(self._h, self._ranks(send, s_end, "send"), cnt, sd,
                                  self._ranks(recv, r_end, "recv"), rd, int(count), dtype, _stream(stream)),
               "hoc_alltoall")

    def sendrecv(self, src_rank, send, dst_rank, recv, count=None, dtype=None, stream=None):
        count = send.numel() if count is None else count
        dtype = _dtype_code(send) if dtype is None else dtype
        n = int(count) * DTYPE_BYTES[dtype]
        _check(lib().hoc_sendrecv(self._h, int(src_rank), _ptr(send, n, "send"), int(dst_rank), _ptr(recv, n, "recv"),
                                  count, dtype, _stream(stream)), "hoc_sendrecv")

    def sendrecv_async(self, src_rank, send, dst_rank, recv, count=None, dtype=None, stream=None, done=None):
        """Send/recv completed by an event, not by `stream`: returns the torch.cuda.Event (`done`, or a new
        one) that the consumer waits on; later work on `stream` does not wait for the copy."""
        import torch
        count = send.numel() if count is None else count
        dtype = _dtype_code(send) if dtype is None else dtype
        if done is None:
            done = torch.cuda.Event()
        if not done.cuda_event:
            done.record(torch.cuda.current_stream() if stream is None else stream)   # creates the CUDA event
        n = int(count) * DTYPE_BYTES[dtype]
        _check(lib().hoc_sendrecv_async(self._h, int(src_rank), _ptr(send, n, "send"), int(dst_rank),
                                        _ptr(recv, n, "recv"), count, dtype, _stream(stream),
                                        C.c_void_p(done.cuda_event)), "hoc_sendrecv_async")
        return done

    def alltoall_device_counts(self, send, recv, d_counts, recv_capacity, dtype=None, stream=None,
                               transpose: bool = False, send_capacity=None):
        """All-to-all(v) whose k x k counts (uint64/int64, elements, row = source) live on the device.

        The counts reach a host proxy through the stream-memory-operation
        handshake; the call returns without waiting (see include/hoc_proxy.h).
        send_capacity defaults to the elements each send tensor holds."""
        dtype = _dtype_code(send[0]) if dtype is None else dtype
        caps = [int(v) for v in recv_capacity]
        if len(caps) != self.k:
            raise ValueError(f"recv_capacity: expected {self.k} values, got {len(caps)}")
        if send_capacity is None:
            scaps = [t.numel() * t.element_size() // DTYPE_BYTES[dtype] if not isinstance(t, int) else None
                     for t in send]
            if any(v is None for v in scaps):
                raise ValueError("send_capacity is needed when send buffers are raw addresses")
        else:
            scaps = [int(v) for v in send_capacity]
        if len(scaps) != self.k:
            raise ValueError(f"send_capacity: expected {self.k} values, got {len(scaps)}")
        cap = (C.c_size_t * self.k)(*caps)
        scap = (C.c_size_t * self.k)(*scaps)
        _check(lib().hoc_alltoall_device_counts(self._h,
                                                self._ranks(send, [v * DTYPE_BYTES[dtype] for v in scaps], "send"),
                                                self._ranks(recv, [v * DTYPE_BYTES[dtype] for v in caps], "recv"),
                                                _ptr(d_counts, 8 * self.k * self.k, "d_counts"),
                                                int(bool(transpose)), scap, cap, dtype, _stream(stream)),
               "hoc_alltoall_device_counts")

    def proxy_status(self) -> dict:
        done = C.c_uint64()
        rel = C.c_uint64()
        err = C.c_int()
        _check(lib().hoc_proxy_status(self._h, C.byref(done), C.byref(rel), C.byref(err)), "hoc_proxy_status")
        return {"completed": done.value, "released_on_error": rel.value, "first_error": err.value}

    # ------------------------------------------------------------- control
    def wait(self, stream=None, timeout_ms: int = 60000):
        _check(lib().hoc_wait(self._h, _stream(stream), int(timeout_ms)), "hoc_wait")

    def last_stats(self) -> dict:
        s = _Stats()
        _check(lib().hoc_last_stats(self._h, C.byref(s)), "hoc_last_stats")
        return {name: getattr(s, name) for name, _ in _Stats._fields_}

    def profile_enable(self, on: bool = True):
        _check(lib().hoc_profile_enable(self._h, int(bool(on))), "hoc_profile_enable")

    def profile_read(self, kernel: int):
        n = C.c_int()
        ms = C.c_double()
        _check(lib().hoc_profile_read(self._h, int(kernel), C.byref(n), C.byref(ms)), "hoc_profile_read")
        return n.value, ms.value

    def profile_stream_finish(self) -> list:
        """Finish time (ms from the fork) of each copy stream of the last call issued while profiling."""
        buf = (C.c_float * 16)()
        n = C.c_int()
        _check(lib().hoc_profile_stream_finish(self._h, buf, 16, C.byref(n)), "hoc_profile_stream_finish")
        return [buf[i] for i in range(min(n.value, 16))]

    def profile_timeline(self) -> list:
        """Per-step (kind, stream, stage, start_ms, end_ms) of the last call issued while profiling."""
        n = C.c_size_t()
        _check(lib().hoc_profile_timeline(self._h, None, 0, C.byref(n)), "hoc_profile_timeline")
        buf = (_StepTime * max(1, n.value))()
        _check(lib().hoc_profile_timeline(self._h, buf, n.value, C.byref(n)), "hoc_profile_timeline")
        kinds = {ITEM_REDUCE: "reduce", ITEM_FUSED: "fused", ITEM_COPY: "copy", ITEM_TMA: "tma"}
        return [dict(kind=kinds.get(b.kind, b.kind), stream=b.stream, stage=b.stage, start_ms=b.start_ms,
                     end_ms=b.end_ms) for b in buf[: n.value]]


# ---------------------------------------------------------------- workload
PROBE_WHOLE_SM, PROBE_PDL = 1, 2


def probe_launch(ctas: int, threads: int, iters: int, sink=None, stream=None, whole_sm: bool = False,
                 pdl: bool = False):
    flags = (PROBE_WHOLE_SM if whole_sm else 0) | (PROBE_PDL if pdl else 0)
    _check(lib().hoc_probe_launch(_stream(stream), int(ctas), int(threads), int(iters), flags,
                                  None if sink is None else _ptr(sink, 12, "sink")), "hoc_probe_launch")


def xor16(src, dst, n: int, key: int, stream=None):
    _check(lib().hoc_xor16_launch(_stream(stream), _ptr(src, 2 * int(n), "src"), _ptr(dst, 2 * int(n), "dst"), int(n),
                                  int(key) & 0xFFFF), "hoc_xor16_launch")


def tma_moves_noalloc(src, dst, nbytes, max_ctas: int = 0, stream=None, wait: bool = True):
    """Byte moves src[i] -> dst[i] on the TMA bulk-copy kernel with no device
    allocation (for callers that cannot call cudaMalloc); see include/hoc.h."""
    n = len(nbytes)
    if len(src) != n or len(dst) != n:
        raise ValueError("src, dst and nbytes must have the same length")
    spans = [int(b) for b in nbytes]
    sizes = (C.c_size_t * max(1, n))(*spans)
    _check(lib().hoc_tma_moves_noalloc(_ptr_array(src, spans, "src"), _ptr_array(dst, spans, "dst"), sizes, n,
                                       int(max_ctas), _stream(stream), int(bool(wait))), "hoc_tma_moves_noalloc")


def topo_schedule(C_matrix, node_of, sym, bw_nvlink: int, bw_rdma: int):
    """Two-domain stage schedule (host only): returns (T, stages, taus, total)."""
    G = len(node_of)
    flat = [int(v) for row in C_matrix for v in row]
    if len(flat) != G * G:
        raise ValueError("C must be G x G")
    cm = (C.c_uint64 * (G * G))(*flat)
    no = (C.c_int * G)(*[int(v) for v in node_of])
    sy = (C.c_int * G)(*[int(v) for v in sym])
    n = C.c_int()
    tot = C.c_double()
    _check(lib().hoc_topo_schedule(G, no, sy, cm, int(bw_nvlink), int(bw_rdma), None, None, None, 0, C.byref(n),
                                   C.byref(tot)), "hoc_topo_schedule")
    T = (C.c_uint64 * (G * G))()
    st = (C.c_uint64 * max(1, n.value * G * G))()
    ta = (C.c_double * max(1, n.value))()
    _check(lib().hoc_topo_schedule(G, no, sy, cm, int(bw_nvlink), int(bw_rdma), T, st, ta, n.value, C.byref(n),
                                   C.byref(tot)), "hoc_topo_schedule")
    Tm = [[T[u * G + v] for v in range(G)] for u in range(G)]
    stages = [[[st[s * G * G + u * G + v] for v in range(G)] for u in range(G)] for s in range(n.value)]
    return Tm, stages, [ta[s] for s in range(n.value)], tot.value


_MOST = (1 << 31) - 1  # what an int of the library holds; ctypes would keep the low 32 bits of more


def _fits(**counts):
    """Refuses counts that an int of the library does not hold."""
    for what, n in counts.items():
        if not -_MOST <= n <= _MOST:
            raise ValueError(f"{what}: {n} is more than 2^31 - 1")


def _int(n) -> int:
    """n, which an int of the library has to hold."""
    n = int(n)
    if not -_MOST <= n <= _MOST:
        raise ValueError(f"a count of {n} is more than 2^31 - 1")
    return n


def ep_pack_workspace(tokens: int, topk: int, experts: int) -> int:
    """int32 entries of scratch that ep_pack needs for this shape."""
    n = C.c_size_t()
    _check(lib().hoc_ep_pack_workspace(_int(tokens), _int(topk), _int(experts), C.byref(n)), "hoc_ep_pack_workspace")
    return n.value


def ep_pack(expert_ids, x, experts: int, nranks: int, send, perm, pos_of, dst_counts, workspace, stream=None):
    """Dispatch-side pack of one source rank (device tensors; see include/hoc_ep.h)."""
    tokens, hidden = x.shape
    topk = expert_ids.numel() // tokens if tokens else 1
    n = tokens * topk
    _check(lib().hoc_ep_pack(_ptr(expert_ids, 4 * n, "expert_ids"), _ptr(x, 2 * tokens * hidden, "x"), _int(tokens),
                             _int(topk), _int(hidden), _int(experts), _int(nranks), _ptr(send, 2 * n * hidden, "send"),
                             _ptr(perm, 4 * n, "perm"), _ptr(pos_of, 4 * n, "pos_of"),
                             _ptr(dst_counts, 8 * int(nranks), "dst_counts"), _ptr(workspace, 0, "workspace"),
                             int(workspace.numel()), _stream(stream)), "hoc_ep_pack")


def ep_combine(rows, pos_of, weights, tokens: int, topk: int, hidden: int, y, stream=None):
    """Gate-weighted top-k combine of one source rank (see include/hoc_ep.h)."""
    n = int(tokens) * int(topk)
    _check(lib().hoc_ep_combine(_ptr(rows, 2 * n * int(hidden), "rows"), _ptr(pos_of, 4 * n, "pos_of"),
                                _ptr(weights, 4 * n, "weights"), _int(tokens), _int(topk), _int(hidden),
                                _ptr(y, 2 * int(tokens) * int(hidden), "y"), _stream(stream)), "hoc_ep_combine")


def _ep_scatter_call(fn_name, expert_ids, x, experts, out, out_capacity, pos_of, counts, workspace, status, stream):
    k = len(x)
    tokens, hidden = x[0].shape
    topk = expert_ids[0].numel() // tokens if tokens else 1
    n = tokens * topk
    caps = [int(v) for v in out_capacity]
    if len(caps) != k or len(expert_ids) != k or len(out) != k or len(pos_of) != k:
        raise ValueError(f"expected {k} per-rank tensors and capacities")
    cap = (C.c_size_t * k)(*caps)
    _check(getattr(lib(), fn_name)(k, _ptr_array(expert_ids, 4 * n, "expert_ids"),
                                   _ptr_array(x, 2 * tokens * hidden, "x"), _int(tokens), _int(topk), _int(hidden),
                                   _int(experts), _ptr_array(out, [2 * c for c in caps], "out"), cap,
                                   _ptr_array(pos_of, 4 * n, "pos_of"), _ptr(counts, 8 * k * k, "counts"),
                                   _ptr(workspace, 0, "workspace"), int(workspace.numel()),
                                   _ptr(status, 4, "status"), _stream(stream)), fn_name)


def ep_pack_all(expert_ids, x, experts: int, send, send_capacity, pos_of, counts, workspace, status, stream=None):
    """hoc_ep_pack for every source rank in one pass (see include/hoc_ep.h): lists of k device tensors."""
    _ep_scatter_call("hoc_ep_pack_all", expert_ids, x, experts, send, send_capacity, pos_of, counts, workspace,
                     status, stream)


def ep_combine_all(rows, rows_capacity, pos_of, weights, tokens: int, topk: int, hidden: int, y, status,
                   stream=None):
    """hoc_ep_combine for every source rank in one pass (see include/hoc_ep.h)."""
    k = len(rows)
    n = int(tokens) * int(topk)
    caps = [int(v) for v in rows_capacity]
    if len(caps) != k or len(pos_of) != k or len(weights) != k or len(y) != k:
        raise ValueError(f"expected {k} per-rank tensors and capacities")
    cap = (C.c_size_t * k)(*caps)
    _check(lib().hoc_ep_combine_all(k, _ptr_array(rows, [2 * c for c in caps], "rows"), cap,
                                    _ptr_array(pos_of, 4 * n, "pos_of"), _ptr_array(weights, 4 * n, "weights"),
                                    _int(tokens), _int(topk), _int(hidden),
                                    _ptr_array(y, 2 * int(tokens) * int(hidden), "y"), _ptr(status, 4, "status"),
                                    _stream(stream)), "hoc_ep_combine_all")


def ep_dispatch_fused(expert_ids, x, experts: int, recv, recv_capacity, pos_of, counts, workspace, status,
                      stream=None):
    """Dispatch of every source rank straight into the receive buffers (see include/hoc_ep.h).

    Lists of k device tensors: expert_ids [tokens*topk] int32, x [tokens, hidden] bf16, recv (room for
    recv_capacity[d] elements each), pos_of [tokens*topk] int32; counts: [k, k] int64; status: int32."""
    k = len(x)
    tokens, hidden = x[0].shape
    topk = expert_ids[0].numel() // tokens if tokens else 1
    n = tokens * topk
    caps = [int(v) for v in recv_capacity]
    if len(caps) != k or len(expert_ids) != k or len(recv) != k or len(pos_of) != k:
        raise ValueError(f"expected {k} per-rank tensors and capacities")
    cap = (C.c_size_t * k)(*caps)
    _check(lib().hoc_ep_dispatch_fused(k, _ptr_array(expert_ids, 4 * n, "expert_ids"),
                                       _ptr_array(x, 2 * tokens * hidden, "x"), _int(tokens), _int(topk), _int(hidden),
                                       _int(experts), _ptr_array(recv, [2 * c for c in caps], "recv"), cap,
                                       _ptr_array(pos_of, 4 * n, "pos_of"), _ptr(counts, 8 * k * k, "counts"),
                                       _ptr(workspace, 0, "workspace"), int(workspace.numel()),
                                       _ptr(status, 4, "status"), _stream(stream)), "hoc_ep_dispatch_fused")


def ep_combine_fused(rows, rows_capacity, expert_ids, pos_of, counts, weights, tokens: int, topk: int, hidden: int,
                     experts: int, y, status, stream=None):
    """Combine of every source rank reading the expert ranks' rows in place (see include/hoc_ep.h)."""
    k = len(rows)
    n = int(tokens) * int(topk)
    caps = [int(v) for v in rows_capacity]
    if len(caps) != k or len(expert_ids) != k or len(pos_of) != k or len(weights) != k or len(y) != k:
        raise ValueError(f"expected {k} per-rank tensors and capacities")
    cap = (C.c_size_t * k)(*caps)
    _check(lib().hoc_ep_combine_fused(k, _ptr_array(rows, [2 * c for c in caps], "rows"), cap,
                                      _ptr_array(expert_ids, 4 * n, "expert_ids"), _ptr_array(pos_of, 4 * n, "pos_of"),
                                      _ptr(counts, 8 * k * k, "counts"), _ptr_array(weights, 4 * n, "weights"),
                                      _int(tokens), _int(topk), _int(hidden), _int(experts),
                                      _ptr_array(y, 2 * int(tokens) * int(hidden), "y"), _ptr(status, 4, "status"),
                                      _stream(stream)), "hoc_ep_combine_fused")


def _combine_grad_args(dy, rows, rows_capacity, pos_of, weights, tokens, topk, hidden, drows, dweights):
    k = len(rows)
    n = int(tokens) * int(topk)
    caps = [int(v) for v in rows_capacity]
    if any(len(v) != k for v in (dy, caps, pos_of, weights, drows, dweights)):
        raise ValueError(f"expected {k} per-rank tensors and capacities")
    span = [2 * c for c in caps]
    return (k, n, (C.c_size_t * k)(*caps), _ptr_array(dy, 2 * int(tokens) * int(hidden), "dy"),
            _ptr_array(rows, span, "rows"), _ptr_array(pos_of, 4 * n, "pos_of"), _ptr_array(weights, 4 * n, "weights"),
            _ptr_array(drows, span, "drows"), _ptr_array(dweights, 4 * n, "dweights"))


def ep_combine_grad(dy, rows, rows_capacity, expert_ids, pos_of, counts, weights, tokens: int, topk: int, hidden: int,
                    experts: int, drows, dweights, status, stream=None):
    """Gradient of ep_combine_fused for the rows and the gate weights (see include/hoc_ep.h)."""
    k, n, cap, dyp, rp, pp, wp, dp, dwp = _combine_grad_args(dy, rows, rows_capacity, pos_of, weights, tokens, topk,
                                                             hidden, drows, dweights)
    if len(expert_ids) != k:
        raise ValueError(f"expected {k} per-rank tensors and capacities")
    _check(lib().hoc_ep_combine_grad(k, dyp, rp, cap, _ptr_array(expert_ids, 4 * n, "expert_ids"), pp,
                                     _ptr(counts, 8 * k * k, "counts"), wp, _int(tokens), _int(topk), _int(hidden),
                                     _int(experts), dp, dwp, _ptr(status, 4, "status"), _stream(stream)),
           "hoc_ep_combine_grad")


def ep_combine_grad_all(dy, rows, rows_capacity, pos_of, weights, tokens: int, topk: int, hidden: int, drows, dweights,
                        status, stream=None):
    """Gradient of ep_combine_all: rows and their gradients in each source's packed order."""
    k, _, cap, dyp, rp, pp, wp, dp, dwp = _combine_grad_args(dy, rows, rows_capacity, pos_of, weights, tokens, topk,
                                                             hidden, drows, dweights)
    _check(lib().hoc_ep_combine_grad_all(k, dyp, rp, cap, pp, wp, _int(tokens), _int(topk), _int(hidden), dp, dwp,
                                         _ptr(status, 4, "status"), _stream(stream)), "hoc_ep_combine_grad_all")


# ------------------------------------------------------- expert and linear layers
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4}


def _act(act) -> int:
    if act not in ACTS:
        raise ValueError(f"act is one of {', '.join(ACTS)}, not {act!r}")
    return ACTS[act]


_TORCH = {}  # torch dtypes by name, once torch is imported


def _dt(name: str):
    if not _TORCH:
        import torch
        _TORCH.update({n: getattr(torch, n) for n in ("bfloat16", "float32", "int32", "int64", "uint8",
                                                            "float8_e4m3fn")})
    return _TORCH[name]


def _typed(x, dtype: str, what: str):
    """`x` checked to be a tensor of `dtype`."""
    if isinstance(x, int) or x.dtype is not _dt(dtype):
        raise TypeError(f"{what}: expected a {dtype} tensor")
    return x


def _shaped(x, shape: tuple, what: str, dtype: str = "bfloat16", rank: int = -1) -> int:
    """Address of the contiguous device tensor `x`, which has to have `shape`."""
    if isinstance(x, int) or x.dtype is not _dt(dtype) or x.shape != shape or not x.is_cuda or not x.is_contiguous():
        name = what if rank < 0 else f"{what}[{rank}]"
        _typed(x, dtype, name)
        if x.shape != shape:
            raise ValueError(f"{name}: expected shape {shape}, got {tuple(x.shape)}")
        return _ptr(x, 0, name)
    return x.data_ptr()


def _strided(x, shape: tuple, what: str):
    """Address and row stride of the bf16 matrix `x`, whose rows' elements are contiguous."""
    if _typed(x, "bfloat16", what).shape != shape:
        raise ValueError(f"{what}: expected shape {shape}, got {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError(f"{what}: must be a CUDA tensor")
    rows, width = shape
    if width > 1 and rows and x.stride(1) != 1:
        raise ValueError(f"{what}: a row's elements must be contiguous")
    if rows > 1 and x.stride(0) < width:
        raise ValueError(f"{what}: rows must not overlap")
    return x.data_ptr(), max(x.stride(0) if rows > 1 else width, width)


def _per_rank(xs, shapes, what: str, dtype: str = "bfloat16") -> C.Array:
    n = len(shapes)
    if len(xs) != n:
        raise ValueError(f"{what}: expected {n} per-rank tensors, got {len(xs)}")
    return (C.c_void_p * n)(*[_shaped(xs[r], shapes[r], what, dtype, r) for r in range(n)])


def _groups(rows, experts: int, seg):
    """The hocRowGroups_t of buffers with `rows[d]` rows each, and what it points to."""
    k = len(rows)
    _typed(seg, "int64", "seg")
    if not experts:
        raise ValueError("weights of at least one expert must be given")
    if seg.dim() != 2 or seg.shape[0] != k or seg.shape[1] < experts + 1 or (seg.shape[1] - 1) % experts:
        raise ValueError(f"seg: expected shape [{k}, sources * {experts} + 1], got {tuple(seg.shape)}")
    cap = (C.c_size_t * max(1, k))(*rows)
    return _RowGroups(k, _int(experts), _int((seg.shape[1] - 1) // experts), _ptr(seg, 0, "seg"), cap), cap


def ep_segments(expert_ids, experts: int, topk: int, seg, stream=None):
    """Row ranges of every expert in the receive layout of a dispatch (see include/hoc_layer.h): expert_ids are the k
    sources' [tokens * topk] int32 ids, experts counts all ranks'; seg: [k, experts + 1] int64."""
    k = len(expert_ids)
    n = expert_ids[0].numel() if k else 0
    if topk < 1 or n % topk:
        raise ValueError("expert_ids must hold topk ids per token")
    for r, v in enumerate(expert_ids):
        _typed(v, "int32", f"expert_ids[{r}]")
    _check(lib().hoc_ep_segments(k, _ptr_array(expert_ids, 4 * n, "expert_ids"), _int(n // topk), _int(topk), _int(experts),
                                 _shaped(seg, (k, int(experts) + 1), "seg", "int64"), _stream(stream)),
           "hoc_ep_segments")


def expert_mm(x, weight, seg, y, *, status, bias=None, act: str = "none", pre=None, stream=None):
    """y[d][r] = act(W[d][e] x[d][r] + bias[d][e]) for the rows r that seg gives to expert e of rank d (see
    include/hoc_layer.h).  Lists of k device tensors: x [capacity, in], weight [experts, out, in] ([experts, 2 * out,
    in] for swiglu), y [capacity, out]; pre keeps the pre-activations for the gradients."""
    a, k = _act(act), len(x)
    if not k or not weight or weight[0].dim() != 3 or x[0].dim() != 2:
        raise ValueError("x: a list of matrices, weight: a list of [experts, out, in] tensors")
    mul = 2 if act == "swiglu" else 1
    experts, wide, inp = weight[0].shape
    if wide % mul:
        raise ValueError("weight: swiglu needs an even number of rows, gates first")
    out, rows = wide // mul, [t.shape[0] for t in x]
    g, _keep = _groups(rows, experts, seg)
    _check(lib().hoc_expert_mm(C.byref(g), _per_rank(x, [(n, inp) for n in rows], "x"),
                               _per_rank(weight, [(experts, wide, inp)] * k, "weight"),
                               None if bias is None else _per_rank(bias, [(experts, wide)] * k, "bias"), _int(inp),
                               _int(out), a,
                               _per_rank(y, [(n, out) for n in rows], "y"),
                               None if pre is None else _per_rank(pre, [(n, wide) for n in rows], "pre"),
                               _ptr(status, 4, "status"), _stream(stream)), "hoc_expert_mm")


def expert_mm_dgrad(dy, weight, seg, dx, *, status, act: str = "none", pre=None, stream=None):
    """dx[d][r] = W[d][e]^T dy[d][r]; with act the layer's input came out of that activation and dx is the gradient
    for what went into it, pre (see include/hoc_layer.h)."""
    a, k = _act(act), len(dy)
    if not k or not weight or weight[0].dim() != 3 or dy[0].dim() != 2:
        raise ValueError("dy: a list of matrices, weight: a list of [experts, out, in] tensors")
    if (act != "none") != (pre is not None):
        raise ValueError("pre is given exactly when there is an activation")
    experts, out, inp = weight[0].shape
    wide, rows = inp * (2 if act == "swiglu" else 1), [t.shape[0] for t in dy]
    g, _keep = _groups(rows, experts, seg)
    _check(lib().hoc_expert_mm_dgrad(C.byref(g), _per_rank(dy, [(n, out) for n in rows], "dy"),
                                     _per_rank(weight, [(experts, out, inp)] * k, "weight"), _int(inp), _int(out), a,
                                     None if pre is None else _per_rank(pre, [(n, wide) for n in rows], "pre"),
                                     _per_rank(dx, [(n, wide) for n in rows], "dx"), _ptr(status, 4, "status"),
                                     _stream(stream)), "hoc_expert_mm_dgrad")


def expert_mm_wgrad(dy, x, seg, dw, *, status, db=None, accumulate: bool = False, stream=None):
    """dw[d][e] (+)= sum of dy[r]^T x[r] over the rows of expert e of rank d, db[d][e] (+)= sum of dy[r]; dw [experts,
    out, in] and db [experts, out] in bf16 or float32 (see include/hoc_layer.h)."""
    k = len(x)
    if not k or not dw or dw[0].dim() != 3:
        raise ValueError("x: a list of matrices, dw: a list of [experts, out, in] tensors")
    experts, out, inp = dw[0].shape
    rows, dt = [t.shape[0] for t in x], "float32" if dw[0].dtype is _dt("float32") else "bfloat16"
    g, _keep = _groups(rows, experts, seg)
    _check(lib().hoc_expert_mm_wgrad(C.byref(g), _per_rank(dy, [(n, out) for n in rows], "dy"),
                                     _per_rank(x, [(n, inp) for n in rows], "x"), _int(inp), _int(out), _dtype_code(dw[0]),
                                     int(bool(accumulate)), _per_rank(dw, [(experts, out, inp)] * k, "dw", dt),
                                     None if db is None else _per_rank(db, [(experts, out)] * k, "db", dt),
                                     _ptr(status, 4, "status"), _stream(stream)), "hoc_expert_mm_wgrad")


def linear(x, weight, y, *, status, bias=None, act: str = "none", pre=None, residual=None, stream=None):
    """y = act(x W^T + bias) + residual; x, y and residual may be rows of wider buffers (see include/hoc_layer.h)."""
    a = _act(act)
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x and weight must be matrices")
    (rows, inp), wide = x.shape, weight.shape[0]
    mul = 2 if act == "swiglu" else 1
    if wide % mul:
        raise ValueError("weight: swiglu needs an even number of rows, gates first")
    out = wide // mul
    xp, ldx = _strided(x, (rows, inp), "x")
    yp, ldy = _strided(y, (rows, out), "y")
    rp, ldr = _strided(residual, (rows, out), "residual") if residual is not None else (None, 0)
    _check(lib().hoc_linear(_int(rows), xp, ldx, _shaped(weight, (wide, inp), "weight"),
                            None if bias is None else _shaped(bias, (wide,), "bias"), rp, ldr, _int(inp), _int(out), a, yp,
                            ldy,
                            None if pre is None else _shaped(pre, (rows, wide), "pre"), _ptr(status, 4, "status"),
                            _stream(stream)), "hoc_linear")


def linear_dgrad(dy, weight, dx, *, status, act: str = "none", pre=None, stream=None):
    """dx = dy W, through the activation below the layer as in expert_mm_dgrad (see include/hoc_layer.h)."""
    a = _act(act)
    if dy.dim() != 2 or weight.dim() != 2:
        raise ValueError("dy and weight must be matrices")
    if (act != "none") != (pre is not None):
        raise ValueError("pre is given exactly when there is an activation")
    out, inp = weight.shape
    rows, wide = dy.shape[0], inp * (2 if act == "swiglu" else 1)
    dp, ldd = _strided(dy, (rows, out), "dy")
    _check(lib().hoc_linear_dgrad(_int(rows), dp, ldd, _shaped(weight, (out, inp), "weight"), _int(inp), _int(out), a,
                                  None if pre is None else _shaped(pre, (rows, wide), "pre"),
                                  _shaped(dx, (rows, wide), "dx"), _ptr(status, 4, "status"), _stream(stream)),
           "hoc_linear_dgrad")


def linear_wgrad(dy, x, dw, *, status, db=None, accumulate: bool = False, stream=None):
    """dw (+)= dy^T x and db (+)= column sums of dy, in bf16 or float32 (see include/hoc_layer.h)."""
    if dw.dim() != 2 or x.dim() != 2:
        raise ValueError("x and dw must be matrices")
    (out, inp), rows = dw.shape, x.shape[0]
    dt = "float32" if dw.dtype is _dt("float32") else "bfloat16"
    dp, ldd = _strided(dy, (rows, out), "dy")
    xp, ldx = _strided(x, (rows, inp), "x")
    _check(lib().hoc_linear_wgrad(_int(rows), dp, ldd, xp, ldx, _int(inp), _int(out), _dtype_code(dw), int(bool(accumulate)),
                                  _shaped(dw, (out, inp), "dw", dt),
                                  None if db is None else _shaped(db, (out,), "db", dt), _ptr(status, 4, "status"),
                                  _stream(stream)), "hoc_linear_wgrad")


def act_grad(dy, pre, dz, act: str, stream=None):
    """dz = dy * act'(pre); dz may be pre, or dy where the activation is not gated (see include/hoc_layer.h)."""
    if dy.dim() != 2:
        raise ValueError("dy must be a matrix")
    rows, width = dy.shape
    wide = width * (2 if act == "swiglu" else 1)
    _check(lib().hoc_act_grad(_int(rows), _int(width), _act(act), _shaped(dy, (rows, width), "dy"),
                              _shaped(pre, (rows, wide), "pre"), _shaped(dz, (rows, wide), "dz"), _stream(stream)),
           "hoc_act_grad")


def layer_trim(keep: int = 0):
    """Gives scratch that products on rows of odd widths left behind back to the device, all but `keep` bytes (see
    include/hoc_layer.h); wait for their streams first."""
    if keep < 0:
        raise ValueError("keep must not be negative")
    _check(lib().hoc_layer_trim(int(keep)), "hoc_layer_trim")


# ------------------------------------- between the residual stream and the dispatch
SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score) -> int:
    if score not in SCORES:
        raise ValueError(f"score is one of {', '.join(SCORES)}, not {score!r}")
    return SCORES[score]


_ROW_DTYPES = {}  # torch dtypes of rows -> codes, once torch is imported


def _row_dtype(x, what: str) -> int:
    """The code of the dtype of `x`, rows of which the calls below take."""
    if not _ROW_DTYPES:
        _ROW_DTYPES.update({_dt("bfloat16"): BFLOAT16, _dt("float32"): FLOAT32})
    code = _ROW_DTYPES.get(getattr(x, "dtype", None))
    if code is None:
        raise TypeError(f"{what}: expected a bfloat16 or float32 tensor")
    return code


_NUMBERS = {}  # host numbers by value, as the library reads them: an address each


def _number(v, kind=C.c_float):
    if type(v) is not float:  # a tensor or an array of one element would be found by its identity, whatever it holds by now
        v = kind(v).value
    got = _NUMBERS.get((kind, v))
    if got is None:
        if len(_NUMBERS) >= 256:
            _NUMBERS.clear()
        got = _NUMBERS[kind, v] = C.byref(kind(v))
    return got


_get_device = _raw_stream = None  # torch's own calls for the current device and its stream, once torch is imported


def _here(x, what: str) -> int:
    """The device of `x`, which has to be the current one: a launch would run there."""
    global _get_device, _raw_stream
    if _get_device is None:
        import torch
        if not torch.cuda.is_available():
            raise ValueError(f"{what}: must be a CUDA tensor, and there is no GPU")
        torch.cuda.init()
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    device = x.get_device()
    if device < 0 or not x.is_cuda:
        raise ValueError(f"{what}: must be a CUDA tensor")
    if device != _get_device():
        raise ValueError(f"{what}: is on another device than the current one")
    return device


def _queue(stream, device: int) -> int:
    """The handle of `stream`, of the current one of `device` for None; _here has been called."""
    return _raw_stream(device) if stream is None and _raw_stream else _stream(stream)


def _rows_of(x, shape, dtype, device: int, what: str):
    """Address and row stride of the matrix `x`, whose rows' elements are contiguous; (None, 0) for None."""
    if x is None:
        return None, 0
    if isinstance(x, int) or x.dtype is not dtype:
        raise TypeError(f"{what}: expected a {str(dtype).split('.')[-1]} tensor")
    if x.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(x.shape)}")
    if x.get_device() != device:
        raise ValueError(f"{what}: must be a CUDA tensor on the device of the others")
    ld, step = x.stride()
    if step == 1 and ld >= shape[1]:
        return x.data_ptr(), ld
    rows, width = shape  # one row, one column or none may have any strides
    if rows and width > 1 and step != 1:
        raise ValueError(f"{what}: a row's elements must be contiguous")
    if rows > 1 and width and ld < width:
        raise ValueError(f"{what}: rows must not overlap")
    return x.data_ptr(), max(ld, width)


def _flat(x, n: int, dtype, device: int, what: str):
    """Address of the contiguous tensor `x` of n elements; None for None."""
    if x is None:
        return None
    if isinstance(x, int) or x.dtype is not dtype:
        raise TypeError(f"{what}: expected a {str(dtype).split('.')[-1]} tensor")
    if x.numel() != n or not x.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous elements, got shape {tuple(x.shape)}")
    if x.get_device() != device:
        raise ValueError(f"{what}: must be a CUDA tensor on the device of the others")
    return x.data_ptr()


_WIRE8 = {}  # width -> (bytes of a row, where its scales start)


def _wire8(width: int):
    if type(width) is not int:  # (as _number)
        width = int(width)
    got = _WIRE8.get(width)
    if got is None:
        _fits(width=width)
        n, at = C.c_size_t(), C.c_size_t()
        _check(lib().hoc_wire8_row(int(width), C.byref(n), C.byref(at)), "hoc_wire8_row")
        got = _WIRE8[width] = (n.value, at.value)
    return got


def wire8_bytes(width: int) -> int:
    """Bytes of a row of `width` values in 8 bits with their scales (see include/hoc_block.h): a dispatch moves such rows,
    a uint8 tensor viewed as bfloat16, as rows of half as many elements."""
    return _wire8(width)[0]


def wire8_views(wire, width: int):
    """The values (float8_e4m3fn, [rows, width]) and scales (float32, [rows, ceil(width / 128)]) in rows of 8 bits."""
    n, at = _wire8(width)
    if wire.dtype is not _dt("uint8") or wire.dim() != 2 or wire.shape[1] != n:
        raise ValueError(f"wire: expected a uint8 tensor of shape [rows, {n}]")
    return (wire.view(_TORCH["float8_e4m3fn"]).narrow(1, 0, width),
            wire.view(_TORCH["float32"]).narrow(1, at // 4, (width + 127) // 128))


def _wire_rows(wire, rows: int, width: int, device: int, what: str) -> Optional[int]:
    if wire is None:
        return None
    if wire.dim() != 2 or wire.shape[0] != rows or wire.shape[1] != _wire8(width)[0]:
        raise ValueError(f"{what}: expected shape {(rows, _wire8(width)[0])}, got {tuple(wire.shape)}")
    return _flat(wire, wire.numel(), _dt("uint8"), device, what)


def rms_norm(x, weight, y=None, *, eps: float, residual=None, h=None, wire=None, stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, stored as it is and / or as rows of 8 bits in wire, uint8
    [rows, wire8_bytes(width)] (see include/hoc_block.h).  x, residual, h and y: [rows, width] in bf16 or float32, may be
    rows of wider buffers; weight: [width] in either."""
    dt = _row_dtype(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    shape, dev = x.shape, _here(x, "x")
    rows, width = shape
    if rows > _MOST or width > _MOST:
        _fits(rows=rows, width=width)
    xp, ldx = _rows_of(x, shape, x.dtype, dev, "x")
    rp, ldr = _rows_of(residual, shape, x.dtype, dev, "residual")
    hp, ldh = _rows_of(h, shape, x.dtype, dev, "h")
    yp, ldy = _rows_of(y, shape, x.dtype, dev, "y")
    wdt = _row_dtype(weight, "weight")
    rc = (_lib or lib()).hoc_rms_norm(rows, width, dt, xp, ldx, rp, ldr, _flat(weight, width, weight.dtype, dev, "weight"), wdt,
                              _number(eps), hp, ldh, yp, ldy, _wire_rows(wire, rows, width, dev, "wire"), _queue(stream, dev))
    if rc:
        _check(rc, "hoc_rms_norm")


def rms_norm_workspace(rows: int, width: int) -> int:
    """int32 entries of scratch that rms_norm_grad needs for a weight gradient."""
    _fits(rows=rows, width=width)
    n = C.c_size_t()
    _check(lib().hoc_rms_norm_workspace(int(rows), int(width), C.byref(n)), "hoc_rms_norm_workspace")
    return n.value


def rms_norm_grad(dy, h, weight, dx, *, eps: float, dy2=None, dres=None, dw=None, accumulate: bool = False,
                  workspace=None, stream=None):
    """Gradients of rms_norm: dx for h (and so for x and the residual) from dy (+ dy2) for y and dres for h itself; dw (+)=
    the weight's, in bf16 or float32, with an int32 workspace of rms_norm_workspace entries (see include/hoc_block.h)."""
    dt = _row_dtype(dy, "dy")
    if dy.dim() != 2:
        raise ValueError("dy must be a matrix")
    shape, dev = dy.shape, _here(dy, "dy")
    rows, width = shape
    if rows > _MOST or width > _MOST:
        _fits(rows=rows, width=width)
    dyp, lddy = _rows_of(dy, shape, dy.dtype, dev, "dy")
    dy2p, lddy2 = _rows_of(dy2, shape, dy.dtype, dev, "dy2")
    hp, ldh = _rows_of(h, shape, dy.dtype, dev, "h")
    drp, lddr = _rows_of(dres, shape, dy.dtype, dev, "dres")
    dxp, lddx = _rows_of(dx, shape, dy.dtype, dev, "dx")
    if hp is None or dxp is None:
        raise ValueError("h and dx must be given")
    wdt, dwdt = _row_dtype(weight, "weight"), FLOAT32 if dw is None else _row_dtype(dw, "dw")
    wsp, ints = None, 0
    if dw is not None:
        if workspace is None:
            raise ValueError("workspace: a weight gradient needs one")
        ints = workspace.numel()
        wsp = _flat(workspace, ints, _dt("int32"), dev, "workspace")
    rc = (_lib or lib()).hoc_rms_norm_grad(rows, width, dt, dyp, lddy, dy2p, lddy2, hp, ldh,
                                   _flat(weight, width, weight.dtype, dev, "weight"), wdt, _number(eps), drp, lddr, dxp, lddx,
                                   None if dw is None else _flat(dw, width, dw.dtype, dev, "dw"), dwdt,
                                   int(bool(accumulate)), wsp, ints, _queue(stream, dev))
    if rc:
        _check(rc, "hoc_rms_norm_grad")


def expert_widen(wire, seg, y, *, counts=None, stream=None):
    """y[d][r] = bf16 of the rows of 8 bits wire[d][r], for the rows that seg covers (see include/hoc_block.h): lists of k
    device tensors, wire uint8 [capacity, wire8_bytes(width)], y bf16 [capacity, width]; seg as expert_mm's.  counts: those
    of the dispatch that moved the rows, int64 [k, k], turned into counts of y's elements for the combine."""
    k = len(y)
    if not k or len(wire) != k or y[0].dim() != 2:
        raise ValueError("wire and y: lists of as many matrices")
    _typed(seg, "int64", "seg")
    if seg.dim() != 2 or seg.shape[0] != k or seg.shape[1] < 2:
        raise ValueError(f"seg: expected shape [{k}, sources * experts + 1], got {tuple(seg.shape)}")
    dev, width = _here(y[0], "y[0]"), y[0].shape[1]
    if seg.shape[1] > _MOST:
        _fits(seg=seg.shape[1])
    n, bf, u8 = wire8_bytes(width), _dt("bfloat16"), _dt("uint8")
    caps, yp, wp, rows, shape, fits = [], [], [], 0, None, False
    for t, w in zip(y, wire):
        if t.shape != shape:
            shape, rows = t.shape, t.shape[0]
            rows_n, fits = (rows, n), t.shape == (rows, width)
        if (t.dtype is not bf or w.dtype is not u8 or not fits or w.shape != rows_n or not t.is_contiguous()
                or not w.is_contiguous() or t.get_device() != dev or w.get_device() != dev):
            d = len(caps)  # the checks once more, by those that name what is wrong
            _flat(t, rows * width, bf, dev, f"y[{d}]")
            _flat(w, rows * n, u8, dev, f"wire[{d}]")
            raise ValueError(f"y[{d}] and wire[{d}]: expected shapes [capacity, {width}] and [capacity, {n}], got "
                             f"{tuple(t.shape)} and {tuple(w.shape)}")
        caps.append(rows)
        yp.append(t.data_ptr())
        wp.append(w.data_ptr())
    arr = C.c_void_p * k
    yp, wp, cap = arr(*yp), arr(*wp), (C.c_size_t * k)(*caps)
    g = _RowGroups(k, seg.shape[1] - 1, 1, _flat(seg, seg.numel(), seg.dtype, dev, "seg"), cap)
    rc = (_lib or lib()).hoc_expert_widen(C.byref(g), wp, width, yp,
                                  None if counts is None else _flat(counts, k * k, _dt("int64"), dev, "counts"),
                                  _queue(stream, dev))
    if rc:
        _check(rc, "hoc_expert_widen")


def _slots(logits, ids, gate, what: str):
    """What both calls of the routing check: tokens, experts, topk, the logits' dtype and the addresses."""
    dt = _row_dtype(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be a matrix [tokens, experts]")
    shape, dev = logits.shape, _here(logits, "logits")
    tokens, experts = shape
    n = ids.numel()
    if n % tokens if tokens else n:
        raise ValueError("ids must hold topk ids per token")
    if n > _MOST or experts > _MOST:  # (n is tokens * topk)
        _fits(tokens=tokens, experts=experts, topk=n // max(tokens, 1))
    lp, ldl = _rows_of(logits, shape, logits.dtype, dev, "logits")
    return (tokens, experts, n // tokens if tokens else 1, lp, dt, ldl, dev, _flat(ids, n, _dt("int32"), dev, "ids"),
            _flat(gate, n, _dt("float32"), dev, what))


def ep_route(logits, ids, gate, *, score: str = "softmax", bias=None, groups: int = 1, top_groups: Optional[int] = None,
             renormalise: bool = False, scale: float = 1.0, stream=None):
    """Routing of tokens to their topk experts (see include/hoc_block.h): logits [tokens, experts] in bf16 or float32, may
    be rows of a wider buffer; ids int32 and gate float32 of tokens * topk elements, as a dispatch and a combine take them;
    bias float32 [experts], for the choice only; of `groups` groups of experts the best top_groups (default: all)."""
    tokens, experts, topk, lp, dt, ldl, dev, ip, gp = _slots(logits, ids, gate, "gate")
    if top_groups is None:
        top_groups = groups
    if (groups != 1 or top_groups != 1) and not (-_MOST <= groups <= _MOST and -_MOST <= top_groups <= _MOST):
        _fits(groups=groups, top_groups=top_groups)
    rc = (_lib or lib()).hoc_ep_route(tokens, experts, topk, lp, dt, ldl, _score(score),
                              _flat(bias, experts, _dt("float32"), dev, "bias"), groups, top_groups,
                              int(bool(renormalise)), _number(scale), ip, gp, _queue(stream, dev))
    if rc:
        _check(rc, "hoc_ep_route")


def ep_route_grad(logits, ids, dgate, dlogits, *, score: str = "softmax", renormalise: bool = False, scale: float = 1.0,
                  stream=None):
    """Gradient of ep_route for the logits, from dgate for the gates; dlogits may be logits (see include/hoc_block.h)."""
    tokens, experts, topk, lp, dt, ldl, dev, ip, gp = _slots(logits, ids, dgate, "dgate")
    dp, ldd = _rows_of(dlogits, logits.shape, logits.dtype, dev, "dlogits")
    rc = (_lib or lib()).hoc_ep_route_grad(tokens, experts, topk, lp, dt, ldl, _score(score), int(bool(renormalise)), _number(scale), ip, gp,
                                   dp, ldd, _queue(stream, dev))
    if rc:
        _check(rc, "hoc_ep_route_grad")


def dropout(x, y, p: float, seed, *, residual=None, stream=None):
    """y = residual + x / (1 - p) where an element is kept, residual (or 0) where it is dropped; which are is drawn from
    seed, two int64 on the device, and not stored: the gradient is the same call on the gradient, without a residual (see
    include/hoc_block.h).  x, y and residual: contiguous, of any shape, or [rows, width] that may be rows of wider buffers."""
    dt, dev = _row_dtype(x, "x"), _here(x, "x")
    shape = x.shape
    if x.dim() != 2 or shape[1] > _MOST:
        for t, what in ((x, "x"), (y, "y"), (residual, "residual")):
            if t is not None and (t.shape != shape or not t.is_contiguous()):
                raise ValueError(f"{what}: expected shape {tuple(shape)}, contiguous (or rows of a matrix, below 2^31 wide)")
        n = x.numel()
        width = 1
        for w in reversed(shape):  # rows of the last dimensions, as wide as an int holds; there may be more rows than that
            if width * w > _MOST:
                break
            width *= w
        shape = (n // width if width else 0, width)
        x, y, residual = x.view(shape), y.view(shape), None if residual is None else residual.view(shape)
    xp, ldx = _rows_of(x, shape, x.dtype, dev, "x")
    yp, ldy = _rows_of(y, shape, x.dtype, dev, "y")
    rp, ldr = _rows_of(residual, shape, x.dtype, dev, "residual")
    rc = (_lib or lib()).hoc_dropout(shape[0], shape[1], dt, xp, ldx, rp, ldr, _number(p, C.c_double), _flat(seed, 2, _dt("int64"), dev, "seed"), yp,
                             ldy, _queue(stream, dev))
    if rc:
        _check(rc, "hoc_dropout")


# ------------------------------------------------------------- gradient clipping
class TensorList:
    """Device tensors of one dtype (float32 or bfloat16), as a table the gradient kernels read.

    Holds references to the tensors; free it with close() or as a context manager."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        dts = {t.dtype for t in self.tensors}
        if len(dts) > 1:
            raise TypeError("the tensors of a list must have one dtype")
        dtype = _dtype_code(self.tensors[0]) if self.tensors else FLOAT32
        n = len(self.tensors)
        counts = (C.c_size_t * max(1, n))(*[t.numel() for t in self.tensors])
        h = C.c_void_p()
        _check(lib().hoc_tensor_list_create(C.byref(h), n, _ptr_array(self.tensors, 0, "tensors"), counts, dtype),
               "hoc_tensor_list_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            _check(lib().hoc_tensor_list_destroy(self._h), "hoc_tensor_list_destroy")
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def grad_workspace(tensors: TensorList) -> int:
    """int32 entries of scratch that grad_norm and grad_clip need for this list."""
    n = C.c_size_t()
    _check(lib().hoc_grad_workspace(tensors._h, C.byref(n)), "hoc_grad_workspace")
    return n.value


def grad_norm(tensors: TensorList, norm, workspace, stream=None):
    """norm[0] = the global 2-norm of the list (see include/hoc_grad.h); norm: float32, workspace: int32 tensors."""
    _check(lib().hoc_grad_norm(tensors._h, _ptr(_typed(norm, "float32", "norm"), 4, "norm"),
                               _ptr(_typed(workspace, "int32", "workspace"), 0, "workspace"),
                               int(workspace.numel()), _stream(stream)), "hoc_grad_norm")


def grad_clip(src: TensorList, dst: TensorList, max_norm: float, norm, workspace, stream=None):
    """dst = min(1, max_norm / (norm + 1e-6)) * src with the global norm of src, which is left in norm[0]; dst may be
    src (see include/hoc_grad.h)."""
    _check(lib().hoc_grad_clip(src._h, dst._h, C.byref(C.c_float(max_norm)), _ptr(_typed(norm, "float32", "norm"), 4, "norm"),
                               _ptr(_typed(workspace, "int32", "workspace"), 0, "workspace"),
                               int(workspace.numel()), _stream(stream)), "hoc_grad_clip")


def sm_count(device: int = 0) -> int:
    n = C.c_int()
    _check(lib().hoc_device_sm_count(int(device), C.byref(n)), "hoc_device_sm_count")
    return n.value


def plan_query(nranks: int, op: int, count: int, dtype: int, counts=None, config: Optional[Config] = None):
    """The plan the scheduler would run, as a list of dicts (host only, no GPU)."""
    cfg = (config or Config()).to_c()
    cnt = _sizes(counts, nranks * nranks) if counts is not None else None
    n = C.c_size_t()
    _check(lib().hoc_plan_query(nranks, C.byref(cfg), op, int(count), dtype, cnt, None, 0, C.byref(n)),
           "hoc_plan_query")
    items = (_PlanItem * max(1, n.value))()
    _check(lib().hoc_plan_query(nranks, C.byref(cfg), op, int(count), dtype, cnt, items, n.value, C.byref(n)),
           "hoc_plan_query")
    return [{name: getattr(items[i], name) for name, _ in _PlanItem._fields_} for i in range(n.value)]
