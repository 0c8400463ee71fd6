"""Python binding of libra.so: argument marshalling only.

The functions carry the C ABI's names (include/ra.h). Tensors supply device
pointers (``data_ptr()``) and the stream is torch's current CUDA stream unless
one is given; every step of a call runs in the library's kernels.
The library must be built (``python -m ring_all_reduce_02_gb300.build``); if
it is missing, the first call raises instead of falling back to anything.
"""

from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libra.so")

RA_SUCCESS, RA_ERR_INVALID_ARG, RA_ERR_UNSUPPORTED, RA_ERR_ALIAS, RA_ERR_CUDA, RA_ERR_SCRATCH_LIMIT = range(6)
RA_NOALLOC_STATUS_WORDS = 16
DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2, "i32": 3}
OP_CODES = {"sum": 0, "avg": 1, "min": 2, "max": 3, "prod": 4}
ORDER_CODES = {"ring": 0, "tree": 1, "rabenseifner": 2}
ACCUM_CODES = {"dtype": 0, "fp32": 1}
RA_MAX_RANKS = 64

# every symbol include/ra.h declares
EXPORTS = ("ra_allreduce", "ra_reduce_scatter", "ra_allgather", "ra_allreduce_ex", "ra_reduce_scatter_ex",
           "ra_bucket_plan", "ra_allreduce_buckets", "ra_allreduce_ringsteps", "ra_chunk_range", "ra_plan_chunk",
           "ra_status_string", "ra_last_cuda_error", "ra_vector_bytes", "ra_selftest_bulk_timeout",
           "ra_allreduce_bulk_noalloc", "ra_layernorm_forward", "ra_layernorm_backward", "ra_layernorm_workspace",
           "ra_grad_norm", "ra_grad_norm_workspace", "ra_adamw")
ENGINE_CODES = {"registers": 0, "bulk": 1}
RA_STATE_F32, RA_STATE_E4M3 = 0, 1
RA_ADAMW_BLOCK = 256  # elements per scale of an 8-bit moment


class Options(ctypes.Structure):
    """ra_options_t."""

    _fields_ = [("order", ctypes.c_int), ("accum", ctypes.c_int), ("max_sms", ctypes.c_int),
                ("engine", ctypes.c_int), ("status", ctypes.c_void_p)]


class AdamwTensor(ctypes.Structure):
    """ra_adamw_tensor_t."""

    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("count", ctypes.c_size_t),
                ("weight_decay", ctypes.c_double)]


class AdamwOptions(ctypes.Structure):
    """ra_adamw_options_t."""

    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("grad_scale", ctypes.c_void_p),
                ("state", ctypes.c_int), ("copy_dtype", ctypes.c_int), ("seed", ctypes.c_uint64)]


def options(order: str = "ring", accum: str = "dtype", max_sms: int = 0, engine: str = "registers",
            status=None) -> Options:
    """ra_options_t; ``status`` is a device int32 tensor (or address) for the bulk engine."""
    st = status.data_ptr() if hasattr(status, "data_ptr") else status
    return Options(ORDER_CODES[order], ACCUM_CODES[accum], max_sms, ENGINE_CODES[engine], st or None)


class RaError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        name = lib().ra_status_string(status).decode()
        extra = f" (cudaError {lib().ra_last_cuda_error()})" if status == RA_ERR_CUDA else ""
        super().__init__(f"{call}: {name}{extra}")


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m ring_all_reduce_02_gb300.build` (no fallback exists)")
            L = ctypes.CDLL(LIB_PATH)
            VP, SZ, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
            PP = ctypes.POINTER(ctypes.c_void_p)
            PSZ = ctypes.POINTER(ctypes.c_size_t)
            POPT = ctypes.POINTER(Options)
            for name in ("ra_allreduce", "ra_reduce_scatter", "ra_allgather"):
                f = getattr(L, name)
                f.argtypes = [PP, PP, SZ, I, I, I, VP]
                f.restype = I
            for name in ("ra_allreduce_ex", "ra_reduce_scatter_ex"):
                f = getattr(L, name)
                f.argtypes = [PP, PP, SZ, I, I, I, POPT, VP]
                f.restype = I
            L.ra_bucket_plan.argtypes = [PSZ, I, SZ, I, PSZ, PSZ, I, ctypes.POINTER(I)]
            L.ra_bucket_plan.restype = I
            L.ra_allreduce_buckets.argtypes = [PP, PP, SZ, I, I, I, I, PSZ, PSZ, PP, POPT, VP]
            L.ra_allreduce_buckets.restype = I
            L.ra_allreduce_ringsteps.argtypes = [PP, PP, SZ, I, I, I, I, VP]
            L.ra_allreduce_ringsteps.restype = I
            L.ra_chunk_range.argtypes = [SZ, I, I, PSZ, PSZ]
            L.ra_chunk_range.restype = I
            L.ra_plan_chunk.argtypes = [SZ, I, I, I, I, I, PSZ, PSZ, PSZ, PSZ]
            L.ra_plan_chunk.restype = I
            L.ra_status_string.argtypes = [I]
            L.ra_status_string.restype = ctypes.c_char_p
            L.ra_last_cuda_error.argtypes = []
            L.ra_last_cuda_error.restype = I
            L.ra_vector_bytes.argtypes = []
            L.ra_vector_bytes.restype = I
            L.ra_selftest_bulk_timeout.argtypes = [PP, PP, SZ, I, I, I, I, VP, I, VP]
            L.ra_selftest_bulk_timeout.restype = I
            L.ra_allreduce_bulk_noalloc.argtypes = [PP, PP, SZ, I, I, I, I, VP, VP]
            L.ra_allreduce_bulk_noalloc.restype = I
            L.ra_layernorm_forward.argtypes = [VP, SZ, VP, VP, VP, SZ, VP, VP, SZ, SZ, ctypes.c_double, I, I, VP]
            L.ra_layernorm_forward.restype = I
            L.ra_layernorm_backward.argtypes = [VP, SZ, VP, SZ, VP, VP, VP, VP, SZ, VP, VP, I, SZ, SZ, I, I, VP, SZ,
                                                VP]
            L.ra_layernorm_backward.restype = I
            L.ra_layernorm_workspace.argtypes = [SZ, SZ]
            L.ra_layernorm_workspace.restype = SZ
            L.ra_grad_norm.argtypes = [PP, PSZ, I, I, ctypes.c_double, ctypes.c_double, VP, VP, SZ, VP]
            L.ra_grad_norm.restype = I
            L.ra_grad_norm_workspace.argtypes = []
            L.ra_grad_norm_workspace.restype = SZ
            L.ra_adamw.argtypes = [ctypes.POINTER(AdamwTensor), I, I, I, ctypes.POINTER(AdamwOptions), VP]
            L.ra_adamw.restype = I
            _lib = L
    return _lib


def ptr_array(ptrs) -> ctypes.Array:
    return (ctypes.c_void_p * len(ptrs))(*[int(p) if p else None for p in ptrs])


def dtype_code(t) -> int:
    import torch

    codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int32: 3}
    if t.dtype not in codes:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return codes[t.dtype]


def _stream_ptr(stream) -> int:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check(tensors, what):
    dt = tensors[0].dtype
    for t in tensors:
        if not (t.is_cuda or (t.device.type == "cpu" and t.is_pinned())):
            raise ValueError(f"{what}: every buffer must be a CUDA tensor or pinned host memory")
        if t.dtype != dt:
            raise ValueError(f"{what}: all buffers must share one dtype")
        if not t.is_contiguous():
            raise ValueError(f"{what}: buffers must be contiguous")


def _check_full(sendbufs, recvbufs, what):
    _check(list(sendbufs) + list(recvbufs), what)
    count = sendbufs[0].numel()
    if any(t.numel() != count for t in list(sendbufs) + list(recvbufs)) or len(recvbufs) != len(sendbufs):
        raise ValueError(f"{what}: N send and N recv buffers of one length")
    return count


def _chunk_len(count: int, n: int, c: int) -> int:
    return (c + 1) * count // n - c * count // n


def call(name: str, send_ptrs, recv_ptrs, count: int, dtype: int, op: int, nranks: int, stream: int) -> int:
    """Raw C call with integer pointers; returns the ra_status_t."""
    f = getattr(lib(), name)
    return f(ptr_array(send_ptrs), ptr_array(recv_ptrs), count, dtype, op, nranks, ctypes.c_void_p(stream or None))


def call_ex(name: str, send_ptrs, recv_ptrs, count: int, dtype: int, op: int, nranks: int, order: int,
            accum: int, stream: int, max_sms: int = 0, engine: int = 0, status: int = 0) -> int:
    """Raw C call of ra_allreduce_ex / ra_reduce_scatter_ex; returns the ra_status_t."""
    f = getattr(lib(), name)
    opts = Options(order, accum, max_sms, engine, status or None)
    return f(ptr_array(send_ptrs), ptr_array(recv_ptrs), count, dtype, op, nranks, ctypes.byref(opts),
             ctypes.c_void_p(stream or None))


def ra_allreduce(sendbufs, recvbufs, op: str = "sum", stream=None) -> None:
    """All-reduce of N equal-length tensors into N tensors (recv may be send: in place)."""
    count = _check_full(sendbufs, recvbufs, "ra_allreduce")
    st = call("ra_allreduce", [t.data_ptr() for t in sendbufs], [t.data_ptr() for t in recvbufs], count,
              dtype_code(sendbufs[0]), OP_CODES[op], len(sendbufs), _stream_ptr(stream))
    if st:
        raise RaError(st, "ra_allreduce")


def ra_allreduce_ex(sendbufs, recvbufs, op: str = "sum", order: str = "ring", accum: str = "dtype",
                    max_sms: int = 0, engine: str = "registers", status=None, stream=None) -> None:
    """All-reduce with a reduction order (ring | tree | rabenseifner), accumulation (dtype | fp32),
    an SM budget (0 = all SMs) and an engine (registers | bulk; bulk needs a device int32 ``status``)."""
    count = _check_full(sendbufs, recvbufs, "ra_allreduce_ex")
    st_ptr = status.data_ptr() if status is not None else 0
    st = call_ex("ra_allreduce_ex", [t.data_ptr() for t in sendbufs], [t.data_ptr() for t in recvbufs], count,
                 dtype_code(sendbufs[0]), OP_CODES[op], len(sendbufs), ORDER_CODES[order], ACCUM_CODES[accum],
                 _stream_ptr(stream), max_sms, ENGINE_CODES[engine], st_ptr)
    if st:
        raise RaError(st, "ra_allreduce_ex")


def ra_reduce_scatter(sendbufs, recvbufs, op: str = "sum", stream=None) -> None:
    """Reduce-scatter: recvbufs[r] receives chunk r (compact) of the reduction."""
    _check(list(sendbufs) + [t for t in recvbufs if t.numel()], "ra_reduce_scatter")
    count, n = sendbufs[0].numel(), len(sendbufs)
    for r, t in enumerate(recvbufs):
        if t.numel() != _chunk_len(count, n, r):
            raise ValueError(f"ra_reduce_scatter: recvbufs[{r}] must hold chunk {r}")
    st = call("ra_reduce_scatter", [t.data_ptr() for t in sendbufs], [t.data_ptr() for t in recvbufs], count,
              dtype_code(sendbufs[0]), OP_CODES[op], n, _stream_ptr(stream))
    if st:
        raise RaError(st, "ra_reduce_scatter")


def ra_reduce_scatter_ex(sendbufs, recvbufs, op: str = "sum", order: str = "ring", accum: str = "dtype",
                         max_sms: int = 0, stream=None) -> None:
    """Reduce-scatter with a reduction order, accumulation and SM budget; recvbufs[r] receives chunk r."""
    _check(list(sendbufs) + [t for t in recvbufs if t.numel()], "ra_reduce_scatter_ex")
    count, n = sendbufs[0].numel(), len(sendbufs)
    for r, t in enumerate(recvbufs):
        if t.numel() != _chunk_len(count, n, r):
            raise ValueError(f"ra_reduce_scatter_ex: recvbufs[{r}] must hold chunk {r}")
    st = call_ex("ra_reduce_scatter_ex", [t.data_ptr() for t in sendbufs], [t.data_ptr() for t in recvbufs],
                 count, dtype_code(sendbufs[0]), OP_CODES[op], n, ORDER_CODES[order], ACCUM_CODES[accum],
                 _stream_ptr(stream), max_sms)
    if st:
        raise RaError(st, "ra_reduce_scatter_ex")


def ra_allgather(sendbufs, recvbufs, stream=None) -> None:
    """All-gather: sendbufs[r] is chunk r (compact); every recvbufs[r] receives all chunks."""
    _check([t for t in sendbufs if t.numel()] + list(recvbufs), "ra_allgather")
    count, n = recvbufs[0].numel(), len(recvbufs)
    for r, t in enumerate(sendbufs):
        if t.numel() != _chunk_len(count, n, r):
            raise ValueError(f"ra_allgather: sendbufs[{r}] must hold chunk {r}")
    st = call("ra_allgather", [t.data_ptr() for t in sendbufs], [t.data_ptr() for t in recvbufs], count,
              dtype_code(recvbufs[0]), OP_CODES["sum"], n, _stream_ptr(stream))
    if st:
        raise RaError(st, "ra_allgather")


def ra_allreduce_ringsteps(sendbufs, recvbufs, op: str = "sum", nsteps: int = -1, stream=None) -> None:
    """The literal ring schedule, one launch per step (first ``nsteps`` of 2(N-1); -1 = all)."""
    count = _check_full(sendbufs, recvbufs, "ra_allreduce_ringsteps")
    st = lib().ra_allreduce_ringsteps(ptr_array([t.data_ptr() for t in sendbufs]),
                                      ptr_array([t.data_ptr() for t in recvbufs]), count,
                                      dtype_code(sendbufs[0]), OP_CODES[op], len(sendbufs), nsteps,
                                      ctypes.c_void_p(_stream_ptr(stream) or None))
    if st:
        raise RaError(st, "ra_allreduce_ringsteps")


def ra_bucket_plan(param_counts, bucket_bytes: int, elem_size: int):
    """DDP-style buckets over a flat buffer: list of (begin, count) in the order they become ready."""
    n = len(param_counts)
    counts = (ctypes.c_size_t * max(n, 1))(*param_counts)
    nb = ctypes.c_int()
    st = lib().ra_bucket_plan(counts, n, bucket_bytes, elem_size, None, None, 0, ctypes.byref(nb))
    if st and not (st == RA_ERR_INVALID_ARG and nb.value > 0):
        raise RaError(st, "ra_bucket_plan")
    m = nb.value
    begin = (ctypes.c_size_t * max(m, 1))()
    cnt = (ctypes.c_size_t * max(m, 1))()
    st = lib().ra_bucket_plan(counts, n, bucket_bytes, elem_size, begin, cnt, m, ctypes.byref(nb))
    if st:
        raise RaError(st, "ra_bucket_plan")
    return [(begin[b], cnt[b]) for b in range(m)]


def ra_allreduce_buckets(sendbufs, recvbufs, buckets, op: str = "sum", ready_events=None, order: str = "ring",
                         accum: str = "dtype", max_sms: int = 0, engine: str = "registers", status=None,
                         stream=None) -> None:
    """All-reduce every bucket (begin, count) of the flat buffers, each after its ready event."""
    count = _check_full(sendbufs, recvbufs, "ra_allreduce_buckets")
    m = len(buckets)
    begin = (ctypes.c_size_t * max(m, 1))(*[b for b, _ in buckets])
    cnt = (ctypes.c_size_t * max(m, 1))(*[c for _, c in buckets])
    events = None
    if ready_events is not None:
        events = ptr_array([int(e.cuda_event) if e is not None else 0 for e in ready_events])
    opts = options(order, accum, max_sms, engine, status)
    st = lib().ra_allreduce_buckets(ptr_array([t.data_ptr() for t in sendbufs]),
                                    ptr_array([t.data_ptr() for t in recvbufs]), count, dtype_code(sendbufs[0]),
                                    OP_CODES[op], len(sendbufs), m, begin, cnt, events, ctypes.byref(opts),
                                    ctypes.c_void_p(_stream_ptr(stream) or None))
    if st:
        raise RaError(st, "ra_allreduce_buckets")


def ra_chunk_range(count: int, nranks: int, c: int) -> tuple[int, int]:
    b, e = ctypes.c_size_t(), ctypes.c_size_t()
    st = lib().ra_chunk_range(count, nranks, c, ctypes.byref(b), ctypes.byref(e))
    if st:
        raise RaError(st, "ra_chunk_range")
    return b.value, e.value


def ra_plan_chunk(count: int, nranks: int, c: int, elem_size: int, phase_bytes: int, align_bytes: int = 0):
    """(begin, end, vec_begin, vec_end) of chunk c: which part takes the vector path. ``align_bytes``
    is the grid's alignment (a power of two from ra_vector_bytes() to 512; 0: ra_vector_bytes())."""
    align_bytes = align_bytes or lib().ra_vector_bytes()
    out = [ctypes.c_size_t() for _ in range(4)]
    st = lib().ra_plan_chunk(count, nranks, c, elem_size, align_bytes, phase_bytes, *[ctypes.byref(o) for o in out])
    if st:
        raise RaError(st, "ra_plan_chunk")
    return tuple(o.value for o in out)


def ra_status_string(status: int) -> str:
    return lib().ra_status_string(status).decode()


def ra_selftest_bulk_timeout(sendbufs, recvbufs, status, op: str = "sum", withhold_chunk: int = 0,
                             per_chunk: bool = False, stream=None) -> None:
    """Run the bulk engine with chunk ``withhold_chunk``'s first tile withheld: that chunk's bounded
    wait must give up and set its status word. ``status``: a device int32 tensor, one word
    (``per_chunk`` False) or nranks words, word c for chunk c (``per_chunk`` True)."""
    count = _check_full(sendbufs, recvbufs, "ra_selftest_bulk_timeout")
    if status.numel() < (len(sendbufs) if per_chunk else 1):
        raise ValueError("ra_selftest_bulk_timeout: status is too small")
    st = lib().ra_selftest_bulk_timeout(ptr_array([t.data_ptr() for t in sendbufs]),
                                        ptr_array([t.data_ptr() for t in recvbufs]), count, dtype_code(sendbufs[0]),
                                        OP_CODES[op], len(sendbufs), withhold_chunk,
                                        ctypes.c_void_p(status.data_ptr()), 1 if per_chunk else 0,
                                        ctypes.c_void_p(_stream_ptr(stream) or None))
    if st:
        raise RaError(st, "ra_selftest_bulk_timeout")


def ra_vector_bytes() -> int:
    return lib().ra_vector_bytes()


def ra_allreduce_bulk_noalloc(sendbufs, recvbufs, op: str = "sum", max_sms: int = 0, chunk_status=None,
                              stream=None) -> None:
    """The bulk-engine all-reduce with the status words kept by the library, so no device memory
    beyond the buffers is needed. ``chunk_status``: optional int32 tensor of nranks words (device or
    host) that receives each chunk's wait code (0 = finished) once the stream has passed the call."""
    import torch

    count = _check_full(sendbufs, recvbufs, "ra_allreduce_bulk_noalloc")
    if chunk_status is not None and (chunk_status.dtype != torch.int32 or not chunk_status.is_contiguous()
                                     or chunk_status.numel() < len(sendbufs)):
        raise ValueError("ra_allreduce_bulk_noalloc: chunk_status must be a contiguous int32 tensor of nranks words")
    cs = chunk_status.data_ptr() if chunk_status is not None else None
    st = lib().ra_allreduce_bulk_noalloc(ptr_array([t.data_ptr() for t in sendbufs]),
                                         ptr_array([t.data_ptr() for t in recvbufs]), count,
                                         dtype_code(sendbufs[0]), OP_CODES[op], len(sendbufs), max_sms,
                                         ctypes.c_void_p(cs), ctypes.c_void_p(_stream_ptr(stream) or None))
    if st:
        raise RaError(st, "ra_allreduce_bulk_noalloc")


# ---- layer norm, gradient norm, AdamW ---------------------------------------


class _Torch:
    """What the calls below need of torch, looked up by the first of them: importing this module does not import
    torch, and looking names up again would cost a call more than its checks."""

    codes: dict = {}  # torch dtype -> ra_dtype_t
    f32 = None
    current_stream = None  # device index -> handle of torch's current stream there
    current_device = None  # () -> index of torch's current device

    @classmethod
    def load(cls):
        import torch

        cls.f32 = torch.float32
        cls.current_stream = torch._C._cuda_getCurrentRawStream
        cls.current_device = torch._C._cuda_getDevice
        cls.codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
        return cls


def _float_code(t, what: str) -> int:
    code = (_Torch.codes or _Torch.load().codes).get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}")
    return code


def _stream_on(device: int, stream, what: str) -> int:
    """The stream handle a call whose tensors are on ``device`` goes to: ``stream``, or torch's current one there
    (read without building a Stream object, which would cost as much as the launch). The library launches on the
    current device, so that has to be the tensors'."""
    if _Torch.current_device() != device:
        raise ValueError(f"{what}: the tensors are on cuda:{device}, which is not torch's current CUDA device")
    return _Torch.current_stream(device) if stream is None else _stream_ptr(stream)


def _rows_contiguous(t) -> bool:
    """Whether the rows of a matrix are contiguous, whatever lies between them."""
    return t.stride(1) == 1 or t.shape[1] <= 1


def _row_stride(t, cols: int) -> int:
    return max(t.stride(0), cols) if t.shape[0] <= 1 else t.stride(0)


def _is_vector(t, n: int, dtype, device: int) -> bool:
    """A contiguous tensor of n elements on CUDA device ``device``, or None."""
    return t is None or (t.get_device() == device and t.dtype is dtype and t.numel() == n and t.is_contiguous())


def _address(t):
    return None if t is None else t.data_ptr()


def _check_vectors(what: str, device: int, **vectors) -> None:
    """Raises for the first of ``name=(tensor, count, dtype)`` that is not a vector of that kind on ``device``."""
    for name, (t, n, dtype) in vectors.items():
        if not _is_vector(t, n, dtype, device):
            raise ValueError(f"{what}: {name} must be a contiguous CUDA tensor of {n} elements of {dtype}, "
                             f"on cuda:{device}")


def ra_layernorm_forward(x, weight, bias, y, mean=None, rstd=None, eps: float = 1e-5, stream=None) -> None:
    """Layer norm of the rows of x [rows, cols] into y (which may be x); weight and bias ([cols], of x's type
    or float32, or None), mean and rstd ([rows] float32, kept for the backward pass, or None)."""
    codes = _Torch.codes or _Torch.load().codes
    dtype = x.dtype
    w = weight if weight is not None else bias
    wdtype = dtype if w is None else w.dtype
    shape = x.shape
    dense = x.is_contiguous() and y.is_contiguous()
    device = x.get_device()
    if not (device >= 0 and y.get_device() == device and len(shape) == 2 and y.shape == shape and y.dtype is dtype
            and (dense or (_rows_contiguous(x) and _rows_contiguous(y)))):
        raise ValueError("ra_layernorm_forward: x and y must be 2-D CUDA tensors of one shape, dtype and device, "
                         "rows contiguous")
    if dtype not in codes or wdtype not in codes:
        raise TypeError(f"ra_layernorm_forward: unsupported dtype {dtype} with weights of {wdtype}")
    rows, cols = shape
    f32 = _Torch.f32
    if not (_is_vector(weight, cols, wdtype, device) and _is_vector(bias, cols, wdtype, device)
            and _is_vector(mean, rows, f32, device) and _is_vector(rstd, rows, f32, device)):
        _check_vectors("ra_layernorm_forward", device, weight=(weight, cols, wdtype), bias=(bias, cols, wdtype),
                       mean=(mean, rows, f32), rstd=(rstd, rows, f32))
    st = (_lib or lib()).ra_layernorm_forward(
        x.data_ptr(), cols if dense else _row_stride(x, cols), _address(weight), _address(bias), y.data_ptr(),
        cols if dense else _row_stride(y, cols), _address(mean), _address(rstd), rows, cols, eps, codes[dtype],
        codes[wdtype], _stream_on(device, stream, "ra_layernorm_forward"))
    if st:
        raise RaError(st, "ra_layernorm_forward")


def ra_layernorm_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace ra_layernorm_backward needs."""
    return lib().ra_layernorm_workspace(rows, cols)


def ra_layernorm_backward(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, workspace=None,
                          accumulate: bool = False, stream=None) -> None:
    """Gradients of layer norm: dx [rows, cols] (may be dy or x), and the sums over the rows dweight and dbias
    ([cols], of weight's type; None: not wanted), added to what they hold with ``accumulate``. ``workspace``: a
    contiguous CUDA tensor of ra_layernorm_workspace(rows, cols) bytes, needed for the sums."""
    codes = _Torch.codes or _Torch.load().codes
    dtype = x.dtype
    w = weight if weight is not None else dweight if dweight is not None else dbias
    wdtype = dtype if w is None else w.dtype
    shape = x.shape
    dense = x.is_contiguous() and dy.is_contiguous() and dx.is_contiguous()
    device = x.get_device()
    if not (device >= 0 and dy.get_device() == device and dx.get_device() == device and len(shape) == 2
            and dy.shape == shape and dx.shape == shape and dy.dtype is dtype and dx.dtype is dtype
            and (dense or (_rows_contiguous(x) and _rows_contiguous(dy) and _rows_contiguous(dx)))):
        raise ValueError("ra_layernorm_backward: x, dy and dx must be 2-D CUDA tensors of one shape, dtype and "
                         "device, rows contiguous")
    if dtype not in codes or wdtype not in codes:
        raise TypeError(f"ra_layernorm_backward: unsupported dtype {dtype} with weights of {wdtype}")
    rows, cols = shape
    f32 = _Torch.f32
    if mean is None or rstd is None or not (
            _is_vector(weight, cols, wdtype, device) and _is_vector(dweight, cols, wdtype, device)
            and _is_vector(dbias, cols, wdtype, device) and _is_vector(mean, rows, f32, device)
            and _is_vector(rstd, rows, f32, device)
            and (workspace is None or (workspace.get_device() == device and workspace.is_contiguous()))):
        if mean is None or rstd is None:
            raise ValueError("ra_layernorm_backward: mean and rstd are needed, as ra_layernorm_forward stored them")
        _check_vectors("ra_layernorm_backward", device, weight=(weight, cols, wdtype), dweight=(dweight, cols, wdtype),
                       dbias=(dbias, cols, wdtype), mean=(mean, rows, f32), rstd=(rstd, rows, f32))
        raise ValueError(f"ra_layernorm_backward: workspace must be a contiguous CUDA tensor, on cuda:{device}")
    st = (_lib or lib()).ra_layernorm_backward(
        dy.data_ptr(), cols if dense else _row_stride(dy, cols), x.data_ptr(), cols if dense else _row_stride(x, cols),
        _address(weight), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), cols if dense else _row_stride(dx, cols),
        _address(dweight), _address(dbias), accumulate, rows, cols, codes[dtype], codes[wdtype], _address(workspace),
        0 if workspace is None else workspace.nbytes, _stream_on(device, stream, "ra_layernorm_backward"))
    if st:
        raise RaError(st, "ra_layernorm_backward")


def _same_type(tensors, what: str, device: int):
    """Raises unless the tensors are contiguous, of one dtype and on CUDA device ``device``."""
    dt = tensors[0].dtype if tensors else None
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{what}: every tensor must be a contiguous CUDA tensor")
        if t.get_device() != device:
            raise ValueError(f"{what}: all tensors must be on one device")
        if t.dtype != dt:
            raise ValueError(f"{what}: all tensors must share one dtype")


class GradTensors:
    """A list of gradient tensors, checked once: their addresses and counts, and the tensors themselves (kept
    alive). Its values are read at every call; the list itself is fixed."""

    def __init__(self, grads):
        self.tensors = list(grads)
        self.device = self.tensors[0].get_device() if self.tensors else None
        _same_type(self.tensors, "grad_tensors", self.device)
        self.dtype = _float_code(self.tensors[0], "grad_tensors") if self.tensors else 0
        n = len(self.tensors)
        self.addresses = (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in self.tensors])
        self.counts = (ctypes.c_size_t * max(n, 1))(*[t.numel() for t in self.tensors])


def grad_tensors(grads) -> GradTensors:
    """The list that ra_grad_norm takes, checked once."""
    return GradTensors(grads)


def ra_grad_norm_workspace() -> int:
    """Bytes of workspace ra_grad_norm needs (zeroed before its first use)."""
    return lib().ra_grad_norm_workspace()


def ra_grad_norm(grads, max_norm: float, out, workspace, prescale: float = 1.0, stream=None) -> None:
    """The 2-norm of all gradients (a grad_tensors() list, or tensors of one dtype) into out[0], and the factor
    that clips it to max_norm into out[1]: out[1:] is ra_adamw's grad_scale. ``workspace``: a CUDA tensor of
    ra_grad_norm_workspace() bytes, zeroed once."""
    g = grads if isinstance(grads, GradTensors) else GradTensors(grads)
    f32 = _Torch.f32 or _Torch.load().f32
    device = out.get_device() if g.device is None and out is not None else g.device
    if (out is None or workspace is None or not (out.is_cuda and _is_vector(out, 2, f32, device))
            or not (workspace.get_device() == device and workspace.is_contiguous())):
        raise ValueError("ra_grad_norm: out must be a contiguous CUDA tensor of 2 float32, workspace a contiguous CUDA "
                         "tensor, both on the gradients' device")
    st = (_lib or lib()).ra_grad_norm(g.addresses, g.counts, len(g.tensors), g.dtype, prescale, max_norm,
                                      out.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                                      _stream_on(device, stream, "ra_grad_norm"))
    if st:
        raise RaError(st, "ra_grad_norm")


class AdamwTensors:
    """The tensors of an AdamW step, checked once: the C table of their addresses, counts and weight decays,
    and the tensors themselves (kept alive)."""

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, exp_avg_scales=None, exp_avg_sq_scales=None,
                 weight_decay=0.0, copies=None):
        import torch

        what = "adamw_tensors"
        params = list(params)
        n = len(params)
        lists = {"params": params, "grads": list(grads), "exp_avgs": list(exp_avgs),
                 "exp_avg_sqs": list(exp_avg_sqs)}
        eight = exp_avg_scales is not None or exp_avg_sq_scales is not None
        if eight:
            if exp_avg_scales is None or exp_avg_sq_scales is None:
                raise ValueError(f"{what}: 8-bit moments need both lists of scales")
            lists["exp_avg_scales"], lists["exp_avg_sq_scales"] = list(exp_avg_scales), list(exp_avg_sq_scales)
        if copies is not None:
            lists["copies"] = list(copies)
        decay = list(weight_decay) if hasattr(weight_decay, "__iter__") else [weight_decay] * n
        if len(decay) != n or any(len(v) != n for v in lists.values()):
            raise ValueError(f"{what}: every list must have one entry per parameter")
        self.device = params[0].get_device() if n else None
        for name, tensors in lists.items():
            _same_type(tensors, f"{what}: {name}", self.device)
            for t, p in zip(tensors, params):
                want = -(-p.numel() // RA_ADAMW_BLOCK) if name.endswith("scales") else p.numel()
                if t.numel() != want:
                    raise ValueError(f"{what}: {name} must match the parameters' sizes")
        for name in ("exp_avgs", "exp_avg_sqs"):
            for t in lists[name][:1]:
                if t.dtype not in ((torch.float8_e4m3fn, torch.uint8) if eight else (torch.float32,)):
                    raise TypeError(f"{what}: {name} must be " +
                                    ("float8_e4m3fn or uint8" if eight else "float32") + f", not {t.dtype}")
        for name in ("exp_avg_scales", "exp_avg_sq_scales"):
            for t in lists.get(name, [])[:1]:
                if t.dtype != torch.float32:
                    raise TypeError(f"{what}: {name} must be float32")
        self.lists = lists
        self.state = RA_STATE_E4M3 if eight else RA_STATE_F32
        self.param_dtype = _float_code(params[0], what) if n else 0
        self.grad_dtype = _float_code(lists["grads"][0], what) if n else 0
        self.copy_dtype = _float_code(lists["copies"][0], what) if n and copies is not None else 0
        self.table = (AdamwTensor * max(n, 1))()
        fields = (("param", "params"), ("grad", "grads"), ("exp_avg", "exp_avgs"), ("exp_avg_sq", "exp_avg_sqs"),
                  ("exp_avg_scale", "exp_avg_scales"), ("exp_avg_sq_scale", "exp_avg_sq_scales"), ("copy", "copies"))
        for field, name in fields:
            for entry, t in zip(self.table, lists.get(name, ())):
                setattr(entry, field, t.data_ptr() or None)
        for entry, p, wd in zip(self.table, params, decay):
            entry.count, entry.weight_decay = p.numel(), wd


def adamw_tensors(params, grads, exp_avgs, exp_avg_sqs, exp_avg_scales=None, exp_avg_sq_scales=None,
                  weight_decay=0.0, copies=None) -> AdamwTensors:
    """The list that ra_adamw takes, checked once. Moments: float32, or, with both lists of scales
    (ceil(n / RA_ADAMW_BLOCK) float32 for a tensor of n), float8_e4m3fn (exp_avg_sqs then hold square roots).
    ``weight_decay``: one number or one per parameter. ``copies``: low-precision copies of the parameters to
    write along."""
    return AdamwTensors(params, grads, exp_avgs, exp_avg_sqs, exp_avg_scales, exp_avg_sq_scales, weight_decay,
                        copies)


def ra_adamw(tensors: AdamwTensors, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999,
             eps: float = 1e-8, grad_scale=None, seed: int = 0, stream=None) -> None:
    """One AdamW step over an adamw_tensors() list. ``step`` counts from 1. ``grad_scale``: a float32 CUDA
    tensor of one element the gradients are multiplied by (out[1:] of ra_grad_norm); not finite: nothing is
    written. ``seed``: of the stochastic rounding of 8-bit moments."""
    params = tensors.lists["params"]
    if not params:
        return
    if not _is_vector(grad_scale, 1, _Torch.f32 or _Torch.load().f32, tensors.device):
        raise ValueError("ra_adamw: grad_scale must be a CUDA tensor of one float32, on the parameters' device")
    opts = AdamwOptions(lr, beta1, beta2, eps, step, _address(grad_scale), tensors.state, tensors.copy_dtype, seed)
    st = (_lib or lib()).ra_adamw(tensors.table, len(params), tensors.param_dtype, tensors.grad_dtype,
                                  ctypes.byref(opts), _stream_on(tensors.device, stream, "ra_adamw"))
    if st:
        raise RaError(st, "ra_adamw")
