"""Python binding of libq4k.so: packed GGUF Q4_K dequant-matmul on MI355X.

Argument marshalling only.  Every step of the product runs in the HIP kernels
of ``libq4k.so``; PyTorch provides device memory and the current stream.  If
the library has not been built this module raises on first use: there is no
CPU fallback.

    y = matmul(w_packed, x)           # w_packed: uint8 [N, K/256*144] on cuda
                                      # x: float32 [M, K] on cuda -> y [M, N]
    matmul_batched([(w, x, y), ...])  # one launch per kernel family
    call = prepare_batched([(w, x, y), ...])  # validate once ...
    call()                                    # ... launch many times (same buffers)
    index, value = matmul_argmax(w, x)  # greedy selection on the device: int32 [M], float32 [M]
    h = matmul_swiglu(w_gate, w_up, x)  # silu(x.Wg^T) * (x.Wu^T), the down projection's input
    ws = load_q4k("model.gguf")         # Q4_K tensors of a GGUF file, bytes unchanged, on the device

    r = moe_route(router_logits, top_k)  # experts, weights and the groups of a mixture-of-experts layer
    h = matmul_grouped_swiglu(w_gate, w_up, x, r.offsets, r.rows, x_div=top_k)  # w: uint8 [E, N, K/256*144]
    y = matmul_grouped_combine(w_down, h, r)   # each token's weighted sum over its experts
    a = Adjustment(history=recent, repetition=r, mask=grammar)  # penalties, biases, allowed tokens
    index, value = matmul_argmax(w, x, adjustment=a)  # greedy selection under them

A call runs on the current stream, or on ``stream`` (a torch stream or a raw
handle); the outputs that it makes come from that stream's memory, as they would
inside ``torch.cuda.stream(stream)``.

Names and semantics mirror include/q4k.h, include/q4k_moe.h, include/q4k_select.h and include/q4a.h.
"""
from __future__ import annotations

import ctypes
import os
from typing import Iterable, NamedTuple, Optional, Sequence, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_PKG, "libq4k.so")

BLOCK_WEIGHTS = 256
BLOCK_BYTES = 144
MAX_BATCH = 32
INT_MAX = 2 ** 31 - 1  # the library counts in int; ctypes would keep a longer number's low 32 bits

OK = 0
ERR_NULL = -1
ERR_BAD_DIM = -2
ERR_LAUNCH = -3
ERR_ALIGN = -4
ERR_DEVICE = -5
ERR_ALLOC = -6
ERR_FORMAT = -7
ERR_IO = -8
ERR_SCRATCH = -9
NOALLOC_SCRATCH_BYTES = 128 << 20
GGUF_TYPE_Q4_K = 12

PATH_AUTO = 0
PATH_DECODE = 1
PATH_PREFILL = 2
PATH_GEMV = 3

# Exported symbols of libq4k.so, as declared in the headers under include/.
EXPORTED = ("q4k_matmul", "q4k_matmul_batched", "q4k_matmul_path", "q4k_matmul_batched_path",
            "q4k_matmul_batched_noalloc", "q4a_matmul", "q4a_matmul_batched",
            "q4k_matmul_argmax", "q4k_matmul_swiglu", "q4k_gguf_list", "q4k_select_path", "q4k_strerror",
            "q4k_version", "q4k_moe_route", "q4k_moe_group", "q4k_matmul_grouped", "q4k_matmul_grouped_swiglu",
            "q4k_matmul_grouped_combine", "q4k_grouped_tile", "q4k_logits_adjust", "q4k_logits_argmax",
            "q4k_matmul_argmax_adjusted")


class Q4KError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} ({code})" if what else f"{strerror(code)} ({code})")


class _Problem(ctypes.Structure):
    _fields_ = [("w_packed", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int), ("K", ctypes.c_int)]


class _Adjustment(ctypes.Structure):
    _fields_ = [("history", ctypes.c_void_p), ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("bias_id", ctypes.c_void_p), ("bias_value", ctypes.c_void_p),
                ("mask", ctypes.c_void_p), ("history_len", ctypes.c_int), ("bias_len", ctypes.c_int)]


class GgufTensor(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 128), ("type", ctypes.c_uint32), ("n_dims", ctypes.c_uint32),
                ("dims", ctypes.c_uint64 * 4), ("offset", ctypes.c_uint64), ("nbytes", ctypes.c_uint64)]


_lib = None


def library() -> ctypes.CDLL:
    """The loaded libq4k.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY_PATH):
        raise ImportError(f"{LIBRARY_PATH} is missing: build it with "
                          "`python -m gguf_q4_dequant_amd.build` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIBRARY_PATH)
    vp, ci = ctypes.c_void_p, ctypes.c_int
    lib.q4k_matmul.argtypes = [vp, vp, vp, ci, ci, ci, vp]
    lib.q4k_matmul.restype = ci
    lib.q4k_matmul_path.argtypes = [vp, vp, vp, ci, ci, ci, ci, vp]
    lib.q4k_matmul_path.restype = ci
    lib.q4k_matmul_batched.argtypes = [ctypes.POINTER(_Problem), ci, ci, vp]
    lib.q4k_matmul_batched.restype = ci
    lib.q4k_matmul_batched_path.argtypes = [ctypes.POINTER(_Problem), ci, ci, ci, vp]
    lib.q4k_matmul_batched_path.restype = ci
    lib.q4k_matmul_batched_noalloc.argtypes = [ctypes.POINTER(_Problem), ci, ci, vp]
    lib.q4k_matmul_batched_noalloc.restype = ci
    lib.q4k_matmul_argmax.argtypes = [vp, vp, ci, ci, ci, vp, vp, vp]
    lib.q4k_matmul_argmax.restype = ci
    lib.q4k_matmul_swiglu.argtypes = [vp, vp, vp, vp, ci, ci, ci, vp]
    lib.q4k_matmul_swiglu.restype = ci
    lib.q4a_matmul.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, vp]
    lib.q4a_matmul.restype = ci
    lib.q4a_matmul_batched.argtypes = [ctypes.POINTER(_QaProblem), ci, ci, vp]
    lib.q4a_matmul_batched.restype = ci
    cf, adj = ctypes.c_float, ctypes.POINTER(_Adjustment)
    lib.q4k_moe_route.argtypes = [vp, vp, ci, ci, ci, ci, cf, vp, vp, vp, vp, vp]
    lib.q4k_moe_route.restype = ci
    lib.q4k_moe_group.argtypes = [vp, ci, ci, vp, vp, vp]
    lib.q4k_moe_group.restype = ci
    lib.q4k_matmul_grouped.argtypes = [vp, vp, ci, vp, vp, vp, ci, ci, ci, ci, vp]
    lib.q4k_matmul_grouped.restype = ci
    lib.q4k_matmul_grouped_swiglu.argtypes = [vp, vp, vp, ci, vp, vp, vp, ci, ci, ci, ci, vp]
    lib.q4k_matmul_grouped_swiglu.restype = ci
    lib.q4k_matmul_grouped_combine.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, vp]
    lib.q4k_matmul_grouped_combine.restype = ci
    lib.q4k_grouped_tile.argtypes = [ci, ci, ci, ci, ci, ctypes.POINTER(ci)]
    lib.q4k_grouped_tile.restype = ci
    lib.q4k_logits_adjust.argtypes = [vp, vp, adj, ci, ci, vp]
    lib.q4k_logits_adjust.restype = ci
    lib.q4k_logits_argmax.argtypes = [vp, adj, ci, ci, vp, vp, vp]
    lib.q4k_logits_argmax.restype = ci
    lib.q4k_matmul_argmax_adjusted.argtypes = [vp, vp, adj, ci, ci, ci, vp, vp, vp]
    lib.q4k_matmul_argmax_adjusted.restype = ci
    lib.q4k_gguf_list.argtypes = [ctypes.c_char_p, ctypes.POINTER(GgufTensor), ci, ctypes.POINTER(ci)]
    lib.q4k_gguf_list.restype = ci
    lib.q4k_select_path.argtypes = [ci, ci, ci]
    lib.q4k_select_path.restype = ci
    lib.q4k_strerror.argtypes = [ci]
    lib.q4k_strerror.restype = ctypes.c_char_p
    lib.q4k_version.argtypes = []
    lib.q4k_version.restype = ci
    _lib = lib
    return lib


def strerror(code: int) -> str:
    return library().q4k_strerror(int(code)).decode()


def version() -> int:
    return library().q4k_version()


def select_path(M: int, N: int, K: int) -> int:
    return library().q4k_select_path(M, N, K)


def _stream_handle(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(like, shape, dtype, stream):
    """An output for a call on ``stream``, on like's device and from that stream's
    memory: memory of the current stream may be what was freed there a moment
    ago, and still be in use by kernels that have not run.  (The callers whose
    kernels take a few microseconds make theirs themselves where ``stream`` is None.)"""
    import torch
    if stream is None or not like.is_cuda:
        return like.new_empty(shape, dtype=dtype)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_handle(stream)
        stream = torch.cuda.ExternalStream(handle, device=like.device) if handle else torch.cuda.default_stream(like.device)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _check_operands(w, x, y):
    import torch
    if w.dtype != torch.uint8 or x.dtype != torch.float32 or y.dtype != torch.float32:
        raise TypeError("expected w uint8, x float32, y float32")
    for name, t in (("w", w), ("x", x), ("y", y)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if x.dim() != 2 or y.dim() != 2:
        raise ValueError("x must be [M, K] and y [M, N]")
    M, K = x.shape
    if y.shape[0] != M:
        raise ValueError("x and y disagree on M")
    N = y.shape[1]
    if K % BLOCK_WEIGHTS != 0:
        raise Q4KError(ERR_BAD_DIM, f"K={K}")
    if w.numel() != N * (K // BLOCK_WEIGHTS) * BLOCK_BYTES:
        raise ValueError(f"w has {w.numel()} bytes, expected N*K/256*144 = "
                         f"{N * (K // BLOCK_WEIGHTS) * BLOCK_BYTES}")
    return M, N, K


def matmul(w, x, y=None, path: int = PATH_AUTO, stream=None):
    """y[M, N] = x[M, K] . dequant(w)^T, w packed Q4_K bytes of an [N, K] matrix.

    ``y`` is allocated when not given (N taken from w's leading dimension)."""
    import torch
    if y is None:
        if w.dim() != 2:
            raise ValueError("pass y, or w shaped [N, K/256*144]")
        y = _new(x, (x.shape[0], w.shape[0]), torch.float32, stream)
    M, N, K = _check_operands(w, x, y)
    lib = library()
    if int(path) == PATH_AUTO:
        rc = lib.q4k_matmul(w.data_ptr(), x.data_ptr(), y.data_ptr(), M, N, K, _stream_handle(stream))
    else:
        rc = lib.q4k_matmul_path(w.data_ptr(), x.data_ptr(), y.data_ptr(), M, N, K, int(path),
                                 _stream_handle(stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_matmul")
    return y


def _check_outputs(x, index, value, M):
    """index int32 [M] and value float32 [M], contiguous, on x's device: the
    library writes them from the GPU and cannot check any of this itself."""
    import torch
    if index.dtype != torch.int32 or value.dtype != torch.float32 or index.numel() < M or value.numel() < M:
        raise ValueError("index must be int32 [M] and value float32 [M]")
    for name, t in (("index", index), ("value", value)):
        if not t.is_cuda or t.device != x.device:
            raise ValueError(f"{name} must be a device tensor on {x.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def matmul_argmax(w, x, N: Optional[int] = None, index=None, value=None, stream=None, adjustment=None):
    """(index int32 [M], value float32 [M]): for each row of x, the lowest n with
    the largest y[m, n] of y = x . dequant(w)^T, and that value.  The logits stay
    on the device (library workspace).  N defaults to w's leading dimension.
    With an ``Adjustment`` the choice is made under its penalties, biases and
    mask (as by logits_argmax; a row that has nothing but NaN then gives index -1
    and value -inf, and index 0 and NaN without)."""
    import torch
    if N is None:
        if w.dim() != 2:
            raise ValueError("pass N, or w shaped [N, K/256*144]")
        N = w.shape[0]
    if x.dim() != 2 or x.dtype != torch.float32 or w.dtype != torch.uint8:
        raise TypeError("expected w uint8 and x float32 [M, K]")
    if not (w.is_cuda and x.is_cuda and w.is_contiguous() and x.is_contiguous()):
        raise ValueError("w and x must be contiguous device tensors")
    M, K = x.shape
    if K % BLOCK_WEIGHTS != 0:
        raise Q4KError(ERR_BAD_DIM, f"K={K}")
    if w.numel() != N * (K // BLOCK_WEIGHTS) * BLOCK_BYTES:
        raise ValueError(f"w has {w.numel()} bytes, expected N*K/256*144 = "
                         f"{N * (K // BLOCK_WEIGHTS) * BLOCK_BYTES}")
    if index is None:
        index = _new(x, M, torch.int32, stream)
    if value is None:
        value = _new(x, M, torch.float32, stream)
    _check_outputs(x, index, value, M)
    if adjustment is not None:
        dev = x.get_device()
        if w.get_device() != dev:
            raise ValueError(f"w must be on cuda:{dev}, as x is")
        rc = library().q4k_matmul_argmax_adjusted(w.data_ptr(), x.data_ptr(), adjustment._checked(dev, M, N), M, N, K,
                                                  index.data_ptr(), value.data_ptr(), _stream_for(dev, stream))
        if rc != OK:
            raise Q4KError(rc, "q4k_matmul_argmax_adjusted")
        return index, value
    rc = library().q4k_matmul_argmax(w.data_ptr(), x.data_ptr(), M, N, K, index.data_ptr(),
                                     value.data_ptr(), _stream_handle(stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_matmul_argmax")
    return index, value


def _checked_tensor(name, t, dtype, shape, dev):
    """t is a contiguous tensor of this dtype and shape on GPU number dev; its address."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be shaped {list(shape)}, not {list(t.shape)}")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be a device tensor on cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _stream_for(dev, stream) -> int:
    """The handle of the given stream, or of the current one; the tensors (on GPU
    number dev) have to be on the current device, whose context the library
    launches in."""
    import torch
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream_handle(stream)


class Adjustment:
    """What is applied to logits [M, N] before a token is chosen (include/q4k_select.h);
    every part is optional, all are device tensors:

    history int32 [M, L]: recent tokens of each sequence, entries outside [0, N)
        (padding) count for nothing; with it, float32 [M] each:
        repetition: z > 0 ? z / r : z * r for tokens that occur in the history,
        frequency: z - f * (number of occurrences), presence: z - p;
    bias_id int32 [M, B], bias_value float32 [M, B]: added to the named tokens
        (several for one token add up; ids outside [0, N) are skipped);
    mask int32 or uint32 [M, ceil(N / 32)]: token n is allowed where bit n % 32
        of word n / 32 is set, else its logit is -inf.

    The tensors are read by the calls that are given the object, not before."""

    __slots__ = ("history", "repetition", "frequency", "presence", "bias_id", "bias_value", "mask")

    def __init__(self, history=None, repetition=None, frequency=None, presence=None, bias_id=None, bias_value=None,
                 mask=None):
        if (bias_id is None) != (bias_value is None):
            raise ValueError("bias_id and bias_value come together")
        if history is None and not (repetition is None and frequency is None and presence is None):
            raise ValueError("repetition, frequency and presence need a history")
        self.history, self.repetition, self.frequency, self.presence = history, repetition, frequency, presence
        self.bias_id, self.bias_value, self.mask = bias_id, bias_value, mask

    def _checked(self, dev, M, N):
        """The C struct for logits [M, N] on GPU number dev."""
        import torch
        history = repetition = frequency = presence = bias_id = bias_value = mask = None
        L = B = 0
        if self.history is not None:
            if self.history.dim() != 2:
                raise ValueError("history must be int32 [M, L]")
            L = self.history.shape[1]
            history = _checked_tensor("history", self.history, torch.int32, (M, L), dev)
            if self.repetition is not None:
                repetition = _checked_tensor("repetition", self.repetition, torch.float32, (M,), dev)
            if self.frequency is not None:
                frequency = _checked_tensor("frequency", self.frequency, torch.float32, (M,), dev)
            if self.presence is not None:
                presence = _checked_tensor("presence", self.presence, torch.float32, (M,), dev)
        if self.bias_id is not None:
            if self.bias_id.dim() != 2:
                raise ValueError("bias_id must be int32 [M, B]")
            B = self.bias_id.shape[1]
            bias_id = _checked_tensor("bias_id", self.bias_id, torch.int32, (M, B), dev)
            bias_value = _checked_tensor("bias_value", self.bias_value, torch.float32, (M, B), dev)
        if self.mask is not None:
            dtype = torch.uint32 if self.mask.dtype == torch.uint32 else torch.int32
            mask = _checked_tensor("mask", self.mask, dtype, (M, (N + 31) // 32), dev)
        return _Adjustment(history, repetition, frequency, presence, bias_id, bias_value, mask, L, B)


def _checked_logits(logits):
    import torch
    shape, dev = logits.shape, logits.get_device()
    if len(shape) != 2 or logits.dtype is not torch.float32:
        raise TypeError("logits must be float32 [M, N]")
    if shape[0] > INT_MAX or shape[1] > INT_MAX:
        raise Q4KError(ERR_BAD_DIM, f"logits {list(shape)}")
    if dev < 0 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous device tensor")
    return shape[0], shape[1], dev


def logits_adjust(logits, adjustment, out=None, stream=None):
    """The logits float32 [M, N] under an ``Adjustment`` (penalties, biases, -inf
    where the mask forbids), in a new tensor or in ``out`` (which may be logits)."""
    import torch
    M, N, dev = _checked_logits(logits)
    if out is None:
        out = torch.empty_like(logits) if stream is None else _new(logits, (M, N), torch.float32, stream)
    elif out is not logits:
        _checked_tensor("out", out, torch.float32, (M, N), dev)
    rc = library().q4k_logits_adjust(logits.data_ptr(), out.data_ptr(), adjustment._checked(dev, M, N), M, N,
                                     _stream_for(dev, stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_logits_adjust")
    return out


def logits_argmax(logits, adjustment, index=None, value=None, stream=None):
    """(index int32 [M], value float32 [M]): for each row of logits [M, N] the lowest
    allowed token with the largest adjusted logit, and that logit; index -1 and
    value -inf where the mask (or NaN) leaves nothing.  The adjusted logits are
    not written."""
    import torch
    M, N, dev = _checked_logits(logits)
    if index is None and value is None and stream is None:
        index, value = logits.new_empty(M, dtype=torch.int32), logits.new_empty(M)
    else:
        index = _new(logits, M, torch.int32, stream) if index is None else index
        value = _new(logits, M, torch.float32, stream) if value is None else value
        _check_outputs(logits, index, value, M)
    rc = library().q4k_logits_argmax(logits.data_ptr(), adjustment._checked(dev, M, N), M, N, index.data_ptr(),
                                     value.data_ptr(), _stream_for(dev, stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_logits_argmax")
    return index, value


MAX_EXPERTS = 1024
MAX_TOP_K = 64
ROUTE_SIGMOID = 1
ROUTE_NORMALIZE = 2


class Routing(NamedTuple):
    """A routed batch: expert int32 [M, top_k] (-1: none), weight float32 [M, top_k],
    and the groups of its pairs p = m * top_k + j: offsets int32 [E + 1] and
    rows int32 [M * top_k], group e being rows[offsets[e]:offsets[e + 1]]."""
    expert: object
    weight: object
    offsets: object
    rows: object


def moe_route(logits, top_k: int, bias=None, sigmoid: bool = False, normalize: bool = True, scale: float = 1.0,
              out: Optional[Routing] = None, stream=None) -> Routing:
    """Each token's top_k experts, their weights, and the pairs grouped by expert
    (q4k_moe_route).  logits float32 [M, E]; scores are their softmax, or with
    ``sigmoid`` their sigmoid; ``bias`` float32 [E] takes part in the choice
    only; ``normalize`` divides a token's weights by their sum."""
    import torch
    M, E, dev = _checked_logits(logits)
    k = int(top_k)
    if not (1 <= E <= MAX_EXPERTS and 1 <= k <= min(E, MAX_TOP_K)):
        raise Q4KError(ERR_BAD_DIM, f"E={E} top_k={k}")
    bias_ptr = None if bias is None else _checked_tensor("bias", bias, torch.float32, (E,), dev)
    if out is None:
        if stream is None:
            expert, weight = logits.new_empty((M, k), dtype=torch.int32), logits.new_empty((M, k))
            out = Routing(expert, weight, expert.new_empty(E + 1), expert.new_empty(M * k))
        else:
            out = Routing(_new(logits, (M, k), torch.int32, stream), _new(logits, (M, k), torch.float32, stream),
                          _new(logits, E + 1, torch.int32, stream), _new(logits, M * k, torch.int32, stream))
    else:
        _checked_tensor("expert", out.expert, torch.int32, (M, k), dev)
        _checked_tensor("weight", out.weight, torch.float32, (M, k), dev)
        _checked_tensor("offsets", out.offsets, torch.int32, (E + 1,), dev)
        _checked_tensor("rows", out.rows, torch.int32, (M * k,), dev)
    flags = (ROUTE_SIGMOID if sigmoid else 0) | (ROUTE_NORMALIZE if normalize else 0)
    rc = library().q4k_moe_route(logits.data_ptr(), bias_ptr, M, E, k, flags, float(scale), out.expert.data_ptr(),
                                 out.weight.data_ptr(), out.offsets.data_ptr(), out.rows.data_ptr(),
                                 _stream_for(dev, stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_moe_route")
    return out


def moe_group(expert, E: int, stream=None):
    """(offsets int32 [E + 1], rows int32 [P]): the groups of an existing table of
    choices, int32 of any shape with P entries (outside [0, E): in no group)."""
    import torch
    if expert.dtype != torch.int32:
        raise TypeError("expert must be int32")
    if expert.numel() > INT_MAX:
        raise Q4KError(ERR_BAD_DIM, f"P={expert.numel()}")
    if not expert.is_cuda or not expert.is_contiguous():
        raise ValueError("expert must be a contiguous device tensor")
    P, E = expert.numel(), int(E)
    if not 1 <= E <= MAX_EXPERTS:
        raise Q4KError(ERR_BAD_DIM, f"E={E}")
    offsets, rows = _new(expert, E + 1, torch.int32, stream), _new(expert, P, torch.int32, stream)
    rc = library().q4k_moe_group(expert.data_ptr(), P, E, offsets.data_ptr(), rows.data_ptr(),
                                 _stream_for(expert.get_device(), stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_moe_group")
    return offsets, rows


def _grouped_checked(ws, x, offsets, rows, x_div):
    """Validate the operands of a grouped product; returns (P, E, N, K, their GPU,
    addresses of the matrices, of offsets and of rows)."""
    import torch
    w_shape, x_shape = ws[0].shape, x.shape
    if x.dtype is not torch.float32 or len(x_shape) != 2 or len(w_shape) != 3 or ws[0].dtype is not torch.uint8:
        raise TypeError("expected w uint8 [E, N, K/256*144] and x float32 [rows, K]")
    E, N, _ = w_shape
    x_rows, K = x_shape
    P = x_rows * x_div if rows is None else rows.numel()
    if P > INT_MAX or N > INT_MAX or x_div > INT_MAX:
        raise Q4KError(ERR_BAD_DIM, f"P={P} N={N} x_div={x_div}")
    if K % BLOCK_WEIGHTS != 0 or K == 0 or K > INT_MAX:
        raise Q4KError(ERR_BAD_DIM, f"K={K}")
    dev = x.get_device()
    if dev < 0 or not x.is_contiguous():
        raise ValueError("x must be a contiguous device tensor")
    if not 1 <= E <= MAX_EXPERTS:
        raise Q4KError(ERR_BAD_DIM, f"E={E}")
    if x_div < 1:
        raise Q4KError(ERR_BAD_DIM, f"x_div={x_div}")
    shape = (E, N, K // BLOCK_WEIGHTS * BLOCK_BYTES)
    w_ptrs = [_checked_tensor("w", w, torch.uint8, shape, dev) for w in ws]
    offsets_ptr = _checked_tensor("offsets", offsets, torch.int32, (E + 1,), dev)
    if rows is None:
        return P, E, N, K, dev, w_ptrs, offsets_ptr, None
    rows_ptr = _checked_tensor("rows", rows, torch.int32, (P,), dev)
    if (P + x_div - 1) // x_div != x_rows:
        raise ValueError(f"x has {x_rows} rows, expected {P} pairs / x_div {x_div}")
    return P, E, N, K, dev, w_ptrs, offsets_ptr, rows_ptr


def matmul_grouped(w, x, offsets, rows=None, y=None, x_div: int = 1, stream=None):
    """y[p] = x[p // x_div] . dequant(w[e])^T for every pair p = rows[i] of group e
    (offsets[e] <= i < offsets[e + 1]); w uint8 [E, N, K/256*144], y float32
    [P, N].  Rows of pairs in no group are left as they were (in a ``y`` made
    here they hold nothing meaningful).  rows None: pairs already in expert order."""
    import torch
    P, E, N, K, dev, (w_ptr,), offsets_ptr, rows_ptr = _grouped_checked((w,), x, offsets, rows, x_div)
    if y is None:
        y = x.new_empty((P, N)) if stream is None else _new(x, (P, N), torch.float32, stream)
    else:
        _checked_tensor("y", y, torch.float32, (P, N), dev)
    rc = library().q4k_matmul_grouped(w_ptr, x.data_ptr(), x_div, offsets_ptr, rows_ptr, y.data_ptr(), E, P, N, K,
                                      _stream_for(dev, stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_matmul_grouped")
    return y


def matmul_grouped_swiglu(w_gate, w_up, x, offsets, rows=None, out=None, x_div: int = 1, stream=None):
    """out[p] = silu(x[p // x_div] . dequant(w_gate[e])^T) * (x[p // x_div] . dequant(w_up[e])^T)
    for every pair p of group e; arguments as for matmul_grouped."""
    import torch
    P, E, N, K, dev, w_ptrs, offsets_ptr, rows_ptr = _grouped_checked((w_gate, w_up), x, offsets, rows, x_div)
    if out is None:
        out = x.new_empty((P, N)) if stream is None else _new(x, (P, N), torch.float32, stream)
    else:
        _checked_tensor("out", out, torch.float32, (P, N), dev)
    rc = library().q4k_matmul_grouped_swiglu(*w_ptrs, x.data_ptr(), x_div, offsets_ptr, rows_ptr, out.data_ptr(),
                                             E, P, N, K, _stream_for(dev, stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_matmul_grouped_swiglu")
    return out


def matmul_grouped_combine(w, x, routing: Routing, out=None, stream=None):
    """out[m] = sum_j weight[m, j] * (x[m * top_k + j] . dequant(w[expert[m, j]])^T),
    the experts' down projections and each token's weighted sum; x float32
    [M * top_k, K], out float32 [M, N]."""
    import torch
    expert, weight, offsets, rows = routing
    P, E, N, K, dev, (w_ptr,), offsets_ptr, rows_ptr = _grouped_checked((w,), x, offsets, rows, 1)
    choices = expert.shape
    if len(choices) != 2 or choices[0] * choices[1] != P:
        raise ValueError(f"expert must be [M, top_k] with {P} entries")
    M, top_k = choices
    expert_ptr = _checked_tensor("expert", expert, torch.int32, choices, dev)
    weight_ptr = _checked_tensor("weight", weight, torch.float32, choices, dev)
    if out is None:
        out = x.new_empty((M, N)) if stream is None else _new(x, (M, N), torch.float32, stream)
    else:
        _checked_tensor("out", out, torch.float32, (M, N), dev)
    rc = library().q4k_matmul_grouped_combine(w_ptr, x.data_ptr(), expert_ptr, weight_ptr, offsets_ptr, rows_ptr,
                                              out.data_ptr(), E, M, top_k, N, K, _stream_for(dev, stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_matmul_grouped_combine")
    return out


def grouped_tile(E: int, P: int, N: int, K: int, swiglu: bool = False) -> Tuple[int, int]:
    """(rows, parts) of the kernel that a grouped product of these sizes runs: tiles
    of 4, 16, 32 or 48 rows (0: nothing to compute), K split into ``parts`` within
    a workgroup (q4k_grouped_tile)."""
    if max(abs(E), abs(P), abs(N), abs(K)) > INT_MAX:
        raise Q4KError(ERR_BAD_DIM, f"E={E} P={P} N={N} K={K}")
    parts = ctypes.c_int(0)
    rows = library().q4k_grouped_tile(E, P, N, K, int(swiglu), ctypes.byref(parts))
    if rows < 0:
        raise Q4KError(rows, "q4k_grouped_tile")
    return rows, parts.value


def matmul_swiglu(w_gate, w_up, x, out=None, stream=None):
    """out[M, N] = silu(x . dequant(w_gate)^T) * (x . dequant(w_up)^T)."""
    import torch
    if out is None:
        if w_gate.dim() != 2:
            raise ValueError("pass out, or w_gate shaped [N, K/256*144]")
        out = _new(x, (x.shape[0], w_gate.shape[0]), torch.float32, stream)
    M, N, K = _check_operands(w_gate, x, out)
    _check_operands(w_up, x, out)
    rc = library().q4k_matmul_swiglu(w_gate.data_ptr(), w_up.data_ptr(), x.data_ptr(), out.data_ptr(), M, N, K,
                                     _stream_handle(stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_matmul_swiglu")
    return out


def raw_matmul_swiglu(wg_ptr: int, wu_ptr: int, x_ptr: int, out_ptr: int, M: int, N: int, K: int,
                      stream: Optional[int] = None) -> int:
    """Direct C-ABI call of q4k_matmul_swiglu with raw device addresses; returns the status."""
    return library().q4k_matmul_swiglu(wg_ptr, wu_ptr, x_ptr, out_ptr, M, N, K, stream)


def raw_matmul_argmax(w_ptr: int, x_ptr: int, M: int, N: int, K: int, index_ptr: int,
                      value_ptr: Optional[int], stream: Optional[int] = None) -> int:
    """Direct C-ABI call of q4k_matmul_argmax with raw device addresses; returns the status."""
    return library().q4k_matmul_argmax(w_ptr, x_ptr, M, N, K, index_ptr, value_ptr, stream)


def matmul_batched(problems: Sequence[Tuple], path: int = PATH_AUTO, stream=None):
    """Run several (w, x, y) products that share M with one launch per kernel family."""
    problems = list(problems)
    if not problems:
        raise Q4KError(ERR_BAD_DIM, "empty batch")
    arr = (_Problem * len(problems))()
    M = None
    for i, (w, x, y) in enumerate(problems):
        m, n, k = _check_operands(w, x, y)
        if M is None:
            M = m
        elif m != M:
            raise ValueError("all problems of a batch share M")
        arr[i] = _Problem(w.data_ptr(), x.data_ptr(), y.data_ptr(), n, k)
    lib = library()
    if int(path) == PATH_AUTO:
        rc = lib.q4k_matmul_batched(arr, len(problems), M, _stream_handle(stream))
    else:
        rc = lib.q4k_matmul_batched_path(arr, len(problems), M, int(path), _stream_handle(stream))
    if rc != OK:
        raise Q4KError(rc, "q4k_matmul_batched")
    return [p[2] for p in problems]


class PreparedBatch:
    """A validated batched call on fixed buffers: the argument array is built
    once and every call goes straight to ``q4k_matmul_batched_path``.  The
    tensors must stay alive (and in place) while the object is used."""

    def __init__(self, problems: Sequence[Tuple], path: int = PATH_AUTO):
        problems = list(problems)
        if not problems:
            raise Q4KError(ERR_BAD_DIM, "empty batch")
        self._keep = problems
        self._arr = (_Problem * len(problems))()
        M = None
        for i, (w, x, y) in enumerate(problems):
            m, n, k = _check_operands(w, x, y)
            if M is None:
                M = m
            elif m != M:
                raise ValueError("all problems of a batch share M")
            self._arr[i] = _Problem(w.data_ptr(), x.data_ptr(), y.data_ptr(), n, k)
        self.M, self.count, self.path = M, len(problems), int(path)
        lib = library()
        if self.path == PATH_AUTO:
            fn = lib.q4k_matmul_batched
            self._call = lambda st: fn(self._arr, self.count, self.M, st)
        else:
            fn = lib.q4k_matmul_batched_path
            self._call = lambda st: fn(self._arr, self.count, self.M, self.path, st)

    def __call__(self, stream=None) -> None:
        rc = self._call(_stream_handle(stream))
        if rc != OK:
            raise Q4KError(rc, "q4k_matmul_batched")


def prepare_batched(problems: Sequence[Tuple], path: int = PATH_AUTO) -> PreparedBatch:
    """Validate a batch of (w, x, y) once; the returned object launches it."""
    return PreparedBatch(problems, path)


def raw_matmul(w_ptr: int, x_ptr: int, y_ptr: int, M: int, N: int, K: int,
               path: int = PATH_AUTO, stream: Optional[int] = None) -> int:
    """Direct C-ABI call with raw device addresses; returns the status code."""
    return library().q4k_matmul_path(w_ptr, x_ptr, y_ptr, M, N, K, path, stream)


def raw_matmul_batched(items: Iterable[Tuple[int, int, int, int, int]], M: int,
                       path: int = PATH_AUTO, stream: Optional[int] = None) -> int:
    """Direct C-ABI batched call; items are (w_ptr, x_ptr, y_ptr, N, K); returns the status."""
    items = list(items)
    arr = (_Problem * max(len(items), 1))()
    for i, (w, x, y, n, k) in enumerate(items):
        arr[i] = _Problem(w, x, y, n, k)
    return library().q4k_matmul_batched_path(arr, len(items), M, path, stream)


def raw_matmul_batched_noalloc(items: Iterable[Tuple[int, int, int, int, int]], M: int,
                               stream: Optional[int] = None) -> int:
    """Direct call of q4k_matmul_batched_noalloc (no device allocation; scratch
    from the library's fixed per-GPU array); items are (w_ptr, x_ptr, y_ptr, N,
    K); returns the status."""
    items = list(items)
    arr = (_Problem * max(len(items), 1))()
    for i, (w, x, y, n, k) in enumerate(items):
        arr[i] = _Problem(w, x, y, n, k)
    return library().q4k_matmul_batched_noalloc(arr, len(items), M, stream)


Q4A_GROUP = 64


def _q4a_checked(w_q, scales, biases, x, y, stream=None):
    """Validate one q4a product's tensors (shapes, dtypes, device, contiguity);
    returns (y, M, N, K) with y allocated if None."""
    import torch
    if x.dtype != torch.float32 or x.dim() != 2:
        raise TypeError("x must be float32 [M, K]")
    M, K = x.shape
    if K % Q4A_GROUP != 0:
        raise Q4KError(ERR_BAD_DIM, f"K={K}")
    if scales.dtype != torch.float16 or biases.dtype != torch.float16:
        raise TypeError("scales and biases must be float16")
    if w_q.dtype not in (torch.uint32, torch.int32, torch.uint8):
        raise TypeError("w_q must hold 32-bit words (uint32/int32) or their bytes (uint8)")
    N = scales.shape[0] if scales.dim() == 2 else scales.numel() // (K // Q4A_GROUP)
    if w_q.numel() * w_q.element_size() != N * K // 2 or scales.numel() != N * K // 64 or \
            biases.numel() != N * K // 64:
        raise ValueError(f"w_q must hold N*K/2 = {N * K // 2} bytes and scales/biases N*K/64 = {N * K // 64} values")
    if y is None:
        y = _new(x, (M, N), torch.float32, stream)
    if y.dtype != torch.float32 or tuple(y.shape) != (M, N):
        raise ValueError("y must be float32 [M, N]")
    for name, t in (("w_q", w_q), ("scales", scales), ("biases", biases), ("x", x), ("y", y)):
        if not t.is_cuda or t.device != x.device:
            raise ValueError(f"{name} must be a device tensor on {x.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return y, M, N, K


def q4a_matmul(w_q, scales, biases, x, y=None, stream=None):
    """y[M, N] = x[M, K] . dequant(W)^T for W in the affine 4-bit group layout
    of include/q4a.h: w_q uint32 [N, K/8] (or uint8 [N, K/2]), scales and
    biases float16 [N, K/64], w = s * q + b per group of 64."""
    y, M, N, K = _q4a_checked(w_q, scales, biases, x, y, stream)
    rc = library().q4a_matmul(w_q.data_ptr(), scales.data_ptr(), biases.data_ptr(), x.data_ptr(), y.data_ptr(),
                              M, N, K, _stream_handle(stream))
    if rc != OK:
        raise Q4KError(rc, "q4a_matmul")
    return y


class _QaProblem(ctypes.Structure):
    _fields_ = [("w_q", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("N", ctypes.c_int), ("K", ctypes.c_int)]


def q4a_matmul_batched(problems, stream=None):
    """Several q4a products sharing M in one call (q4a_matmul_batched):
    problems is a list of (w_q, scales, biases, x, y) with y preallocated
    float32 [M, N_i]; returns the list of y."""
    problems = list(problems)
    if not 1 <= len(problems) <= MAX_BATCH:
        raise Q4KError(ERR_BAD_DIM, f"{len(problems)} problems")
    arr = (_QaProblem * len(problems))()
    Ms = set()
    ys = []
    for i, (w_q, scales, biases, x, y) in enumerate(problems):
        if y is None:
            raise ValueError("batched q4a products need their y tensors")
        y, M, N, K = _q4a_checked(w_q, scales, biases, x, y)
        Ms.add(M)
        arr[i] = _QaProblem(w_q.data_ptr(), scales.data_ptr(), biases.data_ptr(), x.data_ptr(), y.data_ptr(), N, K)
        ys.append(y)
    if len(Ms) != 1:
        raise ValueError("every problem of a batch has the same M")
    rc = library().q4a_matmul_batched(arr, len(problems), Ms.pop(), _stream_handle(stream))
    if rc != OK:
        raise Q4KError(rc, "q4a_matmul_batched")
    return ys


def raw_q4a_matmul_batched(items, M: int, stream: Optional[int] = None) -> int:
    """Direct C-ABI call of q4a_matmul_batched; items are (wq_ptr, s_ptr,
    b_ptr, x_ptr, y_ptr, N, K); returns the status."""
    items = list(items)
    arr = (_QaProblem * max(len(items), 1))()
    for i, (w, sc, bi, x, y, n, k) in enumerate(items):
        arr[i] = _QaProblem(w, sc, bi, x, y, n, k)
    return library().q4a_matmul_batched(arr, len(items), M, stream)


def raw_q4a_matmul(wq_ptr: int, s_ptr: int, b_ptr: int, x_ptr: int, y_ptr: int, M: int, N: int, K: int,
                   stream: Optional[int] = None) -> int:
    """Direct C-ABI call of q4a_matmul with raw device addresses; returns the status."""
    return library().q4a_matmul(wq_ptr, s_ptr, b_ptr, x_ptr, y_ptr, M, N, K, stream)


def gguf_tensors(path) -> list:
    """Tensor directory of a GGUF file (q4k_gguf_list): a list of dicts with
    name, type, dims (innermost first), offset (absolute) and nbytes."""
    lib = library()
    n = ctypes.c_int(0)
    p = os.fsencode(path)
    rc = lib.q4k_gguf_list(p, None, 0, ctypes.byref(n))
    if rc != OK:
        raise Q4KError(rc, f"q4k_gguf_list({path!r})")
    arr = (GgufTensor * max(n.value, 1))()
    rc = lib.q4k_gguf_list(p, arr, n.value, ctypes.byref(n))
    if rc != OK:
        raise Q4KError(rc, f"q4k_gguf_list({path!r})")
    return [{"name": e.name.decode(), "type": int(e.type), "dims": tuple(int(d) for d in e.dims[:e.n_dims]),
             "offset": int(e.offset), "nbytes": int(e.nbytes)} for e in arr[:n.value]]


def load_q4k(path, names=None, device=None) -> dict:
    """The Q4_K tensors of a GGUF file (all, or those in ``names``) uploaded with
    their bytes unchanged into one device buffer: name -> uint8 view shaped
    [N, K/256*144] (N = product of dims[1:], K = dims[0]), ready for matmul."""
    import numpy as np
    import torch
    entries = [e for e in gguf_tensors(path) if e["type"] == GGUF_TYPE_Q4_K]
    if names is not None:
        want = set(names)
        missing = want - {e["name"] for e in entries}
        if missing:
            raise KeyError(f"no Q4_K tensor named {sorted(missing)} in {path}")
        entries = [e for e in entries if e["name"] in want]
    offs, total = [], 0
    for e in entries:
        offs.append(total)
        total += (e["nbytes"] + 255) // 256 * 256
    arena = torch.empty(max(total, 1), dtype=torch.uint8, device=device or "cuda")
    out = {}
    for e, o in zip(entries, offs):
        data = np.fromfile(path, dtype=np.uint8, count=e["nbytes"], offset=e["offset"])
        view = arena[o:o + e["nbytes"]]
        view.copy_(torch.from_numpy(data))
        rows = e["nbytes"] // (e["dims"][0] // BLOCK_WEIGHTS * BLOCK_BYTES)
        out[e["name"]] = view.view(rows, e["dims"][0] // BLOCK_WEIGHTS * BLOCK_BYTES)
    return out
