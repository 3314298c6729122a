"""ctypes binding of ``libspark_attn.so`` (the C ABI in ``include/spark_attn.h``,
``include/spark_layer.h``, ``include/spark_paged.h``, ``include/spark_score.h``
and ``include/spark_beam.h``).

Argument marshalling only: every step of the block runs in the library's CUDA
kernels.  Tensors are PyTorch CUDA tensors (PyTorch provides device memory and
streams); the functions carry the C entry points' names and check only what
the C side cannot see (tensor devices, dtypes, contiguity and shapes).  The
library must have been built (``decode_attention_block_gb300.build_lib.build``);
importing the binding without it raises instead of falling back to anything.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field

import torch

from .build_lib import LIB_PATH

SPARK_OK = 0
SPARK_PATH_AUTO, SPARK_PATH_GEMV, SPARK_PATH_MMA = 0, 1, 2
SPARK_F32 = 0
SPARK_BF16 = 1
SPARK_FP4 = 2             # pages only
SPARK_FP4_BLOCK_BYTES = 2304
SPARK_SLIDING = 0
SPARK_FULL = 1
SPARK_MAX_BATCH = 1024
SPARK_MAX_TOP = 32
SPARK_MAX_BEAMS = 32
# bits of a workspace's error word (spark_attn_error_word)
SPARK_ERRBIT_TIMEOUT, SPARK_ERRBIT_INDEX, SPARK_ERRBIT_PAGES = 1, 2, 4

_DTYPE_CODE = {torch.float32: SPARK_F32, torch.bfloat16: SPARK_BF16}


class SparkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {spark_attn_status_string(status)} (status {status})")


class SparkGeom(ctypes.Structure):
    _fields_ = [
        ("hidden", ctypes.c_int32),
        ("n_q", ctypes.c_int32),
        ("n_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("full_rotary_dim", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("full_theta", ctypes.c_float),
        ("sliding_theta", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("scale", ctypes.c_float),
    ]


class SparkLayerWeights(ctypes.Structure):
    _fields_ = [
        ("norm_w", ctypes.c_void_p),
        ("qkv_w", ctypes.c_void_p),
        ("g_w", ctypes.c_void_p),
        ("o_w", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
    ]


class SparkKvLayer(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("capacity", ctypes.c_int64),
        ("ring_capacity", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


class SparkMlpWeights(ctypes.Structure):
    _fields_ = [
        ("norm_w", ctypes.c_void_p),
        ("gate_w", ctypes.c_void_p),
        ("up_w", ctypes.c_void_p),
        ("down_w", ctypes.c_void_p),
        ("intermediate", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


class SparkPagePool(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("n_pages", ctypes.c_int64),
        ("page_size", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


class SparkPagedBatch(ctypes.Structure):
    _fields_ = [
        ("table", ctypes.c_void_p),
        ("q_start", ctypes.c_void_p),
        ("seq_len", ctypes.c_void_p),
        ("n_seqs", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("n_tokens", ctypes.c_int32),
        ("max_q_len", ctypes.c_int32),
    ]


class SparkBeamState(ctypes.Structure):
    _fields_ = [
        ("src", ctypes.c_void_p),
        ("dst", ctypes.c_void_p),
        ("pitch", ctypes.c_int64),
        ("elem", ctypes.c_int32),
        ("push", ctypes.c_void_p),
    ]


# every symbol include/*.h declares, with its ctypes signature
_P = ctypes.c_void_p
_SIGNATURES = {
    "spark_geom_default": (None, [ctypes.POINTER(SparkGeom)]),
    "spark_attn_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(SparkGeom), ctypes.c_int32]),
    "spark_attn_workspace_init": (ctypes.c_int, [_P, ctypes.c_size_t, _P]),
    "spark_attn_error_word": (ctypes.c_int, [_P, ctypes.c_size_t, ctypes.POINTER(ctypes.c_uint32), _P]),
    "spark_attn_decode": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, ctypes.POINTER(SparkLayerWeights),
                                         ctypes.POINTER(SparkKvLayer), ctypes.c_int32,
                                         ctypes.POINTER(ctypes.c_int32), ctypes.c_int32, _P, _P,
                                         ctypes.c_size_t, _P]),
    "spark_attn_prefill": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, ctypes.POINTER(SparkLayerWeights),
                                          ctypes.POINTER(SparkKvLayer), ctypes.c_int32, ctypes.c_int32,
                                          ctypes.c_int32, _P, _P, ctypes.c_size_t, _P]),
    "spark_attn_decode_stack": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, ctypes.c_int32,
                                               ctypes.POINTER(SparkLayerWeights), ctypes.POINTER(SparkKvLayer),
                                               ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                                               ctypes.c_int32, _P, _P, ctypes.c_size_t, _P]),
    "spark_dbg_qkv_rope": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, ctypes.POINTER(SparkLayerWeights),
                                          ctypes.POINTER(SparkKvLayer), ctypes.c_int32,
                                          ctypes.POINTER(ctypes.c_int32), ctypes.c_int32, _P, _P,
                                          ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "spark_dbg_attention": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, ctypes.POINTER(SparkKvLayer),
                                           ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), ctypes.c_int32,
                                           _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "spark_dbg_attention_noalloc": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, ctypes.POINTER(SparkKvLayer),
                                                   ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), ctypes.c_int32,
                                                   _P, _P]),
    "spark_dbg_attention_noalloc_error_word": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), _P]),
    "spark_dbg_gate_oproj": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, _P, _P,
                                            ctypes.POINTER(SparkLayerWeights), ctypes.c_int32, _P,
                                            ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "spark_dbg_wait_timeout": (ctypes.c_int, [_P, ctypes.c_size_t, ctypes.c_uint64, _P]),
    "spark_mlp_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(SparkGeom), ctypes.c_int32, ctypes.c_int32]),
    "spark_mlp_decode": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, ctypes.POINTER(SparkMlpWeights),
                                        ctypes.c_int32, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "spark_head_logits": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, _P, _P, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_int32, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "spark_paged_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(SparkGeom)]),
    "spark_paged_append": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, _P, ctypes.c_int64, ctypes.c_int32,
                                          ctypes.POINTER(SparkPagePool), ctypes.POINTER(SparkPagedBatch), _P,
                                          ctypes.c_size_t, _P]),
    "spark_paged_attention": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, ctypes.c_int64, ctypes.c_int32,
                                             ctypes.POINTER(SparkPagePool), ctypes.c_int32,
                                             ctypes.POINTER(SparkPagedBatch), _P, _P, ctypes.c_size_t, _P]),
    "spark_rope_table": (ctypes.c_int, [ctypes.POINTER(SparkGeom), ctypes.c_int32, ctypes.c_int32, _P, _P]),
    "spark_paged_rope_append": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, _P, _P, ctypes.c_int64, ctypes.c_int32,
                                               ctypes.c_int32, _P, ctypes.c_int32, ctypes.POINTER(SparkPagePool),
                                               ctypes.POINTER(SparkPagedBatch), _P, ctypes.c_int64, _P,
                                               ctypes.c_size_t, _P]),
    "spark_paged_read": (ctypes.c_int, [ctypes.POINTER(SparkGeom), ctypes.POINTER(SparkPagePool),
                                        ctypes.POINTER(SparkPagedBatch), _P, _P, ctypes.c_int64, ctypes.c_int32, _P,
                                        ctypes.c_size_t, _P]),
    "spark_attn_paged": (ctypes.c_int, [ctypes.POINTER(SparkGeom), _P, ctypes.POINTER(SparkLayerWeights),
                                        ctypes.POINTER(SparkPagePool), ctypes.c_int32,
                                        ctypes.POINTER(SparkPagedBatch), ctypes.POINTER(ctypes.c_int32), _P, _P,
                                        ctypes.c_size_t, _P, ctypes.c_size_t, _P]),
    "spark_pages_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int32]),
    "spark_pages_remap": (ctypes.c_int, [ctypes.POINTER(SparkGeom), ctypes.POINTER(SparkPagePool), ctypes.c_int32,
                                         _P, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.c_size_t,
                                         _P]),
    "spark_pages_compact": (ctypes.c_int, [ctypes.POINTER(SparkGeom), ctypes.POINTER(SparkPagePool), ctypes.c_int32,
                                           _P, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, ctypes.c_size_t, _P]),
    "spark_logprobs_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "spark_token_logprobs": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P,
                                            ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "spark_beam_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "spark_beam_select": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_int32, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P, _P,
                                         ctypes.c_size_t, _P]),
    # (states: an array of SparkBeamState, or its bytes)
    "spark_beam_reorder": (ctypes.c_int, [_P, _P, _P, ctypes.c_int32, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "spark_attn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "spark_attn_abi_version": (ctypes.c_int32, []),
}

_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library once and bind every declared entry point."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "decode_attention_block_gb300.build_lib.build() (needs nvcc)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def declared_symbols() -> list[str]:
    return list(_SIGNATURES)


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

# the current stream's handle without building a torch.cuda.Stream around it
# (0.2 us a call instead of 3)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# the current device without asking whether CUDA is initialised: a call's
# tensors have done that
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev_ptr(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _not_here(t, name: str) -> Exception:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return TypeError(f"{name} must be a CUDA tensor")
    return ValueError(f"{name} is on device {t.get_device()}, the current device is {_current_device()}")


def _here(t: torch.Tensor, name: str, dtype=None) -> int:
    """As _dev_ptr, of a tensor on the current device: the call goes to its
    stream, and its memory alone the kernels are sure to reach."""
    if not isinstance(t, torch.Tensor) or t.get_device() != _current_device():
        raise _not_here(t, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _check(status: int, where: str) -> None:
    if status != SPARK_OK:
        raise SparkError(status, where)


class _CachedC:
    """Mixin of the weight and cache descriptors: the C struct is built and
    checked once and reused while no field is reassigned (the tensors' device
    addresses do not change in place), which keeps the per-call marshalling
    of a decode step short."""

    def __setattr__(self, name, value):
        if name != "_c":
            object.__setattr__(self, "_c", None)
        object.__setattr__(self, name, value)

    def to_c(self):
        if self._c is None:
            object.__setattr__(self, "_c", self._build_c())
        return self._c


def _positions(positions) -> ctypes.Array:
    vals = [int(p) for p in positions]
    return (ctypes.c_int32 * max(1, len(vals)))(*vals)


@dataclass
class LayerWeights(_CachedC):
    """One layer's weights as CUDA tensors (all float32 or all bfloat16):
    ``norm_w [hidden]``, ``qkv_w [n_q*d + 2*n_kv*d, hidden]``,
    ``g_w [n_q, hidden]``, ``o_w [hidden, n_q*d]``."""

    norm_w: torch.Tensor
    qkv_w: torch.Tensor
    g_w: torch.Tensor
    o_w: torch.Tensor
    _c: object = field(default=None, init=False, repr=False, compare=False)

    def _build_c(self) -> SparkLayerWeights:
        dt = self.qkv_w.dtype
        if dt not in _DTYPE_CODE:
            raise TypeError(f"weights must be float32 or bfloat16, got {dt}")
        return SparkLayerWeights(_dev_ptr(self.norm_w, "norm_w", dt), _dev_ptr(self.qkv_w, "qkv_w", dt),
                                 _dev_ptr(self.g_w, "g_w", dt), _dev_ptr(self.o_w, "o_w", dt),
                                 _DTYPE_CODE[dt])


@dataclass
class KvLayer(_CachedC):
    """One layer's cache as CUDA tensors ``k``, ``v`` of shape
    ``[batch, capacity, n_kv, head_dim]`` (float32 or bfloat16) and the ring
    capacity (0 = linear addressing)."""

    k: torch.Tensor
    v: torch.Tensor
    ring_capacity: int = 0
    _c: object = field(default=None, init=False, repr=False, compare=False)

    def _build_c(self) -> SparkKvLayer:
        dt = self.k.dtype
        if dt not in _DTYPE_CODE:
            raise TypeError(f"cache must be float32 or bfloat16, got {dt}")
        if self.k.dim() != 4 or self.k.shape != self.v.shape:
            raise ValueError("k and v must both be [batch, capacity, n_kv, head_dim]")
        return SparkKvLayer(_dev_ptr(self.k, "k", dt), _dev_ptr(self.v, "v", dt),
                            int(self.k.shape[1]), int(self.ring_capacity), _DTYPE_CODE[dt])


@dataclass
class MlpWeights(_CachedC):
    """The MLP half of one layer as CUDA tensors (all float32 or all
    bfloat16): ``norm_w [hidden]`` (post_attention_layernorm), ``gate_w`` and
    ``up_w [intermediate, hidden]``, ``down_w [hidden, intermediate]``."""

    norm_w: torch.Tensor
    gate_w: torch.Tensor
    up_w: torch.Tensor
    down_w: torch.Tensor
    _c: object = field(default=None, init=False, repr=False, compare=False)

    def _build_c(self) -> SparkMlpWeights:
        dt = self.gate_w.dtype
        if dt not in _DTYPE_CODE:
            raise TypeError(f"weights must be float32 or bfloat16, got {dt}")
        if self.gate_w.dim() != 2 or self.up_w.shape != self.gate_w.shape or \
                self.down_w.shape != (self.gate_w.shape[1], self.gate_w.shape[0]):
            raise ValueError("gate_w, up_w must be [intermediate, hidden] and down_w [hidden, intermediate]")
        return SparkMlpWeights(_dev_ptr(self.norm_w, "norm_w", dt), _dev_ptr(self.gate_w, "gate_w", dt),
                               _dev_ptr(self.up_w, "up_w", dt), _dev_ptr(self.down_w, "down_w", dt),
                               int(self.gate_w.shape[0]), _DTYPE_CODE[dt])


def _rows(t: torch.Tensor, name: str) -> tuple:
    """Address, row stride (elements) and dtype code of a matrix on the current
    device whose rows are contiguous but may lie apart (a slice of a fused
    projection's output)."""
    if not isinstance(t, torch.Tensor) or t.get_device() != _current_device():
        raise _not_here(t, name)
    code = _DTYPE_CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or stride[1] != 1 and shape[1] > 1:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1], code


def _matrix(t: torch.Tensor, name: str, shape: tuple, device: int) -> tuple:
    """As _rows, of a matrix of this shape."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise _not_here(t, name)
    code = _DTYPE_CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be [n_tokens, {shape[1]}]")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    return t.data_ptr(), ld if shape[0] > 1 else shape[1], code


@dataclass
class PagePool(_CachedC):
    """One layer's pages as CUDA tensors ``k``, ``v`` of shape
    ``[n_pages, page_size, n_kv, head_dim]`` (float32 or bfloat16), or, held in
    4 bits, uint8 ``[n_pages, page_size / 16, n_kv, 2304]`` (the header's
    blocks)."""

    k: torch.Tensor
    v: torch.Tensor
    _c: object = field(default=None, init=False, repr=False, compare=False)

    def _build_c(self) -> tuple:
        """The C struct, its bytes (for arrays of them) and (n_kv, head_dim, device)."""
        dt = self.k.dtype
        if dt not in _DTYPE_CODE and dt != torch.uint8:
            raise TypeError(f"pages must be float32, bfloat16 or uint8 (4 bits), got {dt}")
        if self.k.dim() != 4 or self.k.shape != self.v.shape:
            raise ValueError("k and v must both be [n_pages, page_size, n_kv, head_dim]")
        n_pages, page_size, n_kv, head_dim = (int(x) for x in self.k.shape)
        code = _DTYPE_CODE.get(dt)
        if code is None:
            if head_dim != SPARK_FP4_BLOCK_BYTES:
                raise ValueError(f"4-bit pages must be [n_pages, page_size / 16, n_kv, {SPARK_FP4_BLOCK_BYTES}]")
            code, page_size, head_dim = SPARK_FP4, 16 * page_size, 256
        c = SparkPagePool(_dev_ptr(self.k, "k", dt), _dev_ptr(self.v, "v", dt), n_pages, page_size, code)
        if self.v.get_device() != self.k.get_device():
            raise ValueError("k and v must be on the same device")
        return c, bytes(c), (n_kv, head_dim, self.k.get_device())


@dataclass
class PagedBatch(_CachedC):
    """The sequences of a call: int32 CUDA tensors ``table [n_seqs,
    max_pages]``, ``q_start [n_seqs + 1]`` and ``seq_len [n_seqs]``, whose
    values are read when the work runs, the rows ``n_tokens`` of the call's
    token tensors and the most new tokens of a sequence ``max_q_len``."""

    table: torch.Tensor
    q_start: torch.Tensor
    seq_len: torch.Tensor
    n_tokens: int
    max_q_len: int
    _c: object = field(default=None, init=False, repr=False, compare=False)

    def _build_c(self) -> tuple:
        """The C struct and the device its arrays are on."""
        if self.table.dim() != 2 or self.q_start.shape != (self.table.shape[0] + 1,) or \
                self.seq_len.shape != (self.table.shape[0],):
            raise ValueError("table must be [n_seqs, max_pages], q_start [n_seqs + 1], seq_len [n_seqs]")
        c = SparkPagedBatch(_dev_ptr(self.table, "table", torch.int32),
                            _dev_ptr(self.q_start, "q_start", torch.int32),
                            _dev_ptr(self.seq_len, "seq_len", torch.int32), int(self.table.shape[0]),
                            int(self.table.shape[1]), int(self.n_tokens), int(self.max_q_len))
        device = self.table.get_device()
        if self.q_start.get_device() != device or self.seq_len.get_device() != device:
            raise ValueError("table, q_start and seq_len must be on the same device")
        return c, device


def _batch_c(batch: PagedBatch) -> SparkPagedBatch:
    c, device = batch.to_c()
    if device != _current_device():
        raise _not_here(batch.table, "the batch's table")
    return c


def _pool_differs(got, want) -> ValueError:
    return ValueError(f"pages of {got[0]} heads of {got[1]} on device {got[2]}: the geometry has {want[0]} of {want[1]}, "
                      f"the current device is {want[2]}")


def _pool_c(geom: SparkGeom, pool: PagePool) -> SparkPagePool:
    c, _, heads = pool.to_c()
    want = (geom.n_kv, geom.head_dim, _current_device())
    if heads != want:
        raise _pool_differs(heads, want)
    return c


def _pools_c(geom: SparkGeom, pools) -> ctypes.Array:
    built = [p._c for p in pools]
    if None in built:
        built = [p.to_c() for p in pools]
    want = (geom.n_kv, geom.head_dim, _current_device())
    for heads in {b[2] for b in built}:
        if heads != want:
            raise _pool_differs(heads, want)
    return (SparkPagePool * len(built)).from_buffer_copy(b"".join([b[1] for b in built]))


# ---------------------------------------------------------------------------
# the entry points
# ---------------------------------------------------------------------------

def spark_geom_default() -> SparkGeom:
    g = SparkGeom()
    load().spark_geom_default(ctypes.byref(g))
    return g


def spark_attn_workspace_bytes(geom: SparkGeom, batch: int) -> int:
    return int(load().spark_attn_workspace_bytes(ctypes.byref(geom), int(batch)))


def spark_attn_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _check(load().spark_attn_workspace_init(_dev_ptr(ws, "workspace"), ws.numel() * ws.element_size(),
                                            _stream(stream)), "spark_attn_workspace_init")


def spark_attn_error_word(ws: torch.Tensor, stream=None) -> int:
    word = ctypes.c_uint32(0)
    _check(load().spark_attn_error_word(_dev_ptr(ws, "workspace"), ws.numel() * ws.element_size(),
                                        ctypes.byref(word), _stream(stream)), "spark_attn_error_word")
    return int(word.value)


def make_workspace(geom: SparkGeom, batch: int, device=None, stream=None) -> torch.Tensor:
    """Allocate (through PyTorch) and initialise a workspace for ``batch``."""
    nbytes = spark_attn_workspace_bytes(geom, batch)
    if nbytes == 0:
        raise ValueError("invalid geometry or batch for a workspace")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    spark_attn_workspace_init(ws, stream)
    return ws


def spark_attn_decode(geom: SparkGeom, h: torch.Tensor, weights: LayerWeights, kv: KvLayer,
                      layer_class: int, positions, out: torch.Tensor, ws: torch.Tensor,
                      stream=None) -> None:
    batch = len(positions)
    wc, kc, pos = weights.to_c(), kv.to_c(), _positions(positions)
    _check(load().spark_attn_decode(ctypes.byref(geom), _dev_ptr(h, "h", torch.float32),
                                    ctypes.byref(wc), ctypes.byref(kc), int(layer_class), pos,
                                    batch, _dev_ptr(out, "out", torch.float32),
                                    _dev_ptr(ws, "workspace"), ws.numel() * ws.element_size(),
                                    _stream(stream)), "spark_attn_decode")


def spark_attn_prefill(geom: SparkGeom, h: torch.Tensor, weights: LayerWeights, kv: KvLayer,
                       layer_class: int, p0: int, out: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """h.shape[0] consecutive tokens of one sequence (positions p0, p0+1, ...)
    through one layer; kv is that sequence's cache ([1, capacity, n_kv, 256])."""
    wc, kc = weights.to_c(), kv.to_c()
    _check(load().spark_attn_prefill(ctypes.byref(geom), _dev_ptr(h, "h", torch.float32), ctypes.byref(wc),
                                     ctypes.byref(kc), int(layer_class), int(p0), int(h.shape[0]),
                                     _dev_ptr(out, "out", torch.float32), _dev_ptr(ws, "workspace"),
                                     ws.numel() * ws.element_size(), _stream(stream)),
           "spark_attn_prefill")


def spark_attn_decode_stack(geom: SparkGeom, h: torch.Tensor, weights: list, kvs: list, layer_classes,
                            positions, out: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """One decode step through len(weights) layers (each layer's output is the
    next one's input); ``out`` receives the last layer's output."""
    n = len(weights)
    if len(kvs) != n or len(layer_classes) != n:
        raise ValueError("weights, kvs and layer_classes must have one entry per layer")
    wc = (SparkLayerWeights * n)(*[w.to_c() for w in weights])
    kc = (SparkKvLayer * n)(*[k.to_c() for k in kvs])
    cls = (ctypes.c_int32 * n)(*[int(c) for c in layer_classes])
    pos = _positions(positions)
    _check(load().spark_attn_decode_stack(ctypes.byref(geom), _dev_ptr(h, "h", torch.float32), n, wc, kc, cls,
                                          pos, len(positions), _dev_ptr(out, "out", torch.float32),
                                          _dev_ptr(ws, "workspace"), ws.numel() * ws.element_size(),
                                          _stream(stream)), "spark_attn_decode_stack")


def spark_dbg_qkv_rope(geom: SparkGeom, h: torch.Tensor, weights: LayerWeights, kv: KvLayer,
                       layer_class: int, positions, q_rot: torch.Tensor, g_logits: torch.Tensor,
                       ws: torch.Tensor, path: int = 0, stream=None) -> None:
    wc, kc, pos = weights.to_c(), kv.to_c(), _positions(positions)
    _check(load().spark_dbg_qkv_rope(ctypes.byref(geom), _dev_ptr(h, "h", torch.float32), ctypes.byref(wc),
                                     ctypes.byref(kc), int(layer_class), pos, len(positions),
                                     _dev_ptr(q_rot, "q_rot", torch.float32),
                                     _dev_ptr(g_logits, "g_logits", torch.float32), int(path),
                                     _dev_ptr(ws, "workspace"), ws.numel() * ws.element_size(),
                                     _stream(stream)),
           "spark_dbg_qkv_rope")


def spark_dbg_attention(geom: SparkGeom, q_rot: torch.Tensor, kv: KvLayer, layer_class: int, positions,
                        a: torch.Tensor, ws: torch.Tensor, n_ctas: int = 0, stream=None) -> None:
    kc, pos = kv.to_c(), _positions(positions)
    _check(load().spark_dbg_attention(ctypes.byref(geom), _dev_ptr(q_rot, "q_rot", torch.float32),
                                      ctypes.byref(kc), int(layer_class), pos, len(positions),
                                      _dev_ptr(a, "a", torch.float32), int(n_ctas),
                                      _dev_ptr(ws, "workspace"), ws.numel() * ws.element_size(),
                                      _stream(stream)), "spark_dbg_attention")


def spark_dbg_attention_noalloc(geom: SparkGeom, q_rot: torch.Tensor, kv: KvLayer, layer_class: int,
                                positions, a: torch.Tensor, stream=None) -> None:
    """spark_dbg_attention without a workspace: the library's fixed scratch
    array is used instead (for callers that cannot allocate device memory)."""
    kc, pos = kv.to_c(), _positions(positions)
    _check(load().spark_dbg_attention_noalloc(ctypes.byref(geom), _dev_ptr(q_rot, "q_rot", torch.float32),
                                              ctypes.byref(kc), int(layer_class), pos, len(positions),
                                              _dev_ptr(a, "a", torch.float32), _stream(stream)),
           "spark_dbg_attention_noalloc")


def spark_dbg_attention_noalloc_error_word(stream=None) -> int:
    """Read and clear the error word of the no-workspace attention's fixed
    array on the current device (synchronises the stream)."""
    word = ctypes.c_uint32(0)
    _check(load().spark_dbg_attention_noalloc_error_word(ctypes.byref(word), _stream(stream)),
           "spark_dbg_attention_noalloc_error_word")
    return int(word.value)


def spark_dbg_gate_oproj(geom: SparkGeom, a: torch.Tensor, g_logits: torch.Tensor, h: torch.Tensor,
                         weights: LayerWeights, out: torch.Tensor, ws: torch.Tensor, path: int = 0,
                         stream=None) -> None:
    wc = weights.to_c()
    _check(load().spark_dbg_gate_oproj(ctypes.byref(geom), _dev_ptr(a, "a", torch.float32),
                                       _dev_ptr(g_logits, "g_logits", torch.float32),
                                       _dev_ptr(h, "h", torch.float32), ctypes.byref(wc), int(h.shape[0]),
                                       _dev_ptr(out, "out", torch.float32), int(path),
                                       _dev_ptr(ws, "workspace"), ws.numel() * ws.element_size(),
                                       _stream(stream)),
           "spark_dbg_gate_oproj")


def spark_dbg_wait_timeout(ws: torch.Tensor, limit_ns: int, stream=None) -> None:
    """Run a bounded wait that nothing satisfies (see the header)."""
    _check(load().spark_dbg_wait_timeout(_dev_ptr(ws, "workspace"), ws.numel() * ws.element_size(),
                                         int(limit_ns), _stream(stream)), "spark_dbg_wait_timeout")


def spark_mlp_workspace_bytes(geom: SparkGeom, intermediate: int, batch: int) -> int:
    return int(load().spark_mlp_workspace_bytes(ctypes.byref(geom), int(intermediate), int(batch)))


def make_mlp_workspace(geom: SparkGeom, intermediate: int, batch: int, device=None, stream=None) -> torch.Tensor:
    """Allocate (through PyTorch) and initialise a workspace for
    spark_mlp_decode at this intermediate size (0: spark_head_logits only)."""
    nbytes = spark_mlp_workspace_bytes(geom, intermediate, batch)
    if nbytes == 0:
        raise ValueError("invalid geometry, intermediate size or batch for a workspace")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    spark_attn_workspace_init(ws, stream)
    return ws


def spark_mlp_decode(geom: SparkGeom, h: torch.Tensor, weights: MlpWeights, out: torch.Tensor,
                     ws: torch.Tensor, path: int = 0, stream=None) -> None:
    wc = weights.to_c()
    _check(load().spark_mlp_decode(ctypes.byref(geom), _dev_ptr(h, "h", torch.float32), ctypes.byref(wc),
                                   int(h.shape[0]), _dev_ptr(out, "out", torch.float32), int(path),
                                   _dev_ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream(stream)),
           "spark_mlp_decode")


def spark_head_logits(geom: SparkGeom, h: torch.Tensor, norm_w: torch.Tensor, embed: torch.Tensor,
                      logits: torch.Tensor, ws: torch.Tensor, path: int = 0, stream=None) -> None:
    """logits [batch, vocab] = embed [vocab, hidden] @ rms(h) * norm_w."""
    dt = embed.dtype
    if dt not in _DTYPE_CODE:
        raise TypeError(f"embed must be float32 or bfloat16, got {dt}")
    if embed.dim() != 2 or logits.dim() != 2 or logits.shape != (h.shape[0], embed.shape[0]):
        raise ValueError("embed must be [vocab, hidden] and logits [batch, vocab]")
    _check(load().spark_head_logits(ctypes.byref(geom), _dev_ptr(h, "h", torch.float32),
                                    _dev_ptr(norm_w, "norm_w", dt), _dev_ptr(embed, "embed", dt),
                                    int(embed.shape[0]), _DTYPE_CODE[dt], int(h.shape[0]),
                                    _dev_ptr(logits, "logits", torch.float32), int(path),
                                    _dev_ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream(stream)),
           "spark_head_logits")


def _workspace(nbytes: int, what: str, device, stream) -> torch.Tensor:
    if nbytes == 0:
        raise ValueError(f"invalid {what} for a workspace")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    spark_attn_workspace_init(ws, stream)
    return ws


def spark_paged_workspace_bytes(geom: SparkGeom) -> int:
    return int(load().spark_paged_workspace_bytes(ctypes.byref(geom)))


def make_paged_workspace(geom: SparkGeom, device=None, stream=None) -> torch.Tensor:
    """Allocate (through PyTorch) and initialise a workspace for
    spark_paged_append and spark_paged_attention (any batch)."""
    return _workspace(spark_paged_workspace_bytes(geom), "geometry", device, stream)


def spark_paged_append(geom: SparkGeom, k: torch.Tensor, v: torch.Tensor, pool: PagePool, batch: PagedBatch,
                       ws: torch.Tensor, stream=None) -> None:
    """Write the new tokens' rows k, v [n_tokens, n_kv * 256] into their pages."""
    kp, ld, dt = _rows(k, "k")
    vp, vld, vdt = _rows(v, "v")
    kv_dim = geom.n_kv * geom.head_dim
    if k.shape != (batch.n_tokens, kv_dim) or v.shape != k.shape:
        raise ValueError(f"k and v must be [n_tokens, {kv_dim}]")
    if vdt != dt or vld != ld:
        raise ValueError("k and v must have the same dtype and row stride")
    pc, bc = _pool_c(geom, pool), _batch_c(batch)
    _check(load().spark_paged_append(ctypes.byref(geom), kp, vp, ld, dt, ctypes.byref(pc), ctypes.byref(bc),
                                     _here(ws, "workspace"), ws.nbytes, _stream(stream)),
           "spark_paged_append")


def spark_rope_table(geom: SparkGeom, layer_class: int, rope: torch.Tensor, stream=None) -> None:
    """rope [n_positions, r / 2, 2] (float32, r the class's rotary dim) = (cos,
    sin) of the class's angles."""
    _check(load().spark_rope_table(ctypes.byref(geom), int(layer_class), _rope_rows(geom, layer_class, rope),
                                   _here(rope, "rope", torch.float32), _stream(stream)), "spark_rope_table")


def _rope_rows(geom: SparkGeom, layer_class: int, rope: torch.Tensor) -> int:
    half = (geom.full_rotary_dim if layer_class == SPARK_FULL else geom.head_dim) // 2
    shape = rope.shape
    if shape[1:] != (half, 2):
        raise ValueError(f"rope must be [n_positions, {half}, 2]")
    return shape[0]


def spark_paged_rope_append(geom: SparkGeom, q, k: torch.Tensor, v: torch.Tensor, layer_class: int, rope: torch.Tensor,
                            pool: PagePool, batch: PagedBatch, q_out, ws: torch.Tensor, stream=None) -> None:
    """Rotate the new tokens' queries q [n_tokens, n_q * 256] into q_out (which
    may be q; both None: no queries) and their keys, and write the rows k, v
    [n_tokens, n_kv * 256] into their pages.  q, k and v have one row stride
    (slices of a fused projection's rows); rope: spark_rope_table's."""
    device, head_dim = _current_device(), geom.head_dim
    kv_shape = (batch.n_tokens, geom.n_kv * head_dim)
    kp, ld, dt = _matrix(k, "k", kv_shape, device)
    vp, vld, vdt = _matrix(v, "v", kv_shape, device)
    qp, op, old = None, None, 0
    if q is not None:
        q_shape = (batch.n_tokens, geom.n_q * head_dim)
        qp, qld, qdt = _matrix(q, "q", q_shape, device)
        op, old, odt = _matrix(q_out, "q_out", q_shape, device)
        if batch.n_tokens == 1:  # a single row has no stride
            ld = vld = qld
        if qdt != dt or odt != dt or qld != ld:
            raise ValueError("q, q_out, k and v must have the same dtype, q, k and v the same row stride")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if vdt != dt or vld != ld:
        raise ValueError("k and v must have the same dtype and row stride")
    pc, bc = _pool_c(geom, pool), _batch_c(batch)
    _check(load().spark_paged_rope_append(ctypes.byref(geom), qp, kp, vp, ld, dt, layer_class,
                                          _here(rope, "rope", torch.float32), _rope_rows(geom, layer_class, rope),
                                          ctypes.byref(pc), ctypes.byref(bc), op, old, _here(ws, "workspace"), ws.nbytes,
                                          _stream(stream)), "spark_paged_rope_append")


def spark_paged_read(geom: SparkGeom, pool: PagePool, batch: PagedBatch, k: torch.Tensor, v: torch.Tensor,
                     ws: torch.Tensor, stream=None) -> None:
    """k, v [n_tokens, n_kv * 256] = the batch's rows out of their pages."""
    kp, ld, dt = _rows(k, "k")
    vp, vld, vdt = _rows(v, "v")
    kv_dim = geom.n_kv * geom.head_dim
    if k.shape != (batch.n_tokens, kv_dim) or v.shape != k.shape:
        raise ValueError(f"k and v must be [n_tokens, {kv_dim}]")
    if vdt != dt or vld != ld:
        raise ValueError("k and v must have the same dtype and row stride")
    pc, bc = _pool_c(geom, pool), _batch_c(batch)
    _check(load().spark_paged_read(ctypes.byref(geom), ctypes.byref(pc), ctypes.byref(bc), kp, vp, ld, dt,
                                   _here(ws, "workspace"), ws.nbytes, _stream(stream)), "spark_paged_read")


def spark_paged_attention(geom: SparkGeom, q: torch.Tensor, pool: PagePool, layer_class: int, batch: PagedBatch,
                          a: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """a [n_tokens, n_q * 256] = attention of the rotated queries q (float32
    or bfloat16, a alike) over each sequence's pages."""
    qp, ld, dt = _rows(q, "q")
    if q.shape != (batch.n_tokens, geom.n_q * geom.head_dim) or a.shape != q.shape:
        raise ValueError(f"q and a must be [n_tokens, {geom.n_q * geom.head_dim}]")
    pc, bc = _pool_c(geom, pool), _batch_c(batch)
    _check(load().spark_paged_attention(ctypes.byref(geom), qp, ld, dt, ctypes.byref(pc), int(layer_class),
                                        ctypes.byref(bc), _here(a, "a", q.dtype), _here(ws, "workspace"),
                                        ws.nbytes, _stream(stream)), "spark_paged_attention")


def spark_attn_paged(geom: SparkGeom, h: torch.Tensor, weights: LayerWeights, pool: PagePool, layer_class: int,
                     batch: PagedBatch, positions, out: torch.Tensor, ws: torch.Tensor, paged_ws: torch.Tensor,
                     stream=None) -> None:
    """The attention block for the batch's new tokens on a paged cache: h,
    out [n_tokens, hidden]; positions: each row's rope position (host; a
    captured call keeps those of its capture, whatever the lengths become)."""
    if h.shape != (batch.n_tokens, geom.hidden) or out.shape != h.shape or len(positions) != batch.n_tokens:
        raise ValueError("h and out must be [n_tokens, hidden], with one position per row")
    wc, pc, bc = weights.to_c(), _pool_c(geom, pool), _batch_c(batch)
    for name in ("norm_w", "qkv_w", "g_w", "o_w"):
        if getattr(weights, name).get_device() != _current_device():
            raise _not_here(getattr(weights, name), name)
    _check(load().spark_attn_paged(ctypes.byref(geom), _here(h, "h", torch.float32), ctypes.byref(wc),
                                   ctypes.byref(pc), int(layer_class), ctypes.byref(bc), _positions(positions),
                                   _here(out, "out", torch.float32), _here(ws, "workspace"),
                                   ws.nbytes, _here(paged_ws, "paged workspace"),
                                   paged_ws.nbytes, _stream(stream)), "spark_attn_paged")


def spark_pages_workspace_bytes(n_pages: int, n_slots: int) -> int:
    return int(load().spark_pages_workspace_bytes(int(n_pages), int(n_slots)))


def make_pages_workspace(n_pages: int, n_slots: int, device=None, stream=None) -> torch.Tensor:
    """Allocate (through PyTorch) and initialise a workspace for
    spark_pages_remap and spark_pages_compact."""
    return _workspace(spark_pages_workspace_bytes(n_pages, n_slots), "number of pages or slots", device, stream)


def spark_pages_remap(geom: SparkGeom, pools, table: torch.Tensor, parent: torch.Tensor, keep_len: torch.Tensor,
                      new_len: torch.Tensor, new_table: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """The page tables of a step: row s of new_table holds the first
    keep_len[s] positions of table's row parent[s] (-1: nothing) and has room
    for new_len[s]; ``pools``: every layer's PagePool."""
    n = table.shape[0]
    if table.dim() != 2 or new_table.shape != table.shape or not parent.shape == keep_len.shape == new_len.shape == (n,):
        raise ValueError("table and new_table must be [n_slots, max_pages], the lists [n_slots]")
    i32 = torch.int32
    _check(load().spark_pages_remap(ctypes.byref(geom), _pools_c(geom, pools), len(pools), _here(table, "table", i32),
                                    n, int(table.shape[1]), _here(parent, "parent", i32),
                                    _here(keep_len, "keep_len", i32), _here(new_len, "new_len", i32),
                                    _here(new_table, "new_table", i32), _here(ws, "workspace"),
                                    ws.nbytes, _stream(stream)), "spark_pages_remap")


def spark_pages_compact(geom: SparkGeom, pools, table: torch.Tensor, new_table: torch.Tensor, n_live: torch.Tensor,
                        ws: torch.Tensor, stream=None) -> None:
    """Move the pages in use to the front of every pool; n_live (int32, one
    element) receives their number.  new_table may be table."""
    if table.dim() != 2 or new_table.shape != table.shape or n_live.numel() != 1:
        raise ValueError("table and new_table must be [n_slots, max_pages], n_live one element")
    i32 = torch.int32
    _check(load().spark_pages_compact(ctypes.byref(geom), _pools_c(geom, pools), len(pools),
                                      _here(table, "table", i32), int(table.shape[0]), int(table.shape[1]),
                                      _here(new_table, "new_table", i32), _here(n_live, "n_live", i32),
                                      _here(ws, "workspace"), ws.nbytes, _stream(stream)),
           "spark_pages_compact")


def spark_logprobs_workspace_bytes(n_rows: int, top_k: int) -> int:
    return int(load().spark_logprobs_workspace_bytes(int(n_rows), int(top_k)))


def make_logprobs_workspace(n_rows: int, top_k: int, device=None, stream=None) -> torch.Tensor:
    """Allocate (through PyTorch) and initialise a workspace for
    spark_token_logprobs."""
    return _workspace(spark_logprobs_workspace_bytes(n_rows, top_k), "number of rows or alternatives", device, stream)


def spark_token_logprobs(logits: torch.Tensor, targets: torch.Tensor, logprob: torch.Tensor, entropy: torch.Tensor,
                         top_ids: torch.Tensor, top_logprobs: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """Log probabilities of the targets [n] under logits [n, vocab] (float32
    or bfloat16; -1: none), the rows' entropies, and their top_ids.shape[1]
    highest logits' indices and log probabilities (None, None: none)."""
    lp, ld, dt = _rows(logits, "logits")
    n, vocab = logits.shape
    k = 0 if top_ids is None else int(top_ids.shape[1])
    if targets.shape != (n,) or logprob.shape != (n,) or entropy.shape != (n,):
        raise ValueError("targets, logprob and entropy must be [n]")
    if k and (top_ids.shape != (n, k) or top_logprobs.shape != (n, k)):
        raise ValueError("top_ids and top_logprobs must be [n, k]")
    _check(load().spark_token_logprobs(lp, ld, dt, n, vocab, _here(targets, "targets", torch.int32), k,
                                       _here(logprob, "logprob", torch.float32),
                                       _here(entropy, "entropy", torch.float32),
                                       _here(top_ids, "top_ids", torch.int32) if k else None,
                                       _here(top_logprobs, "top_logprobs", torch.float32) if k else None,
                                       _here(ws, "workspace"), ws.nbytes, _stream(stream)),
           "spark_token_logprobs")


def spark_beam_workspace_bytes(n_groups: int, n_beams: int) -> int:
    return int(load().spark_beam_workspace_bytes(int(n_groups), int(n_beams)))


def make_beam_workspace(n_groups: int, n_beams: int, device=None, stream=None) -> torch.Tensor:
    """Allocate (through PyTorch) and initialise a workspace for
    spark_beam_select and spark_beam_reorder."""
    return _workspace(spark_beam_workspace_bytes(n_groups, n_beams), "number of groups or beams", device, stream)


def _slots(t, name: str, shape: tuple, device: int, dtype=torch.int32):
    """Address of a list of a value for each slot; None: none."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise _not_here(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be [{shape[0]}] and contiguous")
    return t.data_ptr()


def spark_beam_select(logits: torch.Tensor, score: torch.Tensor, done, length, n_beams: int, eos: int,
                      new_score: torch.Tensor, token: torch.Tensor, parent: torch.Tensor, new_done, keep_len, new_len,
                      ws: torch.Tensor, stream=None) -> None:
    """The n_beams best continuations of every group of n_beams slots under
    logits [slots, vocab] (float32 or bfloat16); lists [slots], float32 scores
    and int32 otherwise.  done (and new_done, with eos -1) or the three lengths
    may be None."""
    lp, ld, dt = _rows(logits, "logits")
    n, vocab = logits.shape
    if n_beams < 1 or n % n_beams:
        raise ValueError("logits must have a row for each beam of every group")
    f32, device, of = torch.float32, _current_device(), (n,)
    _check(load().spark_beam_select(lp, ld, dt, n // n_beams, n_beams, vocab, _slots(score, "score", of, device, f32),
                                    _slots(done, "done", of, device), _slots(length, "length", of, device), eos,
                                    _slots(new_score, "new_score", of, device, f32), _slots(token, "token", of, device),
                                    _slots(parent, "parent", of, device), _slots(new_done, "new_done", of, device),
                                    _slots(keep_len, "keep_len", of, device), _slots(new_len, "new_len", of, device),
                                    _here(ws, "workspace"), ws.nbytes, _stream(stream)), "spark_beam_select")


@dataclass
class BeamState(_CachedC):
    """A state of the beams as two CUDA tensors of the same shape, [slots, ...]
    with rows of a multiple of 4 bytes: ``dst`` receives ``src``'s rows in their
    new order.  ``positions``: the second dimension is a beam's positions, of
    which the kept ones go along; ``push`` (int32 [slots], for int32 [slots,
    positions]) is what to write behind them."""

    src: torch.Tensor
    dst: torch.Tensor
    positions: bool = False
    push: torch.Tensor | None = None
    _c: object = field(default=None, init=False, repr=False, compare=False)

    def _build_c(self) -> tuple:
        """The C struct's bytes and (slots, device)."""
        n, device = int(self.src.shape[0]), self.src.get_device()
        if self.src.shape != self.dst.shape or self.src.dim() < 1 + bool(self.positions):
            raise ValueError("src and dst must both be [slots, ...], with positions [slots, positions, ...]")
        pitch = self.src.nbytes // max(1, n)
        elem = pitch // max(1, int(self.src.shape[1])) if self.positions else 0
        push = None
        if self.push is not None:
            if self.src.dtype != torch.int32 or self.src.dim() != 2 or self.push.shape != (n,):
                raise ValueError("push must be [slots], of a state of positions that are int32")
            push = _dev_ptr(self.push, "push", torch.int32)
        for t in (self.dst, self.push):
            if t is not None and t.get_device() != device:
                raise ValueError("src, dst and push must be on the same device")
        c = SparkBeamState(_dev_ptr(self.src, "src"), _dev_ptr(self.dst, "dst", self.src.dtype), pitch, elem, push)
        return bytes(c), (n, device)


def spark_beam_reorder(parent: torch.Tensor, keep_len, new_len, states, ws: torch.Tensor, stream=None) -> None:
    """Rows of every BeamState to their new slots (spark_beam_select's parent,
    keep_len and new_len; the lengths may be None without ``positions``)."""
    device = _current_device()
    if not isinstance(parent, torch.Tensor):
        raise _not_here(parent, "parent")
    of = parent.shape
    if len(of) != 1:
        raise ValueError("parent must be a list, one slot each")
    built = [st._c or st.to_c() for st in states]
    for st, b in zip(states, built):
        if b[1] != (of[0], device):
            if b[1][0] != of[0]:
                raise ValueError("every state must have a row for each slot")
            raise _not_here(st.src, "a state")
    _check(load().spark_beam_reorder(_slots(parent, "parent", of, device), _slots(keep_len, "keep_len", of, device),
                                     _slots(new_len, "new_len", of, device), of[0], b"".join([b[0] for b in built]),
                                     len(built), _here(ws, "workspace"), ws.nbytes, _stream(stream)), "spark_beam_reorder")


def spark_attn_status_string(status: int) -> str:
    return load().spark_attn_status_string(int(status)).decode()


def spark_attn_abi_version() -> int:
    return int(load().spark_attn_abi_version())
