"""Python binding of libq8k (the C ABI in include/q8k.h).

Argument marshalling only: every step of the path runs in the gfx950 kernels
behind the C ABI.  PyTorch provides device memory and streams.  There is no
CPU fallback: if libq8k.so is missing the import raises.

Functions keep the C names and argument order; tensors are passed for device
buffers (their ``data_ptr()`` is used) and the stream defaults to torch's
current stream.  A refusal raises :class:`Q8KError` carrying the status name
and the library's message.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "Q8K_Q4_K", "Q8K_Q5_K", "Q8K_Q6_K_RELAID", "Q8K_Q6_K_GGUF", "Q8K_COLS_MAX", "Q8K_MOE_MAX_TOKENS", "Q8K_MOE_MAX_TOPK", "Q8KError",
    "lib", "LIB_PATH", "q8k_act_bytes", "q8k_act_layout", "q8k_weight_bytes", "q8k_pack", "q8k_bind_q6k",
    "qmatvec", "qmatvec_batched", "qmatvec_f32", "qmatvec_moe", "qmatmul_prefill_workspace_bytes", "qmatmul_prefill",
    "qmatmul_prefill_f32_workspace_bytes", "qmatmul_prefill_f32",
    "qmatmul_prefill_moe_workspace_bytes", "qmatmul_prefill_moe", "qmatmul_prefill_moe_noalloc",
    "Q8K_NOALLOC_SCRATCH_BYTES", "Q8K_F32", "Q8K_F16", "Q8K_BF16", "Q8K_KV_PAGE", "Q8K_TOP_MAX", "Q8K_ROPE_HALF",
    "Q8K_ROPE_ADJACENT", "KVCache", "Rope", "q8k_kv_bytes", "q8k_kv_append", "q8k_kv_read", "qattend_workspace_bytes",
    "qattend", "qlogprobs_workspace_bytes", "qlogprobs", "q8k_debug_subblock_sums", "q8k_debug_prefill_block_sums", "q8k_debug_moe_subblock_sums",
    "q8k_debug_wave_sums", "q8k_debug_last_launches", "q8k_status_str", "q8k_last_error", "EXPORTED",
]

Q8K_Q4_K = 1
Q8K_Q6_K_RELAID = 2
Q8K_Q6_K_GGUF = 3
Q8K_Q5_K = 4
Q8K_COLS_MAX = 8
Q8K_MOE_MAX_TOKENS = 256
Q8K_MOE_MAX_TOPK = 64
Q8K_NOALLOC_SCRATCH_BYTES = 64 << 20
Q8K_F32 = 0
Q8K_F16 = 1
Q8K_BF16 = 2
Q8K_KV_PAGE = 64
Q8K_TOP_MAX = 32
Q8K_ROPE_HALF = 0
Q8K_ROPE_ADJACENT = 1

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libq8k.so")

# every symbol declared in include/q8k.h
EXPORTED = (
    "q8k_act_bytes", "q8k_act_layout", "q8k_weight_bytes", "q8k_pack", "q8k_bind_q6k", "qmatvec",
    "qmatvec_batched", "qmatvec_f32", "qmatvec_moe", "qmatmul_prefill_workspace_bytes", "qmatmul_prefill",
    "qmatmul_prefill_f32_workspace_bytes", "qmatmul_prefill_f32",
    "qmatmul_prefill_moe_workspace_bytes", "qmatmul_prefill_moe", "qmatmul_prefill_moe_noalloc",
    "q8k_kv_bytes", "q8k_kv_append", "q8k_kv_read", "qattend_workspace_bytes", "qattend", "qlogprobs_workspace_bytes",
    "qlogprobs", "q8k_debug_subblock_sums", "q8k_debug_prefill_block_sums", "q8k_debug_moe_subblock_sums",
    "q8k_debug_wave_sums", "q8k_debug_last_launches", "q8k_status_str", "q8k_last_error",
)

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libq8k.so not found at {LIB_PATH}: build it first "
        "(python -m quantized_q8kpack_fp32_amd.build or __graft_entry__.build())"
    )

# torch first: its HIP runtime carries the same soname (libamdhip64.so.7) as
# the ROCm copy libq8k.so was linked against, so once torch has loaded it the
# library binds to that same runtime.  Loaded the other way round, torch
# would bring a second HIP runtime into the process, and the library's
# launches would not see the device that torch's tensors live on.
import torch  # noqa: E402,F401

lib = ctypes.CDLL(LIB_PATH)
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_INT = ctypes.c_int

lib.q8k_act_bytes.restype = _SZ
lib.q8k_act_bytes.argtypes = [_I64, _I64]
lib.q8k_act_layout.restype = _SZ
lib.q8k_act_layout.argtypes = [_I64, _I64, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]
lib.q8k_weight_bytes.restype = _SZ
lib.q8k_weight_bytes.argtypes = [_INT, _I64, _I64]
lib.q8k_pack.restype = _INT
lib.q8k_pack.argtypes = [_P, _I64, _I64, _P, _P]
lib.q8k_bind_q6k.restype = _INT
lib.q8k_bind_q6k.argtypes = [_P, _I64, _I64, _P, _P]
lib.qmatvec.restype = _INT
lib.qmatvec.argtypes = [_INT, _P, _I64, _I64, _P, _P, _P]
lib.qmatvec_batched.restype = _INT
lib.qmatvec_batched.argtypes = [_INT, _P, _I64, _I64, _P, _I64, _P, _P]
lib.qmatvec_f32.restype = _INT
lib.qmatvec_f32.argtypes = [_INT, _P, _I64, _I64, _P, _I64, _P, _P, _P]
lib.qmatvec_moe.restype = _INT
lib.qmatvec_moe.argtypes = [_INT, _P, _I64, _I64, _I64, _P, _I64, _P, _P, ctypes.c_int32, _P, _P]
lib.qmatmul_prefill_workspace_bytes.restype = _SZ
lib.qmatmul_prefill_workspace_bytes.argtypes = [_INT, _I64, _I64, _I64]
lib.qmatmul_prefill.restype = _INT
lib.qmatmul_prefill.argtypes = [_INT, _P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P]
lib.qmatmul_prefill_f32_workspace_bytes.restype = _SZ
lib.qmatmul_prefill_f32_workspace_bytes.argtypes = [_INT, _I64, _I64, _I64]
lib.qmatmul_prefill_f32.restype = _INT
lib.qmatmul_prefill_f32.argtypes = [_INT, _P, _I64, _I64, _P, _I64, _P, _P, _P, _SZ, _P]
lib.qmatmul_prefill_moe_workspace_bytes.restype = _SZ
lib.qmatmul_prefill_moe_workspace_bytes.argtypes = [_INT, _I64, _I64, _I64, _I64, ctypes.c_int32]
lib.qmatmul_prefill_moe.restype = _INT
lib.qmatmul_prefill_moe.argtypes = [_INT, _P, _I64, _I64, _I64, _P, _I64, _P, _P, ctypes.c_int32, _P, _P, _SZ, _P]
lib.qmatmul_prefill_moe_noalloc.restype = _INT
lib.qmatmul_prefill_moe_noalloc.argtypes = [_INT, _P, _I64, _I64, _I64, _P, _I64, _P, _P, ctypes.c_int32, _P, _P]


class _KVStruct(ctypes.Structure):
    _fields_ = [("data", _P), ("pages", _I64), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _RopeStruct(ctypes.Structure):
    _fields_ = [("table", _P), ("positions", _I64), ("dim", ctypes.c_int32), ("pairs", ctypes.c_int32)]


lib.q8k_kv_bytes.restype = _SZ
lib.q8k_kv_bytes.argtypes = [_I64, _I64, _I64]
lib.q8k_kv_append.restype = _INT
lib.q8k_kv_append.argtypes = [_INT, _P, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P]
lib.q8k_kv_read.restype = _INT
lib.q8k_kv_read.argtypes = [_INT, _P, _P, _I64, _P, _P, _P]
lib.qattend_workspace_bytes.restype = _SZ
lib.qattend_workspace_bytes.argtypes = [_P, _I64, _I64, _I64, _I64, _I64]
lib.qattend.restype = _INT
lib.qattend.argtypes = [_INT, _P, _I64, _I64, _P, _I64, _P, _I64, _I64, _P, _I64, _P, _I64, ctypes.c_float, _I64, _P,
                        _P, _P, _P, _P, _SZ, _P]
lib.qlogprobs_workspace_bytes.restype = _SZ
lib.qlogprobs_workspace_bytes.argtypes = [_I64, _I64, ctypes.c_int32]
lib.qlogprobs.restype = _INT
lib.qlogprobs.argtypes = [_INT, _P, _I64, _I64, _I64, _P, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _SZ, _P]
lib.q8k_debug_subblock_sums.restype = _INT
lib.q8k_debug_subblock_sums.argtypes = [_INT, _P, _I64, _I64, _P, _P, _P, _P]
lib.q8k_debug_prefill_block_sums.restype = _INT
lib.q8k_debug_prefill_block_sums.argtypes = [_INT, _P, _I64, _I64, _P, _I64, _P, _P, _P]
lib.q8k_debug_moe_subblock_sums.restype = _INT
lib.q8k_debug_moe_subblock_sums.argtypes = [_INT, _P, _I64, _I64, _I64, _P, _I64, _P, _P, ctypes.c_int32, _P, _P, _P]
lib.q8k_debug_wave_sums.restype = _INT
lib.q8k_debug_wave_sums.argtypes = [_P, _P]
lib.q8k_debug_last_launches.restype = _INT
lib.q8k_debug_last_launches.argtypes = [ctypes.POINTER(_P), _INT]
lib.q8k_status_str.restype = ctypes.c_char_p
lib.q8k_status_str.argtypes = [_INT]
lib.q8k_last_error.restype = ctypes.c_char_p
lib.q8k_last_error.argtypes = []


class Q8KError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.name = q8k_status_str(status)
        super().__init__(f"{self.name}: {message}")


def q8k_status_str(status: int) -> str:
    return lib.q8k_status_str(int(status)).decode()


def q8k_last_error() -> str:
    return lib.q8k_last_error().decode()


def _ptr(t) -> int | None:
    """Device pointer of a tensor, or an int passed through (None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# torch's current stream as the handle it is; building the stream object that
# torch.cuda.current_stream() returns takes 2.8 us, most of a small call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int) -> None:
    if st != 0:
        raise Q8KError(st, q8k_last_error())


# ------------------------------------------------------------------ sizing
def q8k_act_bytes(T: int, K: int) -> int:
    return int(lib.q8k_act_bytes(T, K))


def q8k_act_layout(T: int, K: int):
    """-> (total_bytes, off_d, off_bsums) of a q8_K buffer of T tokens."""
    od, ob = _SZ(0), _SZ(0)
    total = lib.q8k_act_layout(T, K, ctypes.byref(od), ctypes.byref(ob))
    return int(total), int(od.value), int(ob.value)


def q8k_weight_bytes(qtype: int, rows: int, K: int) -> int:
    return int(lib.q8k_weight_bytes(qtype, rows, K))


def qmatmul_prefill_workspace_bytes(qtype: int, rows: int, K: int, M: int) -> int:
    return int(lib.qmatmul_prefill_workspace_bytes(qtype, rows, K, M))


# -------------------------------------------------------------- operations
def q8k_pack(x, T: int, K: int, xq, stream=None) -> None:
    _check(lib.q8k_pack(_ptr(x), T, K, _ptr(xq), _stream(stream)))


def q8k_bind_q6k(w_gguf, rows: int, K: int, w_relaid, stream=None) -> None:
    _check(lib.q8k_bind_q6k(_ptr(w_gguf), rows, K, _ptr(w_relaid), _stream(stream)))


def qmatvec(qtype: int, w, rows: int, K: int, xq, y, stream=None) -> None:
    _check(lib.qmatvec(qtype, _ptr(w), rows, K, _ptr(xq), _ptr(y), _stream(stream)))


def qmatvec_batched(qtype: int, w, rows: int, K: int, xq, ncols: int, y, stream=None) -> None:
    _check(lib.qmatvec_batched(qtype, _ptr(w), rows, K, _ptr(xq), ncols, _ptr(y), _stream(stream)))


def qmatvec_f32(qtype: int, w, rows: int, K: int, x, ncols: int, y, xq_out=None, stream=None) -> None:
    _check(lib.qmatvec_f32(qtype, _ptr(w), rows, K, _ptr(x), ncols, _ptr(y), _ptr(xq_out), _stream(stream)))


def qmatvec_moe(qtype: int, w, E: int, rows: int, K: int, xq, T: int, ids, rw, topk: int, y, stream=None) -> None:
    _check(lib.qmatvec_moe(qtype, _ptr(w), E, rows, K, _ptr(xq), T, _ptr(ids), _ptr(rw), topk, _ptr(y),
                           _stream(stream)))


def qmatmul_prefill(qtype: int, w, rows: int, K: int, xq, M: int, y, ws=None, ws_bytes: int = 0,
                    stream=None) -> None:
    _check(lib.qmatmul_prefill(qtype, _ptr(w), rows, K, _ptr(xq), M, _ptr(y), _ptr(ws), ws_bytes,
                               _stream(stream)))


def qmatmul_prefill_f32_workspace_bytes(qtype: int, rows: int, K: int, M: int) -> int:
    return int(lib.qmatmul_prefill_f32_workspace_bytes(qtype, rows, K, M))


def qmatmul_prefill_f32(qtype: int, w, rows: int, K: int, x, M: int, xq, y, ws=None, ws_bytes: int = 0,
                        stream=None) -> None:
    _check(lib.qmatmul_prefill_f32(qtype, _ptr(w), rows, K, _ptr(x), M, _ptr(xq), _ptr(y), _ptr(ws), ws_bytes,
                                   _stream(stream)))


def qmatmul_prefill_moe_workspace_bytes(qtype: int, E: int, rows: int, K: int, T: int, topk: int) -> int:
    return int(lib.qmatmul_prefill_moe_workspace_bytes(qtype, E, rows, K, T, topk))


def qmatmul_prefill_moe(qtype: int, w, E: int, rows: int, K: int, xq, T: int, ids, rw, topk: int, y, ws=None,
                        ws_bytes: int = 0, stream=None) -> None:
    _check(lib.qmatmul_prefill_moe(qtype, _ptr(w), E, rows, K, _ptr(xq), T, _ptr(ids), _ptr(rw), topk, _ptr(y),
                                   _ptr(ws), ws_bytes, _stream(stream)))


def qmatmul_prefill_moe_noalloc(qtype: int, w, E: int, rows: int, K: int, xq, T: int, ids, rw, topk: int, y,
                                stream=None) -> None:
    _check(lib.qmatmul_prefill_moe_noalloc(qtype, _ptr(w), E, rows, K, _ptr(xq), T, _ptr(ids), _ptr(rw), topk,
                                           _ptr(y), _stream(stream)))


# ---- the key/value cache, attention and log probabilities.  These check their
# tensors' devices, types, strides and sizes, which the C side cannot see (it
# takes addresses; so do these functions, as ints, unchecked).
def _flat(dev, what, t, dtype, need):
    """Device pointer of a contiguous tensor of at least ``need`` elements on GPU ``dev`` (None -> NULL, an int
    passes through)."""
    if t.__class__ is int or t is None:
        return t
    if t.get_device() != dev or t.numel() < need or (dtype is not None and t.dtype is not dtype) or not t.is_contiguous():
        _refuse(dev, what, t, dtype, need)
    return t.data_ptr()


def _bytes(dev, what, t, need):
    """_flat of a workspace of at least ``need`` bytes."""
    if t.__class__ is int or t is None:
        return t
    return _flat(dev, what, t, None, -(-need // t.element_size()))


def _rows(dev, what, t, dtype, T, stride, row):
    """Device pointer of T rows of ``row`` values each, ``stride`` elements apart (None and ints as in _flat)."""
    if t.__class__ is int or t is None:
        return t
    if t.get_device() != dev or (dtype is not None and t.dtype is not dtype):
        _refuse(dev, what, t, dtype)
    s = t.stride()
    if len(s) == 2:
        n, m = t.shape
        fine = s[0] == stride and s[1] == 1
    elif len(s) == 3:
        n, heads, m = t.shape
        fine = s[0] == stride and s[1] == m and s[2] == 1
        m *= heads
    else:
        fine = False
    if not fine or n < T or m < row:
        _check_rows(what, t, T, stride, row)
    return t.data_ptr()


def _check_rows(what, t, T, stride, row):
    """Any tensor's rows: a row lies in the last axes whose elements follow each other, and rows begin where one of
    the axes before has its next element (or a whole number of them on).  Axes of one element, the rows of a flat
    buffer and a single row's stride are free."""
    axes = [(n, s) for n, s in zip(t.shape, t.stride()) if n != 1]
    run, starts = 1, [1]
    while axes and axes[-1][1] == run:
        run *= axes.pop()[0]
        starts.append(run)
    if axes:
        n, step = axes[-1]
        one = all(outer[1] == inner[0] * inner[1] for outer, inner in zip(axes, axes[1:]))
        fine = run >= row and (T <= 1 or (step > 0 and stride % step == 0 and (one or (T - 1) * stride < n * step)))
    else:
        fine = T <= 1 or t.dim() == 1 or any(n >= row and stride % n == 0 for n in starts)
    reach = run + sum((n - 1) * s for n, s in axes) if t.numel() else 0
    if not fine or (T - 1) * stride + row > reach and T > 0:
        raise ValueError(f"{what}, of shape {tuple(t.shape)} and strides {t.stride()}, does not hold {T} rows of "
                         f"{row} values, {stride} elements apart")


def _refuse(dev, what, t, dtype, need=0):
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{what} is {t.dtype}, {dtype} is taken")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, the call's device is cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    raise ValueError(f"{what} has {t.numel()} elements, {need} are needed")


def _device() -> int:
    """The current device, on which the calls below run (-1 on a machine without one)."""
    return torch.cuda.current_device() if torch.cuda.is_available() else -1


if torch.cuda.device_count() > 0:
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(dev, stream) -> int | None:
    """_stream(stream), the current device being known."""
    if stream is None and _raw_stream is not None and dev >= 0:
        return _raw_stream(dev)
    return _stream(stream)


_TYPES = {Q8K_F32: torch.float32, Q8K_F16: torch.float16, Q8K_BF16: torch.bfloat16}


class KVCache:
    """A paged 8-bit key/value cache (q8k_kv_cache): ``data`` is a device buffer of
    ``q8k_kv_bytes(pages, kv_heads, head_dim)`` bytes, kept alive by this object."""

    def __init__(self, data, pages: int, kv_heads: int, head_dim: int):
        need = q8k_kv_bytes(pages, kv_heads, head_dim)
        if not isinstance(data, int) and data is not None:
            if not data.is_contiguous() or data.numel() * data.element_size() < need:
                raise ValueError(f"a cache of {pages} pages, {kv_heads} heads of {head_dim} is {need} contiguous bytes")
        self.data, self.pages, self.kv_heads, self.head_dim = data, pages, kv_heads, head_dim
        self.device = data.get_device() if isinstance(data, torch.Tensor) else None
        self.struct = _KVStruct(_ptr(data), pages, kv_heads, head_dim)
        self.ref = ctypes.addressof(self.struct)


class Rope:
    """A position rotation (q8k_rope): ``table`` fp32 [positions][dim], cosines then sines,
    kept alive by this object; ``pairs`` Q8K_ROPE_HALF or Q8K_ROPE_ADJACENT."""

    def __init__(self, table, positions: int, dim: int, pairs: int = Q8K_ROPE_HALF):
        if not isinstance(table, int) and table is not None:
            if table.dtype is not torch.float32 or not table.is_contiguous() or table.numel() < positions * dim:
                raise ValueError(f"a rotation table is contiguous fp32 [{positions}][{dim}]")
        self.table, self.positions, self.dim, self.pairs = table, positions, dim, pairs
        self.device = table.get_device() if isinstance(table, torch.Tensor) else None
        self.struct = _RopeStruct(_ptr(table), positions, dim, pairs)
        self.ref = ctypes.addressof(self.struct)


def _kv(dev, kv):
    if kv.device != dev and kv.device is not None:
        _refuse(dev, "kv", kv.data, None)
    return kv.ref


def _rope(dev, rope):
    if rope is None:
        return None
    if rope.device != dev and rope.device is not None:
        _refuse(dev, "rope", rope.table, None)
    return rope.ref


def q8k_kv_bytes(pages: int, kv_heads: int, head_dim: int) -> int:
    return int(lib.q8k_kv_bytes(pages, kv_heads, head_dim))


def q8k_kv_append(dtype: int, k, k_stride: int, v, v_stride: int, T: int, pos, rope, slots, kv, stream=None) -> None:
    dev, t = _device(), _TYPES.get(dtype)
    row = kv.kv_heads * kv.head_dim
    _check(lib.q8k_kv_append(dtype, _rows(dev, "k", k, t, T, k_stride, row), k_stride,
                             _rows(dev, "v", v, t, T, v_stride, row), v_stride, T,
                             _flat(dev, "pos", pos, torch.int32, 0 if rope is None else T), _rope(dev, rope),
                             _flat(dev, "slots", slots, torch.int32, T), _kv(dev, kv), _stream_of(dev, stream)))


def q8k_kv_read(dtype: int, kv, slots, T: int, k, v, stream=None) -> None:
    dev, t = _device(), _TYPES.get(dtype)
    n = T * kv.kv_heads * kv.head_dim
    _check(lib.q8k_kv_read(dtype, _kv(dev, kv), _flat(dev, "slots", slots, torch.int32, T), T, _flat(dev, "k", k, t, n),
                           _flat(dev, "v", v, t, n), _stream_of(dev, stream)))


def qattend_workspace_bytes(kv, q_heads: int, B: int, Tq: int, max_q: int, max_len: int) -> int:
    return int(lib.qattend_workspace_bytes(kv.ref, q_heads, B, Tq, max_q, max_len))


def qattend(dtype: int, q, q_stride: int, q_heads: int, kv, B: int, cu_q, Tq: int, max_q: int, page_table,
            max_pages: int, kv_len, max_len: int, scale: float, window: int, pos, rope, out, lse=None, ws=None,
            ws_bytes: int = 0, stream=None) -> None:
    dev, t = _device(), _TYPES.get(dtype)
    i32 = torch.int32
    row = q_heads * kv.head_dim
    _check(lib.qattend(dtype, _rows(dev, "q", q, t, Tq, q_stride, row), q_stride, q_heads, _kv(dev, kv), B,
                       _flat(dev, "cu_q", cu_q, i32, B + 1), Tq, max_q,
                       _flat(dev, "page_table", page_table, i32, B * max_pages), max_pages,
                       _flat(dev, "kv_len", kv_len, i32, B), max_len, scale, window,
                       _flat(dev, "pos", pos, i32, 0 if rope is None else Tq), _rope(dev, rope),
                       _flat(dev, "out", out, t, Tq * row), _flat(dev, "lse", lse, torch.float32, Tq * q_heads),
                       _bytes(dev, "ws", ws, ws_bytes), ws_bytes, _stream_of(dev, stream)))


def qlogprobs_workspace_bytes(T: int, V: int, topn: int) -> int:
    return int(lib.qlogprobs_workspace_bytes(T, V, topn))


def qlogprobs(dtype: int, logits, stride: int, T: int, V: int, targets, logprob, entropy=None, lse=None, topn: int = 0,
              top_ids=None, top_logprob=None, ws=None, ws_bytes: int = 0, stream=None) -> None:
    dev, f32 = _device(), torch.float32
    _check(lib.qlogprobs(dtype, _rows(dev, "logits", logits, _TYPES.get(dtype), T, stride, V), stride, T, V,
                         _flat(dev, "targets", targets, torch.int32, T), _flat(dev, "logprob", logprob, f32, T),
                         _flat(dev, "entropy", entropy, f32, T), _flat(dev, "lse", lse, f32, T), topn,
                         _flat(dev, "top_ids", top_ids, torch.int32, T * topn),
                         _flat(dev, "top_logprob", top_logprob, f32, T * topn), _bytes(dev, "ws", ws, ws_bytes), ws_bytes,
                         _stream_of(dev, stream)))


def q8k_debug_subblock_sums(qtype: int, w, rows: int, K: int, xq, y, S, stream=None) -> None:
    _check(lib.q8k_debug_subblock_sums(qtype, _ptr(w), rows, K, _ptr(xq), _ptr(y), _ptr(S), _stream(stream)))


def q8k_debug_prefill_block_sums(qtype: int, w, rows: int, K: int, xq, M: int, y, I, stream=None) -> None:
    _check(lib.q8k_debug_prefill_block_sums(qtype, _ptr(w), rows, K, _ptr(xq), M, _ptr(y), _ptr(I),
                                            _stream(stream)))


def q8k_debug_moe_subblock_sums(qtype: int, w, E: int, rows: int, K: int, xq, T: int, ids, rw, topk: int, y, S,
                                stream=None) -> None:
    _check(lib.q8k_debug_moe_subblock_sums(qtype, _ptr(w), E, rows, K, _ptr(xq), T, _ptr(ids), _ptr(rw), topk,
                                           _ptr(y), _ptr(S), _stream(stream)))


def q8k_debug_wave_sums(out, stream=None) -> None:
    _check(lib.q8k_debug_wave_sums(_ptr(out), _stream(stream)))


def q8k_debug_last_launches() -> list:
    """Host kernel handles the calling thread's last operation enqueued, in order."""
    buf = (_P * 16)()
    n = int(lib.q8k_debug_last_launches(buf, 16))
    return [int(buf[i] or 0) for i in range(min(n, 16))] + [0] * max(0, n - 16)
