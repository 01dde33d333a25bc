"""Python binding of the C ABI in include/cpt.h (argument marshalling only).

Every function has the name of the C call it wraps. Tensors are torch CUDA
tensors; the binding turns them into device pointers, passes the current
torch stream (or the one given), and raises ``CptError`` on any non-zero
status with the library's message. ctypes releases the GIL for the length of
each call, as the pages' binding does ("Add stream-ordered CP gradient
return primitive", TransformerEngine PR 3235, "Greptile Summary": the
function is registered with a GIL-release guard).

The shared library must have been built (``context_attention_token_gb300.build``);
importing this module without it raises ImportError: there is no fallback.
With CPT_LIBRARY_VARIANT=checked in the environment the binding loads the
bounds-checked build (libcpt_checked.so) instead of libcpt.so.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_VARIANT = os.environ.get("CPT_LIBRARY_VARIANT", "release")
if _VARIANT not in ("release", "checked"):
    raise ImportError(f"CPT_LIBRARY_VARIANT={_VARIANT!r}: expected 'release' or 'checked'")
_LIB_PATH = os.path.join(_PKG, "libcpt.so" if _VARIANT == "release" else "libcpt_checked.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is missing: build it with `python -m context_attention_token_gb300.build` "
        "(the CUDA path has no fallback)")

_lib = ctypes.CDLL(_LIB_PATH)

# ------------------------------------------------------------------ constants
CPT_OK = 0
CPT_ERR_INVALID_ARG = 1
CPT_ERR_NOT_DIVISIBLE = 2
CPT_ERR_UNSUPPORTED = 3
CPT_ERR_ALIAS = 4
CPT_ERR_DEVICE = 5
CPT_ERR_ALIGNMENT = 6
CPT_ERR_TIMEOUT = 7
CPT_ERR_CUDA = 8
CPT_ERR_WORKSPACE = 9
CPT_ERR_NOT_PUBLISHED = 10

CPT_LAYOUT_DUAL_CHUNK_SWAP = 0
CPT_LAYOUT_PACKED_CONTIGUOUS = 1
CPT_LAYOUT_RETIRED_PACKED_SUPER_SEQUENCE = 2
CPT_LAYOUT_DUAL_CHUNK_SWAP_PADDED = 3
CPT_F32 = 0
CPT_BF16 = 1
CPT_WAIT_BOUNDED = 0
CPT_WAIT_DRIVER = 1
CPT_MAX_CP_SIZE = 8
CPT_KERNEL_AUTO = 0
CPT_KERNEL_LOADS = 1
CPT_KERNEL_BULK = 2
CPT_CALL_ROW_GATHER = 0
CPT_CALL_GRAD_RETURN = 1
CPT_CALL_SLOT_REDUCE = 2
CPT_ROTARY_HALF = 0
CPT_ROTARY_INTERLEAVED = 1
CPT_ROTARY_MAX_AXES = 8
CPT_ORDER_GLOBAL = 0
CPT_ORDER_LOCAL = 1
CPT_GATE_NONE = 0
CPT_GATE_TOKEN = 1
CPT_GATE_DOCUMENT = 2
CPT_RESIDUAL_MAX_ROW = 8192
CPT_ATTENTION_MAX_HEADS = 1024
CPT_ATTENTION_MAX_TOKENS = 2147482624

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_u64 = ctypes.c_uint64
_sz = ctypes.c_size_t


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("cpt_last_error_string", ctypes.c_char_p)
_sig("cpt_status_string", ctypes.c_char_p, ctypes.c_int)
_sig("cpt_validate_layout", ctypes.c_int, ctypes.c_int, _i32, _vp, _i32, _i64)
_sig("cpt_plan_workspace_bytes", _sz, ctypes.c_int, _i32, _i32, _i64)
_sig("cpt_plan_create", ctypes.c_int, ctypes.c_int, _i32, _vp, _i32, _i64, _vp, _sz, _vp,
     ctypes.POINTER(_vp))
_sig("cpt_plan_destroy", ctypes.c_int, _vp)
_sig("cpt_plan_info", ctypes.c_int, _vp, ctypes.POINTER(_i64), ctypes.POINTER(_i32), ctypes.POINTER(_i32))
_sig("cpt_plan_padded_tokens", ctypes.c_int, _vp, ctypes.POINTER(_i64))
_sig("cpt_layout_padded_tokens", ctypes.c_int, ctypes.c_int, _i32, _vp, _i32, _i64,
     ctypes.POINTER(_i64))
_sig("cpt_thd_real_lengths", ctypes.c_int, _vp, _vp, _vp)
_sig("cpt_index_map", ctypes.c_int, _vp, _vp, _vp, _vp)
_sig("cpt_thd_metadata", ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp)
_sig("cpt_partition", ctypes.c_int, _vp, _i32, _vp, _vp, _i64, ctypes.c_int, _vp)
_sig("cpt_grad_return_accumulate", ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64, ctypes.c_int,
     ctypes.c_int, _vp)
_sig("cpt_partition_rows", ctypes.c_int, _vp, _i32, _vp, _vp, _i64, ctypes.c_int, _i64, _i64, _vp)
_sig("cpt_grad_return_rows", ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64, ctypes.c_int, ctypes.c_int,
     _i64, _i64, _vp)
_sig("cpt_restore", ctypes.c_int, _vp, _i32, _vp, _vp, _i64, ctypes.c_int, _vp)
_sig("cpt_grad_return", ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64, ctypes.c_int, ctypes.c_int, _vp)
_sig("cpt_grad_return_noalloc", ctypes.c_int, ctypes.c_int, _i32, _vp, _i32, _i64, _vp, _vp, _vp, _vp,
     _i64, ctypes.c_int, ctypes.c_int, _vp)
_sig("cpt_grad_scatter", ctypes.c_int, _vp, _i32, _vp, _vp, _vp, _i64, ctypes.c_int, _vp)
_sig("cpt_epoch_create", ctypes.c_int, _i32, _vp, _vp, _vp, ctypes.POINTER(_vp))
_sig("cpt_epoch_destroy", ctypes.c_int, _vp)
_sig("cpt_epoch_advance", ctypes.c_int, _vp, ctypes.POINTER(ctypes.c_uint32))
_sig("cpt_epoch_set", ctypes.c_int, _vp, ctypes.c_uint32)
_sig("cpt_epoch_publish", ctypes.c_int, _vp, _i32, _vp)
_sig("cpt_epoch_wait", ctypes.c_int, _vp, _i32, _u64, ctypes.c_int, _vp)
_sig("cpt_epoch_status", ctypes.c_int, _vp, _i32, _vp, ctypes.POINTER(_i32))
_sig("cpt_kernel_wait_timeouts", ctypes.c_int, ctypes.POINTER(ctypes.c_uint32), _i32)
_sig("cpt_set_kernel_path", ctypes.c_int, _i32)
_sig("cpt_test_stall_bulk_waits", ctypes.c_int, _i32)
_sig("cpt_kernel_path_of", ctypes.c_int, _i32, _i32, _i32, _i32, _i32, _i64, _i64, ctypes.POINTER(_i32))
_sig("cpt_slot_reduce", ctypes.c_int, _vp, _i32, _i64, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp)
_sig("cpt_stream_ceiling", ctypes.c_int, _vp, _i32, _vp, _i64, _i32, _i32, _i32, _vp)
_sig("cpt_rotary_create", ctypes.c_int, _i32, _i32, _vp, _vp, _i32, ctypes.c_int, ctypes.POINTER(_vp))
_sig("cpt_rotary_destroy", ctypes.c_int, _vp)
_sig("cpt_rotary_apply", ctypes.c_int, _vp, _vp, _i32, _vp, _vp, _vp, ctypes.c_int, _vp, ctypes.c_int,
     ctypes.c_int, _i32, _vp)
_sig("cpt_attention", ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, ctypes.c_int,
     ctypes.c_float, _i64, _i32, _vp)
_sig("cpt_attention_backward_workspace_bytes", _sz, _vp, _i32, _i32, _i32)
_sig("cpt_attention_backward", ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
     _i32, ctypes.c_int, ctypes.c_float, _i64, _i32, _vp, _sz, _vp)


class _Residual(ctypes.Structure):
    """struct cpt_residual"""

    _fields_ = [("post_weight", _vp), ("pre_weight", _vp), ("gate", _vp), ("gate_kind", ctypes.c_int),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float), ("p", ctypes.c_double), ("rng", _vp),
                ("site", ctypes.c_uint32)]


_sig("cpt_dropout", ctypes.c_int, _vp, _vp, _vp, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_double, _vp,
     ctypes.c_uint32, _vp)
_sig("cpt_residual_norm", ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64, ctypes.c_int, ctypes.c_int,
     ctypes.POINTER(_Residual), _vp)
_sig("cpt_residual_norm_backward_workspace_bytes", _sz, _vp, _i64, ctypes.c_int)
_sig("cpt_residual_norm_backward", ctypes.c_int, *[_vp] * 10, _i64, ctypes.c_int, ctypes.c_int,
     ctypes.POINTER(_Residual), _vp, _sz, _vp)
_sig("cpt_token_logprob", ctypes.c_int, *[_vp] * 5, _i64, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_float, _vp)
_sig("cpt_token_logprob_backward", ctypes.c_int, *[_vp] * 6, _i64, _i64, ctypes.c_int, ctypes.c_int,
     ctypes.c_float, _vp)
_sig("cpt_policy_loss", ctypes.c_int, *[_vp] * 7, ctypes.c_double, ctypes.c_double, ctypes.c_double, _vp, _vp, _vp)
_sig("cpt_bounds_checked", _i32)
_sig("cpt_bounds_violations", ctypes.c_int, ctypes.POINTER(ctypes.c_uint32), _i32)


def library_path() -> str:
    return _LIB_PATH


def exported_symbols(names):
    """Names (of the given ones) the loaded library exports."""
    out = []
    for n in names:
        try:
            getattr(_lib, n)
            out.append(n)
        except AttributeError:
            pass
    return out


class CptError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        name = _lib.cpt_status_string(status).decode()
        super().__init__(f"{name}: {message}")


def _check(status: int):
    if status != CPT_OK:
        raise CptError(status, _lib.cpt_last_error_string().decode())


def cpt_last_error_string() -> str:
    return _lib.cpt_last_error_string().decode()


def cpt_status_string(status: int) -> str:
    return _lib.cpt_status_string(status).decode()


# ------------------------------------------------------------------ marshalling

# The current stream's handle without building a Stream object (3 us less a
# call); torch builds that lack these calls take the public way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None and _raw_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return CPT_F32
    if t.dtype == torch.bfloat16:
        return CPT_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# ctypes array types of n device pointers, built once per n
_PTR_ARRAYS = {}


def _ptr_array(items):
    """Device pointers of the items as a C array (passed by its address)."""
    n = len(items)
    kind = _PTR_ARRAYS.get(n)
    if kind is None:
        kind = _PTR_ARRAYS.setdefault(n, _vp * n)
    return kind(*[_ptr(x) for x in items])


class _Parts:
    """Device pointers of `parts` equally shaped tensors, given as one
    contiguous [parts, ...] tensor or as a sequence of tensors, with the
    shape and dtype of one part."""

    __slots__ = ("ptrs", "shape", "dtype", "part_bytes")

    def __init__(self, t, parts: int):
        if isinstance(t, torch.Tensor):
            if t.dim() == 0 or t.shape[0] != parts:
                raise ValueError(f"leading dimension of {tuple(t.shape)} != {parts}")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
            base = t.data_ptr()
            step = t.stride(0) * t.element_size()
            self.ptrs = [base + i * step for i in range(parts)]
            self.shape = tuple(t.shape[1:])
            self.dtype = t.dtype
            self.part_bytes = step
        else:
            t = list(t)
            if len(t) != parts:
                raise ValueError(f"expected {parts} tensors, got {len(t)}")
            first = t[0]
            shape, dtype = first.shape, first.dtype
            ptrs = []
            for x in t:
                if isinstance(x, int):
                    raise TypeError("parts must be tensors")
                if x.shape != shape or x.dtype != dtype:
                    raise ValueError("the parts differ in shape or dtype")
                if not x.is_contiguous():
                    raise ValueError("tensors must be contiguous")
                ptrs.append(x.data_ptr())
            self.ptrs = ptrs
            self.shape = tuple(shape)
            self.dtype = dtype
            self.part_bytes = first.numel() * first.element_size()

    def array(self):
        """The pointers as a C array; ctypes passes an array argument by its
        address, and the call keeps the array alive while it runs."""
        n = len(self.ptrs)
        kind = _PTR_ARRAYS.get(n)
        if kind is None:
            kind = _PTR_ARRAYS.setdefault(n, _vp * n)
        return kind(*self.ptrs)

    def row_elems(self) -> int:
        n = 1
        for d in self.shape[1:]:
            n *= int(d)
        return n

    def code(self) -> int:
        if self.dtype == torch.float32:
            return CPT_F32
        if self.dtype == torch.bfloat16:
            return CPT_BF16
        raise TypeError(f"unsupported dtype {self.dtype} (float32 or bfloat16)")


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


_ELEM_BYTES = {torch.float32: 4, torch.bfloat16: 2, torch.int32: 4}


def _elem_bytes(dtype) -> int:
    n = _ELEM_BYTES.get(dtype)
    return n if n is not None else torch.empty(0, dtype=dtype).element_size()


def _need(t, nbytes: int, what: str, dtype=None):
    """Refuse a buffer smaller than the bytes the call will touch (the C ABI
    sees only its address), or of the wrong element type."""
    if t is None:
        return
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} has dtype {t.dtype}, expected {dtype}")
    if _nbytes(t) < nbytes:
        raise ValueError(f"{what} holds {_nbytes(t)} bytes but the call touches {nbytes}")


def _need_parts(parts, rows: int, row_elems: int, what: str):
    """Every part of `parts` must hold `rows` rows of `row_elems` elements."""
    if parts is None:
        return
    if parts.row_elems() != row_elems:
        raise ValueError(f"{what} rows have {parts.row_elems()} elements, expected {row_elems}")
    need = rows * row_elems * _elem_bytes(parts.dtype)
    if parts.part_bytes < need:
        raise ValueError(f"each part of {what} holds {parts.part_bytes} bytes but the call touches {need}")


def _same_kind(ts, what: str):
    """Tensors of one call that must share dtype and row width."""
    for t in ts[1:]:
        if t.dtype != ts[0].dtype or _row_elems(t) != _row_elems(ts[0]):
            raise ValueError(f"the {what} tensors differ in dtype or row width")


def _cu_array(cu_seqlens):
    vals = [int(v) for v in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    return (_i32 * len(vals))(*vals), len(vals) - 1


# ------------------------------------------------------------------ host-only

def cpt_validate_layout(layout: int, cp_size: int, cu_seqlens, total_tokens: int) -> int:
    """Status code of the host-side partition check (0 = valid)."""
    arr, n = _cu_array(cu_seqlens)
    return _lib.cpt_validate_layout(layout, cp_size, ctypes.cast(arr, _vp), n, total_tokens)


def cpt_plan_workspace_bytes(layout: int, cp_size: int, n_docs: int, total_tokens: int) -> int:
    return int(_lib.cpt_plan_workspace_bytes(layout, cp_size, n_docs, total_tokens))


def cpt_layout_padded_tokens(layout: int, cp_size: int, cu_seqlens, total_tokens: int) -> int:
    """Tokens of the buffer the layout partitions (the padded total for the
    padded layout, else total_tokens); raises CptError for a batch the
    layout rejects."""
    arr, n = _cu_array(cu_seqlens)
    v = _i64(0)
    _check(_lib.cpt_layout_padded_tokens(layout, cp_size, ctypes.cast(arr, _vp), n, total_tokens,
                                         ctypes.byref(v)))
    return int(v.value)


# ------------------------------------------------------------------ plan

class Plan:
    """Host handle of a plan plus the workspace tensor it lives in."""

    def __init__(self, handle: int, workspace: torch.Tensor, layout: int, cp_size: int,
                 n_docs: int, total_tokens: int, padded_tokens: int):
        self.handle = handle
        self.workspace = workspace
        self.layout = layout
        self.cp_size = cp_size
        self.n_docs = n_docs
        self.total_tokens = total_tokens
        self.padded_tokens = padded_tokens

    @property
    def local_tokens(self) -> int:
        return self.padded_tokens // self.cp_size

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            _lib.cpt_plan_destroy(h)


def cpt_plan_create(layout: int, cp_size: int, cu_seqlens, total_tokens: int,
                    workspace: torch.Tensor | None = None, stream=None) -> Plan:
    arr, n = _cu_array(cu_seqlens)
    need = cpt_plan_workspace_bytes(layout, cp_size, n, total_tokens)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    h = _vp()
    _check(_lib.cpt_plan_create(layout, cp_size, ctypes.cast(arr, _vp), n, total_tokens,
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream), ctypes.byref(h)))
    tp = _i64()
    _check(_lib.cpt_plan_padded_tokens(h.value, ctypes.byref(tp)))
    return Plan(h.value, workspace, layout, cp_size, n, total_tokens, tp.value)


def cpt_plan_destroy(plan: Plan) -> None:
    h, plan.handle = plan.handle, None
    if h:
        _check(_lib.cpt_plan_destroy(h))


def cpt_plan_info(plan: Plan):
    """(total_tokens, cp_size, n_docs) as the library holds them."""
    T, P, n = _i64(), _i32(), _i32()
    _check(_lib.cpt_plan_info(plan.handle, ctypes.byref(T), ctypes.byref(P), ctypes.byref(n)))
    return T.value, P.value, n.value


def cpt_plan_padded_tokens(plan: Plan) -> int:
    v = _i64()
    _check(_lib.cpt_plan_padded_tokens(plan.handle, ctypes.byref(v)))
    return v.value


def cpt_thd_real_lengths(plan: Plan, real_len: torch.Tensor, stream=None):
    """real_len[r][i] ([P, n] int32) = real tokens of document i on rank r."""
    _need(real_len, 4 * plan.cp_size * plan.n_docs, "real_len", torch.int32)
    _check(_lib.cpt_thd_real_lengths(plan.handle, _ptr(real_len), _stream(stream)))


def cpt_index_map(plan: Plan, l2g: torch.Tensor, g2l: torch.Tensor | None = None, stream=None):
    _need(l2g, 4 * plan.padded_tokens, "l2g", torch.int32)
    _need(g2l, 4 * plan.padded_tokens, "g2l", torch.int32)
    _check(_lib.cpt_index_map(plan.handle, _ptr(l2g), _ptr(g2l), _stream(stream)))


def cpt_thd_metadata(plan: Plan, num_segs, seg_doc_first, cu_local, seg_offsets, stream=None):
    P = plan.cp_size
    _need(num_segs, 4 * P, "num_segs", torch.int32)
    _need(seg_doc_first, 4 * P, "seg_doc_first", torch.int32)
    _need(cu_local, 4 * P * (plan.n_docs + 1), "cu_local", torch.int32)
    _need(seg_offsets, 4 * (P + 1), "seg_offsets", torch.int32)
    _check(_lib.cpt_thd_metadata(plan.handle, _ptr(num_segs), _ptr(seg_doc_first), _ptr(cu_local),
                                 _ptr(seg_offsets), _stream(stream)))


def cpt_partition(plan: Plan, srcs, dsts, stream=None):
    """dsts[t] ([P, T/P, ...]) = rank-local reorder of srcs[t] ([T, ...])."""
    srcs, dsts = list(srcs), list(dsts)
    _check_gather(plan, srcs, dsts, plan.total_tokens, plan.padded_tokens, _row_elems(srcs[0]) if srcs else 0)
    _check(_lib.cpt_partition(plan.handle, len(srcs), _ptr_array(srcs),
                              _ptr_array(dsts), _row_elems(srcs[0]), _dtype_code(srcs[0]),
                              _stream(stream)))


def cpt_partition_rows(plan: Plan, srcs, dsts, local_begin: int, local_count: int, stream=None):
    """cpt_partition for flattened local rows [local_begin, local_begin + local_count) only."""
    srcs, dsts = list(srcs), list(dsts)
    _check_gather(plan, srcs, dsts, plan.total_tokens, plan.padded_tokens, _row_elems(srcs[0]) if srcs else 0)
    _check(_lib.cpt_partition_rows(plan.handle, len(srcs), _ptr_array(srcs),
                                   _ptr_array(dsts), _row_elems(srcs[0]),
                                   _dtype_code(srcs[0]), local_begin, local_count, _stream(stream)))


def cpt_restore(plan: Plan, srcs, dsts, stream=None):
    """dsts[t] ([T, ...]) = global-order copy of the rank-local srcs[t] ([P, T/P, ...])."""
    srcs, dsts = list(srcs), list(dsts)
    _check_gather(plan, srcs, dsts, plan.padded_tokens, plan.total_tokens, _row_elems(dsts[0]) if dsts else 0)
    _check(_lib.cpt_restore(plan.handle, len(srcs), _ptr_array(srcs),
                            _ptr_array(dsts), _row_elems(dsts[0]),
                            _dtype_code(srcs[0]), _stream(stream)))


def _check_gather(plan: Plan, srcs, dsts, src_rows: int, dst_rows: int, row: int):
    """Partition, restore: as many sources as destinations, one dtype, every
    buffer large enough for its rows of `row` elements."""
    if len(srcs) != len(dsts):
        raise ValueError("srcs and dsts differ in length")
    if not srcs:
        return
    esz = srcs[0].element_size()
    for i, (a, b) in enumerate(zip(srcs, dsts)):
        if a.dtype != srcs[0].dtype or b.dtype != srcs[0].dtype:
            raise ValueError("srcs and dsts must share one dtype")
        _need(a, src_rows * row * esz, f"srcs[{i}]")
        _need(b, dst_rows * row * esz, f"dsts[{i}]")


def _row_elems(t: torch.Tensor) -> int:
    """Elements of one token row of a [T, ...] tensor."""
    n = 1
    for d in t.shape[1:]:
        n *= int(d)
    return n


def _check_grad_return(Tpad: int, P: int, dkw, dvw, dko, dvo):
    """Writers of Tpad rows, owners of Tpad / P rows, one row width; the dV
    pair like the dK pair."""
    row = dkw.row_elems()
    _need_parts(dkw, Tpad, row, "dk_writers")
    _need_parts(dko, Tpad // P, row, "dk_owners")
    if dvw is not None and dvo is not None:  # one without the other: the library refuses it
        if dvw.dtype != dkw.dtype or dvo.dtype != dko.dtype:
            raise ValueError("the dV pair must have the dtypes of the dK pair")
        _need_parts(dvw, Tpad, row, "dv_writers")
        _need_parts(dvo, Tpad // P, row, "dv_owners")


def _grad_return(fn, plan: Plan, dk_writers, dv_writers, dk_owners, dv_owners, stream):
    P = plan.cp_size
    dkw = _Parts(dk_writers, P)
    dko = _Parts(dk_owners, P)
    dvw = _Parts(dv_writers, P) if dv_writers is not None else None
    dvo = _Parts(dv_owners, P) if dv_owners is not None else None
    _check_grad_return(plan.padded_tokens, P, dkw, dvw, dko, dvo)
    _check(fn(plan.handle, dkw.array(), dvw.array() if dvw is not None else None, dko.array(),
              dvo.array() if dvo is not None else None, dkw.row_elems(), dkw.code(), dko.code(),
              _stream(stream)))


def cpt_grad_return(plan: Plan, dk_writers, dv_writers, dk_owners, dv_owners, stream=None):
    """Owners' local dK (and dV) = ordered sum over writers' global gradients.

    Each of the four arguments is a [P, ...] tensor or a list of P tensors;
    the dV pair may be None.
    """
    _grad_return(_lib.cpt_grad_return, plan, dk_writers, dv_writers, dk_owners, dv_owners, stream)


def cpt_grad_return_rows(plan: Plan, dk_writers, dv_writers, dk_owners, dv_owners,
                         local_begin: int, local_count: int, stream=None):
    """cpt_grad_return for flattened owner-major local rows [local_begin, +local_count) only."""
    P = plan.cp_size
    dkw = _Parts(dk_writers, P)
    dko = _Parts(dk_owners, P)
    dvw = _Parts(dv_writers, P) if dv_writers is not None else None
    dvo = _Parts(dv_owners, P) if dv_owners is not None else None
    _check_grad_return(plan.padded_tokens, P, dkw, dvw, dko, dvo)
    _check(_lib.cpt_grad_return_rows(
        plan.handle, dkw.array(), dvw.array() if dvw is not None else None, dko.array(),
        dvo.array() if dvo is not None else None, dkw.row_elems(), dkw.code(), dko.code(),
        local_begin, local_count, _stream(stream)))


def cpt_grad_return_accumulate(plan: Plan, dk_writers, dv_writers, dk_owners, dv_owners,
                               stream=None):
    """As cpt_grad_return, but the owners' current values start the sums."""
    _grad_return(_lib.cpt_grad_return_accumulate, plan, dk_writers, dv_writers, dk_owners,
                 dv_owners, stream)


CPT_NOALLOC_MAX_TOKENS = 1048576
CPT_NOALLOC_MAX_DOCS = 65536


def cpt_grad_return_noalloc(layout: int, cp_size: int, cu_seqlens, total_tokens: int, dk_writers,
                            dv_writers, dk_owners, dv_owners, stream=None):
    """cpt_grad_return without a plan or workspace, for callers that cannot
    allocate device memory: the map lives in a fixed-size array inside the
    library (at most CPT_NOALLOC_MAX_TOKENS tokens). Calls that overlap on
    the GPU share that array and race."""
    arr, n = _cu_array(cu_seqlens)
    P = cp_size
    dkw = _Parts(dk_writers, P)
    dko = _Parts(dk_owners, P)
    dvw = _Parts(dv_writers, P) if dv_writers is not None else None
    dvo = _Parts(dv_owners, P) if dv_owners is not None else None
    # the library sizes the map; batches it refuses (on layout or size
    # grounds) are left to the call itself to report
    Tmap = _i64(0)
    if _lib.cpt_layout_padded_tokens(layout, P, ctypes.cast(arr, _vp), n, total_tokens,
                                     ctypes.byref(Tmap)) != CPT_OK:
        Tmap.value = 0
    if 0 < Tmap.value <= CPT_NOALLOC_MAX_TOKENS and n <= CPT_NOALLOC_MAX_DOCS:
        _check_grad_return(Tmap.value, P, dkw, dvw, dko, dvo)
    _check(_lib.cpt_grad_return_noalloc(
        layout, P, ctypes.cast(arr, _vp), n, total_tokens, dkw.array(),
        dvw.array() if dvw is not None else None, dko.array(),
        dvo.array() if dvo is not None else None, dkw.row_elems(), dkw.code(), dko.code(),
        _stream(stream)))


def cpt_grad_scatter(plan: Plan, writer: int, src: torch.Tensor, slots, self_slot, stream=None):
    """slots[o] ([T/P, ...]) = writer's rows owned by o; self_slot must be slots[writer]."""
    sl = _Parts(slots, plan.cp_size)
    row = _row_elems(src)
    _need(src, plan.padded_tokens * row * src.element_size(), "src")
    if sl.dtype != src.dtype:
        raise ValueError("slots must have the dtype of src")
    _need_parts(sl, plan.padded_tokens // plan.cp_size, row, "slots")
    _check(_lib.cpt_grad_scatter(plan.handle, writer, _ptr(src), sl.array(), _ptr(self_slot),
                                 _row_elems(src), _dtype_code(src), _stream(stream)))


def cpt_slot_reduce(slots, dst: torch.Tensor, status: torch.Tensor | int | None = None, stream=None):
    n = slots.shape[0] if isinstance(slots, torch.Tensor) else len(slots)
    sl = _Parts(slots, n)
    numel = 1
    for d in sl.shape:
        numel *= int(d)
    _need(dst, numel * dst.element_size(), "dst")
    if isinstance(status, torch.Tensor):
        _need(status, 4, "status", torch.int32)
    _check(_lib.cpt_slot_reduce(sl.array(), n, numel, sl.code(), _dtype_code(dst), _ptr(dst),
                                _ptr(status), _stream(stream)))


# ------------------------------------------------------------------ attention layer

class Rotary:
    """Host handle of a rotation's frequencies and axes."""

    def __init__(self, handle: int, head_dim: int, n_axes: int):
        self.handle = handle
        self.head_dim = head_dim
        self.n_axes = n_axes

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            _lib.cpt_rotary_destroy(h)


def cpt_rotary_create(head_dim: int, inv_freq, axis_of_pair, n_axes: int,
                      pairing: int = CPT_ROTARY_HALF) -> Rotary:
    """Pair i of a head turns by pos[axis_of_pair[i]] * inv_freq[i]."""
    freq = [float(f) for f in inv_freq]
    axis = [int(a) for a in axis_of_pair]
    if len(freq) != len(axis):
        raise ValueError("inv_freq and axis_of_pair differ in length")
    n = len(freq)
    h = _vp()
    _check(_lib.cpt_rotary_create(head_dim, n, (ctypes.c_double * n)(*freq), (_i32 * n)(*axis), n_axes,
                                  pairing, ctypes.byref(h)))
    return Rotary(h.value, head_dim, n_axes)


def cpt_rotary_destroy(rotary: Rotary) -> None:
    h, rotary.handle = rotary.handle, None
    if h:
        _check(_lib.cpt_rotary_destroy(h))


def cpt_rotary_apply(rotary: Rotary, plan: Plan, srcs, dsts, positions: torch.Tensor,
                     src_order: int = CPT_ORDER_GLOBAL, dst_order: int = CPT_ORDER_LOCAL,
                     inverse: bool = False, stream=None):
    """dsts[t] = srcs[t] rotated by its tokens' positions ([n_axes, T] int32),
    moved from src_order to dst_order. Tensors are [T, heads, head_dim] in
    global and [P, T_pad/P, heads, head_dim] in local order."""
    srcs, dsts = list(srcs), list(dsts)
    if len(srcs) != len(dsts):
        raise ValueError("srcs and dsts differ in length")
    if not srcs:
        raise ValueError("no tensors")
    if src_order not in (0, 1) or dst_order not in (0, 1):
        raise ValueError("unknown order")
    rows_in = plan.padded_tokens if src_order else plan.total_tokens
    rows_out = plan.padded_tokens if dst_order else plan.total_tokens
    dtype, d, heads, n = srcs[0].dtype, rotary.head_dim, [], len(srcs)
    for i in range(n):
        a, b = srcs[i], dsts[i]
        if a.dtype != dtype or b.dtype != dtype:
            raise ValueError("srcs and dsts must share one dtype")
        sa, sb = a.shape, b.shape
        if len(sa) < 2 or sa[-1] != d or len(sb) < 2 or sb[-1] != d:
            raise ValueError(f"srcs[{i}] or dsts[{i}] has no heads of {d} elements")
        h = sa[-2]
        if sb[-2] != h:
            raise ValueError(f"srcs[{i}] and dsts[{i}] differ in heads")
        heads.append(h)
        if a.numel() < rows_in * h * d or b.numel() < rows_out * h * d:
            raise ValueError(f"srcs[{i}] or dsts[{i}] holds fewer than {rows_in} and {rows_out} rows")
    if positions.dtype != torch.int32 or positions.numel() < rotary.n_axes * plan.total_tokens:
        raise ValueError("positions must hold n_axes * total_tokens int32 values")
    _check(_lib.cpt_rotary_apply(rotary.handle, plan.handle, n, _ptr_array(srcs), _ptr_array(dsts),
                                 (_i32 * n)(*heads), _dtype_code(srcs[0]), _ptr(positions),
                                 src_order, dst_order, 1 if inverse else 0, _stream(stream)))


def _attention_shape(plan: Plan, q, k, like_q, like_k, lse):
    """(q_heads, kv_heads, head_dim, dtype code), every buffer large enough."""
    qs, ks = q.shape, k.shape
    if len(qs) < 2 or len(ks) < 2 or qs[-1] != ks[-1]:
        raise ValueError("q and k must end in [heads, head_dim] with one head_dim")
    hq, hk, d, dtype = qs[-2], ks[-2], qs[-1], q.dtype
    for group, heads, rows in ((like_q, hq, plan.padded_tokens), (like_k, hk, plan.total_tokens)):
        need = rows * heads * d
        for t in group:
            s = t.shape
            if t.dtype != dtype or len(s) < 2 or s[-1] != d or s[-2] != heads:
                raise ValueError("tensors of q's or k's kind differ in dtype, heads or head_dim")
            if t.numel() < need:
                raise ValueError(f"a tensor of {heads} heads holds {t.numel()} elements but the call touches {need}")
    if lse.dtype != torch.float32 or lse.numel() < hq * plan.padded_tokens:
        raise ValueError("lse must hold q_heads * padded_tokens float32 values")
    return hq, hk, d, _dtype_code(q)


_WINDOW_MAX, _SINKS_MAX = (1 << 63) - 1, (1 << 31) - 1


def _mask_argument(x, most: int):
    """A window or a number of sinks beyond the C type's range as its largest value (no document is
    longer), one below as -1, which the library refuses: ctypes would keep their lowest bits."""
    return x if -1 <= x <= most else (most if x > most else -1)


def cpt_attention(plan: Plan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                  lse: torch.Tensor, scale: float, window: int, sinks: int = 0, stream=None):
    """out ([P, T_pad/P, Hq, D], like q) and lse ([Hq, T_pad]) = causal attention
    of rank-local queries over the packed documents' keys and values ([T, Hkv,
    D], global order) with a sliding window and `sinks` first tokens."""
    hq, hk, d, code = _attention_shape(plan, q, k, (q, out), (k, v), lse)
    window, sinks = _mask_argument(window, _WINDOW_MAX), _mask_argument(sinks, _SINKS_MAX)
    _check(_lib.cpt_attention(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), hq, hk, d, code,
                              scale, window, sinks, _stream(stream)))


def cpt_attention_backward_workspace_bytes(plan: Plan, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(_lib.cpt_attention_backward_workspace_bytes(plan.handle, q_heads, kv_heads, head_dim))


def cpt_attention_backward(plan: Plan, q, k, v, out, lse, dout, dq, dk_writers, dv_writers, scale: float,
                           window: int, sinks: int = 0, workspace: torch.Tensor | None = None, stream=None):
    """dq (like q) and every writer's dk and dv ([P, T_pad, Hkv, D] or lists of P
    tensors) of cpt_attention. Without a workspace the binding allocates one
    from torch on the current stream."""
    hq, hk, d, code = _attention_shape(plan, q, k, (q, out, dout, dq), (k, v), lse)
    window, sinks = _mask_argument(window, _WINDOW_MAX), _mask_argument(sinks, _SINKS_MAX)
    P = plan.cp_size
    dkw, dvw = _Parts(dk_writers, P), _Parts(dv_writers, P)
    for parts, what in ((dkw, "dk_writers"), (dvw, "dv_writers")):
        if parts.dtype != q.dtype:
            raise ValueError(f"{what} must have the dtype of q")
        _need_parts(parts, plan.padded_tokens, hk * d, what)
    if workspace is None:
        if stream is not None:
            raise ValueError("give a workspace with a stream: torch allocates on its current stream only")
        need = cpt_attention_backward_workspace_bytes(plan, hq, hk, d)
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    _check(_lib.cpt_attention_backward(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                       _ptr(dq), dkw.array(), dvw.array(), hq, hk, d, code, scale, window, sinks,
                                       _ptr(workspace), _nbytes(workspace), _stream(stream)))


# ------------------------------------------------------------------ token rows

def _row_count(plan: Plan, order: int) -> int:
    if order not in (CPT_ORDER_GLOBAL, CPT_ORDER_LOCAL):
        raise ValueError("unknown order")
    return plan.padded_tokens if order else plan.total_tokens


def _row_width(plan: Plan, order: int, t: torch.Tensor) -> int:
    """Elements of a row of [P, T_pad/P, ...] or [T_pad, ...] (LOCAL), [T, ...] (GLOBAL)."""
    rows, shape = _row_count(plan, order), t.shape
    dims = len(shape)
    if order and dims > 2 and shape[0] == plan.cp_size and shape[0] * shape[1] == rows:
        lead = 2
    elif dims > 1 and shape[0] == rows:
        lead = 1
    else:
        raise ValueError(f"a tensor of shape {tuple(shape)} does not hold {rows} rows")
    if rows:
        return t.numel() // rows
    width = 1
    for n in shape[lead:]:
        width *= n
    return width


def _rows_of(plan: Plan, order: int, first, others, what: str) -> int:
    """Elements of a row of `first`, like which the others must be."""
    width, shape, dtype = _row_width(plan, order, first), first.shape, first.dtype
    for t in others:
        if t is None:
            continue
        if t.dtype != dtype:
            raise ValueError(f"{what} differ in dtype")
        if t.shape != shape and _row_width(plan, order, t) != width:
            raise ValueError(f"{what} differ in width")
    return width


def _there(t) -> int:
    """The pointer of an optional tensor. One without elements (an empty batch) has none, but is given all the
    same: the library does not look at it, only whether it is NULL."""
    return 0 if t is None else _ptr(t) or 16


def _rng_ptr(rng, p: float) -> int:
    if rng is None:
        return 0
    if rng.dtype not in (torch.int64, torch.uint64) or rng.numel() < 2:
        raise ValueError("rng must hold two 64-bit integers, seed and step")
    return _ptr(rng)


def cpt_dropout(plan: Plan, src: torch.Tensor, dst: torch.Tensor, p: float, rng: torch.Tensor | None = None,
                site: int = 0, order: int = CPT_ORDER_LOCAL, stream=None):
    """dst = dropout of src (dst may be src); the mask follows every row's token. `rng` is an int64
    tensor {seed, step} on the device. The gradient is the same call on the gradient."""
    width = _rows_of(plan, order, src, (dst,), "src and dst")
    _check(_lib.cpt_dropout(plan.handle, _ptr(src), _ptr(dst), width, _dtype_code(src), order, p, _rng_ptr(rng, p),
                            site & 0xFFFFFFFF, _stream(stream)))


def _floats(t, count: int, what: str) -> int:
    """The pointer of an optional float32 tensor of at least `count` elements."""
    if t is None:
        return 0
    if t.dtype != torch.float32 or t.numel() < count:
        raise ValueError(f"{what} must hold {count} float32 values")
    return _ptr(t)


def _row_weights(t, width: int, what: str) -> int:
    """The pointer of an optional row of float32 weights, one for every element of the rows."""
    if t is not None and t.numel() != width:
        raise ValueError(f"{what} must hold {width} float32 values, not {t.numel()}")
    return _floats(t, width, what)


def _check_gate(plan: Plan, t, width: int, order: int, per_document: bool, what: str):
    """A gate or its gradient: rows like h's, or one for every document (flat, too)."""
    rows = plan.n_docs if per_document else _row_count(plan, order)
    if t.numel() == rows * width and (t.dim() == 1 or (per_document and t.shape[0] == rows)):
        return
    if per_document or _row_width(plan, order, t) != width:
        raise ValueError(f"{what} must hold {rows} rows of {width} elements, not {tuple(t.shape)}")


def _residual_options(plan: Plan, width: int, dtype, order: int, post_weight, gate, gate_per_document, scale, p, rng,
                      site, pre_weight, eps):
    gate_ptr, kind = 0, CPT_GATE_NONE
    if gate is not None:
        if gate.dtype != dtype:
            raise ValueError("gate must be of the tensors' dtype")
        _check_gate(plan, gate, width, order, gate_per_document, "gate")
        gate_ptr, kind = _there(gate), CPT_GATE_DOCUMENT if gate_per_document else CPT_GATE_TOKEN
    return _Residual(_row_weights(post_weight, width, "post_weight"), _row_weights(pre_weight, width, "pre_weight"), gate_ptr,
                     kind, scale, eps, p, _rng_ptr(rng, p), site & 0xFFFFFFFF)


def cpt_residual_norm(plan: Plan, x: torch.Tensor, h, y, n, *, post_weight=None, gate=None,
                      gate_per_document: bool = False, scale: float = 1.0, p: float = 0.0, rng=None, site: int = 0,
                      pre_weight=None, eps: float = 1e-6, order: int = CPT_ORDER_LOCAL, stream=None):
    """y = x + scale * dropout(gate * norm(h) * post_weight) and n = norm(y) * pre_weight. What is None is left
    out: post_weight, gate (like h, or [n_docs, row] with gate_per_document), pre_weight with n, h with y. y may be x."""
    width = _rows_of(plan, order, x, (h, y, n), "x, h, y and n")
    o = _residual_options(plan, width, x.dtype, order, post_weight, gate, gate_per_document, scale, p, rng, site,
                          pre_weight, eps)
    _check(_lib.cpt_residual_norm(plan.handle, _ptr(x), _there(h), _there(y), _there(n), width, _dtype_code(x), order,
                                  ctypes.byref(o), _stream(stream)))


def cpt_residual_norm_backward_workspace_bytes(plan: Plan, row_elems: int, dtype: torch.dtype) -> int:
    code = {torch.float32: CPT_F32, torch.bfloat16: CPT_BF16}.get(dtype, -1)
    return int(_lib.cpt_residual_norm_backward_workspace_bytes(plan.handle, row_elems, code))


def cpt_residual_norm_backward(plan: Plan, h, y, dy, dn, dx: torch.Tensor, dh, *, dgate=None, dpost_weight=None,
                               dpre_weight=None, post_weight=None, gate=None, gate_per_document: bool = False,
                               scale: float = 1.0, p: float = 0.0, rng=None, site: int = 0, pre_weight=None,
                               eps: float = 1e-6, order: int = CPT_ORDER_LOCAL, workspace=None, stream=None):
    """Gradients of cpt_residual_norm from h, y (x where there was no h), dy and dn. dgate is float32 [n_docs, row]
    with gate_per_document; the weights' gradients are float32. dx may be dy. Without a workspace the
    binding allocates one from torch on the current stream."""
    width = _rows_of(plan, order, dx, (h, y, dy, dn, dh), "h, y, dy, dn, dx and dh")
    o = _residual_options(plan, width, dx.dtype, order, post_weight, gate, gate_per_document, scale, p, rng, site,
                          pre_weight, eps)
    dpost, dpre = _row_weights(dpost_weight, width, "dpost_weight"), _row_weights(dpre_weight, width, "dpre_weight")
    if dgate is not None:
        kind = torch.float32 if gate_per_document else dx.dtype
        if dgate.dtype != kind:
            raise ValueError(f"dgate must be of {kind}")
        _check_gate(plan, dgate, width, order, gate_per_document, "dgate")
    if workspace is None:
        if stream is not None:
            raise ValueError("give a workspace with a stream: torch allocates on its current stream only")
        need = cpt_residual_norm_backward_workspace_bytes(plan, width, dx.dtype)
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    _check(_lib.cpt_residual_norm_backward(plan.handle, _there(h), _there(y), _there(dy), _there(dn), _there(dx),
                                           _there(dh), _there(dgate), dpost, dpre, width,
                                           _dtype_code(dx), order, ctypes.byref(o), _ptr(workspace), _nbytes(workspace),
                                           _stream(stream)))


def _check_logits(t, rows: int, width: int, what: str):
    """The rows and no others, or a longer table of rows."""
    if t.dim() == 0 or t.shape[-1] != width or (t.numel() != rows * width and (t.dim() != 2 or t.shape[0] < rows)):
        raise ValueError(f"{what} of shape {tuple(t.shape)} do not hold {rows} rows of {width}")


def _check_columns(t, columns: int, what: str):
    """A buffer of so many values a row, flat or of that shape."""
    if t.dim() > 1 and t.shape[-1] != columns:
        raise ValueError(f"{what} must hold {columns} values a row, not {tuple(t.shape)}")


def _logits_shape(plan: Plan, logits, vocab, order, targets, stats, per_token):
    """(vocab, vocab_padded) of rows of logits, every buffer large enough."""
    rows, T = _row_count(plan, order), plan.total_tokens
    width = logits.shape[-1] if logits.dim() > 0 else 0
    _check_logits(logits, rows, width, "logits")
    _check_columns(stats, 2, "stats")
    if targets.dtype != torch.int32 or targets.numel() < T:
        raise ValueError(f"targets must hold {T} int32 values")
    for t, count, what in per_token:
        if t.dtype != torch.float32 or t.numel() < count * T:
            raise ValueError(f"{what} must hold {count * T} float32 values")
    if vocab is None:
        return width, width
    if not 1 <= vocab <= width:     # before ctypes cuts it to 64 bits
        raise ValueError(f"vocab {vocab} outside 1..{width}")
    return vocab, width


def cpt_token_logprob(plan: Plan, logits: torch.Tensor, targets: torch.Tensor, logp: torch.Tensor,
                      stats: torch.Tensor, *, vocab: int | None = None, scale: float = 1.0,
                      order: int = CPT_ORDER_LOCAL, stream=None):
    """logp[g] = log of the probability that token g's logits give to targets[g] (int32, global order; negative:
    none), over the first `vocab` columns (all, if None); stats [T, 2] for the gradient."""
    v, width = _logits_shape(plan, logits, vocab, order, targets, stats, ((logp, 1, "logp"), (stats, 2, "stats")))
    _check(_lib.cpt_token_logprob(plan.handle, _ptr(logits), _ptr(targets), _ptr(logp), _ptr(stats), v, width,
                                  _dtype_code(logits), order, scale, _stream(stream)))


def cpt_token_logprob_backward(plan: Plan, logits: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor,
                               dlogp: torch.Tensor, dlogits: torch.Tensor, *, vocab: int | None = None,
                               scale: float = 1.0, order: int = CPT_ORDER_LOCAL, stream=None):
    """dlogits (may be logits) of cpt_token_logprob from the gradient of logp."""
    v, width = _logits_shape(plan, logits, vocab, order, targets, stats, ((stats, 2, "stats"), (dlogp, 1, "dlogp")))
    if dlogits.dtype != logits.dtype:
        raise ValueError("dlogits must be like logits")
    _check_logits(dlogits, _row_count(plan, order), width, "dlogits")
    _check(_lib.cpt_token_logprob_backward(plan.handle, _ptr(logits), _ptr(targets), _ptr(stats), _ptr(dlogp),
                                           _ptr(dlogits), v, width, _dtype_code(logits), order, scale,
                                           _stream(stream)))


def cpt_policy_loss(plan: Plan, logp: torch.Tensor, logp_old: torch.Tensor, advantages: torch.Tensor,
                    terms: torch.Tensor, dlogp: torch.Tensor, *, logp_ref=None, mask=None, weights=None,
                    clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0, stream=None):
    """terms [n_docs, 4] (loss, KL, clipped share, tokens) of the clipped policy loss and dlogp [T], the gradient
    of the documents' losses, weighted. mask is bool or uint8 [T]; weights None: 1 / n_docs each."""
    T, n = plan.total_tokens, plan.n_docs
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or mask.numel() < T):
        raise ValueError(f"mask must hold {T} values of bool or uint8")
    _check_columns(terms, 4, "terms")
    _check(_lib.cpt_policy_loss(plan.handle, _floats(logp, T, "logp"), _floats(logp_old, T, "logp_old"),
                                _floats(logp_ref, T, "logp_ref") or _there(logp_ref), _ptr(mask), _floats(advantages, n, "advantages"),
                                _floats(weights, n, "weights"), clip_low, clip_high, kl_coef,
                                _floats(terms, 4 * n, "terms"), _floats(dlogp, T, "dlogp"), _stream(stream)))


# ------------------------------------------------------------------ epochs

class Epoch:
    def __init__(self, handle: int, flags: torch.Tensor, status: torch.Tensor, cp_size: int):
        self.handle = handle
        self.flags = flags
        self.status = status
        self.cp_size = cp_size

    def status_ptr(self, owner: int) -> int:
        return self.status.data_ptr() + 4 * owner

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            _lib.cpt_epoch_destroy(h)


def cpt_epoch_create(cp_size: int, flags: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     stream=None) -> Epoch:
    if flags is None:
        flags = torch.zeros(cp_size * cp_size, dtype=torch.int32, device="cuda")
    if status is None:
        status = torch.zeros(cp_size, dtype=torch.int32, device="cuda")
    h = _vp()
    _check(_lib.cpt_epoch_create(cp_size, _ptr(flags), _ptr(status), _stream(stream), ctypes.byref(h)))
    return Epoch(h.value, flags, status, cp_size)


def cpt_epoch_destroy(ep: Epoch) -> None:
    h, ep.handle = ep.handle, None
    if h:
        _check(_lib.cpt_epoch_destroy(h))


def cpt_epoch_advance(ep: Epoch) -> int:
    e = ctypes.c_uint32()
    _check(_lib.cpt_epoch_advance(ep.handle, ctypes.byref(e)))
    return e.value


def cpt_epoch_set(ep: Epoch, epoch: int) -> None:
    _check(_lib.cpt_epoch_set(ep.handle, epoch))


def cpt_epoch_publish(ep: Epoch, writer: int, stream=None) -> None:
    _check(_lib.cpt_epoch_publish(ep.handle, writer, _stream(stream)))


def cpt_epoch_wait(ep: Epoch, owner: int, timeout_ns: int = 1_000_000_000,
                   mode: int = CPT_WAIT_BOUNDED, stream=None) -> None:
    _check(_lib.cpt_epoch_wait(ep.handle, owner, timeout_ns, mode, _stream(stream)))


def cpt_epoch_status(ep: Epoch, owner: int, stream=None) -> int:
    v = _i32()
    _check(_lib.cpt_epoch_status(ep.handle, owner, _stream(stream), ctypes.byref(v)))
    return v.value


def cpt_set_kernel_path(kernel: int):
    """Process-wide kernel choice of the row gather, the gradient return and
    the slot reduce: CPT_KERNEL_AUTO (measured rule), _LOADS or _BULK."""
    _check(_lib.cpt_set_kernel_path(kernel))


def cpt_kernel_path_of(call: int, cp_size: int, in_dtype: int, out_dtype: int, accumulate: bool,
                       row_bytes: int, rows: int) -> int:
    """CPT_KERNEL_LOADS or CPT_KERNEL_BULK: the kernel the call would run now."""
    v = _i32()
    _check(_lib.cpt_kernel_path_of(call, cp_size, in_dtype, out_dtype, 1 if accumulate else 0,
                                   row_bytes, rows, ctypes.byref(v)))
    return v.value


def cpt_bounds_checked() -> bool:
    """Whether the loaded library is the bounds-checked build."""
    return bool(_lib.cpt_bounds_checked())


def cpt_bounds_violations(reset: bool = False) -> int:
    """Failed device bounds checks so far (bounds-checked build only)."""
    v = ctypes.c_uint32(0)
    _check(_lib.cpt_bounds_violations(ctypes.byref(v), 1 if reset else 0))
    return int(v.value)


def cpt_test_stall_bulk_waits(on: bool):
    """Test switch: make every bulk-copy wait of later launches of the row gather,
    the gradient return and the slot reduce run out of its budget (on) or
    behave normally (off)."""
    _check(_lib.cpt_test_stall_bulk_waits(1 if on else 0))


def cpt_kernel_wait_timeouts(reset: bool = False) -> int:
    """Waits in the library's kernels (on bulk copies, and between the warps of the
    attention kernels) that ran out of their budget on the current device (blocking; non-zero means an earlier output is not
    valid)."""
    v = ctypes.c_uint32()
    _check(_lib.cpt_kernel_wait_timeouts(ctypes.byref(v), 1 if reset else 0))
    return v.value


def cpt_stream_ceiling(srcs, dst: torch.Tensor, block_bytes: int, stages: int, ctas_per_sm: int = 1,
                       stream=None):
    """dst = copy of srcs[0], every other source read and discarded: the
    read/write mix of an HBM-bound call with no arithmetic (a roofline
    ceiling). All tensors hold the same number of bytes."""
    sl = _Parts(srcs, len(srcs) if not isinstance(srcs, torch.Tensor) else srcs.shape[0])
    nbytes = sl.part_bytes
    _need(dst, nbytes, "dst")
    _check(_lib.cpt_stream_ceiling(sl.array(), len(sl.ptrs), _ptr(dst), nbytes, block_bytes, stages,
                                   ctas_per_sm, _stream(stream)))


def declared_functions(header_path: str) -> list[str]:
    """Function names declared in a C header (for the export check)."""
    with open(header_path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(cpt_[a-z0-9_]+)\s*\(", text)))
