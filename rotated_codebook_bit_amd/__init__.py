"""Python binding of libcq, the CQ rotated-codebook quantizer for MI355X.

Thin ctypes marshalling over the C ABI declared in ``include/libcq.h``: the
names match the C entry points without the ``cq_`` prefix.  Every step of the
computation runs in libcq's HIP kernels; PyTorch only provides device memory
and the current stream.  There is no fallback: if ``libcq.so`` is missing or
a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Any, NamedTuple

import numpy as np

__all__ = [
    "TERNARY", "TERNARY_TRITS", "GROUP", "group_bytes", "repack", "CQError", "lib", "storage_bits", "n_levels", "layout",
    "model_bytes", "codebook", "codebook_train", "quantize", "dequantize", "dequant_matvec", "dequant_matvec_many",
    "dequant_matvec_many_noalloc",
    "fake_quant", "blob_layout", "quantize_many", "dequantize_many", "dequant_gemm",
    "dequant_gemm_many", "embed", "embed_packed", "embed_grad", "add_rms_norm", "add_rms_norm_q8", "rms_norm_grad",
    "Q8Table", "q8_levels", "dequant_gemm_q8", "qk_norm_rope", "qk_norm_rope_grad", "attention", "attention_grad",
    "TokenLogprobs", "token_logprobs", "token_logprobs_grad",
]

TERNARY = 158
TERNARY_TRITS = 159  # the ternary code stored five indices per byte
GROUP = 128
F32, BF16 = 0, 1

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcq.so")
_lib = None


class CQError(RuntimeError):
    """A libcq call returned an error status."""

    def __init__(self, func: str, status: int, detail: str):
        super().__init__(f"{func}: {detail} (status {status})")
        self.status = status


class QuantDesc(ctypes.Structure):
    """cq_quant_desc: one tensor of cq_quantize_many."""
    _fields_ = [("w", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("packed", ctypes.c_void_p), ("norms", ctypes.c_void_p)]


class DequantDesc(ctypes.Structure):
    """cq_dequant_desc: one tensor of cq_dequantize_many."""
    _fields_ = [("packed", ctypes.c_void_p), ("norms", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("out", ctypes.c_void_p)]


class MatvecDesc(ctypes.Structure):
    """cq_matvec_desc: one matrix of cq_dequant_matvec_many."""
    _fields_ = [("packed", ctypes.c_void_p), ("norms", ctypes.c_void_p), ("n_out", ctypes.c_int64),
                ("k", ctypes.c_int64), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p)]


class Heads(ctypes.Structure):
    """cq_heads: a tensor of heads, strides in values."""
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class Sequences(ctypes.Structure):
    """cq_sequences: the sequences of an attention call."""
    _fields_ = [("n_seq", ctypes.c_int64), ("rows_q", ctypes.c_int64), ("rows_k", ctypes.c_int64),
                ("q_starts", ctypes.c_void_p), ("k_starts", ctypes.c_void_p), ("k_lens", ctypes.c_void_p),
                ("index_bytes", ctypes.c_int)]


class TokenLogprobs(NamedTuple):
    """What token_logprobs returns, per row: the token's log probability, the
    entropy, the log of the sum, and the most probable tokens (of width 0 without)."""
    logprob: Any
    entropy: Any
    lse: Any
    top: Any
    top_logprob: Any


class Q8Table(ctypes.Structure):
    """cq_q8_table: the 16-bit levels of the 8-bit product, made by
    q8_levels() once per codebook."""
    _fields_ = [("hi", ctypes.c_int8 * 16), ("lo", ctypes.c_int8 * 16), ("scale", ctypes.c_float),
                ("n_levels", ctypes.c_int32)]


def lib() -> ctypes.CDLL:
    """Load libcq.so (built in place by ``rotated_codebook_bit_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m rotated_codebook_bit_amd.build`")
        # PyTorch brings a HIP runtime of its own.  Loaded after libcq it would
        # be a second one in the process, and streams and memory of one mean
        # nothing to the other: calls failed and the process crashed.
        try:
            import torch  # noqa: F401
        except ImportError:
            pass  # the host-only calls work without it
        L = ctypes.CDLL(LIB_PATH)
        i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
        L.cq_layout.argtypes = [i64, i64, i32, i32, ctypes.POINTER(i64), ctypes.POINTER(i64)]
        L.cq_model_bytes.argtypes = [i32, ctypes.POINTER(i64), ctypes.POINTER(i64), i32, i32,
                                     ctypes.POINTER(ctypes.c_uint64)]
        L.cq_codebook.argtypes = [i32, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(i32)]
        L.cq_codebook_train.argtypes = [i32, ctypes.POINTER(ctypes.c_double), i64, i32,
                                        ctypes.POINTER(ctypes.c_float), ctypes.POINTER(i32)]
        L.cq_quantize.argtypes = [vp, i32, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_float), i32,
                                  vp, vp, vp]
        L.cq_dequantize.argtypes = [vp, vp, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_float), i32,
                                    vp, i32, vp]
        L.cq_blob_layout.argtypes = [i32, ctypes.POINTER(i64), ctypes.POINTER(i64), i32, i32,
                                     ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i64)]
        L.cq_quantize_many.argtypes = [i32, ctypes.POINTER(QuantDesc), i32, i32, i32,
                                       ctypes.POINTER(ctypes.c_float), i32, vp]
        L.cq_dequantize_many.argtypes = [i32, ctypes.POINTER(DequantDesc), i32, i32,
                                         ctypes.POINTER(ctypes.c_float), i32, i32, vp]
        L.cq_dequant_gemm.argtypes = [vp, vp, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_float),
                                      i32, vp, i64, vp, vp]
        L.cq_dequant_gemm_many.argtypes = [i32, ctypes.POINTER(MatvecDesc), i32, i32,
                                           ctypes.POINTER(ctypes.c_float), i32, i64, vp]
        L.cq_repack.argtypes = [vp, i32, vp, i32, i64, i32, vp]
        L.cq_fake_quant.argtypes = [vp, i32, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_float), i32,
                                    vp, i32, vp]
        L.cq_dequant_matvec.argtypes = [vp, vp, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_float),
                                        i32, vp, i64, vp, vp]
        L.cq_dequant_matvec_many.argtypes = [i32, ctypes.POINTER(MatvecDesc), i32, i32,
                                             ctypes.POINTER(ctypes.c_float), i32, i64, vp]
        L.cq_dequant_matvec_many_noalloc.argtypes = L.cq_dequant_matvec_many.argtypes
        f32, fp, p64 = ctypes.c_float, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(i64)
        L.cq_embed.argtypes = [vp, i32, i64, vp, i32, i64, i64, f32, vp, i32, vp]
        L.cq_embed_packed.argtypes = [vp, i32, i64, vp, vp, i64, i64, i32, i32, vp, i32, f32, vp, i32, vp]
        L.cq_embed_grad_workspace.argtypes = [i64, i64, i64, p64]
        L.cq_embed_grad.argtypes = [vp, i32, i64, vp, i32, i64, i64, f32, i32, vp, i32, vp, i64, vp]
        L.cq_add_rms_norm.argtypes = [vp, vp, i32, vp, i32, i64, i64, f32, vp, vp, i32, vp]
        L.cq_add_rms_norm_q8.argtypes = [vp, vp, i32, vp, i32, i64, i64, i32, f32, vp, vp, vp, vp]
        L.cq_rms_norm_grad_workspace.argtypes = [i64, i64, i32, p64]
        L.cq_rms_norm_grad.argtypes = [vp, vp, vp, i32, vp, i32, i64, i64, f32, vp, vp, vp, i64, vp]
        L.cq_q8_levels.argtypes = [i32, fp, i32, ctypes.POINTER(Q8Table)]
        L.cq_dequant_gemm_q8_workspace.argtypes = [i64, i64, i64, i32, p64]
        L.cq_dequant_gemm_q8.argtypes = [vp, vp, i64, i64, i32, i32, ctypes.POINTER(Q8Table), vp, vp, i64, vp, i32, vp,
                                         i64, vp]
        hp = sp = vp  # cq_heads and cq_sequences, packed or by reference
        rotation = [i32, i64, i32, i32, i32, i32, vp, vp, i32, f32, vp, i32, vp, i32, i32]
        L.cq_qk_norm_rope.argtypes = [hp, hp, hp, *rotation, hp, hp, hp, vp, i32, i64, vp]
        L.cq_qk_norm_rope_grad_workspace.argtypes = [i64, i32, i32, i32, p64]
        L.cq_qk_norm_rope_grad.argtypes = [hp, hp, hp, hp, *rotation, hp, hp, vp, vp, vp, i64, vp]
        L.cq_attention_workspace.argtypes = [sp, i32, i32, i32, i32, p64]
        L.cq_attention.argtypes = [hp, hp, hp, i32, sp, i32, i32, i32, i32, f32, hp, vp, vp, i64, vp]
        L.cq_attention_grad_workspace.argtypes = L.cq_attention_workspace.argtypes
        L.cq_attention_grad.argtypes = [hp, hp, hp, hp, hp, vp, i32, sp, i32, i32, i32, i32, f32, hp, hp, hp, vp, i64, vp]
        L.cq_token_logprobs.argtypes = [vp, i32, i64, i64, i64, f32, vp, i32, vp, vp, vp, i32, vp, vp, vp]
        L.cq_token_logprobs_grad.argtypes = [vp, i32, i64, i64, i64, f32, vp, i32, vp, vp, vp, vp, vp, i64, vp]
        for name in ("cq_qk_norm_rope", "cq_qk_norm_rope_grad_workspace", "cq_qk_norm_rope_grad", "cq_attention_workspace",
                     "cq_attention", "cq_attention_grad_workspace", "cq_attention_grad", "cq_token_logprobs",
                     "cq_token_logprobs_grad"):
            getattr(L, name).restype = i32
        for name in ("cq_embed", "cq_embed_packed", "cq_embed_grad_workspace", "cq_embed_grad", "cq_add_rms_norm",
                     "cq_add_rms_norm_q8", "cq_rms_norm_grad_workspace", "cq_rms_norm_grad", "cq_q8_levels",
                     "cq_dequant_gemm_q8_workspace", "cq_dequant_gemm_q8"):
            getattr(L, name).restype = i32
        for name in ("cq_layout", "cq_model_bytes", "cq_codebook", "cq_codebook_train", "cq_quantize", "cq_dequantize",
                     "cq_fake_quant", "cq_dequant_matvec", "cq_dequant_matvec_many",
                     "cq_dequant_matvec_many_noalloc", "cq_blob_layout",
                     "cq_quantize_many", "cq_dequantize_many", "cq_dequant_gemm",
                     "cq_dequant_gemm_many", "cq_repack"):
            getattr(L, name).restype = i32
        L.cq_status_str.argtypes = [i32]
        L.cq_status_str.restype = ctypes.c_char_p
        L.cq_last_error.argtypes = []
        L.cq_last_error.restype = ctypes.c_char_p
        L.cq_version.argtypes = []
        L.cq_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(func: str, status: int) -> None:
    if status != 0:
        L = lib()
        detail = L.cq_last_error().decode() or L.cq_status_str(status).decode()
        raise CQError(func, status, detail)


def storage_bits(bits: int) -> int:
    return 2 if bits in (TERNARY, TERNARY_TRITS) else int(bits)


def group_bytes(bits: int, group_size: int = GROUP) -> int:
    """Packed bytes per group (ceil(G/5) for trit storage)."""
    if bits == TERNARY_TRITS:
        return -(-group_size // 5)
    return group_size * storage_bits(bits) // 8


def n_levels(bits: int) -> int:
    return 3 if bits in (TERNARY, TERNARY_TRITS) else 1 << int(bits)


def _levels_arg(levels) -> tuple[np.ndarray | None, ctypes.POINTER(ctypes.c_float)]:
    """(kept-alive array, pointer) for a levels argument; None passes NULL,
    which selects the library's built-in table."""
    if levels is None:
        return None, ctypes.POINTER(ctypes.c_float)()
    arr = np.ascontiguousarray(np.asarray(levels, dtype=np.float32))
    return arr, arr.ctypes.data_as(ctypes.POINTER(ctypes.c_float))


def _nlev(arr) -> int:
    return 0 if arr is None else int(arr.size)


def _stream_ptr(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


# -- host-only calls ------------------------------------------------------------

def layout(rows: int, cols: int, bits: int, group_size: int = GROUP) -> tuple[int, int]:
    """(n_groups, packed_bytes) of a rows x cols tensor."""
    ng, pb = ctypes.c_int64(), ctypes.c_int64()
    _check("cq_layout", lib().cq_layout(rows, cols, bits, group_size, ctypes.byref(ng),
                                        ctypes.byref(pb)))
    return ng.value, pb.value


def model_bytes(shapes, bits: int, group_size: int = GROUP) -> int:
    """Storage bytes of a list of tensor shapes (last axis is the grouped one)."""
    rows, cols = [], []
    for shape in shapes:
        shape = tuple(int(s) for s in shape)
        cols.append(shape[-1])
        rows.append(int(np.prod(shape[:-1], dtype=np.int64)) if len(shape) > 1 else 1)
    n = len(rows)
    r = (ctypes.c_int64 * max(n, 1))(*rows)
    c = (ctypes.c_int64 * max(n, 1))(*cols)
    out = ctypes.c_uint64()
    _check("cq_model_bytes", lib().cq_model_bytes(n, r, c, bits, group_size, ctypes.byref(out)))
    return out.value


def codebook(bits: int) -> np.ndarray:
    """The built-in float32 codebook of a width (N(0,1) units): the table
    every call uses when its levels argument is None."""
    out = (ctypes.c_float * 16)()
    n = ctypes.c_int()
    _check("cq_codebook", lib().cq_codebook(bits, out, ctypes.byref(n)))
    return np.array(out[:n.value], dtype=np.float32)


def codebook_train(bits: int, samples, iters: int = 200) -> np.ndarray:
    """float32 Lloyd-Max codebook (N(0,1) units) trained by the library on the
    given float64 samples."""
    s = np.ascontiguousarray(np.zeros(0) if samples is None else samples, dtype=np.float64)
    out = (ctypes.c_float * 16)()
    n = ctypes.c_int()
    _check("cq_codebook_train", lib().cq_codebook_train(
        bits, s.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), s.size, iters, out, ctypes.byref(n)))
    return np.array(out[:n.value], dtype=np.float32)


# -- device calls ---------------------------------------------------------------

def _rows_cols(shape) -> tuple[int, int]:
    rows = 1
    for d in shape[:-1]:
        rows *= int(d)
    return rows, int(shape[-1])


def _desc_array(cls, columns):
    """A ctypes array of the descriptor struct `cls`, field i taken from the
    sequence columns[i].  It is filled through a NumPy record array of the
    same layout (every field is 8 bytes), one vectorised assignment per field
    instead of one ctypes construction per element."""
    n = len(columns[0])
    dt = np.dtype([(name, "<u8" if typ is ctypes.c_void_p else "<i8") for name, typ in cls._fields_])
    assert dt.itemsize == ctypes.sizeof(cls)
    rec = np.zeros(max(n, 1), dt)
    if n:
        for (name, _), col in zip(cls._fields_, columns):
            rec[name] = col
    return (cls * max(n, 1)).from_buffer(rec)


def _ptr_or_0(t) -> int:
    return t.data_ptr() if t.numel() else 0


def quantize(w, bits: int, levels, group_size: int = GROUP, packed=None, norms=None, stream=None):
    """Quantize a CUDA tensor (float32 or bfloat16, any rank; the last axis is
    grouped).  Returns (packed uint8 [rows, ngroups, G*sbits/8],
    norms float16 [rows, ngroups]) on w's device."""
    import torch
    if w.dtype == torch.float32:
        dt = F32
    elif w.dtype == torch.bfloat16:
        dt = BF16
    else:
        raise TypeError(f"unsupported dtype {w.dtype}")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    rows, cols = _rows_cols(w.shape)
    ng = -(-cols // group_size) if cols else 0
    pb = group_bytes(bits, group_size)
    if packed is None:
        packed = torch.empty((rows, ng, pb), dtype=torch.uint8, device=w.device)
    if norms is None:
        norms = torch.empty((rows, ng), dtype=torch.float16, device=w.device)
    lv, lvp = _levels_arg(levels)
    _check("cq_quantize", lib().cq_quantize(_ptr(w), dt, rows, cols, bits, group_size, lvp, _nlev(lv),
                                            _ptr(packed), _ptr(norms), _stream_ptr(stream)))
    return packed, norms


def dequantize(packed, norms, rows: int, cols: int, bits: int, levels, out_dtype=None,
               group_size: int = GROUP, out=None, stream=None):
    """Dequantize to a [rows, cols] CUDA tensor (float32 by default, or
    bfloat16)."""
    import torch
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    dt = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    if out is None:
        out = torch.empty((rows, cols), dtype=out_dtype, device=packed.device)
    lv, lvp = _levels_arg(levels)
    _check("cq_dequantize", lib().cq_dequantize(_ptr(packed), _ptr(norms), rows, cols, bits,
                                                group_size, lvp, _nlev(lv), _ptr(out), dt,
                                                _stream_ptr(stream)))
    return out


def fake_quant(w, bits: int, levels, out_dtype=None, group_size: int = GROUP, out=None,
               stream=None):
    """Quantize and reconstruct a CUDA tensor in one pass (float32 or
    bfloat16 in, float32 or bfloat16 out, w's shape; default out dtype = w's).
    ``out=w`` fake-quantizes in place."""
    import torch
    dts = {torch.float32: F32, torch.bfloat16: BF16}
    if w.dtype not in dts:
        raise TypeError(f"unsupported dtype {w.dtype}")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    if out is None:
        out = torch.empty(w.shape, dtype=w.dtype if out_dtype is None else out_dtype, device=w.device)
    if out.dtype not in dts or not out.is_contiguous() or out.numel() != w.numel():
        raise ValueError("out must be a contiguous float32/bfloat16 tensor of w's size")
    rows, cols = _rows_cols(w.shape)
    lv, lvp = _levels_arg(levels)
    _check("cq_fake_quant", lib().cq_fake_quant(_ptr(w), dts[w.dtype], rows, cols, bits, group_size,
                                                lvp, _nlev(lv), _ptr(out), dts[out.dtype],
                                                _stream_ptr(stream)))
    return out


def dequant_matvec(packed, norms, n_out: int, k: int, bits: int, levels, x, group_size: int = GROUP,
                   y=None, stream=None):
    """y = x . W_hat^T with W the quantized n_out x k matrix; x float32
    [batch, k] on the device.  Returns float32 [batch, n_out]."""
    import torch
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise TypeError("x must be a contiguous float32 tensor")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [batch, {k}], got {tuple(x.shape)}")
    x2 = x
    batch = x2.shape[0]
    if y is None:
        y = torch.empty((batch, n_out), dtype=torch.float32, device=x.device)
    lv, lvp = _levels_arg(levels)
    _check("cq_dequant_matvec", lib().cq_dequant_matvec(_ptr(packed), _ptr(norms), n_out, k, bits,
                                                        group_size, lvp, _nlev(lv), _ptr(x2), batch,
                                                        _ptr(y), _stream_ptr(stream)))
    return y


def _matvec_descs(items):
    return _desc_array(MatvecDesc, (
        [_ptr_or_0(it[0]) for it in items], [_ptr_or_0(it[1]) for it in items],
        [it[2] for it in items], [it[3] for it in items],
        [_ptr_or_0(it[4]) for it in items], [_ptr_or_0(it[5]) for it in items]))


def dequant_matvec_many(items, bits: int, levels, batch: int, group_size: int = GROUP, stream=None):
    """Run y = x . W_hat^T for every (packed, norms, n_out, k, x, y) in items
    as one call (the y tensors, float32 [batch, n_out], are written in place).
    Returns the list of y tensors."""
    n = len(items)
    arr = _matvec_descs(items)
    lv, lvp = _levels_arg(levels)
    _check("cq_dequant_matvec_many", lib().cq_dequant_matvec_many(n, arr, bits, group_size, lvp, _nlev(lv),
                                                                  batch, _stream_ptr(stream)))
    return [it[5] for it in items]


def dequant_matvec_many_noalloc(items, bits: int, levels, batch: int, group_size: int = GROUP, stream=None):
    """dequant_matvec_many with the library's fixed 16 MiB workspace instead of
    memory allocated per call (cq_dequant_matvec_many_noalloc).  Calls that
    overlap on one GPU race on that workspace."""
    n = len(items)
    arr = _matvec_descs(items)
    lv, lvp = _levels_arg(levels)
    _check("cq_dequant_matvec_many_noalloc",
           lib().cq_dequant_matvec_many_noalloc(n, arr, bits, group_size, lvp, _nlev(lv), batch,
                                                _stream_ptr(stream)))
    return [it[5] for it in items]


def blob_layout(shapes, bits: int, group_size: int = GROUP):
    """Offsets of the serialized form (all packed indices, then all norms) of
    tensors with the given shapes: (packed_offsets, norm_offsets, total)."""
    dims = [_rows_cols(tuple(sh)) for sh in shapes]
    n = len(dims)
    rc = np.zeros((2, max(n, 1)), np.int64)
    if n:
        rc[:, :n] = np.array(dims, np.int64).T
    out = np.zeros((2, max(n, 1)), np.int64)
    p64 = ctypes.POINTER(ctypes.c_int64)
    total = ctypes.c_int64()
    _check("cq_blob_layout", lib().cq_blob_layout(n, rc[0].ctypes.data_as(p64), rc[1].ctypes.data_as(p64), bits,
                                                  group_size, out[0].ctypes.data_as(p64),
                                                  out[1].ctypes.data_as(p64), ctypes.byref(total)))
    return out[0, :n].tolist(), out[1, :n].tolist(), total.value


def quantize_many(ws, bits: int, levels, blob=None, group_size: int = GROUP, stream=None,
                  views: bool = True):
    """Quantize a list of CUDA tensors (all float32 or all bfloat16) in one
    call, writing the serialized blob (uint8, all packed indices then all
    norms).  Returns (blob, [(packed [rows, ng, G*sbits/8], norms float16
    [rows, ng]) views into the blob, one per tensor]); with views=False the
    list is empty (blob_layout gives the offsets)."""
    import torch
    if not ws:
        return torch.zeros(0, dtype=torch.uint8), []
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(ws[0].dtype)
    if dt is None or any(w.dtype != ws[0].dtype for w in ws):
        raise TypeError("all tensors must be float32, or all bfloat16")
    if any(not w.is_contiguous() for w in ws):
        raise ValueError("tensors must be contiguous")
    po, no, total = blob_layout([tuple(w.shape) for w in ws], bits, group_size)
    if blob is None:
        blob = torch.empty(total, dtype=torch.uint8, device=ws[0].device)
        # An odd-length index section is followed by a pad byte the library
        # does not write: zero it, so the blob is fully defined.
        packed_end = group_bytes(bits, group_size) * sum(
            r * -(-c // group_size) for r, c in (_rows_cols(tuple(w.shape)) for w in ws))
        if packed_end % 2:
            blob[packed_end:packed_end + 1].zero_()
    if blob.dtype != torch.uint8 or blob.numel() != total or not blob.is_contiguous():
        raise ValueError(f"blob must be a contiguous uint8 tensor of {total} bytes")
    pb = group_bytes(bits, group_size)
    base = blob.data_ptr() if total else 0
    dims = [_rows_cols(tuple(w.shape)) for w in ws]
    live = [r * c != 0 for r, c in dims]
    arr = _desc_array(QuantDesc, (
        [w.data_ptr() if a else 0 for w, a in zip(ws, live)], [r for r, _ in dims], [c for _, c in dims],
        [base + o if a else 0 for o, a in zip(po, live)], [base + o if a else 0 for o, a in zip(no, live)]))
    out_views = []
    if views:
        for i, (rows, cols) in enumerate(dims):
            ng = -(-cols // group_size) if cols else 0
            pk = blob[po[i]:po[i] + rows * ng * pb].view(rows, ng, pb)
            nm = blob[no[i]:no[i] + 2 * rows * ng].view(torch.float16).view(rows, ng)
            out_views.append((pk, nm))
    lv, lvp = _levels_arg(levels)
    _check("cq_quantize_many", lib().cq_quantize_many(len(ws), arr, dt, bits, group_size, lvp, _nlev(lv),
                                                      _stream_ptr(stream)))
    return blob, out_views


def dequantize_many(items, bits: int, levels, out_dtype=None, outs=None, group_size: int = GROUP,
                    stream=None):
    """Dequantize every (packed, norms, rows, cols) of items in one call.
    Returns the list of [rows, cols] outputs (float32 by default, or
    bfloat16; ``outs`` supplies them)."""
    import torch
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    dt = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    if outs is None:
        dev = items[0][0].device if items else "cpu"
        outs = [torch.empty((r, c), dtype=out_dtype, device=dev) for _, _, r, c in items]
    for i, ((_, _, rows, cols), out) in enumerate(zip(items, outs)):
        if out.dtype != out_dtype or out.numel() != rows * cols or not out.is_contiguous():
            raise ValueError(f"outs[{i}] must be a contiguous {out_dtype} tensor of {rows}x{cols}")
    arr = _desc_array(DequantDesc, (
        [_ptr_or_0(it[0]) for it in items], [_ptr_or_0(it[1]) for it in items], [it[2] for it in items],
        [it[3] for it in items], [_ptr_or_0(o) for o in outs]))
    lv, lvp = _levels_arg(levels)
    _check("cq_dequantize_many", lib().cq_dequantize_many(len(items), arr, bits, group_size, lvp,
                                                          _nlev(lv), dt, _stream_ptr(stream)))
    return outs


def dequant_gemm(packed, norms, n_out: int, k: int, bits: int, levels, x, group_size: int = GROUP,
                 y=None, stream=None):
    """y = x . W_hat^T on the matrix cores (split-bf16 MFMA, see
    cq_dequant_gemm); x float32 [batch, k].  Returns float32 [batch, n_out]."""
    import torch
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise TypeError("x must be a contiguous float32 tensor")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [batch, {k}], got {tuple(x.shape)}")
    batch = x.shape[0]
    if y is None:
        y = torch.empty((batch, n_out), dtype=torch.float32, device=x.device)
    lv, lvp = _levels_arg(levels)
    _check("cq_dequant_gemm", lib().cq_dequant_gemm(_ptr(packed), _ptr(norms), n_out, k, bits, group_size,
                                                    lvp, _nlev(lv), _ptr(x), batch, _ptr(y),
                                                    _stream_ptr(stream)))
    return y


def dequant_gemm_many(items, bits: int, levels, batch: int, group_size: int = GROUP, stream=None):
    """dequant_gemm for every (packed, norms, n_out, k, x, y) in items as one
    call (y float32 [batch, n_out] written in place).  Returns the y list."""
    n = len(items)
    arr = _matvec_descs(items)
    lv, lvp = _levels_arg(levels)
    _check("cq_dequant_gemm_many", lib().cq_dequant_gemm_many(n, arr, bits, group_size, lvp, _nlev(lv), batch,
                                                              _stream_ptr(stream)))
    return [it[5] for it in items]


def repack(src, src_bits: int, dst_bits: int, dst=None, group_size: int = GROUP, stream=None):
    """Convert packed ternary indices between 2-bit fields (TERNARY) and trit
    storage (TERNARY_TRITS).  src: uint8 CUDA tensor whose last dimension is
    one group's bytes ([..., 32] or [..., 26]).  Returns dst ([..., 26] or
    [..., 32])."""
    import torch
    sb, db = group_bytes(src_bits, group_size), group_bytes(dst_bits, group_size)
    if src.dtype != torch.uint8 or src.shape[-1] != sb or not src.is_contiguous():
        raise ValueError(f"src must be a contiguous uint8 tensor [..., {sb}]")
    n_groups = src.numel() // sb
    if dst is None:
        dst = torch.empty(tuple(src.shape[:-1]) + (db,), dtype=torch.uint8, device=src.device)
    _check("cq_repack", lib().cq_repack(_ptr(src), src_bits, _ptr(dst), dst_bits, n_groups, group_size,
                                        _stream_ptr(stream)))
    return dst


# -- around the products: embedding, norm, 8-bit activations ---------------------

def _device(named) -> int:
    """Index of the one CUDA device that holds every contiguous tensor of
    `named`, (name, tensor or None) pairs."""
    dev = -1
    for name, t in named:
        if t is None:
            continue
        d = t.get_device()
        if d < 0:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dev < 0:
            dev = d
        elif d != dev:
            raise ValueError(f"{name} is on device {d}, the other tensors on {dev}")
    return dev


def _raw_stream(dev: int):
    """The current stream of device `dev` as a pointer."""
    import torch
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # 2.5 us less per call than current_stream()
    return torch.cuda.current_stream(dev).cuda_stream if get is None else get(dev)


def _elsewhere(dev: int, stream, named, call):
    """call() with device `dev` and `stream` (if given) current, so that what
    it allocates belongs to that stream; the tensors handed to it are recorded
    on a stream that is not the caller's."""
    import torch
    with torch.cuda.device(dev):
        if stream is None:
            return call()
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on device {dev}")
        if stream != torch.cuda.current_stream():
            for _, t in named:
                if t is not None:
                    t.record_stream(stream)
        with torch.cuda.stream(stream):
            return call()


def _here(dev: int, stream) -> bool:
    import torch
    return stream is None and dev == torch.cuda.current_device()


def _levels_address(levels):
    """(kept-alive float32 array or None, its address or None, count)."""
    if levels is None:
        return None, None, 0
    arr = np.ascontiguousarray(levels, dtype=np.float32)
    return arr, arr.ctypes.data, arr.size


def _dtype_code(name, t_or_dtype) -> int:
    import torch
    dt = getattr(t_or_dtype, "dtype", t_or_dtype)
    if dt == torch.float32:
        return F32
    if dt == torch.bfloat16:
        return BF16
    raise TypeError(f"{name}: unsupported dtype {dt}")


def _out_tensor(name, given, shape, dtype, like):
    """`given` if it has the wanted shape and dtype, or a new tensor on the
    device of `like`."""
    if given is None:
        return like.new_empty(shape, dtype=dtype)
    if given.dtype != dtype or tuple(given.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {given.dtype} {tuple(given.shape)}")
    return given


def _opt(t):
    return None if t is None else t.data_ptr()


def _token_bytes(tokens) -> int:
    import torch
    if tokens.dtype == torch.int64:
        return 8
    if tokens.dtype == torch.int32:
        return 4
    raise TypeError(f"tokens must be int32 or int64, got {tokens.dtype}")


def _workspace(query, args, given, like):
    """(tensor or None, bytes) for a call that needs `query(*args)` bytes."""
    import torch
    if given is not None:
        return given, given.numel() * given.element_size()
    need = ctypes.c_int64()
    _check(query, getattr(lib(), query)(*args, ctypes.byref(need)))
    return (like.new_empty(need.value, dtype=torch.uint8) if need.value else None), need.value


def embed(tokens, table, scale: float = 1.0, out_dtype=None, out=None, stream=None):
    """scale * table[tokens] for int32 or int64 tokens of any shape and a
    [vocab, dim] float32 or bfloat16 table: [*tokens.shape, dim] in out_dtype
    (default: the table's).  Tokens outside the table give zero rows."""
    if table.dim() != 2:
        raise ValueError("table must be [vocab, dim]")
    tb, td = _token_bytes(tokens), _dtype_code("table", table)
    od = table.dtype if out_dtype is None else out_dtype
    oc = _dtype_code("out_dtype", od)
    vocab, dim = table.shape
    named = (("table", table), ("tokens", tokens), ("out", out))
    dev = _device(named)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, named, lambda: embed(tokens, table, scale, od, out))
    out = _out_tensor("out", out, (*tokens.shape, dim), od, table)
    _check("cq_embed", lib().cq_embed(tokens.data_ptr(), tb, tokens.numel(), table.data_ptr(), td, vocab, dim, scale,
                                      out.data_ptr(), oc, _raw_stream(dev)))
    return out


def embed_packed(tokens, packed, norms, vocab: int, dim: int, bits: int, levels, scale: float = 1.0, out_dtype=None,
                 group_size: int = GROUP, out=None, stream=None):
    """The same lookup from the CQ form of a [vocab, dim] table (packed and
    norms as quantize() returns them): scale * the dequantized rows, float32
    by default or bfloat16."""
    import torch
    tb = _token_bytes(tokens)
    od = torch.float32 if out_dtype is None else out_dtype
    oc = _dtype_code("out_dtype", od)
    _check_stored(packed, norms, vocab, dim, bits, group_size)
    named = (("packed", packed), ("norms", norms), ("tokens", tokens), ("out", out))
    dev = _device(named)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, named, lambda: embed_packed(tokens, packed, norms, vocab, dim, bits, levels, scale, od,
                                                                   group_size, out))
    keep, lv, nl = _levels_address(levels)
    out = _out_tensor("out", out, (*tokens.shape, dim), od, packed)
    _check("cq_embed_packed", lib().cq_embed_packed(
        tokens.data_ptr(), tb, tokens.numel(), packed.data_ptr(), norms.data_ptr(), vocab, dim, bits, group_size, lv, nl, scale,
        out.data_ptr(), oc, _raw_stream(dev)))
    return out


def _check_stored(packed, norms, rows, cols, bits, group_size):
    """The stored form's tensors hold what the call will read."""
    import torch
    if group_size < 1 or rows < 0 or cols < 0:
        raise ValueError("negative size")
    ng = rows * -(-cols // group_size)
    if packed.dtype != torch.uint8 or packed.numel() != ng * group_bytes(bits, group_size):
        raise ValueError(f"packed must hold {ng * group_bytes(bits, group_size)} uint8 values")
    if norms.dtype != torch.float16 or norms.numel() != ng:
        raise ValueError(f"norms must hold {ng} float16 values")


def embed_grad(tokens, dout, vocab: int, scale: float = 1.0, grad_dtype=None, grad=None, accumulate: bool = False,
               workspace=None, stream=None):
    """Gradient of the lookup with respect to the [vocab, dim] table:
    row v is scale * the sum of dout over the positions with token v (dout
    [*tokens.shape, dim], float32 or bfloat16).  grad_dtype float32 by default;
    accumulate=True adds to the given `grad`."""
    import torch
    tb, dd = _token_bytes(tokens), _dtype_code("dout", dout)
    if tuple(dout.shape[:-1]) != tuple(tokens.shape):
        raise ValueError(f"dout must be [*{tuple(tokens.shape)}, dim], got {tuple(dout.shape)}")
    if accumulate and grad is None:
        raise ValueError("accumulate needs grad")
    gd = grad.dtype if grad is not None else torch.float32 if grad_dtype is None else grad_dtype
    gc = _dtype_code("grad", gd)
    n, dim = tokens.numel(), dout.shape[-1]
    named = (("dout", dout), ("tokens", tokens), ("grad", grad), ("workspace", workspace))
    dev = _device(named)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, named, lambda: embed_grad(tokens, dout, vocab, scale, gd, grad, accumulate, workspace))
    grad = _out_tensor("grad", grad, (vocab, dim), gd, dout)
    ws, wb = _workspace("cq_embed_grad_workspace", (n, vocab, dim), workspace, dout)
    _check("cq_embed_grad", lib().cq_embed_grad(
        tokens.data_ptr(), tb, n, dout.data_ptr(), dd, vocab, dim, scale, int(bool(accumulate)), grad.data_ptr(), gc, _opt(ws),
        wb, _raw_stream(dev)))
    return grad


def _norm_args(x, residual, weight, sum_out):
    xd = _dtype_code("x", x)
    rows, cols = _rows_cols(x.shape)
    for name, t in (("residual", residual), ("sum_out", sum_out)):
        if t is not None and (t.dtype != x.dtype or t.shape != x.shape):
            raise ValueError(f"{name} must be {x.dtype} of shape {tuple(x.shape)}")
    return xd, rows, cols, _weight_code(weight, cols)


def _weight_code(weight, cols):
    if weight is None:
        return F32
    if weight.numel() != cols:
        raise ValueError(f"weight must hold {cols} values")
    return _dtype_code("weight", weight)


def add_rms_norm(x, residual=None, weight=None, eps: float = 1e-6, out_dtype=None, sum_out=None, out=None, stream=None):
    """(out, sum): sum = x + residual and out = its root-mean-square norm over
    the last axis times weight.  x and residual float32 or bfloat16 of one
    shape, weight float32 or bfloat16 [cols] (None: ones).  sum has x's dtype
    and is x itself without a residual; sum_out may be x or residual.  out is
    out_dtype (default x's)."""
    import torch
    xd, rows, cols, wd = _norm_args(x, residual, weight, sum_out)
    od = x.dtype if out_dtype is None else out_dtype
    oc = _dtype_code("out_dtype", od)
    named = (("x", x), ("residual", residual), ("weight", weight), ("sum_out", sum_out), ("out", out))
    dev = _device(named)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, named, lambda: add_rms_norm(x, residual, weight, eps, od, sum_out, out))
    if sum_out is None and residual is not None:
        sum_out = torch.empty_like(x)
    out = _out_tensor("out", out, x.shape, od, x)
    _check("cq_add_rms_norm", lib().cq_add_rms_norm(
        x.data_ptr(), _opt(residual), xd, _opt(weight), wd, rows, cols, eps, _opt(sum_out), out.data_ptr(), oc,
        _raw_stream(dev)))
    return out, x if sum_out is None else sum_out


def add_rms_norm_q8(x, residual=None, weight=None, eps: float = 1e-6, group_size: int = GROUP, sum_out=None, q=None,
                    scale=None, stream=None):
    """(q, scale, sum): add_rms_norm with its output rotated per group and
    held in 8 bits: q int8 of x's shape, scale float32 [*x.shape[:-1]]; q *
    scale are the rotated activations that dequant_gemm_q8 reads."""
    import torch
    xd, rows, cols, wd = _norm_args(x, residual, weight, sum_out)
    named = (("x", x), ("residual", residual), ("weight", weight), ("sum_out", sum_out), ("q", q), ("scale", scale))
    dev = _device(named)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, named, lambda: add_rms_norm_q8(x, residual, weight, eps, group_size, sum_out, q, scale))
    if sum_out is None and residual is not None:
        sum_out = torch.empty_like(x)
    q = _out_tensor("q", q, x.shape, torch.int8, x)
    scale = _out_tensor("scale", scale, x.shape[:-1], torch.float32, x)
    _check("cq_add_rms_norm_q8", lib().cq_add_rms_norm_q8(
        x.data_ptr(), _opt(residual), xd, _opt(weight), wd, rows, cols, group_size, eps, _opt(sum_out), q.data_ptr(),
        scale.data_ptr(), _raw_stream(dev)))
    return q, scale, x if sum_out is None else sum_out


def rms_norm_grad(dout, sum, weight=None, dsum=None, eps: float = 1e-6, dx=None, dweight=None, workspace=None,
                  stream=None):
    """(dx, dweight) of add_rms_norm at its sum: dx (for x and residual alike)
    in sum's dtype, dweight float32 [cols].  dout and dsum (the gradient that
    reaches sum by other ways, None: zero) have sum's dtype and shape; dx may
    be dsum."""
    import torch
    sd = _dtype_code("sum", sum)
    for name, t in (("dout", dout), ("dsum", dsum), ("dx", dx)):
        if t is not None and (t.dtype != sum.dtype or t.shape != sum.shape):
            raise ValueError(f"{name} must be {sum.dtype} of shape {tuple(sum.shape)}")
    rows, cols = _rows_cols(sum.shape)
    wd = _weight_code(weight, cols)
    named = (("sum", sum), ("dout", dout), ("weight", weight), ("dsum", dsum), ("dx", dx), ("dweight", dweight),
             ("workspace", workspace))
    dev = _device(named)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, named, lambda: rms_norm_grad(dout, sum, weight, dsum, eps, dx, dweight, workspace))
    dx = torch.empty_like(sum) if dx is None else dx
    dweight = _out_tensor("dweight", dweight, (cols,), torch.float32, sum)
    ws, wb = _workspace("cq_rms_norm_grad_workspace", (rows, cols, sd), workspace, sum)
    _check("cq_rms_norm_grad", lib().cq_rms_norm_grad(
        dout.data_ptr(), sum.data_ptr(), _opt(dsum), sd, _opt(weight), wd, rows, cols, eps, dx.data_ptr(), dweight.data_ptr(),
        _opt(ws), wb, _raw_stream(dev)))
    return dx, dweight


def q8_levels(bits: int, levels=None) -> Q8Table:
    """The 16-bit form of a codebook (None: the built-in one) that
    dequant_gemm_q8 multiplies with; made once per codebook (a search on the
    host, up to 0.9 ms).  The built-in tables' levels are met to 4e-8 of the
    values (root mean square; ternary and 2 bits), 1e-6 (3) and 7e-6 (4)."""
    table = Q8Table()
    lv, lvp = _levels_arg(levels)
    _check("cq_q8_levels", lib().cq_q8_levels(bits, lvp, _nlev(lv), ctypes.byref(table)))
    return table


def dequant_gemm_q8(packed, norms, n_out: int, k: int, bits: int, table: Q8Table, q, scale, group_size: int = GROUP,
                    out_dtype=None, y=None, workspace=None, stream=None):
    """y = x . W_hat^T with W the quantized n_out x k matrix and x given as
    add_rms_norm_q8 writes it (q int8 [..., k], scale float32 [...]): [...,
    n_out], float32 by default or bfloat16."""
    import torch
    od = torch.float32 if out_dtype is None else out_dtype
    oc = _dtype_code("out_dtype", od)
    if not isinstance(table, Q8Table):
        raise TypeError("table must come from q8_levels()")
    if q.dtype != torch.int8 or q.dim() < 1 or q.shape[-1] != k:
        raise ValueError(f"q must be int8 [..., {k}], got {q.dtype} {tuple(q.shape)}")
    if scale.dtype != torch.float32 or scale.shape != q.shape[:-1]:
        raise ValueError(f"scale must be float32 {tuple(q.shape[:-1])}, got {scale.dtype} {tuple(scale.shape)}")
    _check_stored(packed, norms, n_out, k, bits, group_size)
    batch = scale.numel()
    named = (("packed", packed), ("norms", norms), ("q", q), ("scale", scale), ("y", y), ("workspace", workspace))
    dev = _device(named)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, named, lambda: dequant_gemm_q8(packed, norms, n_out, k, bits, table, q, scale, group_size,
                                                                      od, y, workspace))
    y = _out_tensor("y", y, (*q.shape[:-1], n_out), od, q)
    ws, wb = _workspace("cq_dequant_gemm_q8_workspace", (n_out, k, batch, group_size), workspace, q)
    _check("cq_dequant_gemm_q8", lib().cq_dequant_gemm_q8(
        packed.data_ptr(), norms.data_ptr(), n_out, k, bits, group_size, ctypes.byref(table), q.data_ptr(), scale.data_ptr(),
        batch, y.data_ptr(), oc, _opt(ws), wb, _raw_stream(dev)))
    return y


# -- an attention block and a model's end ------------------------------------------

# cq_heads and cq_sequences as bytes: building the ctypes structures costs the
# call of one token 4 us more.
_pack_heads = struct.Struct("Pqq").pack
_pack_sequences = struct.Struct("qqqPPPi4x").pack


def _heads(named, dev: int = -1):
    """(device, cq_heads of every tensor): the tensors of `named`, (name,
    tensor or None), are [rows, heads, head_dim] on one CUDA device (`dev`, if
    given) and may be strided, but for a head's values."""
    packed = []
    for name, t in named:
        if t is None:
            packed.append(None)
            continue
        shape, stride = t.shape, t.stride()
        if len(shape) != 3:
            raise ValueError(f"{name} must be [rows, heads, head_dim], got {tuple(shape)}")
        if stride[2] != 1 and shape[2] > 1:
            raise ValueError(f"{name}: a head's values must be contiguous")
        d = t.get_device()
        if d < 0:
            raise ValueError(f"{name} must be a CUDA tensor")
        if dev < 0:
            dev = d
        elif d != dev:
            raise ValueError(f"{name} is on device {d}, the other tensors on {dev}")
        packed.append(_pack_heads(t.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0))
    return dev, packed


def _new_heads(like, shape):
    """A new tensor of heads and its cq_heads."""
    t = like.new_empty(shape)
    return t, _pack_heads(t.data_ptr(), shape[1] * shape[2], shape[2])


def _same_kind(like_name, like, pairs):
    """Every tensor of `pairs`, (name, tensor or None, shape), has the dtype
    of `like` and its shape."""
    dtype = like.dtype
    for name, t, shape in pairs:
        if t is not None and (t.dtype != dtype or t.shape != shape):
            raise ValueError(f"{name} must be {dtype} (as {like_name}) of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _index_bytes(name, t) -> int:
    import torch
    if t.dtype == torch.int64:
        return 8
    if t.dtype == torch.int32:
        return 4
    raise TypeError(f"{name} must be int32 or int64, got {t.dtype}")


def _rotation_args(q, k, positions, freqs, q_weight, k_weight, eps, norm, interleaved):
    """The arguments that qk_norm_rope and its gradient share, checked: the C
    call's from dtype to interleaved."""
    import torch
    code = _dtype_code("q", q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [rows, heads, head_dim]")
    n, qh, d = q.shape
    if k.dtype != q.dtype or k.shape[0] != n or k.shape[2] != d:
        raise ValueError(f"k must be {q.dtype} [{n}, heads, {d}], got {k.dtype} {tuple(k.shape)}")
    rotary = 0 if freqs is None else 2 * freqs.numel()
    pb = 8
    if rotary:
        if freqs.dtype != torch.float32:
            raise TypeError(f"freqs must be float32, got {freqs.dtype}")
        if positions is None or positions.numel() != n:
            raise ValueError(f"positions must hold {n} values")
        pb = _index_bytes("positions", positions)
    wc = F32
    weights = [(name, w) for name, w in (("q_weight", q_weight), ("k_weight", k_weight)) if w is not None]
    for name, w in weights:
        if not norm:
            raise ValueError(f"{name} belongs to the norm")
        if w.numel() != d:
            raise ValueError(f"{name} must hold {d} values")
        if w.dtype != weights[0][1].dtype:
            raise TypeError("q_weight and k_weight must have one dtype")
        wc = _dtype_code(name, w)
    return (code, n, qh, k.shape[1], d, int(bool(norm)), _opt(q_weight), _opt(k_weight), wc, eps,
            positions.data_ptr() if rotary else None, pb, freqs.data_ptr() if rotary else None, rotary, int(bool(interleaved)))


def qk_norm_rope(q, k, positions=None, freqs=None, q_weight=None, k_weight=None, eps: float = 1e-6, norm: bool = True,
                 interleaved: bool = False, v=None, slots=None, q_out=None, k_out=None, v_out=None, stream=None):
    """(q_out, k_out), with v (q_out, k_out, v_out): queries [n, q_heads, D] and
    keys [n, kv_heads, D], each head through its root-mean-square norm times
    q_weight / k_weight [D] (norm=False: as it is), the first 2 * len(freqs)
    values then turned in pairs by positions[i] * freqs[j] (values j and j + len(freqs), or
    neighbours with interleaved=True).  Tensors of heads may be strided, e.g.
    parts of one projection's output.  slots [n]: key row i (and v's) goes to row
    slots[i] of k_out and v_out, a cache [rows, kv_heads, D] given by the caller;
    slots outside it write nothing, a row that two slots name may mix both.
    Without slots the outputs may be given too,
    q_out=q and k_out=k among them."""
    args = _rotation_args(q, k, positions, freqs, q_weight, k_weight, eps, norm, interleaved)
    n, kvh, d = k.shape
    rows = n
    if slots is not None:
        if slots.numel() != n:
            raise ValueError(f"slots must hold {n} values")
        if k_out is None or (v is not None and v_out is None):
            raise ValueError("slots need k_out (and v_out with v)")
        rows = k_out.shape[0]
    if v is None and v_out is not None:
        raise ValueError("v_out needs v")
    _same_kind("q", q, (("v", v, (n, kvh, d)), ("q_out", q_out, q.shape), ("k_out", k_out, (rows, kvh, d)),
                        ("v_out", v_out, (rows, kvh, d))))
    heads = (("q", q), ("k", k), ("v", v), ("q_out", q_out), ("k_out", k_out), ("v_out", v_out))
    flat = (("positions", positions), ("freqs", freqs), ("q_weight", q_weight), ("k_weight", k_weight), ("slots", slots))
    dev, (qp, kp, vp, qo, ko, vo) = _heads(heads, _device(flat))
    if not _here(dev, stream):
        return _elsewhere(dev, stream, heads + flat, lambda: qk_norm_rope(
            q, k, positions, freqs, q_weight, k_weight, eps, norm, interleaved, v, slots, q_out, k_out, v_out))
    if q_out is None:
        q_out, qo = _new_heads(q, q.shape)
    if k_out is None:
        k_out, ko = _new_heads(q, k.shape)
    if v is not None and v_out is None:
        v_out, vo = _new_heads(q, k.shape)
    _check("cq_qk_norm_rope", lib().cq_qk_norm_rope(
        qp, kp, vp, *args, qo, ko, vo, _opt(slots), 8 if slots is None else _index_bytes("slots", slots), rows, _raw_stream(dev)))
    return (q_out, k_out) if v is None else (q_out, k_out, v_out)


def qk_norm_rope_grad(dq_out, dk_out, q, k, positions=None, freqs=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                      norm: bool = True, interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of qk_norm_rope at its inputs, from what
    reaches its outputs; the weights' gradients are float32 [D] (norm=False:
    None).  dq may be dq_out, dk may be dk_out."""
    import torch
    args = _rotation_args(q, k, positions, freqs, q_weight, k_weight, eps, norm, interleaved)
    _, n, qh, kvh, d = args[:5]
    _same_kind("q", q, (("dq_out", dq_out, q.shape), ("dk_out", dk_out, k.shape), ("dq", dq, q.shape), ("dk", dk, k.shape)))
    heads = (("q", q), ("k", k), ("dq_out", dq_out), ("dk_out", dk_out), ("dq", dq), ("dk", dk))
    flat = (("positions", positions), ("freqs", freqs), ("q_weight", q_weight), ("k_weight", k_weight), ("workspace", workspace))
    dev, (qp, kp, dqo, dko, dqp, dkp) = _heads(heads, _device(flat))
    if not _here(dev, stream):
        return _elsewhere(dev, stream, heads + flat, lambda: qk_norm_rope_grad(
            dq_out, dk_out, q, k, positions, freqs, q_weight, k_weight, eps, norm, interleaved, dq, dk, workspace))
    if dq is None:
        dq, dqp = _new_heads(q, q.shape)
    if dk is None:
        dk, dkp = _new_heads(q, k.shape)
    dqw = dkw = ws = None
    wb = 0
    if norm:
        dqw, dkw = q.new_empty(d, dtype=torch.float32), q.new_empty(d, dtype=torch.float32)
        ws, wb = _workspace("cq_qk_norm_rope_grad_workspace", (n, qh, kvh, d), workspace, q)
    _check("cq_qk_norm_rope_grad", lib().cq_qk_norm_rope_grad(
        dqo, dko, qp, kp, *args, dqp, dkp, _opt(dqw), _opt(dkw), _opt(ws), wb, _raw_stream(dev)))
    return dq, dk, dqw, dkw


def _attention_args(q, k, v, sequences, q_starts, k_starts, k_lens, scale):
    """(cq_sequences, their number, dtype code, q_heads, kv_heads, head_dim,
    scale) of an attention call, checked."""
    code = _dtype_code("q", q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [rows, heads, head_dim]")
    rows_q, qh, d = q.shape
    rows_k, kvh, _ = k.shape
    _same_kind("q", q, (("k", k, (rows_k, kvh, d)), ("v", v, k.shape)))
    n = sequences
    for name, t, more in (("q_starts", q_starts, 1), ("k_lens", k_lens, 0), ("k_starts", k_starts, 0 if k_lens is not None else 1)):
        if t is None:
            continue
        if t.dim() != 1 or t.numel() < more:
            raise ValueError(f"{name} must be [sequences{' + 1' if more else ''}]")
        if n is None:
            n = t.numel() - more
        elif t.numel() != n + more:
            raise ValueError(f"{name} must hold {n + more} values for {n} sequences, got {t.numel()}")
    n = 1 if n is None else n
    bytes_ = {_index_bytes(name, t) for name, t in (("q_starts", q_starts), ("k_starts", k_starts), ("k_lens", k_lens))
              if t is not None}
    if len(bytes_) > 1:
        raise TypeError("q_starts, k_starts and k_lens must have one dtype")
    seqs = _pack_sequences(n, rows_q, rows_k, _opt(q_starts) or 0, _opt(k_starts) or 0, _opt(k_lens) or 0, bytes_.pop() if bytes_ else 4)
    return seqs, n, code, qh, kvh, d, 1.0 / math.sqrt(max(d, 1)) if scale is None else scale


def attention(q, k, v, sequences=None, q_starts=None, k_starts=None, k_lens=None, causal: bool = True, scale=None, out=None,
              lse=None, workspace=None, stream=None):
    """(out, lse): attention of queries [rows_q, q_heads, D] over keys and values
    [rows_k, kv_heads, D] (q_heads a multiple of kv_heads; strided heads allowed), out
    of q's shape, lse float32 [rows_q, q_heads].  Sequences, int32 or int64 on the
    device: q_starts and k_starts [n + 1] for a packed batch; neither for
    `sequences` (1) equal parts; k_lens [n] for keys that are the first of their
    part, or from k_starts [n] on, as in a cache.  With causal the last query of a
    sequence sees all its keys.  scale: 1 / sqrt(D) by default.  Rows of no
    sequence are zeros (lse 0), or left as they are where out or lse is given."""
    import torch
    seqs, n, code, qh, kvh, d, scale = _attention_args(q, k, v, sequences, q_starts, k_starts, k_lens, scale)
    _same_kind("q", q, (("out", out, q.shape),))
    heads = (("q", q), ("k", k), ("v", v), ("out", out))
    flat = (("q_starts", q_starts), ("k_starts", k_starts), ("k_lens", k_lens), ("lse", lse), ("workspace", workspace))
    dev, (qp, kp, vp, op) = _heads(heads, _device(flat))
    if not _here(dev, stream):
        return _elsewhere(dev, stream, heads + flat, lambda: attention(
            q, k, v, sequences, q_starts, k_starts, k_lens, causal, scale, out, lse, workspace))
    gaps = q_starts is not None or n == 0  # starts may leave rows out
    if out is None:
        out, op = _new_heads(q, q.shape)
        if gaps:
            out.zero_()
    if lse is None:
        lse = q.new_empty(q.shape[:2], dtype=torch.float32)
        if gaps:
            lse.zero_()
    else:
        _out_tensor("lse", lse, q.shape[:2], torch.float32, q)
    ws, wb = _workspace("cq_attention_workspace", (seqs, code, qh, kvh, d), workspace, q)
    _check("cq_attention", lib().cq_attention(
        qp, kp, vp, code, seqs, qh, kvh, d, int(bool(causal)), scale, op, lse.data_ptr(), _opt(ws), wb, _raw_stream(dev)))
    return out, lse


def attention_grad(dout, q, k, v, out, lse, sequences=None, q_starts=None, k_starts=None, k_lens=None, causal: bool = True,
                   scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """(dq, dk, dv) of attention at its inputs, its out and its lse, from what
    reaches out (dout, of out's shape).  Every key row may belong to one
    sequence only.  Rows of no sequence are zeros, or left as they are in
    tensors that are given."""
    import torch
    seqs, n, code, qh, kvh, d, scale = _attention_args(q, k, v, sequences, q_starts, k_starts, k_lens, scale)
    _same_kind("q", q, (("dout", dout, q.shape), ("out", out, q.shape), ("dq", dq, q.shape), ("dk", dk, k.shape),
                        ("dv", dv, k.shape)))
    if lse.dtype != torch.float32 or lse.shape != q.shape[:2]:
        raise ValueError(f"lse must be float32 {tuple(q.shape[:2])}, got {lse.dtype} {tuple(lse.shape)}")
    heads = (("q", q), ("k", k), ("v", v), ("dout", dout), ("out", out), ("dq", dq), ("dk", dk), ("dv", dv))
    flat = (("q_starts", q_starts), ("k_starts", k_starts), ("k_lens", k_lens), ("lse", lse), ("workspace", workspace))
    dev, (qp, kp, vp, dop, op, dqp, dkp, dvp) = _heads(heads, _device(flat))
    if not _here(dev, stream):
        return _elsewhere(dev, stream, heads + flat, lambda: attention_grad(
            dout, q, k, v, out, lse, sequences, q_starts, k_starts, k_lens, causal, scale, dq, dk, dv, workspace))
    if dq is None:
        dq, dqp = _new_heads(q, q.shape)
        if q_starts is not None or n == 0:
            dq.zero_()  # starts may leave rows out
    gaps = k_starts is not None or k_lens is not None or n == 0
    if dk is None:
        dk, dkp = _new_heads(q, k.shape)
        if gaps:
            dk.zero_()
    if dv is None:
        dv, dvp = _new_heads(q, k.shape)
        if gaps:
            dv.zero_()
    ws, wb = _workspace("cq_attention_grad_workspace", (seqs, code, qh, kvh, d), workspace, q)
    _check("cq_attention_grad", lib().cq_attention_grad(
        dop, qp, kp, vp, op, lse.data_ptr(), code, seqs, qh, kvh, d, int(bool(causal)), scale, dqp, dkp, dvp, _opt(ws), wb,
        _raw_stream(dev)))
    return dq, dk, dv


def _logit_rows(name, t, shape):
    """Row stride of logits [*shape, vocab]: contiguous, or a matrix whose rows are."""
    if t.dim() < 1 or tuple(t.shape[:-1]) != tuple(shape):
        raise ValueError(f"{name} must be [*{tuple(shape)}, vocab], got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.shape[-1]
    if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must be contiguous, or a matrix of contiguous rows")
    return t.stride(0)


def _logits_device(logits, named) -> int:
    if logits.get_device() < 0:
        raise ValueError("logits must be a CUDA tensor")
    dev = _device(named)
    if dev >= 0 and dev != logits.get_device():
        raise ValueError(f"logits are on device {logits.get_device()}, the other tensors on {dev}")
    return logits.get_device()


def token_logprobs(logits, tokens, scale: float = 1.0, top: int = 0, stream=None):
    """TokenLogprobs(logprob, entropy, lse, top, top_logprob) of logits [..., vocab]
    (float32 or bfloat16) times scale, one over a temperature: log probability
    of tokens [...] (0 for a token outside the vocabulary), entropy and log of
    the sum, float32 [...], and the `top` most probable tokens, int64 [..., top],
    equal ones by lower index, with their log probabilities."""
    import torch
    code, tb = _dtype_code("logits", logits), _token_bytes(tokens)
    stride = _logit_rows("logits", logits, tokens.shape)
    dev = _logits_device(logits, (("tokens", tokens),))
    if not _here(dev, stream):
        return _elsewhere(dev, stream, (("logits", logits), ("tokens", tokens)), lambda: token_logprobs(logits, tokens, scale, top))
    rows, vocab = tokens.numel(), logits.shape[-1]
    shape = tokens.shape
    logprob, entropy, lse = logits.new_empty((3, *shape), dtype=torch.float32).unbind(0)
    ids = logits.new_empty((*shape, max(top, 0)), dtype=torch.int64)
    lps = logits.new_empty((*shape, max(top, 0)), dtype=torch.float32)
    _check("cq_token_logprobs", lib().cq_token_logprobs(
        logits.data_ptr(), code, rows, vocab, stride, scale, tokens.data_ptr(), tb, logprob.data_ptr(), entropy.data_ptr(),
        lse.data_ptr(), top, ids.data_ptr(), lps.data_ptr(), _raw_stream(dev)))
    return TokenLogprobs(logprob, entropy, lse, ids, lps)


def token_logprobs_grad(logits, tokens, lse, dlogprob, dentropy=None, entropy=None, scale: float = 1.0, dlogits=None,
                        stream=None):
    """Gradient of token_logprobs with respect to the logits, from its lse
    (and entropy, with dentropy) and what reaches logprob and entropy, float32 of
    tokens' shape.  Of logits' dtype and shape; dlogits may be logits."""
    import torch
    code, tb = _dtype_code("logits", logits), _token_bytes(tokens)
    stride = _logit_rows("logits", logits, tokens.shape)
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs entropy")
    named = (("tokens", tokens), ("lse", lse), ("dlogprob", dlogprob), ("dentropy", dentropy), ("entropy", entropy))
    for name, t in named[1:]:
        if t is not None and (t.dtype != torch.float32 or t.shape != tokens.shape):
            raise ValueError(f"{name} must be float32 {tuple(tokens.shape)}, got {t.dtype} {tuple(t.shape)}")
    if dlogits is not None and (dlogits.dtype != logits.dtype or dlogits.shape != logits.shape
                                or dlogits.get_device() != logits.get_device()):
        raise ValueError(f"dlogits must be {logits.dtype} {tuple(logits.shape)} on logits' device")
    out_stride = logits.shape[-1] if dlogits is None else _logit_rows("dlogits", dlogits, tokens.shape)
    dev = _logits_device(logits, named)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, named + (("logits", logits), ("dlogits", dlogits)), lambda: token_logprobs_grad(
            logits, tokens, lse, dlogprob, dentropy, entropy, scale, dlogits))
    if dlogits is None:
        dlogits = logits.new_empty(logits.shape)
    _check("cq_token_logprobs_grad", lib().cq_token_logprobs_grad(
        logits.data_ptr(), code, tokens.numel(), logits.shape[-1], stride, scale, tokens.data_ptr(), tb, lse.data_ptr(),
        dlogprob.data_ptr(), _opt(dentropy), _opt(entropy), dlogits.data_ptr(), out_stride, _raw_stream(dev)))
    return dlogits
