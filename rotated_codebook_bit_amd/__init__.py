"""Python binding of libcq, the CQ rotated-codebook quantizer for MI355X.

Thin ctypes marshalling over the C ABI declared in ``include/libcq.h``: the
names match the C entry points without the ``cq_`` prefix.  Every step of the
computation runs in libcq's HIP kernels; PyTorch only provides device memory
and the current stream.  There is no fallback: if ``libcq.so`` is missing or
a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np

__all__ = [
    "TERNARY", "TERNARY_TRITS", "GROUP", "group_bytes", "repack", "CQError", "lib", "storage_bits", "n_levels", "layout",
    "model_bytes", "codebook", "codebook_train", "quantize", "dequantize", "dequant_matvec", "dequant_matvec_many",
    "dequant_matvec_many_noalloc",
    "fake_quant", "blob_layout", "quantize_many", "dequantize_many", "dequant_gemm",
    "dequant_gemm_many", "embed", "embed_packed", "embed_grad", "add_rms_norm", "add_rms_norm_q8", "rms_norm_grad",
    "Q8Table", "q8_levels", "dequant_gemm_q8",
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
