"""Binding of libqgmm_mm.so (C ABI in ``include/qgmm_mm.h``): grouped products in bf16,
fp16 and MXFP4, the gradients of the bf16 / fp16 product, and the MXFP4 quantiser.
Argument marshalling only; the package re-exports every name here.

    p = q.make_mm_problem(m, k, n, e, x_type=q.QGMM_T_BF16, out_type=q.QGMM_T_BF16)
    ws = torch.empty(q.grouped_mm_workspace(p), dtype=torch.uint8, device="cuda")
    q.grouped_mm(p, x, w, group_list, y, ws)                        # y  = x W, expert by expert
    q.grouped_mm_dgrad(p, dy, w, group_list, dx, ws)                # dx = dy W^T
    q.grouped_mm_wgrad(p, x, dy, group_list, dw, ws)                # dW = x^T dy

    q.per_token_quant_mxfp4(x, codes, scales)                       # rows, or weights (e, n, k)
    q.mxfp4_dequant(codes, scales, out)
    p4 = q.make_mm_problem(m, k, n, e, x_type=q.QGMM_T_MXFP4, out_type=q.QGMM_T_BF16, transpose_w=True)
    ws4 = torch.empty(q.grouped_mm_workspace(p4), dtype=torch.uint8, device="cuda")
    q.grouped_mm(p4, codes, w_codes, group_list, y, ws4, x_scale=scales, w_scale=w_scales)

One workspace serves the three calls of its problem, one at a time, and the same problem with fewer
rows; 20 MB are enough for any bf16 or fp16 problem.

Tensors must lie on the current device, with the types and at least the elements that the
problem names, contiguous or with rows ``ld_x`` / ``ld_w`` / ``ld_y`` apart, weights of three
dimensions not in the other layout's shape; ``QgmmError`` is raised before any launch
otherwise.  Device pointers given as ints are passed on unchecked (``x`` of the quantiser and
``out`` of its inverse, which tell the type and the rows, have to be tensors).
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from typing import Optional

from . import (QGMM_ERR_DTYPE, QGMM_ERR_NULL_PTR, QGMM_ERR_SHAPE, QGMM_ERR_UNSUPPORTED, QGMM_GROUP_CUMSUM, QgmmError,
               _check, _stream)

HERE = os.path.dirname(os.path.abspath(__file__))
MM_LIB_PATH = os.path.join(HERE, "libqgmm_mm.so")

QGMM_T_BF16 = 0
QGMM_T_F16 = 1
QGMM_T_F32 = 2
QGMM_T_MXFP4 = 3

MM_EXPORTS = ("qgmm_grouped_mm_workspace", "qgmm_grouped_mm", "qgmm_grouped_mm_dgrad", "qgmm_grouped_mm_wgrad",
              "qgmm_per_token_quant_mxfp4", "qgmm_mxfp4_dequant")


class QgmmMmProblem(C.Structure):
    """Mirror of ``qgmm_mm_problem`` (same field order, natural C alignment)."""
    _fields_ = [
        ("m", C.c_int64), ("k", C.c_int64), ("n", C.c_int64), ("e", C.c_int64),
        ("x_type", C.c_int32), ("out_type", C.c_int32), ("group_list_type", C.c_int32), ("transpose_w", C.c_int32),
        ("accumulate", C.c_int32),
        ("ld_x", C.c_int64), ("ld_w", C.c_int64), ("ld_y", C.c_int64),
    ]


    # all fields at once: one attribute access of a ctypes structure costs as much
    unpack = struct.Struct("@4q5i3q").unpack_from


_mm_lib = None


def mm_lib():
    """Load libqgmm_mm.so (built in-tree by ``build.py``); raise if it is absent."""
    global _mm_lib
    if _mm_lib is None:
        if not os.path.exists(MM_LIB_PATH):
            raise ImportError(f"libqgmm_mm.so not built at {MM_LIB_PATH}; run "
                              "quantized_moe_grouped_persistent_b200/build.py")
        L = C.CDLL(MM_LIB_PATH)
        P, I32, I64, U, PP = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t, C.POINTER(QgmmMmProblem)
        L.qgmm_grouped_mm_workspace.argtypes = [PP, C.POINTER(C.c_size_t)]
        L.qgmm_grouped_mm.argtypes = [PP, P, P, P, P, P, P, P, U, P]
        L.qgmm_grouped_mm_dgrad.argtypes = [PP, P, P, P, P, P, U, P]
        L.qgmm_grouped_mm_wgrad.argtypes = [PP, P, P, P, P, P, U, P]
        L.qgmm_per_token_quant_mxfp4.argtypes = [P, I32, I64, I64, P, P, P]
        L.qgmm_mxfp4_dequant.argtypes = [P, P, I64, I64, P, I32, P]
        for name in MM_EXPORTS:
            getattr(L, name).restype = C.c_int
        _mm_lib = L
    return _mm_lib


_torch = None
_TYPES = ()          # torch dtype of each QGMM_T_* code
_CODES = {}          # and back, without the packed type


def _load_torch():
    global _torch, _TYPES, _CODES
    import torch
    _TYPES = (torch.bfloat16, torch.float16, torch.float32, torch.uint8)
    _CODES = {t: i for i, t in enumerate(_TYPES[:3])}
    _torch = torch
    return torch


def _device() -> int:
    """The current CUDA device; raises where there is none."""
    torch = _torch or _load_torch()
    try:
        return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else torch.cuda.current_device()
    except (AssertionError, AttributeError, RuntimeError) as e:
        raise QgmmError(QGMM_ERR_UNSUPPORTED, f"no CUDA device ({e})") from None


def _stream_of(stream, device: int) -> int:
    if stream is None:
        try:
            return _torch._C._cuda_getCurrentRawStream(device)
        except AttributeError:
            pass
    return _stream(stream)


def _extent(rows: int, row: int, ld: int) -> int:
    """Elements from the first to the last of `rows` rows of `row` elements, `ld` apart (0: dense)."""
    return (rows - 1) * (ld or row) + row if rows > 0 else 0


def _fits(what: str, name: str, t, dtype, elements: int, device: int, ld: int = 0) -> Optional[int]:
    """Data pointer of ``t``; raises unless it is a tensor on ``device``, of ``dtype``, reaches over
    ``elements`` elements and lies in memory as the call reads it: contiguous, or rows ``ld`` apart
    (an int is a pointer, and goes through)."""
    if t is None or t.__class__ is int:
        return t
    if t.get_device() != device:
        raise QgmmError(QGMM_ERR_UNSUPPORTED, f"{what}: {name} is not on the current CUDA device")
    if t.dtype is not dtype:
        raise QgmmError(QGMM_ERR_DTYPE, f"{what}: {name} is {t.dtype}, not {dtype}")
    have = t.numel()
    if not t.is_contiguous():
        shape, step = t.shape, t.stride()
        rows = all(step[i] == shape[i + 1] * step[i + 1] for i in range(len(step) - 2))
        if len(step) < 2 or step[-1] != 1 or step[-2] != ld or not rows:
            raise QgmmError(QGMM_ERR_SHAPE, f"{what}: {name} has strides {tuple(step)}; rows are {ld or 'not'} apart")
        have = 1 + sum((s - 1) * d for s, d in zip(shape, step)) if have else 0
    if have < elements:
        raise QgmmError(QGMM_ERR_SHAPE, f"{what}: {name} reaches over {have} elements, needs {elements}")
    return t.data_ptr()


def make_mm_problem(m: int, k: int, n: int, e: int, *, x_type: int = QGMM_T_BF16, out_type: int = QGMM_T_BF16,
                    group_list_type: int = QGMM_GROUP_CUMSUM, transpose_w: bool = False, accumulate: bool = False,
                    ld_x: int = 0, ld_w: int = 0, ld_y: int = 0) -> QgmmMmProblem:
    return QgmmMmProblem(m, k, n, e, x_type, out_type, group_list_type, int(bool(transpose_w)),
                         int(bool(accumulate)), ld_x, ld_w, ld_y)


def grouped_mm_workspace(problem: QgmmMmProblem) -> int:
    out = C.c_size_t(0)
    _check(mm_lib().qgmm_grouped_mm_workspace(C.byref(problem), C.byref(out)), "qgmm_grouped_mm_workspace")
    return out.value


def _read(what: str, p: QgmmMmProblem):
    """m, k, n, e, x_type, out_type, transpose_w, ld_x, ld_w, ld_y, the types in range."""
    m, k, n, e, xt, ot, _, t, _, ldx, ldw, ldy = p.unpack(p)
    if not (0 <= xt <= QGMM_T_MXFP4 and 0 <= ot <= QGMM_T_MXFP4):
        raise QgmmError(QGMM_ERR_DTYPE, what)
    return m, k, n, e, xt, ot, t, ldx, ldw, ldy


def _workspace(what: str, workspace, ws_bytes: Optional[int], device: int):
    if workspace.__class__ is int:
        if ws_bytes is None:
            raise QgmmError(QGMM_ERR_SHAPE, f"{what}: ws_bytes is needed with a workspace pointer")
        return workspace, ws_bytes
    if workspace is None:
        raise QgmmError(QGMM_ERR_NULL_PTR, f"{what}: workspace")
    have = workspace.numel() * workspace.element_size()
    ptr = _fits(what, "workspace", workspace, workspace.dtype, 0, device)
    return ptr, have if ws_bytes is None else min(ws_bytes, have)


def _fits_w(what: str, name: str, w, dtype, e: int, k: int, n: int, t: int, device: int, ld: int):
    """``_fits`` for weights; a tensor of e matrices of the other layout, which has as many elements, is refused."""
    rows, row = (n, k) if t else (k, n)
    p = _fits(what, name, w, dtype, (e * rows - 1) * (ld or row) + row, device, ld)
    if rows != row and w.__class__ is not int and w is not None and w.dim() == 3 and w.shape[1:] == (row, rows):
        raise QgmmError(QGMM_ERR_SHAPE, f"{what}: {name} is {tuple(w.shape)}, the problem's layout (e, {rows}, {row})")
    return p


def grouped_mm(problem: QgmmMmProblem, x, w, group_list, y, workspace, x_scale=None, w_scale=None,
               ws_bytes: Optional[int] = None, stream=None) -> None:
    """``y[i] = x[i] W(g)`` for every row i of every expert g."""
    what, dev = "qgmm_grouped_mm", _device()
    m, k, n, e, xt, ot, t, ldx, ldw, ldy = _read(what, problem)
    dx, u8 = _TYPES[xt], _TYPES[3]
    ps = pt = None
    if x_scale is not None:
        ps = _fits(what, "x_scale", x_scale, u8, _extent(m, k // 32, ldx // 32), dev, ldx // 32)
    if w_scale is not None:
        pt = _fits_w(what, "w_scale", w_scale, u8, e, k // 32, n, 1, dev, ldw // 32)
    py = _fits(what, "y", y, _TYPES[ot], _extent(m, n, ldy), dev, ldy)
    if xt == QGMM_T_MXFP4:         # two values per byte
        k, ldx, ldw = k // 2, ldx // 2, ldw // 2
    px = _fits(what, "x", x, dx, _extent(m, k, ldx), dev, ldx)
    pw = _fits_w(what, "w", w, dx, e, k, n, t, dev, ldw)
    pg = _fits(what, "group_list", group_list, _torch.int64, e, dev)
    ws, nbytes = _workspace(what, workspace, ws_bytes, dev)
    rc = (_mm_lib or mm_lib()).qgmm_grouped_mm(C.byref(problem), px, ps, pw, pt, pg, py, ws, nbytes, _stream_of(stream, dev))
    if rc:
        _check(rc, what)


def grouped_mm_dgrad(problem: QgmmMmProblem, dy, w, group_list, dx, workspace, ws_bytes: Optional[int] = None,
                     stream=None) -> None:
    """``dx[i] = dy[i] W(g)^T``: the gradient of ``grouped_mm`` in x, of ``problem.out_type``."""
    what, dev = "qgmm_grouped_mm_dgrad", _device()
    m, k, n, e, xt, ot, t, ldx, ldw, ldy = _read(what, problem)
    pd = _fits(what, "dy", dy, _TYPES[xt], _extent(m, n, ldy), dev, ldy)
    pw = _fits_w(what, "w", w, _TYPES[xt], e, k, n, t, dev, ldw)
    pg = _fits(what, "group_list", group_list, _torch.int64, e, dev)
    px = _fits(what, "dx", dx, _TYPES[ot], _extent(m, k, ldx), dev, ldx)
    ws, nbytes = _workspace(what, workspace, ws_bytes, dev)
    rc = (_mm_lib or mm_lib()).qgmm_grouped_mm_dgrad(C.byref(problem), pd, pw, pg, px, ws, nbytes, _stream_of(stream, dev))
    if rc:
        _check(rc, what)


def grouped_mm_wgrad(problem: QgmmMmProblem, x, dy, group_list, dw, workspace, ws_bytes: Optional[int] = None,
                     stream=None) -> None:
    """``dW(g) = sum_i x[i]^T dy[i]`` over the expert's rows: the gradient in w, of ``problem.out_type``
    and in w's layout, added to ``dw`` with ``problem.accumulate``."""
    what, dev = "qgmm_grouped_mm_wgrad", _device()
    m, k, n, e, xt, ot, t, ldx, ldw, ldy = _read(what, problem)
    px = _fits(what, "x", x, _TYPES[xt], _extent(m, k, ldx), dev, ldx)
    pd = _fits(what, "dy", dy, _TYPES[xt], _extent(m, n, ldy), dev, ldy)
    pg = _fits(what, "group_list", group_list, _torch.int64, e, dev)
    pw = _fits_w(what, "dw", dw, _TYPES[ot], e, k, n, t, dev, ldw)
    ws, nbytes = _workspace(what, workspace, ws_bytes, dev)
    rc = (_mm_lib or mm_lib()).qgmm_grouped_mm_wgrad(C.byref(problem), px, pd, pg, pw, ws, nbytes, _stream_of(stream, dev))
    if rc:
        _check(rc, what)


def _rows_of(what: str, t, *packed):
    """(type code, rows, row length) of a contiguous tensor; its packed companions must be contiguous too
    (or pointers)."""
    if t is None or any(c is None for c in packed):
        raise QgmmError(QGMM_ERR_NULL_PTR, what)
    if t.__class__ is int:
        raise QgmmError(QGMM_ERR_SHAPE, f"{what}: a pointer does not tell type, rows and k; give a tensor")
    code = _CODES.get(t.dtype)
    if code is None:
        raise QgmmError(QGMM_ERR_DTYPE, f"{what}: {t.dtype}")
    if not (t.is_contiguous() and all(c.__class__ is int or c.is_contiguous() for c in packed)):
        raise QgmmError(QGMM_ERR_SHAPE, f"{what}: contiguous tensors only")
    k = t.shape[-1] if t.dim() else 0
    return code, t.numel() // k if k else 0, k


def per_token_quant_mxfp4(x, q_out, sf_out, stream=None) -> None:
    """MXFP4 codes of ``x`` (a contiguous tensor, its last dimension the rows' length k) into ``q_out``
    (uint8, k/2 per row) and E8M0 codes into ``sf_out`` (uint8, k/32 per row)."""
    what, dev = "qgmm_per_token_quant_mxfp4", _device()
    code, rows, k = _rows_of(what, x, q_out, sf_out)
    px = _fits(what, "x", x, x.dtype, 0, dev)
    pq = _fits(what, "q_out", q_out, _torch.uint8, rows * (k // 2), dev)
    ps = _fits(what, "sf_out", sf_out, _torch.uint8, rows * (k // 32), dev)
    rc = (_mm_lib or mm_lib()).qgmm_per_token_quant_mxfp4(px, code, rows, k, pq, ps, _stream_of(stream, dev))
    if rc:
        _check(rc, what)


def mxfp4_dequant(q, sf, out, stream=None) -> None:
    """The values that MXFP4 codes stand for, into ``out`` (its last dimension the rows' length k)."""
    what, dev = "qgmm_mxfp4_dequant", _device()
    code, rows, k = _rows_of(what, out, q, sf)
    pq = _fits(what, "q", q, _torch.uint8, rows * (k // 2), dev)
    ps = _fits(what, "sf", sf, _torch.uint8, rows * (k // 32), dev)
    po = _fits(what, "out", out, out.dtype, 0, dev)
    rc = (_mm_lib or mm_lib()).qgmm_mxfp4_dequant(pq, ps, rows, k, po, code, _stream_of(stream, dev))
    if rc:
        _check(rc, what)
