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
    q.grouped_mm(p4, codes, w_codes, group_list, y, ws, x_scale=scales, w_scale=w_scales)

Tensors must lie on the current device, with the types and at least the elements that the
problem names; ``QgmmError`` is raised before any launch otherwise.  Device pointers
given as ints are passed on unchecked.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional

from . import (QGMM_ERR_DTYPE, QGMM_ERR_SHAPE, QGMM_ERR_UNSUPPORTED, QGMM_GROUP_CUMSUM, QgmmError, _check, _ptr,
               _stream)

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


_TORCH_TYPES = None


def _dtypes():
    global _TORCH_TYPES
    if _TORCH_TYPES is None:
        import torch
        _TORCH_TYPES = {QGMM_T_BF16: torch.bfloat16, QGMM_T_F16: torch.float16, QGMM_T_F32: torch.float32,
                        QGMM_T_MXFP4: torch.uint8}
    return _TORCH_TYPES


def _extent(rows: int, row: int, ld: int) -> int:
    """Elements from the first to the last of `rows` rows of `row` elements, `ld` apart (0: dense)."""
    return (rows - 1) * (ld or row) + row if rows > 0 else 0


def _fits(what: str, name: str, t, dtype, elements: int) -> None:
    """Raise unless tensor ``t`` is on the current device, of ``dtype`` and reaches over ``elements`` elements."""
    if t is None or isinstance(t, int):
        return
    import torch
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise QgmmError(QGMM_ERR_UNSUPPORTED, f"{what}: {name} is not on the current CUDA device")
    if t.dtype != dtype:
        raise QgmmError(QGMM_ERR_DTYPE, f"{what}: {name} is {t.dtype}, not {dtype}")
    # a contiguous tensor's own elements; of a strided view, what lies between its first and last
    have = t.numel()
    if have and not t.is_contiguous():
        have = 1 + sum((s - 1) * d for s, d in zip(t.shape, t.stride()))
    if have < elements:
        raise QgmmError(QGMM_ERR_SHAPE, f"{what}: {name} reaches over {have} elements, needs {elements}")


def make_mm_problem(m: int, k: int, n: int, e: int, *, x_type: int = QGMM_T_BF16, out_type: int = QGMM_T_BF16,
                    group_list_type: int = QGMM_GROUP_CUMSUM, transpose_w: bool = False, accumulate: bool = False,
                    ld_x: int = 0, ld_w: int = 0, ld_y: int = 0) -> QgmmMmProblem:
    return QgmmMmProblem(m, k, n, e, x_type, out_type, group_list_type, int(bool(transpose_w)),
                         int(bool(accumulate)), ld_x, ld_w, ld_y)


def grouped_mm_workspace(problem: QgmmMmProblem) -> int:
    out = C.c_size_t(0)
    _check(mm_lib().qgmm_grouped_mm_workspace(C.byref(problem), C.byref(out)), "qgmm_grouped_mm_workspace")
    return out.value


def _check_mm(what, p, rows, w, group_list, out_name, out, scales=(None, None)) -> None:
    """``rows``: (name, tensor, width, ld) of the row operands; ``out``: the output, with its extent."""
    import torch
    types = _dtypes()
    if p.x_type not in types or p.out_type not in types:
        raise QgmmError(QGMM_ERR_DTYPE, what)
    pack = 2 if p.x_type == QGMM_T_MXFP4 else 1          # MXFP4 values per byte
    for name, t, width, ld in rows:
        _fits(what, name, t, types[p.x_type], _extent(p.m, width // pack, ld // pack))
    w_rows, w_row = (p.n, p.k) if p.transpose_w else (p.k, p.n)
    w_extent = _extent(p.e * w_rows, w_row // pack, p.ld_w // pack)
    if w is not None:
        _fits(what, "w", w, types[p.x_type], w_extent)
    _fits(what, "group_list", group_list, torch.int64, p.e)
    _fits(what, out_name, out[0], types[p.out_type], w_extent if out[1] is None else out[1])
    if scales[0] is not None:
        _fits(what, "x_scale", scales[0], torch.uint8, _extent(p.m, p.k // 32, p.ld_x // 32))
    if scales[1] is not None:
        _fits(what, "w_scale", scales[1], torch.uint8, _extent(p.e * p.n, p.k // 32, p.ld_w // 32))


def _ws(what, workspace, ws_bytes: Optional[int]) -> int:
    import torch
    if not isinstance(workspace, int):
        have = workspace.numel() * workspace.element_size()
        _fits(what, "workspace", workspace, workspace.dtype, 0)
        return have if ws_bytes is None else min(ws_bytes, have)
    if ws_bytes is None:
        raise QgmmError(QGMM_ERR_SHAPE, f"{what}: ws_bytes is needed with a workspace pointer")
    return ws_bytes


def grouped_mm(problem: QgmmMmProblem, x, w, group_list, y, workspace, x_scale=None, w_scale=None,
               ws_bytes: Optional[int] = None, stream=None) -> None:
    """``y[i] = x[i] W(g)`` for every row i of every expert g."""
    p = problem
    _check_mm("qgmm_grouped_mm", p, (("x", x, p.k, p.ld_x),), w, group_list, "y", (y, _extent(p.m, p.n, p.ld_y)),
              (x_scale, w_scale))
    rc = mm_lib().qgmm_grouped_mm(C.byref(p), _ptr(x), _ptr(x_scale), _ptr(w), _ptr(w_scale), _ptr(group_list),
                                  _ptr(y), _ptr(workspace), _ws("qgmm_grouped_mm", workspace, ws_bytes),
                                  _stream(stream))
    _check(rc, "qgmm_grouped_mm")


def grouped_mm_dgrad(problem: QgmmMmProblem, dy, w, group_list, dx, workspace, ws_bytes: Optional[int] = None,
                     stream=None) -> None:
    """``dx[i] = dy[i] W(g)^T``: the gradient of ``grouped_mm`` in x, of ``problem.out_type``."""
    p = problem
    _check_mm("qgmm_grouped_mm_dgrad", p, (("dy", dy, p.n, p.ld_y),), w, group_list, "dx",
              (dx, _extent(p.m, p.k, p.ld_x)))
    rc = mm_lib().qgmm_grouped_mm_dgrad(C.byref(p), _ptr(dy), _ptr(w), _ptr(group_list), _ptr(dx), _ptr(workspace),
                                        _ws("qgmm_grouped_mm_dgrad", workspace, ws_bytes), _stream(stream))
    _check(rc, "qgmm_grouped_mm_dgrad")


def grouped_mm_wgrad(problem: QgmmMmProblem, x, dy, group_list, dw, workspace, ws_bytes: Optional[int] = None,
                     stream=None) -> None:
    """``dW(g) = sum_i x[i]^T dy[i]`` over the expert's rows: the gradient in w, of ``problem.out_type``
    and in w's layout, added to ``dw`` with ``problem.accumulate``."""
    p = problem
    _check_mm("qgmm_grouped_mm_wgrad", p, (("x", x, p.k, p.ld_x), ("dy", dy, p.n, p.ld_y)), None, group_list, "dw",
              (dw, None))
    rc = mm_lib().qgmm_grouped_mm_wgrad(C.byref(p), _ptr(x), _ptr(dy), _ptr(group_list), _ptr(dw), _ptr(workspace),
                                        _ws("qgmm_grouped_mm_wgrad", workspace, ws_bytes), _stream(stream))
    _check(rc, "qgmm_grouped_mm_wgrad")


def _type_of(what: str, t) -> int:
    for code, dtype in _dtypes().items():
        if t.dtype == dtype and code != QGMM_T_MXFP4:
            return code
    raise QgmmError(QGMM_ERR_DTYPE, f"{what}: {t.dtype}")


def per_token_quant_mxfp4(x, q_out, sf_out, stream=None) -> None:
    """MXFP4 codes of ``x`` (a contiguous tensor, its last dimension the rows' length k) into ``q_out``
    (uint8, k/2 per row) and E8M0 codes into ``sf_out`` (uint8, k/32 per row)."""
    import torch
    what = "qgmm_per_token_quant_mxfp4"
    k = int(x.shape[-1])
    rows = x.numel() // k if k else 0
    if not (x.is_contiguous() and q_out.is_contiguous() and sf_out.is_contiguous()):
        raise QgmmError(QGMM_ERR_SHAPE, f"{what}: contiguous tensors only")
    _fits(what, "x", x, x.dtype, 0)
    _fits(what, "q_out", q_out, torch.uint8, rows * (k // 2))
    _fits(what, "sf_out", sf_out, torch.uint8, rows * (k // 32))
    _check(mm_lib().qgmm_per_token_quant_mxfp4(_ptr(x), _type_of(what, x), rows, k, _ptr(q_out), _ptr(sf_out),
                                               _stream(stream)), what)


def mxfp4_dequant(q, sf, out, stream=None) -> None:
    """The values that MXFP4 codes stand for, into ``out`` (its last dimension the rows' length k)."""
    import torch
    what = "qgmm_mxfp4_dequant"
    k = int(out.shape[-1])
    rows = out.numel() // k if k else 0
    if not (q.is_contiguous() and sf.is_contiguous() and out.is_contiguous()):
        raise QgmmError(QGMM_ERR_SHAPE, f"{what}: contiguous tensors only")
    _fits(what, "q", q, torch.uint8, rows * (k // 2))
    _fits(what, "sf", sf, torch.uint8, rows * (k // 32))
    _fits(what, "out", out, out.dtype, 0)
    _check(mm_lib().qgmm_mxfp4_dequant(_ptr(q), _ptr(sf), rows, k, _ptr(out), _type_of(what, out), _stream(stream)),
           what)
