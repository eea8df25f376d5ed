"""Python binding of the MXFP4 experts' operators (include/fp8blk_mxfp4.h).

The functions named ``fp8_*`` forward tensors' device pointers, sizes and a
stream to the entry point of the same name, after the checks that the library
cannot make from pointers: every tensor on one GPU, contiguous, of the
documented type and shape.  Every output is the caller's.  The functions
without the prefix allocate their outputs.

Streams are as in the mixture-of-experts operators (``moe``): torch's current
stream of the tensors' device, or ``stream``.
"""

import ctypes

import torch

from .moe import (_BF, _CODES, _E8M0, _FLOATS, _I32, _RULES, _U8, _allocating, _choice, _dims, _is_f32, _lib, _may,
                  _need, _run)

__all__ = [
    "fp8_mxfp4_quantize", "fp8_mxfp4_dequantize", "fp8_mxfp4_gemm", "fp8_mxfp4_grouped_gemm",
    "fp8_mxfp4_matvec", "fp8_mxfp4_grouped_matvec", "fp8_grouped_dgrad", "fp8_grouped_wgrad",
    "fp8_mxfp4_abi_version",
    "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_grouped_gemm", "mxfp4_matvec", "mxfp4_grouped_matvec",
    "grouped_dgrad", "grouped_wgrad",
]

MXFP4_ABI_VERSION = 1
_ELEMS = {"e4m3": 0, "e2m1": 1, 0: 0, 1: 1}


def declare(lib):
    """Argument types of the entry points in a loaded library."""
    i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    for name, args in (
            ("fp8_mxfp4_quantize", [vp, i64, i64, ci, vp, vp, vp, vp]),
            ("fp8_mxfp4_dequantize", [vp, vp, i64, i64, vp, vp]),
            ("fp8_mxfp4_gemm", [vp, vp, ci, vp, vp, i64, i64, i64, vp, ci, vp]),
            ("fp8_mxfp4_grouped_gemm", [vp, vp, ci, i64, vp, vp, vp, vp, i64, i64, i64, i64, vp, ci, vp]),
            ("fp8_mxfp4_matvec", [vp, vp, vp, i64, i64, i64, vp, ci, vp]),
            ("fp8_mxfp4_grouped_matvec", [vp, i64, vp, vp, vp, vp, i64, i64, i64, i64, vp, ci, vp]),
            ("fp8_grouped_dgrad", [vp, vp, vp, i64, i64, i64, i64, vp, ci, vp]),
            ("fp8_grouped_wgrad", [vp, vp, i64, vp, vp, i64, i64, i64, i64, vp, ci, vp]),
            ("fp8_mxfp4_abi_version", [])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ci
    if lib.fp8_mxfp4_abi_version() != MXFP4_ABI_VERSION:
        raise ImportError("libfp8blk.so ABI version mismatch (MXFP4 experts)")


# ------------------------------------------------------------- entry points

def fp8_mxfp4_quantize(x, rule, q, scale, xdq=None, stream=None):
    """x bf16 [rows, cols] -> q uint8 [rows, cols/2] (two E2M1 codes per
    byte), scale uint8 / float8_e8m0fnu [rows, cols/32]; rule "ceil" or
    "floor"; xdq: optional bf16 [rows, cols] of the fake-quant values."""
    where = "fp8_mxfp4_quantize"
    shape = _dims(where, "x", x, 2)
    rows, cols = shape
    dev = x.get_device()
    _run(where, dev, stream, _lib().fp8_mxfp4_quantize, _need(where, "x", x, (_BF,), shape, dev), rows, cols,
         _choice(where, "rule", rule, _RULES), _need(where, "q", q, (_U8,), (rows, cols // 2), dev),
         _need(where, "scale", scale, _E8M0, (rows, cols // 32), dev),
         _may(where, "xdq", xdq, (_BF,), shape, dev))


def fp8_mxfp4_dequantize(q, scale, x, stream=None):
    """q uint8 [rows, cols/2], scale [rows, cols/32] -> x bf16 [rows, cols]."""
    where = "fp8_mxfp4_dequantize"
    shape = _dims(where, "x", x, 2)
    rows, cols = shape
    dev = x.get_device()
    _run(where, dev, stream, _lib().fp8_mxfp4_dequantize, _need(where, "q", q, (_U8,), (rows, cols // 2), dev),
         _need(where, "scale", scale, _E8M0, (rows, cols // 32), dev), rows, cols,
         _need(where, "x", x, (_BF,), shape, dev))


def _rows_of(where, a_q, a_elem):
    """(element, rows, k, types of the codes) of a product's rows."""
    elem = _choice(where, "a_elem", a_elem, _ELEMS)
    rows, width = _dims(where, "a_q", a_q, 2)
    return elem, rows, 2 * width if elem else width, (_U8,) if elem else _CODES


def fp8_mxfp4_gemm(a_q, a_scale, a_elem, b_q, b_scale, y, stream=None):
    """y = deq(A) . deq(B)^T for B in MXFP4 and A in MXFP8 (a_elem "e4m3") or
    MXFP4 ("e2m1"): a_q uint8 / float8_e4m3fn [m, k] or uint8 [m, k/2];
    b_q uint8 [n, k/2]; scales uint8 / float8_e8m0fnu [m, k/32] and
    [n, k/32]; y bf16 or float32 [m, n].  Sums are fp32's, except those of
    E4M3 rows for a bf16 y: each run of 8 products is off by up to
    7 * 2^-12 of its largest."""
    where = "fp8_mxfp4_gemm"
    elem, m, k, types = _rows_of(where, a_q, a_elem)
    n = _dims(where, "b_q", b_q, 2)[0]
    dev = a_q.get_device()
    _run(where, dev, stream, _lib().fp8_mxfp4_gemm, _need(where, "a_q", a_q, types, a_q.shape, dev),
         _need(where, "a_scale", a_scale, _E8M0, (m, k // 32), dev), elem,
         _need(where, "b_q", b_q, (_U8,), (n, k // 2), dev),
         _need(where, "b_scale", b_scale, _E8M0, (n, k // 32), dev), m, n, k,
         _need(where, "y", y, _FLOATS, (m, n), dev), _is_f32(y))


def fp8_mxfp4_grouped_gemm(a_q, a_scale, a_elem, row_index, b_q, b_scale, group_offsets, y, stream=None):
    """fp8_mxfp4_gemm over routed experts: rows [off[g], off[g+1]) of y take
    matrix g of b_q [groups, n, k/2] (b_scale [groups, n, k/32]); row i reads
    row row_index[i] of A (int32 [total_m]), or row i where that is None.
    group_offsets int32 [groups + 1]; y [total_m, n]: rows behind
    off[groups] are left as they were."""
    where = "fp8_mxfp4_grouped_gemm"
    elem, a_rows, k, types = _rows_of(where, a_q, a_elem)
    groups, n, _ = _dims(where, "b_q", b_q, 3)
    total_m = _dims(where, "y", y, 2)[0]
    dev = a_q.get_device()
    if row_index is None and a_rows != total_m:
        raise ValueError(f"{where}: a_q has {a_rows} rows and y {total_m}: without row_index they must agree")
    _run(where, dev, stream, _lib().fp8_mxfp4_grouped_gemm, _need(where, "a_q", a_q, types, a_q.shape, dev),
         _need(where, "a_scale", a_scale, _E8M0, (a_rows, k // 32), dev), elem, a_rows,
         _may(where, "row_index", row_index, (_I32,), (total_m,), dev),
         _need(where, "b_q", b_q, (_U8,), (groups, n, k // 2), dev),
         _need(where, "b_scale", b_scale, _E8M0, (groups, n, k // 32), dev),
         _need(where, "group_offsets", group_offsets, (_I32,), (groups + 1,), dev), groups, total_m, n, k,
         _need(where, "y", y, _FLOATS, (total_m, n), dev), _is_f32(y))


def fp8_mxfp4_matvec(x, q, scale, y, stream=None):
    """y = x . W^T for MXFP4 W: x bf16 [m, k] (m up to about 32); q uint8
    [n, k/2], scale uint8 / float8_e8m0fnu [n, k/32]; y bf16 or float32
    [m, n]."""
    where = "fp8_mxfp4_matvec"
    m, k = _dims(where, "x", x, 2)
    n = _dims(where, "q", q, 2)[0]
    dev = x.get_device()
    _run(where, dev, stream, _lib().fp8_mxfp4_matvec, _need(where, "x", x, (_BF,), (m, k), dev),
         _need(where, "q", q, (_U8,), (n, k // 2), dev), _need(where, "scale", scale, _E8M0, (n, k // 32), dev), m, n, k,
         _need(where, "y", y, _FLOATS, (m, n), dev), _is_f32(y))


def fp8_mxfp4_grouped_matvec(x, row_index, q, scale, group_offsets, y, stream=None):
    """fp8_mxfp4_matvec over routed experts: rows [off[g], off[g+1]) of y
    take matrix g of q uint8 [groups, n, k/2] (scale [groups, n, k/32]); row i
    reads x[row_index[i]], or x[i] where row_index is None.  group_offsets
    int32 [groups + 1] and row_index int32 [total_m]; y [total_m, n]: rows
    behind off[groups] are left as they were."""
    where = "fp8_mxfp4_grouped_matvec"
    x_rows, k = _dims(where, "x", x, 2)
    groups, n, _ = _dims(where, "q", q, 3)
    total_m = _dims(where, "y", y, 2)[0]
    dev = x.get_device()
    if row_index is None and x_rows != total_m:
        raise ValueError(f"{where}: x has {x_rows} rows and y {total_m}: without row_index they must agree")
    _run(where, dev, stream, _lib().fp8_mxfp4_grouped_matvec, _need(where, "x", x, (_BF,), (x_rows, k), dev), x_rows,
         _may(where, "row_index", row_index, (_I32,), (total_m,), dev),
         _need(where, "q", q, (_U8,), (groups, n, k // 2), dev),
         _need(where, "scale", scale, _E8M0, (groups, n, k // 32), dev),
         _need(where, "group_offsets", group_offsets, (_I32,), (groups + 1,), dev), groups, total_m, n, k,
         _need(where, "y", y, _FLOATS, (total_m, n), dev), _is_f32(y))


def fp8_grouped_dgrad(dy, w, group_offsets, dx, stream=None):
    """dx[i] = dy[i] . W[g] for the rows i of group g: dy bf16 [total_m, n];
    w bf16 [groups, n, k]; group_offsets int32 [groups + 1]; dx bf16 or
    float32 [total_m, k]: rows behind off[groups] are left as they were."""
    where = "fp8_grouped_dgrad"
    total_m, n = _dims(where, "dy", dy, 2)
    groups, _, k = _dims(where, "w", w, 3)
    dev = dy.get_device()
    _run(where, dev, stream, _lib().fp8_grouped_dgrad, _need(where, "dy", dy, (_BF,), (total_m, n), dev),
         _need(where, "w", w, (_BF,), (groups, n, k), dev),
         _need(where, "group_offsets", group_offsets, (_I32,), (groups + 1,), dev), groups, total_m, n, k,
         _need(where, "dx", dx, _FLOATS, (total_m, k), dev), _is_f32(dx))


def fp8_grouped_wgrad(dy, x, row_index, group_offsets, dw, stream=None):
    """dw[g] = dy[rows of g]^T . x[rows of g]: dy bf16 [total_m, n]; x bf16
    [x_rows, k], its row of grouped row i row_index[i] (int32 [total_m]) or i
    where that is None; group_offsets int32 [groups + 1]; dw bf16 or float32
    [groups, n, k], all of it written (zeros for groups without rows)."""
    where = "fp8_grouped_wgrad"
    total_m, n = _dims(where, "dy", dy, 2)
    x_rows, k = _dims(where, "x", x, 2)
    groups = _dims(where, "dw", dw, 3)[0]
    dev = dy.get_device()
    if row_index is None and x_rows != total_m:
        raise ValueError(f"{where}: x has {x_rows} rows and dy {total_m}: without row_index they must agree")
    _run(where, dev, stream, _lib().fp8_grouped_wgrad, _need(where, "dy", dy, (_BF,), (total_m, n), dev),
         _need(where, "x", x, (_BF,), (x_rows, k), dev), x_rows,
         _may(where, "row_index", row_index, (_I32,), (total_m,), dev),
         _need(where, "group_offsets", group_offsets, (_I32,), (groups + 1,), dev), groups, total_m, n, k,
         _need(where, "dw", dw, _FLOATS, (groups, n, k), dev), _is_f32(dw))


def fp8_mxfp4_abi_version():
    return _lib().fp8_mxfp4_abi_version()


# --------------------------------------------- allocating conveniences (torch)

def mxfp4_quantize(x, rule="ceil", dequant=False, stream=None):
    """Allocate outputs and run fp8_mxfp4_quantize: returns (q uint8
    [rows, cols/2], scale uint8 [rows, cols/32][, xdq])."""
    rows, cols = _dims("mxfp4_quantize", "x", x, 2)
    with _allocating(stream, x.device):
        q = torch.empty((rows, cols // 2), dtype=_U8, device=x.device)
        scale = torch.empty((rows, cols // 32), dtype=_U8, device=x.device)
        xdq = torch.empty_like(x) if dequant else None
        fp8_mxfp4_quantize(x, rule, q, scale, xdq, stream)
    return (q, scale, xdq) if dequant else (q, scale)


def mxfp4_dequantize(q, scale, stream=None):
    """Allocate the bf16 output and run fp8_mxfp4_dequantize."""
    rows, half = _dims("mxfp4_dequantize", "q", q, 2)
    with _allocating(stream, q.device):
        x = torch.empty((rows, 2 * half), dtype=_BF, device=q.device)
        fp8_mxfp4_dequantize(q, scale, x, stream)
    return x


def mxfp4_gemm(a_q, a_scale, a_elem, b_q, b_scale, out_dtype=torch.bfloat16, stream=None):
    """Allocate y and run fp8_mxfp4_gemm."""
    m = _dims("mxfp4_gemm", "a_q", a_q, 2)[0]
    n = _dims("mxfp4_gemm", "b_q", b_q, 2)[0]
    with _allocating(stream, a_q.device):
        y = torch.empty((m, n), dtype=out_dtype, device=a_q.device)
        fp8_mxfp4_gemm(a_q, a_scale, a_elem, b_q, b_scale, y, stream)
    return y


def mxfp4_grouped_gemm(a_q, a_scale, a_elem, b_q, b_scale, group_offsets, row_index=None, out_dtype=torch.bfloat16,
                       stream=None):
    """Allocate y and run fp8_mxfp4_grouped_gemm.  Rows behind off[groups]
    are zero."""
    total_m = _dims("mxfp4_grouped_gemm", "a_q", a_q, 2)[0] if row_index is None else row_index.numel()
    n = _dims("mxfp4_grouped_gemm", "b_q", b_q, 3)[1]
    with _allocating(stream, a_q.device):
        y = torch.zeros((total_m, n), dtype=out_dtype, device=a_q.device)
        fp8_mxfp4_grouped_gemm(a_q, a_scale, a_elem, row_index, b_q, b_scale, group_offsets, y, stream)
    return y


def mxfp4_matvec(x, q, scale, out_dtype=torch.bfloat16, stream=None):
    """Allocate y and run fp8_mxfp4_matvec."""
    m = _dims("mxfp4_matvec", "x", x, 2)[0]
    n = _dims("mxfp4_matvec", "q", q, 2)[0]
    with _allocating(stream, x.device):
        y = torch.empty((m, n), dtype=out_dtype, device=x.device)
        fp8_mxfp4_matvec(x, q, scale, y, stream)
    return y


def mxfp4_grouped_matvec(x, q, scale, group_offsets, row_index=None, out_dtype=torch.bfloat16, stream=None):
    """Allocate y and run fp8_mxfp4_grouped_matvec.  Rows behind off[groups]
    are zero."""
    total_m = _dims("mxfp4_grouped_matvec", "x", x, 2)[0] if row_index is None else row_index.numel()
    n = _dims("mxfp4_grouped_matvec", "q", q, 3)[1]
    with _allocating(stream, x.device):
        y = torch.zeros((total_m, n), dtype=out_dtype, device=x.device)
        fp8_mxfp4_grouped_matvec(x, row_index, q, scale, group_offsets, y, stream)
    return y


def grouped_dgrad(dy, w, group_offsets, out_dtype=torch.bfloat16, stream=None):
    """Allocate dx and run fp8_grouped_dgrad.  Rows behind off[groups] are
    zero."""
    total_m = _dims("grouped_dgrad", "dy", dy, 2)[0]
    k = _dims("grouped_dgrad", "w", w, 3)[2]
    with _allocating(stream, dy.device):
        dx = torch.zeros((total_m, k), dtype=out_dtype, device=dy.device)
        fp8_grouped_dgrad(dy, w, group_offsets, dx, stream)
    return dx


def grouped_wgrad(dy, x, group_offsets, row_index=None, out_dtype=torch.float32, stream=None):
    """Allocate dw and run fp8_grouped_wgrad."""
    n = _dims("grouped_wgrad", "dy", dy, 2)[1]
    k = _dims("grouped_wgrad", "x", x, 2)[1]
    groups = _dims("grouped_wgrad", "group_offsets", group_offsets, 1)[0] - 1
    with _allocating(stream, dy.device):
        dw = torch.empty((groups, n, k), dtype=out_dtype, device=dy.device)
        fp8_grouped_wgrad(dy, x, row_index, group_offsets, dw, stream)
    return dw
