"""Python binding of the mixture-of-experts operators (include/fp8blk_moe.h).

The functions named ``fp8_*`` forward tensors' device pointers, sizes and a
stream to the entry point of the same name, after the checks that the
library cannot make from pointers: every tensor on one GPU, contiguous, of
the documented type and shape.  Every output and workspace is the caller's.
The functions without the prefix allocate their outputs.

Streams: a call runs on torch's current stream of its tensors' device, or on
``stream`` (a torch stream or a raw handle).  With ``stream``, the allocating
functions allocate on it, so that what they return belongs to it; tensors
passed in have to be ready on it and to stay alive until it has used them
(``Tensor.record_stream``), as for any kernel launched on another stream.
"""

import contextlib
import ctypes

import torch

__all__ = [
    "fp8_rmsnorm_quantize", "fp8_rmsnorm_backward", "fp8_rmsnorm_backward_workspace",
    "fp8_moe_route", "fp8_moe_route_backward", "fp8_moe_plan", "fp8_moe_plan_workspace",
    "fp8_nvfp4_matvec", "fp8_nvfp4_grouped_matvec",
    "fp8_moe_combine", "fp8_moe_combine_backward", "fp8_moe_abi_version",
    "rmsnorm_quantize", "rmsnorm_backward", "moe_route", "moe_route_backward", "moe_plan",
    "nvfp4_matvec", "nvfp4_grouped_matvec", "moe_combine", "moe_combine_backward",
]

MOE_ABI_VERSION = 1
_BLOCKS = {"1x32": 0, "1x128": 1, 0: 0, 1: 1}
_RULES = {"ceil": 0, "floor": 1, 0: 0, 1: 1}
_SCORES = {"softmax": 0, "sigmoid": 1, 0: 0, 1: 1}
_GROUP_SCORES = {"max": 0, "top2": 1, 0: 0, 1: 1}

_BF, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_FLOATS = (_BF, _F32)
_CODES = (torch.uint8, torch.float8_e4m3fn)
_E8M0 = (torch.uint8, torch.float8_e8m0fnu)

_native = None


def declare(lib):
    """Argument types of the entry points in a loaded library."""
    i64, vp, ci, cf, cs = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    size_out = ctypes.POINTER(cs)
    for name, args in (
            ("fp8_rmsnorm_quantize", [vp, vp, vp, ci, i64, i64, cf, ci, ci, vp, vp, vp, vp, vp, vp, vp]),
            ("fp8_rmsnorm_backward", [vp, vp, vp, ci, vp, vp, i64, i64, vp, cs, vp, vp, vp]),
            ("fp8_rmsnorm_backward_workspace", [i64, i64, size_out]),
            ("fp8_moe_route", [vp, ci, vp, i64, ci, ci, ci, ci, ci, ci, ci, cf, vp, vp, vp]),
            ("fp8_moe_route_backward", [vp, ci, vp, vp, i64, ci, ci, ci, ci, cf, vp, vp]),
            ("fp8_moe_plan", [vp, i64, ci, ci, vp, cs, vp, vp, vp, vp]),
            ("fp8_moe_plan_workspace", [i64, ci, ci, size_out]),
            ("fp8_nvfp4_matvec", [vp, vp, vp, vp, i64, i64, i64, i64, vp, ci, vp]),
            ("fp8_nvfp4_grouped_matvec", [vp, i64, vp, vp, vp, vp, i64, vp, i64, i64, i64, i64, vp, ci, vp]),
            ("fp8_moe_combine", [vp, ci, i64, vp, vp, vp, i64, ci, i64, vp, ci, vp]),
            ("fp8_moe_combine_backward", [vp, ci, vp, ci, i64, vp, vp, i64, ci, i64, vp, vp, vp]),
            ("fp8_moe_abi_version", [])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ci
    if lib.fp8_moe_abi_version() != MOE_ABI_VERSION:
        raise ImportError("libfp8blk.so ABI version mismatch (mixture-of-experts operators)")


def _lib():
    global _native
    if _native is None:
        from . import library
        _native = library()
    return _native


def _raise(status, where):
    from . import Fp8Error
    raise Fp8Error(status, where)


def _choice(where, name, value, table):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{where}: {name} {value!r}, expected one of "
                         f"{', '.join(repr(k) for k in table if isinstance(k, str))}") from None


def _bad(where, name, t, dtypes, shape, dev):
    """Why ``t`` is refused (called when a check has failed)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{where}: {name} must be a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise ValueError(f"{where}: {name} has dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")
    raise ValueError(f"{where}: tensors on different devices ({_device(dev)} and {t.device} for {name})")


def _device(dev):
    return torch.device("cuda", dev) if dev >= 0 else torch.device("cpu")


def _need(where, name, t, dtypes, shape, dev):
    """The address of a contiguous tensor of one of ``dtypes`` and exactly
    ``shape`` on GPU number ``dev`` (-1: the host, which _run refuses)."""
    try:
        if t.dtype in dtypes and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _bad(where, name, t, dtypes, shape, dev)


def _may(where, name, t, dtypes, shape, dev):
    return None if t is None else _need(where, name, t, dtypes, shape, dev)


def _dims(where, name, t, count):
    try:
        if t.dim() == count:
            return t.shape
    except AttributeError:
        raise ValueError(f"{where}: {name} must be a tensor, got {type(t).__name__}") from None
    raise ValueError(f"{where}: {name} must have {count} dimensions, got shape {tuple(t.shape)}")


def _workspace(where, t, dev):
    """(address, bytes) of a workspace tensor of any type; None where none is needed."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{where}: the workspace must be a contiguous tensor on {_device(dev)}")
    return t.data_ptr(), t.numel() * t.element_size()


# torch's current stream of a GPU as a raw handle, and the current GPU.  The
# public calls build a Stream object and look whether torch is initialized
# first, 2.0 of the 8.8 us of a small call; torch's own compiled code takes
# both directly too.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_gpu = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(where, dev, stream, fn, *args):
    """Calls an entry point on ``stream`` (None: torch's current one) with GPU number ``dev`` as the current device,
    which is the one the library launches on."""
    if dev < 0:
        raise ValueError(f"{where}: every tensor must be on a GPU")
    if stream is None:
        handle = _raw_stream(dev)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if dev == _current_gpu():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status:
        _raise(status, where)


def _allocating(stream, dev):
    """Context in which an allocating function allocates and calls: with an
    explicit stream its memory has to come from that stream."""
    if stream is None or dev.type != "cuda":
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return torch.cuda.stream(stream)


def _is_f32(t):
    return 1 if t.dtype == _F32 else 0


# ------------------------------------------------------------- entry points

def fp8_rmsnorm_quantize(x, weight, eps, kind, rule, q, scale, residual=None, h=None, y=None, ydq=None, rstd=None,
                         stream=None):
    """h = x + residual; y = h * rstd * weight; q, scale = y in FP8 with
    "1x128" tiles or "1x32" blocks.

    x, residual, h, y, ydq bf16 [rows, cols]; weight bf16 or float32 [cols];
    q uint8 / float8_e4m3fn [rows, cols]; scale float32 [rows, cols/128] or
    uint8 / float8_e8m0fnu [rows, cols/32]; rstd float32 [rows].  h is
    required with a residual (and may be x or residual itself); y (bf16 of
    the normed rows), ydq (the fake-quant values) and rstd are written if
    given."""
    where = "fp8_rmsnorm_quantize"
    block = _choice(where, "kind", kind, _BLOCKS)
    shape = _dims(where, "x", x, 2)
    rows, cols = shape
    dev = x.get_device()
    px = _need(where, "x", x, (_BF,), shape, dev)
    pw = _need(where, "weight", weight, _FLOATS, (cols,), dev)
    pq = _need(where, "q", q, _CODES, shape, dev)
    if block == 0:
        ps = _need(where, "scale", scale, _E8M0, (rows, cols // 32), dev)
    else:
        ps = _need(where, "scale", scale, (_F32,), (rows, cols // 128), dev)
    _run(where, dev, stream, _lib().fp8_rmsnorm_quantize, px, _may(where, "residual", residual, (_BF,), shape, dev), pw,
         _is_f32(weight), rows, cols, eps, block, _choice(where, "rule", rule, _RULES), pq, ps,
         _may(where, "h", h, (_BF,), shape, dev), _may(where, "y", y, (_BF,), shape, dev),
         _may(where, "ydq", ydq, (_BF,), shape, dev), _may(where, "rstd", rstd, (_F32,), (rows,), dev))


def fp8_rmsnorm_backward_workspace(rows, cols):
    """Workspace bytes fp8_rmsnorm_backward needs for these sizes."""
    out = ctypes.c_size_t(0)
    status = _lib().fp8_rmsnorm_backward_workspace(rows, cols, ctypes.byref(out))
    if status:
        _raise(status, "fp8_rmsnorm_backward_workspace")
    return out.value


def fp8_rmsnorm_backward(dy, h, weight, rstd, workspace, dx, dweight, dres=None, stream=None):
    """Gradients of y = h * rstd * weight, straight through the quantization.

    dy, h, dres, dx bf16 [rows, cols]; weight and dweight [cols], both bf16
    or both float32; rstd float32 [rows] of the forward call; workspace of
    fp8_rmsnorm_backward_workspace(rows, cols) bytes.  dres (the gradient
    that reaches h past the norm) is added to dx, which is the gradient of x
    and of the residual."""
    where = "fp8_rmsnorm_backward"
    shape = _dims(where, "dy", dy, 2)
    rows, cols = shape
    dev = dy.get_device()
    pdy = _need(where, "dy", dy, (_BF,), shape, dev)
    pw = _need(where, "weight", weight, _FLOATS, (cols,), dev)
    ws, ws_bytes = _workspace(where, workspace, dev)
    _run(where, dev, stream, _lib().fp8_rmsnorm_backward, pdy, _need(where, "h", h, (_BF,), shape, dev), pw,
         _is_f32(weight), _need(where, "rstd", rstd, (_F32,), (rows,), dev),
         _may(where, "dres", dres, (_BF,), shape, dev), rows, cols,
         ws, ws_bytes, _need(where, "dx", dx, (_BF,), shape, dev),
         _need(where, "dweight", dweight, (weight.dtype,), (cols,), dev))


def fp8_moe_route(logits, ids, weights, bias=None, score="softmax", groups=1, topk_groups=1, group_score="max",
                  renorm=False, scale=1.0, stream=None):
    """The top_k experts of every token (highest key first, ties to the
    lowest index) and their weights.

    logits bf16 or float32 [tokens, experts]; ids int32 and weights float32
    [tokens, top_k] outputs; bias float32 [experts], added to the scores for
    the ranking only; score "softmax" or "sigmoid"; the experts of the
    ``topk_groups`` best of ``groups`` groups are ranked, groups by their
    best key ("max") or their two best keys' sum ("top2"); renorm divides the
    weights by their sum; scale multiplies them.  Logits of -inf or NaN mask
    an expert; places without an expert get id -1 and weight 0."""
    where = "fp8_moe_route"
    tokens, experts = _dims(where, "logits", logits, 2)
    shape = _dims(where, "ids", ids, 2)
    dev = logits.get_device()
    pl = _need(where, "logits", logits, _FLOATS, (tokens, experts), dev)
    if shape[0] != tokens:
        raise ValueError(f"{where}: ids has shape {tuple(shape)}, expected ({tokens}, top_k)")
    _run(where, dev, stream, _lib().fp8_moe_route, pl, _is_f32(logits),
         _may(where, "bias", bias, (_F32,), (experts,), dev), tokens, experts, shape[1],
         _choice(where, "score", score, _SCORES), groups, topk_groups,
         _choice(where, "group_score", group_score, _GROUP_SCORES), 1 if renorm else 0, scale,
         _need(where, "ids", ids, (_I32,), shape, dev), _need(where, "weights", weights, (_F32,), shape, dev))


def fp8_moe_route_backward(logits, ids, dweights, dlogits, score="softmax", renorm=False, scale=1.0, stream=None):
    """Gradient of fp8_moe_route's weights with respect to the logits.

    logits as there; ids its output; dweights float32 [tokens, top_k];
    dlogits [tokens, experts] output of the logits' type."""
    where = "fp8_moe_route_backward"
    tokens, experts = _dims(where, "logits", logits, 2)
    shape = _dims(where, "ids", ids, 2)
    dev = logits.get_device()
    pl = _need(where, "logits", logits, _FLOATS, (tokens, experts), dev)
    if shape[0] != tokens:
        raise ValueError(f"{where}: ids has shape {tuple(shape)}, expected ({tokens}, top_k)")
    _run(where, dev, stream, _lib().fp8_moe_route_backward, pl, _is_f32(logits),
         _need(where, "ids", ids, (_I32,), shape, dev), _need(where, "dweights", dweights, (_F32,), shape, dev),
         tokens, experts, shape[1], _choice(where, "score", score, _SCORES), 1 if renorm else 0, scale,
         _need(where, "dlogits", dlogits, (logits.dtype,), (tokens, experts), dev))


def fp8_moe_plan_workspace(tokens, top_k, experts):
    """Workspace bytes fp8_moe_plan needs for these sizes (0 for a few tokens)."""
    out = ctypes.c_size_t(0)
    status = _lib().fp8_moe_plan_workspace(tokens, top_k, experts, ctypes.byref(out))
    if status:
        _raise(status, "fp8_moe_plan_workspace")
    return out.value


def fp8_moe_plan(ids, experts, workspace, offsets, row_index, slot, stream=None):
    """Sorts (token, choice) pairs by expert: ids int32 [tokens, top_k] ->
    offsets int32 [experts + 1], row_index int32 [tokens * top_k] (the token
    of each grouped row), slot int32 [tokens, top_k] (the grouped row of each
    pair, -1 where its id is outside [0, experts)).  workspace: at least
    fp8_moe_plan_workspace(tokens, top_k, experts) bytes, None where that is
    0."""
    where = "fp8_moe_plan"
    shape = _dims(where, "ids", ids, 2)
    tokens, top_k = shape
    dev = ids.get_device()
    ws, ws_bytes = _workspace(where, workspace, dev)
    _run(where, dev, stream, _lib().fp8_moe_plan, _need(where, "ids", ids, (_I32,), shape, dev), tokens, top_k, experts,
         ws, ws_bytes, _need(where, "offsets", offsets, (_I32,), (experts + 1,), dev),
         _need(where, "row_index", row_index, (_I32,), (tokens * top_k,), dev),
         _need(where, "slot", slot, (_I32,), shape, dev))


def fp8_nvfp4_matvec(x, q, block_scale, global_scale, rows_per_tensor, y, stream=None):
    """y = x . W^T for NVFP4 W: x bf16 [m, k] (m up to about 32); q uint8
    [n, k/2], block_scale uint8 / float8_e4m3fn [n, k/16], global_scale
    float32 [n / rows_per_tensor] as written by fp8_nvfp4_quantize; y bf16 or
    float32 [m, n]."""
    where = "fp8_nvfp4_matvec"
    m, k = _dims(where, "x", x, 2)
    n = _dims(where, "q", q, 2)[0]
    dev = x.get_device()
    if rows_per_tensor < 1 or n % rows_per_tensor:
        raise ValueError(f"{where}: rows_per_tensor {rows_per_tensor} does not divide n {n}")
    _run(where, dev, stream, _lib().fp8_nvfp4_matvec, _need(where, "x", x, (_BF,), (m, k), dev),
         _need(where, "q", q, (_U8,), (n, k // 2), dev),
         _need(where, "block_scale", block_scale, _CODES, (n, k // 16), dev),
         _need(where, "global_scale", global_scale, (_F32,), (n // rows_per_tensor,), dev), rows_per_tensor, m, n, k,
         _need(where, "y", y, _FLOATS, (m, n), dev), _is_f32(y))


def fp8_nvfp4_grouped_matvec(x, row_index, q, block_scale, global_scale, rows_per_tensor, group_offsets, y,
                             stream=None):
    """fp8_nvfp4_matvec over routed experts: rows [off[g], off[g+1]) of y
    take matrix g of q uint8 [groups, n, k/2] (block_scale [groups, n, k/16],
    global_scale [groups * n / rows_per_tensor]); row i reads
    x[row_index[i]], or x[i] where row_index is None.  group_offsets int32
    [groups + 1] and row_index int32 [total_m] on the device; y [total_m, n]:
    rows behind off[groups] are left as they were."""
    where = "fp8_nvfp4_grouped_matvec"
    x_rows, k = _dims(where, "x", x, 2)
    groups, n, _ = _dims(where, "q", q, 3)
    total_m = _dims(where, "y", y, 2)[0]
    dev = x.get_device()
    if rows_per_tensor < 1 or n % rows_per_tensor:
        raise ValueError(f"{where}: rows_per_tensor {rows_per_tensor} does not divide n {n}")
    if row_index is None and x_rows != total_m:
        raise ValueError(f"{where}: x has {x_rows} rows and y {total_m}: without row_index they must agree")
    _run(where, dev, stream, _lib().fp8_nvfp4_grouped_matvec, _need(where, "x", x, (_BF,), (x_rows, k), dev), x_rows,
         _may(where, "row_index", row_index, (_I32,), (total_m,), dev),
         _need(where, "q", q, (_U8,), (groups, n, k // 2), dev),
         _need(where, "block_scale", block_scale, _CODES, (groups, n, k // 16), dev),
         _need(where, "global_scale", global_scale, (_F32,), (groups * (n // rows_per_tensor),), dev),
         rows_per_tensor, _need(where, "group_offsets", group_offsets, (_I32,), (groups + 1,), dev), groups, total_m,
         n, k, _need(where, "y", y, _FLOATS, (total_m, n), dev), _is_f32(y))


def fp8_moe_combine(rows, slot, weights, y, residual=None, stream=None):
    """y[t] = residual[t] + sum_j weights[t, j] * rows[slot[t, j]]: rows bf16
    or float32 [total_m, n]; slot int32 and weights float32 [tokens, top_k];
    residual bf16 [tokens, n]; y bf16 or float32 [tokens, n] (a bf16 y may be
    residual itself).  Slots outside [0, total_m) take no part."""
    where = "fp8_moe_combine"
    total_m, n = _dims(where, "rows", rows, 2)
    shape = _dims(where, "slot", slot, 2)
    dev = rows.get_device()
    out = (shape[0], n)
    _run(where, dev, stream, _lib().fp8_moe_combine, _need(where, "rows", rows, _FLOATS, (total_m, n), dev),
         _is_f32(rows), total_m, _need(where, "slot", slot, (_I32,), shape, dev),
         _need(where, "weights", weights, (_F32,), shape, dev), _may(where, "residual", residual, (_BF,), out, dev),
         shape[0], shape[1], n, _need(where, "y", y, _FLOATS, out, dev), _is_f32(y))


def fp8_moe_combine_backward(dy, rows, slot, weights, drows, dweights, stream=None):
    """drows[slot[t, j]] = weights[t, j] * dy[t] and dweights[t, j] =
    <dy[t], rows[slot[t, j]]>: dy bf16 or float32 [tokens, n]; drows like
    rows; dweights float32 like weights.  Rows that no slot names are left as
    they were; slots are distinct."""
    where = "fp8_moe_combine_backward"
    total_m, n = _dims(where, "rows", rows, 2)
    shape = _dims(where, "slot", slot, 2)
    dev = rows.get_device()
    _run(where, dev, stream, _lib().fp8_moe_combine_backward,
         _need(where, "dy", dy, _FLOATS, (shape[0], n), dev), _is_f32(dy),
         _need(where, "rows", rows, _FLOATS, (total_m, n), dev), _is_f32(rows), total_m,
         _need(where, "slot", slot, (_I32,), shape, dev), _need(where, "weights", weights, (_F32,), shape, dev),
         shape[0], shape[1], n, _need(where, "drows", drows, (rows.dtype,), (total_m, n), dev),
         _need(where, "dweights", dweights, (_F32,), shape, dev))


def fp8_moe_abi_version():
    return _lib().fp8_moe_abi_version()


# --------------------------------------------- allocating conveniences (torch)

def rmsnorm_quantize(x, weight, eps, residual=None, block="1x128", rule="ceil", normed=False, dequant=False,
                     save_rstd=False, stream=None):
    """Allocate outputs and run fp8_rmsnorm_quantize.  Returns a dict with q
    (float8_e4m3fn), scale, h (x itself without a residual) and, if asked
    for, y (normed), ydq (dequant) and rstd (save_rstd)."""
    rows, cols = _dims("rmsnorm_quantize", "x", x, 2)
    with _allocating(stream, x.device):
        q = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=x.device)
        mx = _choice("rmsnorm_quantize", "block", block, _BLOCKS) == 0
        scale = torch.empty((rows, cols // (32 if mx else 128)), dtype=_U8 if mx else _F32, device=x.device)
        h = torch.empty_like(x) if residual is not None else None
        y = torch.empty_like(x) if normed else None
        ydq = torch.empty_like(x) if dequant else None
        rstd = torch.empty((rows,), dtype=_F32, device=x.device) if save_rstd else None
        fp8_rmsnorm_quantize(x, weight, eps, block, rule, q, scale, residual, h, y, ydq, rstd, stream)
    out = {"q": q, "scale": scale, "h": x if h is None else h}
    out.update({k: v for k, v in (("y", y), ("ydq", ydq), ("rstd", rstd)) if v is not None})
    return out


def rmsnorm_backward(dy, h, weight, rstd, dres=None, workspace=None, stream=None):
    """Allocate (dx, dweight) and, unless given, the workspace, and run
    fp8_rmsnorm_backward."""
    rows, cols = _dims("rmsnorm_backward", "dy", dy, 2)
    with _allocating(stream, dy.device):
        if workspace is None:
            workspace = torch.empty(fp8_rmsnorm_backward_workspace(rows, cols), dtype=_U8, device=dy.device)
        dx = torch.empty_like(dy)
        dweight = torch.empty_like(weight)
        fp8_rmsnorm_backward(dy, h, weight, rstd, workspace, dx, dweight, dres, stream)
    return dx, dweight


def moe_route(logits, top_k, bias=None, score="softmax", groups=1, topk_groups=1, group_score="max", renorm=False,
              scale=1.0, stream=None):
    """Allocate (ids, weights) and run fp8_moe_route."""
    tokens = _dims("moe_route", "logits", logits, 2)[0]
    with _allocating(stream, logits.device):
        ids = torch.empty((tokens, top_k), dtype=_I32, device=logits.device)
        weights = torch.empty((tokens, top_k), dtype=_F32, device=logits.device)
        fp8_moe_route(logits, ids, weights, bias, score, groups, topk_groups, group_score, renorm, scale, stream)
    return ids, weights


def moe_route_backward(logits, ids, dweights, score="softmax", renorm=False, scale=1.0, stream=None):
    """Allocate dlogits and run fp8_moe_route_backward."""
    _dims("moe_route_backward", "logits", logits, 2)
    with _allocating(stream, logits.device):
        dlogits = torch.empty_like(logits)
        fp8_moe_route_backward(logits, ids, dweights, dlogits, score, renorm, scale, stream)
    return dlogits


def moe_plan(ids, experts, stream=None):
    """Allocate (offsets, row_index, slot) and the workspace, and run
    fp8_moe_plan."""
    tokens, top_k = _dims("moe_plan", "ids", ids, 2)
    with _allocating(stream, ids.device):
        size = fp8_moe_plan_workspace(tokens, top_k, experts)
        workspace = torch.empty(size, dtype=_U8, device=ids.device) if size else None
        offsets = torch.empty((experts + 1,), dtype=_I32, device=ids.device)
        row_index = torch.empty((tokens * top_k,), dtype=_I32, device=ids.device)
        slot = torch.empty((tokens, top_k), dtype=_I32, device=ids.device)
        fp8_moe_plan(ids, experts, workspace, offsets, row_index, slot, stream)
    return offsets, row_index, slot


def nvfp4_matvec(x, q, block_scale, global_scale, rows_per_tensor=None, out_dtype=torch.bfloat16, stream=None):
    """Allocate y and run fp8_nvfp4_matvec (one tensor unless
    rows_per_tensor is given)."""
    m = _dims("nvfp4_matvec", "x", x, 2)[0]
    n = _dims("nvfp4_matvec", "q", q, 2)[0]
    with _allocating(stream, x.device):
        y = torch.empty((m, n), dtype=out_dtype, device=x.device)
        fp8_nvfp4_matvec(x, q, block_scale, global_scale, max(n, 1) if rows_per_tensor is None else rows_per_tensor,
                         y, stream)
    return y


def nvfp4_grouped_matvec(x, q, block_scale, global_scale, group_offsets, rows_per_tensor=None, row_index=None,
                         out_dtype=torch.bfloat16, stream=None):
    """Allocate y and run fp8_nvfp4_grouped_matvec (one tensor scale per
    group unless rows_per_tensor is given).  Rows behind off[groups] are
    zero."""
    total_m = _dims("nvfp4_grouped_matvec", "x", x, 2)[0] if row_index is None else row_index.numel()
    n = _dims("nvfp4_grouped_matvec", "q", q, 3)[1]
    with _allocating(stream, x.device):
        y = torch.zeros((total_m, n), dtype=out_dtype, device=x.device)
        fp8_nvfp4_grouped_matvec(x, row_index, q, block_scale, global_scale,
                                 max(n, 1) if rows_per_tensor is None else rows_per_tensor, group_offsets, y, stream)
    return y


def moe_combine(rows, slot, weights, residual=None, out_dtype=torch.bfloat16, stream=None):
    """Allocate y and run fp8_moe_combine."""
    n = _dims("moe_combine", "rows", rows, 2)[1]
    tokens = _dims("moe_combine", "slot", slot, 2)[0]
    with _allocating(stream, rows.device):
        y = torch.empty((tokens, n), dtype=out_dtype, device=rows.device)
        fp8_moe_combine(rows, slot, weights, y, residual, stream)
    return y


def moe_combine_backward(dy, rows, slot, weights, stream=None):
    """Allocate (drows, dweights) and run fp8_moe_combine_backward; rows that
    no slot names get a zero gradient."""
    _dims("moe_combine_backward", "rows", rows, 2)
    with _allocating(stream, rows.device):
        drows = torch.zeros_like(rows)
        dweights = torch.empty_like(weights)
        fp8_moe_combine_backward(dy, rows, slot, weights, drows, dweights, stream)
    return drows, dweights
