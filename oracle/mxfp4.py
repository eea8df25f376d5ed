"""MXFP4 codec, products and the experts' gradients (oracle).

TEST INFRASTRUCTURE ONLY (see the package docstring).

E2M1 elements (as NVFP4's) with an E8M0 scale per 32 consecutive elements of
a row: the microscaled format of [prequant] "Formats" with 4-bit elements.
  * CEIL: the smallest integer X with amax <= 6 * 2^X; FLOOR: floor(log2
    amax) - 2; clamped to [-127, 127], -127 for an all-zero block.
  * code = e2m1(x * 2^-X), value e2m1(code) * 2^X.
Products and gradients are evaluated in float64 on the decoded values.
"""

import numpy as np

from .codec import bf16_to_f32, e4m3_decode, f32_to_bf16
from .nvfp4 import e2m1_decode, e2m1_encode, pack, unpack

BLOCK = 32


def exponent(amax, rule):
    """E8M0 exponent X of each non-negative amax (float64)."""
    amax = np.asarray(amax, dtype=np.float64)
    m, e = np.frexp(np.where(amax > 0, amax, 1.0))       # amax = m 2^e, m in [1/2, 1)
    if rule == "floor":
        x = e - 1 - 2
    else:                                                # amax <= 6 2^X: 2^X >= m 2^e / 6, 6 = 0.75 2^3
        x = np.where(m <= 0.75, e - 3, e - 2)
    return np.where(amax > 0, np.clip(x, -127, 127), -127).astype(np.int64)


def quantize(x_bits, rule="ceil"):
    """bf16 bits [R, C] -> (packed codes [R, C/2], E8M0 bytes [R, C/32], fake-quant bf16 bits [R, C])."""
    x = bf16_to_f32(x_bits).astype(np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // BLOCK, BLOCK)
    e = exponent(np.abs(b).max(-1) if cols else np.zeros((rows, 0)), rule)
    codes = e2m1_encode(np.ldexp(b, -e[..., None])).reshape(rows, cols)
    q, s = pack(codes), (e + 127).astype(np.uint8)
    return q, s, dequantize(q, s)


def matrix(q, s):
    """Values (float64) of packed codes [..., C/2] with E8M0 bytes [..., C/32]; byte 255 is NaN."""
    lead = q.shape[:-1]
    v = e2m1_decode(unpack(q.reshape(-1, q.shape[-1]))).reshape(*lead, s.shape[-1], BLOCK)
    sv = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return (v * sv[..., None]).reshape(*lead, 2 * q.shape[-1])


def matrix8(q, s):
    """The same for E4M3 codes [..., C]."""
    sv = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    v = e4m3_decode(q).astype(np.float64).reshape(*s.shape, BLOCK)
    return (v * sv[..., None]).reshape(q.shape)


def dequantize(q, s):
    with np.errstate(over="ignore"):
        return f32_to_bf16(matrix(q, s).astype(np.float32))


def spans(offsets, total_m):
    """(group, first row, end) of every group, clamped as the library does."""
    out = []
    for g in range(len(offsets) - 1):
        lo = min(max(int(offsets[g]), 0), total_m)
        out.append((g, lo, min(max(int(offsets[g + 1]), lo), total_m)))
    return out


def grouped(x, w, offsets, row_index=None, keep=None):
    """y[rows of g] = x[row_index] . w[g]^T (float64); other rows are ``keep``'s, or zeros."""
    total = len(x) if row_index is None else len(row_index)
    y = np.zeros((total, w.shape[1])) if keep is None else np.array(keep, np.float64)
    for g, lo, hi in spans(offsets, total):
        at = np.arange(lo, hi) if row_index is None else np.clip(row_index[lo:hi], 0, len(x) - 1)
        y[lo:hi] = x[at] @ w[g].T
    return y


def dgrad(dy, w, offsets, keep=None):
    """dx[rows of g] = dy . w[g] (float64); other rows are ``keep``'s, or zeros."""
    dx = np.zeros((len(dy), w.shape[2])) if keep is None else np.array(keep, np.float64)
    for g, lo, hi in spans(offsets, len(dy)):
        dx[lo:hi] = dy[lo:hi] @ w[g]
    return dx


def wgrad(dy, x, offsets, row_index=None):
    """dw[g] = dy[rows of g]^T . x[rows of g] (float64)."""
    dw = np.zeros((len(offsets) - 1, dy.shape[1], x.shape[1]))
    for g, lo, hi in spans(offsets, len(dy)):
        at = np.arange(lo, hi) if row_index is None else np.clip(row_index[lo:hi], 0, len(x) - 1)
        dw[g] = dy[lo:hi].T @ x[at]
    return dw
