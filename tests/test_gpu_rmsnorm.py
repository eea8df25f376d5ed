"""GPU parity of fp8_rmsnorm_quantize / fp8_rmsnorm_backward against the oracle (oracle/moe.py, float64).

Tolerances from the kernels' arithmetic.  The sum of squares of a row of n values is added up in at most
32 + 6 + 16 dependent fp32 additions, each off by at most 2^-24 of sums of positive terms, so rstd (a square root
halves that; a division and a root add one step each) is within 2^-18 of its value, and y = h rstd w, two more
roundings, within D = 2^-17.  From there:
  * codes: rounding is monotone, so a code lies between the codes of the exact quotient times (1 - D) and (1 + D);
  * bf16 outputs add half a step, 2^-8;
  * gradients: dx adds a dot product over the row, off by at most 2^-18 of its terms' magnitudes; dw is a sum over
    the rows in at most 2^8 dependent additions (four rows, or a 256th of them, in a workgroup, then a tree over
    the partials), so within 2^-16 of the magnitudes for the row counts here.
"""

import numpy as np
import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from oracle import moe, quant
from oracle.codec import bf16_to_f32, e4m3_decode, e4m3_encode, f32_to_bf16
from tests.gpu_helpers import assert_bytes_equal, bf16_from_bits
from workloads import bf16_bits

pytestmark = pytest.mark.gpu
D = 2.0 ** -17
EPS = 1e-6


def _f64(bits):
    return bf16_to_f32(bits).astype(np.float64)


def _bits(a):
    return f32_to_bf16(np.asarray(a, dtype=np.float32))


def _values(rng, rows, cols, dist):
    if dist == "normal":
        x = rng.standard_normal((rows, cols))
        x[:, rng.integers(0, cols, max(1, cols // 100))] *= 50
    elif dist == "wide":
        x = np.exp2(rng.uniform(-60, 60, (rows, cols))) * rng.choice([-1, 1], (rows, cols))
    elif dist == "huge":                     # squares beyond the fp32 range
        x = rng.standard_normal((rows, cols)) * 1e30
    else:                                    # "tiny": eps carries the norm, zero rows and zero tiles among them
        x = rng.standard_normal((rows, cols)) * 1e-30
        x[0] = 0.0
        x[:, : min(cols, 128)] = 0.0
    return _bits(x)


def _check_codes(q, scale_val, y, what):
    """Codes against the exact quotients; scale_val per element."""
    with np.errstate(divide="ignore", invalid="ignore"):
        v = np.where(scale_val > 0, y / scale_val, 0.0 * y)
    a, b = e4m3_decode(e4m3_encode(v * (1 - D))), e4m3_decode(e4m3_encode(v * (1 + D)))
    got = e4m3_decode(q)
    bad = np.argwhere((got < np.minimum(a, b)) | (got > np.maximum(a, b)))
    assert len(bad) == 0, (what, len(bad), bad[0], got[tuple(bad[0])], v[tuple(bad[0])])


def _run(xb, rb, w, block, rule="ceil", eps=EPS, inplace=False):
    rows, cols = xb.shape
    x = bf16_from_bits(xb)
    res = None if rb is None else bf16_from_bits(rb)
    n = 32 if block == "1x32" else 128
    q = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.empty((rows, cols // n), dtype=torch.uint8 if n == 32 else torch.float32, device="cuda")
    h = None if rb is None else (res if inplace else torch.empty_like(x))
    y, ydq = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(rows, dtype=torch.float32, device="cuda")
    fb.fp8_rmsnorm_quantize(x, w, eps, block, rule, q, scale, res, h, y, ydq, rstd)
    torch.cuda.synchronize()
    return (q.cpu().numpy(), scale.cpu().numpy(), xb if h is None else bf16_bits(h), bf16_bits(y), bf16_bits(ydq),
            rstd.cpu().numpy())


def _weight(rng, cols, dtype):
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(cols)).astype(np.float32)).to(dtype)
    return w.cuda(), w.double().numpy()


def _check(xb, rb, wdtype, block, rule, seed, eps=EPS, inplace=False):
    rng = np.random.default_rng(seed)
    rows, cols = xb.shape
    w, w64 = _weight(rng, cols, wdtype)
    q, scale, h, yb, ydq, rstd = _run(xb, rb, w, block, rule, eps, inplace)
    hb = xb if rb is None else moe.add_residual(xb, rb)
    assert_bytes_equal(h, hb, "h")
    y, r = moe.rmsnorm(_f64(hb), w64, eps)
    assert np.all(np.abs(rstd - r) <= 2.0 ** -18 * r + 1e-45), "rstd"
    assert np.all(np.abs(_f64(yb) - y) <= (2.0 ** -8 + D) * np.abs(y) + 2.0 ** -133), "y"
    n = 32 if block == "1x32" else 128
    amax = np.abs(y).reshape(rows, cols // n, n).max(-1)
    if block == "1x32":
        lo, hi = quant.e8m0_exponent(amax * (1 - D), rule), quant.e8m0_exponent(amax * (1 + D), rule)
        X = scale.astype(np.int64) - 127
        assert np.all((X == lo) | (X == hi)), "E8M0 scale"
        sv = np.exp2(X.astype(np.float64))
    else:
        assert np.all(np.abs(scale - amax / 448) <= 2 * D * amax / 448 + 2.0 ** -149), "fp32 scale"
        sv = scale.astype(np.float64)
    tiny = np.repeat(sv < 2.0 ** -126 if block == "1x128" else np.zeros_like(sv, bool), n, axis=1)
    per = np.repeat(sv, n, axis=1)
    # an fp32 scale below the normal range has few bits: there only the code's sign is fixed by this check
    _check_codes(np.where(tiny, 0, q), per, np.where(tiny, 0.0, y), f"codes {block}")
    assert_bytes_equal(ydq, quant.dequantize(q, scale, block), "ydq")


@pytest.mark.parametrize("block,rule", [("1x128", "ceil"), ("1x32", "ceil"), ("1x32", "floor")])
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (1, 7168), (37, 1152), (5, 8192), (2, 16384), (2, 32768),
                                       (300, 384)])
def test_forward_shapes(rows, cols, block, rule):
    print(f"[rmsnorm] {rows}x{cols} {block} {rule}", flush=True)
    rng = np.random.default_rng(rows + cols)
    x, r = _values(rng, rows, cols, "normal"), _bits(4 * rng.standard_normal((rows, cols)))
    _check(x, r, torch.float32, block, rule, 1)
    _check(x, None, torch.bfloat16, block, rule, 2)


@pytest.mark.parametrize("cols", [32, 96, 5152, 8224, 32736])
def test_forward_odd_blocks(cols):
    print(f"[rmsnorm] 1x32, {cols} columns", flush=True)
    rng = np.random.default_rng(cols)
    _check(_values(rng, 5, cols, "normal"), None, torch.bfloat16, "1x32", "ceil", 3)


@pytest.mark.parametrize("dist", ["wide", "huge", "tiny"])
@pytest.mark.parametrize("block", ["1x128", "1x32"])
def test_forward_ranges(dist, block):
    print(f"[rmsnorm] {dist} {block}", flush=True)
    rng = np.random.default_rng(7)
    x = _values(rng, 9, 1024, dist)
    _check(x, None, torch.float32, block, "ceil", 4)
    if dist != "huge":
        _check(x, _values(rng, 9, 1024, dist), torch.float32, block, "ceil", 5, eps=1e-20 if dist == "wide" else EPS)


def test_h_written_over_the_residual():
    rng = np.random.default_rng(8)
    _check(_values(rng, 33, 2048, "normal"), _values(rng, 33, 2048, "normal"), torch.float32, "1x128", "ceil", 6,
           inplace=True)


def test_h_written_over_x():
    rng = np.random.default_rng(18)
    xb, rb = _values(rng, 17, 1152, "normal"), _values(rng, 17, 1152, "normal")
    x, r = bf16_from_bits(xb), bf16_from_bits(rb)
    w = torch.ones(1152, device="cuda")
    want = fb.rmsnorm_quantize(x, w, EPS, residual=r)
    q, s = torch.empty_like(want["q"]), torch.empty_like(want["scale"])
    fb.fp8_rmsnorm_quantize(x, w, EPS, "1x128", "ceil", q, s, residual=r, h=x)
    assert torch.equal(x, want["h"]) and torch.equal(q.view(torch.uint8), want["q"].view(torch.uint8))
    assert torch.equal(s, want["scale"])


@pytest.mark.parametrize("over", ["dy", "dres"])
@pytest.mark.parametrize("rows,cols", [(700, 1152), (300, 12288), (300, 20480), (6000, 7168)])
def test_dx_written_over_an_input(over, rows, cols):
    g = torch.Generator("cuda").manual_seed(rows + cols)
    h, dy, dres = (torch.randn((rows, cols), device="cuda", generator=g).to(torch.bfloat16) for _ in range(3))
    w, r = torch.rand(cols, device="cuda", generator=g), torch.rand(rows, device="cuda", generator=g)
    want, dw = fb.rmsnorm_backward(dy, h, w, r, dres=dres)
    ws = torch.empty(fb.fp8_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dx, dw2 = dy if over == "dy" else dres, torch.empty_like(dw)
    fb.fp8_rmsnorm_backward(dy, h, w, r, ws, dx, dw2, dres=dres)
    assert torch.equal(dx, want) and torch.equal(dw, dw2)


def test_rows_beyond_32_bit_offsets():
    rows, cols = 262144 + 3, 16384
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, cols), device="cuda").to(torch.bfloat16)
    w = torch.ones(cols, device="cuda")
    whole = fb.rmsnorm_quantize(x, w, EPS, save_rstd=True)
    tail = fb.rmsnorm_quantize(x[-3:].contiguous(), w, EPS, save_rstd=True)
    assert torch.equal(whole["q"][-3:].view(torch.uint8), tail["q"].view(torch.uint8))
    assert torch.equal(whole["scale"][-3:], tail["scale"]) and torch.equal(whole["rstd"][-3:], tail["rstd"])
    dx, dw = fb.rmsnorm_backward(x, x, w, whole["rstd"])
    dx2, dw2 = fb.rmsnorm_backward(x[-3:].contiguous(), x[-3:].contiguous(), w, tail["rstd"])
    assert torch.equal(dx[-3:], dx2)
    assert torch.all((dw - dw2).abs() <= 2.0 ** -22 * dw2.abs())          # three rows, added in another order


@pytest.mark.parametrize("block", ["1x32", "1x128"])
@pytest.mark.parametrize("cols", [1152, 7168, 16384, 20480])
def test_a_large_call_is_its_small_ones(block, cols):
    """Calls past the size of the last cache (nontemporal) against the same rows in calls below it."""
    rows = 80_000_000 // cols + 3
    g = torch.Generator("cuda").manual_seed(cols)
    x, r = (torch.randn((rows, cols), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    w = torch.rand(cols, device="cuda", generator=g) + 0.5
    whole = fb.rmsnorm_quantize(x, w, EPS, residual=r, block=block, normed=True, dequant=True, save_rstd=True)
    dx, dw = fb.rmsnorm_backward(r, whole["h"], w, whole["rstd"], dres=x)
    total, mag = torch.zeros_like(w).double(), torch.zeros_like(w).double()
    step = rows // 8
    for t in range(0, rows, step):
        cut = slice(t, min(t + step, rows))
        one = fb.rmsnorm_quantize(x[cut].contiguous(), w, EPS, residual=r[cut].contiguous(), block=block, normed=True,
                                  dequant=True, save_rstd=True)
        for name, v in one.items():
            assert torch.equal(whole[name][cut].view(torch.uint8), v.view(torch.uint8)), name
        dxc, dwc = fb.rmsnorm_backward(r[cut].contiguous(), one["h"], w, one["rstd"], dres=x[cut].contiguous())
        assert torch.equal(dx[cut], dxc)
        total += dwc.double()
        mag += (r[cut].float() * one["h"].float() * one["rstd"][:, None]).abs().sum(0, dtype=torch.float64)
    assert torch.all((dw.double() - total).abs() <= 2.0 ** -14 * mag)     # both sums of up to 2^9 additions


def test_same_bytes_every_time():
    rng = np.random.default_rng(19)
    h, dy = (bf16_from_bits(_values(rng, 3000, 1152, "normal")) for _ in range(2))
    w, r = torch.ones(1152, device="cuda"), torch.rand(3000, device="cuda")
    first = fb.rmsnorm_backward(dy, h, w, r)
    for _ in range(5):
        again = fb.rmsnorm_backward(dy, h, w, r)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1].view(torch.int32), again[1].view(torch.int32))


def test_more_rows_than_workgroups():
    """Rows past the launch's largest grid are taken by the same workgroups."""
    rows, cols = (1 << 20) + 3, 128
    x = torch.randn((rows, cols), device="cuda", generator=torch.Generator("cuda").manual_seed(5)).to(torch.bfloat16)
    w = torch.ones(cols, dtype=torch.float32, device="cuda")
    whole = fb.rmsnorm_quantize(x, w, EPS, normed=True)
    tail = fb.rmsnorm_quantize(x[1 << 20:].contiguous(), w, EPS, normed=True)
    for k in ("q", "scale", "y"):
        assert torch.equal(whole[k][1 << 20:].view(torch.uint8), tail[k].view(torch.uint8)), k


def _grad_check(rows, cols, wdtype, dres, seed, inplace=None):
    rng = np.random.default_rng(seed)
    hb = _values(rng, rows, cols, "normal")
    dyb = _bits(1e-3 * rng.standard_normal((rows, cols)))
    drb = _bits(1e-3 * rng.standard_normal((rows, cols))) if dres else None
    w, w64 = _weight(rng, cols, wdtype)
    h, dy = bf16_from_bits(hb), bf16_from_bits(dyb)
    dr = None if drb is None else bf16_from_bits(drb)
    rstd = torch.from_numpy((1 / np.sqrt((_f64(hb) ** 2).mean(1) + EPS)).astype(np.float32)).cuda()
    ws = torch.empty(fb.fp8_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda").fill_(0xFF)
    dx = {None: torch.empty_like(h), "dy": dy, "dres": dr}[inplace]
    dw = torch.empty_like(w)
    fb.fp8_rmsnorm_backward(dy, h, w, rstd, ws, dx, dw, dres=dr)
    torch.cuda.synchronize()
    dy64, h64, r64 = _f64(dyb), _f64(hb), rstd.double().cpu().numpy()
    want, wantw = moe.rmsnorm_backward(dy64, h64, w64, r64, None if drb is None else _f64(drb))
    xh, wd = np.abs(h64 * r64[:, None]), np.abs(dy64 * w64)
    mag = r64[:, None] * (wd + xh * (wd * xh).mean(1)[:, None]) + (0 if drb is None else np.abs(_f64(drb)))
    assert np.all(np.abs(_f64(bf16_bits(dx)) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * mag), "dx"
    magw = (np.abs(dy64) * xh).sum(0)
    tol = 2.0 ** -16 * magw + (2.0 ** -8 * np.abs(wantw) if wdtype == torch.bfloat16 else 0)
    assert np.all(np.abs(dw.double().cpu().numpy() - wantw) <= tol), "dw"


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 128), (7, 40), (513, 1152), (1300, 256), (3, 7168), (2, 32768)])
@pytest.mark.parametrize("wdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dres", [False, True])
def test_backward(rows, cols, wdtype, dres):
    print(f"[rmsnorm backward] {rows}x{cols} {wdtype} dres={dres}", flush=True)
    _grad_check(rows, cols, wdtype, dres, rows + cols)


@pytest.mark.parametrize("over", ["dy", "dres"])
def test_backward_over_its_input(over):
    _grad_check(70, 1024, torch.float32, True, 11, inplace=over)


def test_backward_of_no_rows_writes_zeros():
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    dw = torch.full_like(w, 3.0)
    fb.fp8_rmsnorm_backward(none, none, w, torch.empty(0, device="cuda"), None, none.clone(), dw)
    assert torch.all(dw == 0)


def test_backward_against_differences_of_the_kernel():
    """The kernel's own forward, differenced along a direction: y (bf16 out) carries half a step 2^-8 of each
    term, so the directional derivative of sum(dy y) is known to 2 * 2^-8 * sum|dy y| / step."""
    rng = np.random.default_rng(12)
    rows, cols, step = 4, 256, 0.25
    h = _bits(rng.standard_normal((rows, cols)))
    v = rng.choice([-1.0, 1.0], (rows, cols))
    dyb = _bits(rng.standard_normal((rows, cols)))
    w, _ = _weight(rng, cols, torch.float32)
    up, dn = _bits(_f64(h) + step * v), _bits(_f64(h) - step * v)
    dy = _f64(dyb)
    ys = [_f64(_run(b, None, w, "1x128")[3]) for b in (up, dn)]
    moved = _f64(up) - _f64(dn)                                  # what the rounded inputs moved by
    got = (dy * (ys[0] - ys[1])).sum()
    out = fb.rmsnorm_quantize(bf16_from_bits(h), w, EPS, save_rstd=True)
    dx, _ = fb.rmsnorm_backward(bf16_from_bits(dyb), bf16_from_bits(h), w, out["rstd"])
    # the differences' own error: y's rounding, and the third derivative along the step (measured in float64)
    w64 = w.double().cpu().numpy()
    f = [(dy * moe.rmsnorm(_f64(b), w64, EPS)[0]).sum() for b in (up, dn)]
    curve = abs((f[0] - f[1]) - (moe.rmsnorm_backward(dy, _f64(h), w64, moe.rmsnorm(_f64(h), w64, EPS)[1])[0]
                                 * moved).sum())
    tol = 2.0 ** -8 * (np.abs(dy) * (np.abs(ys[0]) + np.abs(ys[1]))).sum() + curve
    dxf = _f64(bf16_bits(dx))
    assert abs(got - (dxf * moved).sum()) <= tol + 2.0 ** -8 * np.abs(dxf * moved).sum()


# The largest rows: rstd is below the normal range there, where its own rounding is half a step of 2^-149, at most
# 2^-22 of 1 / 2^128, within the 2^-18 that rstd is checked to and the D of y.
@pytest.mark.parametrize("block", ["1x128", "1x32"])
@pytest.mark.parametrize("cols", [128, 1152, 7168, 32768])
@pytest.mark.parametrize("size", [1e36, 1e37, 1e38, 3.38e38])
def test_forward_of_rows_up_to_the_largest_value(size, cols, block):
    print(f"[rmsnorm] rows of {size}, {cols} columns, {block}", flush=True)
    rng = np.random.default_rng(cols)
    x = rng.uniform(0.5, 1, (4, cols)) * size * rng.choice([-1, 1], (4, cols))
    x[0] = size                                  # no smaller element
    x[1, 1:] *= 1e-30                            # one large element among small ones
    _check(_bits(x), None, torch.float32, block, "ceil", 21)
    half = _bits(x / 2)
    _check(half, half, torch.bfloat16, block, "ceil", 22)


@pytest.mark.parametrize("cols", [32, 96])
@pytest.mark.parametrize("size", [1e36, 7e37, 3.38e38])
def test_forward_of_narrow_rows_up_to_the_largest_value(size, cols):
    x = np.full((3, cols), size) * np.random.default_rng(cols).choice([-1, 1], (3, cols))
    _check(_bits(x), None, torch.float32, "1x32", "floor", 23)


@pytest.mark.parametrize("cols", [128, 7168])
def test_forward_where_the_sum_of_squares_leaves_the_fp32_range(cols):
    """Rows whose sum of squares is just below and just above 2^128, with an eps that does not count and ones that
    do."""
    edge = 2.0 ** 64 / np.sqrt(cols)
    x = np.stack([np.full(cols, f * edge) for f in (0.5, 0.98, 0.995, 1.0, 1.005, 1.02, 1.5, 2.0)])
    for eps in (1e-6, 1e30, 1e38):
        _check(_bits(x), None, torch.float32, "1x128", "ceil", 24, eps=eps)


@pytest.mark.parametrize("rows,cols", [(5, 128), (300, 7168), (3, 32768)])
@pytest.mark.parametrize("size", [1e37, 3.38e38])
def test_backward_of_rows_up_to_the_largest_value(size, rows, cols):
    """With the rstd of the forward call, which is below the normal range."""
    rng = np.random.default_rng(rows)
    hb = _bits(rng.uniform(0.5, 1, (rows, cols)) * size * rng.choice([-1, 1], (rows, cols)))
    dyb = _bits(1e30 * rng.standard_normal((rows, cols)))
    w, w64 = _weight(rng, cols, torch.float32)
    h, dy = bf16_from_bits(hb), bf16_from_bits(dyb)
    rstd = fb.rmsnorm_quantize(h, w, EPS, save_rstd=True)["rstd"]
    dx, dw = fb.rmsnorm_backward(dy, h, w, rstd)
    dy64, h64, r64 = _f64(dyb), _f64(hb), rstd.double().cpu().numpy()
    assert np.all(np.abs(r64 * np.sqrt((h64 ** 2).mean(1)) - 1) <= 2.0 ** -18)
    want, wantw = moe.rmsnorm_backward(dy64, h64, w64, r64)
    xh, wd = np.abs(h64 * r64[:, None]), np.abs(dy64 * w64)
    mag = r64[:, None] * (wd + xh * (wd * xh).mean(1)[:, None])
    assert np.all(np.abs(_f64(bf16_bits(dx)) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * mag), "dx"
    assert np.all(np.abs(dw.double().cpu().numpy() - wantw) <= 2.0 ** -16 * (np.abs(dy64) * xh).sum(0)), "dw"


@pytest.mark.parametrize("cols", [128, 7168])
def test_forward_where_the_mean_and_eps_leave_the_fp32_range(cols):
    """Their sum can where the sum of squares does not: eps is any finite value."""
    rng = np.random.default_rng(25)
    sign, top = rng.choice([-1, 1], (4, cols)), 0.999 * 2.0 ** 64 / np.sqrt(cols)
    rows = [_bits(top * sign), _bits(1.001 * top * sign), _bits(1e15 * rng.standard_normal((4, cols))),
            _bits(3e38 * sign)]
    for eps in (3.3e38, 3.4028234e38):
        for x in rows:
            _check(x, None, torch.float32, "1x128", "ceil", 27, eps=eps)


@pytest.mark.parametrize("wdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block,rule", [("1x128", "ceil"), ("1x32", "ceil"), ("1x32", "floor")])
def test_forward_of_values_below_the_normal_range(block, rule, wdtype):
    """Tiles of y from 1e-35 down to zeros: fp32 scales with few bits or none, E8M0 scales at their least.  y itself
    is rounded to a multiple of 2^-149 there, at most half of that off besides D, and so is an fp32 scale; a code
    lies between those of the quotients at both ends of y, by the scale that was stored, and has y's sign.  Where
    that scale is 0 the code is 0."""
    rng = np.random.default_rng(31)
    rows, cols, n = 7, 2048, 32 if block == "1x32" else 128
    xb = _values(rng, rows, cols, "normal")
    size = np.repeat(10.0 ** -np.arange(35, 35 + cols // 128, dtype=np.float64), 128)
    w = torch.from_numpy((size * rng.uniform(0.5, 1, cols) * rng.choice([-1, 1], cols)).astype(np.float32)).to(wdtype)
    w64 = w.double().numpy()
    q, scale, _, yb, ydq, rstd = _run(xb, None, w.cuda(), block, rule)
    y, r = moe.rmsnorm(_f64(xb), w64, EPS)
    half = 2.0 ** -150
    assert np.all(np.abs(rstd - r) <= 2.0 ** -18 * r)
    assert np.all(np.abs(_f64(yb) - y) <= (2.0 ** -8 + D) * np.abs(y) + half + 2.0 ** -134), "y"
    amax = np.abs(y).reshape(rows, cols // n, n).max(-1)
    if block == "1x32":
        lo, hi = (quant.e8m0_exponent(amax * (1 + s * D) + s * half, rule) for s in (-1, 1))
        X = scale.astype(np.int64) - 127
        assert np.all((X == lo) | (X == hi)) and np.any(X == -127)
        sv = np.exp2(X.astype(np.float64))
    else:
        assert np.all(np.abs(scale - amax / 448) <= (2 * D * amax + half) / 448 + half), "fp32 scale"
        assert np.any(scale == 0) and np.any((scale > 0) & (scale < 2.0 ** -126))
        sv = scale.astype(np.float64)
    per = np.repeat(sv, n, axis=1)
    mag, got = np.abs(y), np.abs(e4m3_decode(q).astype(np.float64))
    zero = per == 0
    by = np.where(zero, 1.0, per)
    least = e4m3_decode(e4m3_encode(np.maximum(mag * (1 - D) - half, 0) / by))
    most = e4m3_decode(e4m3_encode((mag * (1 + D) + half) / by))
    bad = np.argwhere(~zero & ((got < least) | (got > most)))
    assert len(bad) == 0, (len(bad), bad[0], q[tuple(bad[0])], y[tuple(bad[0])], per[tuple(bad[0])])
    assert np.all(got[zero] == 0)
    assert np.array_equal(q >= 0x80, np.signbit(y)), "signs"
    assert_bytes_equal(ydq, quant.dequantize(q, scale, block), "ydq")
