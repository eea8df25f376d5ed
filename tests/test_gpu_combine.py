"""GPU parity of fp8_moe_combine / fp8_moe_combine_backward against the oracle (oracle/moe.py, float64).

An fp32 sum of k weighted rows and a residual is off by at most (k + 1) 2^-24 of the terms' magnitudes, a bf16 output
adds 2^-8 of the value; drows is one product (2^-24, or 2^-8 in bf16); a dot product over n columns in fp32 is off
by at most n 2^-24 of the magnitudes in any order.
"""

import numpy as np
import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from oracle import moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _t(a, dtype):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(dtype).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _slots(rng, tokens, top_k, total):
    s = rng.permutation(max(total, tokens * top_k))[: tokens * top_k].reshape(tokens, top_k).astype(np.int32)
    s[s >= total] = -1
    return s


SHAPES = [(1, 1, 8, 1), (1, 8, 7168, 8), (5, 2, 40, 12), (33, 8, 256, 200), (3, 64, 1024, 192), (2, 3, 32768, 6),
          (7, 4, 2056, 0), (260, 6, 128, 1560)]


@pytest.mark.parametrize("tokens,top_k,n,total", SHAPES)
@pytest.mark.parametrize("row_dtype", [BF, F32])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_combine(tokens, top_k, n, total, row_dtype, out_dtype, residual):
    print(f"[combine] {tokens} tokens, {top_k} of {total} rows of {n}, {row_dtype} {out_dtype} res={residual}",
          flush=True)
    rng = np.random.default_rng(tokens + n)
    rows = _t(rng.standard_normal((total, n)), row_dtype)
    slot, w = _slots(rng, tokens, top_k, total), rng.uniform(-1, 1, (tokens, top_k)).astype(np.float32)
    res = _t(4 * rng.standard_normal((tokens, n)), BF) if residual else None
    y = torch.full((tokens, n), 9.0, dtype=out_dtype, device="cuda")
    fb.fp8_moe_combine(rows, torch.from_numpy(slot).cuda(), torch.from_numpy(w).cuda(), y, residual=res)
    r64, s64 = _np(rows), None if res is None else _np(res)
    want = moe.combine(r64, slot, w, s64)
    mag = moe.combine(np.abs(r64), slot, np.abs(w), None if s64 is None else np.abs(s64))
    tol = (top_k + 1) * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(want) if out_dtype == BF else 0)
    assert np.all(np.abs(_np(y) - want) <= tol)


def test_combine_over_the_residual_and_of_left_out_pairs():
    rng = np.random.default_rng(3)
    rows = _t(rng.standard_normal((6, 64)), BF)
    rows[5] = float("nan")                                       # a row no slot names
    slot = np.array([[0, 1], [-1, -1], [6, 2], [np.iinfo(np.int32).min, np.iinfo(np.int32).max]], dtype=np.int32)
    w = np.array([[1, 2], [np.nan, np.inf], [np.nan, 0.5], [np.nan, np.nan]], dtype=np.float32)
    res = _t(rng.standard_normal((4, 64)), BF)
    keep = res.clone()
    fb.fp8_moe_combine(rows, torch.from_numpy(slot).cuda(), torch.from_numpy(w).cuda(), res, residual=res)
    assert torch.equal(res[1], keep[1]) and torch.equal(res[3], keep[3])
    want = moe.combine(_np(rows[:5]), np.where(slot < 5, slot, -1), np.nan_to_num(w), _np(keep))
    assert np.all(np.abs(_np(res) - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -20)


def test_same_row_for_two_tokens():
    """Reading a row twice is fine (a row shared by tokens)."""
    rows = _t(np.arange(32).reshape(2, 16), BF)
    slot = torch.tensor([[1, 1], [1, 0]], dtype=torch.int32, device="cuda")
    y = fb.moe_combine(rows, slot, torch.ones((2, 2), device="cuda"), out_dtype=F32)
    assert torch.equal(y, torch.stack([2 * rows[1].float(), rows[0].float() + rows[1].float()]))


def test_left_out_pairs_add_nothing():
    """Not even a zero: a residual of -0 stays -0."""
    res = torch.full((2, 16), -0.0, dtype=BF, device="cuda")
    slot = torch.tensor([[-1, -1, 4], [-1, 0, 9]], dtype=torch.int32, device="cuda")
    rows = torch.full((4, 16), -0.0, dtype=BF, device="cuda")
    y = fb.moe_combine(rows, slot, torch.ones((2, 3), device="cuda"), residual=res)
    assert torch.all(torch.signbit(y))


def test_rows_beyond_32_bit_offsets():
    total, n = 300000, 16384
    rows = torch.zeros((total, n), dtype=BF, device="cuda")
    rows[-2:] = torch.randn((2, n), device="cuda").to(BF)
    slot = torch.tensor([[total - 1, 0], [5, total - 2]], dtype=torch.int32, device="cuda")
    w = torch.full((2, 2), 0.5, device="cuda")
    y = fb.moe_combine(rows, slot, w, out_dtype=F32)
    assert torch.equal(y, 0.5 * rows[-2:].flip(0).float())
    dy = torch.randn((2, n), device="cuda").to(BF)
    drows = torch.zeros_like(rows)
    dw = torch.empty_like(w)
    fb.fp8_moe_combine_backward(dy, rows, slot, w, drows, dw)
    assert torch.equal(drows[-1], (0.5 * dy[0].float()).to(BF)) and torch.equal(drows[5], (0.5 * dy[1].float()).to(BF))
    want = (dy.double() * rows[-2:].flip(0).double()).sum(1)
    mag = (dy.double() * rows[-2:].flip(0).double()).abs().sum(1)
    assert torch.all((torch.stack([dw[0, 0], dw[1, 1]]).double() - want).abs() <= n * 2.0 ** -24 * mag)
    assert dw[0, 1] == 0 and dw[1, 0] == 0


@pytest.mark.parametrize("row_dtype", [BF, F32])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("top_k", [1, 2, 3, 8])
def test_a_large_call_is_its_small_ones(row_dtype, out_dtype, top_k):
    """Calls past the size of the last cache (nontemporal) against the same tokens in calls below it."""
    n, tokens = 4104, 36000 // top_k + 3
    g = torch.Generator("cuda").manual_seed(top_k)
    rows = torch.randn((tokens * top_k, n), device="cuda", generator=g).to(row_dtype)
    res = torch.randn((tokens, n), device="cuda", generator=g).to(BF)
    slot = torch.randperm(tokens * top_k, device="cuda", generator=g).to(torch.int32).view(tokens, top_k)
    w = torch.rand((tokens, top_k), device="cuda", generator=g)
    y = fb.moe_combine(rows, slot, w, residual=res, out_dtype=out_dtype)
    dy = res if out_dtype == BF else res.float()
    drows, dw = fb.moe_combine_backward(dy, rows, slot, w)
    parts = torch.empty_like(rows)
    step = tokens // 12
    for t in range(0, tokens, step):
        cut = slice(t, min(t + step, tokens))
        one = fb.moe_combine(rows, slot[cut].contiguous(), w[cut].contiguous(), residual=res[cut].contiguous(),
                             out_dtype=out_dtype)
        assert torch.equal(y[cut], one)
        dwc = torch.empty_like(w[cut])
        fb.fp8_moe_combine_backward(dy[cut].contiguous(), rows, slot[cut].contiguous(), w[cut].contiguous(), parts,
                                    dwc)
        assert torch.equal(dw[cut], dwc)
    assert torch.equal(drows, parts)


@pytest.mark.parametrize("tokens,top_k,n,total", SHAPES)
@pytest.mark.parametrize("row_dtype", [BF, F32])
@pytest.mark.parametrize("dy_dtype", [BF, F32])
def test_backward(tokens, top_k, n, total, row_dtype, dy_dtype):
    """Rows that no slot names keep what they held; pairs left out get a weight gradient of 0."""
    print(f"[combine backward] {tokens} tokens, {top_k} of {total} rows of {n}, {row_dtype} {dy_dtype}", flush=True)
    rng = np.random.default_rng(tokens + n + 1)
    rows, dy = _t(rng.standard_normal((total, n)), row_dtype), _t(rng.standard_normal((tokens, n)), dy_dtype)
    slot, w = _slots(rng, tokens, top_k, total), rng.uniform(-1, 1, (tokens, top_k)).astype(np.float32)
    if total > 3:
        slot[slot == 3] = -1
    drows = torch.full_like(rows, 7.0)
    dw = torch.full((tokens, top_k), 9.0, dtype=F32, device="cuda")
    fb.fp8_moe_combine_backward(dy, rows, torch.from_numpy(slot).cuda(), torch.from_numpy(w).cuda(), drows, dw)
    d64, r64 = _np(dy), _np(rows)
    want, wantw = moe.combine_backward(d64, r64, slot, w, np.full((total, n), 7.0))
    step = 2.0 ** -8 if row_dtype == BF else 2.0 ** -24
    assert np.all(np.abs(_np(drows) - want) <= step * np.abs(want))
    _, mag = moe.combine_backward(np.abs(d64), np.abs(r64), slot, w, np.zeros((total, n)))
    assert np.all(np.abs(_np(dw) - wantw) <= n * 2.0 ** -24 * mag)
    assert np.all(_np(dw)[slot < 0] == 0)


def test_backward_against_differences():
    """The combination is linear: its difference along a direction is the gradient's product with it."""
    rng = np.random.default_rng(5)
    rows, dy = _t(rng.standard_normal((12, 64)), F32), _t(rng.standard_normal((4, 64)), F32)
    slot = torch.from_numpy(_slots(rng, 4, 3, 12)).cuda()
    w = _t(rng.uniform(0, 1, (4, 3)), F32)
    drows, dw = fb.moe_combine_backward(dy, rows, slot, w)
    v, u = _t(rng.standard_normal((12, 64)), F32), _t(rng.standard_normal((4, 3)), F32)
    for moved, grad, args in ((v, drows, [(rows + v, w), (rows - v, w)]), (u, dw, [(rows, w + u), (rows, w - u)])):
        up, dn = (_np(fb.moe_combine(r, slot, ww, out_dtype=F32)) for r, ww in args)
        got = (_np(dy) * (up - dn)).sum() / 2
        want = (_np(moved) * _np(grad)).sum()
        mag = (np.abs(_np(dy)) * (np.abs(up) + np.abs(dn))).sum() + (np.abs(_np(moved) * _np(grad))).sum()
        assert abs(got - want) <= 64 * 2.0 ** -24 * mag


@pytest.mark.parametrize("row_dtype", [BF, F32])
@pytest.mark.parametrize("dy_dtype", [BF, F32])
@pytest.mark.parametrize("top_k", [1, 2, 3, 8, 11])
def test_backward_of_left_out_pairs_whatever_dy_holds(top_k, dy_dtype, row_dtype):
    """A slot outside the rows gets a weight gradient of 0 where dy is infinite or NaN too; finite tokens beside such
    ones keep theirs."""
    rng = np.random.default_rng(top_k)
    tokens, n, total = 5, 264, 5 * top_k
    rows, dy = _t(rng.standard_normal((total, n)), row_dtype), _t(rng.standard_normal((tokens, n)), dy_dtype)
    clean = dy.clone()
    dy[1] = float("inf")
    dy[2, 7], dy[2, 260] = float("nan"), -float("inf")
    dy[4] = float("nan")
    slot = _slots(rng, tokens, top_k, total)
    slot[rng.random(slot.shape) < 0.4] = -1
    slot[1, 0], slot[2, top_k - 1] = total, -5
    slot[4] = np.where(np.arange(top_k) % 2, np.iinfo(np.int32).max, np.iinfo(np.int32).min)
    st, w = torch.from_numpy(slot).cuda(), _t(rng.uniform(-1, 1, (tokens, top_k)), F32)
    dw = torch.full((tokens, top_k), 9.0, dtype=F32, device="cuda")
    fb.fp8_moe_combine_backward(dy, rows, st, w, torch.empty_like(rows), dw)
    want = fb.moe_combine_backward(clean, rows, st, w)[1]
    out = torch.from_numpy((slot < 0) | (slot >= total)).cuda()
    assert torch.all(dw[out] == 0)
    assert torch.equal(dw[[0, 3]], want[[0, 3]])
    assert not torch.any(torch.isfinite(dw[[1, 2]]) & ~out[[1, 2]])
