"""Pins of the mixture-of-experts oracle (oracle/moe.py): gradients against central differences of the forward
functions, routing against hand-worked cases and torch's own functions, the plan against its definition."""

import numpy as np
import pytest
import torch

from oracle import moe
from oracle.codec import bf16_to_f32, f32_to_bf16


def _differences(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        g[i] = (f(a) - f(b)) / (2 * step)
    return g


def test_add_residual_is_the_rounded_sum():
    rng = np.random.default_rng(1)
    a = f32_to_bf16(rng.standard_normal((4, 64)).astype(np.float32))
    b = f32_to_bf16((rng.standard_normal((4, 64)) * 300).astype(np.float32))
    want = (torch.from_numpy(bf16_to_f32(a).astype(np.float64)) + torch.from_numpy(bf16_to_f32(b).astype(np.float64)))
    assert np.array_equal(bf16_to_f32(moe.add_residual(a, b)), want.float().to(torch.bfloat16).float().numpy())


def test_rmsnorm_of_a_known_row():
    y, rstd = moe.rmsnorm(np.array([[3.0, -4.0, 0.0, 0.0]]), np.array([1.0, 2.0, 3.0, 4.0]), 0.0)
    assert rstd[0] == pytest.approx(0.4)                       # mean square 25 / 4
    assert y[0] == pytest.approx([1.2, -3.2, 0.0, 0.0])


@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_gradients_against_differences(residual):
    rng = np.random.default_rng(2)
    h, w, dy = rng.standard_normal((3, 8)), rng.standard_normal(8), rng.standard_normal((3, 8))
    dres = rng.standard_normal((3, 8)) if residual else None
    rstd = moe.rmsnorm(h, w, 1e-3)[1]
    dx, dw = moe.rmsnorm_backward(dy, h, w, rstd, dres)

    def loss(hh, ww):
        return (dy * moe.rmsnorm(hh, ww, 1e-3)[0]).sum() + (0.0 if dres is None else (dres * hh).sum())

    assert np.allclose(dx, _differences(lambda v: loss(v, w), h), atol=1e-7)
    assert np.allclose(dw, _differences(lambda v: loss(h, v), w), atol=1e-7)


def test_route_by_hand():
    logits = np.array([[0.0, 1.0, 2.0, 2.0, -1.0, 0.5, 0.25, 3.0]])
    ids, w = moe.route(logits, None, 3, "softmax")
    assert ids.tolist() == [[7, 2, 3]]                         # the tie of 2 and 3 goes to the lower index
    p = np.exp(logits[0]) / np.exp(logits[0]).sum()
    assert w[0] == pytest.approx(p[[7, 2, 3]])
    # two groups of four, one kept: by its best key {4..7}, by its two best scores {0..3}
    assert moe.route(logits, None, 2, "sigmoid", 2, 1, "max")[0].tolist() == [[7, 5]]
    assert moe.route(logits, None, 2, "sigmoid", 2, 1, "top2")[0].tolist() == [[2, 3]]
    # the bias ranks, the weights leave it out
    ids, w = moe.route(logits, np.array([9.0, 0, 0, 0, 0, 0, 0, 0]), 2, "sigmoid", renorm=True, scale=2.0)
    assert ids.tolist() == [[0, 7]]
    s = 1 / (1 + np.exp(-logits[0, [0, 7]]))
    assert w[0] == pytest.approx(2.0 * s / s.sum())


def test_route_masks():
    inf, nan = np.inf, np.nan
    logits = np.array([[-inf, 1.0, nan, 0.0], [-inf, nan, -inf, -inf], [inf, 0.0, inf, 1.0]])
    ids, w = moe.route(logits, None, 3, "softmax", renorm=True)
    assert ids.tolist() == [[1, 3, -1], [-1, -1, -1], [0, 2, 3]]
    assert w[0] == pytest.approx([1 / (1 + np.exp(-1)), 1 / (1 + np.e), 0.0])
    assert w[1].tolist() == [0, 0, 0] and w[2] == pytest.approx([0.5, 0.5, 0.0])
    assert moe.route(logits[:1], np.array([0, -inf, 0, 0]), 2, "sigmoid")[0].tolist() == [[3, -1]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_renormalized_weights_survive_small_scores(score):
    w = moe.route(np.array([[-900.0, -901.0, -2000.0, -2000.0]]), None, 2, score, renorm=True)[1]
    assert w[0] == pytest.approx([1 / (1 + np.exp(-1)), 1 / (1 + np.e)])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    logits, dw = rng.standard_normal((3, 6)), rng.standard_normal((3, 4))
    ids = np.array([[1, 4, 0, -1], [2, 2, 5, 3], [-1, 7, -1, -1]], dtype=np.int32)   # left out, listed twice, empty

    def loss(l):
        return sum((dw[t] * moe.chosen_weights(l[t], ids[t].tolist(), score, renorm, 1.5)).sum() for t in range(3))

    got = moe.route_backward(logits, ids, dw, score, renorm, 1.5)
    assert np.allclose(got, _differences(loss, logits), atol=1e-8)


def test_plan_definition():
    ids = np.array([[2, 0], [1, 2], [-1, 2], [5, 0]], dtype=np.int32)
    off, row, slot = moe.plan(ids, 3)
    assert off.tolist() == [0, 2, 3, 6]
    assert row.tolist() == [0, 3, 1, 0, 1, 2, 0, 0]
    assert slot.tolist() == [[3, 0], [2, 4], [-1, 5], [-1, 1]]


def test_combine_and_gradients_against_differences():
    rng = np.random.default_rng(4)
    rows, w, dy = rng.standard_normal((5, 4)), rng.standard_normal((2, 2)), rng.standard_normal((2, 4))
    slot = np.array([[3, 0], [-1, 4]], dtype=np.int32)
    res = rng.standard_normal((2, 4))
    y = moe.combine(rows, slot, w, res)
    assert y[0] == pytest.approx(res[0] + w[0, 0] * rows[3] + w[0, 1] * rows[0])
    dr, dw = moe.combine_backward(dy, rows, slot, w, np.full((5, 4), 7.0))
    named = [0, 3, 4]
    assert np.all(dr[[1, 2]] == 7.0)
    assert np.allclose(dr[named], _differences(lambda v: (dy * moe.combine(v, slot, w)).sum(), rows)[named], atol=1e-8)
    assert np.allclose(dw, _differences(lambda v: (dy * moe.combine(rows, slot, v)).sum(), w), atol=1e-8)


def test_nvfp4_matrix_and_grouped_product():
    q = np.array([[0x21, 0xF0] + [0] * 6], dtype=np.uint8)            # 0.5, 1, 0, -6, 0 ...
    w = moe.nvfp4_matrix(q, np.array([[0x40]], dtype=np.uint8), [0.25], 1)   # S = 2
    assert w[0, :4].tolist() == [0.25, 0.5, 0.0, -3.0]
    x = np.ones((2, 16))
    y, mag = moe.grouped_matvec(x, np.array([1, 0, 1]), [w, 2 * w], [0, 1, 2], 3)
    assert y[:2, 0].tolist() == [-2.25, -4.5] and np.isnan(y[2, 0]) and mag[1, 0] == 7.5
