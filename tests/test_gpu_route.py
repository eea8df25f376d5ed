"""GPU parity of fp8_moe_route, fp8_moe_route_backward and fp8_moe_plan against the oracle (oracle/moe.py).

Expert ids, offsets, row index and slots are equal.  Weights and gradients are fp32: an exponential of a difference
of two logits that lie L apart is off by at most 2^-24 L (the difference's rounding) and 2^-23, a sum over up to
1024 experts in at most 16 + 6 dependent additions by 22 * 2^-24, and three more operations follow, so a weight is
within W = 2^-18 + 2^-22 L of its value (+ 2^-126 where the result leaves the normal range).  A gradient is a product
of such a weight and a difference of dweights, which a sum of up to 64 of them enters: it is within 2 W + 2^-18 of
the sum of the magnitudes.  bf16 gradients add 2^-8.
"""

import numpy as np
import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from oracle import moe

pytestmark = pytest.mark.gpu


def _logits(rng, tokens, experts, dtype, sigma=1.5):
    l = torch.from_numpy((sigma * rng.standard_normal((tokens, experts))).astype(np.float32)).to(dtype)
    return l.cuda(), l.double().numpy()


def _spread(l):
    fin = np.where(np.isfinite(l), l, np.nan)
    with np.errstate(all="ignore"):
        s = np.nanmax(fin, axis=1) - np.nanmin(fin, axis=1)
    return float(np.nanmax(np.append(s, 0.0)))


def _check(l, l64, bias, top_k, score, groups=1, kept=1, gs="max", renorm=False, scale=1.0):
    ids = torch.full((l.shape[0], top_k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((l.shape[0], top_k), 7.0, dtype=torch.float32, device="cuda")
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    fb.fp8_moe_route(l, ids, w, b, score, groups, kept, gs, renorm, scale)
    torch.cuda.synchronize()
    want, ww = moe.route(l64, None if bias is None else bias.astype(np.float32), top_k, score, groups, kept, gs,
                         renorm, scale)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    bad = np.argwhere(ids != want)
    assert len(bad) == 0, (len(bad), bad[0], ids[bad[0][0]], want[bad[0][0]])
    tol = 2.0 ** -18 + 2.0 ** -22 * _spread(l64)
    assert np.all(np.abs(w - ww) <= tol * np.abs(ww) + 2.0 ** -126), np.abs(w - ww).max()
    return ids, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 256, 8), (5, 8, 2), (3, 8, 8), (130, 64, 6),
                                                  (17, 160, 6), (9, 61, 5), (33, 257, 7), (4, 1024, 64), (6, 100, 64)])
def test_ungrouped(dtype, score, tokens, experts, top_k):
    print(f"[route] {tokens}x{experts} top {top_k} {score} {dtype}", flush=True)
    rng = np.random.default_rng(tokens * 1000 + experts)
    l, l64 = _logits(rng, tokens, experts, dtype)
    bias = 0.1 * rng.standard_normal(experts)
    _check(l, l64, None, top_k, score)
    _check(l, l64, bias, top_k, score, renorm=True, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gs", ["max", "top2"])
@pytest.mark.parametrize("experts,groups,kept,top_k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 64, 9, 9), (64, 2, 1, 32),
                                                       (96, 3, 2, 4), (1024, 64, 5, 16), (8, 4, 4, 8), (36, 12, 1, 3)])
def test_grouped(score, gs, experts, groups, kept, top_k):
    print(f"[route] {experts} experts, {kept} of {groups} groups, top {top_k} {score} {gs}", flush=True)
    rng = np.random.default_rng(experts + groups)
    l, l64 = _logits(rng, 37, experts, torch.float32)
    bias = 0.1 * rng.standard_normal(experts)
    _check(l, l64, None, top_k, score, groups, kept, gs, renorm=True)
    _check(l, l64, bias, top_k, score, groups, kept, gs)


@pytest.mark.parametrize("experts,groups,kept,top_k", [(256, 1, 1, 8), (256, 8, 4, 8), (160, 8, 3, 6), (130, 13, 2, 9),
                                                       (100, 1, 1, 40), (96, 32, 7, 3), (66, 33, 9, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens(experts, groups, kept, top_k, score):
    """The launch shapes for many tokens choose as those for a few do (which are compared with the oracle)."""
    tokens = 4101
    l = 1.5 * torch.randn((tokens, experts), device="cuda", generator=torch.Generator("cuda").manual_seed(experts))
    l[7] = -float("inf")
    l[tokens - 1, 1:] = -float("inf")
    b = 0.1 * torch.randn(experts, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    for bias in (None, b):
        for gs in ("max", "top2"):
            kw = dict(bias=bias, score=score, groups=groups, topk_groups=kept, group_score=gs, renorm=True)
            ids, w = fb.moe_route(l, top_k, **kw)
            for at in range(0, tokens, 1367):
                part = slice(at, min(tokens, at + 1367))
                i2, w2 = fb.moe_route(l[part].contiguous(), top_k, **kw)
                assert torch.equal(ids[part], i2), (bias is not None, gs, at)
                assert torch.all((w[part] - w2).abs() <= 2.0 ** -18 * w2.abs())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(score):
    rng = np.random.default_rng(2)
    l64 = rng.integers(-2, 3, (50, 96)).astype(np.float64)
    l = torch.from_numpy(l64.astype(np.float32)).cuda()
    _check(l, l64, None, 8, score)
    _check(l, l64, np.zeros(96), 8, score)
    _check(l, l64, rng.integers(0, 2, 96).astype(np.float64), 8, score, 8, 3, "top2")
    _check(torch.zeros((3, 96), device="cuda"), np.zeros((3, 96)), None, 8, score, 8, 2, "max")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gs", ["max", "top2"])
def test_keys_closer_than_fp32_tells_apart(score, gs):
    """Every logit a few fp32 steps from the next and a bias that hides the scores' low bits: the order is that of
    double precision."""
    rng = np.random.default_rng(3)
    steps = rng.integers(-40, 41, (64, 128))
    l32 = (np.float32(0.7) + steps.astype(np.float32) * np.float32(2.0 ** -24)).astype(np.float32)
    l, l64 = torch.from_numpy(l32).cuda(), l32.astype(np.float64)
    for bias in (np.full(128, 8.0), rng.integers(0, 2, 128) * 2.0 ** -22 + 3.0):
        _check(l, l64, bias, 8, score)
        _check(l, l64, bias, 8, score, 16, 5, gs)
    _check(l, l64, None, 8, score, 16, 5, gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("base", [0.5, -0.5, 100.0, -1000.0])
@pytest.mark.parametrize("experts,groups,tokens", [(64, 4, 5), (256, 8, 5), (1024, 16, 3), (256, 8, 4100), (96, 3, 40)])
def test_keys_a_few_steps_apart(score, base, experts, groups, tokens):
    """Equal scores and biases one to some fp32 steps apart: the key's own low bits decide."""
    rng = np.random.default_rng(experts + tokens)
    l64 = np.full((tokens, experts), 0.25)
    l = torch.from_numpy(l64.astype(np.float32)).cuda()
    step = float(np.spacing(np.float32(abs(base))))
    bias = base + step * rng.permutation(experts)
    _check(l, l64, bias, 8, score)
    _check(l, l64, bias, 8, score, groups, 2, "top2")
    _check(l, l64, bias, 8, score, groups, 1, "max", renorm=True)


def test_bias_that_is_not_aligned_for_four():
    rng = np.random.default_rng(33)
    for experts, tokens in ((256, 3), (256, 4200), (64, 50)):
        l, _ = _logits(rng, tokens, experts, torch.float32)
        bias = torch.randn(experts + 1, device="cuda")[1:]
        assert bias.data_ptr() % 16
        got = fb.moe_route(l, 6, bias=bias, score="sigmoid", groups=8, topk_groups=3, group_score="top2")
        want = fb.moe_route(l, 6, bias=bias.clone(), score="sigmoid", groups=8, topk_groups=3, group_score="top2")
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_that_cancel(score):
    """Two best keys of a group that are large and of opposite sign: their sum is small, its rounding is not."""
    rng = np.random.default_rng(31)
    l, l64 = _logits(rng, 300, 32, torch.float32)
    bias = np.full(32, -5000.0)
    for g in range(8):
        bias[4 * g], bias[4 * g + 1] = 1000.0 + 0.001 * g, -1000.0 - 0.001 * g
    bias = bias.astype(np.float32).astype(np.float64)
    _check(l, l64, bias, 4, score, 8, 3, "top2")
    _check(l, l64, bias, 4, score, 8, 1, "top2", renorm=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_group_sums_beyond_fp32(score, sign):
    """Two keys of a group near the largest float: fp32 sums of +-inf would tie, or look like a group of none."""
    rng = np.random.default_rng(32)
    l, l64 = _logits(rng, 50, 32, torch.float32)
    l[:, :4] = -float("inf")                                  # a group of none before the others
    l64[:, :4] = -np.inf
    size = np.repeat(np.array([0, 2, 3, 1, 2.5, 3.4, 3.3, 1.5]), 4) * 1e38
    bias = (sign * size).astype(np.float32).astype(np.float64)
    _check(l, l64, bias, 4, score, 8, 2, "top2")
    _check(l, l64, bias, 4, score, 8, 7, "top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_masks(score, renorm):
    """Masked experts are never chosen; rows that mask everything, all but one, or whole groups; NaN and infinities."""
    rng = np.random.default_rng(4)
    l64 = rng.standard_normal((40, 64)).astype(np.float32).astype(np.float64)
    l64[rng.random((40, 64)) < 0.7] = -np.inf
    l64[0] = -np.inf
    l64[1] = np.nan
    l64[2, 1:] = -np.inf
    l64[3, 5] = np.inf
    l64[4, [7, 9]] = np.inf
    l64[5] = np.finfo(np.float32).min
    l64[6, ::2] = np.nan
    l64[7, :32] = -np.inf
    l = torch.from_numpy(l64.astype(np.float32)).cuda()
    bias = 0.1 * rng.standard_normal(64)
    bias[[3, 60]] = -np.inf
    bias[11] = np.nan
    for b in (None, bias):
        ids, w = _check(l, l64, b, 8, score, renorm=renorm)
        assert np.all(ids[0] == -1) and np.all(w[0] == 0) and np.all(ids[1] == -1)
        _check(l, l64, b, 8, score, 8, 3, "top2", renorm=renorm)
        _check(l, l64, b, 8, score, 8, 3, "max", renorm=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(score):
    """Scores that vanish: renormalized weights keep their ratios."""
    l64 = np.array([[-200.0, -201.0, -250.0, -203.0], [90.0, 91.0, -90.0, 0.0], [-1e30, -2e30, -1e30, -3e38],
                    [3e38, 1.0, 2.9e38, -3e38]]).astype(np.float32).astype(np.float64)
    l = torch.from_numpy(l64.astype(np.float32)).cuda()
    ids = torch.empty((4, 3), dtype=torch.int32, device="cuda")
    w = torch.empty((4, 3), dtype=torch.float32, device="cuda")
    fb.fp8_moe_route(l, ids, w, None, score, 1, 1, "max", True, 1.0)
    want, ww = moe.route(l64, None, 3, score, renorm=True)
    assert np.array_equal(ids.cpu().numpy(), want)
    # exp of differences up to 50 here; beyond the double range the weight is 0 or 1
    assert np.all(np.abs(w.cpu().numpy() - ww) <= 2.0 ** -16 * np.abs(ww) + 2.0 ** -126)


def _backward_check(l, l64, ids, dw, score, renorm, scale):
    dl = torch.full_like(l, 5.0)
    fb.fp8_moe_route_backward(l, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), dl, score, renorm, scale)
    torch.cuda.synchronize()
    got = dl.double().cpu().numpy()
    want = moe.route_backward(l64, ids, dw, score, renorm, scale)
    tol = 2.0 ** -17 + 2.0 ** -21 * _spread(l64)
    # magnitudes: |w| times the largest |dweight| of the token
    mag = np.zeros_like(want)
    for t in range(len(ids)):
        clean = moe._clean(l64[t])
        s = moe.scores(clean, score)
        p = moe.chosen_weights(clean, ids[t].tolist(), score, renorm, abs(scale))
        for j, e in enumerate(ids[t]):
            if 0 <= e < l64.shape[1]:
                mag[t, e] += p[j] * 2 * np.abs(dw[t]).max()
        if score == "softmax" and not renorm:
            mag[t] += s * p.sum() * np.abs(dw[t]).max()
    bf = l.dtype == torch.bfloat16
    assert np.all(np.abs(got - want) <= tol * mag + (2.0 ** -8 * np.abs(want) if bf else 0) + 2.0 ** -126)
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (7, 8, 2), (33, 160, 6), (5, 1024, 64), (19, 61, 5)])
def test_backward(dtype, score, renorm, tokens, experts, top_k):
    print(f"[route backward] {tokens}x{experts} top {top_k} {score} {dtype} renorm={renorm}", flush=True)
    rng = np.random.default_rng(tokens + experts)
    l, l64 = _logits(rng, tokens, experts, dtype)
    ids = np.argsort(-l64, axis=1, kind="stable")[:, :top_k].astype(np.int32)
    dw = rng.standard_normal((tokens, top_k)).astype(np.float32)
    _backward_check(l, l64, ids, dw, score, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_of_left_out_repeated_and_masked(score, renorm):
    rng = np.random.default_rng(6)
    l, l64 = _logits(rng, 6, 40, torch.float32)
    l64[4, 3] = -np.inf
    l64[5] = -np.inf
    l = torch.from_numpy(l64.astype(np.float32)).cuda()
    ids = np.array([[-1, 3, 40, 7], [5, 5, 5, 2], [-1, -1, -1, -1], [1 << 30, -5, 39, 0], [3, 4, 5, 6], [0, 1, 2, 3]],
                   dtype=np.int32)
    dw = rng.standard_normal((6, 4)).astype(np.float32)
    got = _backward_check(l, l64, ids, dw, score, renorm, 1.0)
    assert np.all(got[2] == 0) and np.all(got[5] == 0) and got[4, 3] == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_renormalized_choice_has_no_gradient(score):
    """Its weight is the scale whatever the logits: zeros, not the rounding of a difference."""
    l, _ = _logits(np.random.default_rng(41), 300, 75, torch.float32)
    ids, w = fb.moe_route(l, 1, score=score, renorm=True, scale=2.5)
    assert torch.all(w == 2.5)
    d = fb.moe_route_backward(l, ids, torch.randn((300, 1), device="cuda"), score=score, renorm=True, scale=2.5)
    assert torch.all(d == 0)


def test_more_tokens_than_one_launch_takes():
    """Tokens past the largest grid of a launch; 32 tokens of 8 experts to a workgroup."""
    tokens = 32 * (1 << 20) + 37
    l = torch.zeros((tokens, 8), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(3)
    l[-300:] = torch.randn((300, 8), device="cuda", generator=g).to(torch.bfloat16)
    ids, w = fb.moe_route(l, 2, renorm=True)
    i2, w2 = fb.moe_route(l[-300:].contiguous(), 2, renorm=True)
    assert torch.equal(ids[-300:], i2) and torch.equal(w[-300:], w2)
    assert torch.all(ids[:-300] == torch.tensor([0, 1], device="cuda", dtype=torch.int32))
    dw = torch.ones_like(w)
    dw[-300:] = torch.randn((300, 2), device="cuda", generator=g)
    d = fb.moe_route_backward(l, ids, dw, renorm=True)
    d2 = fb.moe_route_backward(l[-300:].contiguous(), i2, dw[-300:].contiguous(), renorm=True)
    assert torch.equal(d[-300:], d2) and torch.all(d[:-300] == 0)


def test_logits_beyond_32_bit_offsets():
    tokens, experts = (1 << 21) + 11, 1024
    l = torch.zeros((tokens, experts), dtype=torch.bfloat16, device="cuda")
    l[-5:] = torch.randn((5, experts), device="cuda").to(torch.bfloat16)
    ids, w = fb.moe_route(l, 8, score="sigmoid", bias=torch.zeros(experts, device="cuda"))
    i2, w2 = fb.moe_route(l[-5:].contiguous(), 8, score="sigmoid", bias=torch.zeros(experts, device="cuda"))
    assert torch.equal(ids[-5:], i2) and torch.equal(w[-5:], w2)


def _plan_check(ids, experts):
    tokens, top_k = ids.shape
    t = torch.from_numpy(ids).cuda()
    off, row, slot = fb.moe_plan(t, experts)
    again = fb.moe_plan(t, experts)
    torch.cuda.synchronize()
    want = moe.plan(ids, experts)
    for name, got, ref, two in zip(("offsets", "row_index", "slot"), (off, row, slot), want, again):
        assert np.array_equal(got.cpu().numpy(), ref), name
        assert torch.equal(got, two), name


@pytest.mark.parametrize("tokens,top_k,experts", [(0, 2, 4), (1, 1, 1), (1, 8, 256), (5, 3, 7), (256, 8, 64),
                                                  (257, 8, 256), (1000, 6, 160), (4099, 8, 256), (700, 64, 1024),
                                                  (131072, 1, 3), (2048, 1, 5), (2049, 1, 5), (300000, 1, 130),
                                                  (35000, 8, 257)])
@pytest.mark.parametrize("kind", ["spread", "one expert", "left out"])
def test_plan(tokens, top_k, experts, kind):
    print(f"[plan] {tokens} tokens, top {top_k} of {experts}, {kind}", flush=True)
    rng = np.random.default_rng(tokens + top_k)
    ids = rng.integers(0, experts, (tokens, top_k)).astype(np.int32)       # the same expert twice in a token too
    if kind == "one expert":
        ids[:] = experts - 1
    if kind == "left out" and tokens:
        ids[rng.random(ids.shape) < 0.3] = -1
        ids[rng.random(ids.shape) < 0.1] = experts
        ids[tokens // 2:] = np.iinfo(np.int32).min
    _plan_check(ids, experts)


def test_plan_workspace_holds_garbage():
    rng = np.random.default_rng(9)
    ids = rng.integers(-1, 64, (5000, 4)).astype(np.int32)
    ws = torch.full((fb.fp8_moe_plan_workspace(5000, 4, 64),), 0xEE, dtype=torch.uint8, device="cuda")
    off = torch.empty(65, dtype=torch.int32, device="cuda")
    row = torch.empty(20000, dtype=torch.int32, device="cuda")
    slot = torch.empty((5000, 4), dtype=torch.int32, device="cuda")
    fb.fp8_moe_plan(torch.from_numpy(ids).cuda(), 64, ws, off, row, slot)
    for got, ref in zip((off, row, slot), moe.plan(ids, 64)):
        assert np.array_equal(got.cpu().numpy(), ref)


def _sampled_check(l, rows, bias, top_k, score, groups, kept, gs, renorm):
    """A call over all tokens against the oracle on the tokens ``rows``."""
    l64 = l[rows].double().cpu().numpy()
    ids, w = fb.moe_route(l, top_k, bias=None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda(),
                          score=score, groups=groups, topk_groups=kept, group_score=gs, renorm=renorm)
    want, ww = moe.route(l64, None if bias is None else bias.astype(np.float32), top_k, score, groups, kept, gs,
                         renorm)
    ids, w = ids[rows].cpu().numpy(), w[rows].cpu().numpy()
    bad = np.argwhere(ids != want)
    assert len(bad) == 0, (len(bad), rows[bad[0][0]], ids[bad[0][0]], want[bad[0][0]])
    tol = 2.0 ** -18 + 2.0 ** -22 * _spread(l64)
    assert np.all(np.abs(w - ww) <= tol * np.abs(ww) + 2.0 ** -126), np.abs(w - ww).max()


@pytest.mark.parametrize("tokens,experts,groups,kept,top_k", [
    # 16 lanes to a token: groups of two lanes, of one, and of parts of lanes
    (4101, 128, 8, 3, 8), (4101, 96, 12, 5, 6), (4101, 120, 8, 3, 7), (4101, 112, 16, 6, 20), (4101, 68, 4, 2, 5),
    # 32 lanes, many tokens
    (4101, 256, 8, 4, 8), (4101, 160, 8, 3, 6), (4101, 192, 24, 7, 4),
    # 64 lanes, eight experts each: whole lanes and parts of them
    (37, 512, 8, 3, 8), (37, 384, 8, 3, 8), (37, 320, 10, 4, 9), (37, 512, 64, 9, 40), (37, 260, 13, 2, 11),
    # 64 lanes, sixteen experts each
    (37, 768, 3, 2, 8), (37, 1000, 8, 3, 64), (37, 600, 12, 5, 6), (37, 1024, 32, 4, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gs", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_of_every_launch_shape(tokens, experts, groups, kept, top_k, score, gs, biased):
    print(f"[route] {tokens}x{experts}, {kept} of {groups} groups, top {top_k} {score} {gs} bias={biased}", flush=True)
    rng = np.random.default_rng(tokens + experts + groups)
    l = 1.5 * rng.standard_normal((tokens, experts)).astype(np.float32)
    l[::3] = np.round(l[::3] * 2) / 2                     # ties, of experts and of groups
    l[1::7][rng.random(l[1::7].shape) < 0.6] = -np.inf
    per = experts // groups
    l[2::9, :per] = -np.inf                               # a group of none
    l[5] = -np.inf
    l[tokens - 1, 1:] = -np.inf
    near = np.float32(0.7) + rng.integers(-40, 41, experts).astype(np.float32) * np.float32(2.0 ** -24)
    l[4] = l[tokens - 3] = near                           # scores closer than fp32 tells apart
    bias = 0.1 * rng.standard_normal(experts)
    bias[rng.integers(0, experts, 3)] = -np.inf
    rows = list(range(37)) + ([] if tokens == 37 else list(range(tokens - 40, tokens)))
    _sampled_check(torch.from_numpy(l).cuda(), rows, bias if biased else None, top_k, score, groups, kept, gs,
                   renorm=experts % 3 == 0)
    if biased:
        flat = np.where(rng.random(experts) < 0.5, 8.0, 8.0 + 2.0 ** -20)      # hides the scores' low bits
        _sampled_check(torch.from_numpy(l).cuda(), rows, flat, top_k, score, groups, kept, gs, renorm=True)


@pytest.mark.parametrize("tokens,experts,top_k", [(4101, 128, 8), (4101, 70, 20), (4101, 255, 8), (37, 512, 8),
                                                  (37, 300, 64), (37, 777, 12)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_no_groups_in_every_launch_shape(tokens, experts, top_k, score, biased):
    rng = np.random.default_rng(tokens + experts)
    l = 1.5 * rng.standard_normal((tokens, experts)).astype(np.float32)
    l[::3] = np.round(l[::3] * 2) / 2
    l[1::7][rng.random(l[1::7].shape) < 0.6] = -np.inf
    bias = 0.1 * rng.standard_normal(experts)
    rows = list(range(37)) + ([] if tokens == 37 else list(range(tokens - 40, tokens)))
    _sampled_check(torch.from_numpy(l).cuda(), rows, bias if biased else None, top_k, score, 1, 1, "max", True)
