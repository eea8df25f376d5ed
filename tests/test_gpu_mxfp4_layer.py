"""The MXFP4 operators together, as a mixture-of-experts layer uses them: a prompt through the grouped products with
MXFP8 or MXFP4 activations, decoded tokens through the products of bf16 rows, a training step with straight-through
gradients; padded tokens, captured graphs, other streams.

Every stage of a layer is compared with float64 from the stage's own inputs, so that tolerances are those of one
operator: k 2^-24 of the sum of magnitudes for fp32 sums of k products, 2^-10 of it where E4M3 products are cut, and
half a step of bf16 (2^-8) of a rounded result.
"""

import numpy as np
import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from workloads import normal_bf16

pytestmark = pytest.mark.gpu
H, INTER, E, K = 512, 256, 16, 4
EPS = 1e-6
F64 = torch.float64
ROUTE = dict(score="sigmoid", groups=4, topk_groups=2, group_score="top2", renorm=True, scale=2.5)


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _model(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, s=0.05):
        return (torch.randn(shape, device="cuda", generator=g) * s).to(torch.bfloat16)

    m = {"norm": 1 + 0.1 * torch.randn(H, device="cuda", generator=g), "gate": r(E, H, s=0.1),
         "bias": 0.05 * torch.randn(E, device="cuda", generator=g), "up": r(E, 2 * INTER, H), "down": r(E, H, INTER)}
    for name in ("up", "down"):
        n, k = m[name].shape[1:]
        q, s, dq = fb.mxfp4_quantize(m[name].view(E * n, k), dequant=True)
        m[name + "4"] = (q.view(E, n, k // 2), s.view(E, n, k // 32))
        m[name + "q"] = dq.view(E, n, k)
    return m


def _inputs(tokens, seed):
    return normal_bf16((tokens, H), 1.0, seed, "cuda"), normal_bf16((tokens, H), 2.0, seed + 1, "cuda")


def _route(m, x, res, padded=()):
    n = fb.rmsnorm_quantize(x, m["norm"], EPS, residual=res, block="1x32", normed=True, dequant=True)
    logits = (n["y"].float()[:, None, :] * m["gate"].float()[None]).sum(-1)
    if padded:
        logits[list(padded)] = -float("inf")
    ids, w = fb.moe_route(logits, K, bias=m["bias"], **ROUTE)
    return n, ids, w, fb.moe_plan(ids, E)


def _silu(gu):
    g, u = gu.float().chunk(2, -1)
    return (torch.nn.functional.silu(g) * u).to(torch.bfloat16)


def _prompt(m, x, res, elem="e4m3", padded=()):
    n, ids, w, (off, row, slot) = _route(m, x, res, padded)
    gu = fb.mxfp4_grouped_gemm(n["q"], n["scale"], "e4m3", *m["up4"], off, row_index=row)
    if elem == "e4m3":
        aq, asc, adq = fb.quantize(_silu(gu), "1x32", dequant=True)
    else:
        aq, asc, adq = fb.mxfp4_quantize(_silu(gu), dequant=True)
    d = fb.mxfp4_grouped_gemm(aq, asc, elem, *m["down4"], off)
    return fb.moe_combine(d, slot, w, residual=n["h"]), (n, w, off, row, slot, gu, adq, d)


def _decode(m, x, res):
    n, ids, w, (off, row, slot) = _route(m, x, res)
    gu = fb.mxfp4_grouped_matvec(n["y"], *m["up4"], off, row_index=row)
    a = _silu(gu)
    d = fb.mxfp4_grouped_matvec(a, *m["down4"], off)
    return fb.moe_combine(d, slot, w, residual=n["h"]), (n, w, off, row, slot, gu, a, d)


def _near(got, x, w, off, cut):
    """got rows of group e against x rows . w[e]^T."""
    at = off.tolist()
    for e in range(len(at) - 1):
        a, b = x[at[e]:at[e + 1]].to(F64), w[e].to(F64)
        want, mag = a @ b.T, a.abs() @ b.abs().T
        tol = (a.shape[1] * 2.0 ** -24 + cut) * mag + 2.0 ** -8 * want.abs()
        assert torch.all((got[at[e]:at[e + 1]].to(F64) - want).abs() <= tol), e


def _combined(y, d, slot, w, h):
    rows = d.to(F64)[slot.long().clamp(min=0).view(-1)].view(*slot.shape, -1)
    rows = rows * (w.to(F64) * (slot >= 0))[..., None]
    want, mag = h.to(F64) + rows.sum(1), h.to(F64).abs() + rows.abs().sum(1)
    assert torch.all((y.to(F64) - want).abs() <= (K + 2) * 2.0 ** -24 * mag + 2.0 ** -8 * want.abs())


@pytest.mark.parametrize("tokens", [1, 7, 150, 700])
@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
def test_prompt_layer(tokens, elem):
    m = _model(1)
    x, res = _inputs(tokens, 40)
    y, (n, w, off, row, slot, gu, adq, d) = _prompt(m, x, res, elem)
    assert off[-1].item() == tokens * K
    _near(gu, n["ydq"][row.long()], m["upq"], off, 2.0 ** -10)
    _near(d, adq, m["downq"], off, 2.0 ** -10 if elem == "e4m3" else 0.0)
    _combined(y, d, slot, w, n["h"])


@pytest.mark.parametrize("tokens", [1, 2, 9, 40])
def test_decode_layer(tokens):
    m = _model(2)
    x, res = _inputs(tokens, 50)
    y, (n, w, off, row, slot, gu, a, d) = _decode(m, x, res)
    _near(gu, n["y"][row.long()], m["upq"], off, 0.0)
    _near(d, a, m["downq"], off, 0.0)
    _combined(y, d, slot, w, n["h"])


def test_a_token_decodes_as_in_the_batch():
    """Rows of the products do not influence each other: a token alone gives the bytes it gives in a batch."""
    m = _model(3)
    x, res = _inputs(6, 60)
    whole, _ = _decode(m, x, res)
    for t in range(6):
        one, _ = _decode(m, x[t:t + 1].contiguous(), res[t:t + 1].contiguous())
        assert _same(one, whole[t:t + 1]), t


def test_padded_tokens():
    """Tokens routed nowhere leave with their residual; the rows that nobody has stay as they were."""
    m = _model(4)
    x, res = _inputs(90, 70)
    y, (n, w, off, row, slot, gu, adq, d) = _prompt(m, x, res, padded=(2, 33, 89))
    assert off[-1].item() == 87 * K and torch.all(slot[[2, 33, 89]] == -1)
    assert _same(y[[2, 33, 89]], n["h"][[2, 33, 89]]) and torch.isfinite(y.float()).all()
    keep = torch.full((90 * K, 2 * INTER), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8_mxfp4_grouped_gemm(n["q"], n["scale"], "e4m3", row, *m["up4"], off, keep)
    assert torch.all(keep[87 * K:] == 7) and _same(keep[:87 * K], gu[:87 * K])
    keep.fill_(7)
    fb.fp8_mxfp4_grouped_matvec(n["y"], row, *m["up4"], off, keep)
    assert torch.all(keep[87 * K:] == 7)
    dx = torch.full((90 * K, H), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.fp8_grouped_dgrad(gu, m["upq"], off, dx)
    assert torch.all(dx[87 * K:] == 7) and torch.isfinite(dx.float()).all()
    gu[87 * K:] = float("nan")                                # and contribute nothing to the weights' gradient
    assert torch.isfinite(fb.grouped_wgrad(gu, n["ydq"], off, row_index=row)).all()


def _backward(m, x, res, dy):
    """Straight-through gradients of a layer's experts: of their weights and of the rows they read."""
    _, (n, w, off, row, slot, gu, adq, d) = _prompt(m, x, res)
    drows, dw = fb.moe_combine_backward(dy, d, slot, w)
    ddown = fb.grouped_wgrad(drows, adq, off)
    da = fb.grouped_dgrad(drows, m["downq"], off)
    g, u = gu.float().chunk(2, -1)
    s = torch.sigmoid(g)
    dgu = torch.cat([da.float() * u * s * (1 + g * (1 - s)), da.float() * g * s], -1).to(torch.bfloat16)
    dup = fb.grouped_wgrad(dgu, n["ydq"], off, row_index=row)
    dx = fb.grouped_dgrad(dgu, m["upq"], off, out_dtype=torch.float32)
    return ddown, dup, dx, drows


def test_training_step_against_autograd():
    """Against autograd in double precision through the layer's own quantized values.  Between the calls the rows'
    gradients are rounded to bf16 three times (2^-8 each, independently): 2^-5 of the norm is eight times that."""
    m = _model(5)
    tokens = 120
    x, res = _inputs(tokens, 80)
    dy = normal_bf16((tokens, H), 1e-2, 90, "cuda")
    ddown, dup, dx, _ = _backward(m, x, res, dy)
    _, (n, w, off, row, slot, gu, adq, d) = _prompt(m, x, res)
    up, down = m["upq"].to(F64).requires_grad_(True), m["downq"].to(F64).requires_grad_(True)
    xr = n["ydq"].to(F64)[row.long()].requires_grad_(True)
    at, outs = off.tolist(), []
    for e in range(E):
        z = xr[at[e]:at[e + 1]] @ up[e].T
        z = z + (gu[at[e]:at[e + 1]].to(F64) - z).detach()                    # the values of the forward call
        g, u = z.chunk(2, -1)
        a = torch.nn.functional.silu(g) * u
        a = a + (adq[at[e]:at[e + 1]].to(F64) - a).detach()
        outs.append(a @ down[e].T)
    out = torch.cat(outs)
    y = (out[slot.long().view(-1)].view(tokens, K, H) * w.to(F64)[..., None]).sum(1)
    gup, gdown, gx = torch.autograd.grad(y, (up, down, xr), dy.to(F64))
    for got, want in ((ddown, gdown), (dup, gup), (dx, gx)):
        assert (got.to(F64) - want).norm() <= 2.0 ** -5 * want.norm()


def test_gradients_against_differences():
    """sum(dy y) for y = x[row] . W^T is linear in W and in x: its difference along any direction is the gradient's
    product with that direction, up to fp32 sums of the gradient."""
    m = _model(6)
    x, res = _inputs(64, 95)
    n, _, _, (off, row, _) = _route(m, x, res)
    dy = normal_bf16((64 * K, 2 * INTER), 1.0, 96, "cuda")
    dw = fb.grouped_wgrad(dy, n["ydq"], off, row_index=row).to(F64)
    dx = fb.grouped_dgrad(dy, m["upq"], off, out_dtype=torch.float32).to(F64)
    at, xr, w = off.tolist(), n["ydq"].to(F64)[row.long()], m["upq"].to(F64)

    def loss(rows, mats):
        return sum((dy[at[e]:at[e + 1]].to(F64) * (rows[at[e]:at[e + 1]] @ mats[e].T)).sum() for e in range(E))

    g = torch.Generator(device="cuda").manual_seed(1)
    ew = torch.randn(w.shape, device="cuda", generator=g, dtype=F64)
    ex = torch.randn(xr.shape, device="cuda", generator=g, dtype=F64)
    for diff, grad, along, terms in ((loss(xr, w + ew) - loss(xr, w - ew), dw, ew, 64 * K),
                                     (loss(xr + ex, w) - loss(xr - ex, w), dx, ex, 2 * INTER)):
        # every element of a gradient is off by terms 2^-24 of its sum of magnitudes, at most terms max|dy| max|x or w|
        mag = terms * dy.abs().max().item() * max(xr.abs().max().item(), w.abs().max().item())
        assert abs((diff / 2 - (grad * along).sum()).item()) <= terms * 2.0 ** -24 * mag * along.abs().sum().item()
        assert abs(diff.item()) > 0


@pytest.mark.parametrize("which", ["prompt", "decode", "backward"])
def test_captured_and_replayed(which):
    """A layer captured once gives the eager bytes on every replay, with eager work on other inputs in between; a
    second graph of the same calls, captured beside it, does not disturb it."""
    m = _model(7)
    tokens = 5 if which == "decode" else 96
    x, res = _inputs(tokens, 100)
    dy = normal_bf16((tokens, H), 1e-2, 101, "cuda")

    def step():
        if which == "backward":
            return list(_backward(m, x, res, dy))
        y, parts = (_prompt if which == "prompt" else _decode)(m, x, res)
        return [y, *parts[1:]]

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i in range(4):
        a, b = _inputs(tokens, 110 + 2 * i)
        x.copy_(a)
        res.copy_(b)
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for o in outs[0] + outs[1]:
            o.fill_(0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for j, (got, ref) in enumerate(zip(outs[0] + outs[1], want + want)):
            assert _same(got, ref), f"{which} replay {i}: output {j}"
        print(f"[mxfp4 layer] {which} replay {i}: {len(want)} outputs of two graphs equal the eager calls", flush=True)


def test_two_streams_at_once():
    """Every operator on two streams, given explicitly, against the same calls one after the other."""
    m = _model(8)
    sets = []
    for seed in (200, 210):
        n, _, _, (off, row, _) = _route(m, *_inputs(200, seed))
        sets.append((n, off, row, normal_bf16((200 * K, 2 * INTER), 1.0, seed + 5, "cuda")))

    def calls(i, stream):
        n, off, row, dy = sets[i]
        q, s, dq = fb.mxfp4_quantize(n["y"], dequant=True, stream=stream)
        return [q, s, dq, fb.mxfp4_dequantize(q, s, stream=stream),
                fb.mxfp4_gemm(n["q"], n["scale"], "e4m3", m["up4"][0][i], m["up4"][1][i], stream=stream),
                fb.mxfp4_grouped_gemm(q, s, "e2m1", *m["up4"], off, row_index=row, stream=stream),
                fb.mxfp4_matvec(n["y"][:5].contiguous(), m["up4"][0][i], m["up4"][1][i], stream=stream),
                fb.mxfp4_grouped_matvec(n["y"], *m["up4"], off, row_index=row, stream=stream),
                fb.grouped_dgrad(dy, m["upq"], off, stream=stream),
                fb.grouped_wgrad(dy, n["ydq"], off, row_index=row, stream=stream),
                fb.grouped_wgrad(dy, n["ydq"], off, row_index=row, out_dtype=torch.bfloat16, stream=stream)]

    want = [calls(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for rep in range(3):
        for i, s in enumerate(streams):
            got[i] = calls(i, s if rep else s.cuda_stream)
    torch.cuda.synchronize()
    for i in range(2):
        for j, (a, b) in enumerate(zip(got[i], want[i])):
            assert _same(a, b), (i, j)


def test_library_errors_reach_the_caller():
    x = torch.zeros((2, 96), dtype=torch.bfloat16, device="cuda")
    q, s = fb.mxfp4_quantize(x)
    with pytest.raises(fb.Fp8Error) as e:
        fb.mxfp4_gemm(q, s, "e2m1", q, s)                                        # 96 is no multiple of 128
    assert e.value.status == 2
    with pytest.raises(fb.Fp8Error) as e:
        fb.mxfp4_quantize(x[:, :80].contiguous())                                # nor 80 of 32
    assert e.value.status == 2
    flat = torch.zeros(2 * 128 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fb.Fp8Error) as e:
        fb.mxfp4_quantize(flat[4:].view(2, 128))                                 # 8-byte aligned
    assert e.value.status == 3
    with pytest.raises(ValueError):
        fb.mxfp4_gemm(q, s, "e5m2", q, s)
