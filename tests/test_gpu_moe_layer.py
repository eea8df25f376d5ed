"""The mixture-of-experts operators together, as a layer uses them: a prompt through the FP8 grouped GEMMs, decoded
tokens through the NVFP4 products, a training step's backward calls; captured into HIP graphs and on other streams."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_amax_amd as fb
from oracle import moe
from oracle.codec import bf16_to_f32
from workloads import bf16_bits, normal_bf16

pytestmark = pytest.mark.gpu
H, INTER, E, K = 512, 256, 16, 4
EPS = 1e-6
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
        flat = m[name].view(E * n, k)
        q, s = fb.quantize(flat, "1x32")
        m[name + "8"] = (q.view(torch.uint8).view(E, n, k), s.view(E, n, k // 32))
        q, s, gs, _ = fb.nvfp4_quantize(flat, rows_per_tensor=n)
        m[name + "4"] = (q.view(E, n, k // 2), s.view(E, n, k // 16), gs)
    return m


def _route(m, x, res):
    """Norm, router product (fp32, so that it does not depend on the batch), routing and plan."""
    n = fb.rmsnorm_quantize(x, m["norm"], EPS, residual=res, normed=True, save_rstd=True)
    logits = (n["y"].float()[:, None, :] * m["gate"].float()[None]).sum(-1)
    ids, w = fb.moe_route(logits, K, bias=m["bias"], **ROUTE)
    return n, logits, ids, w, fb.moe_plan(ids, E)


def _silu(gu):
    g, u = gu.float().chunk(2, -1)
    return (torch.nn.functional.silu(g) * u).to(torch.bfloat16)


def _prompt(m, x, res):
    n, _, ids, w, (off, row, slot) = _route(m, x, res)
    gu = fb.grouped_gemm(n["q"].view(torch.uint8), n["scale"], "1x128", *m["up8"], "1x32", off, row_index=row)
    aq, asc = fb.quantize(_silu(gu), "1x128")
    d = fb.grouped_gemm(aq.view(torch.uint8), asc, "1x128", *m["down8"], "1x32", off)
    return fb.moe_combine(d, slot, w, residual=n["h"]), (n, ids, w, off, row, slot, gu, d)


def _decode(m, x, res):
    n, _, ids, w, (off, row, slot) = _route(m, x, res)
    gu = fb.nvfp4_grouped_matvec(n["y"], *m["up4"], off, row_index=row)
    d = fb.nvfp4_grouped_matvec(_silu(gu), *m["down4"], off)
    return fb.moe_combine(d, slot, w, residual=n["h"]), (n, ids, w, off, row, slot, gu, d)


def _inputs(tokens, seed):
    return normal_bf16((tokens, H), 1.0, seed, "cuda"), normal_bf16((tokens, H), 2.0, seed + 1, "cuda")


def _layer_reference(n, ids, w, up, down):
    """The layer in float64 from the kernel's own h, normed rows, ids and weights (each tested by itself)."""
    x = bf16_to_f32(bf16_bits(n)).astype(np.float64)
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t].tolist()):
            gu = up[e] @ x[t]
            a = gu[:INTER] / (1 + np.exp(-gu[:INTER])) * gu[INTER:]
            y[t] += float(w[t, j]) * (down[e] @ a)
    return y


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("tokens", [1, 7, 150])
def test_prompt_layer(tokens):
    """FP8 codes of the activations carry half a step, 2^-4, per element at two places: the layer's output is within
    a fifth of the reference's norm (and a misplaced row would be off by all of it)."""
    m = _model(1)
    x, res = _inputs(tokens, 40)
    y, (n, ids, w, off, row, slot, gu, d) = _prompt(m, x, res)
    assert off[-1].item() == tokens * K and np.array_equal(slot.cpu().numpy(), moe.plan(ids.cpu().numpy(), E)[2])
    mats = {k: _f64(fb.dequantize(m[k + "8"][0].view(-1, m[k].shape[2]), m[k + "8"][1].view(-1, m[k].shape[2] // 32),
                                  "1x32")).reshape(m[k].shape) for k in ("up", "down")}
    want = _layer_reference(n["y"], ids, w, mats["up"], mats["down"])
    got = _f64(y) - _f64(n["h"])
    # the sum with h is rounded to bf16: half a step of |y|
    err = np.abs(got - want).clip(min=0) - 2.0 ** -8 * np.abs(_f64(y))
    assert np.linalg.norm(err.clip(min=0)) <= 0.2 * np.linalg.norm(want)


@pytest.mark.parametrize("tokens", [1, 2, 9])
def test_decode_layer(tokens):
    """bf16 activations between NVFP4 products: roundings of 2^-8 at three places (gate and up, their product, the
    experts' rows), so within 2^-5 of the norm."""
    m = _model(2)
    x, res = _inputs(tokens, 50)
    y, (n, ids, w, *_rest) = _decode(m, x, res)
    mats = {k: _f64(fb.nvfp4_dequantize(m[k + "4"][0].view(-1, m[k].shape[2] // 2),
                                        m[k + "4"][1].view(-1, m[k].shape[2] // 16), m[k + "4"][2],
                                        m[k].shape[1])).reshape(m[k].shape) for k in ("up", "down")}
    want = _layer_reference(n["y"], ids, w, mats["up"], mats["down"])
    err = np.abs(_f64(y) - _f64(n["h"]) - want) - 2.0 ** -8 * np.abs(_f64(y))
    # the dequantized reference weights are rounded to bf16 themselves: another 2^-8 at each product
    assert np.linalg.norm(err.clip(min=0)) <= 2.0 ** -5 * np.linalg.norm(want)


def test_a_token_decodes_as_in_the_batch():
    """Rows do not influence each other: a token alone gives the bytes it gives in a batch."""
    m = _model(3)
    x, res = _inputs(6, 60)
    whole, parts = _decode(m, x, res)
    for t in range(6):
        one, p1 = _decode(m, x[t:t + 1].contiguous(), res[t:t + 1].contiguous())
        assert torch.equal(p1[1], parts[1][t:t + 1]) and _same(p1[2], parts[2][t:t + 1])
        assert _same(one, whole[t:t + 1]), t


def test_padded_tokens():
    """Tokens whose logits are all masked are routed nowhere and leave with their residual."""
    m = _model(4)
    x, res = _inputs(10, 70)
    n = fb.rmsnorm_quantize(x, m["norm"], EPS, residual=res, normed=True)
    logits = n["y"].float() @ m["gate"].float().t()
    logits[[2, 9]] = -float("inf")
    ids, w = fb.moe_route(logits, K, bias=m["bias"], **ROUTE)
    off, row, slot = fb.moe_plan(ids, E)
    assert off[-1].item() == 8 * K and torch.all(slot[[2, 9]] == -1)
    gu = torch.full((10 * K, 2 * INTER), float("nan"), dtype=torch.bfloat16, device="cuda")
    fb.fp8_nvfp4_grouped_matvec(n["y"], row, *m["up4"], 2 * INTER, off, gu)
    assert torch.isnan(gu[8 * K:]).all() and torch.isfinite(gu[:8 * K]).all()       # rows behind the last stay
    d = torch.full((10 * K, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    fb.fp8_nvfp4_grouped_matvec(_silu(gu), None, *m["down4"], H, off, d)
    y = fb.moe_combine(d, slot, w, residual=n["h"])
    assert _same(y[[2, 9]], n["h"][[2, 9]]) and torch.isfinite(y.float()).all()


def _backward(m, x, res, dy):
    """Backward calls of one layer around the experts (whose own gradient is left to the caller): combination, weights
    to logits, logits and norm."""
    n, logits, ids, w, (off, row, slot) = _route(m, x, res)
    d = torch.arange(x.shape[0] * K, device="cuda")[:, None] % 7 + torch.arange(H, device="cuda") % 5
    d = d.to(torch.bfloat16)
    drows, dw = fb.moe_combine_backward(dy, d, slot, w)
    dl = fb.moe_route_backward(logits, ids, dw, score="sigmoid", renorm=True, scale=2.5)
    dyn = (dl[:, :, None] * m["gate"].float()[None]).sum(1).to(torch.bfloat16)
    dx, dg = fb.rmsnorm_backward(dyn, n["h"], m["norm"], n["rstd"], dres=dy)
    return drows, dw, dl, dx, dg


def test_training_step_against_autograd():
    """The chain of backward calls against autograd in double precision through the same choices.  Between the calls
    the router's gradient is rounded to bf16 (2^-8) and the norm's input gradient once more."""
    m = _model(5)
    tokens = 20
    x, res = _inputs(tokens, 80)
    dy = normal_bf16((tokens, H), 1e-2, 90, "cuda")
    drows, dw, dl, dx, dg = _backward(m, x, res, dy)
    n, _, ids, _, (off, row, slot) = _route(m, x, res)
    d = (torch.arange(tokens * K, device="cuda")[:, None] % 7 + torch.arange(H, device="cuda") % 5).double()
    d.requires_grad_(True)
    h = n["h"].double().requires_grad_(True)
    g = m["norm"].double().requires_grad_(True)
    yn = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * g
    s = torch.sigmoid((yn[:, None, :] * m["gate"].double()[None]).sum(-1)).gather(1, ids.long())
    w = 2.5 * s / s.sum(-1, keepdim=True)
    y = h + (d[slot.long().view(-1)].view(tokens, K, H) * w[..., None]).sum(1)
    gd, gh, gg = torch.autograd.grad(y, (d, h, g), dy.double())
    for got, want, tol in ((drows, gd, 2.0 ** -6), (dx, gh, 2.0 ** -6), (dg, gg, 2.0 ** -6)):
        assert (got.double() - want).norm() <= tol * want.norm()


@pytest.mark.parametrize("which", ["prompt", "decode", "backward"])
def test_captured_and_replayed(which):
    """A layer captured once gives the eager bytes on every replay, with eager work on other inputs in between."""
    m = _model(6)
    tokens = 5 if which == "decode" else 96
    x, res = _inputs(tokens, 100)
    dy = normal_bf16((tokens, H), 1e-2, 101, "cuda")

    def step():
        if which == "backward":
            return list(_backward(m, x, res, dy))
        y, parts = (_prompt if which == "prompt" else _decode)(m, x, res)
        return [y, parts[1], parts[2], parts[3], parts[4], parts[5]]

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(4):
        a, b = _inputs(tokens, 110 + 2 * i)
        x.copy_(a)
        res.copy_(b)
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        for j, (got, ref) in enumerate(zip(outs, want)):
            assert _same(got, ref), f"{which} replay {i}: output {j}"
        print(f"[moe layer] {which} replay {i}: {len(outs)} outputs equal the eager calls", flush=True)


def test_two_streams_at_once():
    """Two layers on two streams, given explicitly, against the same calls one after the other; results are
    allocated on the stream they were asked for."""
    m = _model(7)
    sets = [_inputs(64, 200), _inputs(64, 210)]
    want = [fb.rmsnorm_quantize(a, m["norm"], EPS, residual=b, normed=True) for a, b in sets]
    plans = [fb.moe_plan(fb.moe_route(w["y"].float() @ m["gate"].float().t(), K, **ROUTE)[0], E) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got, gp = [None, None], [None, None]
    logits = [w["y"].float() @ m["gate"].float().t() for w in want]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for rep in range(3):
        for i, s in enumerate(streams):
            a, b = sets[i]
            got[i] = fb.rmsnorm_quantize(a, m["norm"], EPS, residual=b, normed=True,
                                         stream=s if rep else s.cuda_stream)
            ids, _ = fb.moe_route(logits[i], K, **ROUTE, stream=s)
            gp[i] = fb.moe_plan(ids, E, stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(_same(got[i][k], want[i][k]) for k in ("q", "scale", "h", "y"))
        assert all(_same(p, q) for p, q in zip(gp[i], plans[i]))


def test_library_errors_reach_the_caller():
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fb.Fp8Error) as e:
        fb.rmsnorm_quantize(x, torch.ones(64, device="cuda"), EPS)                   # 64 columns, 1x128 tiles
    assert e.value.status == 2
    with pytest.raises(fb.Fp8Error) as e:
        fb.moe_route(torch.zeros((2, 8), device="cuda"), 4, groups=4, topk_groups=1)   # 2 experts left for 4 places
    assert e.value.status == 1
    flat = torch.zeros(2 * 128 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fb.Fp8Error) as e:
        fb.rmsnorm_quantize(flat[4:].view(2, 128), torch.ones(128, device="cuda"), EPS)   # 8-byte aligned
    assert e.value.status == 3
