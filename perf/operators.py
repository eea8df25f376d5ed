"""The operators of a mixture-of-experts layer around the FP8 and FP4 products, as measured cases.

Four operators, each with its directions:
  norm     residual addition, root-mean-square norm and FP8 codes with block scales (and its backward pass);
  route    expert selection and weights, then the offsets, row index and slots that the grouped products take
           (and the gradient of the weights with respect to the logits);
  matvec   products of a few bf16 rows with NVFP4 weights, dense and grouped over experts;
  combine  the weighted sum of the experts' rows back into tokens (and its backward pass).

``own`` false: ``run`` computes the plain form from elementary torch operations.  ``own`` true: ``run`` calls the
library's entry points on the buffers that ``prepare`` made, as a serving or training loop does.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
E4M3_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a single decoded token between two layers: residual stream, codes for the experts, bf16 for the router
        {"name": "norm one token", "op": "norm", "rows": 1, "cols": 7168, "block": "1x128", "residual": True,
         "weight": "f32", "y": True, "dq": False, "rstd": False},
        # a long prompt (or a training batch without recomputation) at the benchmark's token count and hidden size
        {"name": "norm prompt", "op": "norm", "rows": 16384, "cols": 7168, "block": "1x128", "residual": True,
         "weight": "f32", "y": True, "dq": False, "rstd": False},
        # training forward with MXFP8 activations, ragged rows, an odd number of blocks, bf16 weights
        {"name": "norm mxfp8 odd", "op": "norm", "rows": 997, "cols": 5152, "block": "1x32", "residual": False,
         "weight": "bf16", "y": False, "dq": True, "rstd": True},
        # quantization-aware training: gradients of the norm's input and weight at the benchmark's QAT size
        {"name": "norm backward", "op": "norm_backward", "rows": 8192, "cols": 7168, "residual": True,
         "weight": "f32"},
        # one decoded token: sigmoid scores, a balance bias, group-limited choice of 8 among 256 experts
        {"name": "route one token", "op": "route", "tokens": 1, "experts": 256, "top_k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "group_score": "top2", "renorm": True, "logits": "f32"},
        # the same for a prompt of the benchmark's token count
        {"name": "route prompt", "op": "route", "tokens": 16384, "experts": 256, "top_k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "group_score": "top2", "renorm": True, "logits": "f32"},
        # training: gradient of softmax weights, an odd token count, experts that do not fill the wave
        {"name": "route backward odd", "op": "route_backward", "tokens": 4099, "experts": 160, "top_k": 6,
         "score": "softmax", "renorm": False, "logits": "bf16"},
        # one decoded token through one FP4 projection (gate and up rows of one expert, or a dense layer)
        {"name": "matvec one token", "op": "matvec", "m": 1, "n": 4096, "k": 7168, "out": "bf16"},
        # a small odd batch, rows whose bytes are only 8-byte aligned, fp32 out
        {"name": "matvec batch odd", "op": "matvec", "m": 13, "n": 2000, "k": 7184, "out": "f32"},
        # eight decoded tokens through the gate and up rows of their experts: 64 rows on 52 of 256 experts
        {"name": "experts decode", "op": "experts", "rows": 64, "active": 52, "experts": 256, "top_k": 8, "n": 4096,
         "k": 7168, "out": "bf16"},
        # the end of the layer for a prompt: eight expert rows per token, added to the residual stream
        {"name": "combine prompt", "op": "combine", "tokens": 16384, "top_k": 8, "n": 7168, "residual": True},
        # its backward pass for an odd number of tokens
        {"name": "combine backward odd", "op": "combine_backward", "tokens": 4093, "top_k": 8, "n": 7168},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "route", "route", "route_backward", "matvec", "matvec",
                     "experts", "combine", "combine_backward"])
    if op in ("norm", "norm_backward"):
        block = rng.choice(["1x128", "1x32"])
        step = 128 if block == "1x128" else 32
        cols = step * _log_int(rng, max(1, 512 // step), 16384 // step)
        rows = _log_int(rng, 1, max(1, min(16384, 16384 * 7168 // cols)))
        c = {"op": op, "rows": rows, "cols": cols, "residual": rng.random() < 0.7,
             "weight": rng.choice(["f32", "bf16"])}
        if op == "norm":
            c.update(block=block, y=rng.random() < 0.5, dq=rng.random() < 0.3, rstd=rng.random() < 0.5)
        else:
            c["rows"] = max(1, rows // 2)
        return c
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.randint(4, 32)
        experts = groups * per
        topk_groups = rng.randint(1, groups)
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "experts": experts,
                "top_k": rng.randint(1, min(8, per * topk_groups)), "score": rng.choice(["sigmoid", "softmax"]),
                "bias": rng.random() < 0.5, "groups": groups, "topk_groups": topk_groups,
                "group_score": rng.choice(["max", "top2"]), "renorm": rng.random() < 0.6,
                "logits": rng.choice(["f32", "bf16"])}
    if op == "route_backward":
        experts = rng.randint(8, 256)
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "experts": experts, "top_k": rng.randint(1, 8),
                "score": rng.choice(["sigmoid", "softmax"]), "renorm": rng.random() < 0.6,
                "logits": rng.choice(["f32", "bf16"])}
    if op == "matvec":
        k = 16 * _log_int(rng, 32, 512)
        return {"op": op, "m": _log_int(rng, 1, 32), "n": _log_int(rng, 256, 8192), "k": k,
                "out": rng.choice(["bf16", "f32"])}
    if op == "experts":
        experts = rng.randint(8, 256)
        top_k = rng.randint(1, 8)
        rows = top_k * rng.randint(1, 8)
        active = rng.randint(1, min(rows, experts, 52))
        return {"op": op, "rows": rows, "active": active, "experts": experts, "top_k": top_k,
                "n": 16 * _log_int(rng, 16, 256), "k": 32 * _log_int(rng, 16, 224), "out": rng.choice(["bf16", "f32"])}
    top_k = rng.randint(1, 8)
    n = 8 * _log_int(rng, 64, 896)
    tokens = _log_int(rng, 1, 16384 if op == "combine" else 4093)
    c = {"op": op, "tokens": tokens, "top_k": top_k, "n": n}
    if op == "combine":
        c["residual"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, rows, cols, sigma=1.0):
    """bf16 activations with a hundredth of the channels fifty times as large."""
    x = _normal(g, rows, cols) * sigma
    hot = torch.randperm(cols, generator=g, device=DEV)[: max(1, cols // 100)]
    x[:, hot] *= 50.0
    return x.to(torch.bfloat16)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _fp4_rows(g, rows, k):
    """Rows of normal weights in NVFP4 for a tensor scale of 1: packed codes and e4m3 block scales as bytes."""
    w = _normal(g, rows, k // 16, 16)
    s = (w.abs().amax(-1) * (448.0 / 6.0 / 4.5)).clamp(max=448.0).to(torch.float8_e4m3fn)
    v = w / (s.float()[..., None] * (4.5 / 448.0))
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(v.abs(), mid).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    code = code.view(rows, k // 2, 2)
    return (code[..., 0] | (code[..., 1] << 4)).contiguous(), s.view(torch.uint8)


def _weights(g, count, n, k):
    """`count` stacked [n, k] matrices, their rows drawn from a pool of quantized ones; a tensor scale each."""
    pool = min(count * n, 4096)
    q, s = _fp4_rows(g, pool, k)
    if count * n > pool:
        at = torch.randint(0, pool, (count * n,), generator=g, device=DEV)
        q, s = q[at], s[at]
    spread = torch.exp(torch.rand(count, generator=g, device=DEV) * 1.386 - 0.693)
    return q.view(count, n, k // 2), s.view(count, n, k // 16), (0.02 * 4.5 / 448.0) * spread


def _slots(g, tokens, top_k):
    """A row of the experts' output for each (token, choice): every row once, in an order as after routing."""
    return torch.randperm(tokens * top_k, generator=g, device=DEV).to(torch.int32).view(tokens, top_k)


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    s = {"case": c}
    if op == "norm":
        rows, cols = c["rows"], c["cols"]
        s["x"] = _activations(g, rows, cols)
        s["res"] = (4.0 * _normal(g, rows, cols)).to(torch.bfloat16) if c["residual"] else None
        s["w"] = (1.0 + 0.1 * _normal(g, cols)).to(_dtype(c["weight"]))
        s["q"] = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=DEV)
        mx = c["block"] == "1x32"
        s["scale"] = torch.empty((rows, cols // (32 if mx else 128)), dtype=torch.uint8 if mx else torch.float32,
                                 device=DEV)
        s["h"] = torch.empty_like(s["x"]) if c["residual"] else None
        s["y"] = torch.empty_like(s["x"]) if c["y"] else None
        s["ydq"] = torch.empty_like(s["x"]) if c["dq"] else None
        s["rstd"] = torch.empty((rows,), dtype=torch.float32, device=DEV) if c["rstd"] else None
    elif op == "norm_backward":
        rows, cols = c["rows"], c["cols"]
        s["h"] = _activations(g, rows, cols)
        s["dy"] = (1e-3 * _normal(g, rows, cols)).to(torch.bfloat16)
        s["dres"] = (1e-3 * _normal(g, rows, cols)).to(torch.bfloat16) if c["residual"] else None
        s["w"] = (1.0 + 0.1 * _normal(g, cols)).to(_dtype(c["weight"]))
        s["rstd"] = (s["h"].double().square().mean(-1) + EPS).rsqrt().float()
        s["dx"] = torch.empty_like(s["h"])
        s["dw"] = torch.empty((cols,), dtype=_dtype(c["weight"]), device=DEV)
    elif op in ("route", "route_backward"):
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        s["logits"] = (1.5 * _normal(g, t, e)).to(_dtype(c["logits"]))
        if op == "route":
            s["bias"] = 0.1 * _normal(g, e) if c["bias"] else None
            s["ids"] = torch.empty((t, k), dtype=torch.int32, device=DEV)
            s["weights"] = torch.empty((t, k), dtype=torch.float32, device=DEV)
            s["offsets"] = torch.empty((e + 1,), dtype=torch.int32, device=DEV)
            s["row_index"] = torch.empty((t * k,), dtype=torch.int32, device=DEV)
            s["slot"] = torch.empty((t, k), dtype=torch.int32, device=DEV)
        else:
            s["ids"] = s["logits"].float().topk(k, dim=-1).indices.to(torch.int32)
            s["dweights"] = 1e-2 * _normal(g, t, k)
            s["dlogits"] = torch.empty_like(s["logits"])
    elif op == "matvec":
        s["x"] = _activations(g, c["m"], c["k"])
        q, bs, gs = _weights(g, 1, c["n"], c["k"])
        s["q"], s["bs"], s["gs"] = q[0], bs[0], gs
        s["out"] = torch.empty((c["m"], c["n"]), dtype=_dtype(c["out"]), device=DEV)
    elif op == "experts":
        s["x"] = _activations(g, c["rows"] // c["top_k"], c["k"])
        s["q"], s["bs"], s["gs"] = _weights(g, c["experts"], c["n"], c["k"])
        chosen = torch.randperm(c["experts"], generator=g, device=DEV)[: c["active"]]
        more = torch.randint(0, c["active"], (c["rows"] - c["active"],), generator=g, device=DEV)
        of_row = torch.sort(torch.cat([chosen, chosen[more]])).values
        s["offsets"] = torch.searchsorted(of_row, torch.arange(c["experts"] + 1, device=DEV)).to(torch.int32)
        s["row_index"] = (torch.randperm(c["rows"], generator=g, device=DEV) // c["top_k"]).to(torch.int32)
        s["out"] = torch.empty((c["rows"], c["n"]), dtype=_dtype(c["out"]), device=DEV)
    else:
        t, k, n = c["tokens"], c["top_k"], c["n"]
        s["rows"] = _normal(g, t * k, n).to(torch.bfloat16)
        s["slot"] = _slots(g, t, k)
        w = torch.rand((t, k), generator=g, device=DEV) + 0.05
        s["weights"] = 2.5 * w / w.sum(-1, keepdim=True)
        if op == "combine":
            s["res"] = (4.0 * _normal(g, t, n)).to(torch.bfloat16) if c["residual"] else None
            s["out"] = torch.empty((t, n), dtype=torch.bfloat16, device=DEV)
        else:
            s["dy"] = (1e-3 * _normal(g, t, n)).to(torch.bfloat16)
            s["drows"] = torch.empty_like(s["rows"])
            s["dweights"] = torch.empty((t, k), dtype=torch.float32, device=DEV)
    return s


# ----------------------------------------------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


def _run_own(s):
    import block_scaled_fp8_amax_amd as fb
    c = s["case"]
    op = c["op"]
    if op == "norm":
        fb.fp8_rmsnorm_quantize(s["x"], s["w"], EPS, c["block"], "ceil", s["q"], s["scale"], residual=s["res"],
                                h=s["h"], y=s["y"], ydq=s["ydq"], rstd=s["rstd"])
        scale = s["scale"].view(torch.float8_e8m0fnu) if c["block"] == "1x32" else s["scale"]
        return {"q": s["q"], "scale": scale, "h": s["h"], "y": s["y"], "ydq": s["ydq"], "rstd": s["rstd"]}
    if op == "norm_backward":
        if "workspace" not in s:
            s["workspace"] = torch.empty(fb.fp8_rmsnorm_backward_workspace(c["rows"], c["cols"]), dtype=torch.uint8,
                                         device=DEV)
        fb.fp8_rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], s["workspace"], s["dx"], s["dw"], dres=s["dres"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "route":
        if "workspace" not in s:
            s["workspace"] = torch.empty(fb.fp8_moe_plan_workspace(c["tokens"], c["top_k"], c["experts"]),
                                         dtype=torch.uint8, device=DEV)
        fb.fp8_moe_route(s["logits"], s["ids"], s["weights"], bias=s["bias"], score=c["score"], groups=c["groups"],
                         topk_groups=c["topk_groups"], group_score=c["group_score"], renorm=c["renorm"], scale=2.5)
        fb.fp8_moe_plan(s["ids"], c["experts"], s["workspace"], s["offsets"], s["row_index"], s["slot"])
        return {"ids": s["ids"], "weights": s["weights"], "offsets": s["offsets"], "row_index": s["row_index"],
                "slot": s["slot"]}
    if op == "route_backward":
        fb.fp8_moe_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], score=c["score"],
                                  renorm=c["renorm"], scale=2.5)
        return s["dlogits"]
    if op == "matvec":
        fb.fp8_nvfp4_matvec(s["x"], s["q"], s["bs"], s["gs"], c["n"], s["out"])
        return s["out"]
    if op == "experts":
        fb.fp8_nvfp4_grouped_matvec(s["x"], s["row_index"], s["q"], s["bs"], s["gs"], c["n"], s["offsets"], s["out"])
        return s["out"]
    if op == "combine":
        fb.fp8_moe_combine(s["rows"], s["slot"], s["weights"], s["out"], residual=s["res"])
        return s["out"]
    fb.fp8_moe_combine_backward(s["dy"], s["rows"], s["slot"], s["weights"], s["drows"], s["dweights"])
    return {"drows": s["drows"], "dweights": s["dweights"]}


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    h = (x + s["res"].float()).to(torch.bfloat16) if c["residual"] else None
    hf = h.float() if c["residual"] else x
    rstd = 1.0 / torch.sqrt((hf * hf).mean(-1) + EPS)
    y = hf * rstd[:, None] * s["w"].float()
    blk = 32 if c["block"] == "1x32" else 128
    yb = y.view(c["rows"], -1, blk)
    amax = yb.abs().amax(-1)
    if blk == 128:
        scale = amax / E4M3_MAX
        v = torch.where(scale[..., None] > 0, yb / scale[..., None], torch.zeros_like(yb))
        sv, held = scale, scale
    else:
        m, e = torch.frexp(amax / E4M3_MAX)          # smallest X with amax <= 448 2^X
        x2 = torch.where(m > 0.5, e, e - 1).clamp(-127, 127)
        x2 = torch.where(amax > 0, x2, torch.full_like(x2, -127))
        v = torch.ldexp(yb, -x2[..., None])
        sv = torch.ldexp(torch.ones_like(amax), x2)
        held = (x2 + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    q = v.to(torch.float8_e4m3fn)
    return {"q": q.view(c["rows"], c["cols"]), "scale": held, "h": h,
            "y": y.to(torch.bfloat16) if c["y"] else None,
            "ydq": (q.float() * sv[..., None]).to(torch.bfloat16).view(c["rows"], c["cols"]) if c["dq"] else None,
            "rstd": rstd if c["rstd"] else None}


def _plain_norm_backward(s):
    xh = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    wd = dy * s["w"].float()
    dx = s["rstd"][:, None] * (wd - xh * (wd * xh).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * xh).sum(0).to(s["w"].dtype)}


def _plain_route(s):
    # choices between experts are made in 64 bits: the scores of two experts can be closer than 32 bits tell apart
    c = s["case"]
    t, e, k, groups = c["tokens"], c["experts"], c["top_k"], c["groups"]
    logit = s["logits"].double()
    score = 1.0 / (1.0 + torch.exp(-logit)) if c["score"] == "sigmoid" else _softmax(logit)
    key = score + s["bias"].double() if c["bias"] else logit
    summed = key if c["bias"] else score
    if groups > 1:
        if c["group_score"] == "top2":
            per = summed.view(t, groups, e // groups).sort(dim=-1, descending=True).values[..., :2].sum(-1)
        else:
            per = key.view(t, groups, e // groups).amax(-1)
        best = per.sort(dim=-1, descending=True, stable=True).indices[:, : c["topk_groups"]]
        keep = torch.zeros((t, groups), dtype=torch.bool, device=logit.device).scatter_(1, best, True)
        key = torch.where(keep.repeat_interleave(e // groups, 1), key, torch.full_like(key, -math.inf))
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, :k].contiguous()
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    flat = ids.view(-1)
    by_expert, order = flat.sort(dim=0, stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(e + 1, device=flat.device)).to(torch.int32)
    slot = torch.empty_like(order).scatter_(0, order, torch.arange(t * k, device=flat.device))
    return {"ids": ids.to(torch.int32), "weights": (2.5 * w).float(), "offsets": offsets,
            "row_index": (order // k).to(torch.int32), "slot": slot.view(t, k).to(torch.int32)}


def _softmax(x):
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_route_backward(s):
    c = s["case"]
    logit, ids, g = s["logits"].float(), s["ids"].long(), 2.5 * s["dweights"]
    score = 1.0 / (1.0 + torch.exp(-logit)) if c["score"] == "sigmoid" else _softmax(logit)
    chosen = score.gather(1, ids)
    if c["renorm"]:
        total = chosen.sum(-1, keepdim=True)
        g = (g - (g * chosen).sum(-1, keepdim=True) / total) / total
    dscore = torch.zeros_like(score).scatter_add_(1, ids, g)
    if c["score"] == "sigmoid":
        d = dscore * score * (1.0 - score)
    else:
        d = score * (dscore - (dscore * score).sum(-1, keepdim=True))
    return d.to(s["logits"].dtype)


def _decode(q, bs, gs):
    """NVFP4 bytes [..., n, k/2], block scale bytes [..., n, k/16] and tensor scales [...] as fp32 [..., n, k]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=q.device)
    v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], -1)
    v = v.view(*q.shape[:-1], q.shape[-1] // 8, 16) * bs.view(torch.float8_e4m3fn).float()[..., None]
    return v.view(*q.shape[:-1], 2 * q.shape[-1]) * gs[..., None, None]


def _plain_matvec(s):
    w = _decode(s["q"], s["bs"], s["gs"][0])
    return (s["x"].float() @ w.t()).to(s["out"].dtype)


def _plain_experts(s):
    c = s["case"]
    of_row = torch.searchsorted(s["offsets"], torch.arange(c["rows"], dtype=torch.int32, device=DEV), right=True) - 1
    w = _decode(s["q"][of_row], s["bs"][of_row], s["gs"][of_row])
    x = s["x"][s["row_index"].long()].float()
    return torch.bmm(w, x[:, :, None])[..., 0].to(s["out"].dtype)


def _plain_combine(s):
    c = s["case"]
    rows = s["rows"][s["slot"].long().view(-1)].view(c["tokens"], c["top_k"], c["n"])
    y = (rows.float() * s["weights"][..., None]).sum(1)
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(torch.bfloat16)


def _plain_combine_backward(s):
    c = s["case"]
    dy, at = s["dy"].float(), s["slot"].long().view(-1)
    rows = s["rows"][at].view(c["tokens"], c["top_k"], c["n"]).float()
    drows = torch.empty_like(s["rows"])
    drows[at] = (s["weights"][..., None] * dy[:, None]).to(torch.bfloat16).view(-1, c["n"])
    return {"drows": drows, "dweights": (rows * dy[:, None]).sum(-1)}


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "route": _plain_route,
          "route_backward": _plain_route_backward, "matvec": _plain_matvec, "experts": _plain_experts,
          "combine": _plain_combine, "combine_backward": _plain_combine_backward}


# ------------------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    op = c["op"]
    if op == "norm":
        n = c["rows"] * c["cols"]
        blk, sb = (32, 1) if c["block"] == "1x32" else (128, 4)
        per = 2 + 1 + sb / blk + (4 if c["residual"] else 0) + (2 if c["y"] else 0) + (2 if c["dq"] else 0)
        wb = c["cols"] * (4 if c["weight"] == "f32" else 2)
        return {"bytes": n * per + wb + (4 * c["rows"] if c["rstd"] else 0), "flops": 8 * n}
    if op == "norm_backward":
        n = c["rows"] * c["cols"]
        wb = c["cols"] * (4 if c["weight"] == "f32" else 2)
        return {"bytes": n * (6 + (2 if c["residual"] else 0)) + 2 * wb + 4 * c["rows"], "flops": 11 * n}
    if op == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        b = t * e * (4 if c["logits"] == "f32" else 2) + t * k * 16 + 4 * (e + 1) + (4 * e if c["bias"] else 0)
        return {"bytes": b, "flops": t * e * 4}
    if op == "route_backward":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        return {"bytes": 2 * t * e * (4 if c["logits"] == "f32" else 2) + t * k * 8, "flops": t * e * 6}
    if op in ("matvec", "experts"):
        m, x_rows, mats = (c["m"], c["m"], 1) if op == "matvec" else (c["rows"], c["rows"] // c["top_k"], c["active"])
        out = 4 if c["out"] == "f32" else 2
        b = mats * (c["n"] * (c["k"] / 2 + c["k"] / 16) + 4) + x_rows * c["k"] * 2 + m * c["n"] * out
        if op == "experts":
            b += 4 * (c["experts"] + 1) + 4 * c["rows"]
        return {"bytes": b, "flops": 2 * m * c["n"] * c["k"]}
    t, k, n = c["tokens"], c["top_k"], c["n"]
    if op == "combine":
        return {"bytes": t * k * n * 2 + t * n * (4 if c["residual"] else 2) + t * k * 8, "flops": 2 * t * k * n}
    return {"bytes": 2 * t * k * n * 2 + t * n * 2 + t * k * 12, "flops": 3 * t * k * n}


# ------------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What ``run`` returns before its roundings to the outputs' types, in 64 bits.  FP8 codes are given as the
    quotient that the code is the nearest value to; an E8M0 scale is a choice between powers of two and has none."""
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _exact_norm(s, c):
    h = s["x"].double()
    if c["residual"]:
        h = (h + s["res"].double()).to(torch.bfloat16).double()
    r = (h.pow(2).sum(1) / c["cols"] + EPS).pow(-0.5)
    y = torch.einsum("ij,i,j->ij", h, r, s["w"].double())
    blk = 32 if c["block"] == "1x32" else 128
    tiles = y.reshape(c["rows"], c["cols"] // blk, blk)
    top = tiles.abs().max(2).values
    if blk == 128:
        unit = top / E4M3_MAX
    else:
        unit = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp(-127, 127))
    q = (tiles / unit[:, :, None]).nan_to_num(0.0, 0.0, 0.0).reshape(c["rows"], c["cols"])
    # the fake-quantized values have no value beside the codes' own rounding
    return {"q": q, "scale": unit if blk == 128 else None, "h": h if c["residual"] else None,
            "y": y if c["y"] else None, "ydq": None, "rstd": r if c["rstd"] else None}


def _exact_norm_backward(s, c):
    h, dy, w, r = s["h"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()
    proj = (dy * w * h).sum(1)
    dx = r[:, None] * dy * w - h * (r.pow(3) * proj / c["cols"])[:, None]
    if c["residual"]:
        dx = dx + s["dres"].double()
    return {"dx": dx, "dw": ((dy * h) * r[:, None]).sum(0)}


def _exact_route(s, c):
    x = s["logits"].double()
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
    rank = p + s["bias"].double() if c["bias"] else x
    if c["groups"] > 1:
        n = c["experts"] // c["groups"]
        if c["group_score"] == "top2":
            of = (rank if c["bias"] else p).unflatten(1, (c["groups"], n)).topk(min(2, n), 2).values.sum(2)
        else:
            of = rank.unflatten(1, (c["groups"], n)).max(2).values
        # a group stays if fewer than topk_groups are better, or equal and before it
        place = torch.arange(c["groups"], device=DEV)
        before = (of[:, None, :] > of[:, :, None]) | ((of[:, None, :] == of[:, :, None]) & (place[None, :] < place[:, None]))
        out = (before.sum(2) >= c["topk_groups"]).repeat_interleave(n, 1)
        rank = rank.masked_fill(out, -math.inf)
    ids = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, : c["top_k"]]
    w = torch.gather(p, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": None, "weights": 2.5 * w, "offsets": None, "row_index": None, "slot": None}


def _exact_route_backward(s, c):
    x = s["logits"].double().requires_grad_(True)
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
    w = torch.gather(p, 1, s["ids"].long())
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return torch.autograd.grad((2.5 * w * s["dweights"].double()).sum(), x)[0]


def _exact_matrix(q, bs, g):
    sign = 1.0 - 2.0 * ((q >> 3) & 1).double()
    e, m = ((q >> 1) & 3).double(), (q & 1).double()
    v = sign * torch.where(e > 0, torch.exp2(e - 1.0) * (1.0 + 0.5 * m), 0.5 * m)
    return v * bs.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * g.double()


def _nibbles(q):
    out = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.uint8, device=q.device)
    out[:, 0::2] = q & 0x0F
    out[:, 1::2] = q >> 4
    return out


def _exact_matvec(s, c):
    return s["x"].double() @ _exact_matrix(_nibbles(s["q"]), s["bs"], s["gs"][0]).T


def _exact_experts(s, c):
    out = torch.zeros((c["rows"], c["n"]), dtype=torch.float64, device=DEV)
    off = s["offsets"].tolist()
    for e in range(c["experts"]):
        if off[e + 1] > off[e]:
            x = s["x"][s["row_index"][off[e]:off[e + 1]].long()].double()
            out[off[e]:off[e + 1]] = x @ _exact_matrix(_nibbles(s["q"][e]), s["bs"][e], s["gs"][e]).T
    return out


def _exact_combine(s, c):
    y = s["res"].double() if c["residual"] else torch.zeros((c["tokens"], c["n"]), dtype=torch.float64, device=DEV)
    for j in range(c["top_k"]):
        y = y + s["weights"][:, j:j + 1].double() * s["rows"][s["slot"][:, j].long()].double()
    return y


def _exact_combine_backward(s, c):
    drows = torch.zeros((c["tokens"] * c["top_k"], c["n"]), dtype=torch.float64, device=DEV)
    dw = torch.zeros((c["tokens"], c["top_k"]), dtype=torch.float64, device=DEV)
    dy = s["dy"].double()
    for j in range(c["top_k"]):
        at = s["slot"][:, j].long()
        drows[at] = s["weights"][:, j:j + 1].double() * dy
        dw[:, j] = (s["rows"][at].double() * dy).sum(1)
    return {"drows": drows, "dweights": dw}


_EXACT = {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "route": _exact_route,
          "route_backward": _exact_route_backward, "matvec": _exact_matvec, "experts": _exact_experts,
          "combine": _exact_combine, "combine_backward": _exact_combine_backward}
