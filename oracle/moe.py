"""The operators of a mixture-of-experts layer around the products (oracle).

TEST INFRASTRUCTURE ONLY (see the package docstring).  Everything is float64
numpy from the exact input values, written from the formulas; results are
unrounded unless a function says otherwise, and a test allows for the
kernel's own roundings.

  norm     h = RN_bf16(x + r), y = h / sqrt(mean h^2 + eps) * w, and its gradients
  route    scores, group-limited top-k, weights; gradients of the weights
  plan     stable sort of (token, choice) pairs by expert
  combine  weighted sum of the experts' rows, and its gradients
  matvec   x . W^T with NVFP4 W
"""

import numpy as np

from .codec import bf16_to_f32, e4m3_decode, f32_to_bf16
from .nvfp4 import e2m1_decode, unpack


# ------------------------------------------------------------------------ norm

def add_residual(x_bits, r_bits):
    """RN_bf16(x + r) as bf16 bits (the sum of two bf16 values rounded through float32: exact unless the exponents
    are more than 16 apart, and then the smaller value only breaks ties, as in the fp32 sum the kernel takes)."""
    return f32_to_bf16((bf16_to_f32(x_bits) + bf16_to_f32(r_bits)).astype(np.float32))


def rmsnorm(h, w, eps):
    """(y, rstd) in float64 from float64 h [R, C] and w [C]."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * w, rstd


def rmsnorm_backward(dy, h, w, rstd, dres=None):
    """(dx, dw) of y = h rstd(h) w, for the rstd given."""
    cols = h.shape[1]
    xh = h * rstd[:, None]
    wd = dy * w
    dx = rstd[:, None] * (wd - xh * ((wd * xh).sum(axis=1) / cols)[:, None])
    return dx + (0.0 if dres is None else dres), (dy * xh).sum(axis=0)


# --------------------------------------------------------------------- routing

def _clean(v):
    v = np.asarray(v, dtype=np.float64)
    v = np.where(np.isnan(v), -np.inf, v)
    return np.minimum(v, float(np.finfo(np.float32).max))


def scores(logits, score):
    """Scores of one token's cleaned logits; 0 where the logit is -inf."""
    out = np.zeros_like(logits)
    live = logits > -np.inf
    if not live.any():
        return out
    if score == "softmax":
        p = np.exp(logits[live] - logits[live].max())
        out[live] = p / p.sum()
    else:
        with np.errstate(over="ignore"):
            out[live] = 1.0 / (1.0 + np.exp(-logits[live]))
    return out


def chosen_weights(logits, ids, score, renorm, scale):
    """Weights of the listed experts of one token (cleaned logits)."""
    w = np.zeros(len(ids))
    ok = [j for j, e in enumerate(ids) if 0 <= e < len(logits) and logits[e] > -np.inf]
    if not ok:
        return w
    l = logits[[ids[j] for j in ok]]
    if not renorm:
        s = scores(logits, score)[[ids[j] for j in ok]]
    elif score == "softmax":
        s = np.exp(l - l.max())
    else:
        # log sigmoid, so that scores far below the double range keep their ratios
        ls = np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l)))
        s = np.exp(ls - ls.max())
    w[ok] = s / s.sum() if renorm else s
    return w * scale


def route(logits, bias, top_k, score, groups=1, topk_groups=1, group_score="max", renorm=False, scale=1.0):
    """(ids [T, k], weights [T, k]) by sorting each token's keys."""
    logits = _clean(logits)
    b = None if bias is None else _clean(bias)
    tokens, experts = logits.shape
    ids = np.full((tokens, top_k), -1, dtype=np.int32)
    weights = np.zeros((tokens, top_k))
    per = experts // groups
    for t in range(tokens):
        l = logits[t]
        s = scores(l, score)
        key = l.copy() if b is None else np.where((l > -np.inf) & (b > -np.inf), s + b, -np.inf)
        if groups > 1:
            rank = []
            for g in range(groups):
                ks = sorted((float(k), i) for i, k in enumerate(key[g * per:(g + 1) * per]) if k > -np.inf)
                best = [k if (b is not None or group_score == "max") else s[g * per + i] for k, i in ks[::-1][:2]]
                rank.append(-np.inf if not best else best[0] if group_score == "max" else sum(best))
            order = sorted(range(groups), key=lambda g: (-rank[g], g))[:topk_groups]
            keep = np.zeros(experts, dtype=bool)
            for g in order:
                keep[g * per:(g + 1) * per] = True
            key = np.where(keep, key, -np.inf)
        order = [e for e in sorted(range(experts), key=lambda e: (-key[e], e)) if key[e] > -np.inf][:top_k]
        ids[t, :len(order)] = order
        weights[t] = chosen_weights(l, ids[t].tolist(), score, renorm, scale)
    return ids, weights


def route_backward(logits, ids, dw, score, renorm, scale):
    """d logits [T, E] of sum(dw * weights), by the product rule over the chosen experts."""
    logits = _clean(logits)
    tokens, experts = logits.shape
    out = np.zeros((tokens, experts))
    for t in range(tokens):
        l = logits[t]
        s = scores(l, score)
        ok = [j for j, e in enumerate(ids[t]) if 0 <= e < experts and l[e] > -np.inf]
        if not ok:
            continue
        e = [int(ids[t, j]) for j in ok]
        g = dw[t, ok].astype(np.float64) * scale
        if renorm:
            p = chosen_weights(l, e, score, True, 1.0)
            d = p * (g - (g * p).sum())
            if score == "sigmoid":
                d = d * (1.0 / (1.0 + np.exp(np.minimum(l[e], 700.0))))
            np.add.at(out[t], e, d)
        elif score == "sigmoid":
            np.add.at(out[t], e, g * s[e] * (1.0 / (1.0 + np.exp(np.minimum(l[e], 700.0)))))
        else:
            np.add.at(out[t], e, g * s[e])
            out[t] -= s * (g * s[e]).sum()
    return out


def plan(ids, experts):
    """(offsets, row_index, slot) of the stable sort of the pairs by expert."""
    tokens, top_k = ids.shape
    flat = ids.reshape(-1)
    pairs = [p for e in range(experts) for p in np.flatnonzero(flat == e)]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(experts)])]).astype(np.int32)
    row_index = np.zeros(tokens * top_k, dtype=np.int32)
    slot = np.full(tokens * top_k, -1, dtype=np.int32)
    for r, p in enumerate(pairs):
        row_index[r] = p // top_k
        slot[p] = r
    return offsets, row_index, slot.reshape(tokens, top_k)


# ----------------------------------------------------------------- combination

def combine(rows, slot, weights, residual=None):
    tokens, top_k = slot.shape
    y = np.zeros((tokens, rows.shape[1])) if residual is None else residual.astype(np.float64).copy()
    for t in range(tokens):
        for j in range(top_k):
            if 0 <= slot[t, j] < rows.shape[0]:
                y[t] += float(weights[t, j]) * rows[slot[t, j]]
    return y


def combine_backward(dy, rows, slot, weights, drows):
    """(drows, dweights); rows no slot names keep what ``drows`` holds."""
    out = drows.astype(np.float64).copy()
    dw = np.zeros(slot.shape)
    for t in range(slot.shape[0]):
        for j in range(slot.shape[1]):
            s = slot[t, j]
            if 0 <= s < rows.shape[0]:
                out[s] = float(weights[t, j]) * dy[t]
                dw[t, j] = (dy[t] * rows[s]).sum()
    return out, dw


# ---------------------------------------------------------------------- matvec

def nvfp4_matrix(q, block_scale, global_scale, rows_per_tensor):
    """float64 [N, K] from packed codes [N, K/2], e4m3 scale codes [N, K/16] and tensor scales."""
    v = e2m1_decode(unpack(q)).astype(np.float64)
    s = np.repeat(e4m3_decode(block_scale).astype(np.float64), 16, axis=1)
    return v * s * np.repeat(np.asarray(global_scale, np.float64), rows_per_tensor)[:, None]


def grouped_matvec(x, row_index, mats, offsets, total_m):
    """Rows [off[g], off[g+1]) of x[row_index] times mats[g]^T; rows behind the last group are NaN.  Also the sums
    of absolute products, which a rounding bound is relative to."""
    n = mats[0].shape[0]
    y = np.full((total_m, n), np.nan)
    mag = np.full((total_m, n), np.nan)
    for g, w in enumerate(mats):
        r = np.arange(offsets[g], offsets[g + 1])
        xr = x[r if row_index is None else row_index[r]]
        y[r] = xr @ w.T
        mag[r] = np.abs(xr) @ np.abs(w).T
    return y, mag
