"""The layer operators' definitions in 64 bits (numpy), and bounds on how far
an fp32 computation rounded once may be from them.

u is the unit roundoff: 2^-24 for fp32, 2^-8 for bf16, 2^-11 for fp16.  A sum
of n terms in any order of fp32 additions is within n u of the sum of the
terms' magnitudes; the bounds below add that to the roundings of the products
and of the final store.
"""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}  # spacing of subnormals
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def store_bound(x, dt):
    return UNIT[dt] * np.abs(x) + LEAST[dt]


def norm(send, residual, weight, eps):
    """send (N, N*rows, H), residual (N, rows, H) or None, weight (N, H), all
    float64 -> h, rstd, y and bounds of the fp32 computation (before the store)."""
    N, T, H = send.shape
    parts = send.reshape(N, N, T // N, H)
    h = parts.sum(0)
    mag = np.abs(parts).sum(0)
    if residual is not None:
        h = h + residual
        mag = mag + np.abs(residual)
    dh = (N + 2) * U32 * mag
    ms = (h * h).mean(-1, keepdims=True)
    # a thread adds at most 64 squares (96 where a row is taken element by element), then ten levels
    dms = (2 * np.abs(h) * dh + dh * dh).mean(-1, keepdims=True) + 128 * U32 * ms
    rstd = 1 / np.sqrt(ms + eps)
    rel = 0.5 * dms / (ms + eps) * (1 + dms / (ms + eps)) + 6 * U32
    y = h * rstd * weight[:, None, :]
    dy = np.abs(y) * (rel + 4 * U32) + dh * rstd * np.abs(weight[:, None, :])
    return h, rstd[..., 0], y, dh, (rel * rstd)[..., 0], dy


def norm_grad(dout, dres, h, weight, rstd):
    """-> dh, dweight and their bounds; rstd (N, rows)."""
    H = h.shape[-1]
    rs = rstd[..., None]
    g = dout * weight[:, None, :]
    mean = (g * h).mean(-1, keepdims=True)
    dh = rs * (g - h * rs * rs * mean)
    bound = 8 * U32 * rs * np.abs(g) + (128 + 16) * U32 * rs ** 3 * np.abs(h) * np.abs(g * h).mean(-1, keepdims=True)
    bound = bound + 4 * U32 * np.abs(dh)
    if dres is not None:
        dh = dh + dres
        bound = bound + U32 * (np.abs(dres) + np.abs(dh))
    terms = dout * h * rs
    dw = terms.sum(1)
    dw_bound = (h.shape[1] + 20) * U32 * np.abs(terms).sum(1)
    return dh, dw, bound, dw_bound


def scores(l, score):
    """Scores of one row of logits; 0 where a logit is -inf or NaN."""
    there = l > -np.inf
    s = np.zeros_like(l)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s[there] = 1 / (1 + np.exp(-l[there]))
    elif there.any():
        m = l[there].max()
        e = np.array([1.0 if x == m else np.exp(x - m) for x in l[there]])
        s[there] = e / e.sum()
    return s, there


def route_row(l, bias, score, topk, ngroups, keep, top, renorm, scale):
    """One token: ids, weights, and the least gap between two neighbours whose
    order decides, in parts of what each was added up from."""
    s, there = scores(l, score)
    by = s if bias is not None or (ngroups > 1 and top == 2) else l
    c = np.where(there, by + (0 if bias is None else bias), -np.inf)
    c = np.where(c > -np.inf, c, -np.inf)
    size = s + (0 if bias is None else np.abs(bias))
    gap = np.inf
    E = len(l)

    def least(order, v, of):
        # equal things (of equal inputs) tie in fp32 too: their order is by index
        order = [i for i in order if np.isfinite(v[i])]
        return min([(v[a] - v[b]) / max(of[a], of[b], 1e-300) for a, b in zip(order, order[1:]) if v[a] != v[b]],
                   default=np.inf)

    if ngroups > 1:
        each = E // ngroups
        worth, of = np.full(ngroups, -np.inf), np.zeros(ngroups)
        for g in range(ngroups):
            best = np.sort(c[g * each:(g + 1) * each])[::-1]
            best = best[best > -np.inf][:top]
            if len(best):
                worth[g], of[g] = best.sum(), top * size[g * each:(g + 1) * each].max()
        order = sorted(range(ngroups), key=lambda g: (-worth[g], g))
        gap = least(order[keep - 1:keep + 1], worth, of)
        for g in order[keep:]:
            c[g * each:(g + 1) * each] = -np.inf
    order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -np.inf]
    gap = min(gap, least(order[:topk + 1], c, size))
    order = order[:topk]
    ids = np.full(topk, -1, np.int32)
    w = np.zeros(topk)
    ids[:len(order)] = order
    w[:len(order)] = s[order]
    if renorm:
        w = w / max(w.sum(), 2.0 ** -126)
    return ids, w * scale, gap


def route_weights(l, ids, score, renorm, scale):
    """Weights of given choices, a differentiable function of the logits."""
    s, _ = scores(l, score)
    w = np.where(ids >= 0, s[np.maximum(ids, 0)], 0.0)
    if renorm and w.sum() > 0:
        w = w / w.sum()
    return w * scale


def plan(ids, E, cap):
    """ids (N, rows, k) -> slots, offsets, written out as the definition reads."""
    N, rows, k = ids.shape
    each = E // N
    slots = np.full(ids.shape, -1, np.int32)
    offsets = np.zeros((N, each + 1), np.int32)
    flat = ids.reshape(-1)
    for d in range(N):
        row = 0
        for i in range(each):
            offsets[d, i] = min(row, cap)
            at = np.nonzero(flat == d * each + i)[0]
            to = row + np.arange(len(at))
            slots.reshape(-1)[at] = np.where(to < cap, d * cap + to, -1)
            row += len(at)
        offsets[d, each] = min(row, cap)
    return slots, offsets
