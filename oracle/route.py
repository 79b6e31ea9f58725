"""Reference routing of tokens to experts, in float64.  TEST INFRASTRUCTURE ONLY.

The definition, one token at a time and with plain sorts:

* an expert is eligible unless its logit is NaN or -inf (+inf counts as the largest finite
  float32), and with a bias unless its bias is NaN or -inf;
* score = softmax over the experts with an eligible logit, or the logistic function;
* choice value = score + bias; without a bias experts compare by their logits;
* groups are equal runs of experts, valued by their best choice value or the sum of their two
  best (of scores where there is no bias); experts outside the best groups are not eligible;
* the topk largest choice values in descending order, ties to the lowest index, -1 where there are
  too few; weights are the chosen scores, renormalized if asked, times a constant.
"""
from __future__ import annotations

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def scores(logits, scoring: str) -> np.ndarray:
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isposinf(l), FLT_MAX, l)
    out = np.zeros_like(l)
    ok = ~np.isnan(l) & (l > -np.inf)
    if not ok.any():
        return out
    with np.errstate(over="ignore", under="ignore"):
        if scoring == "softmax":
            e = np.exp(l[ok] - l[ok].max())
            out[ok] = e / e.sum()
        else:
            out[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
    return out


def route_token(logits, scoring: str, topk: int, bias=None, groups: int = 1, topk_groups: int = 1, group_top: int = 1,
                renorm: bool = False, scale: float = 1.0):
    """One row of logits (float64 [E]) -> (ids int32 [topk], weights float64 [topk], unrounded)."""
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isposinf(l), FLT_MAX, l)
    e = l.size
    s = scores(l, scoring)
    eligible = ~np.isnan(l) & (l > -np.inf)
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        eligible &= ~np.isnan(b) & (b > -np.inf)
        choice = s + np.where(eligible, b, 0.0)
    else:
        choice = l
    if groups > 1:
        size = e // groups
        base = choice if (bias is not None or group_top == 1) else s
        value = []
        for g in range(groups):
            best = sorted((base[i] for i in range(g * size, (g + 1) * size) if eligible[i]), reverse=True)[:group_top]
            value.append(sum(best) if best else None)
        order = sorted((g for g in range(groups) if value[g] is not None), key=lambda g: (-value[g], g))
        kept = set(order[:topk_groups])
        eligible = eligible & np.array([i // size in kept for i in range(e)])
    order = sorted(np.nonzero(eligible)[0].tolist(), key=lambda i: (-choice[i], i))[:topk]
    ids = np.full(topk, -1, dtype=np.int32)
    w = np.zeros(topk, dtype=np.float64)
    ids[:len(order)] = order
    w[:len(order)] = s[order]
    if renorm:
        total = w.sum()
        w = w / total if total > 0 else np.zeros_like(w)
    return ids, w * float(np.float32(scale))


def route(logits, scoring: str, topk: int, **kw):
    """[T, E] logits -> (ids int32 [T, topk], weights float64 [T, topk])."""
    rows = [route_token(r, scoring, topk, **kw) for r in np.asarray(logits, dtype=np.float64)]
    if not rows:
        return np.zeros((0, topk), np.int32), np.zeros((0, topk))
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])
