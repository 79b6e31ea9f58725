"""References of the operators around a decoder layer's products.  TEST INFRASTRUCTURE ONLY.

Numpy float64 from the definitions: the norms around a block with its gate and residual, low-rank
adapters of many requests, a cache of keys and values in MXFP4 and the causal attention that reads it.
Each also returns the sum of magnitudes that its roundings are bounded against.
"""
from __future__ import annotations

import numpy as np

from .formats import decode_e2m1, decode_ue8m0, unpack_u8_nibbles
from .quant import mxfp4_rows


def normed(v, kind: str, eps: float, weight=None, bias=None, offset: float = 0.0):
    """N(v) by rows, the factor of each value and the rows' means (zeros for RMS)."""
    mean = v.mean(axis=1, keepdims=True) if kind == "layer" else np.zeros((v.shape[0], 1))
    d = v - mean
    factor = 1.0 / np.sqrt(np.mean(d * d, axis=1, keepdims=True) + eps) * np.ones_like(v)
    if weight is not None:
        factor = factor * (offset + weight)
    return d * factor + (0.0 if bias is None else bias), factor, mean


def norm_rows(y=None, res=None, kind="rms", post="", eps=1e-6, weight=None, bias=None, gate=None, post_weight=None,
              offset=0.0, res_scale=1.0):
    """(u, z, magnitude of u's terms, magnitude of z's): the last two are what float32 rounding errors scale with."""
    if y is None:
        u, mag = res, np.abs(res)
    else:
        h, hmag = y, np.abs(y)
        if post:
            h, f, mean = normed(y, post, eps, post_weight, None, offset)
            hmag = (np.abs(y) + np.abs(mean) + np.abs(y).mean(axis=1, keepdims=True)) * np.abs(f)
        g = res_scale * (1.0 if gate is None else gate)
        u, mag = g * h, np.abs(g) * hmag
        if res is not None:
            u, mag = u + res, mag + np.abs(res)
    if not kind:
        return u, None, mag, None
    z, f, mean = normed(u, kind, eps, weight, bias, offset)
    zmag = (mag + mag.mean(axis=1, keepdims=True)) * np.abs(f) + np.abs(z) + (0.0 if bias is None else np.abs(bias))
    return u, z, mag, zmag


def lora(x, a, b, ids, ranks, scales, base, slice_ends):
    """(out, magnitude): a [E][S][R][k], b [E][n][R]; tokens whose id is outside [0, E) keep their row of base."""
    out = base.astype(np.float64).copy()
    mag = np.abs(out)
    for m, e in enumerate(ids):
        if not 0 <= e < a.shape[0]:
            continue
        r = min(max(int(ranks[e]), 0), a.shape[2])
        begin = 0
        for s, end in enumerate(slice_ends):
            t = a[e, s, :r] @ x[m]
            tm = np.abs(a[e, s, :r]) @ np.abs(x[m])
            out[m, begin:end] += scales[e] * (b[e, begin:end, :r] @ t)
            mag[m, begin:end] += abs(scales[e]) * (np.abs(b[e, begin:end, :r]) @ tm)
            begin = end
    return out, mag


def mxfp4_values(x):
    """Rows through MXFP4 and back; a block of 32 that is not finite is NaN."""
    blocks = x.reshape(x.shape[0], -1, 32)
    finite = np.isfinite(blocks).all(axis=2)
    packed, scale = mxfp4_rows(np.where(finite[:, :, None], blocks, 0.0).reshape(x.shape))
    v = decode_e2m1(unpack_u8_nibbles(packed)).reshape(blocks.shape) * decode_ue8m0(scale)[:, :, None]
    v[~finite] = np.nan
    return v.reshape(x.shape)


def attention(q, k, v, lens, counts, scale, seen=None):
    """(out, magnitude): q [tokens][heads][D] rows of the sequences in turn, counts[b] of each; k, v [b] -> [len][kv][D].
    seen [b] -> [len] False: a token that no query sees.  A query that sees nothing gives zeros."""
    heads, dim = q.shape[1:]
    out, mag = np.zeros_like(q), np.zeros_like(q)
    at = 0
    for b, n in enumerate(counts):
        kv = k[b].shape[1]
        for i in range(n):
            place = lens[b] - n + i
            vis = np.arange(lens[b]) <= place
            if seen is not None:
                vis = vis & seen[b]
            if vis.any():
                for h in range(heads):
                    kk, vv = k[b][vis][:, h // (heads // kv)], v[b][vis][:, h // (heads // kv)]
                    s = scale * (kk @ q[at + i, h])
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[at + i, h] = w @ vv
                    # relative errors of the weights go with their scores' terms
                    terms = abs(scale) * (np.abs(kk) @ np.abs(q[at + i, h]))
                    mag[at + i, h] = (w * (1.0 + terms)) @ np.abs(vv) + (w @ terms) * np.abs(out[at + i, h])
        at += n
    return out, mag


def attention_terms(q, k, v, lens, counts, scale, seen=None):
    """attention() with what its roundings are bounded against kept apart, per output: a dict of
    out;  wv: sum_t w_t |V_t|;  dev: a bound of sum_t w_t |V_t - out|;  dev2: sum_t (w_t (V_t - out))^2;
    terms: a bound of sum_t w_t T_t |V_t - out|, T_t = |scale| sum |k q| of the score's terms, plus |score|.
    An error e_t of the weights, relative to each and the same in their sum, moves an output by sum_t w_t e_t (V_t - out)
    to first order: |e_t| <= e gives e * dev, independent errors of root mean square e give e * sqrt(dev2).
    (The bounds are Cauchy's: sum w T |d| <= sqrt(sum w T^2) sqrt(sum w d^2).)"""
    heads, dim = q.shape[1:]
    r = {name: np.zeros(q.shape) for name in ("out", "wv", "dev", "dev2", "terms")}
    at = 0
    for b, n in enumerate(counts):
        if n == 0:
            continue
        kv = k[b].shape[1]
        places = lens[b] - n + np.arange(n)
        vis = np.arange(lens[b])[None, :] <= places[:, None]
        if seen is not None:
            vis = vis & seen[b][None, :]
        some = vis.any(axis=1)
        for h in range(heads):
            kk, vv = k[b][:, h // (heads // kv)], v[b][:, h // (heads // kv)]
            qq = q[at:at + n, h]
            s = np.where(vis, scale * (qq @ kk.T), -np.inf)
            w = np.exp(s - np.where(some, s.max(axis=1, initial=-np.inf), 0.0)[:, None])
            w /= np.where(some, w.sum(axis=1), 1.0)[:, None]
            t = abs(scale) * (np.abs(qq) @ np.abs(kk).T) + np.where(vis, np.abs(s), 0.0)
            out, w2 = w @ vv, w * w
            dev = np.sqrt(np.maximum(w @ (vv * vv) - out * out * w.sum(axis=1)[:, None], 0.0))
            r["out"][at:at + n, h] = out
            r["wv"][at:at + n, h] = w @ np.abs(vv)
            r["dev"][at:at + n, h] = dev
            r["dev2"][at:at + n, h] = np.maximum(w2 @ (vv * vv) - 2 * out * (w2 @ vv) + out * out * w2.sum(axis=1)[:, None], 0.0)
            r["terms"][at:at + n, h] = np.sqrt((w * t * t).sum(axis=1))[:, None] * dev
        at += n
    return r
