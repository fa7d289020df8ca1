"""Serving from a paged cache of keys and values, in plain fp64 numpy: where a token lies, what a new token sees, its
attention, and the 8-bit form of a token's head.
"""
from __future__ import annotations

import math

import numpy as np

from .layer_ops import E4M3_TOP, LEAST_SCALE


def sees(length, new, window, sinks):
    """[new, length] truth values: whether new token i (at position length - new + i) sees token j."""
    p = (length - new + np.arange(new))[:, None]
    j = np.arange(length)[None]
    return (j <= p) & ((window == 0) | (j > p - window) | (j < sinks))


def places(table_row, length, page):
    """(page number, place in it) of a sequence's tokens 0 .. length - 1."""
    j = np.arange(length)
    return np.asarray(table_row)[j // page], j % page


def attention(q, k, v, new, window, sinks, scale=None):
    """q [new, heads_q, D], k and v [length, heads_k, D]; returns (o, lse, size, far): o [new, heads_q, D], lse [new,
    heads_q], size = sum of weights times |v|, and far, the most that a visible key's score adds up in magnitude."""
    length, heads_k, D = k.shape
    heads_q = q.shape[1]
    scale = D ** -0.5 if scale is None else scale
    o, size = np.zeros(q.shape), np.zeros(q.shape)
    lse, far = np.full((new, heads_q), -math.inf), np.zeros((new, heads_q))
    seen = sees(length, new, window, sinks)
    for h in range(heads_q):
        g = h // (heads_q // heads_k)
        for i in range(new):
            at = np.flatnonzero(seen[i])
            if not len(at):
                continue
            s = scale * (k[at, g] @ q[i, h])
            far[i, h] = scale * np.max(np.abs(k[at, g]) @ np.abs(q[i, h]))
            w = np.exp(s - s.max())
            lse[i, h] = s.max() + math.log(w.sum())
            o[i, h], size[i, h] = w @ v[at, g] / w.sum(), w @ np.abs(v[at, g]) / w.sum()
    return o, lse, size, far


def in_8_bits(x):
    """x [..., D]: the quotients by each head's scale before they are rounded, and the scales."""
    scale = np.maximum(np.max(np.abs(x), axis=-1) / E4M3_TOP, LEAST_SCALE)
    return x / scale[..., None], scale
