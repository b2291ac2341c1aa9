"""fp64 oracle of a layer's other parts as calls -- TEST INFRASTRUCTURE ONLY.

* products: y = W x for each row, W dequantized exactly; a pair: silu(W x) * (U x);
* the router's choice over logits, the order of the entries by expert, rows in that order and back with weights, and the
  gradient of that;
* norms after and before a block with the gate and the residual.
Each follows the definition in ``include/strata_window.h`` row by row.
"""
from __future__ import annotations

import numpy as np

from .moe_window import OQMat, dequant, silu


def linear(x: np.ndarray, w: OQMat, up: OQMat = None, offsets=None):
    """y [T][rows] (NaN in rows of no matrix)."""
    x = np.asarray(x, np.float64)
    if offsets is None:
        offsets = [0, len(x)]
    y = np.full((len(x), w.rows), np.nan)
    for i in range(len(offsets) - 1):
        a, b = offsets[i], offsets[i + 1]
        if not 0 <= a < b <= len(x):
            continue
        p = x[a:b] @ dequant(w, i).T
        if up is not None:
            p = silu(p) * (x[a:b] @ dequant(up, i).T)
        y[a:b] = p
    return y


def route(logits: np.ndarray, k: int, renorm: bool, bias=None):
    """(idx [T][k], w [T][k]): largest first, equal logits by the lower expert; -1 and 0 where nothing is left."""
    T = len(logits)
    idx, w = np.full((T, k), -1, np.int64), np.zeros((T, k))
    for t in range(T):
        l = np.asarray(logits[t], np.float32)
        if bias is not None:
            with np.errstate(invalid="ignore"):
                l = l + np.asarray(bias, np.float32)
        l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max)).astype(np.float64)
        order = sorted((e for e in range(len(l)) if l[e] > -np.inf), key=lambda e: (-l[e], e))
        if not order:
            continue
        top = l[order[0]]
        total = sum(np.exp(l[e] - top) for e in (order[:k] if renorm else order))
        for j, e in enumerate(order[:k]):
            idx[t, j], w[t, j] = e, np.exp(l[e] - top) / total
    return idx, w


def order(idx: np.ndarray, E: int):
    """(counts [E], offsets [E + 1], entries [T*k], place [T*k]) of the entries t * k + j."""
    flat = np.asarray(idx).ravel()
    groups = [[i for i, e in enumerate(flat) if e == x] for x in range(E)]
    counts = np.array([len(g) for g in groups])
    entries, place = np.full(len(flat), -1), np.full(len(flat), -1)
    at = 0
    for g in groups:
        for i in g:
            entries[at], place[i] = i, at
            at += 1
    return counts, np.concatenate([[0], np.cumsum(counts)]), entries, place


def gather(x: np.ndarray, place: np.ndarray, k: int):
    """[T*k][width], NaN behind the last expert's rows."""
    xs = np.full((len(place), x.shape[1]), np.nan)
    for i, p in enumerate(place):
        if 0 <= p < len(place):
            xs[p] = x[i // k]
    return xs


def combine(z: np.ndarray, place: np.ndarray, k: int, w=None, base=None):
    T = len(place) // k
    y = np.zeros((T, z.shape[1])) if base is None else np.array(base, np.float64)
    for i, p in enumerate(place):
        if 0 <= p < len(place):
            y[i // k] += (1.0 if w is None else float(w[i // k, i % k])) * z[p]
    return y


def combine_backward(dy: np.ndarray, z: np.ndarray, place: np.ndarray, k: int, w=None):
    """(dz [T*k][width] with NaN behind the last expert's rows, dw [T][k])."""
    T = len(place) // k
    dz, dw = np.full((len(place), dy.shape[1]), np.nan), np.zeros((T, k))
    for i, p in enumerate(place):
        if 0 <= p < len(place):
            dz[p] = (1.0 if w is None else float(w[i // k, i % k])) * dy[i // k]
            dw[i // k, i % k] = dy[i // k] @ z[p]
    return dz, dw


def block_norm(x, y=None, after=None, before=None, gate=None, sigmoid=False, eps=1e-6, residual_scale=1.0,
               block_scale=1.0):
    """(h, n or None); after, before: gains or None for no norm; gate broadcasts against [T][hidden]."""
    h = residual_scale * np.asarray(x, np.float64)
    if y is not None:
        u = np.asarray(y, np.float64)
        if after is not None:
            u = u / np.sqrt(np.square(u).mean(-1, keepdims=True) + eps) * after
        if gate is not None:
            g = np.asarray(gate, np.float64)
            u = u * (1 / (1 + np.exp(-g)) if sigmoid else g)
        h = h + block_scale * u
    n = None if before is None else h / np.sqrt(np.square(h).mean(-1, keepdims=True) + eps) * before
    return h, n
