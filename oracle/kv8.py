"""fp64 oracle of the attention-side calls: per-head norms with the rotation by
position, and the 8-bit KV caches (test infrastructure only).

Code arrays hold the numbers that the codes stand for (float64), exponent
arrays hold e itself.  Exponents and roundings are integer decisions and are
exact here: every operand is a power of two times a short number.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

QMAX = {"e4m3": 448.0, "int8": 127.0}
E_MIN, E_MAX, BIAS = -48, 47, 127


def qknorm(x: np.ndarray, position: np.ndarray, freqs, gain=None, eps: float = 1e-6, norm: bool = True,
           interleaved: bool = False) -> np.ndarray:
    """x [T][heads][head_dim] -> the normed and rotated rows, fp64."""
    y = x.astype(np.float64)
    if norm:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps)
        if gain is not None:
            y = y * gain.astype(np.float64)
    out = y.copy()
    half = len(freqs)
    two_pi = Fraction(6283185307179586476925286766559005768394338798750, 10 ** 48)
    for t, p in enumerate(position):
        for i, f in enumerate(freqs):
            a = Fraction(float(f)) * int(p)
            a -= two_pi * (a // two_pi)
            c, s = math.cos(float(a)), math.sin(float(a))
            j0, j1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            out[t, :, j0] = y[t, :, j0] * c - y[t, :, j1] * s
            out[t, :, j1] = y[t, :, j0] * s + y[t, :, j1] * c
    return out


def code_values(codes: np.ndarray, fmt: str) -> np.ndarray:
    """uint8 codes -> the numbers they stand for."""
    c = codes.astype(np.int64)
    if fmt == "int8":
        return np.where(c >= 128, c - 256, c).astype(np.float64)
    sign = np.where(c >= 128, -1.0, 1.0)
    exp, man = (c >> 3) & 15, c & 7
    return sign * np.where(exp == 0, np.ldexp(man.astype(np.float64), -9), np.ldexp(8.0 + man, exp - 10))


def nearest(v: np.ndarray, fmt: str) -> np.ndarray:
    """The code number nearest to v (ties to even), saturated; NaN gives 0."""
    v = np.where(np.isnan(v), 0.0, np.clip(v, -QMAX[fmt], QMAX[fmt])).astype(np.float64)
    if fmt == "int8":
        return np.rint(v)
    _, x = np.frexp(v)  # |v| in [2^(x-1), 2^x)
    step = np.ldexp(1.0, np.maximum(x - 1, -6) - 3)
    return np.rint(v / step) * step


def least_exponent(a: float, fmt: str) -> int:
    """The least e with a <= qmax 2^e, clamped."""
    if a == 0:
        return E_MIN
    e = math.ceil(math.log2(a / QMAX[fmt])) - 1
    while a > math.ldexp(QMAX[fmt], e):
        e += 1
    return min(max(e, E_MIN), E_MAX)


def rows_of(row_start, slot, length):
    """(first row, rows, slot, length) of each sequence."""
    return [(int(row_start[i]), int(row_start[i + 1] - row_start[i]), int(slot[i]), int(length[i]))
            for i in range(len(slot))]


def append(codes: np.ndarray, exps: np.ndarray, x: np.ndarray, seqs, block: int, fmt: str) -> None:
    """Write x [T][kv_heads][hd] into codes [slots][kv_heads][ctx][hd] and exps [slots][kv_heads][blocks]."""
    for row0, n, slot, length in seqs:
        p0 = length - n
        for b in range(p0 // block, (length + block - 1) // block) if n else ():
            lo, hi = max(p0, b * block), min(length, (b + 1) * block)
            for h in range(codes.shape[1]):
                new = x[row0 + lo - p0:row0 + hi - p0, h].astype(np.float64)
                fin = np.abs(new[np.isfinite(new)])
                e = least_exponent(float(fin.max()) if fin.size else 0.0, fmt)
                if lo > b * block:
                    held = int(exps[slot, h, b])
                    e = max(e, held)
                    codes[slot, h, b * block:lo] = nearest(np.ldexp(codes[slot, h, b * block:lo], held - e), fmt)
                codes[slot, h, lo:hi] = nearest(np.ldexp(new, -e), fmt)
                exps[slot, h, b] = e


def held_values(codes, exps, slot: int, lo: int, hi: int, block: int) -> np.ndarray:
    """[kv_heads][hi - lo][hd] values that a slot holds."""
    e = exps[slot][:, np.arange(lo, hi) // block]
    return np.ldexp(codes[slot, :, lo:hi], e[..., None].astype(np.int64))


def attend(q: np.ndarray, kc, ke, vc, ve, seqs, block: int, scale: float) -> np.ndarray:
    """q [T][heads][hd] over the caches (codes and exponents of keys and values); NaN rows of no sequence."""
    T, heads, hd = q.shape
    out = np.full((T, heads, hd), np.nan)
    for row0, n, slot, length in seqs:
        k, v = held_values(kc, ke, slot, 0, length, block), held_values(vc, ve, slot, 0, length, block)
        group = heads // k.shape[0]
        for r in range(n):
            seen = length - n + r + 1
            for h in range(heads):
                if seen <= 0:
                    out[row0 + r, h] = 0.0
                    continue
                s = scale * (k[h // group, :seen] @ q[row0 + r, h].astype(np.float64))
                p = np.exp(s - s.max())
                out[row0 + r, h] = (p @ v[h // group, :seen]) / p.sum()
    return out
