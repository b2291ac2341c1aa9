"""Glue between KvCache8 and its oracle, and the error bounds of its results.

Half a step of rounding relative to the value is u = finfo.eps / 2.

Attention.  For a row and head with weights p, values V and scores s:
* a score's products are exact in the matrix unit, its hd/16 partial sums (twice that with two parts of q) and the
  scaling each lose at most 2^-23 of c = scale sum |q||K|: under 18 * 2^-23 c; two 11-bit parts of q leave 2^-22 of
  the row's largest element: d = 2^-18 c + 2^-22 scale max|q| sum |K|.
* a weight is off by 2 d (its score's and the maximum's), by 2^-20 (exp2) and by its 16-bit parts: one part 2^-11,
  two 2^-22.  Below 2^-14 an f16 loses relative precision: weights are held relative to W = max p 2^ev and times 2^14,
  so half of f16's least step, 2^-25, is 2^-39 W, and every position may add that times its code: 2^-39 W sum |code|.
* the sums over n positions lose at most 2^-23 in each of n/16 + 24 steps (the splits' joins among them), in numerator
  and in denominator.
The numerator's error is relative to A = sum p |V|; the result's rounding adds u |out|.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv8 as ok

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def rows_of(B, seqs, n_rows=None, max_rows=None):
    """seqs: (rows, slot, length) of each sequence, rows back to back.  Returns (KvRows, oracle sequences)."""
    start = np.concatenate([[0], np.cumsum([s[0] for s in seqs])]).astype(int)
    slot, length = [s[1] for s in seqs], [s[2] for s in seqs]
    r = B.KvRows(i32(list(start)), i32(slot), i32(length), n_rows=int(n_rows or start[-1]),
                 max_rows=int(max_rows or max(s[0] for s in seqs) or 1))
    return r, ok.rows_of(start, slot, length)


def held(cache, layer: int, fmt: str):
    """The cache's state as the oracle has it: codes and exponents of keys and of values."""
    L = cache.n_layers
    out = []
    for t, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        c = t.reshape(L, -1, cache.kv_heads, t.shape[-2], cache.head_dim)[layer].cpu().numpy()
        x = e.reshape(L, -1, cache.kv_heads, e.shape[-1])[layer].cpu().numpy()
        out += [ok.code_values(c, fmt), x.astype(np.int64) - ok.BIAS]
    return out


def fill(cache, fmt: str, seed: int, spread: float = 2.0):
    """Every code a finite number, block exponents spread over 2^+-spread."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        c = torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.int32)
        if fmt == "e4m3":
            c = torch.where((c & 127) > 0x76, c & 0xF0, c)  # below the largest, no NaN
        else:
            c = torch.where(c == 128, torch.zeros_like(c), c)
        t.copy_(c.to(torch.uint8))
        lo = (-8 if fmt == "e4m3" else -7) + ok.BIAS
        e.copy_((lo + spread * torch.randn(e.shape, generator=g, device="cuda")).round().to(torch.uint8))


def attend_bound(q, kc, ke, vc, ve, seqs, block, scale, dtype, want):
    """The bound above, for each element of want."""
    b = np.full(want.shape, np.inf)
    part = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -11
    for row0, n, slot, length in seqs:
        k, v = ok.held_values(kc, ke, slot, 0, length, block), ok.held_values(vc, ve, slot, 0, length, block)
        group = q.shape[1] // k.shape[0]
        for r in range(n):
            seen = length - n + r + 1
            for h in range(q.shape[1]):
                if seen <= 0:
                    b[row0 + r, h] = 0
                    continue
                x, kk = q[row0 + r, h].astype(np.float64), k[h // group, :seen]
                s = scale * (kk @ x)
                p = np.exp(s - s.max())
                p /= p.sum()
                c = scale * (np.abs(kk) @ np.abs(x))
                d = 2.0 ** -18 * c + 2.0 ** -22 * scale * np.abs(x).max() * np.abs(kk).sum(-1)
                w = 2 * d.max() + 2.0 ** -20 + part + (seen / 16 + 24) * 2.0 ** -23
                a = p @ np.abs(v[h // group, :seen])
                step = np.exp2(ve[slot, h // group][np.arange(seen) // block].astype(np.float64))
                floor = 2.0 ** -39 * (p * step).max() * (np.abs(v[h // group, :seen]) / step[:, None]).sum(0)
                off = 2 * w * a + 2 * floor
                b[row0 + r, h] = off + half_step(dtype) * (np.abs(want[row0 + r, h]) + off)
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149}[dtype]
    return b + tiny


def check_attend(out, q, state, seqs, block, scale):
    """out and q are the call's tensors; state as held() gives it."""
    qn = q.double().cpu().numpy()
    want = ok.attend(qn, *state, seqs, block, scale)
    bound = attend_bound(qn, *state, seqs, block, scale, q.dtype, want)
    got = out.double().cpu().numpy()
    inside = ~np.isnan(want)
    assert np.isfinite(got[inside]).all()
    err = np.abs(got - want)
    worst = (err / bound)[inside].max() if inside.any() else 0.0
    assert worst <= 1, f"error is {worst:.3g} of its bound"
    return worst
