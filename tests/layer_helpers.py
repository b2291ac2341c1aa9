"""Inputs of the layer calls' tests, and the error bounds of the products.

u(t) = finfo(t).eps / 2 is half a step relative to the value; a matrix unit's f32 add may truncate: 2^-23 of the larger operand.

Products.  For a row and a weight row with weights W = s q + m, block by block:
* few rows (at most 8 of one matrix; of a small one, up to 64: few = None takes either path's bound): weights and x exact.  A block's products are of (16 + q) x and 16 s - m
  times its sum: B = sum over blocks of (31 |s| + |m - 16 s|) sum |x| bounds every partial sum's terms.  A term passes at most 6
  adds in its block, one per step of a warp, 16 of the join and 4 scalings: (nks + 32) 2^-23 B.
* bf16 rows: weights are one f16 of the row's scale: 2^-11 |W|, or half of f16's least step, 2^-25, where a weight is below
  2^-14; a row's largest scale is at least 2^-10 there (or its largest min at least 4): 2^-15 max(max |s|, max |m| / 2^12).  x is
  brought to at most 2^15: exact but for 2^-25 2^-14 of the row's largest.  4 adds a step and 16: (4 nks + 16) 2^-23 sum |W||x|.
* f16 and f32 rows: s (q - 8), 8 s and m exact but below 2^-24 of the row's scale (2^-27 of its largest weights, that is, 2^-24 of
  its largest scale): terms C = sum (|s| |q - 8| |x|) + (8 |s| + |m|) sum |x|; a block's sum of x is two f16: 2^-21 of itself.
  f16: at most 12 adds a step, one accumulator: (12 nks + 24) 2^-23 C, x exact but for 2^-34 of the row's largest.
  f32: x in two f16 parts (2^-22), the product of both second parts left out (2^-22), 32 adds between sums in f32, and nks of
  those: (32 + nks) 2^-23 C.
A cluster's join is 8 more adds.
* a pair: silu(g) u with |silu'| <= 1.1; silu itself within 2^-19 (16-bit rows) or 2^-21 of its size.
"""
from __future__ import annotations

import numpy as np
import torch

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def parts64(q):
    """(s, m, codes) of a QMat in 64 bits, each [n][rows][cols]."""
    s = q.scale.view(torch.float16).double().repeat_interleave(q.block, -1)
    m = q.min.view(torch.float16).double().repeat_interleave(q.block, -1)
    c = torch.stack((q.codes & 15, q.codes >> 4), -1).flatten(-2).double()
    return s, m, c


def product_bound(x, q, i, few):
    """(W x, its error's bound before the result's own rounding) of rows x with matrix i, in 64 bits on the GPU."""
    s, m, c = (t[i] for t in parts64(q))
    W, xd = s * c + m, x.double()
    ax, nks = xd.abs(), q.cols // 64
    y = xd @ W.T
    top = ax.amax(-1, keepdim=True) * q.cols  # the row's largest, once per column
    big = torch.maximum(s.abs().amax(-1), m.abs().amax(-1) / 4096)
    if few:
        return y, (nks + 32) * 2.0 ** -23 * (ax @ (31 * s.abs() + (m - 16 * s).abs()).T)
    if x.dtype == torch.bfloat16:
        A = ax @ W.abs().T
        return y, 2.0 ** -11 * A + 2.0 ** -15 * ax.sum(-1, keepdim=True) * big + 2.0 ** -39 * top * W.abs().amax(-1) + \
            (4 * nks + 24) * 2.0 ** -23 * A
    C = ax @ ((s * (c - 8)).abs() + 8 * s.abs() + m.abs()).T
    adds = (12 * nks + 32) if x.dtype == torch.float16 else 40 + nks
    return y, (adds * 2.0 ** -23 + 2.0 ** -20) * C + 2.0 ** -24 * ax.sum(-1, keepdim=True) * big + \
        2.0 ** -34 * top * (s.abs() * 16 + m.abs()).amax(-1)


def linear_bound(x, w, up, i=0, few=False):
    """(y, bound) of the call's rows with matrix i."""
    if few is None:
        y, a = linear_bound(x, w, up, i, False)
        return y, torch.maximum(a, linear_bound(x, w, up, i, True)[1])
    g, eg = product_bound(x, w, i, few)
    if up is not None:
        v, ev = product_bound(x, up, i, few)
        sg = g * torch.sigmoid(g)
        e = 1.1 * eg * (v.abs() + ev) + (sg.abs() + 1.1 * eg) * ev
        g, eg = sg * v, e + (2.0 ** -21 if x.dtype == torch.float32 else 2.0 ** -18) * (sg * v).abs() + 2.0 ** -100
    h = half_step(x.dtype)
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -130
    return g, eg * (1 + h) + h * g.abs() + tiny


def check_rows(got, want, bound):
    assert torch.isfinite(got).all()
    err = (got.double() - want).abs()
    assert (err <= bound).all(), (err / bound).max().item()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
