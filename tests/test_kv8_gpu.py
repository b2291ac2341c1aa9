"""The 8-bit KV caches on the GPU against the fp64 oracle: writing (codes and
exponents bit for bit), reading back (bit for bit), attention (within the bound
derived in tests/kv8_helpers.py), refusals, and a run of the calls together."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv8 as ok
from tests.kv8_helpers import DTYPES, check_attend, fill, held, i32, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from slot_decode_window_gb300 import binding, build
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()
    return binding


def _values(seed, shape, dtype, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.exp2(spread * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))).to(DTYPES[dtype])


def _same(cache, state, fmt, layer=0):
    for got, want, name in zip(held(cache, layer, fmt), state, ("k", "k_exp", "v", "v_exp")):
        np.testing.assert_array_equal(got, want, err_msg=name)


def _append(B, cache, state, k, v, seqs, block, fmt, layer=0, **kw):
    rows, os_ = rows_of(B, seqs, **kw)
    cache.append(layer, k, v, rows)
    for c, e, x in ((state[0], state[1], k), (state[2], state[3], v)):
        ok.append(c, e, x.float().cpu().numpy(), os_, block, fmt)


# calls in turn: (rows, slot, length after them) of each sequence
CALLS = [
    [[(1, 0, 1)], [(1, 0, 2)], [(2, 0, 4), (1, 1, 1)]],                                # token by token
    [[(37, 2, 37), (100, 0, 100), (1, 1, 1)], [(5, 2, 42), (30, 0, 130), (2, 1, 3)]],  # prompts, then more
    [[(16, 0, 16), (64, 1, 64), (0, 2, 0)], [(16, 0, 32), (1, 1, 65), (128, 2, 128)]], # block borders, no rows
    [[(131, 3, 131)], [(9, 3, 133)], [(1, 3, 20)]],                                    # the last position; written over
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,hd,kvh", [("f32", 128, 2), ("bf16", 64, 3), ("f16", 128, 1), ("f32", 64, 1),
                                          ("bf16", 128, 4)])
@pytest.mark.parametrize("calls", range(len(CALLS)))
def test_append_bit_for_bit(B, fmt, block, dtype, hd, kvh, calls):
    cache = B.KvCache8(2, 4, kvh * 2, kvh, hd, 133, block=block, format=fmt)
    fill(cache, fmt, seed=calls)
    state, other = held(cache, 1, fmt), held(cache, 0, fmt)
    for n, seqs in enumerate(CALLS[calls]):
        T = sum(s[0] for s in seqs)
        k, v = (_values(10 * n + i, (T, kvh, hd), dtype) * 2.0 ** (n - 1) for i in (1, 2))
        _append(B, cache, state, k, v, seqs, block, fmt, layer=1)
        cache.sync()
        _same(cache, state, fmt, layer=1)
    _same(cache, other, fmt, layer=0)  # the other layer is untouched


def test_append_values_at_the_format_borders(B):
    """Zeros, the largest of a format exactly and just past it, values below and above the exponents' range."""
    for fmt in ("e4m3", "int8"):
        q = ok.QMAX[fmt]
        vals = [0.0, q, float(np.nextafter(np.float32(q), np.float32(1e9))), q * 2.0 ** -48, 2.0 ** -70, 1e-42,
                q * 2.0 ** 47, 3e38, 1.0, -q]
        cache = B.KvCache8(1, len(vals), 1, 1, 64, 16, block=16, format=fmt)
        fill(cache, fmt, 0)
        state = held(cache, 0, fmt)
        k = torch.zeros(len(vals), 1, 64, device="cuda")
        k[:, 0, 5] = torch.tensor(vals)
        k[:, 0, 6] = torch.tensor(vals) * 0.3
        _append(B, cache, state, k, -k, [(1, i, 1) for i in range(len(vals))], 16, fmt)
        cache.sync()
        _same(cache, state, fmt)


def test_append_strided_rows_and_rows_behind_the_last_sequence(B):
    cache = B.KvCache8(1, 2, 4, 2, 128, 50, block=16)
    fill(cache, "e4m3", 1)
    state = held(cache, 0, "e4m3")
    fused = _values(3, (12, 8, 128), "bf16")  # q, k, v of a row side by side
    k, v = fused[:, 4:6], fused[:, 6:8]
    assert not k.is_contiguous()
    _append(B, cache, state, k, v, [(4, 1, 30), (3, 0, 3)], 16, "e4m3", n_rows=12)
    cache.sync()
    _same(cache, state, "e4m3")


def test_append_reports_and_bounds_what_is_not_finite(B):
    for fmt in ("e4m3", "int8"):
        cache = B.KvCache8(1, 1, 1, 1, 64, 16, block=16, format=fmt)
        fill(cache, fmt, 2)
        state = held(cache, 0, fmt)
        k = _values(4, (3, 1, 64), "f32")
        k[0, 0, 0], k[1, 0, 1], k[2, 0, 2] = float("nan"), float("inf"), float("-inf")
        v = _values(5, (3, 1, 64), "f32")
        _append(B, cache, state, k, v, [(3, 0, 3)], 16, fmt)
        with pytest.raises(B.StrataError) as e:
            cache.sync()
        assert e.value.status == B.STRATA_EDEVICE
        _same(cache, state, fmt)
        assert state[0][0, 0, 0, 0] == 0 and state[0][0, 0, 1, 1] == ok.QMAX[fmt]
        cache.sync()  # reported once


@pytest.mark.parametrize("fmt,dtype,hd,kvh,block", [("e4m3", "f32", 128, 2, 16), ("int8", "bf16", 64, 3, 64),
                                                    ("e4m3", "f16", 64, 1, 128), ("int8", "f32", 128, 1, 32)])
def test_read_bit_for_bit(B, fmt, dtype, hd, kvh, block):
    cache = B.KvCache8(2, 3, kvh, kvh, hd, 301, block=block, format=fmt)
    fill(cache, fmt, 3)
    kc, ke, vc, ve = held(cache, 1, fmt)
    rows, seqs = rows_of(B, [(301, 2, 301), (1, 0, 1), (0, 1, 7), (45, 1, 100)], n_rows=400)
    out = [torch.full((400, kvh, hd), 7.0, dtype=DTYPES[dtype], device="cuda") for _ in range(2)]
    cache.read(1, rows, k=out[0], v=out[1])
    cache.sync()
    for got, c, e in ((out[0], kc, ke), (out[1], vc, ve)):
        for row0, n, slot, length in seqs:
            want = ok.held_values(c, e, slot, length - n, length, block).transpose(1, 0, 2)
            want = torch.from_numpy(np.ascontiguousarray(want)).float().to(DTYPES[dtype])
            assert torch.equal(got[row0:row0 + n].cpu(), want)
        assert (got[347:] == 7).all()


SHAPES = [  # heads, kv_heads, head_dim, block, format, dtype
    (32, 4, 128, 32, "e4m3", "f32"), (8, 2, 64, 16, "int8", "f32"), (4, 4, 128, 64, "int8", "bf16"),
    (28, 4, 128, 128, "e4m3", "f16"), (5, 5, 64, 16, "e4m3", "bf16"), (20, 1, 128, 16, "int8", "f32"),
    (64, 2, 64, 64, "e4m3", "f16"), (3, 1, 128, 32, "e4m3", "f32"),
]
MIXES = [  # rows, slot, length
    [(1, 0, 1)],
    [(2, 1, 2), (1, 0, 16), (2, 3, 18), (1, 2, 17)],
    [(1, 0, 64), (1, 1, 65), (1, 2, 63), (1, 3, 129), (1, 0, 128)],  # tile borders; a slot twice
    [(2, 2, 700), (0, 1, 40), (1, 0, 0), (3, 1, 2)],                  # no rows; an empty slot; a row that sees nothing
    [(9, 0, 9), (17, 1, 60), (8, 2, 333)],
    [(65, 0, 65), (40, 3, 500)],
    [(130, 1, 701), (1, 0, 5), (129, 2, 129)],
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("mix", range(len(MIXES)))
def test_attend(B, shape, mix):
    heads, kvh, hd, block, fmt, dtype = shape
    cache = B.KvCache8(2, 4, heads, kvh, hd, 701, block=block, format=fmt)
    fill(cache, fmt, 10 + mix)
    state = held(cache, 1, fmt)
    rows, seqs = rows_of(B, MIXES[mix])
    q = _values(20 + mix, (rows.n_rows, heads, hd), dtype, spread=0.5)
    out = cache.attend(1, q, rows)
    cache.sync()
    check_attend(out, q, state, seqs, block, hd ** -0.5)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows_", [1, 40])
def test_attend_never_sees_past_a_row(B, fmt, dtype, rows_):
    """Codes of NaN (e4m3), of the largest magnitude (int8) and exponents at their ends wherever a row must not look:
    the same bits as with zeros there."""
    heads, kvh, hd, block = 8, 2, 128, 16
    outs = []
    q = _values(7, (rows_ + 1, heads, hd), dtype, spread=0.5)
    for poison in (0, 0x7F if fmt == "e4m3" else 0x80):
        cache = B.KvCache8(1, 3, heads, kvh, hd, 200, block=block, format=fmt)
        fill(cache, fmt, 5)
        for t, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
            t[0, 0, :, 83:] = poison
            t[0, 1, :, rows_:] = poison
            t[0, 2] = poison
            e[0, 0, :, 6:] = 255 if poison else 0
            e[0, 2] = 255 if poison else 0
        rows, _ = rows_of(B, [(rows_, 0, 83), (1, 1, rows_)])
        outs.append(cache.attend(0, q, rows))
        cache.sync()
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])
    # a long row set: row r equals the same row alone in a slot that ends there, within rounding
    if rows_ > 1:
        for r in (0, 11):
            alone, _ = rows_of(B, [(1, 0, 83 - rows_ + r + 1)])
            one = cache.attend(0, q[r:r + 1], alone)
            cache.sync()
            tol = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -17
            scale = outs[0][r].float().abs().max()
            assert (one[0].float() - outs[0][r].float()).abs().max() <= tol * scale


@pytest.mark.parametrize("n", [2, 40])
def test_attend_blocks_of_far_apart_exponents(B, n):
    """Exponents from one end of the range to the other in one row: weights and values span 2^90."""
    for fmt in ("e4m3", "int8"):
        for dtype in ("f32", "bf16"):
            cache = B.KvCache8(1, 1, 2, 1, 64, 128, block=16, format=fmt)
            fill(cache, fmt, 6, spread=0.0)
            cache.v_exp[0, 0, 0] = torch.tensor([79, 120, 174, 100, 127, 90, 140, 80], dtype=torch.uint8)
            cache.k_exp[0, 0, 0] = torch.tensor([118, 122, 79, 121, 117, 120, 119, 120], dtype=torch.uint8)
            state = held(cache, 0, fmt)
            rows, seqs = rows_of(B, [(n, 0, 128)])
            q = _values(8, (n, 2, 64), dtype, spread=0.0)
            out = cache.attend(0, q, rows)
            cache.sync()
            check_attend(out, q, state, seqs, 16, 0.125)


@pytest.mark.parametrize("n", [3, 40])
def test_attend_large_and_small_queries_and_scales(B, n):
    cache = B.KvCache8(1, 1, 4, 2, 128, 300, block=32)
    fill(cache, "e4m3", 9)
    state = held(cache, 0, "e4m3")
    rows, seqs = rows_of(B, [(n, 0, 300)])
    for mul, scale in ((2.0 ** 20, 2.0 ** -24), (2.0 ** -30, 2.0 ** 26), (1.0, 0.0), (1.0, -0.1)):
        q = _values(9, (n, 4, 128), "f32", spread=0.5) * mul
        out = cache.attend(0, q, rows, scale=scale)
        cache.sync()
        want = ok.attend(q.double().cpu().numpy(), *state, seqs, 32, scale)
        rms = np.sqrt(np.mean(want ** 2))
        assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0 ** -14 * rms


def test_attend_a_row_of_nan_stays_alone(B):
    cache = B.KvCache8(1, 2, 8, 2, 128, 400, block=64)
    fill(cache, "e4m3", 11)
    for n in (2, 33):
        rows, _ = rows_of(B, [(n, 0, 400), (1, 1, 10)])
        q = _values(12, (n + 1, 8, 128), "f32", spread=0.5)
        good = cache.attend(0, q, rows)
        q2 = q.clone()
        q2[1, 3] = float("nan")
        bad = cache.attend(0, q2, rows)
        cache.sync()
        assert torch.isnan(bad[1, 3]).all()
        bad[1, 3] = good[1, 3]
        assert torch.equal(bad, good)


def test_attend_long_rows_are_split_and_joined(B):
    """One row, a few and many over thousands of positions; twice the same bits."""
    for heads, kvh, hd, n, length, dtype in ((8, 1, 128, 1, 4099, "f32"), (16, 2, 64, 3, 5000, "bf16"),
                                             (4, 1, 128, 70, 2500, "f16")):
        cache = B.KvCache8(1, 2, heads, kvh, hd, 5003, block=64)
        fill(cache, "e4m3", 13)
        state = held(cache, 0, "e4m3")
        rows, seqs = rows_of(B, [(n, 1, length), (1, 0, 77)])
        q = _values(14, (n + 1, heads, hd), dtype, spread=0.5)
        a, b = cache.attend(0, q, rows), cache.attend(0, q, rows)
        cache.sync()
        assert torch.equal(a, b)
        check_attend(a, q, state, seqs, 64, hd ** -0.5)


def test_offsets_past_32_bits(B):
    """A cache of more than 2^32 codes: the last slot's last layer is written, read and attended over."""
    kvh, hd, ctx = 4, 128, 131072
    slots = (1 << 32) // (kvh * hd * ctx) + 1
    cache = B.KvCache8(1, slots, kvh, kvh, hd, ctx, block=64)
    assert cache.k.numel() > 1 << 32
    rows, seqs = rows_of(B, [(100, slots - 1, ctx)])
    k, v, q = (_values(i, (100, kvh, hd), "bf16", spread=0.5) for i in (1, 2, 3))
    # the same rows at the same places within their blocks: positions ctx - 100 on, and 28 on of a small cache
    small = B.KvCache8(1, 1, kvh, kvh, hd, 128, block=64)
    cache.k[0, slots - 1, :, :ctx - 100] = 0
    cache.v[0, slots - 1, :, :ctx - 100] = 0
    cache.k_exp[0, slots - 1] = 79
    cache.v_exp[0, slots - 1] = 79
    small.k.zero_(), small.v.zero_(), small.k_exp.fill_(79), small.v_exp.fill_(79)
    cache.append(0, k, v, rows)
    small.append(0, k, v, rows_of(B, [(100, 0, 128)])[0])
    a, b = cache.read(0, rows), small.read(0, rows_of(B, [(100, 0, 128)])[0])
    cache.sync(), small.sync()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    out = cache.attend(0, q, rows, scale=0.5)
    cache.sync()
    # zero keys score 0 and zero values add nothing: the oracle on the rows that count
    kk, vv, qq = (x.double().cpu() for x in (a[0], a[1], q))
    for r in (0, 57, 99):
        for h in (0, kvh - 1):
            s = 0.5 * (kk[:r + 1, h] @ qq[r, h])
            m = max(0.0, s.max().item())
            p = torch.exp(s - m)
            want = (p @ vv[:r + 1, h]) / (p.sum() + (ctx - 100) * np.exp(-m))
            err = (out[r, h].double().cpu() - want).abs().max()
            assert err <= 2.0 ** -8 * want.abs().max() + 2.0 ** -9 * (p.abs() @ vv[:r + 1, h].abs()).max() / (
                p.sum() + (ctx - 100) * np.exp(-m))
    one = cache.attend(0, q[99:], rows_of(B, [(1, slots - 1, ctx)])[0], scale=0.5)  # the few-row path's offsets
    cache.sync()
    assert (one[0].float() - out[99].float()).abs().max() <= 2.0 ** -7 * out[99].float().abs().max()


def test_captured_calls_follow_their_buffers(B):
    """append and attend captured once and replayed as the slots grow, against the same calls made directly."""
    kw = dict(block=16, format="int8")
    one, two = (B.KvCache8(1, 3, 8, 2, 64, 90, **kw) for _ in range(2))
    for c in (one, two):
        fill(c, "int8", 15)
    k, v, q = (_values(i, (4, h, 64), "f32") for i, h in ((1, 2), (2, 2), (3, 8)))
    out = torch.empty_like(q)
    start, slot, length = i32([0, 2, 3, 3]), i32([2, 0, 1]), i32([40, 1, 0])
    rows = B.KvRows(start, slot, length, n_rows=4, max_rows=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one.attend(0, q, rows, out=out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one.append(0, k, v, rows)
        one.attend(0, q, rows, out=out)
    for step in range(6):
        for t in (k, v, q):
            t.normal_()
        out.fill_(5.0)
        g.replay()
        two.append(0, k, v, rows)
        want = torch.full_like(q, 5.0)
        two.attend(0, q, rows, out=want)
        one.sync(), two.sync()
        assert torch.equal(out, want) and (out[3] == 5).all()
        for a, b in ((one.k, two.k), (one.v, two.v), (one.k_exp, two.k_exp), (one.v_exp, two.v_exp)):
            assert torch.equal(a, b)
        length += i32([2, 1, 0])


def test_bad_sequences_are_left_out_and_reported(B):
    """A slot or a length out of range: zeros; row bounds out of order or too many rows: not touched; one slot twice
    in an append: the first is written."""
    cache = B.KvCache8(1, 3, 4, 2, 64, 40, block=16)
    fill(cache, "e4m3", 16)
    clean = held(cache, 0, "e4m3")
    q, k = _values(1, (6, 4, 64), "f32"), _values(2, (6, 2, 64), "f32")

    def reported():
        with pytest.raises(B.StrataError) as e:
            cache.sync()
        assert e.value.status == B.STRATA_EDEVICE
        cache.sync()

    bad = [([0, 2, 4], [3, 0], [5, 6], 2), ([0, 2, 4], [-1, 0], [5, 6], 2), ([0, 2, 4], [1, 0], [41, 6], 2),
           ([0, 2, 4], [1, 0], [-1, 6], 2)]
    for start, slot, length, most in bad:
        rows = B.KvRows(i32(start), i32(slot), i32(length), n_rows=6, max_rows=most)
        out = torch.full_like(q, 3.0)
        cache.attend(0, q, rows, out=out)
        reported()
        assert (out[:2] == 0).all() and (out[4:] == 3).all()
        good, seqs = rows_of(B, [(2, 0, 6)])
        check_attend(out[2:4], q[2:4], clean, seqs, 16, 0.125)
        ko, vo = torch.full_like(k, 3.0), torch.full_like(k, 3.0)
        cache.read(0, rows, k=ko, v=vo)
        reported()
        assert (ko[:2] == 0).all() and (ko[4:] == 3).all() and (ko[2:4] != 0).any()
    for start, most in (([0, -1, 2], 2), ([4, 2, 4], 2), ([0, 7, 7], 8), ([0, 3, 4], 2)):
        rows = B.KvRows(i32(start), i32([1, 0]), i32([5, 6]), n_rows=6, max_rows=most)
        out = torch.full_like(q, 3.0)
        cache.attend(0, q, rows, out=out)
        reported()
        assert torch.isfinite(out).all()
        cache.append(0, k, k, rows)
        reported()
    fill(cache, "e4m3", 16)
    state = held(cache, 0, "e4m3")
    rows = B.KvRows(i32([0, 2, 4, 5]), i32([1, 1, 2]), i32([5, 9, 1]), n_rows=6, max_rows=2)
    cache.append(0, k, k, rows)
    reported()
    for c, e in (state[:2], state[2:]):
        ok.append(c, e, k.cpu().numpy(), [(0, 2, 1, 5), (4, 1, 2, 1)], 16, "e4m3")
    _same(cache, state, "e4m3")
    rows = B.KvRows(i32([0, 4]), i32([1]), i32([3]), n_rows=6, max_rows=4)  # more rows than positions
    cache.append(0, k, k, rows)
    reported()
    _same(cache, state, "e4m3")


def test_refusals(B):
    cache = B.KvCache8(1, 2, 4, 2, 64, 40, block=16)
    rows, _ = rows_of(B, [(2, 0, 6)])
    h, q = cache.handle, torch.zeros(2, 4, 64, device="cuda")
    p, s = q.data_ptr(), 256
    EI, EU = B.STRATA_EINVAL, B.STRATA_EUNSUPPORTED
    assert B.strata_kv8_attend(None, 0, p, s, p, s, 0, 1.0, rows.c) == EI
    for kw in (dict(layer=1), dict(layer=-1), dict(dtype=3), dict(q=p + 4), dict(s=255), dict(s=257), dict(q=0),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        a = dict(layer=0, q=p, s=s, dtype=0, scale=1.0)
        a.update(kw)
        assert B.strata_kv8_attend(h, a["layer"], a["q"], a["s"], p, s, a["dtype"], a["scale"], rows.c) == EI, kw
    for field, val, st in (("n_seq", -1, EI), ("n_rows", -1, EI), ("max_rows", -1, EI), ("n_seq", 1025, EU),
                           ("row_start", None, EI), ("slot", None, EI), ("length", None, EI)):
        c = B.strata_kv8_rows(*(getattr(rows.c, n) for n, _ in rows.c._fields_))
        setattr(c, field, val)
        assert B.strata_kv8_append(h, 0, p, s, p, s, 0, c) == st
        assert B.strata_kv8_read(h, 0, p, s, p, s, 0, c) == st
        assert B.strata_kv8_attend(h, 0, p, s, p, s, 0, 1.0, c) == st
    for field in ("n_seq", "n_rows", "max_rows"):  # nothing to do
        c = B.strata_kv8_rows(*(getattr(rows.c, n) for n, _ in rows.c._fields_))
        setattr(c, field, 0)
        assert B.strata_kv8_attend(h, 0, 0, 0, 0, 0, 0, 1.0, c) == B.STRATA_OK
    cache.sync()
    for bad in (torch.zeros(2, 4, 64, device="cuda", dtype=torch.float64), torch.zeros(2, 3, 64, device="cuda"),
                torch.zeros(3, 4, 64, device="cuda"), torch.zeros(2, 4, 64), torch.zeros(2, 64, 4, device="cuda").mT):
        with pytest.raises(B.StrataError):
            cache.attend(0, bad, rows)
    with pytest.raises(B.StrataError):
        cache.append(0, q[:, :2], q[:, :2].half(), rows)
    for kw in (dict(dtype=torch.float64), dict(k=q[:, :2].double()), dict(k=q[:, :2], v=q[:, :2].half()),
               dict(v=q[:, :3]), dict(k=q[:1, :2])):
        with pytest.raises(B.StrataError):
            cache.read(0, rows, **kw)
    with pytest.raises(B.StrataError):
        B.KvRows(torch.zeros(3, dtype=torch.int64, device="cuda"), i32([0, 1]), i32([1, 1]), 2, 1)
    with pytest.raises(B.StrataError):
        B.KvCache8(1, 2, 4, 2, 64, 40, buffers=(torch.zeros(4, dtype=torch.uint8, device="cuda"),) * 4)


def test_steps_of_a_conversation_together(B):
    """Norms and rotation, append, attention: a prompt and then windows of a token and a proposal, some proposals
    rejected, against the same steps in 64 bits.  The keys are rotated, so far positions are part of it."""
    heads, kvh, hd, block, fmt, L = 8, 2, 128, 32, "int8", 2
    gain = 1 + 0.2 * torch.randn(hd, device="cuda", generator=torch.Generator("cuda").manual_seed(0))
    qk = B.QkNorm(heads, kvh, hd, theta=1e6, q_gain=gain, k_gain=None)
    freqs = [1e6 ** (-2.0 * i / hd) for i in range(hd // 2)]
    cache = B.KvCache8(L, 2, heads, kvh, hd, 120, block=block, format=fmt)
    fill(cache, fmt, 17)
    states = [held(cache, l, fmt) for l in range(L)]
    lengths = [0, 0]
    for step, rows_ in enumerate(([50, 33], [2, 1], [2, 2], [1, 2], [2, 0])):
        lengths = [n + r for n, r in zip(lengths, rows_)]
        rows, seqs = rows_of(B, [(r, s, n) for s, (r, n) in enumerate(zip(rows_, lengths))])
        position = np.concatenate([np.arange(n - r, n) for r, n in zip(rows_, lengths)])
        for layer in range(L):
            fused = _values(100 + 10 * step + layer, (rows.n_rows, heads + 2 * kvh, hd), "f32", spread=0.5)
            q, k, v = fused[:, :heads], fused[:, heads:heads + kvh], fused[:, heads + kvh:]
            qr, kr = qk.forward(q, k, i32(list(position)))
            cache.append(layer, kr, v, rows)
            out = cache.attend(layer, qr, rows)
            cache.sync()
            for got, x, g in ((qr, q, gain.cpu().numpy()), (kr, k, None)):
                want = ok.qknorm(x.cpu().numpy(), position, freqs, g)
                assert np.abs(got.double().cpu().numpy() - want).max() <= 2.0 ** -19 * np.abs(want).max()
            st = states[layer]
            ok.append(st[0], st[1], kr.cpu().numpy(), seqs, block, fmt)
            ok.append(st[2], st[3], v.cpu().numpy(), seqs, block, fmt)
            _same(cache, st, fmt, layer)
            check_attend(out, qr, st, seqs, block, hd ** -0.5)
        if step in (1, 3):
            lengths[step // 2] -= 1  # the last proposal was rejected
    qk.close(), cache.close()


@pytest.mark.parametrize("n", [1, 3, 50])
def test_attend_at_the_most_sequences_and_padded_rows(B, n):
    """1024 sequences in one call (one more is refused), some without rows or positions; rows behind the last one stay
    as they were; on another stream than the tensors'."""
    heads, kvh, hd = 4, 1, 64
    cache = B.KvCache8(1, 64, heads, kvh, hd, 150, block=16, format="int8")
    fill(cache, "int8", 18)
    state = held(cache, 0, "int8")
    some = [(i * 7) % (n + 1) if i % 5 else n for i in range(1024)]
    seqs = [(r, i % 64, max(r, (i * 13) % 150)) for i, r in enumerate(some)]
    T = sum(some)
    rows, os_ = rows_of(B, seqs, n_rows=T + 9)
    q = _values(3, (T + 9, heads, hd), "bf16", spread=0.5)
    out = torch.full_like(q, 3.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.attend(0, q, rows, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    cache.sync()
    assert (out[T:] == 3).all()
    # the oracle on a few of them
    pick = [0, 5, 512, 1019, 1020, 1023]
    part = [(s[0], s[1], s[2], s[3]) for s in (os_[i] for i in pick) if s[1] > 0]
    assert part
    check_attend(out, q, state, part, 16, 0.125)
    with pytest.raises(B.StrataError):
        cache.attend(0, q, rows_of(B, seqs + [(0, 0, 0)], n_rows=T + 9)[0], out=out)


def test_two_captured_graphs_of_one_handle_in_turn(B):
    """Two graphs share the handle's workspace; replayed one after the other, with split rows in both, each gives what
    the call gives by itself."""
    cache = B.KvCache8(1, 2, 8, 2, 128, 3000, block=64)
    fill(cache, "e4m3", 19)
    calls = []
    for n, seqs in ((1, [(1, 0, 2900), (1, 1, 700)]), (60, [(60, 1, 2999), (2, 0, 70)])):
        rows, _ = rows_of(B, seqs)
        q = _values(n, (rows.n_rows, 8, 128), "bf16", spread=0.5)
        want = cache.attend(0, q, rows)
        cache.sync()
        out = torch.zeros_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.attend(0, q, rows, out=out)
        calls.append((g, want, out, q, rows))
    for i in (0, 1, 1, 0, 0, 1):
        g, want, out = calls[i][:3]
        out.zero_()
        g.replay()
        cache.sync()
        assert torch.equal(out, want)


def test_appends_on_two_streams_to_different_slots(B):
    """append uses no workspace: two at once on one handle, each to its own slots."""
    cache = B.KvCache8(1, 2, 2, 2, 128, 4000, block=32)
    fill(cache, "e4m3", 20)
    state = held(cache, 0, "e4m3")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = []
    for i in range(2):
        rows, os_ = rows_of(B, [(3000, i, 3500)])
        k, v = _values(30 + i, (3000, 2, 128), "f16"), _values(40 + i, (3000, 2, 128), "f16")
        calls.append((rows, os_, k, v))
    torch.cuda.synchronize()
    for st, (rows, _, k, v) in zip(streams, calls):
        cache.append(0, k, v, rows, stream=st)
    cache.sync()
    for _, os_, k, v in calls:
        ok.append(state[0], state[1], k.float().cpu().numpy(), os_, 32, "e4m3")
        ok.append(state[2], state[3], v.float().cpu().numpy(), os_, 32, "e4m3")
    _same(cache, state, "e4m3")


def test_a_layer_by_its_parts(B):
    """The attention half as calls beside the MoE window: a decode step's hidden rows through q, k, v products, norms
    and rotation, append, attention, the o product and strata_moe_window_forward, against the fp64 oracle."""
    import oracle
    from slot_decode_window_gb300 import workloads as wlm
    from tests.helpers import margin_accept, omoe
    d, heads, kvh, hd = 256, 4, 2, 64
    wl = wlm.WORKLOADS["tiny"]
    layer = wlm.make_moe_layer(wl.moe, seed=0, cfg_id=wl.cfg_id, device="cuda")
    assert wl.moe.hidden == d
    g = torch.Generator(device="cuda").manual_seed(4)
    wqkv = torch.randn((heads + 2 * kvh) * hd, d, generator=g, device="cuda") / d ** 0.5
    wo = torch.randn(d, heads * hd, generator=g, device="cuda") / (heads * hd) ** 0.5
    cache = B.KvCache8(1, 3, heads, kvh, hd, 40, block=16)
    fill(cache, "e4m3", 21)
    state = held(cache, 0, "e4m3")
    qk, win = B.QkNorm(heads, kvh, hd, theta=1e4), B.Window(layer, max_rows=8)
    freqs = [1e4 ** (-2.0 * i / hd) for i in range(hd // 2)]
    rows, seqs = rows_of(B, [(2, 2, 21), (1, 0, 9), (2, 1, 40)])
    position = np.array([19, 20, 8, 38, 39])
    x = torch.randn(5, d, generator=g, device="cuda")
    fused = (x.double() @ wqkv.double().T).float().view(5, heads + 2 * kvh, hd)
    q, k, v = fused[:, :heads], fused[:, heads:heads + kvh], fused[:, heads + kvh:]
    qr, kr = qk.forward(q, k, i32(list(position)))
    cache.append(0, kr, v, rows)
    att = cache.attend(0, qr, rows)
    x1 = (x.double() + att.view(5, -1).double() @ wo.double().T).float()
    y, rt = win.forward(x1, routing=True)
    win.sync(), cache.sync()
    # the same in 64 bits, from the same fused rows
    qn, kn = ok.qknorm(q.cpu().numpy(), position, freqs), ok.qknorm(k.cpu().numpy(), position, freqs)
    assert np.abs(qr.double().cpu().numpy() - qn).max() <= 2.0 ** -19 * np.abs(qn).max()
    assert np.abs(kr.double().cpu().numpy() - kn).max() <= 2.0 ** -19 * np.abs(kn).max()
    ok.append(state[0], state[1], kr.cpu().numpy(), seqs, 16, "e4m3")
    ok.append(state[2], state[3], v.cpu().numpy(), seqs, 16, "e4m3")
    _same(cache, state, "e4m3")
    check_attend(att, qr, state, seqs, 16, hd ** -0.5)
    ref = oracle.moe_window(x1.cpu().numpy(), omoe(layer))
    keep = np.array([margin_accept(omoe(layer))(r) for r in x1.cpu().numpy()])
    assert keep.any()
    assert np.array_equal(rt["topk_idx"].cpu().numpy()[keep], ref["topk_idx"][keep])
    rms = np.sqrt(np.mean(ref["y"] ** 2))
    assert np.abs(y.double().cpu().numpy() - ref["y"])[keep].max() <= 2e-3 * rms
    win.close(), qk.close(), cache.close()


def test_refuses_outputs_over_inputs(B):
    cache = B.KvCache8(1, 1, 2, 2, 64, 40, block=16)
    fill(cache, "e4m3", 3)
    rows, _ = rows_of(B, [(2, 0, 6)])
    q = torch.ones(2, 2, 64, device="cuda")
    with pytest.raises(B.StrataError):
        cache.attend(0, q, rows, out=q)
    with pytest.raises(B.StrataError):
        cache.read(0, rows, k=q, v=q)
    cache.sync()
    assert (q == 1).all()


FIRST = """
import torch
from slot_decode_window_gb300 import binding as B
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
torch.manual_seed(5)
caches = [B.KvCache8(1, 1, 8, 2, 64, 200, block=16) for _ in range(2)]
qk = B.QkNorm(8, 2, 64)
q, k, v = (torch.randn(40, h, 64, device="cuda") for h in (8, 2, 2))
pos = torch.arange(40, dtype=torch.int32, device="cuda")
calls = [(B.KvRows(i32([0, 40]), i32([0]), i32([40]), 40, 40), slice(0, 40)),
         (B.KvRows(i32([0, 1]), i32([0]), i32([41]), 1, 1), slice(0, 1))]
def run(cache):
    out = []
    qq, kk = qk.forward(q, k, pos)
    for rows, part in calls:  # the kernels for many rows and for few
        cache.append(0, kk[part], v[part], rows)
        out += [cache.attend(0, qq[part], rows), *cache.read(0, rows)]
    return out
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run(caches[0])
g.replay()
want = run(caches[1])
for c in caches:
    c.sync()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0].abs().max() > 0
print("same")
"""


def test_the_first_calls_of_a_process_are_captured(B):
    """No call has run before the capture: nothing that a launch needs is made by an earlier one."""
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.split() == ["same"], r.stderr[-2000:]
