"""The 8-bit caches' calls at the ends of what their documentation allows: scores of any size, sums over long caches,
batches of very unlike sequences, sequences that are left out, and a workspace that a forbidden overlap disturbed."""
import numpy as np
import pytest
import torch

from oracle import kv8 as ok
from tests.kv8_helpers import DTYPES, check_attend, fill, half_step, held, i32, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from slot_decode_window_gb300 import binding, build
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()
    return binding


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("n", [2, 3, 40])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("way", [1, -1])
@pytest.mark.parametrize("power", [14, 20, 24, 25, 26, 27, 28, 30, 60, 90])
def test_attend_scores_of_any_size(B, n, dtype, way, power):
    """Three equal keys, in units of their own, score 2^power times what keys do otherwise and far above the rest (way
    = -1: all scores are negative, theirs least so): a row is the mean of their values.

    Bound: equal scores give equal weights, whatever they are, and every other weight is below 2^-60 of them, so what
    is left are f32 roundings (the sums, the joins, exp2 and the quotient: under 16 of 2^-24 relative to the values'
    mean magnitude) and the result's own."""
    heads, kvh, hd, block, length = 4, 2, 128, 32, 300
    cache = B.KvCache8(1, 1, heads, kvh, hd, length, block=block)
    fill(cache, "e4m3", 1)
    u = _randn(1, kvh, hd)
    k, v = 0.1 * _randn(2, length, kvh, hd), _randn(3, length, kvh, hd).clamp(-3.9, 3.9)
    k += 0 if way > 0 else -3 * u
    same = [5, 130, 250]
    k[same] = way * u  # (way = -1: -u scores above -3 u)
    k.clamp_(-15.5, 15.5)
    k[..., 0] = 16.0  # every block has the same exponent
    v[..., 0] = 4.0
    cache.append(0, k, v, rows_of(B, [(length, 0, length)])[0])
    state = held(cache, 0, "e4m3")
    q = u.repeat_interleave(heads // kvh, 0) + 0.02 * _randn(4, n, heads, hd)
    q[..., 0] = 0
    q = q.to(DTYPES[dtype])
    scale = 2.0 ** power
    rows, _ = rows_of(B, [(n, 0, length)])
    out = cache.attend(0, q, rows, scale=scale)
    again = cache.attend(0, -q, rows, scale=-scale)
    cache.sync()
    assert torch.equal(out, again)
    kk, vv = ok.held_values(state[0], state[1], 0, 0, length, block), ok.held_values(state[2], state[3], 0, 0, length, block)
    got, qq = out.double().cpu().numpy(), q.double().cpu().numpy()
    for r in range(n):
        for h in range(heads):
            s = scale * np.log2(np.e) * (kk[h // 2, :length - n + r + 1] @ qq[r, h])
            rest = np.delete(s, same)
            assert (s[same] == s[5]).all() and s[5] - rest.max() > 60 and (way > 0 or s.max() < 0)
            want, size = vv[h // 2, same].mean(0), np.abs(vv[h // 2, same]).mean(0)
            off = 16 * 2.0 ** -24 * size
            bound = off + half_step(q.dtype) * (np.abs(want) + off)
            assert (np.abs(got[r, h] - want) <= bound).all(), (r, h, np.abs(got[r, h] - want).max())


@pytest.mark.parametrize("n", [2, 40])
def test_attend_zero_keys_under_the_largest_factors(B, n):
    """Keys of zero in blocks of the largest exponent, queries near the end of f32's range: every score is 0, and the
    product of the powers of two that it is multiplied with does not fit f32."""
    cache = B.KvCache8(1, 1, 4, 2, 128, 200, block=16)
    fill(cache, "e4m3", 2)
    cache.k.zero_()
    cache.k_exp.fill_(ok.E_MAX + ok.BIAS)
    state = held(cache, 0, "e4m3")
    rows, seqs = rows_of(B, [(n, 0, 200)])
    for scale in (1.0, -3.0):
        q = _randn(5, n, 4, 128) * 2.0 ** 110
        out = cache.attend(0, q, rows, scale=scale)
        cache.sync()
        check_attend(out, q, state, seqs, 16, abs(scale))


@pytest.mark.parametrize("fmt,kvh,group,n,hd", [("e4m3", 8, 1, 1, 128), ("int8", 4, 8, 2, 128), ("int8", 8, 1, 1, 64),
                                                ("e4m3", 4, 8, 2, 64)])
def test_attend_long_sums_of_f32_rows_do_not_drift(B, fmt, kvh, group, n, hd):
    """More items than CTAs, each of 131071 positions, so that whole items are summed by one CTA: positive values under
    nearly equal weights, whose mean error over rows and dims shows what sums lose on one side.

    Bound: products that cut off lose under 2^-23 of a sum at each of the 32 adds (16 times 16 positions, two parts)
    that it stays in one accumulator, half of that for a sum that grows evenly: 16 * 2^-23.  What rounds errs to
    both sides: the denominator's adds (one a unit of 64 positions and warp, at most 12 warps a CTA in groups of 4) by
    less than 2^-24 of the sum each, independently for each of the rows looked at; six standard deviations of their mean."""
    length, n_seq, heads = 131071, 152, kvh * group
    cache = B.KvCache8(1, 2, heads, kvh, hd, length, block=64, format=fmt)
    fill(cache, fmt, 3, spread=0.0)
    cache.v &= 0x7F
    q = 0.02 * _randn(6, n_seq * n, heads, hd)
    rows, _ = rows_of(B, [(n, i % 2, length) for i in range(n_seq)])
    out = cache.attend(0, q, rows)
    cache.sync()
    off, seqs = [], (0, 51, 76, 151)
    table = torch.from_numpy(ok.code_values(np.arange(256), fmt)).cuda()
    for h in range(kvh):
        for slot in range(2):
            k, v = (table[c[0, slot, h].int()] * torch.exp2(e[0, slot, h].double() - ok.BIAS).repeat_interleave(64)[:length, None]
                    for c, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)))
            for i in seqs:
                if i % 2 != slot:
                    continue
                for r in range(n):
                    at, seen = i * n + r, length - n + r + 1
                    p = torch.softmax(q[at, h * group:(h + 1) * group].double() @ k[:seen].T * hd ** -0.5, -1)
                    want = p @ v[:seen]
                    off.append(((out[at, h * group:(h + 1) * group].double() - want) / want).mean(-1))
    off = torch.cat(off)
    units = length / 64 / (3 if n * group <= 8 else 2)
    assert abs(off.mean().item()) <= 16 * 2.0 ** -23 + 6 * 2.0 ** -24 * (units / len(off)) ** 0.5, off.mean().item()


def _reported(B, cache):
    with pytest.raises(B.StrataError) as e:
        cache.sync()
    assert e.value.status == B.STRATA_EDEVICE
    cache.sync()  # reported once


@pytest.mark.parametrize("start,length", [([0, 2, 4], [41, 9]), ([0, 2, 4], [-1, 9]), ([0, 2, 4], [1, 9]),
                                          ([0, 3, 5], [9, 9]), ([4, 2, 4], [9, 9])])
def test_append_a_sequence_that_is_left_out_takes_no_slot(B, start, length):
    """The first of two sequences of one slot has a length out of range or below its rows, too many rows, or rows out of
    order: the second is written."""
    cache = B.KvCache8(1, 2, 4, 2, 64, 40, block=16)
    fill(cache, "e4m3", 22)
    state = held(cache, 0, "e4m3")
    k, v = _randn(7, 6, 2, 64), _randn(8, 6, 2, 64)
    cache.append(0, k, v, B.KvRows(i32(start), i32([1, 1]), i32(length), n_rows=6, max_rows=2))
    _reported(B, cache)
    for c, e, x in ((state[0], state[1], k), (state[2], state[3], v)):
        ok.append(c, e, x.cpu().numpy(), [(start[1], start[2] - start[1], 1, length[1])], 16, "e4m3")
    for got, want in zip(held(cache, 0, "e4m3"), state):
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("fmt,dtype,hd,kvh,block", [("e4m3", "f32", 128, 2, 16), ("int8", "bf16", 64, 3, 32),
                                                    ("e4m3", "f16", 128, 1, 128), ("int8", "f32", 64, 1, 64)])
@pytest.mark.parametrize("n_seq", [9, 70, 300])
def test_append_and_read_of_very_unlike_sequences(B, fmt, dtype, hd, kvh, block, n_seq):
    """Single rows, sequences without rows, a prompt and some that are left out in one call, where the places of the
    longest sequence for each would be many times the rows: codes, exponents and values bit for bit, and what is left
    out is not touched."""
    big, ctx = 601, 700
    cache = B.KvCache8(1, n_seq, kvh, kvh, hd, ctx, block=block, format=fmt)
    fill(cache, fmt, n_seq)
    state = held(cache, 0, fmt)
    rng = np.random.default_rng(n_seq)
    n = rng.choice([0, 1, 1, 1, 2, 20], n_seq)
    at = n_seq // 2
    n[at], n[0] = big, 1
    start = np.concatenate([[0], np.cumsum(n)])
    length = np.minimum(ctx, n + rng.integers(0, 70, n_seq))
    slot = rng.permutation(n_seq)
    rows = int(start[-1])
    bad = [i for i in (1, n_seq - 2) if i != at]  # a length out of range; a slot out of range
    length[1], slot[n_seq - 2] = ctx + 1, -1
    r = B.KvRows(i32(start), i32(slot), i32(length), n_rows=rows + 5, max_rows=big)
    k, v = (_randn(s, rows + 5, kvh, hd).to(DTYPES[dtype]) for s in (9, 10))
    cache.append(0, k, v, r)
    _reported(B, cache)
    good = [(int(start[i]), int(n[i]), int(slot[i]), int(length[i])) for i in range(n_seq) if i not in bad]
    for c, e, x in ((state[0], state[1], k), (state[2], state[3], v)):
        ok.append(c, e, x.float().cpu().numpy(), good, block, fmt)
    for got, want in zip(held(cache, 0, fmt), state):
        np.testing.assert_array_equal(got, want)
    ko, vo = (torch.full_like(k, 7.0) for _ in range(2))
    cache.read(0, r, k=ko, v=vo)
    _reported(B, cache)
    for got, c, e in ((ko, state[0], state[1]), (vo, state[2], state[3])):
        want = torch.full(got.shape, 7.0)
        for i in bad:
            want[start[i]:start[i + 1]] = 0
        for row0, m, s, end in good:
            x = ok.held_values(c, e, s, end - m, end, block).transpose(1, 0, 2)
            want[row0:row0 + m] = torch.from_numpy(np.ascontiguousarray(x)).float()
        assert torch.equal(got.cpu(), want.to(got.dtype))


@pytest.mark.parametrize("n", [120, 600])
def test_append_and_read_of_sequences_over_one_another(B, n):
    """row_start that goes back: every other sequence is out of order, those between share their rows, so the pieces are
    more than the rows could need."""
    cache = B.KvCache8(1, 40, 2, 2, 64, n + 80, block=16)
    fill(cache, "e4m3", 23)
    state = held(cache, 0, "e4m3")
    start = [0, n] * 30 + [0]
    slot = [i // 2 for i in range(60)]
    length = [n + 30] * 60
    k, v = _randn(11, n + 10, 2, 64), _randn(12, n + 10, 2, 64)
    r = B.KvRows(i32(start), i32(slot), i32(length), n_rows=n + 10, max_rows=n + 5)
    cache.append(0, k, v, r)
    _reported(B, cache)
    for c, e, x in ((state[0], state[1], k), (state[2], state[3], v)):
        ok.append(c, e, x.cpu().numpy(), [(0, n, i, n + 30) for i in range(30)], 16, "e4m3")
    for got, want in zip(held(cache, 0, "e4m3"), state):
        np.testing.assert_array_equal(got, want)
    ko, vo = (torch.full_like(k, 7.0) for _ in range(2))
    cache.read(0, B.KvRows(i32(start), i32([3] * 60), i32(length), n_rows=n + 10, max_rows=n + 5), k=ko, v=vo)
    _reported(B, cache)
    for got, c, e in ((ko, state[0], state[1]), (vo, state[2], state[3])):
        want = ok.held_values(c, e, 3, 30, n + 30, 16).transpose(1, 0, 2)
        assert np.array_equal(got[:n].cpu().numpy(), want.astype(np.float32)) and (got[n:] == 7).all()


def test_append_of_the_most_sequences_beside_one_long_prompt(B):
    """1024 sequences of which one has 2^18 + 3 rows, 64 kv heads and blocks of 16: the same bits as that one alone."""
    n, kvh, hd = (1 << 18) + 3, 64, 64
    x = _randn(13, n, 1, hd).bfloat16() * torch.exp2(torch.arange(kvh, device="cuda") % 7 - 3.0)[:, None].bfloat16()
    cache = [B.KvCache8(1, 1, kvh, kvh, hd, n, block=16) for _ in range(2)]
    for c, seqs in zip(cache, ([(0, 0, 0)] * 500 + [(n, 0, n)] + [(0, 0, 0)] * 523, [(n, 0, n)])):
        for t in (c.k, c.v, c.k_exp, c.v_exp):
            t.zero_()
        c.append(0, x, x, rows_of(B, seqs)[0])
        c.sync()
    assert torch.equal(cache[0].k, cache[1].k) and torch.equal(cache[0].k_exp, cache[1].k_exp)
    assert torch.equal(cache[0].v, cache[1].v) and torch.equal(cache[0].v_exp, cache[1].v_exp)
    assert cache[0].k.any() and torch.equal(cache[0].k, cache[0].v)


def test_sync_reports_and_clears_joins_that_were_left_unfinished(B, monkeypatch):
    """Counters of the joins that are not back at zero, as an overlap of two attends may leave them (put there by the
    host): the next sync reports them and the call after it is right again."""
    cache = B.KvCache8(1, 1, 8, 2, 128, 6000, block=64)
    fill(cache, "e4m3", 24)
    state = held(cache, 0, "e4m3")
    for n in (1, 60):
        rows, seqs = rows_of(B, [(n, 0, 6000)])
        q = _randn(14, n, 8, 128)
        want = cache.attend(0, q, rows)
        cache.sync()
        check_attend(want, q, state, seqs, 64, 128 ** -0.5)
        monkeypatch.setenv("STRATA_FAULT", "overlap")
        cache.attend(0, q, rows)
        monkeypatch.delenv("STRATA_FAULT")
        _reported(B, cache)
        again = cache.attend(0, q, rows)
        cache.sync()
        assert torch.equal(again, want)


def _valid(start, slot, length, n_rows, max_rows, n_slots, ctx):
    """(sequences whose rows may be touched, those of them that are not left out), as the header has it."""
    rows = [(a, b - a, s, n) for a, b, s, n in zip(start, start[1:], slot, length)
            if 0 <= a <= b <= n_rows and b - a <= max_rows]
    return rows, [q for q in rows if 0 <= q[2] < n_slots and 0 <= q[3] <= ctx]


@pytest.mark.parametrize("by", [1, 20])  # few rows, many rows
@pytest.mark.parametrize("start,slot,length,most", [
    ([0, -1, 2], [1, 0], [5, 6], 2), ([4, 2, 4], [1, 0], [5, 6], 2), ([0, 7, 7], [1, 0], [5, 6], 8),
    ([0, 3, 4], [1, 0], [5, 6], 2), ([0, 2, 1, 3], [1, 0, 2], [5, 6, 7], 2),
    ([0, 2, 4], [3, 0], [5, 6], 2), ([0, 2, 4], [-1, 0], [5, 6], 2), ([0, 2, 4], [1, 0], [50, 6], 2),
    ([0, 2, 4], [1, 0], [-1, 6], 2), ([0, 2, 4], [1, 0], [6, 50], 2)])
def test_what_is_skipped_or_left_out_is_not_touched(B, start, slot, length, most, by):
    """Every row and code against the header's rules: rows of a skipped sequence stay, rows of one that is left out become
    zero, and neither changes the caches.  Rows that two sequences name (row_start goes back) have no defined output."""
    start, length, most, n_rows, ctx = [a * by for a in start], [n * by for n in length], most * by, 6 * by, 40 * by
    cache = B.KvCache8(1, 3, 4, 2, 64, ctx, block=16)
    fill(cache, "e4m3", 25)
    state = held(cache, 0, "e4m3")
    q, k, v = _randn(15, n_rows, 4, 64), _randn(16, n_rows, 2, 64), _randn(17, n_rows, 2, 64)
    r = B.KvRows(i32(start), i32(slot), i32(length), n_rows=n_rows, max_rows=most)
    rows, good = _valid(start, slot, length, n_rows, most, 3, ctx)
    out = torch.full_like(q, 3.0)
    cache.attend(0, q, r, out=out)
    _reported(B, cache)
    ko, vo = torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    cache.read(0, r, k=ko, v=vo)
    _reported(B, cache)
    mine, owners = np.full(n_rows, -1), np.zeros(n_rows, int)
    for i, x in enumerate(rows):
        mine[x[0]:x[0] + x[1]] = i if x in good else -2
        owners[x[0]:x[0] + x[1]] += 1
    assert (out[mine == -1] == 3).all() and (ko[mine == -1] == 3).all() and (vo[mine == -1] == 3).all()
    assert (out[mine == -2] == 0).all() and (ko[mine == -2] == 0).all() and (vo[mine == -2] == 0).all()
    for row0, n, s, end in good:
        one = owners[row0:row0 + n] == 1
        for got, c, e in ((ko, state[0], state[1]), (vo, state[2], state[3])):
            want = ok.held_values(c, e, s, end - n, end, 16).transpose(1, 0, 2).astype(np.float32)
            assert np.array_equal(got[row0:row0 + n].cpu().numpy()[one], want[one])
        for j in np.flatnonzero(one):  # as a sequence of this row alone, at the position that it has
            check_attend(out[row0 + j:row0 + j + 1], q[row0 + j:row0 + j + 1], state, [(0, 1, s, end - n + j + 1)], 16, 0.125)
    cache.append(0, k, v, r)
    _reported(B, cache)
    for c, e, x in ((state[0], state[1], k), (state[2], state[3], v)):
        ok.append(c, e, x.cpu().numpy(), good, 16, "e4m3")
    for got, want in zip(held(cache, 0, "e4m3"), state):
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("heads,kvh", [(8, 2), (3, 3), (16, 1)])
@pytest.mark.parametrize("seqs", [[(400, 0, 37)], [(400, 0, 37), (70, 1, 300)], [(70, 1, 300), (400, 0, 37), (1, 2, 0)],
                                  [(400, 0, 0), (129, 2, 128)], [(400, 0, 400), (300, 1, 1), (300, 2, 129)]])
def test_attend_whole_tiles_of_rows_that_see_nothing(B, heads, kvh, seqs):
    """Lengths so far below the rows that row tiles at a sequence's start have nothing to do."""
    for dtype in ("f32", "bf16"):
        cache = B.KvCache8(1, 3, heads, kvh, 64, 400, block=32, format="int8")
        fill(cache, "int8", 26)
        state = held(cache, 0, "int8")
        rows, os_ = rows_of(B, seqs, n_rows=sum(s[0] for s in seqs) + 3)
        q = _randn(18, rows.n_rows, heads, 64).to(DTYPES[dtype])
        out = torch.full_like(q, 3.0)
        cache.attend(0, q, rows, out=out)
        cache.sync()
        assert (out[-3:] == 3).all()
        check_attend(out, q, state, os_, 32, 0.125)


@pytest.mark.parametrize("n", [1, 6, 12, 70])  # one row tile of 8, of 16, two of 16, the many-row kernel
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt,heads,kvh,hd", [("int8", 4, 2, 128), ("int8", 4, 2, 64), ("e4m3", 4, 2, 64), ("e4m3", 6, 2, 128)])
@pytest.mark.parametrize("length", [300, 2300])  # in one part, and in parts that are joined
def test_attend_large_scores_in_every_variant(B, n, dtype, fmt, heads, kvh, hd, length):
    """As test_attend_scores_of_any_size, at 2^26 and with the equal keys far apart: a row is the mean of their values, under
    the bound derived there."""
    block, scale, group = 32, 2.0 ** 26, heads // kvh
    cache = B.KvCache8(1, 1, heads, kvh, hd, length, block=block, format=fmt)
    fill(cache, fmt, 1)
    u = _randn(1, kvh, hd).sign()
    k, v = 0.1 * _randn(2, length, kvh, hd), _randn(3, length, kvh, hd).clamp(-3.9, 3.9)
    same = [5, 130, length - 80]
    k[same] = u
    k[..., 0] = 16.0
    v[..., 0] = 4.0
    cache.append(0, k, v, rows_of(B, [(length, 0, length)])[0])
    kc, ke, vc, ve = held(cache, 0, fmt)
    q = u.repeat_interleave(group, 0) + 0.02 * _randn(4, n, heads, hd)
    q[..., 0] = 0
    q = q.to(DTYPES[dtype])
    out = cache.attend(0, q, rows_of(B, [(n, 0, length)])[0], scale=scale)
    cache.sync()
    kk, vv = ok.held_values(kc, ke, 0, 0, length, block), ok.held_values(vc, ve, 0, 0, length, block)
    got, qq = out.double().cpu().numpy(), q.double().cpu().numpy()
    for r in range(n):
        for h in range(heads):
            s = scale * np.log2(np.e) * (kk[h // group, :length - n + r + 1] @ qq[r, h])
            assert (s[same] == s[5]).all() and s[5] - np.delete(s, same).max() > 60
            want, size = vv[h // group, same].mean(0), np.abs(vv[h // group, same]).mean(0)
            off = 16 * 2.0 ** -24 * size
            assert (np.abs(got[r, h] - want) <= off + half_step(q.dtype) * (np.abs(want) + off)).all(), (r, h)


def test_captured_append_and_read_of_unlike_sequences_follow_their_buffers(B):
    """The list of pieces is made on the device: captured once, replayed as other sequences take the rows."""
    n_seq, n_rows, most = 60, 700, 640
    one, two = (B.KvCache8(1, n_seq, 2, 2, 64, 700, block=16, format="int8") for _ in range(2))
    for c in (one, two):
        fill(c, "int8", 27)
    start, slot, length = i32([0] * (n_seq + 1)), i32(range(n_seq)), i32([0] * n_seq)
    rows = B.KvRows(start, slot, length, n_rows=n_rows, max_rows=most)
    k, v = _randn(19, n_rows, 2, 64), _randn(20, n_rows, 2, 64)
    out, want = ([torch.empty_like(k), torch.empty_like(k)] for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one.append(0, k, v, rows)
        one.read(0, rows, k=out[0], v=out[1])
    for big in (0, 59, 31):
        n = [1 if i % 3 else 0 for i in range(n_seq)]
        n[big] = most
        start.copy_(i32([0] + list(np.cumsum(n))))
        length.copy_(i32([x + (7 * i + big) % 50 for i, x in enumerate(n)]))
        k.normal_(), v.normal_()
        for t in out + want:
            t.fill_(5.0)
        graph.replay()
        for i in range(n_seq):  # one sequence at a time
            if n[i]:
                a = int(start[i])
                alone, _ = rows_of(B, [(n[i], i, int(length[i]))])
                two.append(0, k[a:a + n[i]], v[a:a + n[i]], alone)
                two.read(0, alone, k=want[0][a:a + n[i]], v=want[1][a:a + n[i]])
        one.sync(), two.sync()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        for a, b in ((one.k, two.k), (one.v, two.v), (one.k_exp, two.k_exp), (one.v_exp, two.v_exp)):
            assert torch.equal(a, b)
