"""Pins of the oracle of the head norms, the rotation and the 8-bit caches (no GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import kv8 as ok


def test_e4m3_codes_are_the_formats_numbers():
    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    finite = np.isfinite(want)
    assert finite.sum() == 254
    np.testing.assert_array_equal(ok.code_values(c, "e4m3")[finite], want[finite])
    np.testing.assert_array_equal(ok.code_values(c, "int8"), c.view(np.int8).astype(np.float64))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_nearest_by_search(fmt):
    """Against the nearest of all code numbers; ties go to the even code."""
    nums = np.unique(ok.code_values(np.array([c for c in range(256) if fmt == "int8" and c != 128
                                              or fmt == "e4m3" and c & 127 != 127], dtype=np.uint8), fmt))
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(4000) * 60, (nums[1:] + nums[:-1]) / 2, nums, [1e9, -1e9]])
    for x, y in zip(v, ok.nearest(v, fmt)):
        d = np.abs(nums - x)
        best = nums[d == d.min()]
        assert y in best
        if len(best) == 2:  # a tie: the even one is a multiple of twice the step
            assert (y / abs(best[1] - best[0])) % 2 == 0
    assert ok.nearest(np.array([np.nan]), fmt)[0] == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_least_exponent_by_trying(fmt):
    q = ok.QMAX[fmt]
    rng = np.random.default_rng(1)
    some = [float(np.float32(x)) for x in np.exp2(rng.uniform(-60, 60, 500))]
    edges = [q * 2.0 ** e * f for e in (-48, -5, 0, 9, 47) for f in (1.0, 1 + 2 ** -23, 1 - 2 ** -24)]
    for a in some + edges:
        fits = [e for e in range(-48, 48) if a <= q * 2.0 ** e]
        assert ok.least_exponent(a, fmt) == (fits[0] if fits else 47)
    assert ok.least_exponent(0.0, fmt) == -48


def test_append_hand_worked():
    """int8, block 16: 1.0 needs e = -6 (127/64 > 1 > 127/128); 3.0 next to it needs e = -5 and halves the held code."""
    codes, exps = np.zeros((1, 1, 32, 1)), np.zeros((1, 1, 2), dtype=np.int64)
    ok.append(codes, exps, np.array([[[1.0]]]), [(0, 1, 0, 1)], 16, "int8")
    assert codes[0, 0, 0, 0] == 64 and exps[0, 0, 0] == -6
    ok.append(codes, exps, np.array([[[3.0]], [[0.1]]]), [(0, 2, 0, 3)], 16, "int8")
    assert list(codes[0, 0, :3, 0]) == [32, 96, 3] and exps[0, 0, 0] == -5
    ok.append(codes, exps, np.array([[[0.25]]]), [(0, 1, 0, 17)], 16, "int8")  # the next block starts anew
    assert codes[0, 0, 16, 0] == 64 and exps[0, 0, 1] == -8


@pytest.mark.parametrize("fmt,rel", [("e4m3", 2.0 ** -4), ("int8", 2.0 ** -7)])
def test_round_trip_error(fmt, rel):
    """e4m3: half a step is 2^-4 of a normal value; int8: half a step is at most 1/128 of the block's largest."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((40, 2, 8))
    codes, exps = np.zeros((1, 2, 48, 8)), np.zeros((1, 2, 3), dtype=np.int64)
    ok.append(codes, exps, x, [(0, 40, 0, 40)], 16, fmt)
    back = ok.held_values(codes, exps, 0, 0, 40, 16).transpose(1, 0, 2)
    for b in range(3):
        s = slice(16 * b, min(40, 16 * b + 16))
        for h in range(2):
            a = np.abs(x[s, h]).max()
            bound = np.abs(x[s, h]) * rel + a * 2.0 ** -18 if fmt == "e4m3" else a * rel
            assert (np.abs(back[s, h] - x[s, h]) <= bound).all()


def test_attention_equals_the_fp16_cache_oracle_on_the_held_values():
    rng = np.random.default_rng(3)
    kc, ke = np.zeros((2, 2, 20, 8)), np.zeros((2, 2, 2), dtype=np.int64)
    vc, ve = kc.copy(), ke.copy()
    for c, e in ((kc, ke), (vc, ve)):
        ok.append(c, e, rng.standard_normal((18, 2, 8)), [(0, 18, 1, 18)], 16, "e4m3")
    q = rng.standard_normal((2, 4, 8))
    got = ok.attend(q, kc, ke, vc, ve, [(0, 2, 1, 18)], 16, 1 / math.sqrt(8))
    hk = np.stack([ok.held_values(kc, ke, s, 0, 20, 16) for s in range(2)])
    hv = np.stack([ok.held_values(vc, ve, s, 0, 20, 16) for s in range(2)])
    for r in range(2):
        want = oa.attention_row(q[r].reshape(-1), hk, hv, 1, 16 + r, heads=4)
        np.testing.assert_allclose(got[r].reshape(-1), want, rtol=1e-13, atol=1e-14)
    empty = ok.attend(q, kc, ke, vc, ve, [(0, 2, 1, 1)], 16, 1.0)  # the first row sees nothing
    assert (empty[0] == 0).all() and np.isfinite(empty[1]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_and_norm(interleaved):
    """Position 0 is the norm alone; the rotation keeps lengths; products of rotated rows depend on distance only;
    a quarter turn by hand."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((1, 2, 8))
    f = [1.0, 0.1, 0.01]
    n = ok.qknorm(x, [0], f, interleaved=interleaved)
    np.testing.assert_allclose(np.mean(n * n, -1), 1, rtol=1e-5)
    np.testing.assert_allclose(np.linalg.norm(ok.qknorm(x, [77], f, interleaved=interleaved), axis=-1),
                               np.linalg.norm(n, axis=-1), rtol=1e-14)
    y = rng.standard_normal((1, 2, 8))
    d = [np.sum(ok.qknorm(x, [a], f, interleaved=interleaved) * ok.qknorm(y, [a + 5], f, interleaved=interleaved))
         for a in (0, 10 ** 6)]
    assert abs(d[0] - d[1]) < 1e-12
    e = np.zeros((1, 1, 8))
    e[..., 0] = 1
    z = ok.qknorm(e, [1], [math.pi / 2], norm=False, interleaved=interleaved)
    want = np.zeros(8)
    want[1] = 1  # one pair: dims 0 and 1 either way
    np.testing.assert_allclose(z[0, 0], want, atol=1e-15)
