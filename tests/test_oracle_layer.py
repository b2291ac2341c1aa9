"""Pins of the oracle of a layer's other parts to something other than itself."""
import numpy as np
import pytest

import oracle
from oracle import layer as ol
from slot_decode_window_gb300 import workloads as wlm
from tests.helpers import oqmat


def test_linear_is_the_dense_product_row_by_row():
    q = wlm.make_qmat(3, 32, 64, 4, 32, [1, 2, 3], "cpu")
    w = oqmat(q)
    x = np.random.default_rng(0).standard_normal((7, 64))
    y = ol.linear(x, w, offsets=[1, 3, 3, 6])
    assert np.isnan(y[0]).all() and np.isnan(y[6]).all()
    for t, m in ((1, 0), (2, 0), (3, 2), (4, 2), (5, 2)):
        W = oracle.dequant(w, m)
        assert np.allclose(y[t], [sum(W[r, c] * x[t, c] for c in range(64)) for r in range(32)], rtol=1e-12)


def test_linear_pair_and_sorting_make_the_moe_window():
    """Router's choice, order, products and back over a layer's experts are the window oracle's rows."""
    spec = wlm.MoESpec(64, 6, 2, 32, 0, 4, 32)
    layer = wlm.make_moe_layer(spec, seed=0, cfg_id=70, device="cpu")
    from tests.helpers import omoe
    om = omoe(layer)
    x = np.random.default_rng(1).standard_normal((5, 64))
    logits = (x @ om.router_w.astype(np.float64).T).astype(np.float32)
    idx, w = ol.route(logits, 2, False)
    counts, offsets, entries, place = ol.order(idx, 6)
    xs = ol.gather(x, place, 2)
    h = ol.linear(xs, om.gate, om.up, offsets)
    y = ol.combine(ol.linear(h, om.down, offsets=offsets), place, 2, w)
    for t in range(5):
        ref = oracle.moe_row(x[t], om)[0]
        assert np.abs(y[t] - ref).max() <= 1e-5 * np.sqrt(np.mean(ref * ref))
    assert counts.sum() == 10 and sorted(entries) == list(range(10))
    got = oracle.group_rows(idx, 6)
    assert np.array_equal(got[0], counts)


def test_route_against_brute_force_and_masks():
    l = np.array([[1.0, 3.0, 3.0, -np.inf], [np.nan, -np.inf, -np.inf, -np.inf], [np.inf, 0, np.inf, 1]], np.float32)
    idx, w = ol.route(l, 3, False)
    assert idx.tolist() == [[1, 2, 0], [-1, -1, -1], [0, 2, 3]]
    e = np.exp(np.array([3.0, 3.0, 1.0]) - 3)
    assert np.allclose(w[0], e / e.sum()) and not w[1].any() and np.allclose(w[2], [0.5, 0.5, 0])
    _, wr = ol.route(l[:1], 2, True)
    assert np.allclose(wr, 0.5)


def test_gradient_against_differences():
    rng = np.random.default_rng(2)
    place = np.array([3, -1, 0, 2, 1, 5])
    z, w, dy = rng.standard_normal((6, 4)), rng.standard_normal((3, 2)), rng.standard_normal((3, 4))
    f = lambda z, w: (ol.combine(z, place, 2, w) * dy).sum()
    dz, dw = ol.combine_backward(dy, z, place, 2, w)
    for p in range(6):
        for c in range(4):
            d = np.zeros_like(z)
            d[p, c] = 1e-5
            num = (f(z + d, w) - f(z - d, w)) / 2e-5
            assert abs(num - (dz[p, c] if p != 4 else 0)) < 1e-8
    for t in range(3):
        for j in range(2):
            d = np.zeros_like(w)
            d[t, j] = 1e-5
            assert abs((f(z, w + d) - f(z, w - d)) / 2e-5 - dw[t, j]) < 1e-8


def test_block_norm_by_hand():
    x, y = np.array([[3.0, 4.0]]), np.array([[6.0, -8.0]])
    h, n = ol.block_norm(x, y, after=np.array([1.0, 2.0]), before=np.ones(2), gate=np.array([[0.0]]), sigmoid=True, eps=0.0,
                         residual_scale=2.0, block_scale=4.0)
    r = np.sqrt(50.0)
    assert np.allclose(h, [[6 + 4 * 0.5 * 6 / r, 8 - 4 * 0.5 * 2 * 8 / r]])
    assert np.allclose((n * n).mean(), 1.0)
    assert np.allclose(ol.block_norm(x, before=np.ones(2), eps=0.0)[1], oracle.rmsnorm(x[0]), atol=1e-6)
    assert ol.block_norm(x, y)[1] is None and np.allclose(ol.block_norm(x, y)[0], x + y)
