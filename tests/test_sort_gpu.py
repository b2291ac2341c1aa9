"""Tokens sorted by expert and back on the GPU against the oracle."""
import numpy as np
import pytest
import torch

from oracle import layer as ol
from tests.layer_helpers import DTYPES, half_step, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from slot_decode_window_gb300 import binding, build
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()
    return binding


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("E,k", [(1, 1), (4, 4), (33, 3), (128, 8), (160, 8), (300, 16), (1024, 5)])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(B, E, k, renorm):
    """Equal logits, masked experts, rows with too few and with none, NaN, infinities, a bias, padded rows of logits.  The weights are
    quotients of sums of at most 1024 exponentials: ceil(E / 32) + 5 adds, the exponentials' 2 ulp and the differences' rounding
    (below 2^-24 of 60): under (E / 32 + 80) 2^-24."""
    g = torch.Generator(device="cuda").manual_seed(E)
    for T in (1, 5, 67):
        whole = torch.round(torch.randn(T, E + 3, generator=g, device="cuda") * 8) / 8
        l = whole[:, :E]
        l[T // 2, ::2] = -float("inf")
        if T > 4:
            l[1] = -float("inf")
            l[2, 0] = float("nan")
            l[3, E - 1] = float("inf")
            l[4] = 0.0
            l[4, ::3] = -0.0
        bias = torch.round(torch.randn(E, generator=g, device="cuda") * 4) / 4
        h = B.ExpertSort(E, k, renorm=renorm)
        for b in (None, bias):
            idx, w = h.route(l, bias=b)
            ri, rw = ol.route(l.cpu().numpy(), k, renorm, None if b is None else b.cpu().numpy())
            assert np.array_equal(idx.cpu().numpy(), ri)
            assert np.abs(_np(w) - rw).max() <= (E / 32 + 80) * 2.0 ** -24
        h.close()


def _check_plan(plan, idx, E):
    counts, offsets, entries, place = ol.order(idx.cpu().numpy(), E)
    for got, want in ((plan.counts, counts), (plan.offsets, offsets), (plan.entries, entries), (plan.place, place)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("E,k", [(1, 1), (7, 2), (128, 8), (1024, 3)])
def test_plan(B, E, k):
    """From no rows to more than one pass of every warp; all entries of one expert; none of any; values far outside."""
    rng = np.random.default_rng(E)
    h = B.ExpertSort(E, k)
    for T in (0, 1, 3, 255, 2100):
        idx = rng.integers(-1, E, (T, k))
        _check_plan(h.plan(i32(idx).reshape(T, k)), i32(idx).reshape(T, k), E)
    for fill in (E - 1, -1, E, 2 ** 31 - 1, -2 ** 31):
        idx = i32(np.full((700, k), fill))
        _check_plan(h.plan(idx), idx, E)
    h.close()


def test_plan_of_a_long_prompt(B):
    """Against a stable sort: 400,000 entries, skewed."""
    g = torch.Generator(device="cuda").manual_seed(1)
    idx = (torch.rand(50000, 8, generator=g, device="cuda") ** 3 * 132).to(torch.int32)  # 128 and above: no expert's
    h = B.ExpertSort(128, 8)
    plan = h.plan(idx)
    key = torch.where(idx.flatten() < 128, idx.flatten(), 128)
    order = torch.argsort(key, stable=True).to(torch.int32)
    n = int((key < 128).sum())
    assert torch.equal(plan.entries[:n], order[:n]) and (plan.entries[n:] == -1).all()
    assert torch.equal(plan.counts, torch.bincount(key, minlength=129)[:128].to(torch.int32))
    assert int(plan.offsets[-1]) == n
    live = plan.place >= 0
    assert int(live.sum()) == n and torch.equal(plan.entries[plan.place[live].long()], torch.nonzero(live).flatten().to(torch.int32))
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,k,width", [(1, 4, 1, 8), (37, 5, 3, 24), (130, 60, 8, 520), (9, 16, 16, 2048), (300, 8, 2, 4104)])
def test_rows_there_and_back(B, dtype, T, E, k, width):
    """gather, combine with and without weights and base, the gradient; padded rows, rows of no expert, in place; what is behind
    the last expert's rows and beside the rows stays.  Sums of at most 17 terms: 17 u32 of their sizes; dot products of n
    elements in 256 partial sums: (n / 256 + 16) u32 of theirs."""
    dt, u = DTYPES[dtype], 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(T)
    rng = np.random.default_rng(T)
    idx = rng.integers(0, E, (T, k))
    idx[rng.random((T, k)) < 0.2] = -1
    if T > 2:
        idx[T // 2] = -1
    h = B.ExpertSort(E, k)
    plan = h.plan(i32(idx))
    place = plan.place.cpu().numpy()
    x = torch.randn(T, width + 8, generator=g, device="cuda").to(dt)[:, :width]
    whole = torch.full((T * k, width + 8), 7.0, dtype=dt, device="cuda")
    xs = h.gather(plan, x, out=whole[:, :width])
    want = ol.gather(_np(x), place, k)
    gone = np.isnan(want[:, 0])
    assert np.array_equal(_np(xs)[~gone], want[~gone]) and (_np(xs)[gone] == 7).all() and (whole[:, width:] == 7).all()
    z = torch.randn(T * k, width, generator=g, device="cuda").to(dt)
    w = torch.rand(T, k, generator=g, device="cuda")
    base = torch.randn(T, width, generator=g, device="cuda").to(dt)
    half = half_step(dt)
    for ww, bb in ((w, base), (w, None), (None, base), (None, None)):
        out = base.clone() if bb is not None else None
        y = h.combine(plan, z, w=ww, base=out if bb is not None else None, out=out)
        wn = None if ww is None else ww.double().cpu().numpy()
        ref = ol.combine(_np(z), place, k, wn, None if bb is None else _np(bb))
        size = ol.combine(np.abs(_np(z)), place, k, wn, None if bb is None else np.abs(_np(bb)))
        tiny = 2.0 ** -25 if dtype == "f16" else 0.0
        assert (np.abs(_np(y) - ref) <= half * np.abs(ref) * (1 + 1e-6) + 17 * u * size * 1.01 + tiny).all()
        if bb is None and T > 2:
            assert (y[T // 2] == 0).all()
    dy = torch.randn(T, width, generator=g, device="cuda").to(dt)
    for ww in (w, None):
        wn = None if ww is None else ww.double().cpu().numpy()
        rz, rw = ol.combine_backward(_np(dy), _np(z), place, k, wn)
        sw = ol.combine_backward(np.abs(_np(dy)), np.abs(_np(z)), place, k)[1]
        for inplace in (False, True):
            zz = z.clone()
            dz = zz if inplace else torch.full_like(z, 7.0)
            dz, dw = h.combine_backward(plan, dy, zz, w=ww, dz=dz)
            live = ~np.isnan(rz[:, 0])
            assert (np.abs(_np(dz)[live] - rz[live]) <= (half + u) * np.abs(rz[live]) * (1 + 1e-6) + (2.0 ** -25 if dtype == "f16" else 0)).all()
            assert np.array_equal(_np(dz)[~live], _np(z)[~live] if inplace else np.full_like(_np(z)[~live], 7.0))
            assert (np.abs(_np(dw) - rw) <= (width / 256 + 16) * u * sw).all()
    # gather's gradient: the sum of the copies' gradients
    dx = h.combine(plan, z)
    assert (np.abs(_np(dx) - ol.combine(_np(z), place, k)) <= half * np.abs(_np(dx)) * 1.01 + 17 * u * ol.combine(np.abs(_np(z)), place, k) + 2.0 ** -25).all()
    h.close()


def test_gradient_against_differences(B):
    """<dz, a> + <dw, b> is the derivative of <combine, dy> along (a, b): combine is bilinear, so the central difference along a
    direction is exact up to rounding (steps of 1/8, f32 sums of 24 terms)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    T, k, E, width = 40, 3, 6, 64
    h = B.ExpertSort(E, k)
    plan = h.plan(torch.randint(-1, E, (T, k), generator=g, device="cuda").to(torch.int32))
    z, a = (torch.randn(T * k, width, generator=g, device="cuda") for _ in range(2))
    w, b = (torch.randn(T, k, generator=g, device="cuda") for _ in range(2))
    dy = torch.randn(T, width, generator=g, device="cuda")
    dz, dw = h.combine_backward(plan, dy, z, w=w, dz=torch.zeros_like(z))
    n = int(plan.offsets[-1])
    a[n:] = 0
    t = 0.125
    up, down = (h.combine(plan, z + s * t * a, w=w + s * t * b) for s in (1, -1))
    num = ((up.double() - down.double()) * dy).sum() / (2 * t)
    ana = (dz.double() * a).sum() + (dw.double() * b * (plan.place.view(T, k) >= 0)).sum()
    size = (z.abs().sum() + a.abs().sum()) * (w.abs().max() + b.abs().max()) * dy.abs().max() * 8
    assert abs(num - ana) <= 2.0 ** -20 * size
    h.close()


def test_places_outside_are_passed_over(B):
    h = B.ExpertSort(4, 2)
    plan = h.plan(i32([[0, 1], [2, 3], [1, 1]]))
    plan.place.copy_(i32([0, 6, -5, 2 ** 31 - 1, 1, -2 ** 31]))
    x = torch.randn(3, 16, device="cuda")
    xs = h.gather(plan, x, out=torch.full((6, 16), 7.0, device="cuda"))
    assert torch.equal(xs[0], x[0]) and torch.equal(xs[1], x[2]) and (xs[2:] == 7).all()
    y = h.combine(plan, xs)
    assert torch.equal(y[0], x[0]) and (y[1] == 0).all() and torch.equal(y[2], x[2])
    dz, dw = h.combine_backward(plan, x, xs, dz=torch.full((6, 16), 7.0, device="cuda"))
    assert (dz[2:] == 7).all() and dw[1].tolist() == [0, 0] and dw[0, 1] == 0
    h.close()


def test_captured_and_on_another_stream(B):
    """One captured run from logits to rows and back follows new contents; a handle may run on several streams at once."""
    T, E, k, d = 500, 128, 8, 256
    h = B.ExpertSort(E, k, renorm=True)
    ls = [torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(i)) for i in range(3)]
    x = torch.randn(T, d, device="cuda")

    def run(l, stream=None):
        idx, w = h.route(l, stream=stream)
        plan = h.plan(idx, stream=stream)
        xs = h.gather(plan, x, stream=stream)
        return idx, w, plan.entries, plan.place, h.combine(plan, xs, w=w, base=x, stream=stream)

    want = [[t.clone() for t in run(l)] for l in ls]
    torch.cuda.synchronize()
    l = ls[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(l)
    for i in (2, 0, 1):
        l.copy_(ls[i])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        got = [run(l, s) for l, s in zip(ls, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o, r in zip(got, want) for a, b in zip(o, r))
    h.close()


def test_refusals(B):
    h = B.ExpertSort(8, 2)
    l = torch.randn(4, 8, device="cuda")
    idx, w = h.route(l)
    plan = h.plan(idx)
    x = torch.randn(4, 16, device="cuda")
    xs = h.gather(plan, x)
    for call in (lambda: h.route(l.half()), lambda: h.route(l[:, :7]), lambda: h.route(l.cpu()), lambda: h.route(l, bias=l[0, :4]),
                 lambda: h.plan(idx.long()), lambda: h.plan(idx[:, :1]), lambda: h.gather(plan, x[:3]), lambda: h.gather(plan, x.double()),
                 lambda: h.gather(plan, x, out=xs[:7]), lambda: h.gather(plan, x[:, :6]), lambda: h.combine(plan, xs, w=w.half()),
                 lambda: h.combine(plan, xs, base=x.half()), lambda: h.combine(plan, xs[:4]), lambda: h.combine(plan, xs, out=xs[:4]),
                 lambda: h.combine_backward(plan, x, xs.half()), lambda: h.combine_backward(plan, x, xs, w=w[:2])):
        with pytest.raises(B.StrataError) as e:
            call()
        assert e.value.status == B.STRATA_EINVAL
    p, q, pl = x.data_ptr(), xs.data_ptr(), plan.place.data_ptr()
    assert B.strata_sort_gather(h.handle, pl, p, 16, p, 16, 0, 4, 16) == B.STRATA_EINVAL
    assert B.strata_sort_gather(h.handle, pl, p, 16, q, 16, 0, 4, 0) == B.STRATA_EINVAL
    assert B.strata_sort_gather(h.handle, None, p, 16, q, 16, 0, 4, 16) == B.STRATA_EINVAL
    assert B.strata_sort_gather(h.handle, pl, p, 16, q, 16, 0, 0, 16) == B.STRATA_OK
    assert B.strata_sort_combine_backward(h.handle, pl, p, 16, q, 16, None, None, 0, None, 0, 4, 16) == B.STRATA_EINVAL
    assert B.strata_sort_combine_backward(h.handle, pl, p, 16, q, 16, None, p, 16, None, 0, 4, 16) == B.STRATA_EINVAL
    o = B.strata_sort_order(None, pl, pl, pl)
    assert B.strata_sort_plan(h.handle, idx.data_ptr(), 4, o) == B.STRATA_EINVAL
    assert B.strata_sort_plan(h.handle, idx.data_ptr(), 1 << 28, B.strata_sort_order(pl, pl, pl, q)) == B.STRATA_EUNSUPPORTED
    assert h.route(l[:0])[0].shape == (0, 2)
    h.close()


def test_a_plan_of_another_number_of_choices_is_refused(B):
    """Its places are fewer (or more) than the call would read."""
    h, other = B.ExpertSort(8, 4), B.ExpertSort(8, 2)
    plan = other.plan(other.route(torch.randn(4, 8, device="cuda"))[0])
    x, z = torch.randn(4, 16, device="cuda"), torch.randn(16, 16, device="cuda")
    for call in (lambda: h.gather(plan, x), lambda: h.combine(plan, z), lambda: h.combine_backward(plan, x, z)):
        with pytest.raises(B.StrataError) as e:
            call()
        assert e.value.status == B.STRATA_EINVAL
    again = B.ExpertSort(16, 2)  # the experts of a plan are in its places alone
    assert torch.equal(again.gather(plan, x), other.gather(plan, x))
    h.close(), other.close(), again.close()


def test_gradient_against_differences_within_the_sums_own_rounding(B):
    """As above, with the bound formed entry by entry: a shifted z and w are rounded once each and a row's k products in f32 take k
    roundings, (k + 2) 2^-24 of |w| |z| each, over 2 t; a product of the gradient's rounds once, a sum of `width` of them in at
    most width / 32 + 16 adds."""
    g = torch.Generator(device="cuda").manual_seed(6)
    T, k, E, width, u = 40, 3, 6, 64, 2.0 ** -24
    h = B.ExpertSort(E, k)
    plan = h.plan(torch.randint(-1, E, (T, k), generator=g, device="cuda").to(torch.int32))
    z, a = (torch.randn(T * k, width, generator=g, device="cuda") for _ in range(2))
    w, b = (torch.randn(T, k, generator=g, device="cuda") for _ in range(2))
    dy = torch.randn(T, width, generator=g, device="cuda")
    dz, dw = h.combine_backward(plan, dy, z, w=w, dz=torch.zeros_like(z))
    live = (plan.place >= 0).view(T, k, 1).double()
    at = plan.place.clamp(min=0).long()
    rows = lambda v: v.double()[at].view(T, k, width) * live
    t, size = 0.125, 0.0
    for s in (1, -1):
        size = size + ((w + s * t * b).double().abs()[..., None] * rows((z + s * t * a).abs())).sum(1)
    bound = (size * (k + 2) * u * dy.double().abs()).sum() / (2 * t)
    bound += (u * rows(dz).abs() * rows(a).abs()).sum()
    bound += ((width / 32 + 16) * u * (dy.double().abs()[:, None] * rows(z).abs()).sum(-1) * b.double().abs()).sum()
    up, down = (h.combine(plan, z + s * t * a, w=w + s * t * b) for s in (1, -1))
    num = ((up.double() - down.double()) * dy.double()).sum() / (2 * t)
    ana = (rows(dz) * rows(a)).sum() + (dw.double() * b.double()).sum()
    assert abs(num - ana) <= bound
    h.close()
