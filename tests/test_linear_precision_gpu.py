"""How exactly the products hold weights and rows, beyond the general bounds of tests/layer_helpers.py: rows that cancel, that meet
one block only, of the largest values, of many columns, and gates far below zero.

Bounds: h = half a step of the result's type; a matrix unit's add may be off by 2^-23 of the larger operand, and only adds of
something other than zero are.  C as in tests/layer_helpers.py: the size of the terms s (q - 8), 8 s and m times x.
"""
import pytest
import torch

from slot_decode_window_gb300 import workloads as wlm
from tests.layer_helpers import DTYPES, check_rows, half_step, i32, linear_bound, parts64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from slot_decode_window_gb300 import binding, build
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()
    return binding


def _qmat(n, rows, cols, seed):
    return wlm.make_qmat(n, rows, cols, 4, 32, [seed * 100 + i for i in range(n)], "cuda")


def _terms(x, q, i=0):
    """(y, C) in 64 bits."""
    s, m, c = (t[i] for t in parts64(q))
    xd = x.double()
    return xd @ (s * c + m).T, xd.abs() @ ((s * (c - 8)).abs() + 8 * s.abs() + m.abs()).T


def _close(got, y, size):
    """size: the bound before the result's own rounding."""
    h = half_step(got.dtype)
    check_rows(got, y, size * (1 + h) + h * y.abs() + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -130))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [8, 33, 70, 300])
def test_rows_that_cancel_meet_the_exact_weights(B, dtype, T):
    """Rows of one 1 and one -1: two weights' difference, where a weight rounded to f16 would show.  At most two instructions with
    products other than zero for each of the two columns, two of their blocks' sums, 4 scalings and sums: 16 2^-23 C."""
    d, out = 512, 208
    g = torch.Generator(device="cuda").manual_seed(T)
    w = _qmat(3, out, d, 40)
    at = torch.randint(0, d - 1, (T, 2), generator=g, device="cuda")
    at[:, 1] += at[:, 1] >= at[:, 0]
    x = torch.zeros(T, d, device="cuda", dtype=DTYPES[dtype])
    x.scatter_(1, at, torch.tensor([1.0, -1.0], device="cuda", dtype=x.dtype).expand(T, 2))
    one = wlm.QMat(w.codes[:1], w.scale[:1], w.min[:1], out, d, 4, 32)
    h, hs = B.Linear(one, max_rows=T), B.Linear(w, max_rows=T)
    y, C = _terms(x, w)
    _close(h.forward(x), y, 16 * 2.0 ** -23 * C)
    off = [0, T // 3, T // 2, T]
    got = hs.forward(x, offsets=i32(off))
    for i in range(3):
        y, C = _terms(x[off[i]:off[i + 1]], w, i)
        _close(got[off[i]:off[i + 1]], y, 16 * 2.0 ** -23 * C)
    hs.sync()
    h.close(), hs.close()


@pytest.mark.parametrize("glu", [False, True])
def test_rounded_weights_are_the_callers_choice(B, glu):
    """With rounded = True many bf16 rows keep to the bound of weights rounded to f16 (one matrix, and a stack's rows); few rows and
    other types have the bits that they have without."""
    d, out, T = 1088, 400, 200
    w, up = _qmat(2, out, d, 55), _qmat(2, out, d, 56) if glu else None
    first = lambda q: wlm.QMat(q.codes[:1], q.scale[:1], q.min[:1], out, d, 4, 32) if q else None
    exact, rounded = (B.Linear(first(w), up=first(up), max_rows=T, rounded=r) for r in (False, True))
    stack = B.Linear(w, up=up, max_rows=T, rounded=True)
    x = torch.randn(T, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    for dtype in DTYPES.values():
        for t in (5, T):
            a, b = exact.forward(x[:t].to(dtype)), rounded.forward(x[:t].to(dtype))
            assert torch.equal(a, b) == (dtype != torch.bfloat16 or t == 5)
    xb = x.bfloat16()
    check_rows(rounded.forward(xb), *linear_bound(xb, w, up, few=False))
    y = stack.forward(xb, offsets=i32([0, 70, T]))
    check_rows(y[:70], *linear_bound(xb[:70], w, up, 0, few=False))
    check_rows(y[70:], *linear_bound(xb[70:], w, up, 1, few=False))
    assert B.strata_linear_round_weights(rounded.handle, 2) == B.STRATA_EINVAL
    assert B.strata_linear_round_weights(rounded.handle, 0) == B.STRATA_OK
    assert torch.equal(rounded.forward(xb), exact.forward(xb))
    for h in (exact, rounded, stack):
        h.sync()
        h.close()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("T", [3, 70])
def test_small_mins_beside_large_scales(B, dtype, T):
    """Mins of 1 / 130 of the scale, codes of zeros, rows of one 1: the result is the min.  Two instructions with products other than
    zero (-8 s; 8 s and m), or two fma of a difference: 4 2^-23 C."""
    d, out = 128, 64
    w = _qmat(1, out, d, 41)
    w.codes.zero_()
    s, m = w.scale.view(torch.float16), w.min.view(torch.float16)
    s.fill_(0.0133)
    m.copy_(1.003e-4 * (1 + torch.rand(m.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))))
    x = torch.zeros(T, d, device="cuda", dtype=DTYPES[dtype])
    x[torch.arange(T), torch.arange(T) * 37 % d] = 1
    h = B.Linear(w, max_rows=T)
    y, C = _terms(x, w)
    _close(h.forward(x), y, 4 * 2.0 ** -23 * C)
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [7, 70])
def test_rows_that_meet_only_a_block_of_small_scale(B, dtype, T):
    """A block's scale is 2^-16 to 2^-22 of its row's largest; rows of x have values in one such block only.  Its columns are two
    instructions of two parts each, six for f32 rows, and one of the sums, with 6 scalings and sums: 16 2^-23 C; a sum of x in two
    parts 2^-21, f32 rows' x in two parts 2^-21: 2^-20 C."""
    d, out = 256, 96
    w = _qmat(1, out, d, 42)
    s, m = w.scale.view(torch.float16), w.min.view(torch.float16)
    g = torch.Generator(device="cuda").manual_seed(4)
    s.copy_((1 + torch.rand(s.shape, generator=g, device="cuda")) * 2.0 ** 10)
    s[..., 1:] *= 2.0 ** -torch.arange(16, 23, device="cuda").half()
    m.copy_(-7.5 * s.float())
    x = torch.randn(T, 8, 32, generator=g, device="cuda")
    x = (x * torch.nn.functional.one_hot(torch.arange(T, device="cuda") % 7 + 1, 8)[..., None]).flatten(1).to(DTYPES[dtype])
    h = B.Linear(w, max_rows=T)
    y, C = _terms(x, w)
    _close(h.forward(x), y, (16 * 2.0 ** -23 + 2.0 ** -20) * C)
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 9, 16, 64])
def test_rows_of_the_few_row_kernel_over_the_range_that_the_header_gives(B, dtype, T):
    """Values from 2^-100 to 2^100, rows of zeros, weights of 2^-9 of the usual; rows of 2^100 that meet weights of zeros beside a
    block of scale 2^15; infinities and NaN stay in their rows."""
    d, out = 128, 32
    w = _qmat(1, out, d, 43)
    s, m = w.scale.view(torch.float16), w.min.view(torch.float16)
    s[0, :, 1], m[0, :, 1] = 2.0 ** 15, 0
    s[0, :, 0], m[0, :, 0] = 0, 0
    x = torch.zeros(T, d, device="cuda", dtype=DTYPES[dtype])
    x[:, :32] = 2.0 ** 100
    h = B.Linear(w, max_rows=T)
    assert (h.forward(x) == 0).all()
    h.close()
    w = _qmat(1, out, d, 44)
    w.scale.view(torch.float16)[0, :16] *= 2.0 ** -9
    w.min.view(torch.float16)[0, :16] *= 2.0 ** -9
    g = torch.Generator(device="cuda").manual_seed(T)
    scale = torch.tensor([2.0 ** -100, 2.0 ** 99, 1.0, 0.0, 2.0 ** -20], device="cuda").repeat(T)[:T, None]
    x = (1 + torch.rand(T, d, generator=g, device="cuda")) * torch.where(torch.rand(T, d, generator=g, device="cuda") < 0.5, -1, 1)
    x = (x * scale).to(DTYPES[dtype])
    h = B.Linear(w, max_rows=T)
    y = h.forward(x)
    check_rows(y, *linear_bound(x, w, None, few=True))
    assert (y[3] == 0).all()
    bad = x.clone()
    bad[2, 5], bad[4, 7] = float("nan"), float("inf")
    z = h.forward(bad)
    keep = [t for t in range(T) if t not in (2, 4)]
    assert torch.equal(z[keep], y[keep]) and not torch.isfinite(z[[2, 4]]).any()
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [4, 70])
def test_gates_far_below_zero(B, dtype, T):
    """silu(z) for z from -80 to -97, where e^-z leaves f32 or its quotient does, times 2^10: e^z is down to 2^-140, 9 bits of a
    subnormal, so the result is within 2^-9 and its own rounding."""
    d, out = 64, 32
    w, up = _qmat(1, out, d, 45), _qmat(1, out, d, 46)
    z = -torch.linspace(80, 97, out, device="cuda").half()
    for q, v in ((w, z), (up, torch.full_like(z, 1024.0))):
        q.scale.zero_(), q.min.zero_()
        q.min.view(torch.float16)[0, :, 0] = v
    x = torch.zeros(T, d, device="cuda", dtype=DTYPES[dtype])
    x[torch.arange(T), torch.arange(T) % 32] = 1
    h = B.Linear(w, up=up, max_rows=T)
    y = h.forward(x)
    zd = z.double()
    want = (zd * torch.exp(zd) / (1 + torch.exp(zd)) * 1024).expand(T, out)
    check_rows(y, want, (2.0 ** -9 + half_step(x.dtype)) * want.abs())
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [4, 70])
def test_the_largest_gates(B, dtype, T):
    """silu is z or 0 at the far ends, and not a number of neither."""
    d, out = 64, 16
    w, up = _qmat(1, out, d, 47), _qmat(1, out, d, 48)
    z = torch.tensor([-6e4, -1e3, -200, -104, 89, 200, 1e3, 6e4] * 2, device="cuda").half()
    for q, v in ((w, z), (up, torch.full_like(z, 1.0))):
        q.scale.zero_(), q.min.zero_()
        q.min.view(torch.float16)[0, :, 0] = v
    x = torch.zeros(T, d, device="cuda", dtype=DTYPES[dtype])
    x[:, 3] = 1
    h = B.Linear(w, up=up, max_rows=T)
    want = z.clamp(min=0).to(x.dtype).expand(T, out)
    y = h.forward(x)
    assert torch.isfinite(y).all() and ((y - want).abs() <= 2 * half_step(x.dtype) * want + 2.0 ** -100).all()
    h.close()


@pytest.mark.parametrize("dtype,d", [("f16", 65536), ("f16", 29184), ("f16", 29120), ("bf16", 65536)])
@pytest.mark.parametrize("glu", [False, True])
def test_long_sums_of_one_sign(B, dtype, d, glu):
    """All products positive, so that adds that truncate drift one way, in tiles enough that no cluster shares their columns.  f16
    rows of more than 29120 columns are added up in f32 registers every two steps of 64 columns: 32 2^-23 within them and one
    rounding each, d / 128 2^-24 in all.  Others take at most 9 adds a step: 9 d / 64 2^-23.  A pair in 16 bits: 2^-18 of its silu."""
    T, out = 1283, 2048 if glu else 4096
    g = torch.Generator(device="cuda").manual_seed(d)

    def mat():  # codes of 8 and more, mins as the scales: C is y
        codes = (torch.randint(0, 256, (1, out, d // 2), generator=g, device="cuda", dtype=torch.int32) | 0x88).to(torch.uint8)
        s = (1.0 / d * (1 + torch.rand(1, out, d // 32, generator=g, device="cuda"))).half()
        return wlm.QMat(codes, s.view(torch.int16), s.clone().view(torch.int16), out, d, 4, 32)

    w, up = mat(), mat() if glu else None
    x = (0.5 + 0.5 * torch.rand(T, d, generator=g, device="cuda")).to(DTYPES[dtype])
    h = B.Linear(w, up=up, max_rows=T)
    got = h.forward(x)[::20, ::64]
    some = lambda q: wlm.QMat(q.codes[:, ::64], q.scale[:, ::64], q.min[:, ::64], q.codes[:, ::64].shape[1], d, 4, 32)
    y, C = _terms(x[::20], some(w))
    rel = 32 * 2.0 ** -23 + d / 128 * 2.0 ** -24 if dtype == "f16" and d > 29120 else 9 * d / 64 * 2.0 ** -23
    size = rel * C
    if glu:
        v, Cv = _terms(x[::20], some(up))
        sg = y * torch.sigmoid(y)
        y, size = sg * v, 1.1 * size * (v + rel * Cv) + sg * rel * Cv + 2.0 ** -18 * sg * v
    _close(got, y, size)
    h.sync()
    h.close()


def test_long_f16_rows_of_stacks_and_clusters(B):
    """f16 rows of more than 29120 columns with offsets, and few tiles (clusters share their columns)."""
    d, out = 29184, 48
    w, up = _qmat(2, out, d, 57), _qmat(2, out, d, 58)
    one = wlm.QMat(w.codes[:1], w.scale[:1], w.min[:1], out, d, 4, 32)
    x = torch.randn(150, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).half()
    h, hs = B.Linear(one, max_rows=150), B.Linear(w, up=up, max_rows=150)
    check_rows(h.forward(x), *linear_bound(x, w, None, few=False))
    y = torch.full((150, out), 7.0, dtype=x.dtype, device="cuda")
    hs.forward(x, y=y, offsets=i32([3, 70, 149]))
    for i, (a, b) in enumerate(((3, 70), (70, 149))):
        check_rows(y[a:b], *linear_bound(x[a:b], w, up, i, few=False))
    assert (y[:3] == 7).all() and (y[149:] == 7).all()
    hs.sync()
    h.close(), hs.close()
