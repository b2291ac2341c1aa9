"""Products with 4-bit matrices on the GPU against a plain product in 64 bits, within the bounds of tests/layer_helpers.py."""
import numpy as np
import pytest
import torch

from slot_decode_window_gb300 import workloads as wlm
from tests.layer_helpers import DTYPES, check_rows, i32, linear_bound

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


def _rows(T, d, dtype, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, d + pad, generator=g, device="cuda") * torch.exp2(torch.randn(T, 1, generator=g, device="cuda"))
    return x.to(DTYPES[dtype])[:, :d]


@pytest.mark.parametrize("d,out", [(64, 16), (64, 272), (192, 400), (1088, 144), (2048, 256)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("glu", [False, True])
def test_one_matrix_any_number_of_rows(B, d, out, dtype, glu):
    """Both paths and the border between them, tiles of x that end anywhere, clusters of every size (few tiles), padded rows
    of x and y; what is beside y's rows stays."""
    w, up = _qmat(1, out, d, 1), _qmat(1, out, d, 2) if glu else None
    h = B.Linear(w, up=up, max_rows=700)
    for T in (1, 2, 7, 8, 9, 31, 33, 64, 65, 129, 193, 200, 385, 700):
        x = _rows(T, d, dtype, T, pad=16)
        whole = torch.full((T + 2, out + 16), 7.0, dtype=x.dtype, device="cuda")
        y = whole[1:T + 1, :out]
        assert h.forward(x, y=y) is y
        want, bound = linear_bound(x, w, up, few=True if T <= 8 else None)
        check_rows(y, want, bound)
        assert (whole[0] == 7).all() and (whole[-1] == 7).all() and (whole[:, out:] == 7).all()
    h.sync()
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_many_tiles_and_long_columns(B, dtype):
    """More tiles than SMs (every CTA takes several), and up to 65536 columns (rows of x that do not fit a CTA's registers)."""
    for T, d, out, glu in ((2003, 128, 5136, False), (1500, 256, 2576, True), (40, 12288, 160, False), (6, 12288, 160, False),
                           (11, 65536, 16, False), (3, 65536, 16, False), (70, 20544, 48, True)):
        w, up = _qmat(1, out, d, 3), _qmat(1, out, d, 4) if glu else None
        h = B.Linear(w, up=up, max_rows=T)
        x = _rows(T, d, dtype, 5)
        y = h.forward(x)
        h.sync()
        check_rows(y, *linear_bound(x, w, up, few=True if T <= 8 else None))
        h.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("glu", [False, True])
def test_few_rows_of_large_matrices(B, dtype, glu):
    """Each number of tiles and warps that the few-row kernel chooses; the last CTA's tiles end early."""
    for d, out in ((128, 5024), (192, 39056)):
        w, up = _qmat(1, out, d, 6), _qmat(1, out, d, 7) if glu else None
        h = B.Linear(w, up=up, max_rows=8)
        for T in (1, 5, 8):
            x = _rows(T, d, dtype, T)
            check_rows(h.forward(x), *linear_bound(x, w, up, few=True))
        h.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("d,out", [(512, 4880), (5184, 4864), (4096, 4096), (16384, 1024)])
def test_nine_to_sixty_four_rows_of_matrices_of_middling_size(B, d, out, dtype, glu):
    """Both sides of the rule that gives small matrices' rows to the few-row kernel; narrow tiles of x whose columns a cluster
    shares."""
    w, up = _qmat(1, out, d, 26), _qmat(1, out, d, 27) if glu else None
    h = B.Linear(w, up=up, max_rows=64)
    for T in (9, 16, 17, 24, 33, 40, 57, 64):
        x = _rows(T, d, dtype, T)
        y = h.forward(x)
        check_rows(y, *linear_bound(x, w, up, few=None))
        assert torch.equal(y, h.forward(x))
    h.sync()
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("glu", [False, True])
def test_rows_sorted_by_matrix(B, dtype, glu):
    """Matrices with no rows, one row and many; rows before the first and behind the last stay as they were."""
    w, up = _qmat(6, 208, 320, 8), _qmat(6, 208, 320, 9) if glu else None
    h = B.Linear(w, up=up, max_rows=600)
    for off in ([3, 3, 4, 41, 41, 450, 590], [0, 0, 0, 0, 0, 0, 1], [0, 5, 5, 5, 5, 5, 5], [0, 100, 200, 300, 400, 500, 600],
                [7, 7, 7, 7, 7, 7, 7]):
        T = 600 if off[-1] > 50 else 9
        x = _rows(T, 320, dtype, 10)
        y = torch.full((T, 208), 7.0, dtype=x.dtype, device="cuda")
        h.forward(x, y=y, offsets=i32(off))
        for i in range(6):
            if off[i] < off[i + 1]:
                check_rows(y[off[i]:off[i + 1]], *linear_bound(x[off[i]:off[i + 1]], w, up, i))
        assert (y[:off[0]] == 7).all() and (y[off[-1]:] == 7).all()
    h.sync()
    h.close()


@pytest.mark.parametrize("T", [8, 100])
def test_offsets_of_one_matrix(B, T):
    w = _qmat(1, 64, 128, 11)
    h = B.Linear(w, max_rows=100)
    x = _rows(T, 128, "bf16", 12)
    y = torch.full((T, 64), 7.0, dtype=x.dtype, device="cuda")
    h.forward(x, y=y, offsets=i32([2, T - 3]))
    check_rows(y[2:T - 3], *linear_bound(x[2:T - 3], w, None, few=T <= 8))
    assert (y[:2] == 7).all() and (y[T - 3:] == 7).all()
    h.close()


def test_ranges_out_of_order_or_outside_are_left_out(B):
    w = _qmat(4, 64, 128, 13)
    h = B.Linear(w, max_rows=64)
    x = _rows(50, 128, "bf16", 14)
    for off, good in (([0, 20, 10, 30, 50], (0, 2, 3)), ([-1, 10, 20, 30, 51], (1, 2)), ([0, 10, 20, 2 ** 31 - 1, 50], (0, 1))):
        y = torch.full((50, 64), 7.0, dtype=x.dtype, device="cuda")
        h.forward(x, y=y, offsets=i32(off))
        with pytest.raises(B.StrataError) as e:
            h.sync()
        assert e.value.status == B.STRATA_EDEVICE
        h.sync()  # reported once
        named = torch.zeros(50, device="cuda")
        for i in good:
            named[off[i]:off[i + 1]] += 1
        for i in good:  # rows that two of them name have no defined output
            rows = torch.nonzero(named[off[i]:off[i + 1]] == 1).flatten() + off[i]
            check_rows(y[rows], *linear_bound(x[rows], w, None, i))
        assert (y[named == 0] == 7).all()
    one = B.Linear(_qmat(1, 64, 128, 13), max_rows=8)
    one.forward(_rows(4, 128, "f32", 1), offsets=i32([0, 5]))
    with pytest.raises(B.StrataError):
        one.sync()
    one.close()
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 70])
def test_rows_and_weights_of_any_size(B, dtype, T):
    """Rows from 1e-30 to 1e30, rows of zeros; matrices with weights of 1e-5, of 3e4, of zeros, blocks of one value far from
    zero, negative scales."""
    d, out = 256, 96
    w = _qmat(1, out, d, 15)
    s, m = w.scale.view(torch.float16), w.min.view(torch.float16)
    s[0, :16] *= 2.0 ** -9
    m[0, :16] *= 2.0 ** -9
    s[0, 16:32] *= 2.0 ** 15
    m[0, 16:32] *= 2.0 ** 15
    s[0, 32:40], m[0, 32:40] = 0, 0
    s[0, 40:48] = 0
    m[0, 48:56, ::3] = 100.0
    s[0, 56:64] *= -1
    x = _rows(T, d, dtype, 16)
    scale = torch.tensor([1e-30, 1e30, 1.0, 0.0, 1e-6], device="cuda").repeat(T)[:T, None]
    x = (x.float() * scale).to(x.dtype)
    h = B.Linear(w, max_rows=100)
    y = h.forward(x)
    check_rows(y, *linear_bound(x, w, None, few=True if T <= 8 else None))
    assert (y[3] == 0).all()
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_rows_with_weights_of_the_largest_scale(B, dtype):
    """A row's and a weight row's powers of two together pass f32's range, their product with a result does not: x of 2^126 meets
    weights of zeros, beside a block of scale 2^15 that meets zeros."""
    d, out, T = 128, 32, 70
    w = _qmat(1, out, d, 28)
    s, m = w.scale.view(torch.float16), w.min.view(torch.float16)
    s[0, :, 1], m[0, :, 1] = 2.0 ** 15, 0
    s[0, :, 0], m[0, :, 0] = 0, 0
    x = torch.zeros(T, d, device="cuda", dtype=DTYPES[dtype])
    x[:, :32] = 2.0 ** 126
    h = B.Linear(w, max_rows=T)
    assert (h.forward(x) == 0).all()
    h.sync()
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [8, 70])
def test_a_row_without_meaning_stays_alone(B, dtype, T):
    w, up = _qmat(1, 160, 192, 17), _qmat(1, 160, 192, 18)
    h = B.Linear(w, up=up, max_rows=100)
    x = _rows(T, 192, dtype, 19).contiguous()
    ref = h.forward(x).clone()
    bad = x.clone()
    bad[3, 5], bad[6, 7] = float("nan"), float("inf")
    y = h.forward(bad)
    keep = [t for t in range(T) if t not in (3, 6)]
    assert torch.equal(y[keep], ref[keep]) and not torch.isfinite(y[3]).any()
    h.sync()
    h.close()


def test_a_row_alone_has_the_bits_of_a_window(B):
    for dtype in DTYPES:
        w = _qmat(1, 176, 640, 20)
        h = B.Linear(w, max_rows=8)
        x = _rows(8, 640, dtype, 21)
        y = h.forward(x)
        for t in range(8):
            assert torch.equal(h.forward(x[t:t + 1])[0], y[t])
        assert torch.equal(h.forward(x.flip(0)).flip(0), y)
        h.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_calls_other_streams_and_the_same_bits(B, dtype):
    """Captured calls of one handle replay with new contents, on another stream, and give an eager call's bits; two handles run at
    the same time."""
    w = _qmat(3, 272, 512, 22)
    h, h2 = B.Linear(w, max_rows=500), B.Linear(w, max_rows=500)
    one = B.Linear(_qmat(1, 272, 512, 23), max_rows=40)
    xs = [_rows(500, 512, dtype, 24 + i).contiguous() for i in range(3)]
    offs = [i32(o) for o in ([0, 100, 300, 500], [0, 0, 490, 495], [5, 250, 251, 400])]
    want = []
    for x, o in zip(xs, offs):
        y = torch.zeros(500, 272, dtype=x.dtype, device="cuda")
        want.append((h.forward(x, y=y, offsets=o).clone(), one.forward(x[:33]).clone(), one.forward(x[:4]).clone()))
    x, o = xs[0].clone(), offs[0].clone()
    y, y33, y4 = torch.zeros_like(want[0][0]), torch.empty_like(want[0][1]), torch.empty_like(want[0][2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        h.forward(x, y=y, offsets=o)
        one.forward(x[:33], y=y33)
        one.forward(x[:4], y=y4)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        o.copy_(offs[i])
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip((y, y33, y4), want[i]):
            assert torch.equal(got, ref)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        ya = torch.zeros_like(y)
        yb = torch.zeros_like(y)
        torch.cuda.synchronize()
        h.forward(xs[0], y=ya, offsets=offs[0], stream=a)
        h2.forward(xs[2], y=yb, offsets=offs[2], stream=b)
        torch.cuda.synchronize()
        assert torch.equal(ya, want[0][0]) and torch.equal(yb, want[2][0])
    for l in (h, h2, one):
        l.sync()
        l.close()


def test_workspace_and_weights_are_counted(B):
    h = B.Linear(_qmat(2, 96, 128, 30), max_rows=1000)
    a, b = h.bytes()
    assert a == 2 * 96 * 128 * 5 // 8 and b >= 1000 * 128 * 4
    few = B.Linear(_qmat(1, 96, 128, 30), max_rows=8)
    assert few.bytes() == (96 * 128 * 5 // 8, 0)
    few.close()
    h.close()


def test_refusals(B):
    w = _qmat(2, 64, 128, 31)
    h = B.Linear(w, max_rows=16)
    x = _rows(16, 128, "bf16", 32).contiguous()
    off = i32([0, 8, 16])
    y = h.forward(x, offsets=off)
    big = torch.zeros(17, 128, dtype=x.dtype, device="cuda")
    for call in (lambda: h.forward(x), lambda: h.forward(big, offsets=off), lambda: h.forward(x[:, :64], offsets=off),
                 lambda: h.forward(x.double(), offsets=off), lambda: h.forward(x, y=y.float(), offsets=off),
                 lambda: h.forward(x, offsets=off.long()), lambda: h.forward(x, offsets=off[:2]),
                 lambda: h.forward(x.T.contiguous().T, offsets=off), lambda: h.forward(x.cpu(), offsets=off),
                 lambda: h.forward(x, y=y[:15], offsets=off), lambda: B.Linear(w, up=_qmat(2, 80, 128, 1)),
                 lambda: B.Linear(_qmat(1, 64, 128, 1), up=w), lambda: B.Linear(w, max_rows=0)):
        with pytest.raises(B.StrataError) as e:
            call()
        assert e.value.status == B.STRATA_EINVAL
    p, q = x.data_ptr(), y.data_ptr()
    f = B.strata_linear_forward
    for args in ((p, 128, p, 128, 2, 4), (p + 2, 128, q, 64, 2, 4), (p, 127, q, 64, 2, 4), (p, 132, q, 64, 2, 4), (p, 128, q, 60, 2, 4),
                 (p, 128, q, 64, 3, 4), (p, 128, q, 64, 2, -1), (None, 128, q, 64, 2, 4), (p, 128, None, 64, 2, 4)):
        assert f(h.handle, *args, off.data_ptr()) == B.STRATA_EINVAL
    assert f(h.handle, p, 128, q, 64, 2, 4, off.data_ptr() + 2) == B.STRATA_EINVAL
    assert f(h.handle, p, 128, q, 64, 2, 0, off.data_ptr()) == B.STRATA_OK
    assert h.forward(x[:0], offsets=off).shape == (0, 64)
    h.sync()
    h.close()


@pytest.mark.parametrize("dtype,rounded", [("f32", False), ("f16", False), ("f16", True), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("d,out", [(2048, 512), (4096, 2048), (4096, 4096), (1024, 4864), (1024, 4880)])
def test_which_kernel_takes_nine_to_sixty_four_rows(B, d, out, dtype, rounded, glu):
    """The rule that the header gives: the few-row kernel's rows have the bits that they have in calls of 8, the others keep to the
    many-row kernel's own bound (and f32 rows, of 22 bits there, do not have those bits)."""
    w, up = _qmat(1, out, d, 51), _qmat(1, out, d, 52) if glu else None
    h = B.Linear(w, up=up, max_rows=64, rounded=rounded)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    most = {"f32": 130, "f16": 440, "bf16": 320 if rounded else 440}[dtype]
    for T in (9, 16, 17, 24, 33, 48, 64):
        x = _rows(T, d, dtype, T)
        y = h.forward(x)
        few = out <= 32 * sms and (2 if glu else 1) * (out // 16) * (-(-T // 8)) * (d // 64) <= most * sms
        eights = torch.cat([h.forward(x[t:t + 8]) for t in range(0, T, 8)])
        assert not few or torch.equal(y, eights)
        if not few:
            check_rows(y, *linear_bound(x, w, up, few=False))
            assert dtype != "f32" or not torch.equal(y, eights)
    h.close()


@pytest.mark.parametrize("d,out", [(64, 272), (192, 400), (2048, 256)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("glu", [False, True])
def test_many_rows_keep_to_their_own_bound(B, d, out, dtype, glu):
    w, up = _qmat(1, out, d, 53), _qmat(1, out, d, 54) if glu else None
    h = B.Linear(w, up=up, max_rows=700)
    for T in (65, 129, 193, 200, 385, 700):
        x = _rows(T, d, dtype, T)
        check_rows(h.forward(x), *linear_bound(x, w, up, few=False))
    h.close()
