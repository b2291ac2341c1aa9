"""The norms of query and key heads with the rotation by position on the GPU
against the fp64 oracle.

Bound: with u = 2^-24, the mean of squares of at most 256 values is off by less
than 16 u (8 sums of a lane, 5 of the warp, products and the division), the
root, the quotient, the two factors and the gain by under 8 u more; a cosine or
sine by under 8 u (the angle's rounding to 24 bits of half a turn, pi u, and
the function's 2 u); the pair's sum by 2 u.  A turned value of a pair of length
r is within 40 u r, and its rounding adds half a step of the type."""
import numpy as np
import pytest
import torch

from oracle import kv8 as ok
from tests.kv8_helpers import DTYPES, half_step, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from slot_decode_window_gb300 import binding, build
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()
    return binding


def _check(got, x, position, freqs, gain, interleaved, norm, eps):
    hd, half = x.shape[-1], len(freqs)
    want = ok.qknorm(x.double().cpu().numpy(), position, freqs, gain, eps, norm, interleaved)
    r = np.abs(want).copy()  # the length of each dim's pair
    one = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    two = one + 1 if interleaved else one + half
    r[..., one] = r[..., two] = np.hypot(want[..., one], want[..., two])
    bound = 40 * 2.0 ** -24 * r * (1 + half_step(x.dtype)) + half_step(x.dtype) * np.abs(want) + 2.0 ** -25
    if x.dtype != torch.float16:
        bound -= 2.0 ** -25 - 2.0 ** -130
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound).all(), (err / bound).max()
    assert hd == got.shape[-1]


@pytest.mark.parametrize("heads,kvh,hd,rd", [(32, 4, 128, 128), (3, 1, 64, 32), (5, 5, 128, 64), (2, 0, 64, 64),
                                             (7, 2, 256, 96), (4, 2, 128, 0), (1, 1, 64, 4)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [1, 7, 60])
def test_against_the_oracle(B, heads, kvh, hd, rd, dtype, interleaved, T):
    g = torch.Generator(device="cuda").manual_seed(T)
    fused = torch.randn(T, heads + 2 * kvh + 1, hd, generator=g, device="cuda").to(DTYPES[dtype])
    q, k = fused[:, :heads], fused[:, heads:heads + kvh]
    gains = [1 + 0.3 * torch.randn(hd, generator=g, device="cuda") for _ in range(2)]
    freqs = [5e5 ** (-2.0 * i / max(rd, 1)) for i in range(rd // 2)]
    position = np.concatenate([[0], np.random.default_rng(T).integers(-5, 2 ** 21, T)])[:T]
    for norm, gain in ((True, gains), (True, (None, None)), (False, (None, None))):
        qk = B.QkNorm(heads, kvh, hd, rotary_dim=rd, freqs=freqs, interleaved=interleaved, norm=norm, eps=1e-5,
                      q_gain=gain[0], k_gain=gain[1])
        qo, ko = qk.forward(q, k if kvh else None, i32(list(position)))
        torch.cuda.synchronize()
        for got, x, w in ((qo, q, gain[0]), (ko, k, gain[1])):
            if x.shape[1]:
                _check(got, x, position, freqs, w.cpu().numpy() if w is not None else None, interleaved, norm, 1e-5)
        qk.close()


def test_far_positions_lose_nothing(B):
    """Positions up to the ends of int32, a frequency of one radian per position."""
    qk = B.QkNorm(1, 0, 64, freqs=[1.0, -0.37] + [1e-4] * 30, norm=False)
    pos = [2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 123456789]
    q = torch.randn(4, 1, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    qo, _ = qk.forward(q, None, i32(pos))
    torch.cuda.synchronize()
    _check(qo, q, pos, [1.0, -0.37] + [1e-4] * 30, None, False, False, 0.0)


def test_in_place_other_stream_and_rows_do_not_matter(B):
    """In place, on another stream, in a captured graph and in a batch of any size: the same bits."""
    qk = B.QkNorm(8, 2, 128, theta=1e4)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k = torch.randn(700, 8, 128, generator=g, device="cuda"), torch.randn(700, 2, 128, generator=g, device="cuda")
    pos = torch.arange(700, dtype=torch.int32, device="cuda")
    a, b = qk.forward(q, k, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, d = qk.forward(q, k, pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    e, f = qk.forward(q[300:301], k[300:301], pos[300:301])
    q1, k1 = q.clone(), k.clone()
    qk.forward(q1, k1, pos, q_out=q1, k_out=k1)
    q2, k2 = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qk.forward(q, k, pos, q_out=q2, k_out=k2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, c) and torch.equal(b, d) and torch.equal(a, q1) and torch.equal(b, k1)
    assert torch.equal(a, q2) and torch.equal(b, k2)
    assert torch.equal(a[300:301], e) and torch.equal(b[300:301], f)


def test_a_row_that_is_not_finite_and_a_zero_row(B):
    qk = B.QkNorm(2, 1, 64)
    q, k = torch.randn(4, 2, 64, device="cuda"), torch.randn(4, 1, 64, device="cuda")
    pos = i32([1, 2, 3, 4])
    good = qk.forward(q, k, pos)[0]
    q2 = q.clone()
    q2[1, 0, 3], q2[2, 1] = float("nan"), 0.0
    bad = qk.forward(q2, k, pos)[0]
    torch.cuda.synchronize()
    assert torch.isnan(bad[1, 0]).all() and (bad[2, 1] == 0).all()
    for r, h in ((0, 0), (0, 1), (1, 1), (2, 0), (3, 0), (3, 1)):
        assert torch.equal(good[r, h], bad[r, h])


def test_refusals(B):
    qk = B.QkNorm(2, 1, 64)
    q, k, pos = torch.zeros(3, 2, 64, device="cuda"), torch.zeros(3, 1, 64, device="cuda"), i32([0, 1, 2])
    for bad in ((q.double(), k.double(), pos), (q[:, :1], k, pos), (q, k.half(), pos), (q, k[:2], pos),
                (q, k, pos[:2]), (q, k, pos.long()), (q.cpu(), k, pos), (q.transpose(0, 1), k, pos)):
        with pytest.raises(B.StrataError):
            qk.forward(*bad)
    p, s = q.data_ptr(), 128
    kp = k.data_ptr()
    for a in ((None, p, s, kp, 64, p, s, kp, 64, 0, pos.data_ptr(), 3), (qk.handle, p + 4, s, kp, 64, p, s, kp, 64, 0, pos.data_ptr(), 3),
              (qk.handle, p, 127, kp, 64, p, s, kp, 64, 0, pos.data_ptr(), 3), (qk.handle, p, s, 0, 64, p, s, kp, 64, 0, pos.data_ptr(), 3),
              (qk.handle, p, s, kp, 64, p, 130, kp, 64, 0, 0, 3), (qk.handle, p, s, kp, 64, p, s, kp, 64, 3, pos.data_ptr(), 3),
              (qk.handle, p, s, kp, 64, p, s, kp, 64, 0, pos.data_ptr(), -1)):
        assert B.strata_qknorm_forward(*a) == B.STRATA_EINVAL
    assert B.strata_qknorm_forward(qk.handle, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) == B.STRATA_OK  # no rows
    empty = qk.forward(q[:0], k[:0], pos[:0])
    assert empty[0].shape == (0, 2, 64)


def test_refuses_overlaps_and_other_devices(B):
    qk = B.QkNorm(2, 2, 64)
    wide = torch.zeros(3, 4, 64, device="cuda")
    q, k, pos = torch.ones(3, 2, 64, device="cuda"), torch.ones(3, 2, 64, device="cuda"), i32([0, 1, 2])
    for kw in (dict(q_out=k), dict(k_out=q), dict(q_out=wide[:, :2], k_out=wide[:, :2])):
        with pytest.raises(B.StrataError):
            qk.forward(q, k, pos, **kw)
    flat = torch.ones(3 * 256, device="cuda")
    tight, spread = flat[:384].view(3, 2, 64), flat.view(3, 4, 64)[:, :2]  # one start, two strides
    for a, b in ((tight, spread), (spread, tight)):
        with pytest.raises(B.StrataError):
            qk.forward(a, k, pos, q_out=b)
        with pytest.raises(B.StrataError):
            qk.forward(q, a, pos, k_out=b)
    with pytest.raises(B.StrataError):
        qk.forward(q, None, pos)
    torch.cuda.synchronize()
    assert (q == 1).all() and (k == 1).all() and (flat == 1).all() and (wide == 0).all()
    one = qk.forward(tight[:1], k[:1], pos[:1], q_out=spread[:1])[0]  # one row has no stride
    both = qk.forward(q, k, pos, q_out=wide[:, :2], k_out=wide[:, 2:])  # halves of one buffer do not overlap
    want = qk.forward(q, k, pos)
    assert torch.equal(one, want[0][:1]) and all(torch.equal(a, b) for a, b in zip(both, want))
    qk.device += 1  # a handle of another device
    with pytest.raises(B.StrataError):
        qk.forward(q, k, pos)
