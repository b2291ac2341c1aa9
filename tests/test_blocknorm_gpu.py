"""Norms after and before a block with the gate and the residual on the GPU against the oracle.

Bound, with u = 2^-24: a mean of d squares in at most 1024 partial sums is off by under (d / 1024 + 20) u, the root, quotient and
the factors by under 12 u more: e = (d / 2048 + 24) u relative on a normed value.  h is off by e on its block's part, 4 u on both
and (with a sigmoid) 8 u; n by that relative to the row's root mean square through h, and e again."""
import numpy as np
import pytest
import torch

from oracle import layer as ol
from tests.layer_helpers import DTYPES, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from slot_decode_window_gb300 import binding, build
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()
    return binding


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _check(got, x, y, after, before, gate, sigmoid, a, b, eps):
    h, n = ol.block_norm(_np(x), _np(y), _np(after), _np(before), _np(gate), sigmoid, eps, a, b)
    d, u = x.shape[1], 2.0 ** -24
    e = (d / 2048 + 24) * u
    part = np.abs(h - a * _np(x)) if y is not None else 0.0
    eh = 4 * u * np.abs(a * _np(x)) + (e + 12 * u) * part
    half, tiny = half_step(x.dtype), 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -130
    if got[0] is not None:
        assert (np.abs(_np(got[0]) - h) <= eh * (1 + half) + half * np.abs(h) + tiny).all()
    assert (got[1] is None) == (before is None)
    if before is not None:
        r = np.sqrt(np.square(h).mean(-1, keepdims=True) + eps)
        en = (eh / r + np.abs(h) / r * (np.square(eh).mean(-1, keepdims=True) ** 0.5 / r + e)) * np.abs(_np(before))
        assert (np.abs(_np(got[1]) - n) <= en * (1 + half) + half * np.abs(n) + tiny).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [8, 24, 512, 1000, 2048, 4104, 8192, 16384])
def test_against_the_oracle(B, dtype, d):
    """Every kernel variant (rows of 1 to 4096 pieces), every gate, both norms or none, padded rows."""
    g = torch.Generator(device="cuda").manual_seed(d)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    T = 5
    x, y, ge = ((rand(T, d + 16) * torch.exp2(2 * rand(T, 1))).to(DTYPES[dtype])[:, :d] for _ in range(3))
    x[2] = 0
    y[3] = 0
    for after, before, gate, sigmoid in ((True, True, "none", False), (False, True, "channel", True), (True, False, "row", False),
                                         (False, True, "element", True), (True, True, "element", False), (False, False, "row", True),
                                         (True, True, "channel", False)):
        ga, gb, gc = 1 + 0.3 * rand(d), 1 + 0.3 * rand(d), rand(d)
        gr = rand(T)
        h = B.BlockNorm(d, after=ga if after else None, before=gb if before else None, gate=gate,
                        channel_gate=gc if gate == "channel" else None, sigmoid=sigmoid, eps=1e-5, residual_scale=0.8,
                        block_scale=-1.5)
        got = h.forward(x, y, gate={"row": gr, "element": ge}.get(gate))
        _check(got, x, y, ga if after else None, gb if before else None,
               {"none": None, "channel": gc, "row": gr[:, None], "element": ge}[gate], sigmoid, 0.8, -1.5, 1e-5)
        h.close()


def test_gains_of_ones_first_norm_and_last_sum(B):
    x, y = torch.randn(3, 256, device="cuda"), torch.randn(3, 256, device="cuda")
    one = torch.ones(256, device="cuda")
    first = B.BlockNorm(256, before=True)
    h, n = first.forward(x, keep=False)
    assert h is None
    _check((None, n), x, None, None, one, None, False, 1.0, 1.0, 1e-6)
    last = B.BlockNorm(256, after=True)
    got = last.forward(x, y)
    _check(got, x, y, one, None, None, False, 1.0, 1.0, 1e-6)


def test_in_place_other_stream_graph_and_rows_do_not_matter(B):
    """h over x, n over y (or the other way round), on another stream, captured, alone or in a batch: the same bits."""
    d, T = 2048, 64
    for dt in DTYPES.values():
        g = torch.Generator(device="cuda").manual_seed(3)
        x, y = (torch.randn(T, d, generator=g, device="cuda").to(dt) for _ in range(2))
        bn = B.BlockNorm(d, after=True, before=True, gate="channel", channel_gate=torch.randn(d, generator=g, device="cuda"))
        h, n = bn.forward(x, y)
        for swap in (False, True):
            a, b = x.clone(), y.clone()
            s = torch.cuda.Stream()
            torch.cuda.synchronize()
            bn.forward(a, b, h_out=b if swap else a, n_out=a if swap else b, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(b if swap else a, h) and torch.equal(a if swap else b, n)
        for t in (0, 17, T - 1):
            h1, n1 = bn.forward(x[t:t + 1], y[t:t + 1])
            assert torch.equal(h1[0], h[t]) and torch.equal(n1[0], n[t])
        a, ho, no = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        a.copy_(x)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            bn.forward(a, y, h_out=ho, n_out=no)
        a.copy_(x.flip(0))
        gr.replay()
        torch.cuda.synchronize()
        want = bn.forward(x.flip(0).contiguous(), y)
        assert torch.equal(ho, want[0]) and torch.equal(no, want[1])
        bn.close()


def test_a_row_without_meaning_stays_alone(B):
    x, y = torch.randn(4, 512, device="cuda"), torch.randn(4, 512, device="cuda")
    bn = B.BlockNorm(512, after=True, before=True)
    h, n = bn.forward(x, y)
    x[1, 3], y[2, 5] = float("nan"), float("inf")
    h2, n2 = bn.forward(x, y)
    assert torch.equal(h2[[0, 3]], h[[0, 3]]) and torch.equal(n2[[0, 3]], n[[0, 3]])


def test_refusals(B):
    d = 64
    bn = B.BlockNorm(d, after=True, before=True, gate="row")
    x, y, g = torch.randn(4, d, device="cuda"), torch.randn(4, d, device="cuda"), torch.randn(4, device="cuda")
    h, n = bn.forward(x, y, gate=g)
    for call in (lambda: bn.forward(x, y), lambda: bn.forward(x, None, gate=g), lambda: bn.forward(x, y.half(), gate=g),
                 lambda: bn.forward(x, y, gate=g[:3]), lambda: bn.forward(x, y, gate=g.half()), lambda: bn.forward(x[:, :32], y, gate=g),
                 lambda: bn.forward(x, y[:3], gate=g), lambda: bn.forward(x.cpu(), y, gate=g), lambda: bn.forward(x.double(), y, gate=g),
                 lambda: bn.forward(x, y, gate=g, h_out=n, n_out=n),
                 lambda: B.BlockNorm(d, before=True).forward(x, y, gate=torch.randn(4, d, device="cuda")),
                 lambda: B.BlockNorm(d).forward(x, y, keep=False), lambda: B.BlockNorm(d).forward(x, y, n_out=n)):
        with pytest.raises(B.StrataError) as e:
            call()
        assert e.value.status == B.STRATA_EINVAL
    f, p, q, r = B.strata_blocknorm_forward, x.data_ptr(), y.data_ptr(), g.data_ptr()
    for args in ((p + 4, d, q, d, r, 0, h.data_ptr(), d, n.data_ptr(), d, 0, 4), (p, d - 4, q, d, r, 0, h.data_ptr(), d, n.data_ptr(), d, 0, 4),
                 (p, d, q, d, r, 0, p, d + 4, n.data_ptr(), d, 0, 4), (p, d, q, d, r, 0, None, d, None, d, 0, 4),
                 (p, d, q, d, r, 0, h.data_ptr(), d, n.data_ptr(), d, 5, 4), (p, d, q, d, r + 2, 0, h.data_ptr(), d, n.data_ptr(), d, 0, 4)):
        assert f(bn.handle, *args) == B.STRATA_EINVAL
    assert f(bn.handle, p, d, q, d, r, 0, h.data_ptr(), d, n.data_ptr(), d, 0, 0) == B.STRATA_OK


def test_a_gain_without_its_norm_is_not_applied(B):
    """after = 0: u = y whatever after_gain is, with a channel gate (which is folded into the same vector) as without."""
    d, T = 64, 3
    x, y, gain, gate = (torch.randn(*s, device="cuda") for s in ((T, d), (T, d), (d,), (d,)))
    for kind, p, g in ((B.STRATA_GATE_CHANNEL, gate.data_ptr(), gate), (B.STRATA_GATE_NONE, None, None)):
        st, h = B.strata_blocknorm_create(B.strata_blocknorm_desc(d, 0, 0, kind, 0, 1e-6, 1.0, 1.0), gain.data_ptr(), None, p)
        assert st == B.STRATA_OK
        out = torch.empty_like(x)
        assert B.strata_blocknorm_forward(h, x.data_ptr(), d, y.data_ptr(), d, None, 0, out.data_ptr(), d, None, 0, 0, T) == B.STRATA_OK
        torch.cuda.synchronize()
        _check((out, None), x, y, None, None, g, False, 1.0, 1.0, 1e-6)
        B.strata_blocknorm_destroy(h)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_over_the_range_that_the_header_gives(B, dtype):
    """Rows of 2^56 in the widest hidden size, and of 2^-60 without eps."""
    d = 16384
    g = torch.Generator(device="cuda").manual_seed(9)
    sign = torch.where(torch.rand(4, d, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    scale = torch.tensor([2.0 ** 56, 2.0 ** -60, 1.0, 2.0 ** 30], device="cuda")[:, None]
    y = (sign * scale).to(DTYPES[dtype])
    x = torch.zeros_like(y)
    one = torch.ones(d, device="cuda")
    for after in (None, one):
        h = B.BlockNorm(d, after=after, before=True, eps=0.0)
        _check(h.forward(x, y), x, y, after, one, None, False, 1.0, 1.0, 0.0)
        h.close()
