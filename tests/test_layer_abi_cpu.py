"""Refusals of the products, the sorting by expert and the block norms that need no GPU."""
import ctypes

import pytest

from slot_decode_window_gb300 import binding as B
from slot_decode_window_gb300 import build as BLD

Q = B.strata_qmat(0x1000, 0x1000, 0x1000)


@pytest.fixture(scope="module")
def lib():
    BLD.build()
    return B.load()


def _desc(cls, base, kw):
    base = dict(base, **kw)
    return cls(*(base[n] for n, _ in cls._fields_))


LINEAR = dict(n=1, out=64, bits=4, block=32, max_rows=8, **{"in": 64})
SORT = dict(n_experts=8, top_k=2, renorm_topk=0)
NORM = dict(hidden=64, after=1, before=1, gate=0, sigmoid=0, eps=1e-6, residual_scale=1.0, block_scale=1.0)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), B.STRATA_EINVAL), ({"in": 0}, B.STRATA_EINVAL), (dict(out=-16), B.STRATA_EINVAL),
    (dict(max_rows=0), B.STRATA_EINVAL), (dict(bits=2, block=16), B.STRATA_EUNSUPPORTED),
    (dict(block=64), B.STRATA_EUNSUPPORTED), ({"in": 96}, B.STRATA_EUNSUPPORTED), (dict(out=24), B.STRATA_EUNSUPPORTED),
    (dict(n=1025), B.STRATA_EUNSUPPORTED), ({"in": 65600}, B.STRATA_EUNSUPPORTED),
    (dict(out=(1 << 22) + 16), B.STRATA_EUNSUPPORTED), (dict(max_rows=(1 << 20) + 1), B.STRATA_EUNSUPPORTED),
])
def test_linear_create_rejects_bad_desc_on_host(lib, kw, status):
    assert B.strata_linear_create(_desc(B.strata_linear_desc, LINEAR, kw), Q) == (status, None)


def test_linear_create_rejects_bad_pointers(lib):
    d = _desc(B.strata_linear_desc, LINEAR, {})
    for q in (B.strata_qmat(None, 0x1000, 0x1000), B.strata_qmat(0x1000, None, 0x1000), B.strata_qmat(0x1000, 0x1000, None),
              B.strata_qmat(0x1000, 0x1001, 0x1000)):
        assert B.strata_linear_create(d, q) == (B.STRATA_EINVAL, None)
        assert B.strata_linear_create(d, Q, q) == (B.STRATA_EINVAL, None)
    assert lib.strata_linear_create(d, None, None, None, ctypes.byref(ctypes.c_void_p())) == B.STRATA_EINVAL
    assert lib.strata_linear_create(d, Q, None, None, None) == B.STRATA_EINVAL
    assert lib.strata_linear_create(None, Q, None, None, ctypes.byref(ctypes.c_void_p())) == B.STRATA_EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(n_experts=0), B.STRATA_EINVAL), (dict(top_k=0), B.STRATA_EINVAL), (dict(top_k=9), B.STRATA_EINVAL),
    (dict(renorm_topk=2), B.STRATA_EINVAL), (dict(n_experts=1025), B.STRATA_EUNSUPPORTED),
    (dict(n_experts=64, top_k=17), B.STRATA_EUNSUPPORTED),
])
def test_sort_create_rejects_bad_desc_on_host(lib, kw, status):
    assert B.strata_sort_create(_desc(B.strata_sort_desc, SORT, kw)) == (status, None)


@pytest.mark.parametrize("kw,status", [
    (dict(hidden=0), B.STRATA_EINVAL), (dict(after=2), B.STRATA_EINVAL), (dict(before=-1), B.STRATA_EINVAL),
    (dict(gate=4), B.STRATA_EINVAL), (dict(gate=B.STRATA_GATE_CHANNEL), B.STRATA_EINVAL), (dict(sigmoid=3), B.STRATA_EINVAL),
    (dict(eps=-1.0), B.STRATA_EINVAL), (dict(eps=float("nan")), B.STRATA_EINVAL), (dict(eps=float("inf")), B.STRATA_EINVAL),
    (dict(residual_scale=float("inf")), B.STRATA_EINVAL), (dict(block_scale=float("nan")), B.STRATA_EINVAL),
    (dict(hidden=12), B.STRATA_EUNSUPPORTED), (dict(hidden=16392), B.STRATA_EUNSUPPORTED),
])
def test_blocknorm_create_rejects_bad_desc_on_host(lib, kw, status):
    assert B.strata_blocknorm_create(_desc(B.strata_blocknorm_desc, NORM, kw)) == (status, None)


def test_fault_hook_alloc_gives_enomem(lib, monkeypatch):
    monkeypatch.setenv("STRATA_FAULT", "alloc")
    assert B.strata_linear_create(_desc(B.strata_linear_desc, LINEAR, {}), Q) == (B.STRATA_ENOMEM, None)
    assert B.strata_sort_create(_desc(B.strata_sort_desc, SORT, {})) == (B.STRATA_ENOMEM, None)
    assert B.strata_blocknorm_create(_desc(B.strata_blocknorm_desc, NORM, {})) == (B.STRATA_ENOMEM, None)


def test_calls_on_null_handles(lib):
    p = 0x1000
    assert B.strata_linear_forward(None, p, 64, p, 64, 0, 1) == B.STRATA_EINVAL
    assert B.strata_linear_sync(None) == B.STRATA_EINVAL and B.strata_linear_query(None)[0] == B.STRATA_EINVAL
    assert B.strata_sort_route(None, p, 8, None, 1, p, p) == B.STRATA_EINVAL
    assert B.strata_sort_plan(None, p, 1, B.strata_sort_order(p, p, p, p)) == B.STRATA_EINVAL
    assert B.strata_sort_gather(None, p, p, 64, p, 64, 0, 1, 64) == B.STRATA_EINVAL
    assert B.strata_sort_combine(None, p, p, 64, None, None, 0, p, 64, 0, 1, 64) == B.STRATA_EINVAL
    assert B.strata_sort_combine_backward(None, p, p, 64, p, 64, None, p, 64, p, 0, 1, 64) == B.STRATA_EINVAL
    assert B.strata_blocknorm_forward(None, p, 64, p, 64, None, 0, p, 64, p, 64, 0, 1) == B.STRATA_EINVAL
    for destroy in (B.strata_linear_destroy, B.strata_sort_destroy, B.strata_blocknorm_destroy):
        assert destroy(None) == B.STRATA_OK


def test_create_without_gpu_reports_cuda_error(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert B.strata_linear_create(_desc(B.strata_linear_desc, LINEAR, {}), Q) == (B.STRATA_ECUDA, None)
    assert B.strata_sort_create(_desc(B.strata_sort_desc, SORT, {})) == (B.STRATA_ECUDA, None)
    assert B.strata_blocknorm_create(_desc(B.strata_blocknorm_desc, NORM, {})) == (B.STRATA_ECUDA, None)


def test_binding_refuses_what_it_can_see():
    import types

    import torch
    cpu = types.SimpleNamespace(codes=torch.zeros(1, 16, 32, dtype=torch.uint8), scale=torch.zeros(1, 16, 2, dtype=torch.int16),
                                min=torch.zeros(1, 16, 2, dtype=torch.int16), rows=16, cols=64, bits=4, block=32)
    for call in (lambda: B.Linear(cpu), lambda: B.BlockNorm(64, gate="rows"), lambda: B.BlockNorm(64, gate="channel"),
                 lambda: B.BlockNorm(64, after=torch.ones(64))):
        with pytest.raises(B.StrataError) as e:
            call()
        assert e.value.status == B.STRATA_EINVAL


def test_round_weights_on_a_null_handle(lib):
    assert B.strata_linear_round_weights(None, 0) == B.STRATA_EINVAL
