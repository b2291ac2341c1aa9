"""The binding of the head norms and the 8-bit caches, as far as it goes without a GPU: a stand-in for torch records what
it asks of it."""
import types

import numpy as np
import pytest
import torch

from slot_decode_window_gb300 import binding as B
from slot_decode_window_gb300 import build as BLD


class Asked(Exception):
    pass


class Gain:
    """A float32 [64] on a device."""
    is_cuda, dtype, shape = True, "float32", (64,)

    def __init__(self, index):
        self.device = types.SimpleNamespace(index=index)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 4096


@pytest.fixture
def torch_(monkeypatch):
    """Two devices, of which 1 is current."""
    BLD.build()
    t = types.SimpleNamespace(uint8="uint8", float32="float32", empty_on=[], current=1)

    def empty(shape, dtype, device):
        t.empty_on.append(device)
        raise Asked

    class Device:
        def __init__(self, device):
            self.to = t.current if device is None else getattr(device, "index", device)

        def __enter__(self):
            self.was, t.current = t.current, self.to

        def __exit__(self, *_):
            t.current = self.was

    t.empty = empty
    t.cuda = types.SimpleNamespace(device=Device, current_device=lambda: t.current,
                                   current_stream=lambda: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(B, "_with_torch", lambda: t)
    t.created_on = []

    def create(*a):
        t.created_on.append(t.current)
        return B.STRATA_OK, 1

    monkeypatch.setattr(B, "strata_qknorm_create", create)
    monkeypatch.setattr(B, "strata_qknorm_destroy", lambda h: B.STRATA_OK)
    return t


@pytest.mark.parametrize("device,want", [(0, 0), (1, 1), (None, "cuda"), ("cuda:0", "cuda:0")])
def test_caches_are_made_on_the_device_that_was_asked_for(torch_, device, want):
    with pytest.raises(Asked):
        B.KvCache8(1, 1, 2, 2, 64, 16, device=device)
    assert torch_.empty_on == [want]


@pytest.mark.parametrize("device,q,k,want", [(0, None, None, 0), (None, None, None, 1), (0, 0, None, 0), (None, 0, 0, 0),
                                             (None, None, 0, 0), (1, 1, 1, 1)])
def test_norms_are_made_on_the_device_that_was_asked_for(torch_, device, q, k, want):
    gains = [None if g is None else Gain(g) for g in (q, k)]
    qk = B.QkNorm(2, 1, 64, device=device, q_gain=gains[0], k_gain=gains[1])
    assert qk.device == want and torch_.created_on == [want] and torch_.current == 1
    qk.close()


@pytest.mark.parametrize("device,q,k", [(0, 1, None), (0, 0, 1), (None, 1, 0), (1, None, 0)])
def test_norms_refuse_gains_of_another_device(torch_, device, q, k):
    gains = [None if g is None else Gain(g) for g in (q, k)]
    with pytest.raises(B.StrataError) as e:
        B.QkNorm(2, 1, 64, device=device, q_gain=gains[0], k_gain=gains[1])
    assert e.value.status == B.STRATA_EINVAL and not torch_.created_on


@pytest.mark.parametrize("form", [list, tuple, np.array, torch.tensor])
@pytest.mark.parametrize("n", [0, 4])
def test_frequencies_come_as_any_sequence(form, n):
    """Lists, arrays and tensors reach the library alike: infinite ones are found there, and none where some are due."""
    BLD.build()
    d = B.strata_qknorm_desc(2, 1, 64, 8, 0, 1, 1e-6)
    assert B.strata_qknorm_create(d, None, None, form([float("inf")] * n)) == (B.STRATA_EINVAL, None)
