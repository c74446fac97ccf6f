"""The binding's objects hold addresses of the tensors that they were made of:
none of their attributes is replaced behind a descriptor's back.  Without a
GPU, on stand-ins that say they are on one."""
import ctypes

import pytest
import torch

from ternary_weight_only_tern_amd import lib as L


class OnGpu:
    """What the binding asks of a device tensor, its memory the host's."""

    device = torch.device("cuda", 0)

    def __init__(self, *shape, dtype=torch.int32):
        self._t = torch.zeros(shape, dtype=dtype)

    def __getattr__(self, name):
        return getattr(self._t, name)


def a_batch():
    return L.KvBatch(OnGpu(2), OnGpu(2, 5), 3, start=OnGpu(3))


def a_cache():
    codes, scales = (lambda: OnGpu(4, 2, 64, 64, dtype=torch.uint8)), (lambda: OnGpu(4, 2, dtype=torch.float32))
    return L.KvCache(codes(), codes(), scales(), scales())


def a_rope():
    return L.Rope(OnGpu(32, dtype=torch.float64), norm=OnGpu(64, dtype=torch.float16))


def a_matrix():
    return L.Q4Matrix(OnGpu(8, 64, dtype=torch.uint8), OnGpu(8, 1, dtype=torch.float16))


OBJECTS = [(a_batch, ("len", "pages", "start", "max_rows", "max_len", "count", "device")),
           (a_cache, ("k", "v", "k_scale", "v_scale", "pages", "heads", "dim")), (a_rope, ("freq", "norm", "dim")),
           (a_matrix, ("codes", "scale", "zero", "n", "k", "group"))]


@pytest.mark.parametrize("make,name", [(make, name) for make, names in OBJECTS for name in names])
def test_attributes_are_not_replaced(make, name):
    held = make()
    before = getattr(held, name)
    with pytest.raises(AttributeError):
        setattr(held, name, OnGpu(2))
    with pytest.raises(AttributeError):
        delattr(held, name)
    assert getattr(held, name) is before


def test_a_batch_passes_on_the_tensors_that_it_shows():
    """For a number of rows that it has met, too."""
    batch = a_batch()
    desc = batch._of(batch.device, 6)
    for name, new in (("len", OnGpu(2)), ("pages", OnGpu(2, 5)), ("start", OnGpu(3)), ("max_len", 7), ("max_rows", 2)):
        try:
            setattr(batch, name, new)
        except AttributeError:
            pass
        now = batch._of(batch.device, 6)
        shown = getattr(batch, name)
        assert getattr(now, name) == (shown if isinstance(shown, int) else shown.data_ptr()), name
    assert ctypes.addressof(batch._of(batch.device, 6)) == ctypes.addressof(desc)
