"""What the Python side of the operators hands to the library: addresses, strides
and streams, without a GPU (tensors that say they are on one, and a library that
only records its calls)."""
import types

import pytest
import torch

from unpermute_stable_counting_gb300 import api

E4M3 = torch.float8_e4m3fn


class OnGpu(torch.Tensor):
    """A tensor in host memory that says it is on device 0."""
    is_cuda = property(lambda self: True)
    index = 0

    def get_device(self):
        return self.index


def gpu(t, index=0):
    t = torch.Tensor._make_subclass(OnGpu, t)
    t.index = index
    return t


class Calls:
    """Every library function: records its arguments, returns MR_OK."""
    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        def call(*args):
            self.made.append(types.SimpleNamespace(name=name, args=args))
            return 0
        return call

    def one(self):
        assert len(self.made) == 1
        return self.made[0]


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(api, "lib", lambda: c)
    monkeypatch.setattr(api, "_device", lambda index: torch.device("cpu"))
    monkeypatch.setattr(api, "_raw_stream", lambda stream, index: 0)
    return c


def quantized_matrices(c, x, values, scales):
    """{batch, row} strides of x and of values that a call for 128 x 128 blocks passed."""
    a = c.one().args
    assert a[0] == x.data_ptr() and a[8] == values.data_ptr() and a[10] == scales.data_ptr()
    return a[2], tuple(a[5]), tuple(a[9])


@pytest.mark.parametrize("cut", [lambda w: w[:, ::2], lambda w: w[:, 0:1], lambda w: w[:, 1:2]])
def test_weights_of_four_dimensions_whose_second_is_one(calls, cut):
    """One matrix of every pair: they lie a pair apart."""
    x = cut(gpu(torch.zeros(4, 2, 6, 32, dtype=torch.bfloat16)))
    values = cut(gpu(torch.zeros(4, 2, 6, 48, dtype=torch.uint8).view(E4M3)))[..., :32]
    scales = gpu(torch.zeros(4, 1, 1, 1))
    assert x.shape == (4, 1, 6, 32) and x.stride(0) == 384
    api.moe_quantize(x, block_rows=128, out=dict(values=values, scales=scales))
    batch, xs, vs = quantized_matrices(calls, x, values, scales)
    assert batch == 4 and xs == (384, 32) and vs == (2 * 6 * 48, 48)


def test_weights_of_four_dimensions_whose_first_is_one(calls):
    x = gpu(torch.zeros(3, 5, 6, 32, dtype=torch.bfloat16))[1:2, ::2]
    out = dict(values=gpu(torch.zeros(1, 3, 6, 32, dtype=torch.uint8).view(E4M3)), scales=gpu(torch.zeros(1, 3, 1, 1)))
    api.moe_quantize(x, block_rows=128, out=out)
    batch, xs, vs = quantized_matrices(calls, x, out["values"], out["scales"])
    assert batch == 3 and xs == (2 * 192, 32) and vs == (192, 32)


def test_weights_that_are_not_evenly_spaced_are_refused(calls):
    x = gpu(torch.zeros(4, 3, 6, 32, dtype=torch.bfloat16))[:, :2]
    out = dict(values=gpu(torch.zeros(4, 2, 6, 32, dtype=torch.uint8).view(E4M3)), scales=gpu(torch.zeros(4, 2, 1, 1)))
    with pytest.raises(ValueError):
        api.moe_quantize(x, block_rows=128, out=out)
    assert not calls.made
