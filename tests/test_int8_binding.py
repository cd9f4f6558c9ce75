"""What the Python side of the INT8 operators hands to the library, and what it
refuses, without a GPU (the fakes are test_expert_binding's)."""
import pytest
import torch

from test_expert_binding import E4M3, calls, gpu, streams, zeros  # noqa: F401
from unpermute_stable_counting_gb300 import api

BF16, F16, I8, F32 = torch.bfloat16, torch.float16, torch.int8, torch.float32


def a_call(name):
    x, w, ws = zeros(4, 128, dtype=BF16), zeros(2, 64, 128, dtype=I8), zeros(2, 64)
    w13, s13, w2, s2 = zeros(2, 2, 64, 128, dtype=I8), zeros(2, 2, 64), zeros(2, 128, 64, dtype=I8), zeros(2, 128)
    return dict(moe_quantize_int8=((x,), {}), moe_add_rms_norm=((x, zeros(128, dtype=BF16)), dict(quantize="int8")),
                moe_grouped_matmul_int8=((x, w, ws), {}), moe_expert_ffn_int8=((x, w13, s13, w2, s2), {}))[name]


ENTRIES = ["moe_quantize_int8", "moe_add_rms_norm", "moe_grouped_matmul_int8", "moe_expert_ffn_int8"]


@pytest.fixture
def counted(monkeypatch, streams):
    for maker in ("empty", "zeros", "empty_strided"):
        monkeypatch.setattr(torch, maker, streams.counted(getattr(torch, maker)))


@pytest.mark.parametrize("name", ENTRIES)
def test_a_call_for_another_stream(calls, streams, counted, name):
    args, kw = a_call(name)
    streams.asked.clear()
    out = getattr(api, name)(*args, **kw, stream=streams.make("side", 9))
    assert streams.asked and set(streams.asked) == {"side"}
    launches = [c for c in calls.made if not c.name.endswith("_size")]
    assert len(launches) == 1 and launches[0].name == name and launches[0].args[-1] == 9
    assert all(t.used_on == ["side"] for t in args)
    assert all(t.used_on == ["main"] for t in out.values())


@pytest.mark.parametrize("name", ENTRIES)
def test_tensors_of_another_device(calls, streams, counted, name):
    args, kw = a_call(name)
    for t in args:
        t.index = 1
    with pytest.raises(ValueError, match="current device"):
        getattr(api, name)(*args, **kw)
    for t in args:
        t.index = 0
    args[-1].index = 1
    with pytest.raises(ValueError):
        getattr(api, name)(*args, **kw)
    assert not [c for c in calls.made if not c.name.endswith("_size")]


@pytest.mark.parametrize("f,error", [
    (lambda x, w: api.moe_quantize_int8(x[0]), ValueError),
    (lambda x, w: api.moe_quantize_int8(x.to(torch.float64)), TypeError),
    (lambda x, w: api.moe_quantize_int8(x.t()), ValueError),
    (lambda x, w: api.moe_quantize_int8(x[:, :6], interleaved=True), ValueError),
    (lambda x, w: api.moe_quantize_int8(x[None], interleaved=True), ValueError),
    (lambda x, w: api.moe_quantize_int8(x, out=dict(values=zeros(4, 8, dtype=torch.uint8), scales=zeros(4))), ValueError),
    (lambda x, w: api.moe_quantize_int8(x, out=dict(values=zeros(4, 8, dtype=I8), scales=zeros(5))), ValueError),
    (lambda x, w: api.moe_quantize_int8(x, out=dict(values=zeros(4, 8, dtype=I8), scales=zeros(1).expand(4))), ValueError),
    (lambda x, w: api.moe_quantize_int8(x, num_rows=zeros(1, dtype=torch.int32)), TypeError),
    (lambda x, w: api.moe_add_rms_norm(x, w, quantize="int4"), ValueError),
    (lambda x, w: api.moe_add_rms_norm(x, w, interleaved=True), ValueError),
    (lambda x, w: api.moe_add_rms_norm(x, w.to(F16)), TypeError),
    (lambda x, w: api.moe_add_rms_norm(x, w[:7]), ValueError),
    (lambda x, w: api.moe_add_rms_norm(x, w, x.to(F16)), ValueError),
    (lambda x, w: api.moe_add_rms_norm(x, w, x[:3]), ValueError),
    (lambda x, w: api.moe_add_rms_norm(x, w, out=dict(y=zeros(4, 9, dtype=BF16))), ValueError),
    (lambda x, w: api.moe_add_rms_norm(x, w, quantize="e4m3", out=dict(y=zeros(4, 8, dtype=BF16), values=zeros(4, 8, dtype=I8),
                                                                      scales=zeros(4, 1))), ValueError),
])
def test_rows_refused(calls, f, error):
    with pytest.raises(error):
        f(zeros(4, 8, dtype=BF16), zeros(8, dtype=BF16))
    assert not calls.made


def product(x=None, xs=None, w=None, ws=None, groups=None, **kw):
    x = zeros(4, 128, dtype=I8) if x is None else x
    w = zeros(2, 64, 128, dtype=I8) if w is None else w
    return api.moe_grouped_matmul_int8(x, w, zeros(2, 64) if ws is None else ws, groups,
                                       x_scales=zeros(4) if xs is None and x.dtype == I8 else xs, **kw)


@pytest.mark.parametrize("kw,error", [
    (dict(x=zeros(4, 128, dtype=F32)), TypeError), (dict(x=zeros(4, 128, dtype=torch.uint8)), TypeError),
    (dict(x=zeros(4, 64, dtype=I8)), ValueError), (dict(xs=zeros(5)), ValueError), (dict(xs=zeros(4, 1)), ValueError),
    (dict(xs=zeros(4, dtype=F16)), TypeError), (dict(w=zeros(2, 64, 128, dtype=torch.uint8)), TypeError),
    (dict(ws=zeros(2, 63)), ValueError), (dict(ws=zeros(2, 1)), ValueError), (dict(groups=zeros(3, 2)), TypeError),
    (dict(groups=zeros(3, 3, dtype=torch.int64)), ValueError), (dict(out_dtype=I8), TypeError),
    (dict(out=dict(y=zeros(4, 63, dtype=BF16))), ValueError),
])
def test_products_refused(calls, kw, error):
    with pytest.raises(error):
        product(**kw)
    assert not [c for c in calls.made if not c.name.endswith("_size")]


def test_int8_rows_need_scales(calls):
    with pytest.raises(ValueError):
        api.moe_grouped_matmul_int8(zeros(4, 128, dtype=I8), zeros(2, 64, 128, dtype=I8), zeros(2, 64))


def test_strides(calls):
    """A slice of interleaved rows, weights with room behind rows and matrices, a slice of y."""
    both = zeros(4, 144, dtype=I8)
    x, xs = both[:, :128], both.view(F32)[:, 32]
    w = zeros(3, 65, 160, dtype=I8)[:2, :64, :128]
    y = zeros(4, 70, dtype=BF16)[:, 3:67]
    product(x=x, xs=gpu(xs), w=w, out=dict(y=y))
    a = [c for c in calls.made if not c.name.endswith("_size")][0].args
    assert a[2] == 144 and a[3] == xs.data_ptr() and a[4] == 36
    assert tuple(a[6]) == (160, 65 * 160) and a[18] == 70


def test_workspaces_go_by_device(calls, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    for index, size in ((0, 1000), (1, 3000), (0, 1000)):
        monkeypatch.setattr(torch.cuda, "current_device", lambda: index)

        def answer(*args):
            args[-1]._obj.value = size
            return 0
        for name in ("moe_grouped_matmul_int8_get_workspace_size", "moe_expert_ffn_int8_get_workspace_size"):
            monkeypatch.setattr(calls, name, answer, raising=False)
        assert api.grouped_matmul_int8_workspace_size(8, 2, 64, 128, api.DT_INT8) == size
        assert api.expert_ffn_int8_workspace_size(8, 2, 64, 128, api.DT_INT8) == size
