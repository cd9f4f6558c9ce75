"""What the Python side of the operators hands to the library: addresses, strides
and streams, without a GPU (tensors that say they are on one, and a library that
only records its calls)."""
import contextlib
import inspect
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

    def record_stream(self, stream):
        self.used_on = getattr(self, "used_on", []) + [stream.name]


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


class Streams:
    """A device's current stream, and the streams that memory was asked for on."""
    def __init__(self):
        self.current, self.asked = self.make("main", 7), []

    def make(self, name, handle):
        return types.SimpleNamespace(name=name, cuda_stream=handle)

    @contextlib.contextmanager
    def use(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before

    def counted(self, allocate):
        def call(*args, **kw):
            self.asked.append(self.current.name)
            return gpu(allocate(*args, **kw))
        return call


@pytest.fixture
def streams(monkeypatch):
    s = Streams()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: s.current)
    monkeypatch.setattr(torch.cuda, "stream", s.use)
    monkeypatch.setattr(api, "_as_stream", lambda stream: stream, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: s.current.cuda_stream, raising=False)
    return s


@pytest.fixture
def calls(monkeypatch, streams):
    c = Calls()
    monkeypatch.setattr(api, "lib", lambda: c)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(api, "_device", lambda index: torch.device("cpu"))
    sizes = [f for f in vars(api).values() if hasattr(f, "cache_clear") and "workspace" in f.__name__]
    for f in sizes:
        f.cache_clear()
    yield c
    for f in sizes:
        f.cache_clear()


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


# ---------------------------------------------------------------------------
# Calls for another stream than the current one
# ---------------------------------------------------------------------------

def zeros(*shape, dtype=torch.float32):
    return gpu(torch.zeros(*shape, dtype=torch.uint8 if dtype is E4M3 else dtype).view(dtype))


def an_expert_call(name):
    BF16 = torch.bfloat16
    x, w, ws = zeros(4, 128, dtype=BF16), zeros(2, 64, 128, dtype=E4M3), zeros(2, 1, 1)
    w13, s13, w2, s2 = zeros(2, 2, 64, 128, dtype=E4M3), zeros(2, 2, 1, 1), zeros(2, 128, 64, dtype=E4M3), zeros(2, 1, 1)
    return dict(moe_quantize=((x,), {}), moe_grouped_matmul=((x, w, ws), {}), moe_expert_ffn=((x, w13, s13, w2, s2), {}),
                moe_layer=((x, zeros(2, 128, dtype=BF16), w13, w2), dict(topk=1, w13_scales=s13, w2_scales=s2)))[name]


def a_call(name):
    i32 = torch.int32
    x, m = zeros(4, 16, dtype=torch.float16), zeros(4, 2, dtype=torch.int8)
    if name == "moe_permute":
        return (x, m), dict(topk=1)
    if name == "moe_unpermute":
        return (x, zeros(4, dtype=i32), m, zeros(4, 2)), {}
    if name == "moe_update_expert":
        return (zeros(4, 2, dtype=i32), zeros(2, 3, dtype=i32)), dict(world_size=1)
    shape = dict(expert_num=2, max_out_shape=(1, 2, 2, 16), token_dtype=api.DT_F16)
    if name == "ffnwb_batching":
        return (zeros(4, dtype=i32), x, zeros(1, dtype=i32), zeros(1, dtype=i32)), shape
    if name == "ffnwb_batching_context":
        return (zeros(1024, dtype=torch.int8),), shape
    return an_expert_call(name)


ENTRIES = ["ffnwb_batching", "ffnwb_batching_context", "moe_permute", "moe_unpermute", "moe_update_expert", "moe_quantize",
           "moe_grouped_matmul", "moe_expert_ffn", "moe_layer"]


@pytest.mark.parametrize("name", ENTRIES)
def test_memory_of_a_call_for_another_stream_is_asked_for_on_that_stream(calls, streams, monkeypatch, name):
    """On the current stream it could be memory that a kernel in flight there still uses."""
    args, kw = a_call(name)
    f = getattr(api, name)
    for maker in ("empty", "zeros", "empty_strided"):
        monkeypatch.setattr(torch, maker, streams.counted(getattr(torch, maker)))
    out = f(*args, **kw)
    assert streams.asked and set(streams.asked) == {"main"}
    assert not any(hasattr(t, "used_on") for t in args)
    launches = [c for c in calls.made if not c.name.endswith("_size")]
    assert len(launches) == 1 and getattr(launches[0].args[-1], "value", launches[0].args[-1]) == 7
    streams.asked.clear(), calls.made.clear()
    out = f(*args, **kw, stream=streams.make("side", 9))
    assert streams.asked and set(streams.asked) == {"side"}
    launches = [c for c in calls.made if not c.name.endswith("_size")]
    assert len(launches) == 1 and getattr(launches[0].args[-1], "value", launches[0].args[-1]) == 9
    # what the caller gave is in use on the side stream, what the call made may be on the caller's
    assert all(t.used_on == ["side"] for t in args)
    assert all(t.used_on == ["main"] for t in out.values() if t is not None)
    assert "stream" in inspect.signature(f).parameters and streams.current.name == "main"


@pytest.mark.parametrize("name", ENTRIES)
def test_the_current_stream_by_name(calls, streams, monkeypatch, name):
    args, kw = a_call(name)
    for maker in ("empty", "zeros", "empty_strided"):
        monkeypatch.setattr(torch, maker, streams.counted(getattr(torch, maker)))
    getattr(api, name)(*args, **kw, stream=streams.current)
    assert not any(hasattr(t, "used_on") for t in args)


# ---------------------------------------------------------------------------
# Tensors of another device than the current one
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", ENTRIES)
def test_tensors_of_another_device_are_refused(calls, streams, monkeypatch, name):
    """The library would launch on the current device, with the other one's addresses."""
    args, kw = a_call(name)
    for t in (*args, *kw.values()):
        if isinstance(t, torch.Tensor):
            t.index = 1
    for maker in ("empty", "zeros", "empty_strided"):
        monkeypatch.setattr(torch, maker, streams.counted(getattr(torch, maker)))
    with pytest.raises(ValueError, match="current device"):
        getattr(api, name)(*args, **kw)
    assert not calls.made and not streams.asked
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for maker in ("empty", "zeros", "empty_strided"):
        monkeypatch.setattr(torch, maker, lambda *a, f=getattr(torch, maker), **k: gpu(f(*a, **k), 1))
    getattr(api, name)(*args, **kw)


def test_the_layer_s_workspace_is_that_of_the_device(calls, monkeypatch):
    """The same sizes on a device with another number of SMs need another workspace."""
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    for index, size in ((0, 1000), (1, 3000), (0, 1000)):
        monkeypatch.setattr(torch.cuda, "current_device", lambda: index)

        def answer(*args):
            args[-1]._obj.value = size
            return 0
        monkeypatch.setattr(calls, "moe_layer_get_workspace_size", answer, raising=False)
        assert api.layer_workspace_size(4, 128, 64, 8, 2, api.DT_E4M3) == size


# ---------------------------------------------------------------------------
# Memory that holds less than it shows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["moe_grouped_matmul", "moe_expert_ffn", "moe_layer"])
def test_an_expanded_workspace_is_refused(calls, streams, monkeypatch, name):
    args, kw = an_expert_call(name)
    with pytest.raises(ValueError, match="contiguous"):
        getattr(api, name)(*args, **kw, workspace=zeros(1, dtype=torch.uint8).expand(1 << 20), out=OUT(name))
    assert all(c.name.endswith("_size") for c in calls.made)
    getattr(api, name)(*args, **kw, workspace=zeros(1 << 20, dtype=torch.uint8)[256:], out=OUT(name))


def OUT(name):
    y = zeros(4, 64 if name == "moe_grouped_matmul" else 128, dtype=torch.bfloat16)
    return dict(y=y, expertIds=zeros(4, 1, dtype=torch.int32), expertWeights=zeros(4, 1))


@pytest.mark.parametrize("scales", [lambda: zeros(1, 1).expand(5, 3), lambda: zeros(1, 3).expand(5, 3),
                                    lambda: zeros(5, 1).expand(5, 3)])
def test_expanded_scales_are_not_written(calls, scales):
    x, values = zeros(5, 300, dtype=torch.bfloat16), zeros(5, 304, dtype=E4M3)[:, :300]
    with pytest.raises(ValueError, match="scales"):
        api.moe_quantize(x, out=dict(values=values, scales=scales()))
    assert not calls.made
    api.moe_quantize(x, out=dict(values=values, scales=zeros(3, 5).T))
    api.moe_quantize(x[:1], out=dict(values=values[:1], scales=zeros(3).as_strided((1, 3), (0, 1))))
    assert [tuple(c.args[11]) for c in calls.made] == [(1, 5), (1, 1)]


# ---------------------------------------------------------------------------
# Waits that ran out
# ---------------------------------------------------------------------------

def test_the_count_of_waits_that_ran_out(calls):
    """A call whose blocks gave up a wait returns like any other: the count is how a user learns of it."""
    import unpermute_stable_counting_gb300 as usc
    assert "waits_out" in usc.__all__

    def answer(count, reset):
        resets.append(reset)
        count._obj.value = 3
        return 0
    resets, calls.mr_waits_out = [], answer
    assert usc.waits_out() == 3 and usc.waits_out(reset=True) == 3 and resets == [0, 1]


@pytest.mark.parametrize("lead", [(0,), (0, 2), (3, 0)])
def test_no_weights_to_quantize(calls, lead):
    """A shard without experts."""
    x = zeros(*lead, 130, 64, dtype=torch.bfloat16)
    out = dict(values=zeros(*lead, 130, 64, dtype=E4M3), scales=zeros(*lead, 2, 1))
    assert api.moe_quantize(x, block_rows=128, out=out) is out and not calls.made
    r = api.moe_quantize(x[..., :0, :], block_rows=128, out=dict(values=out["values"][..., :0, :], scales=zeros(*lead, 0, 1)))
    assert r["values"].shape == (*lead, 0, 64)
