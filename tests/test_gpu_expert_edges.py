"""The expert operators at the edges of what they take: layouts, streams, sizes
and values, against the definitions in 64 bits. Tolerances: see _expert_util."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import unpermute_stable_counting_gb300 as usc  # noqa: E402

import _expert_util as eu  # noqa: E402
import test_gpu_layer as layer  # noqa: E402

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(autouse=True)
def _no_wait_ran_out():
    from unpermute_stable_counting_gb300 import _native
    yield
    n = ctypes.c_uint32(0)
    assert _native.lib().mr_waits_out(ctypes.byref(n), 1) == 0
    assert n.value == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def as_bytes(t):
    return t.contiguous().view(torch.uint8)


# ---------------------------------------------------------------------------
# moe_quantize
# ---------------------------------------------------------------------------

def quantized_blocks(x):
    """(values, scales) of float64 weights [..., n, k] in 128 x 128 blocks."""
    n, k = x.shape[-2:]
    t = torch.nn.functional.pad(x, (0, -k % 128, 0, -n % 128)).unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    s = eu.scale_of(t.abs().amax((-3, -1)))
    return eu.e4m3(x / s.repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]), s


@pytest.mark.parametrize("cut", [lambda w: w[:, ::2], lambda w: w[:, 1:2], lambda w: w[1:2, ::2], lambda w: w[:, :, 3:90],
                                 lambda w: w[::2, 1:2, :130, 8:]])
def test_quantize_weights_of_four_dimensions_in_part(cut):
    """Matrices some way apart, of x and of the values that are written."""
    w = torch.randn(4, 2, 140, 200, generator=gen(3)).to(BF16)
    x = cut(w)
    buf = torch.full((4, 2, 140, 208), 0x55, dtype=torch.uint8, device="cuda")
    values = cut(buf.view(E4M3))[..., :x.shape[-1]]
    q, s = quantized_blocks(x.double())
    out = dict(values=values, scales=torch.empty(s.shape, device="cuda"))
    usc.moe_quantize(cut(w.cuda()), block_rows=128, out=out)
    assert torch.equal(out["scales"].cpu().double(), s) and torch.equal(values.cpu().double(), q)
    left = torch.ones(4, 2, 140, 208, dtype=torch.bool)
    cut(left)[..., :x.shape[-1]] = False
    assert (buf.cpu()[left] == 0x55).all()
    r = usc.moe_quantize(cut(w.cuda()), block_rows=128)
    assert torch.equal(r["scales"].cpu().double(), s) and torch.equal(r["values"].cpu().double(), q)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("lead", [0, 3])
def test_quantize_many_rows(lead, dtype):
    """Enough blocks that each 8 lanes take two of them; rows that start on 16 bytes, and anywhere."""
    n, k, used = 40_001, 513, 39_990             # 5 blocks a row, the last of one value
    g = torch.Generator(device="cuda").manual_seed(4)
    buf = torch.full((lead + n * 520,), float("nan"), dtype=dtype, device="cuda")
    x = buf[lead:].view(n, 520)[:, :k] if lead == 0 else buf[lead:lead + n * 517].view(n, 517)[:, :k]
    x.copy_(torch.randn(n, k, device="cuda", generator=g) * torch.exp(3 * torch.randn(n, 1, device="cuda", generator=g)))
    out = usc.quantize_outputs((n, k), "cuda")
    out["values"].view(torch.uint8).fill_(0x55), out["scales"].fill_(-1.0)
    usc.moe_quantize(x, num_rows=torch.tensor([used], device="cuda"), out=out)
    q, s = eu.quantize(x[:used].double())
    for got, want in ((out["values"][:used].double(), q), (out["scales"][:used].double(), s)):
        bad = want.isnan()                       # f16: blocks with an infinity
        assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], want[~bad])
    assert (out["values"][used:].view(torch.uint8) == 0x55).all() and (out["scales"][used:] == -1).all()
    for rows_in_use, first in ((-5, 0), (n + 7, n)):
        out["scales"].fill_(-1.0)
        usc.moe_quantize(x, num_rows=torch.tensor([rows_in_use], device="cuda"), out=out)
        assert (out["scales"][first:] == -1).all() and (out["scales"][:first] != -1).all()


# ---------------------------------------------------------------------------
# Streams
# ---------------------------------------------------------------------------

def rows(n, k, dtype, g):
    x = torch.randn(n, k, generator=g)
    x[:, torch.randint(0, k, (max(1, k // 100),), generator=g)] *= 10
    return x.to(dtype)


def weights(lead, n, k, g):
    w = (torch.randn(*lead, n, k, generator=g) * 100).clamp(-448, 448).to(E4M3)
    s = torch.exp(0.4 * torch.randn(*lead, eu.blocks(n), eu.blocks(k), generator=g)) / (100 * k**0.5)
    return w, s


@pytest.mark.parametrize("raw", [False, True])
def test_a_call_on_another_stream_beside_one_whose_memory_was_just_freed(raw):
    """The first call's workspace and result are freed on the host with its kernels still queued on the
    current stream: the second call, on a side stream, must not be given them."""
    g = gen(78)
    H, inter, n = 512, 256, 900
    w13, s13 = (t.cuda() for t in weights((2, 2), inter, H, g))
    w2, s2 = (t.cuda() for t in weights((2,), H, inter, g))
    xs = [rows(n, H, BF16, g).cuda() for _ in range(2)]
    lists = [torch.tensor([[0, 400], [1, 500]]).cuda(), torch.tensor([[1, 300], [0, 600]]).cuda()]
    net = lambda i, **kw: usc.moe_expert_ffn(xs[i], w13, s13, w2, s2, lists[i], **kw)["y"]
    want = [net(0), net(1)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    first, second = [], []
    for _ in range(8):
        torch.cuda._sleep(2_000_000)
        first.append(net(0)), net(0)           # the second one's result is dropped at once
        second.append(net(1, stream=side.cuda_stream if raw else side))
    torch.cuda.synchronize()
    assert all(torch.equal(as_bytes(y), as_bytes(want[0])) for y in first)
    assert all(torch.equal(as_bytes(y), as_bytes(want[1])) for y in second)


def test_the_default_stream_by_its_handle():
    x = rows(40, 300, BF16, gen(79)).cuda()
    want = usc.moe_quantize(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = usc.moe_quantize(x, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(as_bytes(want[k]), as_bytes(got[k])) for k in want)


# ---------------------------------------------------------------------------
# moe_grouped_matmul
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("second", [1, 31])
def test_counts_past_the_rows_at_the_largest_number_of_rows(second):
    """2^30 rows and counts that add up to more than 2^31, in one window of 32 groups and over two."""
    n = 1 << 30
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = torch.full((n, 16), 0x38, dtype=torch.uint8, device="cuda").view(E4M3)     # ones
    w = torch.ones(2, 1, 16).to(E4M3)
    w[1] = 2.0
    lst = torch.zeros(second + 2, 2, dtype=torch.int64)
    lst[0, 1], lst[second], lst[second + 1] = n - 3, torch.tensor([1, n]), torch.tensor([0, 7])
    y = torch.zeros(n, 1, dtype=BF16, device="cuda")
    usc.moe_grouped_matmul(x, w.cuda(), torch.ones(2, 1, 1, device="cuda"), lst.cuda(),
                           x_scales=torch.ones(1, 1, device="cuda").expand(n, 1), out=dict(y=y))
    assert (y[:n - 3] == 16).all() and (y[n - 3:] == 32).all()
    # both counts are all of the rows: nothing is left for the others
    lst[0, 1] = n
    usc.moe_grouped_matmul(x, w.cuda(), torch.ones(2, 1, 1, device="cuda"), lst.cuda(),
                           x_scales=torch.ones(1, 1, device="cuda").expand(n, 1), out=dict(y=y))
    assert (y == 16).all()


def eight(n, k, g):
    q = (torch.randn(n, k, generator=g) * 100).clamp(-448, 448).to(E4M3)
    s = torch.exp(0.5 * torch.randn(n, eu.blocks(k), generator=g)) * 0.01
    return q, s, q.double() * eu.spread(s.double(), k)


def apart(t, unit=16):
    """A device copy whose last dimension is contiguous and whose matrices (or rows) start on 16 bytes."""
    lead, n = t.shape[0], t[0].numel()
    buf = torch.zeros(lead, -(-n // unit) * unit, dtype=t.dtype, device="cuda")
    v = buf.as_strided(t.shape, (buf.stride(0), *t.stride()[1:]))
    v.copy_(t.cuda())
    return v


@pytest.mark.parametrize("k", [500, 1, 129])
@pytest.mark.parametrize("n,N,E", [(1, 1, 1), (1, 1, 3), (1, 48, 1), (5, 1, 2)])
def test_single_rows_of_any_length(n, N, E, k):
    """A single e4m3 row (of x, or of each expert's weights) has no stride that 16 would have to divide."""
    g = gen(31 + k)
    q, s, x = eight(n, k, g)
    w, ws = weights((E,), N, k, g)
    xd = q.cuda() if n == 1 else apart(q)
    wd = w.cuda() if N == E == 1 else apart(w) if N == 1 else apart(w[0])[None]
    lst = torch.tensor([[E - 1, n]]).cuda()
    y = usc.moe_grouped_matmul(xd, wd, ws.cuda(), lst, x_scales=s.cuda(), out_dtype=F32)["y"]
    eu.assert_close(y, *eu.product(x, eu.weight(w, ws)[E - 1]))


def test_single_rows_through_the_network_and_the_layer():
    g = gen(32)
    H, inter = 137, 1                            # W1 and W3 have one row, which need not be padded
    w13, s13 = weights((2, 2), inter, H, g)
    w2, s2 = weights((2,), H, inter, g)
    q, s, x = eight(1, H, g)
    w13d = apart(w13.flatten(0, 1)).unflatten(0, (2, 2))
    w2d = apart(w2.flatten(0, 1)).unflatten(0, (2, H))
    assert w13d.stride()[-2] == H and w2d.stride()[-2] == 16
    y = usc.moe_expert_ffn(q.cuda(), w13d, s13.cuda(), w2d, s2.cuda(), torch.tensor([[1, 1]]).cuda(), x_scales=s.cuda(),
                           out_dtype=F32)["y"]
    W13, W2 = eu.weight(w13, s13), eu.weight(w2, s2)
    eu.assert_close(y, *eu.net(x, W13[1, 0], W13[1, 1], W2[1]))
    c = layer.make(3, 2, H, inter, BF16, E4M3, 33)
    r = usc.moe_layer(c["x"].cuda(), c["router"].cuda(), apart(c["w13"].flatten(0, 1)).unflatten(0, (2, 2)),
                      apart(c["w2"].flatten(0, 1)).unflatten(0, (2, H)), topk=2, w13_scales=c["s13"].cuda(),
                      w2_scales=c["s2"].cuda())
    layer.check(c, 2, r)


@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("N", [4092, 4090, 4089, 3970])
def test_rows_of_results_that_end_inside_16_bytes(N, out):
    """Rows that start on 16 bytes, N values in a row of 4096: what lies beside them stays as it is."""
    g = gen(N)
    n, k = 1000, 136
    q, s, x = eight(n, k, g)
    w, ws = weights((1,), N, k, g)
    buf = torch.full((n, 4096), 77.0, dtype=out, device="cuda")
    usc.moe_grouped_matmul(apart(q), apart(w[0])[None], ws.cuda(), x_scales=s.cuda(), out=dict(y=buf[:, :N]))
    eu.assert_close(buf[:, :N], *eu.product(x, eu.weight(w, ws)[0]))
    assert (buf[:, N:] == 77).all()


def test_offsets_past_32_bits():
    """Rows of x, of its 8-bit values and of y that lie past 2^31 elements, and weights past 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(35)
    n, k, N = 560_000, 4096, 4100
    x = torch.empty(n, k, dtype=BF16, device="cuda")
    for i in range(0, n, 40_000):
        x[i:i + 40_000] = torch.randn(40_000, k, device="cuda", generator=g).to(BF16)
    w = torch.randint(0, 256, (258, N, k), dtype=torch.uint8, device="cuda", generator=g).bitwise_and_(0xB7).view(E4M3)
    ws = torch.rand(258, eu.blocks(N), k // 128, device="cuda", generator=g) * 0.01
    lst = torch.tensor([[257, n - 70_001], [1, 70_001]]).cuda()
    q = usc.moe_quantize(x)
    sel = torch.tensor([0, 1, 299_999, 524_287, 524_288, n - 1], device="cuda")
    v, s = eu.quantize(x[sel].double())
    assert torch.equal(q["values"][sel].double(), v) and torch.equal(q["scales"][sel].double(), s)
    rows = v * eu.spread(s, k)
    ref = [eu.product(rows[j:j + 1], eu.weight(w[e], ws[e])) for j, e in enumerate([257, 257, 257, 1, 1, 1])]
    assert n - 70_001 <= 524_287
    ref, bound = (torch.cat(t).cpu() for t in zip(*ref))
    for xx, kw in ((x, {}), (q["values"], dict(x_scales=q["scales"]))):
        y = usc.moe_grouped_matmul(xx, w, ws, lst, **kw)["y"]
        eu.assert_close(y[sel], ref, bound)
        del y


# ---------------------------------------------------------------------------
# moe_layer
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("infinite", [True, False])
def test_bf16_values_of_h_past_the_range(infinite, sign):
    """An infinite h is one in its high part alone: y is infinite, not NaN. fp32's highest finite values,
    which round to an infinite bf16, stay finite."""
    c = layer.make(3, 4, 128, 32, BF16, BF16, 24)
    for k in ("x", "router", "w13", "w2"):
        c[k][:] = 0.0
    c["x"][1, :2] = 2.0**60
    c["w13"][:, 0, 5, 0] = 1.0                   # g = 2^60 = silu(g)
    if infinite:
        c["w13"][:, 1, 5, 0] = sign * 2.0**40    # h = 2^160
    else:                                        # u = 2^60 (256 - 2^-3): h = 2^128 (1 - 2^-11)
        c["w13"][:, 1, 5, 0], c["w13"][:, 1, 5, 1] = sign * 255.0, sign * 0.875
    c["w2"][:, :, 5] = 0.5
    y = layer.run(c, 2)["y"].double().cpu()
    assert (y[[0, 2]] == 0).all()
    if infinite:
        assert (y[1] == sign * float("inf")).all()
    else:                                        # half of h, to the nearest bf16 value
        assert ((y[1] - sign * 2.0**127).abs() <= 2.0**127 * 2.0**-8).all()


def test_f16_keeps_16_bits_of_a_small_h():
    """h of about 3e-5, of which f16 alone holds 9 bits: what cancels in y is known to 16 bits of h."""
    g = gen(25)
    T, E, H, I = 6, 2, 8, 32
    near = lambda *s: 1.0 + 0.02 * torch.rand(*s, generator=g)
    w13 = near(E, 2, I, H)
    w13[:, 1] *= 0.0625
    w2 = 400.0 * near(E, H, I)
    w2[:, :, 1::2] *= -1.0
    c = dict(x=(4e-3 * near(T, H)).to(F16), router=torch.zeros(E, H).to(F16), w13=w13.to(F16), w2=w2.to(F16), s13=None, s2=None)
    r = layer.run(c, 2)
    x, W13, W2 = c["x"].double(), c["w13"].double(), c["w2"].double()
    y, b = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        ye, be = eu.net(x, W13[e, 0], W13[e, 1], W2[e], rounded=False)
        a, u = x @ W13[e, 0].T, x @ W13[e, 1].T
        h = a * torch.sigmoid(a) * u
        assert (h > 2.0**-20).all() and (h < 2.0**-14).all()
        be = be + (h * 2.0**-16) @ W2[e].abs().T
        y += 0.5 * ye
        b += 0.5 * (be + 4 * 2.0**-23 * (ye.abs() + be))
    eu.assert_close(r["y"], y, b)
    # the bound means something: f16's own 2^-25 per value of h would be outside of it
    assert (b < 2.0**-25 * 400 * I**0.5).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_scores_below_fp32_s_range_still_weigh(score):
    """Scores whose sum fp32 does not hold, chosen by a bias: their ratios are those of the definition."""
    c = layer.make(5, 8, 128, 32, BF16, BF16, 26)
    c["x"][:] = 0.0
    c["x"][:, 0] = 1.0
    c["router"][:] = 0.0
    c["router"][:, 0] = torch.tensor([300.0 if score == "softmax" else 3.0, -96.0, -95.0, -95.5, -97.0, -170.0, -94.0, -99.0])
    bias = torch.tensor([0.0, 9.0, 8.0, 7.0, 6.0, 5.0, -1.0, -1.0])
    r = layer.run(c, 5, score=score, select_bias=bias.cuda(), routed_scale=2.5)
    assert torch.equal(r["expertIds"].cpu(), torch.tensor([1, 2, 3, 4, 5], dtype=torch.int32).expand(5, 5))
    assert ((r["expertWeights"].sum(1) - 2.5).abs() < 1e-5).all()
    layer.check(c, 5, r, score=score, routed_scale=2.5, bias=bias)


def test_a_taken_score_that_is_nan_leaves_no_weight():
    """The sum of the taken scores is NaN, and so is every weight of the token; other tokens keep theirs."""
    c = layer.make(3, 4, 128, 32, BF16, BF16, 27)
    c["router"][:, 5] = 0.0
    c["router"][2, 5] = float("nan")             # every token's logit of expert 2
    r = layer.run(c, 4, score="sigmoid")
    assert r["expertWeights"].isnan().all() and (r["expertIds"][:, 3] == 2).all() and r["y"].isnan().all()
    r = layer.run(c, 3, score="sigmoid")         # not taken
    assert ((r["expertWeights"].sum(1) - 1).abs() < 1e-5).all() and r["y"].isfinite().all()
    c["router"][2, 5] = 0.0
    c["x"][1, 9] = float("nan")                  # every logit of token 1
    r = layer.run(c, 2, score="sigmoid")
    assert r["expertWeights"][1].isnan().all() and r["expertWeights"][[0, 2]].isfinite().all()


def test_scores_that_are_all_zero_have_no_ratios():
    c = layer.make(2, 4, 128, 32, BF16, BF16, 28)
    c["x"][:] = 0.0
    c["x"][:, 0] = 1.0
    c["router"][:] = 0.0
    c["router"][:, 0] = float("-inf")
    r = layer.run(c, 2, score="sigmoid")
    assert r["expertWeights"].isnan().all() and torch.equal(r["expertIds"].cpu(), torch.tensor([[0, 1]] * 2, dtype=torch.int32))
    assert (layer.run(c, 2, score="sigmoid", renormalize=False)["expertWeights"] == 0).all()


@pytest.mark.parametrize("T,E,topk,H,I", [(64, 4, 2, 16384, 40), (64, 4, 2, 72, 16384), (64, 1024, 16, 136, 24),
                                          (13, 16, 16, 9800, 136)])
@pytest.mark.parametrize("wdt", [E4M3, BF16])
def test_the_largest_sizes_of_a_layer(T, E, topk, H, I, wdt):
    from unpermute_stable_counting_gb300 import _build, _native
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if H > 128 * (_build.FEW_SMS if _native.few_sms_requested() else sms):
        pytest.skip("a block takes at most 128 rows of y")
    c = layer.make(T, E, H, I, BF16, wdt, T + E + H + I)
    layer.check(c, topk, layer.run(c, topk))


# ---------------------------------------------------------------------------
# The count of waits that ran out
# ---------------------------------------------------------------------------

def test_the_count_of_waits_waits_for_every_stream():
    """Also for streams that the legacy default stream is not ordered with, as PyTorch's are."""
    from unpermute_stable_counting_gb300 import _native
    side, done, n = torch.cuda.Stream(), torch.cuda.Event(), ctypes.c_uint32(9)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)           # about 0.2 s
        done.record()
    assert _native.lib().mr_waits_out(ctypes.byref(n), 0) == 0 and n.value == 0
    assert done.query()


# ---------------------------------------------------------------------------
# The example
# ---------------------------------------------------------------------------

def test_the_example_runs_the_routed_rows_alone(monkeypatch):
    """Groups of as many rows as were routed; a capacity that holds every token gives the same result."""
    import os
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    monkeypatch.setattr(sys, "path", [os.path.join(root, "examples"), *sys.path])
    import moe_step
    T, E, topk, H = 100, 16, 3, 256
    wt = moe_step.make_weights(E, H, 128, seed=5)
    x = torch.randn(T, H, generator=gen(6)).to(BF16).cuda()
    seen, ffn = [], usc.moe_expert_ffn
    monkeypatch.setattr(moe_step.usc, "moe_expert_ffn", lambda r, *a, **k: (seen.append(r.shape[0]), ffn(r, *a, **k))[1])
    y, z = moe_step.routed_step(x, wt, topk), moe_step.routed_step(x, wt, topk, capacity=T)
    assert seen == [T * topk, T * E]
    # the padded way rounds each expert's rows to bf16 (2^-8 of each term), both round the result
    assert ((y - z).float().norm() / y.float().norm()) < 2.0**-7 and (y - z).abs().amax() <= y.abs().amax() * 2.0**-5
