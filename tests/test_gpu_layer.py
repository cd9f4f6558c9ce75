"""moe_layer against its definition in 64 bits. Tolerances: see _expert_util;
a token's experts have to be its highest logits (or biased scores), in order, up
to their fp32 error."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import unpermute_stable_counting_gb300 as usc  # noqa: E402

import _expert_util as eu  # noqa: E402

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


def padded(t):
    """A device copy whose rows start on 16 bytes, NaN bytes between them."""
    unit = 16 // t.element_size()
    wide = -(-t.shape[-1] // unit) * unit + unit
    buf = torch.full((*t.shape[:-1], wide * t.element_size()), 0xFF, dtype=torch.uint8, device="cuda")
    v = buf.view(t.dtype)[..., :t.shape[-1]]
    if t.element_size() == 1:
        v.view(torch.uint8).copy_(t.view(torch.uint8))
    else:
        v.copy_(t)
    return v


def make(T, E, H, I, xdt, wdt, seed, rdt=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g)
    x[:, torch.randint(0, H, (max(1, H // 100),), generator=g)] *= 6
    c = dict(x=x.to(xdt), router=(torch.randn(E, H, generator=g) / H**0.5).to(rdt or xdt))
    if wdt is E4M3:
        def w(*s):
            return (torch.randn(*s, generator=g) * 100).clamp(-448, 448).to(E4M3)

        def sc(*s):
            return torch.exp(0.4 * torch.randn(*s, generator=g)) / (100 * H**0.5)
        c.update(w13=w(E, 2, I, H), s13=sc(E, 2, eu.blocks(I), eu.blocks(H)), w2=w(E, H, I),
                 s2=sc(E, eu.blocks(H), eu.blocks(I)))
    else:
        c.update(w13=(torch.randn(E, 2, I, H, generator=g) / H**0.5).to(wdt), s13=None,
                 w2=(torch.randn(E, H, I, generator=g) / I**0.5).to(wdt), s2=None)
    return c


def run(c, topk, **kw):
    d = lambda t: None if t is None else t.cuda()
    r = usc.moe_layer(c["x"].cuda(), c["router"].cuda(), padded(c["w13"]), padded(c["w2"]), topk=topk,
                      w13_scales=d(c["s13"]), w2_scales=d(c["s2"]), **kw)
    torch.cuda.synchronize()
    return r


def check(c, topk, r, score="softmax", renormalize=True, routed_scale=1.0, bias=None):
    x, R = c["x"].double(), c["router"].double()
    T, E = x.shape[0], R.shape[0]
    logits, dl = eu.product(x, R)
    s = torch.softmax(logits, -1) if score == "softmax" else torch.sigmoid(logits)
    key, dk = (logits, dl) if bias is None else (s + bias.double(), 0 * s)
    ids = r["expertIds"].cpu().long()
    assert (ids >= 0).all() and (ids < E).all()
    assert all(len(set(row.tolist())) == topk for row in ids)
    # in descending order, and none left out above the last one, up to the fp32 error
    v, d = torch.gather(key, 1, ids), torch.gather(dk, 1, ids) + 1e-6
    assert (v[:, :-1] + d[:, :-1] >= v[:, 1:] - d[:, 1:]).all()
    left = (key - dk).scatter(1, ids, float("-inf")).amax(1)
    assert (v[:, -1] + d[:, -1] >= left).all()
    w = torch.gather(s, 1, ids)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    w = w * routed_scale
    gw = r["expertWeights"].cpu().double()
    # the exponents are off by the logits' error, and by a few units of fp32
    assert ((gw - w).abs() <= w.abs() * (4 * dl.max() + (40 + logits.abs().max()) * 2.0**-23)).all()
    eight = c["s13"] is not None
    if eight:
        W13, W2 = eu.weight(c["w13"], c["s13"]), eu.weight(c["w2"], c["s2"])
        q, sx = eu.quantize(x)
        x = q * eu.spread(sx, x.shape[1])
    else:
        W13, W2 = c["w13"].double(), c["w2"].double()
    y, b = torch.zeros_like(c["x"].double()), torch.zeros_like(c["x"].double())
    part = 2.0**-16 if c["x"].dtype == BF16 else 2.0**-20  # h in two parts of 8 (bf16) or 11 bits
    for e in ids.unique().tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        yt, bt = eu.net(x[t], W13[e, 0], W13[e, 1], W2[e], rounded=eight)
        if not eight:
            g, u = x[t] @ W13[e, 0].T, x[t] @ W13[e, 1].T
            h = (g * torch.sigmoid(g) * u).abs()
            # f16: parts below the normal range lose to its steps of 2^-24
            bt = bt + (h * part + (2.0**-24 if c["x"].dtype == F16 else 0.0)) @ W2[e].abs().T
        wt = gw[t, j][:, None]
        y[t] += wt * yt
        b[t] += wt.abs() * (bt + (topk + 2) * 2.0**-23 * (yt.abs() + bt))
    eu.assert_close(r["y"], y, b)


@pytest.mark.parametrize("wdt", [E4M3, BF16, F16])
@pytest.mark.parametrize("T,E,topk,H,I", [
    (1, 8, 1, 128, 64), (1, 64, 8, 1024, 256), (2, 3, 3, 256, 24), (5, 12, 3, 1000, 200), (16, 16, 2, 520, 136),
    (17, 8, 2, 512, 128), (32, 32, 4, 264, 72), (33, 40, 6, 768, 96), (64, 64, 8, 512, 160), (64, 2, 2, 256, 128),
    (7, 300, 5, 136, 48), (3, 700, 16, 144, 16)])
def test_layer(T, E, topk, H, I, wdt):
    c = make(T, E, H, I, BF16 if wdt is E4M3 else wdt, wdt, T + E + H + I)
    check(c, topk, run(c, topk))


@pytest.mark.parametrize("T,E,topk,H,I", [(9, 10, 2, 7168, 40), (20, 6, 2, 100, 2048), (1, 4, 2, 4095, 129),
                                          (4, 5, 3, 129, 7), (6, 6, 6, 1, 1)])
@pytest.mark.parametrize("wdt", [E4M3, BF16])
def test_long_and_odd_sizes(T, E, topk, H, I, wdt):
    c = make(T, E, H, I, BF16, wdt, T + E + H + I)
    check(c, topk, run(c, topk))


@pytest.mark.parametrize("score,renormalize,scale", [("softmax", False, 1.0), ("sigmoid", True, 2.5),
                                                     ("sigmoid", False, 1.0)])
@pytest.mark.parametrize("xdt,rdt,wdt", [(F32, F32, E4M3), (F16, F32, F16), (BF16, F16, BF16)])
def test_scores_and_types(score, renormalize, scale, xdt, rdt, wdt):
    c = make(11, 24, 384, 64, xdt, wdt, 3, rdt=rdt)
    kw = dict(score=score, renormalize=renormalize, routed_scale=scale)
    check(c, 4, run(c, 4, **kw), **kw)


def test_select_bias_chooses_but_does_not_weigh():
    c = make(12, 16, 256, 64, BF16, BF16, 5)
    bias = torch.zeros(16)
    bias[3], bias[7], bias[0] = 5.0, 4.0, -5.0
    r = run(c, 3, score="sigmoid", select_bias=bias.cuda())
    assert (r["expertIds"][:, 0] == 3).all() and (r["expertIds"][:, 1] == 7).all()
    check(c, 3, r, score="sigmoid", bias=bias)


def test_ties_go_to_the_lowest_expert():
    c = make(4, 40, 256, 32, BF16, BF16, 6)
    c["router"][:] = c["router"][0]              # every logit of a token the same
    r = run(c, 5)
    assert torch.equal(r["expertIds"].cpu(), torch.arange(5, dtype=torch.int32).expand(4, 5))
    check(c, 5, r)


def test_all_tokens_to_one_expert_and_every_expert_taken():
    c = make(64, 8, 256, 200, BF16, E4M3, 7)
    bias = torch.zeros(8)
    bias[5] = 10.0
    r = run(c, 1, select_bias=bias.cuda(), renormalize=False)
    assert (r["expertIds"] == 5).all()
    check(c, 1, r, renormalize=False, bias=bias)
    check(c, 8, run(c, 8))


def test_nan_logits_and_tokens():
    c = make(6, 9, 256, 64, BF16, BF16, 8)
    c["router"][4, 10] = float("nan")            # an expert whose logits are NaN is chosen last
    r = run(c, 8, renormalize=False, score="sigmoid")
    assert not (r["expertIds"] == 4).any()
    c = make(6, 9, 256, 64, BF16, E4M3, 9)
    c["x"][2, 7] = float("inf")                  # a bad token spoils its own row only
    y = run(c, 3)["y"].float().cpu()
    assert y[2].isnan().all() and int(y.isnan().any(1).sum()) == 1


def test_f16_values_past_the_range_are_infinities():
    c = make(3, 4, 128, 32, F16, F16, 14)
    c["x"][1] = 300.0
    c["w13"][:] = 2.0                            # h of token 1: (128 * 600)^2
    c["w2"][:] = 1.0
    y = run(c, 2)["y"].float().cpu()
    assert y[1].isinf().all() and (y[1] > 0).all()


def test_strided_rows_and_no_tokens():
    c = make(10, 8, 264, 72, BF16, BF16, 10)
    big = torch.full((20, 300), float("nan"), dtype=BF16, device="cuda")
    big[::2, 3:267] = c["x"].cuda()
    yb = torch.full((10, 280), 77.0, dtype=BF16, device="cuda")
    out = dict(y=yb[:, 5:269], expertIds=torch.empty(10, 2, dtype=torch.int32, device="cuda"),
               expertWeights=torch.empty(10, 2, device="cuda"))
    rb = torch.full((8, 301), float("nan"), dtype=BF16, device="cuda")
    rb[:, 1:265] = c["router"].cuda()
    usc.moe_layer(big[::2, 3:267], rb[:, 1:265], padded(c["w13"]), padded(c["w2"]), topk=2, out=out)
    check(c, 2, out)
    assert (yb[:, :5] == 77).all() and (yb[:, 269:] == 77).all()
    r = usc.moe_layer(torch.empty(0, 264, dtype=BF16, device="cuda"), c["router"].cuda(), padded(c["w13"]),
                      padded(c["w2"]), topk=2)
    assert r["y"].shape == (0, 264)


def test_same_numbers_as_the_grouped_network():
    """With 8-bit weights the layer is the router and moe_expert_ffn: one expert
    per token and weight 1 give the same rows up to the order of fp32 sums."""
    c = make(24, 6, 512, 256, F32, E4M3, 11)
    r = run(c, 1)
    ids = r["expertIds"].cpu()[:, 0].long()
    order = torch.argsort(ids, stable=True)
    groups = torch.stack([torch.arange(6), torch.bincount(ids, minlength=6)], 1).cuda()
    y = usc.moe_expert_ffn(c["x"][order].cuda(), padded(c["w13"]), c["s13"].cuda(), padded(c["w2"]), c["s2"].cuda(),
                           groups)["y"]
    got = r["y"][order.cuda()]
    assert (got - y).abs().max() <= 0.07 * y.abs().max()      # a value of h may round the other way
    assert ((got - y).norm() / y.norm()) < 2e-3


def test_repeats_bit_for_bit_beside_other_streams_and_in_a_graph():
    c = make(40, 32, 512, 192, BF16, E4M3, 12)
    args = (c["x"].cuda(), c["router"].cuda(), padded(c["w13"]), padded(c["w2"]))
    kw = dict(topk=4, w13_scales=c["s13"].cuda(), w2_scales=c["s2"].cuda())
    first = usc.moe_layer(*args, **kw)
    torch.cuda.synchronize()
    same = lambda r: all(torch.equal(first[k], r[k]) for k in first)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            got.append(usc.moe_layer(*args, **kw))
    torch.cuda.synchronize()
    assert all(same(r) for r in got)
    out = {k: torch.zeros_like(v) for k, v in first.items()}
    ws = torch.empty(usc.layer_workspace_size(40, 512, 192, 32, 4, usc.DT_E4M3), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        usc.moe_layer(*args, out=out, workspace=ws, **kw)
    for _ in range(3):
        for v in out.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out)


def test_refusals():
    c = make(4, 8, 128, 32, BF16, BF16, 13)
    args = [c["x"].cuda(), c["router"].cuda(), padded(c["w13"]), padded(c["w2"])]
    with pytest.raises(ValueError):
        usc.moe_layer(*args, topk=2, score="tanh")
    with pytest.raises(ValueError):              # scales with 16-bit weights
        usc.moe_layer(*args, topk=2, w13_scales=torch.ones(1, device="cuda"))
    with pytest.raises(TypeError):               # weights of another 16-bit type
        usc.moe_layer(args[0].half(), args[1], args[2], args[3], topk=2)
    with pytest.raises(ValueError):              # a router of another length
        usc.moe_layer(args[0], args[1][:, :64], args[2], args[3], topk=2)
    with pytest.raises(usc.MoeReorderError):     # more experts per token than there are
        usc.moe_layer(*args, topk=9)
    with pytest.raises(usc.MoeReorderError):     # 65 tokens
        usc.moe_layer(torch.ones(65, 128, dtype=BF16, device="cuda"), *args[1:], topk=2)
    with pytest.raises(usc.MoeReorderError):
        usc.moe_layer(*args, topk=2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):              # e4m3 weights without scales
        usc.moe_layer(args[0], args[1], padded(c["w13"].to(E4M3)), padded(c["w2"].to(E4M3)), topk=2)
