"""moe_quantize, moe_grouped_matmul and moe_expert_ffn against their
definitions in 64 bits. Tolerances: see _expert_util."""
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
    import ctypes
    from unpermute_stable_counting_gb300 import _native
    yield
    n = ctypes.c_uint32(0)
    assert _native.lib().mr_waits_out(ctypes.byref(n), 1) == 0
    assert n.value == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(n, k, dtype, g):
    x = torch.randn(n, k, generator=g)
    x[:, torch.randint(0, k, (max(1, k // 100),), generator=g)] *= 10
    return x.to(dtype)


def padded_cuda(t, fill=0x7F):
    """A device copy whose rows start on 16 bytes; the padding holds NaN bytes (0x7F)."""
    unit = 16 // t.element_size()
    wide = -(-t.shape[-1] // unit) * unit + unit
    buf = torch.full((*t.shape[:-1], wide * t.element_size()), fill, dtype=torch.uint8, device="cuda")
    v = buf.view(t.dtype)[..., :t.shape[-1]]
    v.view(torch.uint8).copy_(t.view(torch.uint8).cuda()) if t.element_size() == 1 else v.copy_(t.cuda())
    return v


def weights(lead, n, k, g):
    w = (torch.randn(*lead, n, k, generator=g) * 100).clamp(-448, 448).to(E4M3)
    s = torch.exp(0.4 * torch.randn(*lead, eu.blocks(n), eu.blocks(k), generator=g)) / (100 * k**0.5)
    return w, s


def group_list(pairs, total):
    out = torch.zeros(total, 2, dtype=torch.int64)
    out[:len(pairs)] = torch.tensor(pairs, dtype=torch.int64).reshape(-1, 2)
    return out.cuda()


def as_bytes(t):
    return t.contiguous().view(torch.uint8)


# ---------------------------------------------------------------------------
# moe_quantize
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("n,k", [(1, 1), (1, 128), (3, 127), (5, 129), (64, 7168), (7, 1000), (300, 136), (2, 4095)])
def test_quantize_rows(n, k, dtype):
    x = rows(n, k, dtype, gen(n * 7 + k))
    q, s = eu.quantize(x.double())
    r = usc.moe_quantize(x.cuda())
    assert r["values"].dtype == E4M3 and r["values"].stride(0) % 16 == 0
    assert torch.equal(r["scales"].cpu().double(), s)
    assert torch.equal(r["values"].cpu().double(), q)


def test_quantize_special_blocks():
    x = torch.zeros(9, 300)
    x[1] = 448.0                                 # the largest value itself: scale 1
    x[2] = 448.0001                              # just above: scale 2
    x[3, :128] = 2.0**-140                       # below the floor
    x[4, 5] = float("inf")
    x[5, 130] = float("nan")
    x[6] = torch.finfo(torch.float32).max
    x[7, ::2] = 17.0 / 16 * 256                  # half way between two values
    x[7, 1::2] = -19.0 / 16 * 256
    x[8, 299] = -3.0
    q, s = eu.quantize(x.double())
    r = usc.moe_quantize(x.cuda())
    gs, gq = r["scales"].cpu().double(), r["values"].cpu().double()
    assert torch.equal(gs.isnan(), s.isnan()) and s.isnan().sum() == 2
    assert torch.equal(gs.nan_to_num(7.0), s.nan_to_num(7.0))
    assert torch.equal(gq.isnan(), q.isnan()) and int(q.isnan().sum()) == 256
    assert torch.equal(gq.nan_to_num(7.0), q.nan_to_num(7.0))
    assert gs[0].tolist() == [2.0**-104] * 3     # an empty block: the floor's scale, values 0


def test_quantize_strides_rows_in_use_and_padding():
    g = gen(5)
    wide = torch.randn(40, 700, generator=g).to(BF16).cuda()
    x = wide[1::2, 3:3 + 385]                    # rows at odd 2-byte offsets
    buf = torch.full((20, 400), 0x55, dtype=torch.uint8, device="cuda")
    out = dict(values=buf.view(E4M3)[:, :385], scales=torch.full((4, 20), -1.0, device="cuda").T)
    used = torch.tensor([13], device="cuda")
    usc.moe_quantize(x, num_rows=used, out=out)
    q, s = eu.quantize(x.cpu().double())
    assert torch.equal(out["values"].cpu().double()[:13], q[:13])
    assert torch.equal(out["scales"].cpu().double()[:13], s[:13])
    assert (out["scales"][13:] == -1).all() and (buf[13:] == 0x55).all()
    assert (buf[:, 385:] == 0x55).all()          # the padding is the caller's


@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (130, 257), (2, 100, 300), (2, 2, 129, 64)])
def test_quantize_weights(shape):
    x = torch.randn(*shape, generator=gen(sum(shape))).to(BF16)
    r = usc.moe_quantize(x.cuda(), block_rows=128)
    v = x.double()
    n, k = shape[-2:]
    t = torch.nn.functional.pad(v, (0, -k % 128, 0, -n % 128))
    t = t.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))      # [.., nb, 128, kb, 128]
    s = eu.scale_of(t.abs().amax((-3, -1)))
    q = eu.e4m3(v / s.repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k])
    assert torch.equal(r["scales"].cpu().double(), s)
    assert torch.equal(r["values"].cpu().double(), q)


# ---------------------------------------------------------------------------
# moe_grouped_matmul
# ---------------------------------------------------------------------------

def reference(x, w, s, pairs, base=0):
    """float64 result and bound of each group's rows; rows of no expert NaN."""
    W = eu.weight(w, s)
    y = torch.full((x.shape[0], w.shape[1]), float("nan"), dtype=torch.float64)
    b = torch.zeros_like(y)
    at = 0
    for e, c in pairs:
        c = max(0, min(c, x.shape[0] - at))
        if 0 <= e - base < w.shape[0]:
            y[at:at + c], b[at:at + c] = eu.product(x[at:at + c], W[e - base])
        at += c
    return y, b


def eight(n, k, g):
    q = (torch.randn(n, k, generator=g) * 100).clamp(-448, 448).to(E4M3)
    s = torch.exp(0.5 * torch.randn(n, eu.blocks(k), generator=g)) * 0.01
    return q, s, q.double() * eu.spread(s.double(), k)


@pytest.mark.parametrize("n,N,k,out", [
    (1, 1, 1, F32), (1, 16, 128, BF16), (1, 2048, 512, BF16), (127, 33, 129, F16), (128, 64, 256, F32),
    (129, 256, 384, BF16), (300, 257, 640, F16), (257, 1000, 1000, F32), (5, 7168, 256, BF16),
    (1000, 4096, 136, BF16), (64, 511, 2000, F32)])
def test_dense_sizes(n, N, k, out):
    g = gen(n + N + k)
    q, s, x = eight(n, k, g)
    w, ws = weights((1,), N, k, g)
    got = usc.moe_grouped_matmul(padded_cuda(q), padded_cuda(w), ws.cuda(), x_scales=s.cuda(), out_dtype=out)["y"]
    assert got.dtype == out
    eu.assert_close(got, *eu.product(x, eu.weight(w, ws)[0]))


@pytest.mark.parametrize("xdt", [E4M3, BF16, F16, F32])
@pytest.mark.parametrize("pairs", [
    [(0, 130), (2, 1), (3, 0), (5, 255), (6, 3)],                  # compacted, one empty
    [(e, 7) for e in range(8)] * 1,                                # one row per expert
    [(7, 128), (0, 128), (7, 40)],                                 # any order, an expert twice
    [(1, 0), (2, -4), (3, 12)],                                    # nothing, a negative count
])
def test_groups(xdt, pairs):
    g = gen(len(pairs))
    total = sum(max(0, c) for _, c in pairs)
    n, N, k = total + 5, 300, 400
    w, ws = weights((8,), N, k, g)
    if xdt is E4M3:
        q, s, x = eight(n, k, g)
        args, kw = padded_cuda(q), dict(x_scales=s.cuda())
    else:
        q = rows(n, k, xdt, g)
        v, s = eu.quantize(q.double())
        x, args, kw = v * eu.spread(s, k), q.cuda(), {}
    y = torch.full((n, N), 77.0, dtype=F32, device="cuda")
    usc.moe_grouped_matmul(args, padded_cuda(w), ws.cuda(), group_list(pairs, len(pairs) + 3), out=dict(y=y), **kw)
    ref, b = reference(x, w, ws, pairs)
    real = ~ref[:, 0].isnan()
    eu.assert_close(y[real.cuda()], ref[real], b[real])
    assert (y[~real.cuda()] == 77.0).all()       # rows of no group keep what they held


def test_many_groups_and_expert_base():
    """More groups than a warp has lanes, most of them empty; layer 3's keys."""
    g = gen(9)
    counts = torch.randint(0, 4, (96,), generator=g) * (torch.rand(96, generator=g) < 0.5)
    counts[70], counts[95] = 200, 131
    pairs = [(3 * 96 + e, int(c)) for e, c in enumerate(counts)]
    n, N, k = int(counts.sum()), 192, 256
    q, s, x = eight(n, k, g)
    w, ws = weights((96,), N, k, g)
    got = usc.moe_grouped_matmul(q.cuda(), w.cuda(), ws.cuda(), group_list(pairs, 96), x_scales=s.cuda(),
                                 expert_base=3 * 96, out_dtype=F32)["y"]
    eu.assert_close(got, *reference(x, w, ws, pairs, base=3 * 96))


@pytest.mark.parametrize("total,present", [(1024, [0, 1, 2]), (1024, [5, 700, 1023]), (257, [255, 256]), (288, [31, 287]),
                                           (600, [])])
def test_long_lists_of_empty_groups(total, present):
    """Whole windows of empty groups before, between and after the others."""
    g = gen(total + len(present))
    n, N, k = 3 + 40 * len(present), 64, 128
    q, s, x = eight(n, k, g)
    w, ws = weights((4,), N, k, g)
    lst = torch.zeros(total, 2, dtype=torch.int64)
    lst[:, 1] = -(torch.arange(total) % 2)                # empty: 0 and -1
    pairs = []
    for j, i in enumerate(present):
        lst[i] = torch.tensor([j, 40])
        pairs.append((j, 40))
    y = torch.full((n, N), 77.0, dtype=F32, device="cuda")
    usc.moe_grouped_matmul(q.cuda(), w.cuda(), ws.cuda(), lst.cuda(), x_scales=s.cuda(), out=dict(y=y))
    ref, b = reference(x, w, ws, pairs)
    real = ~ref[:, 0].isnan()
    if present:
        eu.assert_close(y[real.cuda()], ref[real], b[real])
    assert (y[~real.cuda()] == 77.0).all()


def test_memory_of_a_call_on_another_stream_is_kept_until_it_is_done():
    g = gen(77)
    n, N, k = 4000, 512, 1024
    w, ws = weights((1,), N, k, g)
    w, ws, x = w.cuda(), ws.cuda(), rows(n, k, BF16, g).cuda()
    want = usc.moe_grouped_matmul(x, w, ws)["y"]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append(usc.moe_grouped_matmul(x, w, ws, stream=side)["y"])
        # as large as the call's workspace, on the current stream: must not be its memory
        torch.full((usc.grouped_matmul_workspace_size(n, k, 1),), 0x7F, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(as_bytes(want), as_bytes(y)) for y in got)


def test_experts_outside_and_counts_past_the_rows():
    g = gen(10)
    n, N, k = 150, 64, 128
    q, s, x = eight(n, k, g)
    w, ws = weights((4,), N, k, g)
    big = 1 << 62
    pairs = [(-1, 10), (4, 20), (1, 30), (big, 5), (2, big), (0, 40)]
    y = torch.full((n, N), 77.0, dtype=F32, device="cuda")
    usc.moe_grouped_matmul(q.cuda(), w.cuda(), ws.cuda(), group_list(pairs, 6), x_scales=s.cuda(), out=dict(y=y))
    ref, b = reference(x, w, ws, pairs)
    real = ~ref[:, 0].isnan()
    assert int(real.sum()) == 30 + 85
    eu.assert_close(y[real.cuda()], ref[real], b[real])
    assert (y[~real.cuda()] == 77.0).all()


@pytest.mark.parametrize("xdt", [E4M3, BF16])
def test_strided_operands_and_results(xdt):
    g = gen(11)
    n, N, k, E = 140, 200, 300, 3
    w, ws = weights((E,), N, k, g)
    wbuf = torch.full((E, 2, N, 336), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
    wv = wbuf[:, 1, :, 16:16 + k]                # every second matrix, rows 336 apart, 16 bytes in
    wv.view(torch.uint8).copy_(w.view(torch.uint8).cuda())
    if xdt is E4M3:
        q, s, x = eight(n, k, g)
        xbuf = torch.full((2 * n, 352), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
        xv = xbuf[::2, 32:32 + k]
        xv.view(torch.uint8).copy_(q.view(torch.uint8).cuda())
        kw = dict(x_scales=s.T.contiguous().cuda().T)   # block-major scales
    else:
        q = rows(n, k, xdt, g)
        v, s = eu.quantize(q.double())
        x, kw = v * eu.spread(s, k), {}
        xbuf = torch.full((2 * n, 311), float("nan"), dtype=xdt, device="cuda")
        xv = xbuf[1::2, 5:5 + k]
        xv.copy_(q.cuda())
    ybuf = torch.full((n, N + 9), 77.0, dtype=BF16, device="cuda")
    pairs = [(0, 60), (2, 80)]
    usc.moe_grouped_matmul(xv, wv, ws.cuda(), group_list(pairs, 2), out=dict(y=ybuf[:, 3:3 + N]), **kw)
    ref, b = reference(x, w, ws, pairs)
    eu.assert_close(ybuf[:, 3:3 + N], ref, b)
    assert (ybuf[:, :3] == 77).all() and (ybuf[:, 3 + N:] == 77).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("lead", [0, 1, 2, 3, 5, 7])
def test_quantize_rows_that_start_anywhere(lead, dtype):
    """Rows whose 16-byte words are shared with their neighbours: what lies beside them is not used."""
    g = gen(41)
    n, k = 37, 261
    x = rows(n, k, dtype, g)
    buf = torch.full((lead + n * (k + 2),), float("nan"), dtype=dtype, device="cuda")
    xv = buf[lead:].view(n, k + 2)[:, :k]
    xv.copy_(x.cuda())
    v, s = eu.quantize(x.double())
    r = usc.moe_quantize(xv)
    assert torch.equal(r["scales"].double().cpu(), s)
    assert torch.equal(r["values"].float().double().cpu(), v)


@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("N,lead,step", [(131, 1, 2), (515, 0, 0), (514, 3, 1), (96, 1, 1), (33, 2, 3), (1, 1, 1)])
@pytest.mark.parametrize("pairs", [[(0, 33), (1, 1), (2, 100)], [(1, 700)], [(2, 417), (0, 343)]])
def test_results_that_start_anywhere(N, lead, step, out, pairs):
    """Rows of results that share their words with what lies beside them, which stays as it is."""
    g = gen(42)
    n, k, E = sum(c for _, c in pairs), 130, 3
    q, s, x = eight(n, k, g)
    w, ws = weights((E,), N, k, g)
    ybuf = torch.full((lead + n * (N + step) + 1,), 77.0, dtype=out, device="cuda")
    body = ybuf[lead:lead + n * (N + step)].view(n, N + step)
    usc.moe_grouped_matmul(padded_cuda(q), padded_cuda(w), ws.cuda(), group_list(pairs, len(pairs)), x_scales=s.cuda(),
                           out=dict(y=body[:, :N]))
    ref, b = reference(x, w, ws, pairs)
    eu.assert_close(body[:, :N], ref, b)
    assert (body[:, N:] == 77).all() and (ybuf[:lead] == 77).all() and ybuf[-1] == 77


def test_non_finite_rows_stay_in_their_rows():
    g = gen(12)
    n, N, k = 200, 130, 256
    x = rows(n, k, BF16, g)
    x[17, 40] = float("nan")
    x[150, 200] = float("inf")
    w, ws = weights((1,), N, k, g)
    y = usc.moe_grouped_matmul(x.cuda(), w.cuda(), ws.cuda())["y"].float().cpu()
    bad = y.isnan()
    assert bad[17].all() and bad[150].all() and int(bad.any(1).sum()) == 2


def test_no_rows_and_no_groups():
    g = gen(13)
    w, ws = weights((2,), 64, 128, g)
    y = usc.moe_grouped_matmul(torch.empty(0, 128, dtype=BF16, device="cuda"), w.cuda(), ws.cuda())["y"]
    assert y.shape == (0, 64)
    y = torch.full((3, 64), 5.0, dtype=BF16, device="cuda")
    usc.moe_grouped_matmul(torch.ones(3, 128, dtype=BF16, device="cuda"), w.cuda(), ws.cuda(),
                           torch.empty(0, 2, dtype=torch.int64, device="cuda"), out=dict(y=y))
    assert (y == 5.0).all()


def test_repeats_bit_for_bit_on_two_streams():
    g = gen(14)
    n, N, k, E = 500, 700, 520, 6
    x, (w, ws) = rows(n, k, BF16, g).cuda(), weights((E,), N, k, g)
    w, ws = padded_cuda(w), ws.cuda()
    groups = group_list([(0, 200), (3, 299), (5, 1)], E)
    torch.cuda.synchronize()
    first = usc.moe_grouped_matmul(x, w, ws, groups)["y"]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            got.append(usc.moe_grouped_matmul(x, w, ws, groups)["y"])
    torch.cuda.synchronize()
    assert all(torch.equal(as_bytes(first), as_bytes(y)) for y in got)


# ---------------------------------------------------------------------------
# moe_expert_ffn
# ---------------------------------------------------------------------------

def ffn_reference(x, w13, s13, w2, s2, pairs):
    W13, W2 = eu.weight(w13, s13), eu.weight(w2, s2)
    y = torch.full((x.shape[0], x.shape[1]), float("nan"), dtype=torch.float64)
    b = torch.zeros_like(y)
    at = 0
    for e, c in pairs:
        if c > 0:
            y[at:at + c], b[at:at + c] = eu.net(x[at:at + c], W13[e, 0], W13[e, 1], W2[e])
        at += c
    return y, b


@pytest.mark.parametrize("xdt,H,inter,pairs", [
    (BF16, 256, 128, [(0, 1)]),
    (BF16, 128, 16, [(0, 3)]),
    (F16, 1080, 712, [(0, 130), (1, 1), (3, 77)]),
    (BF16, 392, 100, [(2, 128), (0, 0), (1, 129)]),
    (F32, 513, 257, [(0, 40), (1, 60)]),
    (E4M3, 640, 384, [(3, 200), (2, 5)]),
])
def test_expert_ffn(xdt, H, inter, pairs):
    g = gen(H + inter)
    n = sum(c for _, c in pairs)
    w13, s13 = weights((4, 2), inter, H, g)
    w2, s2 = weights((4,), H, inter, g)
    kw = {}
    if xdt is E4M3:
        q, s, x = eight(n, H, g)
        args, kw = padded_cuda(q), dict(x_scales=s.cuda())
    else:
        q = rows(n, H, xdt, g)
        v, s = eu.quantize(q.double())
        x, args = v * eu.spread(s, H), q.cuda()
    got = usc.moe_expert_ffn(args, padded_cuda(w13), s13.cuda(), padded_cuda(w2), s2.cuda(),
                             group_list(pairs, 4), **kw)["y"]
    assert got.dtype == (BF16 if xdt is E4M3 else xdt)
    eu.assert_close(got, *ffn_reference(x, w13, s13, w2, s2, pairs))


def test_expert_ffn_leaves_rows_of_no_group():
    g = gen(21)
    w13, s13 = weights((2, 2), 128, 256, g)
    w2, s2 = weights((2,), 256, 128, g)
    x = rows(50, 256, BF16, g).cuda()
    y = torch.full((50, 256), 7.0, dtype=BF16, device="cuda")
    used = torch.tensor([31], device="cuda")
    usc.moe_expert_ffn(x, w13.cuda(), s13.cuda(), w2.cuda(), s2.cuda(), group_list([(0, 11), (1, 20)], 2),
                       num_rows=used, out=dict(y=y))
    assert (y[31:] == 7.0).all() and not (y[:31] == 7.0).all(1).any()


def test_captured_into_a_graph():
    g = gen(22)
    w13, s13 = weights((2, 2), 256, 256, g)
    w2, s2 = weights((2,), 256, 256, g)
    a = [t.cuda() for t in (w13, s13, w2, s2)]
    x = rows(70, 256, BF16, g).cuda()
    groups = group_list([(0, 30), (1, 40)], 2)
    eager = usc.moe_expert_ffn(x, *a, groups)["y"]
    out = dict(y=torch.zeros_like(x))
    ws = torch.empty(usc.expert_ffn_workspace_size(70, 256, 256), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        usc.moe_expert_ffn(x, *a, groups, out=out, workspace=ws)
    for _ in range(3):
        out["y"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(as_bytes(out["y"]), as_bytes(eager))


def test_refusals():
    g = gen(23)
    w, ws = weights((2,), 64, 128, g)
    w, ws, x = w.cuda(), ws.cuda(), torch.ones(4, 128, dtype=BF16, device="cuda")
    q = usc.moe_quantize(x)
    with pytest.raises(ValueError):              # e4m3 rows without scales
        usc.moe_grouped_matmul(q["values"], w, ws)
    with pytest.raises(ValueError):              # another row length
        usc.moe_grouped_matmul(x[:, :64], w, ws)
    with pytest.raises(ValueError):              # scales of another shape
        usc.moe_grouped_matmul(x, w, ws[:, :0].contiguous())
    with pytest.raises(TypeError):               # 16-bit weights
        usc.moe_grouped_matmul(x, w.to(BF16), ws)
    with pytest.raises(TypeError):
        usc.moe_grouped_matmul(x.to(torch.float64), w, ws)
    with pytest.raises(TypeError):               # int32 groups
        usc.moe_grouped_matmul(x, w, ws, torch.zeros(2, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(usc.MoeReorderError):     # a workspace that is too small
        usc.moe_grouped_matmul(x, w, ws, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    odd = torch.zeros(2, 64, 136, dtype=torch.uint8, device="cuda").view(E4M3)[..., 8:]
    with pytest.raises(usc.MoeReorderError):     # weights that start on 8 bytes
        usc.moe_grouped_matmul(x, odd, ws)
    with pytest.raises(ValueError):
        usc.moe_quantize(x, block_rows=64)
