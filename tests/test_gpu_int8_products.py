"""moe_grouped_matmul_int8 and moe_expert_ffn_int8 against their definitions in 64 bits."""
import pytest
import torch

from _expert_util import assert_close, product
from _int8_util import net, weight

pytestmark = pytest.mark.gpu

F16, BF16, F32, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def usc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import unpermute_stable_counting_gb300 as u
    return u


@pytest.fixture(autouse=True)
def _no_wait_ran_out(usc):
    yield
    assert usc.waits_out(reset=True) == 0


def wide(t, dtype=None):
    """t on the GPU with rows that start on 16 bytes, other data between them."""
    dtype = dtype or t.dtype
    unit = 16 // torch.empty(0, dtype=dtype).element_size()
    cols = -(-t.shape[-1] // unit) * unit + unit
    buf = torch.full((*t.shape[:-1], cols), 99, dtype=dtype)
    buf[..., :t.shape[-1]] = t
    return buf.cuda()[..., :t.shape[-1]]


def rows_of(rows, K, dtype, seed):
    """(rows, scales or None, the values they stand for in 64 bits)."""
    g = torch.Generator().manual_seed(seed)
    if dtype == I8:
        x = torch.randint(-127, 128, (rows, K), generator=g).to(I8)
        x[:, ::7] = -127
        s = torch.rand(rows, generator=g) * 0.02 + 0.001
        return wide(x), s.cuda(), x.double() * s.double()[:, None]
    x = torch.randn(rows, K, generator=g).to(dtype)
    return wide(x), None, x.double()


def weights_of(lead, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(*lead, N, K, generator=g) * 40).round().clamp(-128, 127).to(I8)
    s = (torch.rand(*lead, N, generator=g) + 0.5) / (40 * K**0.5)
    return w, s


def groups_of(rows, experts, seed, empty=0.3):
    """(group list, [(expert, first row, rows)]) with some groups empty, in no order of their experts."""
    g = torch.Generator().manual_seed(seed)
    cut = torch.sort(torch.randint(0, rows + 1, (experts - 1,), generator=g))[0].tolist()
    counts = [b - a for a, b in zip([0, *cut], [*cut, rows])]
    order = torch.randperm(experts, generator=g).tolist()
    return torch.tensor([[e, c] for e, c in zip(order, counts)], dtype=torch.int64), counts, order


def expected(values, groups, f, cols):
    """f(expert, its rows) -> (y, bound) of every group, put together."""
    y, b = torch.zeros(len(values), cols, dtype=torch.float64), torch.zeros(len(values), cols, dtype=torch.float64)
    at = 0
    for e, c in groups.tolist():
        c = min(c, len(values) - at)
        if c > 0:
            y[at:at + c], b[at:at + c] = f(e, values[at:at + c])
            at += c
    return y, b


def check_matmul(usc, rows, experts, N, K, x_dtype, out, seed=0, groups=None):
    x, xs, values = rows_of(rows, K, x_dtype, seed)
    w, ws = weights_of((experts,), N, K, seed + 1)
    if groups is None:
        groups = groups_of(rows, experts, seed + 2)[0]
    y = usc.moe_grouped_matmul_int8(x, wide(w), ws.cuda(), groups.cuda(), x_scales=xs, out_dtype=out)["y"]
    wd = weight(w, ws)
    want, bound = expected(values, groups, lambda e, v: product(v, wd[e]), N)
    assert_close(y, want, bound + want.abs() * 2.0**-22)  # and two products with scales
    return y


def check_ffn(usc, rows, experts, H, inter, x_dtype, out=None, seed=0, groups=None):
    x, xs, values = rows_of(rows, H, x_dtype, seed)
    w13, s13 = weights_of((experts, 2), inter, H, seed + 1)
    w2, s2 = weights_of((experts,), H, inter, seed + 2)
    if groups is None:
        groups = groups_of(rows, experts, seed + 3)[0]
    y = usc.moe_expert_ffn_int8(x, wide(w13), s13.cuda(), wide(w2), s2.cuda(), groups.cuda(), x_scales=xs,
                                out_dtype=out)["y"]
    a, b = weight(w13, s13), weight(w2, s2)
    want, bound = expected(values, groups, lambda e, v: net(v, a[e, 0], a[e, 1], b[e]), H)
    assert_close(y, want, bound + want.abs() * 2.0**-22)
    return y


@pytest.mark.parametrize("x_dtype", [I8, F16, BF16])
@pytest.mark.parametrize("rows", [1, 2, 16, 17, 33, 64, 65, 200, 500])
def test_rows(usc, rows, x_dtype):
    check_matmul(usc, rows, 1, 300, 256, x_dtype, F32, rows)


@pytest.mark.parametrize("K", [1, 15, 16, 63, 64, 65, 127, 128, 129, 500, 1000, 2048])
@pytest.mark.parametrize("x_dtype", [I8, F16, BF16])
def test_row_lengths(usc, K, x_dtype):
    check_matmul(usc, 40, 3, 130, K, x_dtype, F32, K)
    check_matmul(usc, 300, 2, 130, K, x_dtype, F32, K)


@pytest.mark.parametrize("N", [1, 31, 32, 127, 128, 129, 256, 257, 1100])
@pytest.mark.parametrize("out", [BF16, F16, F32])
def test_widths(usc, N, out):
    check_matmul(usc, 50, 4, N, 192, I8, out, N)
    check_matmul(usc, 400, 4, N, 192, I8, out, N)
    check_matmul(usc, 400, 4, N, 192, BF16, out, N)


@pytest.mark.parametrize("x_dtype", [I8, F16, BF16])
def test_several_tiles_for_each_block(usc, x_dtype):
    check_matmul(usc, 300, 40, 1500, 320, x_dtype, BF16)
    check_matmul(usc, 2600, 9, 2100, 320, x_dtype, BF16)


@pytest.mark.parametrize("x_dtype", [I8, F16, BF16])
@pytest.mark.parametrize("rows,experts,H,inter", [(1, 1, 128, 64), (7, 3, 200, 100), (50, 4, 1080, 712), (515, 6, 136, 200),
                                                  (900, 2, 512, 700)])
def test_ffn(usc, rows, experts, H, inter, x_dtype):
    check_ffn(usc, rows, experts, H, inter, x_dtype, seed=rows)


@pytest.mark.parametrize("out", [BF16, F16, F32])
def test_ffn_outputs(usc, out):
    check_ffn(usc, 30, 2, 264, 136, I8, out)
    check_ffn(usc, 300, 2, 264, 136, I8, out)


# ---------------------------------------------------------------------------
# Group lists, rows that are not the call's, strides
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("x_dtype", [I8, BF16])
@pytest.mark.parametrize("rows", [20, 700])
def test_lists(usc, rows, x_dtype):
    """Empty groups, negative counts, experts that are not there, a group that reaches past the rows; rows of
    none of them stay as they were."""
    E, N, K, base = 5, 200, 160, 100
    x, xs, values = rows_of(rows, K, x_dtype, 1)
    w, ws = weights_of((E,), N, K, 2)
    wd = weight(w, ws)
    a, b = rows // 4, rows // 3
    for groups in ([[101, a], [100, 0], [7, b], [104, -5], [105, 2], [102, 10 * rows]],
                   [[99, a], [100, b]], [[0, 0]] * 40 + [[103, a], [0, 0]] + [[100, b]], [[102, 1]] * rows):
        g = torch.tensor(groups, dtype=torch.int64)
        y = torch.full((rows, N), 5.0, device="cuda")
        usc.moe_grouped_matmul_int8(x, wide(w), ws.cuda(), g.cuda(), x_scales=xs, expert_base=base, out=dict(y=y))
        got, at = y.cpu(), 0
        for e, c in groups:
            c = max(0, min(c, rows - at))
            if base <= e < base + E:
                assert_close(got[at:at + c], *product(values[at:at + c], wd[e - base]))
            else:
                assert (got[at:at + c] == 5.0).all()
            at += c
        assert (got[at:] == 5.0).all()


@pytest.mark.parametrize("groups", [40, 257, 1000])
def test_long_lists(usc, groups):
    """Lists of several windows, and longer than what is walked twice."""
    counts = torch.zeros(groups, dtype=torch.int64)
    counts[::7] = 1
    counts[-1] = 3
    g = torch.stack([torch.arange(groups) % 3, counts], 1)
    rows = int(counts.sum())
    for x_dtype in (I8, F16):
        check_matmul(usc, rows, 3, 300, 2100, x_dtype, F32, 3, g)


def test_no_list_and_no_rows(usc):
    for rows in (1, 90, 300):
        x, xs, values = rows_of(rows, 256, I8, rows)
        w, ws = weights_of((3,), 130, 256, 5)
        y = usc.moe_grouped_matmul_int8(x, wide(w), ws.cuda(), x_scales=xs, out_dtype=F32)["y"]
        assert_close(y, *product(values, weight(w, ws)[0]))
    x = torch.empty(0, 256, dtype=I8, device="cuda")
    assert usc.moe_grouped_matmul_int8(x, wide(w), ws.cuda(), x_scales=torch.empty(0, device="cuda"))["y"].shape == (0, 130)
    y = torch.full((4, 130), 3.0, device="cuda")
    x, xs, _ = rows_of(4, 256, I8, 1)
    usc.moe_grouped_matmul_int8(x, wide(w), ws.cuda(), torch.empty(0, 2, dtype=torch.int64, device="cuda"), x_scales=xs,
                                out=dict(y=y))
    assert (y == 3.0).all()


@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("rows", [9, 300])
def test_results_keep_their_surroundings(usc, rows, out):
    N, K = 133, 200
    x, xs, values = rows_of(rows, K, I8, 3)
    w, ws = weights_of((1,), N, K, 4)
    want, bound = product(values, weight(w, ws)[0])
    for start, pad in ((0, 0), (1, 3), (5, 11)):
        buf = torch.full((start + rows * (N + pad) + 7,), 3.0, dtype=out, device="cuda")
        y = buf.as_strided((rows, N), (N + pad, 1), start)
        usc.moe_grouped_matmul_int8(x, wide(w), ws.cuda(), x_scales=xs, out=dict(y=y))
        assert_close(y, want, bound + want.abs() * 2.0**-22)
        y.fill_(3.0)
        assert (buf == 3.0).all()


def test_strides(usc):
    """Rows of interleaved scales, weights with room behind rows and matrices, single rows and matrices of any stride."""
    E, N, K, rows = 2, 70, 128, 40
    g = torch.Generator().manual_seed(1)
    both = torch.randint(-127, 128, (rows, K + 16), generator=g).to(I8)
    both.view(F32)[:, K // 4] = torch.rand(rows, generator=g)
    w, ws = weights_of((E,), N, K, 2)
    room = torch.full((E, N + 3, K + 32), 77, dtype=I8)
    room[:, :N, :K] = w
    dev = both.cuda()
    groups = torch.tensor([[1, 15], [0, 25]], dtype=torch.int64)
    y = usc.moe_grouped_matmul_int8(dev[:, :K], room.cuda()[:, :N, :K], ws.cuda(), groups.cuda(),
                                    x_scales=dev.view(F32)[:, K // 4], out_dtype=F32)["y"]
    values = both[:, :K].double() * both.view(F32)[:, K // 4].double()[:, None]
    wd = weight(w, ws)
    want, bound = expected(values, groups, lambda e, v: product(v, wd[e]), N)
    assert_close(y, want, bound)
    one = usc.moe_grouped_matmul_int8(dev[:1, :100], room.cuda()[:1, :1, :100], ws.cuda()[:1, :1].contiguous(),
                                      x_scales=dev.view(F32)[:1, K // 4], out_dtype=F32)["y"]
    assert_close(one, *product(values[:1, :100], wd[0, :1, :100]))


@pytest.mark.parametrize("x_dtype", [F16, BF16])
@pytest.mark.parametrize("rows", [12, 300])
def test_scales_of_16_bit_rows(usc, rows, x_dtype):
    x, _, values = rows_of(rows, 300, x_dtype, 6)
    xs = torch.rand(rows, 3)
    w, ws = weights_of((1,), 150, 300, 7)
    y = usc.moe_grouped_matmul_int8(x, wide(w), ws.cuda(), x_scales=xs.cuda()[:, 1], out_dtype=F32)["y"]
    assert_close(y, *product(values * xs[:, 1:2].double(), weight(w, ws)[0]))


@pytest.mark.parametrize("rows", [12, 300])
def test_unusual_values(usc, rows):
    """Infinities and NaN stay in their rows, and behind the rows nothing is read; -128 is a value like any other."""
    K, N = 200, 150
    w = torch.randint(-128, 128, (1, N, K)).to(I8)
    w[0, 3] = -128
    ws = torch.rand(1, N)
    ws[0, 5], ws[0, 6] = 0.0, float("inf")
    x = torch.randn(rows, K).to(BF16)
    x[2, 7], x[4, 9] = float("inf"), float("nan")
    x[5] = 0.0
    y = usc.moe_grouped_matmul_int8(wide(x), wide(w), ws.cuda(), out_dtype=F32)["y"].cpu()
    # (fp32's order of the two products: sum, channel's scale)
    plain = (x.double() @ w[0].double().T) * ws.double()
    assert torch.equal(torch.isnan(y), torch.isnan(plain)) and torch.equal(torch.isinf(y), torch.isinf(plain))
    keep = torch.isfinite(plain)
    _, bound = product(torch.nan_to_num(x.double(), 0, 0, 0), weight(w, torch.nan_to_num(ws, posinf=0.0))[0])
    assert ((y.double() - plain)[keep].abs() <= (bound + plain.abs() * 2.0**-22)[keep]).all()
    q = torch.randint(-128, 128, (rows, K)).to(I8)
    s = torch.rand(rows)
    s[1], s[3] = float("nan"), 0.0
    y = usc.moe_grouped_matmul_int8(wide(q), wide(w), ws.cuda(), x_scales=s.cuda(), out_dtype=F32)["y"].cpu()
    plain = (q.double() @ w[0].double().T) * ws.double() * s.double()[:, None]
    assert torch.equal(torch.isnan(y), torch.isnan(plain))
    assert torch.equal(y[3][torch.isfinite(plain[3])], torch.zeros(N)[torch.isfinite(plain[3])])


@pytest.mark.parametrize("rows,K", [(1, 4096), (30, 3000), (300, 4096)])
def test_sums_of_int8_are_exact(usc, rows, K):
    """Below 2^24 a sum is exact, so with scales of 1 the result is the integer."""
    q = torch.randint(-20, 21, (rows, K)).to(I8)
    w = torch.randint(-20, 21, (1, 260, K)).to(I8)
    y = usc.moe_grouped_matmul_int8(wide(q), wide(w), torch.ones(1, 260, device="cuda"), x_scales=torch.ones(rows, device="cuda"),
                                    out_dtype=F32)["y"].cpu()
    assert torch.equal(y.double(), q.double() @ w[0].double().T)


def test_ffn_lists_and_large_activations(usc):
    """h past f16's range is a bf16 value like any other; rows of no group stay."""
    H, inter, rows = 128, 96, 50
    x = (torch.randn(rows, H) * 300).to(BF16)
    w13, s13 = weights_of((2, 2), inter, H, 1)
    w2, s2 = weights_of((2,), H, inter, 2)
    groups = torch.tensor([[1, 20], [9, 5], [0, 20]], dtype=torch.int64)
    y = torch.full((rows, H), 7.0, dtype=F32, device="cuda")
    usc.moe_expert_ffn_int8(wide(x), wide(w13), s13.cuda(), wide(w2), s2.cuda(), groups.cuda(), out=dict(y=y))
    a, b = weight(w13, s13), weight(w2, s2)
    for e, lo, hi in ((1, 0, 20), (0, 25, 45)):
        want, bound = net(x[lo:hi].double(), a[e, 0], a[e, 1], b[e])
        assert_close(y[lo:hi], want, bound + want.abs() * 2.0**-22)
    assert (y[20:25] == 7.0).all() and (y[45:] == 7.0).all()


# ---------------------------------------------------------------------------
# Streams, graphs, workspaces, the same bits
# ---------------------------------------------------------------------------

SIZES = [(1, 1, 2048, 4096, I8, BF16), (8, 3, 500, 2500, F16, F32), (576, 16, 512, 700, I8, BF16), (600, 3, 700, 2300, BF16, F32)]


def a_case(rows, experts, N, K, x_dtype, seed):
    x, xs, values = rows_of(rows, K, x_dtype, seed)
    w, ws = weights_of((experts,), N, K, seed + 1)
    groups = groups_of(rows, experts, seed + 2)[0]
    want, bound = expected(values, groups, lambda e, v: product(v, weight(w, ws)[e]), N)
    return (x, wide(w), ws.cuda(), groups.cuda()), dict(x_scales=xs), want, bound + want.abs() * 2.0**-22


@pytest.mark.parametrize("size", SIZES)
def test_the_same_bits_twice(usc, size):
    args, kw, _, _ = a_case(*size[:5], 5)
    first = usc.moe_grouped_matmul_int8(*args, **kw, out_dtype=size[5])["y"]
    for _ in range(20):
        assert torch.equal(usc.moe_grouped_matmul_int8(*args, **kw, out_dtype=size[5])["y"], first)


@pytest.mark.parametrize("size", SIZES)
def test_a_workspace_that_holds_anything(usc, size):
    rows, experts, N, K, x_dtype, out = size
    args, kw, want, bound = a_case(rows, experts, N, K, x_dtype, 6)
    dt = {I8: usc.DT_INT8, F16: usc.DT_F16, BF16: usc.DT_BF16}[x_dtype]
    n = usc.grouped_matmul_int8_workspace_size(rows, experts, N, K, dt)
    for fill in (0, 255, 1):
        wsp = torch.full((max(n, 1),), fill, dtype=torch.uint8, device="cuda")
        assert_close(usc.moe_grouped_matmul_int8(*args, **kw, out_dtype=out, workspace=wsp)["y"], want, bound)
    if n:
        with pytest.raises(usc.MoeReorderError):
            usc.moe_grouped_matmul_int8(*args, **kw, out_dtype=out, workspace=wsp[:n - 1].clone())


@pytest.mark.parametrize("size", SIZES)
def test_captured_and_replayed(usc, size):
    rows, experts, N, K, x_dtype, out = size
    args, kw, want, bound = a_case(rows, experts, N, K, x_dtype, 7)
    o = usc.moe_grouped_matmul_int8(*args, **kw, out_dtype=out)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        usc.moe_grouped_matmul_int8(*args, **kw, out=o)
    for seed in (8, 9):
        others, kw2, want, bound = a_case(rows, experts, N, K, x_dtype, seed)
        for t, u in zip((*args, kw["x_scales"]), (*others, kw2["x_scales"])):
            if t is not None:
                t.copy_(u)
        o["y"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert_close(o["y"], want, bound)


def test_two_streams_at_once(usc):
    cases = [a_case(*size[:5], 20 + i) for i, size in enumerate(SIZES)]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        got = [usc.moe_grouped_matmul_int8(*c[0], **c[1], out_dtype=size[5], stream=s)["y"]
               for c, size, s in zip(cases, SIZES, streams)]
    torch.cuda.synchronize()
    for y, c in zip(got, cases):
        assert_close(y, c[2], c[3])


def test_ffn_captured(usc):
    rows, E, H, inter = 70, 3, 2100, 264
    x, xs, values = rows_of(rows, H, I8, 30)
    w13, s13 = weights_of((E, 2), inter, H, 31)
    w2, s2 = weights_of((E,), H, inter, 32)
    groups = groups_of(rows, E, 33)[0]
    args = (x, wide(w13), s13.cuda(), wide(w2), s2.cuda(), groups.cuda())
    for cut in (20, 70):  # few rows share tiles
        o = usc.moe_expert_ffn_int8(x[:cut], *args[1:], x_scales=xs[:cut])
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            usc.moe_expert_ffn_int8(x[:cut], *args[1:], x_scales=xs[:cut], out=o)
        o["y"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        a, b = weight(w13, s13), weight(w2, s2)
        want, bound = expected(values[:cut], groups, lambda e, v: net(v, a[e, 0], a[e, 1], b[e]), H)
        assert_close(o["y"], want, bound + want.abs() * 2.0**-22)


# ---------------------------------------------------------------------------
# Large operands
# ---------------------------------------------------------------------------

def test_results_past_32_bits(usc):
    """A result of more than 2^31 values, weights of more than 2^32 bytes: the last rows, experts and channels."""
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 64 GB")
    rows, N, K = 150_000, 16_000, 32
    x, xs, values = rows_of(rows, K, I8, 40)
    w, ws = weights_of((1,), N, K, 41)
    y = usc.moe_grouped_matmul_int8(x, wide(w), ws.cuda(), x_scales=xs)["y"]
    for rs in (slice(0, 3), slice(rows - 300, rows)):
        assert_close(y[rs, -300:], *product(values[rs], weight(w, ws)[0][-300:]))
    del y
    E, N, K = 40, 16_000, 8192
    w = torch.zeros(E, N, K, dtype=I8, device="cuda")
    assert w.numel() > 1 << 32
    tail, ws = weights_of((1,), N, K, 42)
    w[-1] = tail[0].cuda()
    scales = torch.ones(E, N, device="cuda")
    scales[-1] = ws[0].cuda()
    for rows in (3, 200):
        x, xs, values = rows_of(rows, K, I8, 43)
        g = torch.tensor([[E - 1, rows]], dtype=torch.int64, device="cuda")
        y = usc.moe_grouped_matmul_int8(x, w, scales, g, x_scales=xs)["y"]
        assert_close(y, *product(values, weight(tail, ws)[0]))


@pytest.mark.parametrize("x_dtype", [I8, BF16])
def test_groups_of_few_and_many_rows_in_turn(usc, x_dtype):
    """A block's tiles have their sums in halves of their room, or in all of it."""
    sizes = [5, 90, 17, 33, 48, 49, 1, 96, 16, 97, 2, 64] * 4
    g = torch.tensor([[i % 3, c] for i, c in enumerate(sizes)], dtype=torch.int64)
    check_matmul(usc, sum(sizes), 3, 1500, 200, x_dtype, BF16, 9, g)
    check_ffn(usc, sum(sizes), 3, 520, 300, x_dtype, seed=10, groups=g)


@pytest.mark.parametrize("x_dtype,out", [(I8, F32), (F16, BF16), (BF16, F32)])
def test_more_tiles_than_sms_of_long_rows(usc, x_dtype, out):
    for experts, per, N in ((40, 8, 1500), (34, 70, 1300), (170, 2, 700), (3, 60, 4000)):
        g = torch.tensor([[i % 3, max(0, per - i % 5)] for i in range(experts)], dtype=torch.int64)
        check_matmul(usc, int(g[:, 1].sum()), 3, N, 2100, x_dtype, out, experts, g)
    g = torch.tensor([[i % 3, 1 + i % 14] for i in range(40)], dtype=torch.int64)
    check_ffn(usc, int(g[:, 1].sum()), 3, 2100, 2000, x_dtype, seed=3, groups=g)
