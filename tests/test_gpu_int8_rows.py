"""moe_quantize_int8 and moe_add_rms_norm against their definitions, bit for bit."""
import pytest
import torch

from _int8_util import e4m3_rows, int8_rows, norm

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
COLS = [1, 7, 64, 100, 129, 256, 257, 500, 513, 1000, 1024, 1025, 2048, 2050, 2500, 4096, 4097, 7168, 8192, 9001, 16384, 16392, 20001]


@pytest.fixture(scope="module")
def usc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import unpermute_stable_counting_gb300 as u
    return u


def rows_of(rows, cols, dtype, seed, pad=0, start=0):
    """Rows with a few large channels, in a buffer where they start `start` elements in, `pad` apart."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cols, generator=g)
    v[:, :: max(1, cols // 5)] *= 8.0
    buf = torch.zeros(start + rows * (cols + pad), dtype=dtype)
    t = buf[start:].view(rows, cols + pad)[:, :cols]
    t.copy_(v)
    return t


def on_gpu(t):
    """t on the GPU with its strides and its place in its buffer."""
    if t is None:
        return None
    whole = torch.empty(0, dtype=t.dtype).set_(t.untyped_storage()).cuda()
    return whole.as_strided(t.shape, t.stride(), t.storage_offset())


def same(got, want):
    got = got.cpu()
    assert got.shape == want.shape and got.dtype == want.dtype
    if got.dtype.is_floating_point:
        nan = torch.isnan(want.float())
        assert torch.equal(torch.isnan(got.float()), nan)
        got, want = got.float().masked_fill(nan, 0.0), want.float().masked_fill(nan, 0.0)
    assert torch.equal(got, want), f"{int((got != want).sum())} of {got.numel()} values differ"


def check_int8(usc, x, **kw):
    r = usc.moe_quantize_int8(on_gpu(x), **kw)
    q, s = int8_rows(x.float())
    same(r["values"], q)
    same(r["scales"], s)
    return r


def check_norm(usc, x, w, residual, quantize, eps=1e-6, **kw):
    r = usc.moe_add_rms_norm(on_gpu(x), on_gpu(w), on_gpu(residual), eps=eps, quantize=quantize, **kw)
    h, y = norm(x, residual, w, eps)
    if residual is not None:
        same(r["residual"], h)
    else:
        assert "residual" not in r
    if kw.get("with_y", True):
        same(r["y"], y.to(x.dtype))
    if quantize:
        q, s = int8_rows(y) if quantize == "int8" else e4m3_rows(y)
        same(r["values"], q) if quantize == "int8" else same(r["values"].float(), q.float())
        same(r["scales"], s)
    return r


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_quantize_sizes(usc, cols, dtype):
    for rows, pad, start in ((1, 0, 0), (5, 0, 0), (13, 3, 1)):
        check_int8(usc, rows_of(rows, cols, dtype, cols + rows, pad, start))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_norm_sizes(usc, cols, dtype):
    for k, (quantize, residual, pad, start) in enumerate([("int8", True, 0, 0), ("e4m3", True, 5, 3), (None, False, 0, 0),
                                                          ("int8", False, 1, 1), ("e4m3", False, 8, 0)]):
        rows = (1, 9, 4, 17, 3)[k]
        x = rows_of(rows, cols, dtype, cols + k, pad, start)
        res = rows_of(rows, cols, dtype, cols + k + 50, 0, 0) if residual else None
        w = rows_of(1, cols, F32 if k == 3 else dtype, cols + 99)[0]
        check_norm(usc, x, w, res, quantize)


def test_many_rows(usc):
    check_int8(usc, rows_of(3001, 513, BF16, 1))
    check_norm(usc, rows_of(2049, 1000, F16, 2), rows_of(1, 1000, F16, 3)[0], rows_of(2049, 1000, F16, 4), "int8")
    check_norm(usc, rows_of(700, 7168, BF16, 2), rows_of(1, 7168, BF16, 3)[0], rows_of(700, 7168, BF16, 4), "e4m3")


def test_no_rows(usc):
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    assert usc.moe_quantize_int8(x)["values"].shape == (0, 64)
    w = torch.ones(64, dtype=BF16, device="cuda")
    r = usc.moe_add_rms_norm(x, w, x, quantize="e4m3")
    assert r["y"].shape == (0, 64) and r["scales"].shape == (0, 1)
    assert usc.moe_quantize_int8(torch.empty(0, 3, 64, dtype=BF16, device="cuda"))["scales"].shape == (0, 3)


@pytest.mark.parametrize("cols", [40, 2000, 20001])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_unusual_values(usc, dtype, cols):
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).tiny
    x = rows_of(12, cols, dtype, 5)
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, cols - 1] = float("nan")
    x[3] = big
    x[4, 5] = -big
    x[5] = tiny
    x[6] = -0.0
    x[7] = 0.0
    x[7, 1] = tiny
    x[8, 2], x[8, 4] = float("inf"), float("-inf")
    x[9] = torch.finfo(dtype).smallest_normal / 2  # subnormal
    x[10] = x[10].sign()  # every value at the maximum
    check_int8(usc, x)
    w = rows_of(1, cols, dtype, 6)[0]
    for quantize in ("int8", "e4m3"):
        check_norm(usc, x, w, None, quantize)
        check_norm(usc, x, w, rows_of(12, cols, dtype, 7), quantize)


@pytest.mark.parametrize("eps", [2.0**-100, 1e-30, 1e-5, 0.1, 1e6])
def test_eps(usc, eps):
    x = rows_of(6, 777, F32, 8) * torch.tensor([1.0, 1e-3, 1e-9, 1e3, 1e9, 1e-12])[:, None]
    check_norm(usc, x, rows_of(1, 777, F32, 9)[0], None, "int8", eps=eps)


def test_rows_in_use(usc):
    x, n = rows_of(10, 300, BF16, 10), torch.tensor([7], device="cuda")
    out = dict(values=torch.full((10, 304), 77, dtype=torch.int8, device="cuda")[:, :300],
               scales=torch.full((10,), 9.0, device="cuda"))
    usc.moe_quantize_int8(on_gpu(x), num_rows=n, out=out)
    q, s = int8_rows(x.float())
    same(out["values"][:7], q[:7])
    assert (out["values"][7:] == 77).all() and (out["scales"][7:] == 9.0).all()
    assert (out["values"].as_strided((10, 4), (304, 1), 300) == 77).all()
    w = torch.ones(300, dtype=BF16, device="cuda")
    for count in (0, 4, 10, 12, -3):
        o = dict(residual=torch.full((10, 300), 5.0, dtype=BF16, device="cuda"),
                 y=torch.full((10, 300), 5.0, dtype=BF16, device="cuda"))
        usc.moe_add_rms_norm(on_gpu(x), w, on_gpu(x), num_rows=torch.tensor([count], device="cuda"), out=o)
        k = min(10, max(0, count))
        assert (o["y"][k:] == 5.0).all() and (o["residual"][k:] == 5.0).all()
        h, y = norm(x, x, w.cpu(), 1e-6)
        same(o["y"][:k], y.to(BF16)[:k])


@pytest.mark.parametrize("cols", [36, 1000, 7168, 20004])
def test_interleaved(usc, cols):
    x = rows_of(9, cols, BF16, 11)
    r = check_int8(usc, x, interleaved=True)
    raw = r["rows"].cpu()
    assert raw.shape == (9, cols + 4)
    q, s = int8_rows(x.float())
    assert torch.equal(raw[:, :cols], q) and torch.equal(raw[:, cols:].contiguous().view(F32)[:, 0], s)
    r = check_norm(usc, x, rows_of(1, cols, BF16, 12)[0], None, "int8", interleaved=True, with_y=False)
    assert r["rows"].shape == (9, cols + 4) and "y" not in r


@pytest.mark.parametrize("cols,dtype", [(1000, BF16), (1001, BF16), (8192, F16), (20001, BF16), (999, F32)])
def test_residual_in_place(usc, cols, dtype):
    x, res, w = rows_of(11, cols, dtype, 13), rows_of(11, cols, dtype, 14), rows_of(1, cols, dtype, 15)[0]
    h, y = norm(x, res, w, 1e-6)
    for which in (0, 1):
        t = [on_gpu(x), on_gpu(res)]
        out = dict(residual=t[1 - which], y=torch.empty(11, cols, dtype=dtype, device="cuda"))
        usc.moe_add_rms_norm(t[0], w.cuda(), t[1], out=out)
        same(t[1 - which], h)
        same(t[which], (x, res)[which])
        same(out["y"], y.to(dtype))


def test_outputs_keep_their_surroundings(usc):
    """Rows of outputs that start anywhere, with other data on either side."""
    cols, rows = 1001, 6
    x, res, w = rows_of(rows, cols, BF16, 16, 2, 5), rows_of(rows, cols, BF16, 17), rows_of(1, cols, BF16, 18)[0]
    for start, pad in ((0, 1), (1, 3), (3, 6), (7, 0)):
        bufs = {k: torch.full((start + rows * (cols + pad) + 9,), 3, dtype=d, device="cuda")
                for k, d in (("y", BF16), ("residual", BF16), ("values", torch.int8))}
        out = {k: b.as_strided((rows, cols), (cols + pad, 1), start) for k, b in bufs.items()}
        out["scales"] = torch.empty(rows, device="cuda")
        usc.moe_add_rms_norm(on_gpu(x), w.cuda(), on_gpu(res), quantize="int8", out=out)
        h, y = norm(x, res, w, 1e-6)
        for k, v in (("y", y.to(BF16)), ("residual", h), ("values", int8_rows(y)[0])):
            want = torch.full(bufs[k].shape, 3, dtype=bufs[k].dtype)
            want.as_strided((rows, cols), (cols + pad, 1), start).copy_(v)
            same(bufs[k], want)


def test_weights_of_several_matrices(usc):
    x = rows_of(2 * 3 * 40, 100, F16, 19).view(2, 3, 40, 100)
    check_int8(usc, x)
    apart = torch.zeros(5, 2, 40, 104, dtype=F16)  # matrices and rows with room behind them
    view = apart[:, :, :33, :100]
    view.copy_(torch.randn(5, 2, 33, 100))
    check_int8(usc, view[:, 0])
    r = usc.moe_quantize_int8(apart.cuda()[:, 0, :33, :100])
    same(r["scales"], int8_rows(view[:, 0].float())[1])


def test_expanded_rows(usc):
    x = rows_of(1, 500, BF16, 20).expand(4, 500)
    r = usc.moe_quantize_int8(x.contiguous()[:1].cuda().expand(4, 500))
    same(r["values"], int8_rows(x.float())[0])


def test_captured_and_replayed(usc):
    x, res = rows_of(33, 1000, BF16, 21).cuda(), rows_of(33, 1000, BF16, 22).cuda()
    w = rows_of(1, 1000, BF16, 23)[0].cuda()
    out = usc.moe_add_rms_norm(x, w, res, quantize="int8")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        usc.moe_add_rms_norm(x, w, res, quantize="int8", out=out)
        q = usc.moe_quantize_int8(out["y"])
    for seed in (30, 31):
        x.copy_(rows_of(33, 1000, BF16, seed))
        graph.replay()
        torch.cuda.synchronize()
        h, y = norm(x.cpu(), res.cpu(), w.cpu(), 1e-6)
        same(out["residual"], h)
        same(out["values"], int8_rows(y)[0])
        same(q["values"], int8_rows(y.to(BF16).float())[0])


def test_another_stream(usc):
    x, w = rows_of(50, 640, BF16, 24), rows_of(1, 640, BF16, 25)[0]
    s = torch.cuda.Stream()
    gx, gw = x.cuda(), w.cuda()
    s.wait_stream(torch.cuda.current_stream())
    a = usc.moe_add_rms_norm(gx, gw, quantize="e4m3", stream=s)
    b = usc.moe_quantize_int8(gx, stream=s)
    s.synchronize()
    y = norm(x, None, w, 1e-6)[1]
    same(a["values"].float(), e4m3_rows(y)[0].float())
    same(b["values"], int8_rows(x.float())[0])


def test_norm_to_the_e4m3_product(usc):
    """The norm's e4m3 rows are the product's input as they are."""
    x, w = rows_of(40, 520, BF16, 26), rows_of(1, 520, BF16, 27)[0]
    r = usc.moe_add_rms_norm(x.cuda(), w.cuda(), quantize="e4m3", with_y=False)
    wt = usc.moe_quantize(torch.randn(1, 256, 520, device="cuda", dtype=BF16), block_rows=128)
    y = usc.moe_grouped_matmul(r["values"], wt["values"], wt["scales"], x_scales=r["scales"], out_dtype=F32)["y"]
    q, s = e4m3_rows(norm(x, None, w, 1e-6)[1])
    xd = q.double() * s.double().repeat_interleave(128, 1)[:, :520]
    ws = wt["scales"].cpu().double().repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :256, :520]
    want = xd @ (wt["values"].cpu().float().double() * ws)[0].T
    assert ((y.cpu().double() - want).norm() / want.norm()).item() < 1e-6
