"""Long sums of moe_grouped_matmul_int8 and moe_expert_ffn_int8: values of one sign, whose sums
leave what one fp32 sum of the tensor cores holds."""
import pytest
import torch

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


def rows_on_16(*shape):
    """int8 on the GPU with rows that start on 16 bytes."""
    cols = shape[-1]
    return torch.zeros(*shape[:-1], -(-cols // 16) * 16, dtype=I8, device="cuda")[..., :cols]


def one_sign(shape, seed, low=100, high=128):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = rows_on_16(*shape)
    t.copy_(torch.randint(low, high, shape, device="cuda", generator=g, dtype=torch.int16).to(I8))
    return t


def scales(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, device="cuda", generator=g) + 0.5


def a_list(rows, groups):
    """[groups, 2] of ragged counts, experts in descending order."""
    cut = [rows * (i * i + 1) // (groups * groups + 1) for i in range(groups)] + [rows]
    cut[0] = 0
    return torch.tensor([[groups - 1 - i, cut[i + 1] - cut[i]] for i in range(groups)], dtype=torch.int64)


def exact_sums(x, w, groups):
    """float64 of the integer sums (all below 2^53)."""
    parts, at = [], 0
    for e, c in groups.tolist():
        parts.append(x[at:at + c].double() @ w[e].double().T)
        at += c
    return torch.cat(parts)


# few rows, whose tiles blocks share (the first four); single blocks with tiles of their own; pairs of blocks
INT8_SIZES = [(1, 1, 2048, 4096), (4, 1, 130, 131071), (20, 3, 300, 7168), (32, 2, 513, 2049),
              (200, 20, 2000, 1100), (200, 20, 2000, 7168), (40, 1, 130, 131071), (100, 1, 256, 1041), (300, 3, 700, 7167)]


@pytest.mark.parametrize("rows,experts,N,K", INT8_SIZES)
def test_fp32_results_of_int8_rows_past_24_bits(usc, rows, experts, N, K):
    """Sums of at most 1024 values are exact (at most 2^24) and are added in fp32, where blocks share a tile by
    shares of at least four loads of 128; then two scales. Sums below 2^24 are exact: equal bits."""
    x, w = one_sign((rows, K), rows), one_sign((experts, N, K), rows + 1)
    xs, ws, groups = scales((rows,), 3), scales((experts, N), 4), a_list(rows, experts)
    sums = exact_sums(x, w, groups)
    assert K < 1500 or sums.max() > 2**24
    experts_of = torch.repeat_interleave(groups[:, 0], groups[:, 1]).cuda()
    want = sums.float() * ws[experts_of] * xs[:, None]
    for _ in range(3):
        y = usc.moe_grouped_matmul_int8(x, w, ws, groups.cuda(), x_scales=xs, out_dtype=F32)["y"]
        if K < 1500:
            assert torch.equal(y, want)
        else:
            exact = sums * ws.double()[experts_of] * xs.double()[:, None]
            assert ((y.double() - exact).abs() <= (K // 512 + 4) * 2.0**-24 * exact).all()


@pytest.mark.parametrize("rows", [3, 90])
@pytest.mark.parametrize("K", [1024, 1025, 1041])
def test_fp32_results_next_to_24_bits(usc, rows, K):
    """1024 products of -128 and -128 are 2^24, and 1041 of 127 and 127 are past it."""
    x, w = rows_on_16(rows, K), rows_on_16(1, 300, K)
    x.fill_(127)
    w.fill_(127)
    x[0] = -128
    w[0, 0] = -128
    w[0, 1, ::2] = -127
    groups = torch.tensor([[0, rows]])
    one = torch.ones(rows, device="cuda")
    y = usc.moe_grouped_matmul_int8(x, w, torch.ones(1, 300, device="cuda"), x_scales=one, out_dtype=F32)["y"]
    assert torch.equal(y, exact_sums(x, w, groups).float())


@pytest.mark.parametrize("rows", [3, 90])
def test_fp32_results_at_the_ends_of_32_bits(usc, rows):
    """131071 products of -128 and -128 stay below 2^31, and of -128 and 127 above -2^31."""
    x, w = rows_on_16(rows, 131071), rows_on_16(1, 70, 131071)
    x.fill_(-128)
    w.fill_(-128)
    w[0, ::2] = 127
    one = torch.ones(rows, device="cuda")
    y = usc.moe_grouped_matmul_int8(x, w, torch.ones(1, 70, device="cuda"), x_scales=one, out_dtype=F32)["y"]
    assert torch.equal(y[0], exact_sums(x[:1], w, torch.tensor([[0, 1]]))[0].float()) and (y == y[0]).all()


@pytest.mark.parametrize("rows", [2, 50])
@pytest.mark.parametrize("K", [1 << 17, (1 << 18) + 40])
def test_fp32_results_past_32_bits(usc, rows, K):
    """Sums of 1024 values are exact (at most 2^24), and are added in fp32: one rounding for each sum, and at
    most as many again where blocks share a tile; two for the scales."""
    x, w = one_sign((rows, K), 5), one_sign((1, 66, K), 6)
    xs, ws = scales((rows,), 7), scales((1, 66), 8)
    y = usc.moe_grouped_matmul_int8(x, w, ws, x_scales=xs, out_dtype=F32)["y"].double()
    want = exact_sums(x, w, torch.tensor([[0, rows]])) * ws.double() * xs.double()[:, None]
    assert ((y - want).abs() <= (2 * (K // 1024 + 1) + 2) * 2.0**-24 * want).all()


@pytest.mark.parametrize("rows", [4, 100])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_fp32_results_of_16_bit_rows(usc, dtype, rows):
    """Sums of at most 1024 values, each addition off by at most 2^-23 of what is there, then three roundings
    for each sum. (One sum of all values loses 7.6e-4 here, five times the bound.)"""
    K, N = 131072, 130
    g = torch.Generator(device="cuda").manual_seed(9)
    x = (torch.rand(rows, K, device="cuda", generator=g) + 0.5).to(dtype)
    w, ws = one_sign((1, N, K), 10), scales((1, N), 11) / K
    y = usc.moe_grouped_matmul_int8(x, w, ws, out_dtype=F32)["y"].double()
    want = exact_sums(x, w, torch.tensor([[0, rows]])) * ws.double()
    assert ((y - want).abs() <= (1024 * 2.0**-23 + (K // 1024 + 2) * 2.0**-24) * want).all()


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("K", [2100, 20000])
@pytest.mark.parametrize("rows,experts", [(9, 1), (200, 100), (300, 1)])
def test_results_of_several_sums_keep_their_surroundings(usc, rows, experts, K, out):
    """Results that start anywhere, groups of experts that are not there, rows behind the last group."""
    N = 133
    x, w = one_sign((rows, K), 1, -127, 128), one_sign((2, N, K), 2, -127, 128)
    xs, ws = scales((rows,), 3), scales((2, N), 4)
    each = (rows - 3) // experts
    groups = torch.tensor([[9 if i % 5 == 4 else i % 2, each] for i in range(experts)], dtype=torch.int64)
    used = each * experts
    e = torch.repeat_interleave(groups[:, 0], groups[:, 1]).cuda()
    both = torch.stack([x[:used].double() @ w[i].double().T for i in range(2)])
    there = e < 2
    sums = both[e.clamp_max(1), torch.arange(used, device="cuda")]
    assert sums.abs().max() < 2**23
    want = (sums.float() * ws[e.clamp_max(1)] * xs[:used, None]).to(out)
    for start, pad in ((0, 0), (1, 3), (5, 11)):
        buf = torch.full((start + rows * (N + pad) + 7,), 3.0, dtype=out, device="cuda")
        y = buf.as_strided((rows, N), (N + pad, 1), start)
        usc.moe_grouped_matmul_int8(x, w, ws, groups.cuda(), x_scales=xs, out=dict(y=y))
        got = y[:used][there]
        assert torch.equal(got, want[there])  # (signs differ: no sum on the way leaves 24 bits)
        y[:used][there] = 3.0
        assert (y == 3.0).all()
        y.fill_(3.0)
        assert (buf == 3.0).all()
