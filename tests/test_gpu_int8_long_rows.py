"""16-bit results and the network's h of rows of more than 16384 values, of one sign: one sum of all of them
would lose more than a result's rounding."""
import pytest
import torch

from test_gpu_int8_sums import BF16, F16, I8, _no_wait_ran_out, exact_sums, one_sign, scales, usc  # noqa: F401

pytestmark = pytest.mark.gpu

HALF_STEP = {BF16: 2.0**-8, F16: 2.0**-11}
# each sum takes at most 16384 values, each addition off by at most 2^-23 of what is there; then the sums of a row of
# 2^20 values are added (128 additions at most, a shared tile's among them), scaled twice and rounded to the result's type
SUM = 16384 * 2.0**-23 + 130 * 2.0**-24


def rows_of(rows, K, dtype, seed):
    if dtype == I8:
        return one_sign((rows, K), seed), scales((rows,), seed + 1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(rows, -(-K // 8) * 8, device="cuda", dtype=dtype)[:, :K]  # rows that start on 16 bytes
    x.copy_(torch.rand(rows, K, device="cuda", generator=g) + 0.5)
    return x, None


def values(x, xs):
    return x.double() if xs is None else x.double() * xs.double()[:, None]


@pytest.mark.parametrize("x_dtype", [I8, F16, BF16])
@pytest.mark.parametrize("rows,groups,N", [(3, 1, 70), (100, 1, 130), (200, 100, 300)])
def test_16_bit_results(usc, rows, groups, N, x_dtype):
    """Blocks that share a tile, pairs, single blocks with several tiles."""
    K = 1 << 20
    x, xs = rows_of(rows, K, x_dtype, rows)
    w, ws = one_sign((1, N, K), 3), scales((1, N), 4) / (64.0 * K)
    each = rows // groups
    lists = torch.tensor([[0, each]] * groups, device="cuda")
    want = torch.cat([values(x[i:i + 20], None if xs is None else xs[i:i + 20]) @ w[0].double().T for i in range(0, rows, 20)])
    want *= ws.double()
    for out in (F16, BF16):
        y = usc.moe_grouped_matmul_int8(x, w, ws, lists, x_scales=xs, out_dtype=out)["y"].double()
        assert ((y - want).abs() <= (SUM + HALF_STEP[out]) * want).all()


@pytest.mark.parametrize("x_dtype", [I8, F16, BF16])
@pytest.mark.parametrize("K", [16384, 16385, 18432, 53248])
@pytest.mark.parametrize("rows", [5, 60])
def test_lengths_next_to_the_border(usc, rows, K, x_dtype):
    x, xs = rows_of(rows, K, x_dtype, rows)
    w, ws = one_sign((2, 131, K), 3, -127, 128), scales((2, 131), 4) / (64.0 * K)
    lists = torch.tensor([[1, rows - 2], [0, 2]])
    want = exact_sums(x, w, lists) * ws.double()[lists[:, 0].repeat_interleave(lists[:, 1]).cuda()]
    size = exact_sums(x.abs(), w.abs(), lists) * ws.double()[lists[:, 0].repeat_interleave(lists[:, 1]).cuda()]
    if xs is not None:
        want, size = want * xs.double()[:, None], size * xs.double()[:, None]
    for out in (F16, BF16):
        y = usc.moe_grouped_matmul_int8(x, w, ws, lists.cuda(), x_scales=xs, out_dtype=out)["y"].double()
        assert ((y - want).abs() <= SUM * size + HALF_STEP[out] * want.abs() + 2.0**-25).all()


@pytest.mark.parametrize("x_dtype", [I8, F16, BF16])
@pytest.mark.parametrize("rows,H,inter", [(3, 1 << 20, 70), (40, 1 << 20, 70), (3000, 16500, 700)])
def test_the_networks_first_product(usc, rows, H, inter, x_dtype):
    """g, u > 0 and w2 > 0: what a sum loses is lost by every h and by y."""
    x, xs = rows_of(rows, H, x_dtype, 5)
    w13 = one_sign((1, 2, inter, H), 6)
    s13 = scales((1, 2, inter), 7) / (64.0 * H) / (114.0 if x_dtype == I8 else 1.0)
    w2 = one_sign((1, H, inter), 8)
    s2 = torch.ones(1, H, device="cuda") / (64.0 * inter)
    y = usc.moe_expert_ffn_int8(x, w13, s13, w2, s2, x_scales=xs, out_dtype=F16)["y"].double()
    v = values(x, xs)
    g, u = ((v @ w13[0, j].double().T) * s13[0, j].double() for j in (0, 1))
    h = g * torch.sigmoid(g) * u
    # silu' < 1.1; silu in fp32 is off by a few 2^-23, of |g| 2^-23 in the exponent; h is rounded to bf16
    dh = (1.1 * SUM * g / (g * torch.sigmoid(g)) + SUM + (16 + g) * 2.0**-23) * (1 + SUM) * h + 2.0**-8 * h
    wd = w2[0].double() * s2[0].double()[:, None]
    want, bound = h @ wd.T, dh @ wd.T
    assert ((y - want).abs() <= bound * (1 + 1e-3) + want * (2.0**-11 + (inter + 10) * 2.0**-23)).all()


@pytest.mark.parametrize("out", [F16, BF16])
@pytest.mark.parametrize("rows,groups,N", [(600, 3, 7000), (300, 100, 700)])
def test_several_tiles_for_each_block(usc, rows, groups, N, out):
    """Pairs, single blocks: signs differ, no sum on the way leaves 24 bits, so that the bits are the integers'."""
    K = 16500
    x, w = one_sign((rows, K), 1, -127, 128), one_sign((2, N, K), 2, -127, 128)
    xs, ws = scales((rows,), 3) / 4096.0, scales((2, N), 4) / 4096.0
    lists = torch.tensor([[i % 2, rows // groups] for i in range(groups)])
    sums = exact_sums(x, w, lists)
    assert sums.abs().max() < 2**23
    want = (sums.float() * ws[lists[:, 0].repeat_interleave(lists[:, 1]).cuda()] * xs[:, None]).to(out)
    for _ in range(3):
        y = usc.moe_grouped_matmul_int8(x, w, ws, lists.cuda(), x_scales=xs, out_dtype=out)["y"]
        assert torch.equal(y, want)


@pytest.mark.parametrize("rows", [3, 100])
def test_a_workspace_that_holds_anything(usc, rows):
    K, N = 40000, 300
    x, xs = rows_of(rows, K, I8, 1)
    w, ws = one_sign((1, N, K), 3), scales((1, N), 4) / (64.0 * K)
    n = usc.grouped_matmul_int8_workspace_size(rows, -1, N, K, usc.DT_INT8)
    got = [usc.moe_grouped_matmul_int8(x, w, ws, x_scales=xs, workspace=torch.full((n,), fill, dtype=torch.uint8, device="cuda"))["y"]
           for fill in (0, 255)]
    assert n and torch.equal(got[0], got[1])
    want = exact_sums(x, w, torch.tensor([[0, rows]])) * ws.double() * xs.double()[:, None]
    assert ((got[0].double() - want).abs() <= (SUM + HALF_STEP[BF16]) * want).all()
