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
