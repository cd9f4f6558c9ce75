"""moe_add_rms_norm where a row's squares pass fp32's range and eps still counts beside their mean, bit for bit."""
import pytest
import torch

from test_gpu_int8_rows import BF16, F32, check_norm, rows_of, usc  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [2.0**100, 1.7 * 2.0**99, 2.0**90])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,power", [(40, 63), (1000, 59), (1000, 60), (7168, 58), (20001, 57), (1 << 20, 54)])
def test_eps_beside_squares_past_the_range(usc, cols, power, dtype, eps):
    """The sum of squares is 2^128 at least (but for the second row), eps up to 2^-8 of their mean."""
    x = torch.ones(3, cols) * 2.0**power
    g = torch.Generator().manual_seed(cols)
    x *= 1.0 + torch.rand(3, cols, generator=g)
    x[1] *= 2.0**-20
    x[2, ::2] *= -1.0
    w = rows_of(1, cols, dtype, 9)[0]
    for quantize in ("int8", "e4m3"):
        check_norm(usc, x.to(dtype), w, None, quantize, eps=eps)
