"""Calls none of whose products share tiles leave the workspace's tickets alone (no launch clears them)."""
import pytest
import torch

from test_gpu_int8_products import BF16, F16, F32, I8, a_case, usc, weights_of, wide  # noqa: F401

pytestmark = pytest.mark.gpu


def untouched(size):
    return torch.full((size,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("x_dtype", [F16, BF16])
@pytest.mark.parametrize("rows,experts,N,K", [(1, 1, 2048, 4096), (30, 2, 300, 2000)])
def test_fp32_results_of_16_bit_rows(usc, rows, experts, N, K, x_dtype):
    args, kw, _, _ = a_case(rows, experts, N, K, x_dtype, 1)
    n = usc.grouped_matmul_int8_workspace_size(rows, experts, N, K, usc.DT_F16 if x_dtype == F16 else usc.DT_BF16)
    wsp = untouched(n)
    first = usc.moe_grouped_matmul_int8(*args, **kw, out_dtype=F32)["y"]
    assert n and torch.equal(usc.moe_grouped_matmul_int8(*args, **kw, out_dtype=F32, workspace=wsp)["y"], first)
    assert (wsp == 255).all()


@pytest.mark.parametrize("H,shares", [(1000, False), (2048, True)])
def test_fp32_results_of_the_network(usc, H, shares):
    """The second product has no shares, the first one those of long rows."""
    rows, inter = 4, 2048
    x = torch.randn(rows, H).to(BF16)
    (w13, s13), (w2, s2) = weights_of((1, 2), inter, H, 1), weights_of((1,), H, inter, 2)
    args = (wide(x), wide(w13), s13.cuda(), wide(w2), s2.cuda())
    n = usc.expert_ffn_int8_workspace_size(rows, -1, H, inter, usc.DT_BF16)
    wsp, h = untouched(n), rows * inter * 2
    first = usc.moe_expert_ffn_int8(*args, out_dtype=F32)["y"]
    assert torch.equal(usc.moe_expert_ffn_int8(*args, out_dtype=F32, workspace=wsp)["y"], first)
    assert n > h and bool((wsp[h:] == 255).all()) != shares
