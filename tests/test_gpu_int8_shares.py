"""Tiles that blocks share (few rows, long ones), for every type of rows and in both products of the
network: partial sums, tickets, the last block's sum, on workspaces that hold anything."""
import pytest
import torch

from _expert_util import assert_close, product
from _int8_util import net, weight
from test_gpu_int8_products import BF16, F16, F32, I8, _no_wait_ran_out, expected, groups_of, rows_of, usc, weights_of, wide  # noqa: F401

pytestmark = pytest.mark.gpu

DT = {I8: "DT_INT8", F16: "DT_F16", BF16: "DT_BF16"}


def on_workspaces(call, size):
    """call(workspace) on one of its own and, twice each, on ones of ones and of zeros: the same bits."""
    y = call(None)
    for fill in (255, 0):
        wsp = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            assert torch.equal(call(wsp), y)
    return y


@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("x_dtype", [I8, F16, BF16])
@pytest.mark.parametrize("rows,experts,N,K", [(1, 1, 2048, 4096), (20, 3, 520, 2100), (32, 2, 300, 4096), (9, 9, 130, 2100),
                                              (31, 1, 1, 4096), (16, 40, 60, 2100)])
def test_products(usc, rows, experts, N, K, x_dtype, out):
    x, xs, values = rows_of(rows, K, x_dtype, rows)
    w, ws = weights_of((experts,), N, K, 1)
    groups = groups_of(rows, experts, 2)[0]
    size = usc.grouped_matmul_int8_workspace_size(rows, experts, N, K, getattr(usc, DT[x_dtype]))
    assert size > 0
    dev = (x, wide(w), ws.cuda(), groups.cuda())
    y = on_workspaces(lambda wsp: usc.moe_grouped_matmul_int8(*dev, x_scales=xs, out_dtype=out, workspace=wsp)["y"], size)
    wd = weight(w, ws)
    want, bound = expected(values, groups, lambda e, v: product(v, wd[e]), N)
    assert_close(y, want, bound + want.abs() * 2.0**-22)


@pytest.mark.parametrize("x_dtype", [I8, F16, BF16])
@pytest.mark.parametrize("rows,experts", [(1, 1), (9, 2), (32, 1)])
@pytest.mark.parametrize("H,inter", [(2100, 2048), (264, 2048), (2100, 200)])
def test_networks(usc, H, inter, rows, experts, x_dtype):
    """Both products share tiles, the second one alone, the first one alone."""
    x, xs, values = rows_of(rows, H, x_dtype, rows)
    w13, s13 = weights_of((experts, 2), inter, H, 3)
    w2, s2 = weights_of((experts,), H, inter, 4)
    groups = groups_of(rows, experts, 5)[0]
    size = usc.expert_ffn_int8_workspace_size(rows, experts, H, inter, getattr(usc, DT[x_dtype]))
    assert size > 1 << 20  # (h alone is 128 KB)
    dev = (x, wide(w13), s13.cuda(), wide(w2), s2.cuda(), groups.cuda())
    a, b = weight(w13, s13), weight(w2, s2)
    want, bound = expected(values, groups, lambda e, v: net(v, a[e, 0], a[e, 1], b[e]), H)
    for out in (BF16, F32):
        y = on_workspaces(lambda wsp: usc.moe_expert_ffn_int8(*dev, x_scales=xs, out_dtype=out, workspace=wsp)["y"], size)
        assert_close(y, want, bound + want.abs() * 2.0**-22)


def test_a_workspace_for_calls_of_other_sizes(usc):
    """Tickets and sums of one call are not the next one's."""
    calls = []
    for rows, N, K, x_dtype in ((1, 2048, 4096, BF16), (20, 520, 2100, I8), (32, 300, 4096, F16)):
        x, xs, values = rows_of(rows, K, x_dtype, rows)
        w, ws = weights_of((1,), N, K, 1)
        calls.append(((x, wide(w), ws.cuda()), xs, *product(values, weight(w, ws)[0])))
    wsp = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    for args, xs, want, bound in calls * 3:
        y = usc.moe_grouped_matmul_int8(*args, x_scales=xs, workspace=wsp)["y"]
        assert_close(y, want, bound + want.abs() * 2.0**-22)
