"""The INT8 operators in their place: norm -> batching's INT8 mode -> experts ->
unpermute, and their suites on the bounds-checked builds."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import unpermute_stable_counting_gb300 as usc  # noqa: E402

from _expert_util import assert_close  # noqa: E402
from _int8_util import int8_rows, net, norm, weight  # noqa: E402
from test_gpu_few_sms import run_suites  # noqa: E402

SUITES = ["test_gpu_int8_rows.py", "test_gpu_int8_products.py"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("tokens,topk,experts,H,inter", [(1, 2, 4, 128, 64), (40, 3, 8, 256, 136), (300, 2, 6, 192, 100)])
def test_norm_batching_experts_unpermute(tokens, topk, experts, H, inter):
    g = torch.Generator().manual_seed(tokens)
    x, res = (torch.randn(tokens, H, generator=g).to(torch.bfloat16) for _ in range(2))
    gamma = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16)
    w13 = (torch.randn(experts, 2, inter, H, generator=g) / H**0.5).to(torch.bfloat16)
    w2 = (torch.randn(experts, H, inter, generator=g) / inter**0.5).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(experts, generator=g)[:topk] for _ in range(tokens)]).to(torch.int32)
    ids[torch.rand(tokens, topk, generator=g) < 0.2] = 2**31 - 1  # masked slots
    # the attention side: norm, rows with their scale behind them, one copy for each slot
    rows = usc.moe_add_rms_norm(x.cuda(), gamma.cuda(), res.cuda(), quantize="int8", interleaved=True, with_y=False)
    slots = rows["rows"].repeat_interleave(topk, 0).contiguous()
    zero = torch.zeros(tokens * topk, dtype=torch.int32, device="cuda")
    out = usc.ffnwb_batching(ids.flatten().cuda(), slots, zero, zero, expert_num=experts, max_out_shape=(1, tokens, topk, H),
                             token_dtype=usc.DT_INT8, with_sorted_indices=True)
    # the workers
    q13, q2 = usc.moe_quantize_int8(w13.cuda()), usc.moe_quantize_int8(w2.cuda())
    y = torch.zeros(tokens * topk, H, device="cuda")
    usc.moe_expert_ffn_int8(out["y"], q13["values"], q13["scales"], q2["values"], q2["scales"], out["groupList"],
                            x_scales=out["dynamicScale"], num_rows=out["actualTokenNum"], out=dict(y=y))
    back = usc.moe_unpermute(y, out["sortedIndices"], restore_shape=(tokens, H))["unpermutedTokens"].cpu()
    # the same from the definitions
    h, n = norm(x, res, gamma, 1e-6)
    assert torch.equal(rows["residual"].cpu(), h)
    q, s = int8_rows(n)
    values = q.double() * s.double()[:, None]
    a, b = (weight(*int8_rows(w.float())) for w in (w13, w2))
    want, bound = (torch.zeros(tokens, H, dtype=torch.float64) for _ in range(2))
    for t in range(tokens):
        for e in ids[t].tolist():
            if e < experts:
                v, d = net(values[t:t + 1], a[e, 0], a[e, 1], b[e])
                want[t] += v[0]
                bound[t] += d[0] + v[0].abs() * 2.0**-20
    assert_close(back, want, bound)


def test_suites_on_the_checked_build():
    from unpermute_stable_counting_gb300 import _build, _native
    if _native.checked_requested():
        pytest.skip("this process runs against another build")
    _build.build_library(checked=True)
    run_suites(SUITES, USC_CHECKED="1")


def test_suites_on_few_sms():
    from unpermute_stable_counting_gb300 import _build, _native
    if _native.checked_requested():
        pytest.skip("this process runs against another build")
    _build.build_library(few_sms=True)
    run_suites(SUITES, USC_CHECKED="1", USC_FEW_SMS="1")
