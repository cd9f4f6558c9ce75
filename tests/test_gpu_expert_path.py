"""The expert operators in their place between batching / permute and
unpermute, and their suites on the bounds-checked build."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import unpermute_stable_counting_gb300 as usc  # noqa: E402
import workloads as w  # noqa: E402

import _expert_util as eu  # noqa: E402
from _gpu_util import run_batching  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import moe_step  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("tokens,experts,topk,hidden,inter", [(1, 8, 2, 256, 128), (40, 16, 4, 512, 192),
                                                              (64, 24, 3, 384, 136)])
def test_example_both_ways(tokens, experts, topk, hidden, inter):
    """permute -> experts -> unpermute, and the layer, against 64 bits."""
    wt = moe_step.make_weights(experts, hidden, inter, seed=tokens)
    x = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(tokens)).to(torch.bfloat16)
    xd = x.cuda()
    routed, layer = moe_step.routed_step(xd, wt, topk), moe_step.layer_step(xd, wt, topk)
    c = {k: v.cpu() for k, v in wt.items()}
    W13, W2 = eu.weight(c["w13"], c["w13_scales"]), eu.weight(c["w2"], c["w2_scales"])
    q, s = eu.quantize(x.double())
    xq = q * eu.spread(s, hidden)
    logits = x.double() @ c["router"].double().T
    ids = torch.argsort(logits, dim=-1, descending=True, stable=True)[:, :topk]
    p = torch.gather(torch.softmax(logits, -1), 1, ids)
    p = p / p.sum(1, keepdim=True)
    y, b, terms = (torch.zeros(tokens, hidden, dtype=torch.float64) for _ in range(3))
    for e in ids.unique().tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        ye, be = eu.net(xq[t], W13[e, 0], W13[e, 1], W2[e])
        y[t] += p[t, j][:, None] * ye
        b[t] += p[t, j][:, None] * be
        terms[t] += p[t, j][:, None] * ye.abs()
    # fp32 logits and weights: a few hundred units; the routed way also rounds each expert's rows to bf16
    slack = terms * 512 * 2.0**-23
    eu.assert_close(layer, y, b + slack)
    eu.assert_close(routed, y, b + slack + (terms + b) * 2.0**-8)


@pytest.mark.parametrize("layer_id", [0, 2])
def test_experts_on_a_batching(layer_id):
    """The batching's y, groupList and actualTokenNum go to the experts as they
    are: masked slots and absent experts included, one layer's weights."""
    H, inter, per_layer = 256, 128, 6
    inp = w.make_batching(A=4, BS=8, K1=3, E=4 * per_layer, H=H, dtype=w.DT_BF16, layerNum=4, layer_id=layer_id,
                          ids="zipf", zipf_s=1.2, mask=0.3, seed=11)
    out = run_batching(inp)
    wt = moe_step.make_weights(per_layer, H, inter, seed=3)
    used = int(out["actualTokenNum"].item())
    assert 0 < used < inp["Y"]
    y = torch.full((inp["Y"], H), 7.0, dtype=torch.bfloat16, device="cuda")
    usc.moe_expert_ffn(out["y"], wt["w13"], wt["w13_scales"], wt["w2"], wt["w2_scales"], out["groupList"],
                       num_rows=out["actualTokenNum"], expert_base=layer_id * per_layer, out=dict(y=y))
    c = {k: v.cpu() for k, v in wt.items()}
    W13, W2 = eu.weight(c["w13"], c["w13_scales"]), eu.weight(c["w2"], c["w2_scales"])
    x = out["y"].cpu().double()
    at = 0
    for key, count in out["groupList"].cpu().tolist():
        if count == 0:
            continue
        q, s = eu.quantize(x[at:at + count])
        e = key - layer_id * per_layer
        eu.assert_close(y[at:at + count], *eu.net(q * eu.spread(s, H), W13[e, 0], W13[e, 1], W2[e]))
        at += count
    assert at == used and (y[used:] == 7.0).all()


def test_suites_on_the_checked_build():
    from unpermute_stable_counting_gb300 import _build, _native
    if _native.checked_requested():
        pytest.skip("this process is the checked run")
    _build.build_library(checked=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider",
                        "tests/test_gpu_expert_products.py", "tests/test_gpu_layer.py"],
                       cwd=ROOT, env=dict(os.environ, USC_CHECKED="1"), capture_output=True, text=True, timeout=1500)
    tail = r.stdout[-4000:] + r.stderr[-2000:]
    assert r.returncode == 0 and " passed" in r.stdout and " failed" not in r.stdout, tail
