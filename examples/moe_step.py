"""One mixture-of-experts step on GB300, both ways that this package offers:

* routed_step: any number of tokens. The router's choice becomes a routing map,
  moe_permute groups the rows by expert, moe_expert_ffn runs the experts on the
  groups, moe_unpermute brings the weighted rows back.
* moe_layer: up to 64 tokens, the same step in one launch.

Both use the same 8-bit weights (moe_quantize with 128 x 128 blocks).

    python examples/moe_step.py --tokens 32
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import unpermute_stable_counting_gb300 as usc  # noqa: E402


def make_weights(experts: int, hidden: int, inter: int, seed: int = 0) -> dict:
    """A router and the experts' weights, quantized as a loader does once."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, fan):
        return (torch.randn(*shape, device="cuda", generator=g) / fan**0.5).to(torch.bfloat16)

    w13 = usc.moe_quantize(normal(experts, 2, inter, hidden, fan=hidden), block_rows=128)
    w2 = usc.moe_quantize(normal(experts, hidden, inter, fan=inter), block_rows=128)
    return dict(router=normal(experts, hidden, fan=hidden), w13=w13["values"], w13_scales=w13["scales"],
                w2=w2["values"], w2_scales=w2["scales"])


def route(x, router, topk: int):
    """The routing map [tokens, experts], and each token's experts (ascending) and their weights [tokens, topk]."""
    probs = torch.softmax(x.float() @ router.float().T, -1)
    top, ids = torch.topk(probs, topk, dim=-1)
    ids, order = ids.sort(-1)
    top = torch.gather(top, 1, order)
    routing_map = torch.zeros(probs.shape, dtype=torch.int8, device=x.device).scatter_(1, ids, 1)
    return routing_map, ids, top / top.sum(-1, keepdim=True)


def routed_step(x, w: dict, topk: int, capacity: int | None = None):
    """permute -> experts -> unpermute, of the rows that were routed. With a capacity each expert
    has that many rows: it drops the tokens past them, and rows of zeros fill them up (8 of 64
    experts and room for every token are eight times the rows)."""
    experts, device = w["router"].shape[0], x.device
    weights = (w["w13"], w["w13_scales"], w["w2"], w["w2_scales"])
    routing_map, ids, top = route(x, w["router"], topk)
    expert = torch.arange(experts, device=device)
    if capacity is not None:
        rows = usc.moe_permute(x, routing_map, padded_mode=True, capacity=capacity)
        groups = torch.stack([expert, torch.full_like(expert, capacity)], 1)
        y = usc.moe_expert_ffn(rows["permutedTokens"], *weights, groups)["y"]
        probs = torch.zeros(routing_map.shape, device=device).scatter_(1, ids, top)
        return usc.moe_unpermute(y, rows["sortedIndices"], routing_map, probs, padded_mode=True,
                                 restore_shape=tuple(x.shape))["unpermutedTokens"]
    rows = usc.moe_permute(x, routing_map, topk=topk)
    groups = torch.stack([expert, routing_map.sum(0)], 1)
    y = usc.moe_expert_ffn(rows["permutedTokens"], *weights, groups, out_dtype=torch.float32)["y"]
    # sortedIndices has a token's rows by ascending expert: the weights in the rows' order
    y *= torch.empty_like(y[:, 0]).scatter_(0, rows["sortedIndices"].long(), top.flatten())[:, None]
    return usc.moe_unpermute(y, rows["sortedIndices"], restore_shape=tuple(x.shape))["unpermutedTokens"].to(x.dtype)


def layer_step(x, w: dict, topk: int):
    return usc.moe_layer(x, w["router"], w["w13"], w["w2"], topk=topk, w13_scales=w["w13_scales"],
                         w2_scales=w["w2_scales"])["y"]


def time_us(f, n: int = 50) -> float:
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3 / n


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inter", type=int, default=1024)
    ap.add_argument("--capacity", type=int, default=None, help="rows of each expert (default: those routed to it)")
    args = ap.parse_args()
    w = make_weights(args.experts, args.hidden, args.inter)
    x = torch.randn(args.tokens, args.hidden, device="cuda").to(torch.bfloat16)
    y = routed_step(x, w, args.topk, args.capacity)
    print(f"routed step: {time_us(lambda: routed_step(x, w, args.topk, args.capacity)):.1f} us")
    if args.tokens <= 64:
        z = layer_step(x, w, args.topk)
        off = ((y - z).float().norm() / z.float().norm()).item()
        print(f"one launch:  {time_us(lambda: layer_step(x, w, args.topk)):.1f} us, "
              f"relative difference {off:.2g}")


if __name__ == "__main__":
    main()
