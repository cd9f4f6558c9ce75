"""Every kernel of the grouped product with several tiles for each block: what a
block carries from one tile to the next (its place in the list, the ring, the
buffers, the next tile's scales, the results on their way out) is used. Which
kernel a size reaches is asked of the library (mr_expert_tile), so that another
rule cannot leave one of them out unnoticed. Against 64 bits; tolerances: see
_expert_util."""
import ctypes
import functools

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import unpermute_stable_counting_gb300 as usc  # noqa: E402
from unpermute_stable_counting_gb300 import _native  # noqa: E402

import _expert_util as eu  # noqa: E402

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(autouse=True)
def _no_wait_ran_out():
    yield
    assert usc.waits_out(reset=True) == 0


def several_tiles(pairs, N, tile, network=False):
    """The call is cut into tiles of this size, and there are more of them than are in work at once."""
    got = (ctypes.c_int32 * 3)()
    assert _native.lib().mr_expert_tile(sum(c for _, c in pairs), len(pairs), N, int(network), got) == 0
    assert tuple(got[:2]) == tile, f"this size is cut into tiles of {tuple(got[:2])}"
    tiles = sum(-(-c // tile[0]) for _, c in pairs) * -(-N // tile[1])
    assert tiles > got[2], f"{tiles} tiles, {got[2]} at once"


def ragged(groups, rows, seed):
    """Many groups of a few rows, one of more than a tile, in no order."""
    g = torch.Generator().manual_seed(seed)
    counts = torch.randint(1, 5, (groups,), generator=g)
    counts[groups // 3] = 0
    counts[groups // 3] = rows - int(counts.sum())
    assert counts[groups // 3] > 128
    return [(int(e), int(c)) for e, c in zip(torch.randperm(groups, generator=g), counts)]


FULL = [(1, 1000), (0, 901), (2, 149)]            # row tiles of 256: the last of each has 232, 133 and 149 rows
CASES = {(256, 256): (FULL, 2500), (128, 256): (ragged(64, 330, 1), 1020), (128, 128): (ragged(64, 330, 2), 635)}
K = 1000                                          # eight steps: more than the ring has stages


def eight(n, k, g):
    q = (torch.randn(n, k, generator=g) * 100).clamp(-448, 448).to(E4M3)
    s = torch.exp(0.5 * torch.randn(n, eu.blocks(k), generator=g)) * 0.01
    return q, s, q.double() * eu.spread(s.double(), k)


def weights(lead, n, k, g):
    """e4m3 weights whose rows start on 16 bytes, on the device and here, and their scales."""
    w = (torch.randn(*lead, n, k, generator=g) * 100).clamp(-448, 448).to(E4M3)
    s = torch.exp(0.4 * torch.randn(*lead, eu.blocks(n), eu.blocks(k), generator=g)) / (100 * k**0.5)
    d = torch.full((*lead, n, -(-k // 16) * 16), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)[..., :k]
    d.view(torch.uint8).copy_(w.view(torch.uint8).cuda())
    return d, s.cuda(), eu.weight(w, s)


def over_groups(pairs, one):
    """(result, bound) of one(rows, expert) over the groups."""
    at, parts = 0, []
    for e, c in pairs:
        parts.append(one(slice(at, at + c), e))
        at += c
    return tuple(torch.cat(v) for v in zip(*parts))


@functools.lru_cache(maxsize=None)
def product_case(tile):
    pairs, N = CASES[tile]
    g = torch.Generator().manual_seed(N)
    n = sum(c for _, c in pairs)
    q, s, x = eight(n, -(-K // 16) * 16, g)
    s, x = s[:, :eu.blocks(K)], x[:, :K]
    w, ws, W = weights((len(pairs),), N, K, g)
    ref = over_groups(pairs, lambda r, e: eu.product(x[r], W[e]))
    return pairs, N, q.cuda()[:, :K], s.cuda(), w, ws, torch.tensor(pairs).cuda(), ref


@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("anywhere", [False, True])
@pytest.mark.parametrize("tile", list(CASES))
def test_several_tiles_of_a_product(tile, anywhere, out):
    """Results that start on 16 bytes, and that start anywhere; columns past the last whole tile."""
    pairs, N, x, xs, w, ws, lst, (ref, bound) = product_case(tile)
    several_tiles(pairs, N, tile)
    n = x.shape[0]
    lead, step = (1, N + 1) if anywhere else (0, -(-N // 8) * 8)
    buf = torch.full((lead + n * step,), 77.0, dtype=out, device="cuda")
    rows = buf[lead:].view(n, step)
    usc.moe_grouped_matmul(x, w, ws, lst, x_scales=xs, out=dict(y=rows[:, :N]))
    eu.assert_close(rows[:, :N], ref, bound)
    assert (rows[:, N:] == 77).all() and (buf[:lead] == 77).all()
    first = buf.clone()
    for _ in range(3):
        rows[:, :N] = 5.0
        usc.moe_grouped_matmul(x, w, ws, lst, x_scales=xs, out=dict(y=rows[:, :N]))
        assert torch.equal(first.view(torch.uint8), buf.view(torch.uint8))


@pytest.mark.parametrize("tile,H,inter,second", [((256, 128), 2500, 1250, (256, 256)), ((128, 128), 1020, 380, (128, 256))])
def test_several_tiles_of_the_network(tile, H, inter, second):
    """Both products: rows of h are quantized at the end of tiles of either parity."""
    pairs = FULL if tile[0] == 256 else ragged(64, 330, 3)
    several_tiles(pairs, inter, tile, network=True)
    several_tiles(pairs, H, second)
    g = torch.Generator().manual_seed(H)
    n, E = sum(c for _, c in pairs), len(pairs)
    x = torch.randn(n, H, generator=g).to(BF16)
    w13, s13, W13 = weights((E, 2), inter, H, g)
    w2, s2, W2 = weights((E,), H, inter, g)
    v, s = eu.quantize(x.double())
    v = v * eu.spread(s, H)
    lst = torch.tensor(pairs).cuda()
    y = usc.moe_expert_ffn(x.cuda(), w13, s13, w2, s2, lst)["y"]
    eu.assert_close(y, *over_groups(pairs, lambda r, e: eu.net(v[r], W13[e, 0], W13[e, 1], W2[e])))
    for _ in range(3):
        again = usc.moe_expert_ffn(x.cuda(), w13, s13, w2, s2, lst)["y"]
        assert torch.equal(y.view(torch.uint8), again.view(torch.uint8))


@pytest.mark.parametrize("T,E,topk,I", [(16, 40, 8, 520), (32, 40, 8, 1000), (64, 48, 8, 424), (64, 20, 5, 2056)])
@pytest.mark.parametrize("wdt", [E4M3, BF16, F16])
def test_several_tiles_of_the_layer(T, E, topk, I, wdt):
    """moe_layer's second step takes 16 groups of 8 rows of W1 and W3 at a time: here a block has more, so
    that blocks of 128 values of h are completed over several tiles, of one block and of neighbours."""
    import test_gpu_layer as layer
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c = layer.make(T, E, 200, I, BF16 if wdt is E4M3 else wdt, wdt, T + I)
    r = layer.run(c, topk)
    taken = r["expertIds"].unique().numel()
    assert taken * -(-I // 8) > 16 * sms, f"{taken} experts taken"
    layer.check(c, topk, r)
    for _ in range(3):
        again = layer.run(c, topk)
        assert all(torch.equal(r[k], again[k]) for k in r)
