"""The expert operators' argument checks at the edges (no GPU needed: each call
returns before anything touches the device)."""
import ctypes

import pytest

from test_expert_host import BF16, E4M3, FAKE, INVALID, OK, F16, ffn, layer, matmul, pair, quantize  # noqa: F401

from unpermute_stable_counting_gb300 import _build, _native


@pytest.fixture(scope="module")
def L():
    _build.build_library()
    return _native.lib()


def ffn_rows_in_use(L, num):
    return L.moe_expert_ffn(FAKE, BF16, 512, None, None, FAKE, None, FAKE, FAKE, None, FAKE, FAKE, 4, num, 0, 8, 4, 512, 256,
                            FAKE, BF16, 512, FAKE, 1 << 40, None)


@pytest.mark.parametrize("call,kw", [
    (quantize, dict(num=FAKE + 4)),
    (matmul, dict(xs=FAKE + 2)), (matmul, dict(ws=FAKE + 1)), (matmul, dict(dt=BF16, num=FAKE + 4)),
    (ffn, dict(s13=FAKE + 2)), (ffn, dict(s2=FAKE + 2)), (ffn, dict(dt=E4M3, xs=FAKE + 2)),
    (layer, dict(s13=FAKE + 2)), (layer, dict(s2=FAKE + 3)), (layer, dict(bias=FAKE + 2)), (layer, dict(ids=FAKE + 1)),
    (layer, dict(wts=FAKE + 2)),
    (lambda L, num: ffn_rows_in_use(L, num), dict(num=FAKE + 4)),
])
def test_addresses_that_their_type_cannot_have(L, call, kw):
    """Scales, counts, ids: a kernel would read (or write) them at an address that faults."""
    assert call(L, **kw) == INVALID


def test_the_tile_of_a_product(L):
    t = (ctypes.c_int32 * 3)()
    assert L.mr_expert_tile(16384, -1, 7168, 0, t) == OK and tuple(t[:2]) == (256, 256) and t[2] > 0
    assert L.mr_expert_tile(1, 1, 16, 0, t) == OK and tuple(t[:2]) == (128, 128)
    assert L.mr_expert_tile(32768, 64, 2048, 1, t) == OK and tuple(t[:2]) == (256, 128)
    assert L.mr_expert_tile(4, 1, 16, 0, None) == _NULLPTR
    for bad in ((0, 1, 16), (4, 0, 16), (4, -2, 16), (4, 1, 0), ((1 << 30) + 1, 1, 16)):
        assert L.mr_expert_tile(*bad, 0, t) == INVALID


_NULLPTR = 161001
