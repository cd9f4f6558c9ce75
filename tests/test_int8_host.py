"""The INT8 operators' argument checks (no GPU needed: each call returns before
anything touches the CUDA runtime)."""
import ctypes

import pytest

from unpermute_stable_counting_gb300 import _build, _native

OK, NULLPTR, INVALID, WORKSPACE = 0, 161001, 161002, 561002
F16, BF16, INT8, F32, E4M3 = 0, 1, 2, 3, 6
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    _build.build_library()
    return _native.lib()


def arr(v):
    return None if v is None else (ctypes.c_int64 * 2)(*v)


def quantize(L, **kw):
    a = dict(x=FAKE, dt=BF16, batch=1, rows=4, cols=256, xs=None, num=None, v=FAKE, vs=None, s=FAKE, ss=None)
    a.update(kw)
    return L.moe_quantize_int8(a["x"], a["dt"], a["batch"], a["rows"], a["cols"], arr(a["xs"]), a["num"], a["v"],
                               arr(a["vs"]), a["s"], arr(a["ss"]), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=0, x=None, v=None, s=None), OK),
    (dict(x=None), NULLPTR), (dict(v=None), NULLPTR), (dict(s=None), NULLPTR),
    (dict(dt=INT8), INVALID), (dict(dt=E4M3), INVALID), (dict(dt=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(cols=0), INVALID), (dict(cols=(1 << 24) + 1), INVALID), (dict(rows=(1 << 30) + 1), INVALID),
    (dict(batch=0), INVALID), (dict(batch=1 << 20, rows=1 << 20), INVALID), (dict(batch=2, num=FAKE), INVALID),
    (dict(xs=(0, -1)), INVALID), (dict(vs=(0, 255)), INVALID), (dict(batch=2, vs=(1000, 256)), INVALID),
    (dict(ss=(0, 0)), INVALID), (dict(batch=2, ss=(3, 1)), INVALID),
    (dict(x=FAKE + 1), INVALID), (dict(dt=F32, x=FAKE + 2), INVALID), (dict(s=FAKE + 2), INVALID), (dict(num=FAKE + 4), INVALID),
])
def test_quantize(L, kw, expect):
    assert quantize(L, **kw) == expect


def norm(L, **kw):
    a = dict(x=FAKE, dt=BF16, rows=4, cols=256, xst=256, r=FAKE, rst=256, w=FAKE, wdt=BF16, eps=1e-6, num=None, h=FAKE, hst=256,
             y=FAKE, yst=256, q=INT8, v=FAKE, vst=256, s=FAKE, ss=None)
    a.update(kw)
    return L.moe_add_rms_norm(a["x"], a["dt"], a["rows"], a["cols"], a["xst"], a["r"], a["rst"], a["w"], a["wdt"], a["eps"],
                              a["num"], a["h"], a["hst"], a["y"], a["yst"], a["q"], a["v"], a["vst"], a["s"], arr(a["ss"]),
                              None)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=0), OK), (dict(rows=0, x=None, w=None), OK),
    (dict(x=None), NULLPTR), (dict(w=None), NULLPTR), (dict(v=None), NULLPTR), (dict(s=None), NULLPTR),
    (dict(y=None, h=None, q=-1), NULLPTR),
    (dict(dt=INT8), INVALID), (dict(q=BF16), INVALID), (dict(q=-2), INVALID), (dict(wdt=F16), INVALID), (dict(wdt=E4M3), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=(1 << 30) + 1), INVALID), (dict(cols=0), INVALID), (dict(cols=(1 << 24) + 1), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(xst=-1), INVALID), (dict(rst=-1), INVALID), (dict(hst=255), INVALID), (dict(yst=255), INVALID),
    (dict(vst=255), INVALID), (dict(r=None), INVALID), (dict(ss=(0, 1)), INVALID), (dict(ss=(1, 0)), INVALID),
    (dict(x=FAKE + 1), INVALID), (dict(r=FAKE + 1), INVALID), (dict(h=FAKE + 1), INVALID), (dict(y=FAKE + 1), INVALID),
    (dict(w=FAKE + 1), INVALID), (dict(wdt=F32, w=FAKE + 2), INVALID), (dict(s=FAKE + 1), INVALID), (dict(num=FAKE + 4), INVALID),
])
def test_norm(L, kw, expect):
    assert norm(L, **kw) == expect


def matmul(L, **kw):
    a = dict(x=FAKE, dt=INT8, xst=512, xs=FAKE, xss=1, w=FAKE, wst=None, ws=FAKE, g=FAKE, G=4, num=None, base=0,
             rows=300, E=4, N=64, K=512, y=FAKE, ydt=BF16, yst=64, wsp=FAKE, size=1 << 40)
    a.update(kw)
    return L.moe_grouped_matmul_int8(a["x"], a["dt"], a["xst"], a["xs"], a["xss"], a["w"], arr(a["wst"]), a["ws"],
                                     a["g"], a["G"], a["num"], a["base"], a["rows"], a["E"], a["N"], a["K"], a["y"],
                                     a["ydt"], a["yst"], a["wsp"], a["size"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=0), OK), (dict(rows=0, x=None, y=None), OK), (dict(G=0, g=None), OK), (dict(G=0, g=None, wsp=None, size=0), OK),
    (dict(x=None), NULLPTR), (dict(xs=None), NULLPTR), (dict(w=None), NULLPTR), (dict(ws=None), NULLPTR),
    (dict(y=None), NULLPTR), (dict(g=None), NULLPTR), (dict(wsp=None), NULLPTR), (dict(size=16), WORKSPACE),
    (dict(dt=F32), INVALID), (dict(dt=E4M3), INVALID), (dict(ydt=INT8), INVALID), (dict(ydt=E4M3), INVALID),
    (dict(rows=(1 << 30) + 1), INVALID), (dict(rows=-1), INVALID), (dict(E=0), INVALID), (dict(E=8193), INVALID),
    (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(G=-2), INVALID), (dict(xst=511), INVALID), (dict(xst=520), INVALID),
    (dict(yst=63), INVALID), (dict(K=500, xst=500), INVALID), (dict(dt=BF16, xst=516), INVALID), (dict(xss=-1), INVALID),
    (dict(wst=(511, 64 * 512)), INVALID), (dict(wst=(520, 64 * 528)), INVALID), (dict(wst=(512, 8)), INVALID),
    (dict(wst=(512, 512)), INVALID), (dict(x=FAKE + 8), INVALID), (dict(w=FAKE + 8), INVALID), (dict(g=FAKE + 8), INVALID),
    (dict(y=FAKE + 1), INVALID), (dict(ydt=F32, y=FAKE + 2), INVALID), (dict(wsp=FAKE + 16), INVALID),
    (dict(ws=FAKE + 2), INVALID), (dict(xs=FAKE + 2), INVALID), (dict(num=FAKE + 4), INVALID),
])
def test_matmul(L, kw, expect):
    assert matmul(L, **kw) == expect


def ffn(L, **kw):
    a = dict(x=FAKE, dt=INT8, xst=512, xs=FAKE, xss=1, w13=FAKE, st13=None, s13=FAKE, w2=FAKE, st2=None, s2=FAKE, g=FAKE, G=4,
             num=None, rows=8, E=4, H=512, I=256, y=FAKE, ydt=BF16, yst=512, wsp=FAKE, size=1 << 40)
    a.update(kw)
    return L.moe_expert_ffn_int8(a["x"], a["dt"], a["xst"], a["xs"], a["xss"], a["w13"], arr(a["st13"]), a["s13"], a["w2"],
                                 arr(a["st2"]), a["s2"], a["g"], a["G"], a["num"], 0, a["rows"], a["E"], a["H"], a["I"], a["y"],
                                 a["ydt"], a["yst"], a["wsp"], a["size"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=0), OK), (dict(G=0, g=None, wsp=None, size=0), OK),
    (dict(x=None), NULLPTR), (dict(xs=None), NULLPTR), (dict(w13=None), NULLPTR), (dict(s13=None), NULLPTR),
    (dict(w2=None), NULLPTR), (dict(s2=None), NULLPTR), (dict(y=None), NULLPTR), (dict(wsp=None), NULLPTR), (dict(g=None), NULLPTR),
    (dict(size=16), WORKSPACE),
    (dict(dt=F32), INVALID), (dict(ydt=INT8), INVALID), (dict(H=0), INVALID), (dict(I=0), INVALID), (dict(yst=511), INVALID),
    (dict(xst=511), INVALID), (dict(st13=(512, 8)), INVALID), (dict(st13=(500, 256 * 512)), INVALID),
    (dict(st2=(255, 512 * 256)), INVALID), (dict(I=250), INVALID), (dict(w2=FAKE + 4), INVALID), (dict(w13=FAKE + 4), INVALID),
    (dict(wsp=FAKE + 128), INVALID), (dict(x=FAKE + 4), INVALID), (dict(s13=FAKE + 1), INVALID), (dict(s2=FAKE + 1), INVALID),
])
def test_ffn(L, kw, expect):
    assert ffn(L, **kw) == expect


def test_workspace_sizes(L):
    n = ctypes.c_uint64(7)
    p = ctypes.byref(n)

    def matmul_size(*a):
        assert L.moe_grouped_matmul_int8_get_workspace_size(*a, p) == OK
        return n.value
    assert matmul_size(0, 4, 64, 512, INT8) == 0 and matmul_size(8, 0, 64, 512, INT8) == 0
    assert matmul_size(5000, 4, 4096, 512, BF16) == 0
    assert matmul_size(5000, 4, 4096, 500, INT8) >= 5000 * 512 * 2         # rows of 16 bits
    assert matmul_size(1, -1, 2048, 4096, BF16) >= 8 * 4                   # shares of few tiles
    assert L.moe_grouped_matmul_int8_get_workspace_size(8, 4, 64, 512, F32, p) == INVALID
    assert L.moe_grouped_matmul_int8_get_workspace_size(8, 4, 64, 0, INT8, p) == INVALID
    assert L.moe_grouped_matmul_int8_get_workspace_size(8, 4, 64, 512, INT8, None) == NULLPTR
    assert L.moe_expert_ffn_int8_get_workspace_size(100, 4, 512, 300, INT8, p) == OK and n.value >= 100 * 320 * 2
    assert L.moe_expert_ffn_int8_get_workspace_size(100, -2, 512, 300, INT8, p) == INVALID
    assert L.moe_expert_ffn_int8_get_workspace_size(100, 4, 512, 300, INT8, None) == NULLPTR
