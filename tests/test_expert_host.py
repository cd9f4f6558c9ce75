"""The expert operators' argument checks (no GPU needed: each call returns
before anything touches the CUDA runtime)."""
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


def pair(*v):
    return None if v[0] is None else (ctypes.c_int64 * 2)(*v)


def quantize(L, **kw):
    a = dict(x=FAKE, dt=BF16, batch=1, rows=4, cols=256, xs=None, blk=1, num=None, v=FAKE, vs=None, s=FAKE, ss=None)
    a.update(kw)
    arr = lambda v: None if v is None else pair(*v)
    return L.moe_quantize(a["x"], a["dt"], a["batch"], a["rows"], a["cols"], arr(a["xs"]), a["blk"], a["num"], a["v"],
                          arr(a["vs"]), a["s"], arr(a["ss"]), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=0, x=None, v=None, s=None), OK),
    (dict(x=None), NULLPTR), (dict(v=None), NULLPTR), (dict(s=None), NULLPTR),
    (dict(dt=INT8), INVALID), (dict(dt=E4M3), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(cols=(1 << 24) + 1), INVALID), (dict(rows=1 << 30, cols=512), INVALID), (dict(blk=64), INVALID),
    (dict(batch=2), INVALID), (dict(batch=0), INVALID), (dict(blk=128, num=FAKE), INVALID),
    (dict(xs=(0, -1)), INVALID), (dict(vs=(0, 255)), INVALID), (dict(ss=(0, 1)), INVALID),
    (dict(blk=128, ss=(2, 1)), INVALID), (dict(blk=128, batch=2, vs=(100, 256)), INVALID),
    (dict(x=FAKE + 1), INVALID), (dict(dt=F32, x=FAKE + 2), INVALID), (dict(s=FAKE + 2), INVALID),
])
def test_quantize(L, kw, expect):
    assert quantize(L, **kw) == expect


def matmul(L, **kw):
    a = dict(x=FAKE, dt=E4M3, xst=512, xs=FAKE, xss=None, w=FAKE, wst=None, ws=FAKE, g=FAKE, G=4, num=None, base=0,
             rows=8, E=4, N=64, K=512, y=FAKE, ydt=BF16, yst=64, wsp=FAKE, size=1 << 40)
    a.update(kw)
    arr = lambda v: None if v is None else pair(*v)
    return L.moe_grouped_matmul(a["x"], a["dt"], a["xst"], a["xs"], arr(a["xss"]), a["w"], arr(a["wst"]), a["ws"],
                                a["g"], a["G"], a["num"], a["base"], a["rows"], a["E"], a["N"], a["K"], a["y"],
                                a["ydt"], a["yst"], a["wsp"], a["size"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=0), OK), (dict(rows=0, x=None, y=None), OK), (dict(G=0, g=None), OK),
    (dict(x=None), NULLPTR), (dict(xs=None), NULLPTR), (dict(w=None), NULLPTR), (dict(ws=None), NULLPTR),
    (dict(y=None), NULLPTR), (dict(g=None), NULLPTR), (dict(dt=BF16, wsp=None), NULLPTR),
    (dict(dt=BF16, size=16), WORKSPACE),
    (dict(dt=INT8), INVALID), (dict(ydt=E4M3), INVALID), (dict(rows=(1 << 30) + 1), INVALID), (dict(rows=-1), INVALID),
    (dict(E=0), INVALID), (dict(E=8193), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(G=-2), INVALID),
    (dict(xst=511), INVALID), (dict(xst=520), INVALID), (dict(yst=63), INVALID), (dict(K=500, xst=512), INVALID),
    (dict(wst=(511, 64 * 512)), INVALID), (dict(wst=(520, 64 * 528)), INVALID), (dict(wst=(512, 8)), INVALID),
    (dict(wst=(512, 512)), INVALID), (dict(xss=(-1, 1)), INVALID),
    (dict(x=FAKE + 8), INVALID), (dict(w=FAKE + 8), INVALID), (dict(g=FAKE + 8), INVALID), (dict(y=FAKE + 1), INVALID),
    (dict(dt=BF16, wsp=FAKE + 16), INVALID), (dict(dt=F32, rows=1 << 30), INVALID),
])
def test_matmul(L, kw, expect):
    assert matmul(L, **kw) == expect


def ffn(L, **kw):
    a = dict(x=FAKE, dt=BF16, xst=512, xs=None, w13=FAKE, s13=FAKE, st13=None, w2=FAKE, s2=FAKE, st2=None, g=FAKE, G=4,
             rows=8, E=4, H=512, I=256, y=FAKE, ydt=BF16, yst=512, wsp=FAKE, size=1 << 40)
    a.update(kw)
    arr = lambda v: None if v is None else pair(*v)
    return L.moe_expert_ffn(a["x"], a["dt"], a["xst"], a["xs"], None, a["w13"], arr(a["st13"]), a["s13"], a["w2"],
                            arr(a["st2"]), a["s2"], a["g"], a["G"], None, 0, a["rows"], a["E"], a["H"], a["I"], a["y"],
                            a["ydt"], a["yst"], a["wsp"], a["size"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=0), OK), (dict(G=0, g=None), OK),
    (dict(x=None), NULLPTR), (dict(w13=None), NULLPTR), (dict(s13=None), NULLPTR), (dict(w2=None), NULLPTR),
    (dict(s2=None), NULLPTR), (dict(y=None), NULLPTR), (dict(wsp=None), NULLPTR), (dict(dt=E4M3), NULLPTR),
    (dict(size=16), WORKSPACE),
    (dict(H=0), INVALID), (dict(I=0), INVALID), (dict(yst=511), INVALID), (dict(xst=511), INVALID),
    (dict(st13=(512, 8)), INVALID), (dict(st13=(500, 256 * 512)), INVALID), (dict(st2=(255, 512 * 256)), INVALID),
    (dict(I=250), INVALID), (dict(w2=FAKE + 4), INVALID), (dict(wsp=FAKE + 128), INVALID),
])
def test_ffn(L, kw, expect):
    assert ffn(L, **kw) == expect


def layer(L, **kw):
    a = dict(x=FAKE, xdt=BF16, xst=512, r=FAKE, rdt=BF16, rst=512, bias=None, w13=FAKE, wdt=E4M3, st13=None, s13=FAKE,
             w2=FAKE, st2=None, s2=FAKE, T=4, H=512, I=256, E=8, K=2, flags=0, y=FAKE, yst=512, ids=FAKE, wts=FAKE,
             wsp=FAKE, size=1 << 40)
    a.update(kw)
    arr = lambda v: None if v is None else pair(*v)
    return L.moe_layer(a["x"], a["xdt"], a["xst"], a["r"], a["rdt"], a["rst"], a["bias"], a["w13"], a["wdt"],
                       arr(a["st13"]), a["s13"], a["w2"], arr(a["st2"]), a["s2"], a["T"], a["H"], a["I"], a["E"],
                       a["K"], a["flags"], 1.0, a["y"], a["yst"], a["ids"], a["wts"], a["wsp"], a["size"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=0), OK),
    (dict(x=None), NULLPTR), (dict(r=None), NULLPTR), (dict(w13=None), NULLPTR), (dict(w2=None), NULLPTR),
    (dict(y=None), NULLPTR), (dict(ids=None), NULLPTR), (dict(wts=None), NULLPTR), (dict(wsp=None), NULLPTR),
    (dict(s13=None), NULLPTR), (dict(s2=None), NULLPTR), (dict(wdt=BF16), NULLPTR), (dict(size=16), WORKSPACE),
    (dict(T=65), INVALID), (dict(T=-1), INVALID), (dict(H=16385), INVALID), (dict(I=0), INVALID), (dict(E=1025), INVALID),
    (dict(K=0), INVALID), (dict(K=9), INVALID), (dict(K=17, E=32), INVALID), (dict(wdt=F32), INVALID),
    (dict(xdt=E4M3), INVALID), (dict(rdt=INT8), INVALID), (dict(wdt=F16, s13=None, s2=None), INVALID),
    (dict(flags=4), INVALID), (dict(xst=511), INVALID), (dict(rst=511), INVALID), (dict(yst=511), INVALID),
    (dict(st13=(512, 256 * 512 + 8)), INVALID), (dict(st2=(256, 16)), INVALID), (dict(I=250), INVALID),
    (dict(w13=FAKE + 8), INVALID), (dict(x=FAKE + 1), INVALID), (dict(wsp=FAKE + 64), INVALID),
])
def test_layer(L, kw, expect):
    assert layer(L, **kw) == expect


def test_workspace_sizes(L):
    n = ctypes.c_uint64(7)
    p = ctypes.byref(n)
    assert L.moe_grouped_matmul_get_workspace_size(100, 512, E4M3, p) == OK and n.value == 0
    assert L.moe_grouped_matmul_get_workspace_size(100, 512, BF16, p) == OK and n.value >= 100 * 512 + 100 * 16
    assert L.moe_grouped_matmul_get_workspace_size(100, 512, INT8, p) == INVALID
    assert L.moe_grouped_matmul_get_workspace_size(100, 512, BF16, None) == NULLPTR
    assert L.moe_expert_ffn_get_workspace_size(100, 512, 300, p) == OK and n.value >= 100 * (512 + 384)
    assert L.moe_expert_ffn_get_workspace_size(100, 0, 300, p) == INVALID
    assert L.moe_layer_get_workspace_size(64, 512, 300, 16, 4, E4M3, p) == OK and n.value > 64 * 4 * 384 * 5
    assert L.moe_layer_get_workspace_size(65, 512, 300, 16, 4, E4M3, p) == INVALID
    assert L.moe_layer_get_workspace_size(64, 512, 300, 16, 4, E4M3, None) == NULLPTR
    assert L.mr_waits_out(None, 0) == NULLPTR
