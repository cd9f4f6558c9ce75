"""64-bit definitions of the expert operators on CPU tensors, with the error
that fp32 sums may have, for the GPU tests.

Error of a sum of n fp32 terms with absolute sum S: at most n * 2^-23 * S for
any order of the additions, rounded to nearest or cut (each addition is off by
at most 2^-23 of a partial sum, which is at most S). Results of 16-bit types
are rounded once more: 2^-8 (bf16), 2^-11 (f16) of the value."""
import torch

BLOCK = 128
OUT_ROUND = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11, torch.float32: 2.0**-23}
# below its normal range f16 rounds to multiples of 2^-24
OUT_FLOOR = {torch.bfloat16: 0.0, torch.float16: 2.0**-25, torch.float32: 0.0}


def blocks(n):
    return -(-n // BLOCK)


def e4m3_step(v):
    """Spacing of the e4m3 values around v (float64)."""
    e = torch.frexp(v)[1]                       # |v| in [2^(e-1), 2^e)
    return torch.exp2((e - 1).clamp_min(-6).double() - 3)


def e4m3(v):
    s = e4m3_step(v)
    return torch.round(v / s) * s               # torch.round: ties to even


def scale_of(amax):
    """The smallest power of two s with max(amax, 2^-96) <= 448 s (float64)."""
    a = amax.clamp_min(2.0**-96)
    m, e = torch.frexp(a)
    s = torch.exp2((e - 9 + (m > 0.875)).double())
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, float("nan")))


def quantize(x):
    """(e4m3 values, scales) of float64 rows."""
    K = x.shape[-1]
    v = torch.nn.functional.pad(x, (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))
    bad = ~torch.isfinite(v).all(-1)
    amax = torch.where(bad, torch.full_like(v[..., 0], float("inf")), v.abs().amax(-1))
    s = scale_of(amax)
    q = e4m3(v / s[..., None])
    return q.flatten(-2)[..., :K], s


def spread(s, K):
    return s.repeat_interleave(BLOCK, -1)[..., :K]


def weight(w, s):
    """float64 weights [..., N, K] of e4m3 values and their scales."""
    N, K = w.shape[-2:]
    return w.double() * s.double().repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]


def product(x, w):
    """(x w^T, bound of the fp32 error) of float64 rows and one float64 matrix."""
    return x @ w.T, (x.shape[1] + blocks(x.shape[1])) * 2.0**-23 * (x.abs() @ w.abs().T)


def net(x, w1, w3, w2, rounded=True):
    """(y, bound) of silu(x w1^T) * (x w3^T) [quantized] times w2^T."""
    (g, dg), (u, du) = product(x, w1), product(x, w3)
    sg = g * torch.sigmoid(g)
    h = sg * u
    # |silu'| < 1.1; silu and the two products are fp32 with errors of a few 2^-23, of |g| 2^-23 in the exponent
    dh = 1.1 * dg * (u.abs() + du) + (sg.abs() + 1.1 * dg) * du + h.abs() * (16 + g.abs()) * 2.0**-23
    if not rounded:
        y, dy = product(h, w2)
        return y, dy + dh @ w2.abs().T
    q, s = quantize(h)
    S = spread(s, h.shape[1])
    y, dy = product(q * S, w2)
    # an element may round to either neighbour where the fp32 error reaches a rounding boundary
    v = h / S
    step = e4m3_step(v)
    to_edge = ((v / step - torch.floor(v / step)) - 0.5).abs() * step
    moved = torch.where(to_edge * S <= dh, step * S, torch.zeros_like(v))
    # and a whole block to half as many digits where the error reaches the edge of its scale
    pad = -h.shape[1] % BLOCK
    amax = torch.nn.functional.pad(h.abs(), (0, pad)).unflatten(-1, (-1, BLOCK)).amax(-1)
    off = torch.nn.functional.pad(dh, (0, pad)).unflatten(-1, (-1, BLOCK)).amax(-1)
    other = (scale_of((amax - off).clamp_min(0)) != s) | (scale_of(amax + off) != s)
    moved = torch.where(spread(other, h.shape[1]), 2 * step * S, moved)
    return y, dy + moved @ w2.abs().T


def assert_close(got, ref, bound):
    """|got - ref| within the bound and one rounding to got's type."""
    g = got.detach().cpu().double()
    tol = (ref.abs() + bound) * OUT_ROUND[got.dtype] + bound + OUT_FLOOR[got.dtype]
    bad = ~((g - ref).abs() <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} values outside their bound, the worst by "
                           f"{((g - ref).abs() / tol).nan_to_num(posinf=9e9).max():.3g} times")
