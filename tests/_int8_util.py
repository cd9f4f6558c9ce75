"""Definitions of the INT8 operators on CPU tensors, for the GPU tests.

Rows to 8 bits are defined down to their roundings (each fp32 operation is IEEE's,
the mean of squares is taken in 64 bits), so their tests ask for equal bits. The
products are defined in 64 bits; the error that fp32 sums may have is bounded as
in _expert_util."""
import torch

from _expert_util import BLOCK, blocks, product, scale_of  # noqa: F401

FLOOR = 2.0**-96


def int8_rows(v):
    """(int8 values, scales) of fp32 rows; a row with an infinity or a NaN gets a NaN scale and zeros."""
    bad = ~torch.isfinite(v).all(-1, keepdim=True)
    a = torch.where(bad, torch.ones_like(v[..., :1]), v.abs().amax(-1, keepdim=True)).clamp_min(FLOOR)
    full = torch.full_like(a, 127.0)
    q = torch.where(bad, torch.zeros_like(v), torch.round(v * (full / a)))
    return q.to(torch.int8), torch.where(bad, torch.full_like(a, float("nan")), a / full)[..., 0]


def e4m3_rows(v):
    """(e4m3 values, scales) of fp32 rows."""
    K = v.shape[-1]
    w = torch.nn.functional.pad(v, (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))
    bad = ~torch.isfinite(w).all(-1)
    s = scale_of(torch.where(bad, torch.full_like(w[..., 0], float("inf")), w.abs().amax(-1)).double()).float()
    return (w / s[..., None]).flatten(-2)[..., :K].to(torch.float8_e4m3fn), s


def norm(x, residual, weight, eps):
    """(h of x's type, y in fp32)."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    r = (1.0 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + eps)).float()
    return h, (h.float() * r) * weight.float()


def weight(w, s):
    """float64 weights [..., N, K] of int8 values and a scale per channel."""
    return w.double() * s.double()[..., None]


def net(x, w1, w3, w2):
    """(y, bound) of h = silu(x w1^T) * (x w3^T) rounded to bf16, times w2^T, in float64."""
    (g, dg), (u, du) = product(x, w1), product(x, w3)
    sg = g * torch.sigmoid(g)
    h = sg * u
    # |silu'| < 1.1; silu and the two products are fp32 with errors of a few 2^-23, of |g| 2^-23 in the exponent
    dh = 1.1 * dg * (u.abs() + du) + (sg.abs() + 1.1 * dg) * du + h.abs() * (16 + g.abs()) * 2.0**-23
    rounded = h.to(torch.bfloat16).double()
    y, dy = product(rounded, w2)
    # where the fp32 error reaches the edge between two bf16 values, h may round to either
    step = torch.exp2((torch.frexp(h)[1] - 8).double())  # |h| in [2^(e-1), 2^e): steps of 2^(e-8)
    edge = ((h / step - torch.floor(h / step)) - 0.5).abs() * step
    moved = torch.where(edge <= dh, step + dh, torch.zeros_like(h))
    return y, dy + moved @ w2.abs().T
