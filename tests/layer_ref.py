"""64-bit references and error bounds of the feed-forward operators (test infrastructure).

U[dtype] is the unit roundoff of the 16-bit type (bf16 8, fp16 11 significand
bits): a result rounded once is within U |ref| of the unrounded one, fp16 below
its normal range within half its smallest subnormal.
"""
import math

import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}
EPS32 = 2.0 ** -24  # unit roundoff of fp32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]  # by their MC2_ACT_* value


def rand(seed, *shape, std=1.0, dtype="bf16"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(DT[dtype])


def check(got, ref, bound, what):
    """|got - ref| <= bound element by element (ref, bound in 64 bits on the CPU)."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.numel()} outside the bound; first at {i}: got "
                             f"{got[i].item()!r} ref {ref[i].item()!r} bound {bound[i].item()!r}")


def rounded(ref, dtype):
    """Bound of one rounding of ref to the 16-bit type."""
    return U[dtype] * ref.abs() + TINY[dtype]


def act(z, name):
    """(act(z), act'(z)) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    t = torch.tanh(u)
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


# The kernels' activations are within ACT_ERR (1 + |z|) of the exact ones, and
# their slopes within ACT_ERR (1 + |z|)^3 (the argument of the tanh form's
# exponential is a cubic): the erfc formula's 1.5e-7 and a few roundings of
# fp32 with exponential and reciprocal of 1 ulp.
ACT_ERR = 2e-6


def norm(x, residual, weight, eps):
    s = x.double() if residual is None else x.double() + residual.double()
    rstd = 1 / torch.sqrt((s * s).mean(-1) + eps)
    return s, rstd, s * rstd[..., None] * weight.double()


def norm_grad(dout, dsum, s, weight, rstd):
    s, g = s.double(), dout.double() * weight.double()
    r = rstd.double()[:, None]
    dx = r * (g - s * r * r * (g * s).mean(-1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.double()
    return dx, (dout.double() * s * r).sum(0)


def spans(offsets, m):
    """[(group, begin, end)] as the kernels read the ranges."""
    out, at = [], 0
    for g, e in enumerate(offsets[1:]):
        e = min(max(e, at), m)
        out.append((g, at, e))
        at = e
    return out
