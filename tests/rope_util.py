"""64-bit references of the rotary operators and the error bounds that their
arithmetic gives."""
from __future__ import annotations

import math

import torch

from window_util import HALF_STEP

INTERLEAVED, HALF = 1, 2


def turn(x, cos, sin, layout, inverse=False):
    """Rows of x (any float type) rotated in 64 bits, and the sum of the
    absolute products behind each element (the element itself where it is
    copied).  cos, sin broadcast against x[..., :rope_dim/2]."""
    r = 2 * cos.shape[-1]
    i = torch.arange(r // 2, device=x.device)
    lo, hi = (i, i + r // 2) if layout == HALF else (2 * i, 2 * i + 1)
    x, c, s = x.double(), cos.double(), sin.double()
    if inverse:
        s = -s
    y, size = x.clone(), x.abs()
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    size[..., lo], size[..., hi] = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    return y, size


def check_turned(got, x, cos, sin, layout, what, inverse=False):
    """Two fp32 products, each rounded (2^-24 of it), their sum rounded (2^-24 of
    at most the products' sum), and one rounding to the element type: half a step
    of the value, 2^-25 where fp16 is subnormal.  Copied columns keep their bits."""
    r = 2 * cos.shape[-1]
    ref, size = turn(x, cos, sin, layout, inverse)
    u = HALF_STEP[x.dtype]
    tol = u * ref.abs() + (1 + u) * 2.0 ** -23 * size + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
    off = (got.double() - ref).abs()
    assert got.shape == x.shape and got.dtype == x.dtype, what
    assert bool((off <= tol)[..., :r].all()), f"{what}: worst excess {float((off - tol)[..., :r].max()):.3e}"
    assert torch.equal(got[..., r:].contiguous().view(torch.int16), x[..., r:].contiguous().view(torch.int16)), f"{what}: copied columns"


def frequencies(r, theta, kind="none", factor=1.0, original=0.0, low=0.0, high=0.0, amplitude=1.0):
    """Angles per position, from the definition, in Python's floats."""
    if kind == "base":
        theta = theta * factor ** (r / (r - 2))
    f = [theta ** (-2.0 * i / r) for i in range(r // 2)]
    if kind == "linear":
        return [x / factor for x in f]
    if kind == "turns":
        keep = [(original * x / (2 * math.pi) - low) / (high - low) for x in f]
    elif kind == "index":
        def pair(w):
            return r * math.log(original / (2 * math.pi * w)) / (2 * math.log(theta))
        a, b = max(0, math.floor(pair(high))), min(r - 1, math.ceil(pair(low)))
        keep = [1 - (i - a) / max(b - a, 0.001) for i in range(r // 2)]
    else:
        return f
    keep = [min(1.0, max(0.0, k)) for k in keep]
    return [(1 - k) * x / factor + k * x for x, k in zip(f, keep)]
