"""The angle tables (fa_rope_table) at positions far out, against sixty decimal
digits, within the bound that the header states."""
import decimal
import math
from decimal import Decimal as D

import pytest
import torch

pytestmark = pytest.mark.gpu
PI = D("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def frequencies(r, theta, kind="none", factor=1.0, original=0.0, low=0.0, high=0.0, amplitude=1.0):
    """Angles per position, from the definition."""
    theta, s, original, low, high = (D(x) for x in (theta, factor, original, low, high))
    if kind == "base":
        theta = theta * s ** (D(r) / (r - 2))
    f = [theta ** (D(-2 * i) / r) for i in range(r // 2)]
    if kind == "linear":
        return [x / s for x in f]
    if kind == "turns":
        keep = [(original * x / (2 * PI) - low) / (high - low) for x in f]
    elif kind == "index":
        def pair(w):
            return r * (original / (2 * PI * w)).ln() / (2 * theta.ln())
        a, b = max(0, math.floor(pair(high))), min(r - 1, math.ceil(pair(low)))
        keep = [1 - (i - a) / max(D(b - a), D(0.001)) for i in range(r // 2)]
    else:
        return f
    keep = [min(D(1), max(D(0), k)) for k in keep]
    return [(1 - k) * x / s + k * x for x, k in zip(f, keep)]


def cos_sin(angle):
    """Both to the last places of a double, small values included: the nearest quarter turn is taken off first."""
    q = (2 * angle / PI).to_integral_value()
    x = float(angle - q * PI / 2)
    c, s = math.cos(x), math.sin(x)
    return ((c, s), (-s, c), (-c, -s), (s, -c))[int(q) % 4]


SCALINGS = [dict(kind="none"), dict(kind="linear", factor=3.0), dict(kind="base", factor=8.0),
            dict(kind="turns", factor=8.0, original=8192, low=1.0, high=4.0), dict(kind="turns", factor=2.0, original=1e308, low=0.0, high=1e-3),
            dict(kind="index", factor=40.0, original=4096, low=1.0, high=32.0, amplitude=0.1 * math.log(40.0) + 1.0)]


@pytest.mark.parametrize("sc", SCALINGS, ids=lambda sc: "-".join(str(x) for x in sc.values()))
@pytest.mark.parametrize("r,theta", [(16, 10000.0), (64, 500000.0), (96, 1e6), (128, 10000.0), (256, 1.5)])
@pytest.mark.parametrize("start", [0, 1 << 17, (1 << 26) + 1, (1 << 30) - 40])
def test_tables_far_out(fa, start, r, theta, sc):
    """Two units of fp32's last place.  Relative to the value, in 2^-24: a cosine of a rest of up to pi/4 is off by 0.8
    through the rest's own rounding, 0.5 through its square's, 0.2 through the polynomial (9.1e-9) and 1 through the last
    sum; a sine by 1, 0.3, 0.05 and 1; an amplitude adds 1.  That is less than 4, two units where they are smallest.
    Beside it the frequency, rounded to 2^-64 of a turn (2^-62.3 radians a position), and the rest's last six bits of
    those 64, which are left out (2^-55.3 radians).  The reference itself is off by some 2^-53 of the value."""
    n = 40
    with decimal.localcontext() as context:
        context.prec = 60
        f = frequencies(r, theta, **sc)
        amp = sc.get("amplitude", 1.0)
        ref = torch.tensor([[cos_sin(x * p) for x in f] for p in range(start, start + n)], dtype=torch.float64) * amp
    got = torch.stack(fa.rope_table(n, r, theta, scaling=sc, start=start), -1).cpu().double()
    fa.check_device_error()
    p = torch.arange(start, start + n, dtype=torch.float64)[:, None, None]
    tol = (2.0 ** -22 + 2.0 ** -50) * ref.abs() + abs(amp) * (p + 128) * 2.0 ** -62
    off = (got - ref).abs()
    assert bool((off <= tol).all()), f"worst: {float((off / tol).max()):.3g} times the bound"
