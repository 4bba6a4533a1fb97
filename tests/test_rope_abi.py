"""The rotary entry points refuse bad arguments on the host, before any CUDA
call (CPU only), and the host's frequencies follow their definition."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def fa():
    from exact_attention_forward_09_gb300 import build
    build.build()
    import exact_attention_forward_09_gb300 as fa
    fa.lib()
    return fa


P = 1 << 20  # any aligned non-null value: these calls return before any CUDA call
NAN, INF = float("nan"), float("inf")


def _array(fa, **kw):
    a = dict(x=P, y=P, heads=2, xb=1024, xh=512, xn=64, yb=1024, yh=512, yn=64)
    a.update(kw)
    return fa._ROPE_PACK(*[x or 0 for x in a.values()])


def _rope(fa, arrays=None, **kw):
    a = dict(count=1, B=2, N=8, d=64, pos=None, pos_stride=0, offset=0, cos=P, sin=P, length=8, r=64, layout=2, inverse=0, dtype=0)
    a.update(kw)
    return fa.lib().fa_rope(_array(fa) if arrays is None else arrays, *a.values(), None)


def test_rope_refusals(fa):
    bad, unsup = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for kw in (dict(B=-1), dict(N=-1), dict(count=0), dict(count=3), dict(offset=-1), dict(offset=1), dict(length=7), dict(layout=0),
               dict(layout=3), dict(inverse=2), dict(dtype=2), dict(cos=None), dict(sin=P + 8), dict(pos=P + 2), dict(pos_stride=-1),
               dict(length=-1, pos=P)):
        assert _rope(fa, **kw) == bad, kw
    for kw in (dict(d=96), dict(r=8), dict(r=24), dict(r=80), dict(r=0), dict(N=(1 << 30) + 1), dict(B=1 << 30, N=1 << 10),
               dict(length=(1 << 30) + 1)):
        assert _rope(fa, **kw) == unsup, kw
    for kw in (dict(x=0), dict(y=0), dict(x=P + 8), dict(y=P + 2), dict(heads=-1), dict(xn=-64), dict(xn=60), dict(yn=32), dict(yh=0),
               dict(yb=516), dict(xh=1024)):  # (the last: in place with other strides)
        assert _rope(fa, _array(fa, **kw)) == bad, kw
    assert _rope(fa, _array(fa, heads=(1 << 20) + 1)) == unsup
    assert _rope(fa, _array(fa, xb=1 << 38, yb=1 << 38)) == unsup
    assert _rope(fa, B=0) == fa.FA_OK
    assert _rope(fa, N=0, cos=None) == fa.FA_OK
    assert _rope(fa, _array(fa, heads=0, x=0, y=0)) == fa.FA_OK


def _scaling(fa, **kw):
    a = dict(kind=3, factor=8.0, original=1000.0, low=1.0, high=4.0, amplitude=1.0)
    a.update(kw)
    return fa._SCALING_PACK(*a.values())


def _table(fa, sc=None, **kw):
    a = dict(cos=P, sin=P, n=0, r=64, theta=10000.0, start=0)
    a.update(kw)
    return fa.lib().fa_rope_table(*a.values(), sc, None)


def test_table_refusals(fa):
    bad, unsup = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for kw in (dict(n=-1), dict(start=-1), dict(theta=1.0), dict(theta=-5.0), dict(theta=NAN), dict(theta=INF), dict(n=1, cos=None),
               dict(n=1, sin=P + 4)):
        assert _table(fa, **kw) == bad, kw
    for kw in (dict(r=8), dict(r=0), dict(r=272), dict(r=-16), dict(n=(1 << 30) + 1), dict(start=(1 << 30) + 1)):
        assert _table(fa, **kw) == unsup, kw
    for kw in (dict(kind=5), dict(kind=-1), dict(factor=0.5), dict(factor=NAN), dict(original=0.0), dict(original=INF), dict(low=-1.0),
               dict(low=4.0), dict(high=NAN), dict(amplitude=INF), dict(kind=4, low=0.0), dict(kind=2, factor=1e308)):
        assert _table(fa, _scaling(fa, **kw)) == bad, kw
    for kw in (dict(), dict(kind=0, factor=0.0), dict(kind=1, original=0.0), dict(kind=4), dict(amplitude=-1.0)):
        assert _table(fa, _scaling(fa, **kw)) == fa.FA_OK, kw


def test_append_at_refusals(fa):
    cache = fa._KV_PACK(P, P, 10, 16, 2, 64, 2048, 1024, 64, 0)

    def call(**kw):
        a = dict(q=None, k=P, v=P, q_out=None, qs=0, ks=128, vs=128, table=P, ts=4, mp=4, cu=P, sk=P, B=1, T=0, Hq=0, cos=P, sin=P, n=9,
                 r=64, layout=2, pos=P)
        a.update(kw)
        return fa.lib().fa_cache_append_at(cache, *a.values(), None)

    assert call() == fa.FA_OK
    for r in (0, 8, 40, 80, 128):
        assert call(r=r) == fa.FA_ERR_UNSUPPORTED
    assert call(r=0, layout=0) == fa.FA_OK
    assert call(T=1, pos=P + 2) == fa.FA_ERR_INVALID_ARG


def test_the_packed_structures_are_the_header_s(fa):
    class Array(ctypes.Structure):
        _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p)] + [(n, ctypes.c_int64) for n in "abcdefg"]

    class Scaling(ctypes.Structure):
        _fields_ = [("kind", ctypes.c_int)] + [(n, ctypes.c_double) for n in "abcde"]

    assert bytes(Array(1, 2, 3, 4, 5, 6, 7, 8, 9)) == fa._ROPE_PACK(1, 2, 3, 4, 5, 6, 7, 8, 9)
    assert bytes(Scaling(1, 2.0, 3.0, 4.0, 5.0, 6.0)) == fa._SCALING_PACK(1, 2.0, 3.0, 4.0, 5.0, 6.0)


def test_python_refusals(fa):
    import torch
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    for args in ((x, None, (x, x, 2)), (None, None, (x, x, 2))):
        with pytest.raises(ValueError):
            fa.rope(*args)
    for sc in (dict(kind="other"), dict(kind="linear", speed=2), dict(factor=2.0)):
        with pytest.raises(ValueError):
            fa.rope_table(4, 64, scaling=sc, out=(x, x))
    with pytest.raises(ValueError):
        fa.rope_table(4, 64, out=(x, x))


def test_reference_frequencies():
    from rope_util import frequencies
    f = frequencies(64, 10000.0)
    assert f[0] == 1.0 and f[31] == pytest.approx(10000.0 ** (-62 / 64))
    by = frequencies(64, 10000.0, "turns", 8.0, 4096.0, 1.0, 4.0)
    for x, y in zip(f, by):
        turns = 4096.0 * x / (2 * math.pi)
        assert y == pytest.approx(x if turns >= 4 else x / 8 if turns <= 1 else y)
        assert x / 8 <= y <= x


def test_an_amplitude_beyond_fp32_is_refused(fa):
    # (the tables would hold infinities and NaN)
    for a in (3.5e38, -1e39, 1e308):
        assert _table(fa, _scaling(fa, amplitude=a)) == fa.FA_ERR_INVALID_ARG
    for a in (3.4e38, -3.4e38, 1e-45, 0.0):
        assert _table(fa, _scaling(fa, amplitude=a)) == fa.FA_OK
