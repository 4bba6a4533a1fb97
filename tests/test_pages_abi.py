"""The entry points on a cache's pages refuse bad arguments on the host, before
any CUDA call (CPU only)."""
import pytest


@pytest.fixture(scope="module")
def fa():
    from exact_attention_forward_09_gb300 import build
    build.build()
    import exact_attention_forward_09_gb300 as fa
    fa.lib()
    return fa


P = 1 << 20  # any aligned non-null value: these calls return before any CUDA call


def _cache(fa, **kw):
    a = dict(k=P, v=P, n=10, page=16, heads=2, d=64, ps=2048, hs=1024, ts=64, dtype=0)
    a.update(kw)
    return fa._KV_PACK(*a.values())


def test_resize_refusals(fa):
    def call(**kw):
        a = dict(refs=P, n=10, page=16, table=P, ts=4, mp=4, seq=P, want=P, B=2)
        a.update(kw)
        return fa.lib().fa_pages_resize(*a.values(), None)

    for kw in (dict(B=-1), dict(n=0), dict(refs=None), dict(refs=P + 4), dict(table=None), dict(table=P + 2), dict(ts=3), dict(mp=0),
               dict(seq=None), dict(want=P + 1)):
        assert call(**kw) == fa.FA_ERR_INVALID_ARG, kw
    for kw in (dict(page=8), dict(page=48), dict(page=2048), dict(n=1 << 31), dict(B=49153), dict(mp=(1 << 30) + 1, ts=1 << 31)):
        assert call(**kw) == fa.FA_ERR_UNSUPPORTED, kw
    assert call(B=0, refs=None, table=None, seq=None, want=None) == fa.FA_OK


def test_fork_refusals(fa):
    def call(cache=None, **kw):
        a = dict(layers=2, ls=1 << 20, refs=P, table=P, ts=4, mp=4, seq=P, rows=3, src=P, dst=P, fresh=P, n=2)
        a.update(kw)
        return fa.lib().fa_pages_fork(_cache(fa) if cache is None else cache, *a.values(), None)

    for kw in (dict(layers=-1), dict(layers=0), dict(ls=60), dict(ls=32), dict(refs=P + 4), dict(refs=None), dict(table=None), dict(ts=3),
               dict(mp=0), dict(seq=None), dict(rows=-1), dict(rows=0), dict(src=None), dict(dst=P + 2), dict(fresh=None), dict(n=-1)):
        assert call(**kw) == fa.FA_ERR_INVALID_ARG, kw
    for kw in (dict(rows=(1 << 18) + 1), dict(n=16385), dict(layers=32768), dict(ls=1 << 44)):
        assert call(**kw) == fa.FA_ERR_UNSUPPORTED, kw
    for kw in (dict(k=0), dict(v=P + 8), dict(dtype=7), dict(n=0), dict(ts=60)):
        assert call(_cache(fa, **kw)) == fa.FA_ERR_INVALID_ARG, kw
    for kw in (dict(d=96), dict(page=24), dict(heads=1 << 20, page=1024, ps=1 << 36, hs=1 << 16)):
        assert call(_cache(fa, **kw)) == fa.FA_ERR_UNSUPPORTED, kw
    assert call(n=0, src=None, dst=None, refs=None) == fa.FA_OK


def test_copy_refusals(fa):
    def call(cache=None, **kw):
        a = dict(layers=2, ls=1 << 20, src=P, dst=P, n=2)
        a.update(kw)
        return fa.lib().fa_cache_copy(_cache(fa) if cache is None else cache, *a.values(), None)

    for kw in (dict(layers=-1), dict(ls=60), dict(src=None), dict(dst=P + 2), dict(n=-1)):
        assert call(**kw) == fa.FA_ERR_INVALID_ARG, kw
    assert call(n=(1 << 30) + 1) == fa.FA_ERR_UNSUPPORTED
    assert call(_cache(fa, d=256, page=1024, heads=64, ps=1 << 24, hs=1 << 18, ts=256), n=1 << 22) == fa.FA_ERR_UNSUPPORTED
    assert call(_cache(fa, d=32)) == fa.FA_ERR_UNSUPPORTED
    assert call(n=0, src=None) == fa.FA_OK
    assert call(layers=0) == fa.FA_OK


def test_compact_refusals(fa):
    def call(cache=None, **kw):
        a = dict(layers=2, ls=1 << 20, table=P, ts=4, mp=4, first=P, keep=P, ks=5, mk=5, keep_n=P, out=P, B=2)
        a.update(kw)
        return fa.lib().fa_cache_compact(_cache(fa) if cache is None else cache, *a.values(), None)

    for kw in (dict(layers=-1), dict(layers=0), dict(ls=60), dict(table=None), dict(ts=3), dict(mp=0), dict(first=None), dict(keep=None),
               dict(ks=4), dict(mk=-1), dict(keep_n=P + 2), dict(out=None), dict(B=-1)):
        assert call(**kw) == fa.FA_ERR_INVALID_ARG, kw
    for kw in (dict(B=(1 << 24) + 1), dict(mk=(1 << 30) + 1, ks=1 << 31)):
        assert call(**kw) == fa.FA_ERR_UNSUPPORTED, kw
    assert call(_cache(fa, heads=1 << 19, ps=1 << 34, hs=1 << 12), B=1 << 20) == fa.FA_ERR_UNSUPPORTED
    assert call(_cache(fa, d=32)) == fa.FA_ERR_UNSUPPORTED
    assert call(B=0, table=None, first=None) == fa.FA_OK


def test_python_refusals(fa):
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: fa.pages_resize(i, i[None], i, i, 16), lambda: fa.pages_resize(None, i, i, i, 16),
                 lambda: fa.cache_copy(x, x, i, i), lambda: fa.pages_fork(x, x, i, i[None], i, i, i),
                 lambda: fa.cache_compact(x[None], x, i[None], i, i[None], i)):
        with pytest.raises(ValueError):
            call()
