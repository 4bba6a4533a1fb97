"""The windowed and paged entry points refuse bad arguments on the host,
before any CUDA call (CPU only)."""
import ctypes

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


def _window(fa, **kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, B=1, Hq=4, Hkv=2, Nq=8, Nk=16, d=64, window=4, sinks=1, scale=0.1, dtype=0)
    a.update(kw)
    return fa.lib().fa_fwd_window(*a.values(), None)


def test_fwd_window_refusals(fa):
    bad, unsup = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(scale=NAN), dict(scale=INF), dict(dtype=2), dict(dtype=-1),
               dict(B=-1), dict(Nq=-1), dict(Hq=5), dict(Hkv=0), dict(Nk=0), dict(q=None), dict(k=P + 8), dict(o=P + 2),
               dict(lse=None)):
        assert _window(fa, **kw) == bad, kw
    for kw in (dict(d=96), dict(d=32), dict(Nk=(1 << 30) + 1), dict(Nq=(1 << 30) + 1, Nk=1 << 30)):
        assert _window(fa, **kw) == unsup, kw
    assert _window(fa, B=0, q=None, k=None, v=None, o=None, lse=None) == fa.FA_OK
    assert _window(fa, Nq=0, q=None, o=None, lse=None) == fa.FA_OK


def _bwd(fa, **kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, do=P, dq=P, dk=P, dv=P, B=1, Hq=4, Hkv=2, Nq=8, Nk=16, d=64, window=4, sinks=1, scale=0.1,
             dtype=0, ws=P, ws_bytes=1 << 30)
    a.update(kw)
    return fa.lib().fa_bwd_window(*a.values(), None)


def test_bwd_window_refusals(fa):
    bad, unsup = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for kw in (dict(window=0), dict(sinks=-1), dict(scale=NAN), dict(dtype=2), dict(B=-1), dict(Hq=5), dict(Hkv=0), dict(Nk=0),
               dict(q=None), dict(do=P + 8), dict(dk=None), dict(dv=P + 4), dict(lse=P + 4), dict(ws=None), dict(ws=P + 16),
               dict(ws_bytes=100)):
        assert _bwd(fa, **kw) == bad, kw
    for kw in (dict(d=96), dict(d=256), dict(Nk=(1 << 30) + 1)):
        assert _bwd(fa, **kw) == unsup, kw
    none = {n: None for n in ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv", "ws")}
    assert _bwd(fa, **none, B=0) == fa.FA_OK
    n = ctypes.c_size_t(3)
    size = fa.lib().fa_bwd_window_workspace_bytes
    assert size(1, 4, 2, 8, 16, 64, 0, 0, ctypes.byref(n)) == bad
    assert size(1, 4, 2, 8, 16, 64, 4, -1, ctypes.byref(n)) == bad
    assert size(1, 4, 3, 8, 16, 64, 4, 0, ctypes.byref(n)) == bad
    assert size(1, 4, 2, 8, 16, 256, 4, 0, ctypes.byref(n)) == unsup
    assert size(1, 4, 2, 8, 16, 64, 4, 0, None) == bad
    # without sinks, or where a window covers everything: what the causal backward needs
    base = fa.bwd_workspace_bytes(2, 8, 3000, 128)
    assert fa.bwd_window_workspace_bytes(2, 8, 2, 3000, 3000, 128, 100, 0) == base
    assert fa.bwd_window_workspace_bytes(2, 8, 2, 3000, 3000, 128, 3000, 4) == base
    # with them: shares of the sink tiles, bounded whatever the sizes
    for args in ((2, 8, 2, 3000, 3000, 128, 100, 4), (1, 8, 8, 100000, 100000, 128, 1, 1), (1, 8, 1, 9000, 9000, 64, 10, 9000)):
        more = fa.bwd_window_workspace_bytes(*args) - fa.bwd_workspace_bytes(args[0], args[1], args[3], args[5])
        assert 0 <= more <= 128 << 20


def _cache(fa, **kw):
    a = dict(k=P, v=P, num_pages=10, page_size=16, heads=2, d=64, page_stride=2 * 16 * 64, head_stride=16 * 64,
             token_stride=64, dtype=0)
    a.update(kw)
    return fa._KvCache(*a.values())


def test_the_packed_cache_is_the_structure(fa):
    v = (P, 2 * P, 10, 16, 2, 64, 2048, 1024, 64, 1)
    assert fa._KV_PACK(*v) == bytes(fa._KvCache(*v)) and len(fa._KV_PACK(*v)) == ctypes.sizeof(fa._KvCache)


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=P + 8), dict(num_pages=0), dict(heads=0), dict(page_size=0), dict(dtype=3),
              dict(token_stride=60), dict(token_stride=68), dict(head_stride=1020), dict(head_stride=0), dict(page_stride=-64),
              dict(token_stride=32)]
UNSUPPORTED_CACHES = [dict(d=96), dict(page_size=8), dict(page_size=48), dict(page_size=2048), dict(num_pages=1 << 31),
                      dict(page_stride=1 << 38)]


def _paged(fa, cache=None, **kw):
    a = dict(q=P, cache=None, o=P, lse=P, table=P, table_stride=4, max_pages=4, cu_q=P, seq_k=P, B=2, T=5, Hq=4, q_stride=256,
             max_q=0, window=1 << 30, sinks=0, scale=0.1, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    a["cache"] = bytes(_cache(fa, **(cache or {})))
    return fa.lib().fa_fwd_paged(*a.values(), None)


def test_fwd_paged_refusals(fa):
    bad, unsup = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for c in BAD_CACHES:
        assert _paged(fa, cache=c) == bad, c
    for c in UNSUPPORTED_CACHES:
        assert _paged(fa, cache=c) == unsup, c
    for kw in (dict(window=0), dict(sinks=-1), dict(scale=NAN), dict(B=-1), dict(T=-1), dict(max_q=-1), dict(Hq=5), dict(q=None),
               dict(q=P + 8), dict(o=P + 8), dict(lse=P + 2), dict(lse=None), dict(table=None), dict(table=P + 2),
               dict(cu_q=None), dict(seq_k=None), dict(max_pages=0), dict(table_stride=3), dict(q_stride=255),
               dict(q_stride=260)):
        assert _paged(fa, **kw) == bad, kw
    for kw in (dict(Hq=2 * 129, q_stride=258 * 64), dict(T=(1 << 30) + 1), dict(B=1 << 25), dict(q_stride=1 << 38)):
        assert _paged(fa, **kw) == unsup, kw
    none = dict(q=None, o=None, lse=None, table=None, cu_q=None, seq_k=None, ws=None, ws_bytes=0)
    for kw in (dict(T=0), dict(B=0), dict(Hq=0)):
        assert _paged(fa, **none, **kw) == fa.FA_OK
    n = ctypes.c_size_t(3)
    assert fa.lib().fa_paged_workspace_bytes(96, ctypes.byref(n)) == unsup
    assert fa.lib().fa_paged_workspace_bytes(64, None) == bad
    assert fa.lib().fa_fwd_paged(P, None, P, P, P, 4, 4, P, P, 2, 5, 4, 256, 0, 1, 0, 0.1, P, 1 << 40, None) == bad


def _append(fa, cache=None, **kw):
    a = dict(cache=None, q=P, k=P, v=P, q_out=P, q_stride=256, k_stride=128, v_stride=128, table=P, table_stride=4, max_pages=4,
             cu_q=P, seq_k=P, B=2, T=5, Hq=4, cos=P, sin=P, rope_len=100, layout=fa.FA_ROPE_HALF)
    a.update(kw)
    a["cache"] = bytes(_cache(fa, **(cache or {})))
    return fa.lib().fa_cache_append(*a.values(), None)


def test_cache_append_refusals(fa):
    bad, unsup = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for c in BAD_CACHES:
        assert _append(fa, cache=c) == bad, c
    for c in UNSUPPORTED_CACHES:
        assert _append(fa, cache=c) == unsup, c
    for kw in (dict(layout=3), dict(layout=-1), dict(cos=None), dict(sin=P + 4), dict(k=None), dict(v=P + 8), dict(q=None),
               dict(q_out=None), dict(q_out=P + 8), dict(q_stride=128), dict(k_stride=100), dict(v_stride=132), dict(B=-1),
               dict(T=-1), dict(rope_len=-1), dict(Hq=-1), dict(table=None), dict(cu_q=P + 2), dict(max_pages=0)):
        assert _append(fa, **kw) == bad, kw
    assert _append(fa, T=0, q=None, k=None, v=None, q_out=None, table=None) == fa.FA_OK


def test_unknown_status_and_index_status(fa):
    assert fa.lib().fa_status_string(fa.FA_ERR_INDEX).decode().startswith("FA_ERR_INDEX")
