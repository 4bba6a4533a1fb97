"""The tree entry points refuse bad arguments on the host, before any CUDA call
(CPU only), and the tests' own models agree with one another."""
import random

import pytest


@pytest.fixture(scope="module")
def fa():
    from exact_attention_forward_09_gb300 import build
    build.build()
    import exact_attention_forward_09_gb300 as fa
    fa.lib()
    return fa


P = 1 << 20  # any aligned non-null value: these calls return before any CUDA call


def test_plan_refusals(fa):
    def call(**kw):
        a = dict(parents=P, cu=P, sk=P, B=2, T=9, mask=P, words=1, pos=P)
        a.update(kw)
        return fa.lib().fa_tree_plan(*a.values(), None)

    for kw in (dict(parents=None), dict(cu=None), dict(sk=P + 2), dict(B=-1), dict(T=-1), dict(mask=None), dict(mask=P + 1), dict(words=0),
               dict(words=-1), dict(pos=None)):
        assert call(**kw) == fa.FA_ERR_INVALID_ARG, kw
    for kw in (dict(words=33), dict(B=(1 << 24) + 1), dict(T=(1 << 30) + 1)):
        assert call(**kw) == fa.FA_ERR_UNSUPPORTED, kw
    assert call(B=0, parents=None) == fa.FA_OK
    assert call(T=0, mask=None) == fa.FA_OK


def test_fwd_tree_refusals(fa):
    cache = fa._KV_PACK(P, P, 10, 16, 2, 64, 2048, 1024, 64, 0)

    def call(cache=cache, **kw):
        a = dict(table=P, ts=4, mp=4, cu=P, sk=P, mask=P, words=2, pos=P, B=2, T=9, Hq=4, qs=256, max_q=0, window=5, sinks=0, scale=0.1,
                 ws=P, ws_bytes=1 << 40)
        a.update({k: v for k, v in kw.items() if k in a})
        return fa.lib().fa_fwd_tree(kw.get("q", P), cache, kw.get("o", P), kw.get("lse", P), *a.values(), None)

    for kw in (dict(mask=None), dict(mask=P + 2), dict(words=0), dict(words=-4), dict(pos=P + 2), dict(window=0), dict(sinks=-1),
               dict(scale=float("nan")), dict(Hq=5), dict(q=None), dict(o=P + 8), dict(lse=P + 2), dict(qs=250), dict(T=-1), dict(table=None),
               dict(max_q=-1)):
        assert call(**kw) == fa.FA_ERR_INVALID_ARG, kw
    for kw in (dict(words=33), dict(T=(1 << 30) + 1), dict(Hq=2 * 129)):
        assert call(**kw) == fa.FA_ERR_UNSUPPORTED, kw
    assert call(fa._KV_PACK(P, P, 10, 24, 2, 64, 4096, 2048, 64, 0)) == fa.FA_ERR_UNSUPPORTED
    assert call(T=0, mask=None, q=None) == fa.FA_OK
    assert call(B=0, mask=None, pos=P + 2) == fa.FA_OK


def test_python_refusals(fa):
    import torch
    i = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: fa.tree_plan(i, i, i, 5), lambda: fa.tree_plan(None, i, i, 5),
                 lambda: fa.fwd_tree(x[0], x, x, i[None], i, i, None), lambda: fa.fwd_tree(x[0], x, x, i[None], i, i, i)):
        with pytest.raises(ValueError):
            call()


def test_models_agree():
    import torch
    from tree_util import layout, mask_of, random_tree, sees
    rng = random.Random(1)
    for n in (1, 7, 40, 70):
        parents = random_tree(n, rng)
        rows, depth = layout(parents, 3)
        assert all(len(r) == d + 1 for r, d in zip(rows, depth))
        mask = mask_of(rows, 3)
        for i in range(n):
            assert {k for k in range(96) if int(mask[i, k // 32]) >> (k % 32) & 1} == rows[i]
        see = sees(n, 5, rows, [5 + d for d in depth], 1 << 30, 0)
        assert bool(see[:, :5].all()) and see[:, 5:].sum().item() == sum(len(r) for r in rows)
        line, depth = layout(list(range(-1, n - 1)), 3)
        for window in (1, 4, 1000):  # under a window, nodes lying in a line differ from a chunk in what they see of one another alone
            a = sees(n, 9, line, [9 + d for d in depth], window, 2)
            b = sees(n, 9, None, None, window, 2, chunk=True)
            assert torch.equal(a[:, :9], b[:, :9])


def test_plan_under_a_window_refusals(fa):
    def call(**kw):
        a = dict(parents=P, cu=P, sk=P, B=2, T=9, mask=P, words=1, pos=P, window=4, sinks=0)
        a.update(kw)
        return fa.lib().fa_tree_plan_window(*a.values(), None)

    for kw in (dict(parents=None), dict(mask=P + 1), dict(words=0), dict(pos=None), dict(window=0), dict(window=-1), dict(sinks=-1)):
        assert call(**kw) == fa.FA_ERR_INVALID_ARG, kw
    for kw in (dict(words=33), dict(B=(1 << 24) + 1), dict(T=(1 << 30) + 1)):
        assert call(**kw) == fa.FA_ERR_UNSUPPORTED, kw
    assert call(T=0, mask=None, window=1 << 62, sinks=1 << 62) == fa.FA_OK
