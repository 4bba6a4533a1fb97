"""Seeded random shapes of the windowed and paged operators: sizes, head
groups, windows, sinks, layouts and batches from a fixed generator, every
element against the 64-bit reference within the derived bounds."""
import math
import random

import pytest
import torch

import attn_inputs as gen
from window_util import Paged, check_backward, check_forward, ints, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _normal(shape, seed, stream, dtype):
    return torch.from_numpy(gen.normal(shape, seed, stream)).to(dtype).cuda()


def _spread(r, lo, hi):
    return min(hi, max(lo, int(math.exp(r.uniform(math.log(lo), math.log(hi + 1))))))


def _mask(r, n):
    return r.choice([1, _spread(r, 2, 2 * n + 2), _spread(r, 2, n + 2), 1 << 33]), r.choice([0, 0, 1, 4, 32, 100, 129, 400])


@pytest.mark.parametrize("seed", range(60))
def test_random_window(fa, seed):
    r = random.Random(seed)
    backward = seed % 2 == 0
    d = r.choice([64, 128] if backward else [64, 128, 256])
    dtype = r.choice([torch.bfloat16, torch.float16])
    Hkv, g, B = r.choice([1, 2, 3]), r.choice([1, 2, 4, 5]), r.choice([1, 1, 2])
    Nk = _spread(r, 1, 1500)
    Nq = r.choice([Nk, _spread(r, 1, Nk), _spread(r, 1, 900)])
    w, sinks = _mask(r, Nk)
    scale = r.choice([None, None, 0.2, -0.15, 0.0])
    q, do = (_normal((B, Hkv * g, Nq, d), seed, i, dtype) for i in (0, 3))
    k, v = (_normal((B, Hkv, Nk, d), seed, i, dtype) for i in (1, 2))
    o, lse = fa.fwd_window(q, k, v, w, sinks, scale=scale)
    grads = fa.bwd_window(q, k, v, o, lse, do, w, sinks, scale=scale) if backward else None
    fa.check_device_error()
    s = d ** -0.5 if scale is None else scale
    for b in range(B):
        what = f"seed {seed}: B{B} Hkv{Hkv} g{g} Nq{Nq} Nk{Nk} d{d} w{w} s{sinks} scale {scale} {dtype}"
        ref = reference(q[b], k[b], v[b], w, sinks, s, do[b] if backward else None)
        check_forward(o[b], lse[b], ref, dtype, d, Nk, what)
        if backward:
            check_backward([x[b] for x in grads], q[b], k[b], v[b], do[b], o[b], w, sinks, s, ref, dtype, what)


@pytest.mark.parametrize("seed", range(80))
def test_random_paged(fa, seed):
    r = random.Random(1000 + seed)
    d, dtype, page = r.choice([64, 128, 256]), r.choice([torch.bfloat16, torch.float16]), r.choice([16, 32, 64, 128, 256, 512])
    Hkv, g = r.choice([1, 2, 3, 8]), r.choice([1, 2, 3, 4, 7, 8, 16])
    B = _spread(r, 1, 20)
    chunk = r.choice([1, 1, 4, 40, 300])
    lens = []
    for _ in range(B):
        nq = 0 if r.random() < 0.1 else r.randint(1, chunk)
        lens.append((nq, max(nq if r.random() < 0.9 else nq // 2, _spread(r, 1, 3000 if B < 8 else 700))))
    w, sinks = _mask(r, 800)
    scale = r.choice([None, None, 0.2, -0.15])
    max_q = r.choice([0, max(nq for nq, _ in lens), 1])
    seqs = [tuple(_normal((Hkv, nk, d), seed, 10 * b + i, dtype) for i in (1, 2)) for b, (_, nk) in enumerate(lens)]
    c = Paged(seqs, page, r.choice(["hnd", "nhd", "both"]), seed=seed)
    cu = [0]
    for nq, _ in lens:
        cu.append(cu[-1] + nq)
    q = _normal((cu[-1] + 1, Hkv * g, d), seed, 0, dtype)[:cu[-1]]
    o, lse = fa.fwd_paged(q, c.k, c.v, c.table, ints(cu), ints([nk for _, nk in lens]), window=w, sinks=sinks, scale=scale, max_q=max_q)
    fa.check_device_error()
    s = d ** -0.5 if scale is None else scale
    for b, ((nq, nk), (k, v)) in enumerate(zip(lens, seqs)):
        if nq:
            rows = slice(cu[b], cu[b] + nq)
            ref = reference(q[rows].transpose(0, 1), k, v, w, sinks, s)
            check_forward(o[rows].transpose(0, 1), lse[rows].transpose(0, 1), ref, dtype, d, nk,
                          f"seed {seed}: sequence {b} ({nq}, {nk}) Hkv{Hkv} g{g} d{d} page{page} w{w} s{sinks} max_q{max_q}")
