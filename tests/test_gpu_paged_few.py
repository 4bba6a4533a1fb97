"""Paged attention of batches whose sequences bring a few rows each (a token's
query heads of one key/value head, or a few tokens'): every count of rows up
to 16 and just above, both numbers of blocks per SM, masks, and failures."""
import math

import pytest
import torch

import attn_inputs as gen
from window_util import Paged, check_forward, ints, reference

pytestmark = pytest.mark.gpu
ALL = 1 << 30


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _normal(shape, seed, stream, dtype):
    return torch.from_numpy(gen.normal(shape, seed, stream)).to(dtype).cuda()


def _make(lens, Hq, Hkv, d, dtype, page, seed=7, junk=float("nan")):
    seqs = [tuple(_normal((Hkv, nk, d), seed, 10 * b + i, dtype) for i in (1, 2)) for b, (_, nk) in enumerate(lens)]
    cu = [0]
    for nq, _ in lens:
        cu.append(cu[-1] + nq)
    q = _normal((cu[-1], Hq, d), seed, 0, dtype)
    return q, Paged(seqs, page, junk=junk, seed=seed), ints(cu), ints([nk for _, nk in lens]), seqs


def _run(fa, lens, Hq, Hkv, d, dtype=torch.bfloat16, page=16, window=ALL, sinks=0, max_q=1, scale=None):
    q, c, cu, sk, seqs = _make(lens, Hq, Hkv, d, dtype, page)
    o, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device="cuda")
    fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, window=window, sinks=sinks, max_q=max_q, scale=scale, out=o, lse=lse)
    fa.check_device_error()
    at, s = 0, d ** -0.5 if scale is None else scale
    for b, ((nq, nk), (k, v)) in enumerate(zip(lens, seqs)):
        r = slice(at, at + nq)
        ref = reference(q[r].transpose(0, 1), k, v, window, sinks, s)
        check_forward(o[r].transpose(0, 1), lse[r].transpose(0, 1), ref, q.dtype, d, nk,
                      f"Hq{Hq} Hkv{Hkv} d{d} w{window} s{sinks} max_q{max_q} sequence {b} ({nq}, {nk})")
        at += nq


ONE = [(1, n) for n in (1, 31, 32, 33, 64, 127, 128, 129, 255, 700, 0, 1500)]


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_heads_of_one_token(fa, d, g):
    _run(fa, ONE, 2 * g, 2, d)
    _run(fa, ONE[:4] + [(0, 40)] + ONE[4:], g, 1, d, torch.float16, page=64, max_q=0)  # as many tokens as sequences, or fewer


@pytest.mark.parametrize("nq", [2, 3, 4, 5, 8, 9, 16, 17])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_few_tokens(fa, d, nq):
    lens = [(nq, nq), (1, 500), (nq, 129), (nq - 1, 1000), (nq, 2000), (nq, nq - 2)]
    for g in (1, 2, 3):
        _run(fa, lens, g, 1, d, max_q=nq)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_sequences_that_bring_more_than_announced(fa, d):
    _run(fa, [(1, 300), (50, 400), (1, 7), (300, 300)], 8, 2, d, max_q=1)
    _run(fa, [(0, 9), (7, 200), (0, 5), (0, 100), (0, 0), (0, 1), (0, 2)], 8, 2, d, max_q=0)


@pytest.mark.parametrize("heads", [1, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_sequences(fa, d, heads):
    # with 8 heads more units than SMs: two blocks per SM at d = 128
    lens = [(1, 1 + (b * 53) % 900) for b in range(40)]
    _run(fa, lens, 4 * heads, heads, d)
    _run(fa, lens, 8 * heads, heads, d, torch.float16, page=32, window=200, sinks=3)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (31, 2), (33, 0), (128, 32), (129, 33), (500, 20), (200, 300)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows_and_sinks(fa, d, window, sinks):
    _run(fa, [(1, 40), (1, 129), (2, 1000), (1, 2500), (3, 600), (2, 1)], 8, 2, d, window=window, sinks=sinks, max_q=3)


@pytest.mark.parametrize("scale", [0.0, -0.3, 0.6])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales(fa, d, scale):
    _run(fa, [(1, 400), (2, 200), (1, 3)], 8, 2, d, window=150, sinks=2, max_q=2, scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_growing_maximum(fa, d):
    """Scores that rise by far more than the rescaling threshold from key to key, and fall the other way."""
    n = 700
    ramp = torch.linspace(-6, 6, n).view(1, n, 1).expand(1, n, d)
    for sign in (1.0, -1.0):
        seqs = [((sign * ramp).to(torch.bfloat16).cuda().contiguous(), _normal((1, n, d), 9, 2, torch.bfloat16))]
        c = Paged(seqs, 32)
        q = torch.ones((1, 4, d), dtype=torch.bfloat16, device="cuda")
        q[0, 1] = 0.01
        q[0, 2] = -1
        o, lse = fa.fwd_paged(q, c.k, c.v, c.table, ints([0, 1]), ints([n]), max_q=1)
        fa.check_device_error()
        ref = reference(q.transpose(0, 1), *seqs[0], ALL, 0, d ** -0.5)
        check_forward(o.transpose(0, 1), lse.transpose(0, 1), ref, torch.bfloat16, d, n, f"d{d} sign {sign}")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_nan_query_stays_in_its_row(fa, d):
    q, c, cu, sk, _ = _make([(1, 900), (2, 300)], 4, 1, d, torch.float16, 32)
    want = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, max_q=2)
    q[2, 1] = float("nan")
    o, lse = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, max_q=2)
    fa.check_device_error()
    assert bool(o[2, 1].isnan().all()) and math.isnan(float(lse[2, 1]))
    o[2, 1], lse[2, 1] = want[0][2, 1], want[1][2, 1]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("heads", [1, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_wait_that_runs_out_is_reported(fa, d, heads):
    """A key or value slot that the first block never fills: every wait ends, the four warps that join a
    unit's copies leave together, and the next call is right."""
    q, c, cu, sk, _ = _make([(1, 600)] * 30, 4 * heads, heads, d, torch.bfloat16, 64)
    want = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, max_q=1)
    fa.check_device_error()
    assert fa.lib().fa_debug_inject(1) == fa.FA_OK
    fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, max_q=1)
    with pytest.raises(fa.FaError) as e:
        fa.check_device_error()
    assert e.value.status == fa.FA_ERR_TIMEOUT
    got = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, max_q=1)
    fa.check_device_error()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
