"""Windowed attention of few queries over many keys, where a cluster of blocks
shares each query tile's keys and joins the parts."""
import math

import pytest
import torch

import attn_inputs as gen
from window_util import check_backward, check_forward, reference

pytestmark = pytest.mark.gpu
ALL = 1 << 30


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _inputs(B, Hq, Hkv, Nq, Nk, d, seed, dtype):
    shapes = ((B, Hq, Nq, d), (B, Hkv, Nk, d), (B, Hkv, Nk, d), (B, Hq, Nq, d))
    return [torch.from_numpy(gen.normal(s, seed, i)).to(dtype).cuda() for i, s in enumerate(shapes)]


def _check(fa, B, Hq, Hkv, Nq, Nk, d, window, sinks, dtype=torch.bfloat16, scale=None, seed=61):
    q, k, v, _ = _inputs(B, Hq, Hkv, Nq, Nk, d, seed, dtype)
    o, lse = torch.full_like(q, float("nan")), torch.full((B, Hq, Nq), float("nan"), device="cuda")
    fa.fwd_window(q, k, v, window, sinks, scale=scale, out=o, lse=lse)
    fa.check_device_error()
    s = d ** -0.5 if scale is None else scale
    for b in range(B):
        check_forward(o[b], lse[b], reference(q[b], k[b], v[b], window, sinks, s), dtype, d, Nk,
                      f"B{B} Hq{Hq} Hkv{Hkv} {Nq}x{Nk} d{d} w{window} s{sinks} {dtype} scale {scale}")


@pytest.mark.parametrize("Nq", [1, 2, 127, 128, 129, 300])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_few_queries(fa, d, Nq):
    for Nk in (512, 600, 1024, 1025, 4000):       # 4 and 8 blocks to a cluster
        _check(fa, 1, 2, 1, Nq, Nk, d, ALL, 0)
    _check(fa, 2, 3, 3, Nq, 3000, d, 700, 0, torch.float16)
    _check(fa, 1, 4, 2, Nq, 5000, d, 1500, 33)


@pytest.mark.parametrize("heads", [15, 16, 36, 37, 76, 77])
@pytest.mark.parametrize("d", [64, 256])
def test_as_many_clusters_as_run_at_once(fa, d, heads):
    _check(fa, 1, heads, 1, 5, 1100, d, ALL, 0)
    _check(fa, 1, heads, 1, 128, 1100, d, 500, 9)


@pytest.mark.parametrize("window,sinks", [(1, 600), (20, 513), (400, 1), (400, 32), (400, 33), (513, 0), (600, 700), (1000, 128)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_runs_that_rows_do_not_see(fa, d, window, sinks):
    # rows of one tile whose windows start in different runs, sinks seen alone, the gap between
    for Nq, Nk in ((1, 3000), (130, 3000), (700, 1500)):
        _check(fa, 1, 2, 1, Nq, Nk, d, window, sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_before_the_first_key(fa, d):
    _check(fa, 1, 2, 1, 700, 520, d, ALL, 0)
    _check(fa, 1, 2, 1, 1000, 600, d, 550, 4, torch.float16)
    _check(fa, 1, 1, 1, 2000, 513, d, 513, 513)


@pytest.mark.parametrize("scale", [0.0, -0.3, 0.5])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales(fa, d, scale):
    _check(fa, 1, 2, 2, 60, 2000, d, 900, 3, scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_nan_query_stays_in_its_row(fa, d):
    q, k, v, _ = _inputs(1, 2, 1, 40, 2000, d, 63, torch.bfloat16)
    want = fa.fwd_window(q, k, v, ALL, 0)
    q2 = q.clone()
    q2[0, 1, 7] = float("nan")
    o, lse = fa.fwd_window(q2, k, v, ALL, 0)
    fa.check_device_error()
    assert bool(o[0, 1, 7].isnan().all()) and math.isnan(float(lse[0, 1, 7]))
    o[0, 1, 7], lse[0, 1, 7] = want[0][0, 1, 7], want[1][0, 1, 7]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_what_the_window_hides_may_be_anything(fa):
    # the first query, at position 3990, sees keys from 2991 on and the five sinks
    q, k, v, _ = _inputs(1, 4, 2, 10, 4000, 128, 65, torch.float16)
    want = fa.fwd_window(q, k, v, 1000, 5)
    k[:, :, 5:2991] = float("nan")
    v[:, :, 128:2944] = float("inf")  # key tiles that are not visited
    o, lse = fa.fwd_window(q, k, v, 1000, 5)
    fa.check_device_error()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("d", [64, 128])
def test_with_its_backward(fa, d):
    q, k, v, do = _inputs(1, 4, 1, 200, 1500, d, 67, torch.bfloat16)
    o, lse = fa.fwd_window(q, k, v, 1200, 6)
    grads = fa.bwd_window(q, k, v, o, lse, do, 1200, 6)
    fa.check_device_error()
    ref = reference(q[0], k[0], v[0], 1200, 6, d ** -0.5, do[0])
    check_backward([x[0] for x in grads], q[0], k[0], v[0], do[0], o[0], 1200, 6, d ** -0.5, ref, torch.bfloat16, f"d{d}")


def test_same_bits_on_two_streams_and_from_a_graph(fa):
    q, k, v, _ = _inputs(1, 8, 2, 90, 3000, 128, 69, torch.bfloat16)
    want = fa.fwd_window(q, k, v, ALL, 0)
    g = torch.cuda.CUDAGraph()
    outs = [(torch.empty_like(q), torch.empty((1, 8, 90), device="cuda")) for _ in range(2)]
    with torch.cuda.graph(g):
        for o, lse in outs:
            fa.fwd_window(q, k, v, ALL, 0, out=o, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.replay()
        other = fa.fwd_window(q, k, v, ALL, 0)
    here = fa.fwd_window(q, k, v, ALL, 0)
    torch.cuda.synchronize()
    fa.check_device_error()
    for o, lse in outs + [other, here]:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_wait_that_runs_out_is_reported(fa, d):
    """The first block never fills a key slot; its wait ends, and so does every block of its cluster."""
    q, k, v, _ = _inputs(1, 2, 1, 50, 3000, d, 71, torch.bfloat16)
    want = fa.fwd_window(q, k, v, ALL, 0)
    fa.check_device_error()
    fa.lib().fa_debug_inject(1)
    fa.fwd_window(q, k, v, ALL, 0)
    with pytest.raises(fa.FaError):
        fa.check_device_error()
    o, lse = fa.fwd_window(q, k, v, ALL, 0)
    fa.check_device_error()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
