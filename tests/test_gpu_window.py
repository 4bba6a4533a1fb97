"""Attention under a sliding window with sinks (fa_fwd_window) against the
64-bit reference, on every element, within bounds derived from the kernel's
arithmetic (window_util.check_forward)."""
import math

import pytest
import torch

import attn_inputs as gen
from window_util import check_forward, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _inputs(B, Hq, Hkv, Nq, Nk, d, seed, dtype):
    return [torch.from_numpy(gen.normal(s, seed, i)).to(dtype).cuda()
            for i, s in enumerate([(B, Hq, Nq, d), (B, Hkv, Nk, d), (B, Hkv, Nk, d)])]


def _check(fa, case, dtype, scale=None, window=None):
    B, Hq, Hkv, Nq, Nk, d, w, sinks = case
    q, k, v = _inputs(B, Hq, Hkv, Nq, Nk, d, 400 + Nq + Nk + w % 1000, dtype)
    o, lse = fa.fwd_window(q, k, v, w, sinks, scale=scale)
    fa.check_device_error()
    s = 1 / math.sqrt(d) if scale is None else scale
    for b in range(B):
        ref = reference(q[b], k[b], v[b], w, sinks, s)
        check_forward(o[b], lse[b], ref, dtype, d, Nk, f"{case} {dtype} batch {b}")


CASES = [
    # B, Hq, Hkv, Nq, Nk, d, window, sinks
    (1, 2, 1, 1, 1, 64, 1, 0),             # one token
    (2, 4, 2, 1, 700, 128, 100, 3),        # one query, sinks and window far apart
    (1, 2, 2, 256, 256, 128, 1, 0),        # each query sees itself alone
    (1, 2, 1, 300, 300, 64, 1, 1),
    (1, 4, 2, 300, 130, 128, 50, 2),       # queries before the first key see none
    (1, 2, 1, 200, 3, 256, 7, 1),
    (2, 4, 4, 640, 640, 128, 128, 0),      # window edges on, before and behind a tile edge
    (1, 4, 1, 777, 777, 128, 127, 4),
    (1, 4, 1, 777, 777, 64, 129, 4),
    (1, 4, 2, 777, 901, 256, 130, 4),
    (1, 3, 1, 1000, 1000, 128, 200, 127),  # sinks that end before, on and behind a tile edge
    (1, 3, 1, 1000, 1000, 64, 200, 128),
    (1, 3, 1, 1000, 1000, 128, 200, 129),
    (1, 2, 2, 1500, 1500, 256, 300, 400),  # several tiles of sinks
    (1, 2, 1, 900, 900, 128, 100, 900),    # every key a sink
    (1, 2, 1, 900, 900, 128, 1 << 40, 5),  # a window over everything
    (1, 2, 1, 513, 2049, 64, 1024, 16),    # a chunk at the end of a longer sequence
    (1, 2, 1, 129, 2500, 256, 333, 1),
    (3, 6, 2, 383, 1021, 128, 255, 64),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B{}_Hq{}_Hkv{}_Nq{}_Nk{}_d{}_w{}_s{}".format(*c))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_window_forward(fa, case, dtype):
    _check(fa, case, dtype)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_window_forward_many_units(fa, d):
    # more units than SMs, so that CTAs take over further units
    _check(fa, (2, 16, 4, 2600, 2600, d, 700, 9), torch.bfloat16)


@pytest.mark.parametrize("scale", [0.0, -0.2, 0.7])
@pytest.mark.parametrize("d", [64, 256])
def test_window_forward_scales(fa, scale, d):
    _check(fa, (1, 4, 2, 500, 600, d, 140, 5), torch.bfloat16, scale=scale)
    _check(fa, (1, 2, 2, 200, 60, d, 20, 2), torch.float16, scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_window_over_everything_is_causal(fa, d):
    q, k, v = _inputs(2, 4, 2, 700, 900, d, 21, torch.bfloat16)
    o1, l1 = fa.fwd_gqa(q, k, v, causal=True)
    o2, l2 = fa.fwd_window(q, k, v, 900, 0)
    fa.check_device_error()
    # the same online softmax over the same tiles in the same order
    assert (o1.float() - o2.float()).abs().max().item() <= 2.0 ** -7
    assert (l1 - l2).abs().max().item() <= 1e-5


def test_tiles_outside_every_window_are_not_read(fa):
    B, Hq, Hkv, Nq, Nk, d, w, sinks = 1, 4, 2, 256, 2048, 128, 256, 4
    q, k, v = _inputs(B, Hq, Hkv, Nq, Nk, d, 23, torch.bfloat16)
    ref = reference(q[0], k[0], v[0], w, sinks, 1 / math.sqrt(d))
    # the first query's window starts at 2048 - 256 - 256 + 1 = 1537, in tile 12
    for x in (k, v):
        x[:, :, 128:1536] = float("nan")
    o, lse = fa.fwd_window(q, k, v, w, sinks)
    fa.check_device_error()
    check_forward(o[0], lse[0], ref, torch.bfloat16, d, Nk, "NaN behind the window")


def test_window_outputs_in_place_and_empty(fa):
    q, k, v = _inputs(1, 2, 1, 100, 100, 64, 25, torch.bfloat16)
    o, lse = torch.empty_like(q), torch.empty((1, 2, 100), device="cuda")
    r = fa.fwd_window(q, k, v, 30, 2, out=o, lse=lse)
    assert r[0] is o and r[1] is lse
    o2, l2 = fa.fwd_window(q, k, v, 30, 2)
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    e = torch.empty((0, 2, 100, 64), dtype=torch.bfloat16, device="cuda")
    ek = torch.empty((0, 1, 100, 64), dtype=torch.bfloat16, device="cuda")
    assert fa.fwd_window(e, ek, ek, 30, 2)[0].shape == e.shape
    for bad in (dict(window=0), dict(window=-3), dict(window=5, sinks=-1), dict(window=5, scale=math.inf)):
        with pytest.raises(fa.FaError):
            fa.fwd_window(q, k, v, **bad)
    with pytest.raises(ValueError):
        fa.fwd_window(q, k, v, 5, out=torch.empty((1, 2, 99, 64), dtype=torch.bfloat16, device="cuda"))


def test_window_forward_in_a_graph_and_on_a_stream(fa):
    case = (2, 4, 2, 500, 800, 128, 200, 4)
    q, k, v = _inputs(*case[:6], 27, torch.bfloat16)
    want = fa.fwd_window(q, k, v, *case[6:])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = fa.fwd_window(q, k, v, *case[6:])
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    o, lse = torch.empty_like(q), torch.empty((2, 4, 500), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fwd_window(q, k, v, *case[6:], out=o, lse=lse)
    q2 = _inputs(*case[:6], 28, torch.bfloat16)[0]
    q.copy_(q2)
    g.replay()
    torch.cuda.synchronize()
    want = fa.fwd_window(q2, k, v, *case[6:])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("sinks", [1, 31, 32, 33, 64, 127, 128])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_few_sinks_far_from_the_window(fa, sinks, d):
    # up to 32 sinks in a tile of their own take a narrower path
    _check(fa, (1, 3, 1, 700, 1900, d, 150, sinks), torch.bfloat16)
    _check(fa, (1, 2, 1, 1, 900, d, 3, sinks), torch.float16, scale=-0.1)


@pytest.mark.parametrize("d", [64, 256])
def test_window_wait_that_runs_out_is_reported(fa, d):
    # a ring slot that the kernel leaves unfilled: the waits on it end after
    # their limit, the call is reported, and the next one is right
    q, k, v = _inputs(1, 2, 2, 900, 900, d, 41, torch.bfloat16)
    want = fa.fwd_window(q, k, v, 400, 4)
    fa.check_device_error()
    assert fa.lib().fa_debug_inject(1) == fa.FA_OK
    fa.fwd_window(q, k, v, 400, 4)
    with pytest.raises(fa.FaError) as e:
        fa.check_device_error()
    assert e.value.status == fa.FA_ERR_TIMEOUT
    got = fa.fwd_window(q, k, v, 400, 4)
    fa.check_device_error()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
