"""Windowed attention at d = 64 with more query tiles than SMs, on both sides
of the reach at which two blocks of one query tile share an SM."""
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


def _check(fa, B, Hq, Hkv, Nq, Nk, window, sinks, dtype=torch.bfloat16, scale=None, d=64):
    q, k, v = [torch.from_numpy(gen.normal(s, 81, i)).to(dtype).cuda()
               for i, s in enumerate(((B, Hq, Nq, d), (B, Hkv, Nk, d), (B, Hkv, Nk, d)))]
    o, lse = torch.full_like(q, float("nan")), torch.full((B, Hq, Nq), float("nan"), device="cuda")
    fa.fwd_window(q, k, v, window, sinks, scale=scale, out=o, lse=lse)
    fa.check_device_error()
    for b in range(B):
        check_forward(o[b], lse[b], reference(q[b], k[b], v[b], window, sinks, d ** -0.5 if scale is None else scale),
                      dtype, d, Nk, f"B{B} Hq{Hq} Hkv{Hkv} {Nq}x{Nk} w{window} s{sinks} {dtype} scale {scale}")


@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk", [(64, 3, 1, 100, 100), (1, 153, 9, 1, 300), (2, 77, 7, 100, 200), (1, 16, 4, 1281, 1281),
                                            (3, 26, 13, 250, 130), (1, 12, 4, 1700, 1800)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (128, 33), (300, 0), (640, 0), (636, 4), (636, 5), (500, 140)])
def test_short_windows(fa, B, Hq, Hkv, Nq, Nk, window, sinks):
    _check(fa, B, Hq, Hkv, Nq, Nk, window, sinks, torch.bfloat16 if window % 2 else torch.float16)


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scales(fa, scale):
    _check(fa, 2, 40, 10, 300, 300, 90, 2, scale=scale)


def test_every_head_dimension_agrees_where_rows_are_padded(fa):
    for d in (64, 128, 256):
        _check(fa, 4, 20, 5, 257, 257, 100, 1, d=d)


def test_wait_that_runs_out_is_reported(fa):
    q, k, v = [torch.from_numpy(gen.normal((2, 40, 500, 64), 83, i)).to(torch.bfloat16).cuda() for i in range(3)]
    want = fa.fwd_window(q, k, v, 100, 3)
    fa.check_device_error()
    assert fa.lib().fa_debug_inject(1) == fa.FA_OK
    fa.fwd_window(q, k, v, 100, 3)
    with pytest.raises(fa.FaError) as e:
        fa.check_device_error()
    assert e.value.status == fa.FA_ERR_TIMEOUT
    got = fa.fwd_window(q, k, v, 100, 3)
    fa.check_device_error()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
