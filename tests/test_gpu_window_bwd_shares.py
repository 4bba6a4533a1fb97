"""The windowed backward where key tiles are few and a group's query heads
many: every tile's steps are shared out over several blocks, whose fp32 dK and
dV are summed."""
import pytest
import torch

import attn_inputs as gen
from window_util import check_backward, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _inputs(B, Hq, Hkv, Nq, Nk, d, seed, dtype):
    shapes = ((B, Hq, Nq, d), (B, Hkv, Nk, d), (B, Hkv, Nk, d), (B, Hq, Nq, d))
    return [torch.from_numpy(gen.normal(s, seed, i)).to(dtype).cuda() for i, s in enumerate(shapes)]


CASES = [
    # B, Hq, Hkv, Nq, Nk, window, sinks
    (1, 16, 1, 700, 700, 200, 0),
    (1, 16, 1, 700, 700, 650, 4),       # the sink tile shared out too
    (1, 32, 2, 129, 129, 100, 0),       # one row beyond a tile
    (1, 64, 1, 40, 40, 39, 0),          # less than a tile: one of them, seen by 64 heads
    (1, 16, 1, 100, 1000, 990, 0),      # keys of the first tiles seen by few queries
    (1, 16, 1, 100, 1000, 150, 0),      # and by none: zero gradients
    (1, 16, 1, 700, 200, 199, 3),       # queries that see no key
    (1, 24, 1, 513, 513, 300, 260),     # three sink tiles
    (1, 24, 1, 513, 513, 300, 513),     # every tile a sink tile
    (3, 14, 2, 300, 321, 250, 0),
    (8, 64, 8, 384, 384, 380, 0),       # whole tiles first, the others shared
    (8, 64, 8, 640, 640, 600, 130),     # with sink tiles before them
    (1, 16, 1, 256, 256, 256, 0),       # a window over everything: not shared
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B{}_Hq{}_Hkv{}_Nq{}_Nk{}_w{}_s{}".format(*c))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_shared_tiles(fa, case, d, dtype):
    B, Hq, Hkv, Nq, Nk, w, sinks = case
    q, k, v, do = _inputs(B, Hq, Hkv, Nq, Nk, d, 51, dtype)
    o, lse = fa.fwd_window(q, k, v, w, sinks)
    grads = fa.bwd_window(q, k, v, o, lse, do, w, sinks)
    fa.check_device_error()
    for b in range(B):
        ref = reference(q[b], k[b], v[b], w, sinks, d ** -0.5, do[b])
        check_backward([x[b] for x in grads], q[b], k[b], v[b], do[b], o[b], w, sinks, d ** -0.5, ref, dtype,
                       f"{case} d{d} {dtype}")


@pytest.mark.parametrize("d", [64, 128])
def test_shared_tiles_are_the_same_every_time_and_in_a_graph(fa, d):
    B, Hq, Hkv, N, w, sinks = 1, 32, 2, 500, 300, 2
    q, k, v, do = _inputs(B, Hq, Hkv, N, N, d, 53, torch.bfloat16)
    o, lse = fa.fwd_window(q, k, v, w, sinks)
    need = fa.bwd_window_workspace_bytes(B, Hq, Hkv, N, N, d, w, sinks)
    assert need > fa.bwd_window_workspace_bytes(B, Hq, Hkv, N, N, d, N, 0)  # parts of the shared tiles
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    want = fa.bwd_window(q, k, v, o, lse, do, w, sinks, workspace=ws)
    ws.fill_(255)
    outs = [torch.full_like(x, float("nan")) for x in (q, k, v)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.bwd_window(q, k, v, o, lse, do, w, sinks, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
    for _ in range(2):
        g.replay()
        fa.check_device_error()
        assert torch.equal(outs[1], want[1]) and torch.equal(outs[2], want[2])
        # dQ: fp32 adds in any order, rounded once
        assert (outs[0].float() - want[0].float()).abs().max() <= 2.0 ** -7 * want[0].float().abs().max()
    with pytest.raises(fa.FaError):
        fa.bwd_window(q, k, v, o, lse, do, w, sinks, workspace=ws[:need - 256])
