"""Gradients of windowed attention (fa_bwd_window) against the 64-bit
formulas on every element, within bounds derived from the kernel's arithmetic
(window_util.check_backward)."""
import math

import pytest
import torch

import attn_inputs as gen
from window_util import check_backward, check_forward, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _inputs(B, Hq, Hkv, Nq, Nk, d, seed, dtype):
    return [torch.from_numpy(gen.normal(s, seed, i)).to(dtype).cuda()
            for i, s in enumerate([(B, Hq, Nq, d), (B, Hkv, Nk, d), (B, Hkv, Nk, d), (B, Hq, Nq, d)])]


def _check(fa, case, dtype, scale=None):
    B, Hq, Hkv, Nq, Nk, d, w, sinks = case
    q, k, v, do = _inputs(B, Hq, Hkv, Nq, Nk, d, 500 + Nq + Nk + w % 1000, dtype)
    o, lse = fa.fwd_window(q, k, v, w, sinks, scale=scale)
    grads = fa.bwd_window(q, k, v, o, lse, do, w, sinks, scale=scale)
    fa.check_device_error()
    s = 1 / math.sqrt(d) if scale is None else scale
    for b in range(B):
        what = f"{case} {dtype} batch {b}"
        ref = reference(q[b], k[b], v[b], w, sinks, s, do[b])
        check_forward(o[b], lse[b], ref, dtype, d, Nk, what)
        check_backward([x[b] for x in grads], q[b], k[b], v[b], do[b], o[b], w, sinks, s, ref, dtype, what)


CASES = [
    # B, Hq, Hkv, Nq, Nk, d, window, sinks
    (1, 2, 1, 1, 1, 64, 1, 0),
    (2, 4, 2, 1, 300, 128, 100, 3),
    (1, 2, 2, 256, 256, 128, 1, 0),
    (1, 4, 2, 300, 130, 64, 50, 2),        # queries that see no key
    (2, 4, 4, 640, 640, 128, 128, 0),
    (1, 4, 1, 777, 777, 128, 127, 4),
    (1, 4, 1, 777, 777, 64, 129, 4),
    (1, 6, 2, 1000, 1000, 128, 64, 127),
    (1, 3, 1, 1000, 1000, 64, 65, 128),
    (1, 3, 1, 1000, 1000, 128, 200, 129),
    (1, 2, 1, 900, 900, 64, 100, 900),     # every key a sink
    (1, 2, 1, 900, 900, 128, 1 << 40, 5),  # plain causal
    (1, 2, 1, 200, 2049, 128, 300, 16),    # keys that no query sees get zero gradients
    (1, 8, 1, 2000, 2000, 64, 30, 1),      # the sink tile's queries shared out over many CTAs
    (2, 8, 2, 1100, 1300, 128, 40, 200),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B{}_Hq{}_Hkv{}_Nq{}_Nk{}_d{}_w{}_s{}".format(*c))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_window_backward(fa, case, dtype):
    _check(fa, case, dtype)


@pytest.mark.parametrize("scale", [0.0, -0.2, 0.4])
@pytest.mark.parametrize("d", [64, 128])
def test_window_backward_scales(fa, scale, d):
    _check(fa, (1, 4, 2, 400, 500, d, 140, 5), torch.bfloat16, scale=scale)


@pytest.mark.parametrize("d", [64, 128])
def test_window_over_everything_is_the_causal_backward(fa, d):
    q, k, v, do = _inputs(1, 4, 2, 600, 700, d, 31, torch.bfloat16)
    o, lse = fa.fwd_gqa(q, k, v, causal=True)
    a = fa.bwd(q, k, v, o, lse, do, causal=True)
    b = fa.bwd_window(q, k, v, o, lse, do, 700, 0)
    fa.check_device_error()
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert (a[0].float() - b[0].float()).abs().max() <= 2.0 ** -7 * a[0].float().abs().max()


def test_window_backward_workspace_empty_and_refusals(fa):
    B, Hq, Hkv, N, d, w, sinks = 1, 4, 2, 700, 128, 60, 3
    q, k, v, do = _inputs(B, Hq, Hkv, N, N, d, 33, torch.bfloat16)
    o, lse = fa.fwd_window(q, k, v, w, sinks)
    need = fa.bwd_window_workspace_bytes(B, Hq, Hkv, N, N, d, w, sinks)
    assert need > fa.bwd_workspace_bytes(B, Hq, N, d)  # the sink tile is shared out
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    outs = [torch.full_like(x, float("nan")) for x in (q, k, v)]
    r = fa.bwd_window(q, k, v, o, lse, do, w, sinks, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
    assert all(x is y for x, y in zip(r, outs))
    want = fa.bwd_window(q, k, v, o, lse, do, w, sinks)
    fa.check_device_error()
    assert torch.equal(r[1], want[1]) and torch.equal(r[2], want[2])
    assert (r[0].float() - want[0].float()).abs().max() <= 2.0 ** -7 * want[0].float().abs().max()
    with pytest.raises(fa.FaError):
        fa.bwd_window(q, k, v, o, lse, do, w, sinks, workspace=ws[:need - 256])
    for kw in (dict(window=0), dict(window=5, sinks=-1), dict(window=5, scale=math.nan)):
        with pytest.raises(fa.FaError):
            fa.bwd_window(q, k, v, o, lse, do, **kw)
    with pytest.raises(ValueError):
        fa.bwd_window(q, k, v, o, lse[:, :, :5], do, w)
    with pytest.raises(ValueError):
        fa.bwd_window(q, k, v, o, lse, do, w, dk=q)
    e = q[:, :, :0].contiguous()
    dq, dk, dv = fa.bwd_window(e, k, v, e, lse[:, :, :0].contiguous(), e, w, sinks)
    assert bool((dk == 0).all()) and bool((dv == 0).all()) and dq.numel() == 0


def test_window_training_step_in_a_graph(fa):
    B, Hq, Hkv, N, d, w, sinks = 1, 4, 2, 800, 64, 120, 4
    q, k, v, do = _inputs(B, Hq, Hkv, N, N, d, 35, torch.float16)
    o, lse = torch.empty_like(q), torch.empty((B, Hq, N), device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty((fa.bwd_window_workspace_bytes(B, Hq, Hkv, N, N, d, w, sinks),), dtype=torch.uint8, device="cuda")

    def step():
        fa.fwd_window(q, k, v, w, sinks, out=o, lse=lse)
        fa.bwd_window(q, k, v, o, lse, do, w, sinks, dq=dq, dk=dk, dv=dv, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    q.copy_(_inputs(B, Hq, Hkv, N, N, d, 36, torch.float16)[0])
    g.replay()
    fa.check_device_error()
    ref = reference(q[0], k[0], v[0], w, sinks, 1 / math.sqrt(d), do[0])
    check_backward((dq[0], dk[0], dv[0]), q[0], k[0], v[0], do[0], o[0], w, sinks, 1 / math.sqrt(d), ref, torch.float16, "graph")
