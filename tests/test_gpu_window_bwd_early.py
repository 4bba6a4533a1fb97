"""The windowed backward's first positions, whose D = sum_j P_j dP_j is taken
over their keys: a row of one key has dS = P (dP - D) = 0, which O's rounding
in D = dO . O would hide."""
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,window,sinks", [(2, 6, 2, 300, 300, 100, 0), (1, 4, 4, 200, 200, 1, 0), (1, 4, 1, 77, 77, 76, 3),
                                                         (1, 3, 1, 200, 170, 60, 1), (1, 2, 1, 90, 101, 40, 0), (1, 2, 1, 40, 72, 20, 0),
                                                         (1, 2, 2, 20, 20, 5, 1)])
def test_first_positions(fa, B, Hq, Hkv, Nq, Nk, window, sinks, d, dtype):
    shapes = ((B, Hq, Nq, d), (B, Hkv, Nk, d), (B, Hkv, Nk, d), (B, Hq, Nq, d))
    q, k, v, do = [torch.from_numpy(gen.normal(s, 91, i)).to(dtype).cuda() for i, s in enumerate(shapes)]
    o, lse = fa.fwd_window(q, k, v, window, sinks)
    grads = fa.bwd_window(q, k, v, o, lse, do, window, sinks)
    fa.check_device_error()
    s = d ** -0.5
    for b in range(B):
        ref = reference(q[b], k[b], v[b], window, sinks, s, do[b])
        check_backward([x[b] for x in grads], q[b], k[b], v[b], do[b], o[b], window, sinks, s, ref, dtype, f"{window} {sinks}")
    if Nq >= Nk:
        # Position 0 sees key 0 alone.  With P = 1 + e, e at most the fp32 error
        # of its exponent (its score's sum and LSE, d 2^-22 sum|q||k| s + 2^-20),
        # dP and D sums of d products in fp32 in two orders: |dP - D| is at most
        # d 2^-22 sum|dO||v| + |e| |D|, and dQ that times s |k|.
        i = Nq - Nk
        g = Hq // Hkv
        k0, v0 = (x[:, :, 0].double().abs().repeat_interleave(g, 1) for x in (k, v))
        q0, g0 = q[:, :, i].double().abs(), do[:, :, i].double().abs()
        dp = (g0 * v0).sum(-1, keepdim=True)
        e = d * 2.0 ** -22 * s * (q0 * k0).sum(-1, keepdim=True) + 2.0 ** -20
        bound = s * k0 * (d * 2.0 ** -22 * dp + e * dp)
        assert bool((grads[0][:, :, i].double().abs() <= bound + 2.0 ** -24).all())
