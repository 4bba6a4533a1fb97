"""The windowed backward's rows of few keys.  dS = P (dP - D) hands D's error on
to every key of a row: it averages out over many keys, but with one key dS must
vanish.  Rows that see at most 32 keys, whatever their position, therefore take
D = sum_j P_j dP_j over their keys, which carries fp32 errors alone."""
import pytest
import torch

import attn_inputs as gen
from window_util import HALF_STEP, reference, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def check(got, q, k, v, do, o, window, sinks, scale, ref, dtype, what):
    """window_util.check_backward's bounds (its P, dP, dS, sums and roundings)
    with D's error eD by the row's number of keys n.  Above 32, D = dO . O: O's
    rounding and an fp32 sum.  Up to 32, D = sum_j P_j dP_j: each P_j is off by a
    factor within e, each dP_j by edp, and a sum of at most 32 fp32 terms by
    2^-18 of their absolute sum."""
    u = HALF_STEP[dtype]
    H, Nq, d = q.shape
    Hkv, Nk = k.shape[0], k.shape[1]
    g = H // Hkv
    q, do, o = q.double(), do.double(), o.double()
    k, v = (x.double().repeat_interleave(g, 0) for x in (k, v))
    see = visible(Nq, Nk, window, sinks, q.device)
    lse = torch.where(ref["some"], ref["LSE"], torch.zeros_like(ref["LSE"]))
    p = torch.where(see, torch.exp((q @ k.transpose(1, 2)) * scale - lse[..., None]), torch.zeros(1, dtype=torch.float64, device=q.device))
    dp = do @ v.transpose(1, 2)
    ds = p * (dp - (do * ref["O"]).sum(-1, keepdim=True))
    e = (4 * d * 2.0 ** -23 * ref["S"] + 2.0 ** -18)[..., None]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    edp = d * 2.0 ** -23 * (do.abs() @ v.abs().transpose(1, 2))
    many = (do.abs() * (o - ref["O"]).abs()).sum(-1, keepdim=True) + d * 2.0 ** -23 * (do.abs() * o.abs()).sum(-1, keepdim=True)
    few = (p * (e * dp.abs() + (1 + e) * edp) + 2.0 ** -18 * p * dp.abs()).sum(-1, keepdim=True)
    eD = torch.where(see.sum(-1, keepdim=True) <= 32, few, many)
    eS = torch.where(see, (1 + u) * (e * ds.abs() + (1 + e) * p * (edp + eD)) + u * ds.abs() + tiny, torch.zeros_like(p))
    fold = lambda x: x.view(Hkv, g, Nk, d).sum(1)  # noqa: E731
    aS = ds.abs() + eS
    bounds = (abs(scale) * (eS @ k.abs() + 2.0 ** -18 * (aS @ k.abs())),
              abs(scale) * fold(eS.transpose(1, 2) @ q.abs() + 2.0 ** -18 * (aS.transpose(1, 2) @ q.abs())))
    for name, x, b in zip(("dQ", "dK"), got, bounds):
        r = ref[name]
        tol = b + u * (r.abs() + b) + tiny
        over = (x.double() - r).abs() - tol
        assert bool(torch.isfinite(x).all()) and not bool((over > 0).any()), \
            f"{what} {name}: {int((over > 0).sum())} of {over.numel()} outside, worst excess {float(over.max()):.3e}"


CASES = [
    # B, Hq, Hkv, Nq, Nk, window, sinks
    (1, 4, 2, 300, 300, 1, 0),       # one key to every row: no gradient of Q and K
    (2, 2, 1, 300, 300, 1, 1),
    (1, 3, 1, 333, 333, 5, 3),
    (1, 4, 4, 200, 200, 32, 0),
    (1, 2, 1, 200, 200, 20, 12),     # the most keys a row of few may have
    (1, 2, 1, 200, 200, 20, 13),     # one more: the first positions alone
    (1, 6, 2, 130, 400, 7, 9),       # positions far behind the first ones
    (1, 2, 1, 1, 500, 3, 1),
    (1, 2, 1, 90, 60, 4, 1),         # rows without a key before them
    (1, 2, 1, 300, 300, 300, 0),     # a window over everything
    (1, 2, 1, 260, 250, 1 << 40, 4),
    (1, 2, 2, 20, 20, 20, 20),
    (1, 2, 1, 700, 700, 40, 2),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B{}_Hq{}_Hkv{}_Nq{}_Nk{}_w{}_s{}".format(*c))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_rows_of_few_keys(fa, case, d, dtype):
    B, Hq, Hkv, Nq, Nk, window, sinks = case
    shapes = ((B, Hq, Nq, d), (B, Hkv, Nk, d), (B, Hkv, Nk, d), (B, Hq, Nq, d))
    q, k, v, do = [torch.from_numpy(gen.normal(s, 97, i)).to(dtype).cuda() for i, s in enumerate(shapes)]
    s = d ** -0.5
    o, lse = fa.fwd_window(q, k, v, window, sinks)
    grads = fa.bwd_window(q, k, v, o, lse, do, window, sinks)
    fa.check_device_error()
    for b in range(B):
        ref = reference(q[b], k[b], v[b], window, sinks, s, do[b])
        check([x[b] for x in grads[:2]], q[b], k[b], v[b], do[b], o[b], window, sinks, s, ref, dtype, f"{case} d{d} {dtype}")


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_rows_of_few_keys_scales(fa, scale):
    q, k, v, do = [torch.from_numpy(gen.normal((1, 2, 200, 128), 98, i)).bfloat16().cuda() for i in range(4)]
    o, lse = fa.fwd_window(q, k, v, 6, 2, scale=scale)
    grads = fa.bwd_window(q, k, v, o, lse, do, 6, 2, scale=scale)
    fa.check_device_error()
    ref = reference(q[0], k[0], v[0], 6, 2, scale, do[0])
    check([x[0] for x in grads[:2]], q[0], k[0], v[0], do[0], o[0], 6, 2, scale, ref, torch.bfloat16, f"scale {scale}")
