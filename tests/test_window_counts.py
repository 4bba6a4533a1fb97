"""Windows, sinks and hints of any size: one that 64 bits do not hold means what
the largest one means (and below zero is refused), and nothing is remembered by
the object that held it."""
import pytest
import torch

FAR = [(1 << 63) - 1, 1 << 63, 1 << 64, (1 << 64) + 1, (1 << 70) + 5]


@pytest.fixture(scope="module")
def fa():
    from exact_attention_forward_09_gb300 import build
    build.build()
    import exact_attention_forward_09_gb300 as fa
    fa.lib()
    return fa


@pytest.mark.parametrize("far", FAR)
def test_workspace(fa, far):
    size = lambda w, s: fa.bwd_window_workspace_bytes(1, 8, 2, 1000, 1000, 64, w, s)  # noqa: E731
    assert size(far, 4) == size(1 << 40, 4)
    assert size(30, far) == size(30, 1 << 40) != size(30, 1)  # (without parts: most tiles hold sinks)
    for kw in (dict(w=-far - 1, s=0), dict(w=5, s=-far - 1)):
        with pytest.raises(fa.FaError):
            size(**kw)


def test_workspace_of_a_count_that_changes(fa):
    sinks = torch.tensor(1)
    size = lambda: fa.bwd_window_workspace_bytes(1, 8, 2, 1000, 1000, 64, 30, sinks)  # noqa: E731
    one = size()
    sinks.fill_(900)
    assert size() == fa.bwd_window_workspace_bytes(1, 8, 2, 1000, 1000, 64, 30, 900) != one


@pytest.mark.gpu
@pytest.mark.parametrize("far", FAR)
def test_results(fa, far):
    q, k, v, do = (torch.randn(1, h, 300, 64, device="cuda").bfloat16() for h in (4, 2, 2, 4))
    for w, s, w2, s2 in ((far, 3, 300, 3), (20, far, 20, 300)):
        o, lse = fa.fwd_window(q, k, v, w, s)
        o2, lse2 = fa.fwd_window(q, k, v, w2, s2)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        g, g2 = fa.bwd_window(q, k, v, o, lse, do, w, s), fa.bwd_window(q, k, v, o, lse, do, w2, s2)
        assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])
    pages = [torch.randn(3, 2, 64, 64, device="cuda").bfloat16() for _ in range(2)]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (q[0].transpose(0, 1)[:5].contiguous(), *pages, ints([[2, 0, 1]]), ints([0, 5]), ints([170]))
    a, b = (fa.fwd_paged(*args, window=w, sinks=s, max_q=m) for w, s, m in ((far, 1, far), (1 << 30, 1, 0)))
    fa.check_device_error()
    assert torch.allclose(a[0].float(), b[0].float(), rtol=2.0 ** -7, atol=2.0 ** -9) and torch.allclose(a[1], b[1], atol=1e-5)
    with pytest.raises(fa.FaError):
        fa.fwd_window(q, k, v, -far - 1)
