"""The 64-bit reference of windowed attention: its gradients against central
differences of its forward, its mask against the definition (CPU only)."""
import pytest
import torch

from window_util import reference, visible


@pytest.mark.parametrize("Nq,Nk,window,sinks", [(5, 5, 2, 0), (4, 7, 3, 1), (6, 3, 2, 1), (5, 6, 1, 6), (3, 9, 100, 0)])
def test_mask(Nq, Nk, window, sinks):
    m = visible(Nq, Nk, window, sinks)
    for i in range(Nq):
        p = i + Nk - Nq
        for j in range(Nk):
            assert bool(m[i, j]) == (j <= p and (j > p - window or j < sinks))


@pytest.mark.parametrize("H,Hkv,Nq,Nk,window,sinks", [(2, 1, 5, 5, 2, 1), (4, 2, 3, 6, 3, 0), (2, 2, 6, 4, 2, 1), (3, 1, 4, 4, 9, 0)])
def test_gradients_against_differences(H, Hkv, Nq, Nk, window, sinks):
    gen = torch.Generator().manual_seed(Nq + 10 * Nk)
    q, do = (torch.randn(H, Nq, 4, generator=gen, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(Hkv, Nk, 4, generator=gen, dtype=torch.float64) for _ in range(2))
    ref = reference(q, k, v, window, sinks, 0.6, do)
    h = 1e-5
    for name, i in (("dQ", 0), ("dK", 1), ("dV", 2)):
        x = [q, k, v]
        for n in range(x[i].numel()):
            side = []
            for s in (h, -h):
                y = [t.clone() for t in x]
                y[i].view(-1)[n] += s
                side.append((reference(*y, window, sinks, 0.6)["O"] * do).sum())
            assert abs(float((side[0] - side[1]) / (2 * h)) - float(ref[name].reshape(-1)[n])) < 1e-7
