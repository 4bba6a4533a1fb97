"""64-bit reference of windowed attention (forward and gradients) and of the
paged cache, and the error bounds that the arithmetic of the kernels gives.

Visibility: the query at position p sees key j iff j <= p and
(j > p - window or j < sinks)."""
from __future__ import annotations

import math

import torch

# half a step relative to the value: the most one rounding to nearest moves it
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def visible(Nq, Nk, window, sinks, device="cpu"):
    p = torch.arange(Nq, device=device)[:, None] + (Nk - Nq)
    j = torch.arange(Nk, device=device)[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def reference(q, k, v, window, sinks, scale, do=None):
    """q [H, Nq, d], k, v [Hkv, Nk, d] (any dtype) -> dict of 64-bit tensors:
    O, LSE, the weights' sum of |v| (A) and, with do, dQ, dK, dV."""
    H, Nq, d = q.shape
    Hkv, Nk = k.shape[0], k.shape[1]
    g = H // Hkv
    q, k, v = q.double(), k.double().repeat_interleave(g, 0), v.double().repeat_interleave(g, 0)
    see = visible(Nq, Nk, window, sinks, q.device)
    s = (q @ k.transpose(1, 2)) * scale
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, -1) if Nk else torch.full((H, Nq), -math.inf, dtype=torch.float64, device=q.device)
    some = lse > -math.inf
    p = torch.where(see, torch.exp(s - torch.where(some, lse, torch.zeros_like(lse))[..., None]), torch.zeros_like(s))
    v0 = torch.where(see.any(0)[None, :, None], v, torch.zeros_like(v))  # what no query sees may hold anything
    k0 = torch.where(see.any(0)[None, :, None], k, torch.zeros_like(k))
    out = dict(O=p @ v0, LSE=lse, A=p @ v0.abs(), some=some, vmax=float(v0.abs().max()) if v0.numel() else 0.0,
               # the largest sum of |q||k| behind a visible score, times |scale|
               S=abs(scale) * torch.where(see, q.abs() @ k0.abs().transpose(1, 2), torch.zeros_like(s)).amax(-1)
               if Nk else torch.zeros_like(lse))
    if do is not None:
        do = do.double()
        dp = do @ v0.transpose(1, 2)
        D = (do * out["O"]).sum(-1, keepdim=True)
        ds = p * (dp - D)
        fold = lambda x: x.view(Hkv, g, Nk, d).sum(1)  # noqa: E731
        out.update(dQ=scale * ds @ k0, dK=fold(scale * ds.transpose(1, 2) @ q), dV=fold(p.transpose(1, 2) @ do))
    return out


def check_forward(o, lse, ref, dtype, d, Nk, what):
    """Element-wise bounds.

    Score: products of two 16-bit values are exact in fp32; the sum of d of
    them and its scaling move it by at most delta = d 2^-23 S (S: the sum of
    absolute products), so each weight by a factor within 2 delta, numerator
    and denominator.  exp2, the row sum and the accumulation in fp32 add at
    most 2^-18 of A for these lengths (A = sum of weight * |v|).
    P is rounded to the element type (u A), O once more (u |O|); in fp16,
    weights below 2^-14 of the running maximum lie on a grid of 2^-24, half a
    step of which is 2^-25 each (at most Nk 2^-25 max|v|)."""
    u = HALF_STEP[dtype]
    o, lse = o.double(), lse.double()
    assert o.shape == ref["O"].shape and lse.shape == ref["LSE"].shape, what
    some = ref["some"]
    assert torch.equal(lse == -math.inf, ~some), f"{what}: rows without keys must have LSE = -inf, and no others"
    assert bool((o[~some] == 0).all()), f"{what}: rows without keys must have O = 0"
    assert bool(torch.isfinite(o).all()), f"{what}: non-finite output"
    delta = (d * 2.0 ** -23 * ref["S"])[..., None]
    tol = u * (ref["A"] + ref["O"].abs()) * (1 + 2 * u) + (4 * delta + 2.0 ** -18) * ref["A"]
    if dtype == torch.float16:
        tol = tol + Nk * 2.0 ** -25 * ref["vmax"] + 2.0 ** -25
    bad = (o - ref["O"]).abs() > tol
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst excess " \
                                f"{float(((o - ref['O']).abs() - tol).max()):.3e}"
    if some.any():
        # LSE: the maximum and the logarithm in fp32 (2^-22 of the value and
        # 2^-20 absolute), the scores' delta
        tol = (delta[..., 0] + 2.0 ** -20 + 2.0 ** -21 * ref["LSE"].abs())[some]
        off = (lse[some] - ref["LSE"][some]).abs()
        assert bool((off <= tol).all()), f"{what}: LSE off by {float(off.max()):.3e}"


class Paged:
    """A paged cache with scattered pages that holds given sequences.

    seqs: [(k, v)] per sequence, [Hkv, nk, d]; everything the sequences do not
    hold is filled with ``junk``."""

    def __init__(self, seqs, page, layout="hnd", junk=float("nan"), spare=3, max_pages=None, seed=0, device="cuda"):
        Hkv, _, d = seqs[0][0].shape
        dt = seqs[0][0].dtype
        need = [-(-k.shape[1] // page) for k, _ in seqs]
        n = sum(need) + spare
        if layout == "hnd":
            self.k, self.v = (torch.full((n, Hkv, page, d), junk, dtype=dt, device=device) for _ in range(2))
        elif layout == "nhd":
            self.k, self.v = (torch.full((n, page, Hkv, d), junk, dtype=dt, device=device).transpose(1, 2)
                              for _ in range(2))
        else:  # keys and values interleaved, with padding behind each token
            both = torch.full((n, page, 2, Hkv, d + 8), junk, dtype=dt, device=device)
            self.k, self.v = (both[:, :, i, :, :d].transpose(1, 2) for i in range(2))
        gen = torch.Generator().manual_seed(seed)
        order = torch.randperm(n, generator=gen)
        width = max([1] + need) if max_pages is None else max_pages
        self.table = torch.full((len(seqs), width), -7, dtype=torch.int32)
        at = 0
        for b, (k, v) in enumerate(seqs):
            self.table[b, :need[b]] = order[at:at + need[b]].to(torch.int32)
            at += need[b]
            for x, pages in ((k, self.k), (v, self.v)):
                for i in range(need[b]):
                    part = x[:, i * page:(i + 1) * page]
                    pages[int(self.table[b, i]), :, :part.shape[1]] = part.to(device)
        self.table = self.table.to(device)


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def check_backward(got, q, k, v, do, o, window, sinks, scale, ref, dtype, what):
    """Element-wise bounds of dQ, dK, dV (one batch entry; o: the forward's
    rounded output, which D is formed from).

    P is off by a factor within e = 4 delta + 2^-18 (scores, exp2, the LSE's
    own error; delta as in check_forward) and rounded to the element type (u)
    as dV's left operand; dP by d 2^-23 sum|do||v|; D by sum |do||o - O| and
    its fp32 sum; dS = P (dP - D) is rounded to the element type (u); every
    gradient is a sum of such products in fp32 (2^-18 of the absolute sum)
    and rounded once (u).  In fp16, P and dS below 2^-14 lie on a grid whose
    half step is 2^-25."""
    u = HALF_STEP[dtype]
    H, Nq, d = q.shape
    Hkv, Nk = k.shape[0], k.shape[1]
    g = H // Hkv
    q, do, o = q.double(), do.double(), o.double()
    k, v = (x.double().repeat_interleave(g, 0) for x in (k, v))
    see = visible(Nq, Nk, window, sinks, q.device)
    lse = torch.where(ref["some"], ref["LSE"], torch.zeros_like(ref["LSE"]))
    p = torch.where(see, torch.exp((q @ k.transpose(1, 2)) * scale - lse[..., None]), torch.zeros(1, dtype=torch.float64, device=q.device))
    ds = p * (do @ v.transpose(1, 2) - (do * ref["O"]).sum(-1, keepdim=True))
    e = (4 * d * 2.0 ** -23 * ref["S"] + 2.0 ** -18)[..., None]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    edp = d * 2.0 ** -23 * (do.abs() @ v.abs().transpose(1, 2))
    eD = (do.abs() * (o - ref["O"]).abs()).sum(-1, keepdim=True) + d * 2.0 ** -23 * (do.abs() * o.abs()).sum(-1, keepdim=True)
    eP = torch.where(see, (u + e) * p + tiny, torch.zeros_like(p))
    eS = torch.where(see, (1 + u) * (e * ds.abs() + (1 + e) * p * (edp + eD)) + u * ds.abs() + tiny, torch.zeros_like(p))
    fold = lambda x: x.view(Hkv, g, Nk, d).sum(1)  # noqa: E731
    aP, aS = p + eP, ds.abs() + eS
    bounds = (abs(scale) * (eS @ k.abs() + 2.0 ** -18 * (aS @ k.abs())),
              abs(scale) * fold(eS.transpose(1, 2) @ q.abs() + 2.0 ** -18 * (aS.transpose(1, 2) @ q.abs())),
              fold(eP.transpose(1, 2) @ do.abs() + 2.0 ** -18 * (aP.transpose(1, 2) @ do.abs())))
    for name, x, b in zip(("dQ", "dK", "dV"), got, bounds):
        x, r = x.double(), ref[name]
        assert bool(torch.isfinite(x).all()), f"{what} {name}: non-finite"
        tol = b + u * (r.abs() + b) + tiny
        bad = (x - r).abs() > tol
        assert not bool(bad.any()), f"{what} {name}: {int(bad.sum())} of {bad.numel()} outside, worst excess " \
                                    f"{float(((x - r).abs() - tol).max()):.3e}"
