"""Trees of drafted tokens on the host: plain models of their layout, and the
64-bit reference of attention under any visibility."""
from __future__ import annotations

import math
import random

import torch


def random_tree(n, rng, width=None):
    """Parents of n nodes: a few roots, else an earlier node not far away."""
    width = width or rng.choice([1, 2, 5, 12])
    return [-1 if i == 0 or rng.random() < 0.03 else rng.randrange(max(0, i - width), i) for i in range(n)]


def layout(parents, words):
    """(rows of what each node sees, as sets; depths)."""
    rows, depth = [], []
    for i, p in enumerate(parents):
        rows.append((rows[p] if p >= 0 else frozenset()) | {i})
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return rows, depth


def mask_of(rows, words):
    """Sets of seen nodes -> int32 [n, words]."""
    out = []
    for row in rows:
        bits = sum(1 << k for k in row if k < 32 * words)
        out.append([(bits >> (32 * w)) & 0xffffffff for w in range(words)])
    out = torch.tensor(out, dtype=torch.int64).view(len(rows), words)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def sees(n, ctx, rows, pos, window, sinks, chunk=False):
    """[n, ctx + n] visibility: cached keys by a node's position, new ones by its
    row (a chunk: by where its tokens lie).  ctx may be negative: the first nodes
    then lie before the sequence."""
    nk = max(0, ctx + n)
    see = torch.zeros(n, nk, dtype=torch.bool)
    j = torch.arange(nk)
    for i in range(n):
        if chunk:
            p = ctx + i
            see[i] = (j <= p) & ((j > p - window) | (j < sinks))
            continue
        see[i] = (j < ctx) & ((j > pos[i] - window) | (j < sinks))
        for k in rows[i]:
            if k <= i and ctx + k >= 0:
                see[i, ctx + k] = True
    return see


def reference(q, k, v, see, scale):
    """q [n, Hq, d], k, v [Hkv, nk, d], see [n, nk] -> what check_forward takes."""
    g = q.shape[1] // k.shape[0]
    see = see.to(q.device)
    q = q.transpose(0, 1).double()
    k, v = (x.double().repeat_interleave(g, 0) for x in (k, v))
    any_ = see.any(0)[None, :, None]
    k0, v0 = torch.where(any_, k, torch.zeros_like(k)), torch.where(any_, v, torch.zeros_like(v))
    s = torch.where(see, (q @ k0.transpose(1, 2)) * scale, torch.full((), -math.inf, dtype=torch.float64, device=q.device))
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    some = lse > -math.inf
    p = torch.where(see, torch.exp(s - torch.where(some, lse, torch.zeros_like(lse))[..., None]), torch.zeros_like(s))
    S = abs(scale) * torch.where(see, q.abs() @ k0.abs().transpose(1, 2), torch.zeros_like(s)).amax(-1) if s.shape[-1] else torch.zeros_like(lse)
    return dict(O=p @ v0, LSE=lse, A=p @ v0.abs(), some=some, vmax=float(v0.abs().max()) if v0.numel() else 0.0, S=S)
