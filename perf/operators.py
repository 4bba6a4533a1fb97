"""Windowed and paged attention: the operators' cases, their plain forms and the calls a user makes of them.

Four operators that work together where a model attends to a sliding window or keeps its keys and values in pages:

* ``window``  attention forward with a sliding window and a few first keys (sinks) that stay visible, on dense tensors;
* ``train``   the same forward followed by its backward pass: one training step of the layer;
* ``paged``   attention of a ragged batch of new tokens (one token or a chunk per sequence) over a paged key/value cache;
* ``append``  rotary positions applied to the new queries and keys, and the new keys and values written into the pages.

Visibility, everywhere: with p the position of a query in its sequence, key j is visible iff j <= p and
(j > p - window or j < sinks).  A query that sees no key gets O = 0 and LSE = -inf.
"""
import math
import random

import torch

own = False

NO_WINDOW = 1 << 30  # a window that hides nothing


# ---------------------------------------------------------------- cases --

def listed():
    w = dict(op="window", dtype="bf16", B=1)
    t = dict(op="train", dtype="bf16", B=1)
    p = dict(op="paged", dtype="bf16", d=128, window=NO_WINDOW, sinks=0, qlo=1, qhi=1, long=0, mix=1)
    a = dict(op="append", dtype="bf16", d=128, page=64, mix=1)
    return [
        # a short ragged call against a longer cache, where the launch is what counts
        dict(w, name="window short ragged", dtype="fp16", Hq=4, Hkv=1, Nq=333, Nk=777, d=64, window=100, sinks=3),
        # an ordinary layer of a model with local attention
        dict(w, name="window 4k", B=2, Hq=16, Hkv=4, Nq=4096, Nk=4096, d=128, window=1024, sinks=4),
        # a long document under a wide window
        dict(w, name="window 16k wide", Hq=8, Hkv=2, Nq=16384, Nk=16384, d=128, window=4096, sinks=4),
        # odd length, more sinks than one key tile holds, no shared heads
        dict(t, name="train odd", dtype="fp16", Hq=8, Hkv=8, Nq=1025, Nk=1025, d=64, window=200, sinks=130),
        # an ordinary training sequence with shared key/value heads
        dict(t, name="train 8k", Hq=16, Hkv=4, Nq=8192, Nk=8192, d=128, window=1024, sinks=4),
        # two short conversations, one new token each: latency
        dict(p, name="decode small", B=2, Hq=8, Hkv=1, d=256, page=16, klo=90, khi=140, mix=5),
        # a full serving batch, one new token each, contexts of unequal length
        dict(p, name="decode batch", B=64, Hq=32, Hkv=8, page=64, klo=2000, khi=16000, mix=2),
        # one very long context, one new token
        dict(p, name="decode long", B=1, Hq=16, Hkv=2, page=32, klo=131000, khi=131000, mix=3),
        # chunks of a prompt over what is cached of it already
        dict(p, name="chunk prefill", B=4, Hq=32, Hkv=8, page=16, qlo=2048, qhi=2048, klo=4000, khi=10000, mix=4),
        # a serving step that mixes a few chunks with many single tokens, under a window with sinks
        dict(p, name="mixed window", dtype="fp16", B=33, Hq=16, Hkv=4, d=64, page=32, window=1000, sinks=5, qlo=1, qhi=500,
             long=3, klo=600, khi=4000, mix=6),
        # the new tokens of one decoding step
        dict(a, name="append decode", B=64, Hq=32, Hkv=8, qlo=1, qhi=1, klo=100, khi=4000, half=True),
        # the new tokens of a prefill step, read out of one fused projection
        dict(a, name="append prefill", B=8, Hq=32, Hkv=8, qlo=500, qhi=2000, klo=2000, khi=6000, half=False),
    ]


def spread(rng, lo, hi):
    """A whole number in [lo, hi], even in its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["window", "train", "paged", "paged", "append"])
    dtype = rng.choice(["bf16", "fp16"])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 7, 8])
    if op in ("window", "train"):
        d = rng.choice([64, 128, 256] if op == "window" else [64, 128])
        Nk = spread(rng, 60, 8000)
        Nq = Nk if op == "train" or rng.random() < 0.5 else spread(rng, 1, Nk)
        B = spread(rng, 1, 4)
        while B * Hkv * g * Nq * Nk > (1 << 30) // (2 if op == "train" else 1):
            if B > 1:
                B -= 1
            elif Hkv > 1:
                Hkv //= 2
            elif g > 1:
                g -= 1
            else:
                break
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * g, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, window=spread(rng, 30, 5000),
                    sinks=rng.choice([0, 1, 4, 16, 129]))
    page = rng.choice([16, 32, 64, 128, 256])
    mix = rng.randrange(1 << 20)
    if op == "append":
        B = spread(rng, 1, 64)
        qhi = spread(rng, 1, 1 + 8000 // B)
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * g, Hkv=Hkv, d=rng.choice([64, 128, 256]), page=page, qlo=1, qhi=qhi,
                    klo=qhi, khi=qhi + spread(rng, 1, 4000), half=rng.random() < 0.5, mix=mix)
    windowed = rng.random() < 0.4
    c = dict(op=op, dtype=dtype, Hq=Hkv * g, Hkv=Hkv, d=rng.choice([64, 128, 256]), page=page, qlo=1, long=0, mix=mix,
             window=spread(rng, 30, 5000) if windowed else NO_WINDOW, sinks=rng.choice([0, 1, 4, 130]) if windowed else 0)
    kind = rng.choice(["decode", "chunk", "mixed"])
    if kind == "decode":
        B = spread(rng, 1, 100)
        khi = spread(rng, 20, 300000 // B)
        return dict(c, B=B, qhi=1, klo=max(1, khi // 4), khi=khi)
    B = spread(rng, 1, 4) if kind == "chunk" else spread(rng, 5, 24)
    qhi = spread(rng, 2, 1500 if kind == "chunk" else 300)
    khi = qhi + spread(rng, 20, 5000 if kind == "chunk" else 3000)
    if B * c["Hq"] * qhi * khi > 1 << 30:
        c["Hq"] = c["Hkv"] = 4
    return dict(c, B=B, qhi=qhi, klo=qhi, khi=khi, long=0 if kind == "chunk" else 2)


def lengths(c):
    """The sequences of a ragged case: (new tokens, keys in the cache with them) for each.  With ``long`` > 0 only
    that many of them bring a chunk, the others one token."""
    rng = random.Random(c["mix"])
    got = []
    for b in range(c["B"]):
        nq = rng.randint(c["qlo"], c["qhi"])
        if c.get("long", 0) and b % (c["B"] // c["long"]) != 0:
            nq = 1
        got.append((nq, max(nq, rng.randint(c["klo"], c["khi"]))))
    return got


TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TYPES[c["dtype"]]
    d = c["d"]

    def normal(*shape):
        x = torch.empty(shape, dtype=dt, device="cuda")
        return x.normal_(generator=gen)

    s = dict(c=c, scale=1.0 / math.sqrt(d))
    if c["op"] in ("window", "train"):
        s["q"] = normal(c["B"], c["Hq"], c["Nq"], d)
        s["k"], s["v"] = (normal(c["B"], c["Hkv"], c["Nk"], d) for _ in range(2))
        if c["op"] == "train":
            s["do"] = normal(c["B"], c["Hq"], c["Nq"], d)
        return s
    lens = lengths(c)
    ps, T = c["page"], sum(nq for nq, _ in lens)
    need = [-(-nk // ps) for _, nk in lens]
    pages = sum(need) + 3
    s["k_pages"], s["v_pages"] = (normal(pages, c["Hkv"], ps, d) for _ in range(2))
    # every sequence's pages lie scattered over the cache; table entries past its last page are not in use
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((c["B"], max(need)), -1, dtype=torch.int32, device="cuda")
    at, cu = 0, [0]
    for b, (nq, nk) in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        cu.append(cu[-1] + nq)
    s["table"] = table
    s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["seq_k"] = torch.tensor([nk for _, nk in lens], dtype=torch.int32, device="cuda")
    s["max_q"], s["max_k"] = max(nq for nq, _ in lens), max(nk for _, nk in lens)
    if c["op"] == "paged":
        s["q"] = normal(T, c["Hq"], d)
        return s
    # q, k and v are slices of one projection's output
    qkv = normal(T, c["Hq"] + 2 * c["Hkv"], d)
    s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
    pos = torch.arange(c["khi"], dtype=torch.float64, device="cuda")
    freq = 10000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d)
    ang = pos[:, None] * freq[None, :]
    s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    return s


# ---------------------------------------------------------- plain forms --

def visible(p, j, window, sinks):
    """Whether the query at position p sees key j (the shapes broadcast)."""
    return (j <= p) & ((j > p - window) | (j < sinks))


def softmax_parts(q, k, mask, scale):
    """exp(scale q k^T - max) under the mask, its row sums, and the rows' log-sum-exp."""
    s = q @ k.transpose(-1, -2)
    s.mul_(scale).masked_fill_(~mask, -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = s.sum(-1, keepdim=True)
    return s, l, (m + l.log()).squeeze(-1)


def over(x, l):
    return torch.where(l > 0, x / l, torch.zeros_like(x))


def window_plain(s, backward):
    c = s["c"]
    B, Hq, Hkv, Nq, Nk, d = (c[n] for n in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))
    g, dt = Hq // Hkv, s["q"].dtype
    q = s["q"].float().view(B, Hkv, g * Nq, d)
    k, v = s["k"].float(), s["v"].float()
    at = torch.arange(Nq, device="cuda") + (Nk - Nq)
    mask = visible(at[:, None], torch.arange(Nk, device="cuda")[None, :], c["window"], c["sinks"]).repeat(g, 1)
    p, l, lse = softmax_parts(q, k, mask, s["scale"])
    o = over(p @ v, l)
    out = (o.view(B, Hq, Nq, d).to(dt), lse.view(B, Hq, Nq))
    if not backward:
        return out
    do = s["do"].float().view(B, Hkv, g * Nq, d)
    p.copy_(over(p, l))
    dv = p.transpose(-1, -2) @ do
    ds = do @ v.transpose(-1, -2)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    return (*out, dq.view(B, Hq, Nq, d).to(dt), dk.to(dt), dv.to(dt))


def rows_of(s):
    """For each new token: its sequence and its place among that sequence's new tokens."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    return b, t - s["cu_q"].long()[b]


def paged_plain(s):
    c = s["c"]
    Hq, Hkv, d, ps = c["Hq"], c["Hkv"], c["d"], c["page"]
    B, g, T = c["B"], Hq // Hkv, s["q"].shape[0]
    b, i = rows_of(s)
    j = torch.arange(s["max_k"], device="cuda")
    page = s["table"].long()[:, j // ps].clamp(min=0)
    k, v = (x[page, :, j % ps].permute(0, 2, 1, 3).float() for x in (s["k_pages"], s["v_pages"]))  # [B, Hkv, max_k, d]
    q = torch.zeros(B, s["max_q"], Hq, d, device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, s["max_q"], Hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * s["max_q"], d)
    nq = s["cu_q"][1:].long() - s["cu_q"][:-1].long()
    nk = s["seq_k"].long()
    p = torch.arange(s["max_q"], device="cuda")[None, :] + (nk - nq)[:, None]
    mask = visible(p[:, :, None], j[None, None, :], c["window"], c["sinks"]) & (j[None, None, :] < nk[:, None, None])
    e, l, lse = softmax_parts(q, k, mask.repeat(1, g, 1)[:, None], s["scale"])
    o = over(e @ v, l).view(B, Hkv, g, s["max_q"], d).permute(0, 3, 1, 2, 4)[b, i]
    lse = lse.view(B, Hkv, g, s["max_q"]).permute(0, 3, 1, 2)[b, i]
    return o.reshape(T, Hq, d).to(s["q"].dtype), lse.reshape(T, Hq)


def turned(x, cos, sin, half):
    """Rotary positions: pairs (i, i + d/2) (half) or (2i, 2i + 1)."""
    x = x.float()
    a, b = x.chunk(2, -1) if half else (x[..., 0::2], x[..., 1::2])
    y, z = a * cos - b * sin, a * sin + b * cos
    return torch.cat([y, z], -1) if half else torch.stack([y, z], -1).flatten(-2)


def append_plain(s):
    c, dt = s["c"], s["q"].dtype
    b, i = rows_of(s)
    pos = s["seq_k"].long()[b] - (s["cu_q"][1:].long() - s["cu_q"][:-1].long())[b] + i
    page, at = s["table"].long()[b, pos // c["page"]], pos % c["page"]
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    s["k_pages"][page, :, at] = turned(s["k"], cos, sin, c["half"]).to(dt)
    s["v_pages"][page, :, at] = s["v"]
    return turned(s["q"], cos, sin, c["half"]).to(dt), s["k_pages"], s["v_pages"]


# ------------------------------------------------------------------ run --

def own_run(s):
    import exact_attention_forward_09_gb300 as fa
    c = s["c"]
    if c["op"] == "window":
        return fa.fwd_window(s["q"], s["k"], s["v"], c["window"], c["sinks"])
    if c["op"] == "train":
        o, lse = fa.fwd_window(s["q"], s["k"], s["v"], c["window"], c["sinks"])
        return (o, lse, *fa.bwd_window(s["q"], s["k"], s["v"], o, lse, s["do"], c["window"], c["sinks"]))
    if c["op"] == "paged":
        return fa.fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu_q"], s["seq_k"], window=c["window"],
                            sinks=c["sinks"], max_q=s["max_q"])
    rope = (s["cos"], s["sin"], fa.FA_ROPE_HALF if c["half"] else fa.FA_ROPE_INTERLEAVED)
    q = fa.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cu_q"], s["seq_k"], q=s["q"], rope=rope)
    return q, s["k_pages"], s["v_pages"]


def run(s):
    if own:
        return own_run(s)
    op = s["c"]["op"]
    if op == "paged":
        return paged_plain(s)
    if op == "append":
        return append_plain(s)
    return window_plain(s, op == "train")


def seen(p, nk, window, sinks):
    """How many of nk keys the query at position p sees."""
    p = min(p, nk - 1)
    if p < 0:
        return 0
    lo = max(0, p - window + 1)
    return p + 1 - lo + min(sinks, lo)


def work(c):
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    if c["op"] in ("window", "train"):
        B, Nq, Nk = c["B"], c["Nq"], c["Nk"]
        pairs = B * Hq * sum(seen(i + Nk - Nq, Nk, c["window"], c["sinks"]) for i in range(Nq))
        # the keys that some query sees: the sinks and everything from the first query's window on
        lo = max(0, Nk - Nq - c["window"] + 1)
        keys = B * Hkv * (Nk - lo + min(c["sinks"], lo))
        rows = B * Hq * Nq
        if c["op"] == "window":
            return {"bytes": 2 * d * (2 * rows + 2 * keys) + 4 * rows, "flops": 4 * d * pairs}
        return {"bytes": 2 * d * (4 * rows + 4 * keys) + 4 * rows, "flops": 14 * d * pairs}
    lens = lengths(c)
    T = sum(nq for nq, _ in lens)
    if c["op"] == "append":
        return {"bytes": 2 * d * T * (2 * Hq + 4 * Hkv) + 4 * d * T, "flops": 3 * d * T * (Hq + Hkv)}
    pairs = Hq * sum(seen(nk - nq + i, nk, c["window"], c["sinks"]) for nq, nk in lens for i in range(nq))
    keys = 0
    for nq, nk in lens:
        lo = max(0, nk - nq - c["window"] + 1)
        keys += Hkv * (nk - lo + min(c["sinks"], lo))
    return {"bytes": 2 * d * (2 * T * Hq + 2 * keys) + 4 * T * Hq, "flops": 4 * d * pairs}


# ---------------------------------------------------------------- exact --

def exact_rows(q, k, v, first, window, sinks, scale, do=None):
    """One head in 64 bits: queries q at positions first, first + 1, ...; blocks of rows against the keys that a block
    can see.  Returns O, LSE and, with do, the gradients of sum(do * O)."""
    n, nk = q.shape[0], k.shape[0]
    O, L = torch.zeros_like(q), torch.full((n,), -math.inf, dtype=q.dtype, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for r0 in range(0, n, 1024):
        r1 = min(n, r0 + 1024)
        hi = min(nk, first + r1)
        if hi <= 0:
            continue
        lo = max(0, min(first + r0 - window + 1, hi))
        js = torch.cat([torch.arange(min(sinks, lo)), torch.arange(lo, hi)]).to(q.device)
        p = (first + torch.arange(r0, r1, device=q.device))[:, None]
        dist = p - js[None, :]
        see = (dist >= 0) & ((dist < window) | (js[None, :] < sinks))
        a = torch.einsum("id,jd->ij", q[r0:r1], k[js]) * scale
        a = torch.where(see, a, torch.full_like(a, -math.inf))
        lse = torch.logsumexp(a, 1)
        w = torch.where(see, torch.exp(a - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None]), torch.zeros_like(a))
        O[r0:r1] = torch.einsum("ij,jd->id", w, v[js])
        L[r0:r1] = lse
        if do is not None:
            g = do[r0:r1]
            dv.index_add_(0, js, torch.einsum("ij,id->jd", w, g))
            gw = torch.einsum("id,jd->ij", g, v[js])
            ga = w * (gw - (w * gw).sum(1, keepdim=True)) * scale
            dq[r0:r1] = torch.einsum("ij,jd->id", ga, k[js])
            dk.index_add_(0, js, torch.einsum("ij,id->jd", ga, q[r0:r1]))
    return (O, L) if do is None else (O, L, dq, dk, dv)


def exact(c, seed):
    s = prepare(c, seed)
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    g = Hq // Hkv
    if c["op"] in ("window", "train"):
        if work(c)["flops"] > 6e12:
            return None
        q, k, v = (s[n].double() for n in ("q", "k", "v"))
        O, L = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float64, device="cuda")
        grads = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for b in range(c["B"]):
            for h in range(Hq):
                do = s["do"][b, h].double() if c["op"] == "train" else None
                got = exact_rows(q[b, h], k[b, h // g], v[b, h // g], c["Nk"] - c["Nq"], c["window"], c["sinks"], d ** -0.5, do)
                O[b, h], L[b, h] = got[:2]
                if do is not None:
                    grads[0][b, h] = got[2]
                    grads[1][b, h // g] += got[3]
                    grads[2][b, h // g] += got[4]
        return (O, L) if c["op"] == "window" else (O, L, *grads)
    if c["op"] == "paged":
        if work(c)["flops"] > 6e12:
            return None
        T = s["q"].shape[0]
        O, L = torch.empty(T, Hq, d, dtype=torch.float64, device="cuda"), torch.empty(T, Hq, dtype=torch.float64, device="cuda")
        at = 0
        for b, (nq, nk) in enumerate(lengths(c)):
            ids = s["table"][b, :-(-nk // c["page"])].long()
            k, v = (x[ids].double().transpose(0, 1).reshape(Hkv, -1, d)[:, :nk] for x in (s["k_pages"], s["v_pages"]))
            for h in range(Hq):
                O[at:at + nq, h], L[at:at + nq, h] = exact_rows(s["q"][at:at + nq, h].double(), k[h // g], v[h // g], nk - nq,
                                                                c["window"], c["sinks"], d ** -0.5)
            at += nq
        return O, L
    # append: the turned queries, and the pages with the turned keys in them (the values are copies)
    kp = s["k_pages"].double()
    qs, at = [], 0
    m = torch.arange(d // 2, device="cuda")
    lo, hi = (m, m + d // 2) if c["half"] else (2 * m, 2 * m + 1)
    for b, (nq, nk) in enumerate(lengths(c)):
        pos = torch.arange(nk - nq, nk, device="cuda")
        turn = torch.complex(s["cos"][pos].double(), s["sin"][pos].double())[:, None]
        new = []
        for x in (s["q"][at:at + nq], s["k"][at:at + nq]):
            x = x.double()
            z = torch.complex(x[..., lo], x[..., hi]) * turn
            y = torch.empty_like(x)
            y[..., lo], y[..., hi] = z.real, z.imag
            new.append(y)
        qs.append(new[0])
        kp[s["table"][b, pos // c["page"]].long(), :, pos % c["page"]] = new[1]
        at += nq
    return torch.cat(qs), kp, None
