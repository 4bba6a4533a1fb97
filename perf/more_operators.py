"""Drafted trees, rotary positions and the cache's pages: the operators' cases, their plain forms and the calls a user
makes of them.

Three operators that a serving loop needs around paged attention once it drafts several tokens at a time, continues one
prompt in several ways, or runs past the lengths that a model was trained on; the rotation and its gradient serve
training as well:

* ``tree``    attention for trees of drafted tokens over a paged key/value cache: every node sees the cached keys (under
              a sliding window with sinks) and its own ancestors;
* rotary positions: ``rope`` turns queries and keys of a layer and their gradients back, ``table`` makes the angle tables,
  scaled for long contexts, ``append`` lays out drafted trees and writes their keys, turned in part of the head by the
  nodes' positions, into the cache;
* pages of the cache: ``fork`` drops sequences and continues others in their place, ``copy`` copies pages, ``compact``
  moves the tokens that are kept together.

A cache that pages are moved in has its layers in one tensor, [layers, pages, heads, page_size, d].
"""
import math
import random

import torch

own = False

NO_WINDOW = 1 << 30  # a window that hides nothing


# ---------------------------------------------------------------- cases --

def listed():
    t = dict(op="tree", dtype="bf16", d=128, page=64, window=NO_WINDOW, sinks=0, long=0, chunk=0)
    p = dict(dtype="bf16", Hkv=8, d=128, page=64)
    return [
        # two short conversations with a handful of drafted tokens each: latency
        dict(t, name="tree small", dtype="fp16", B=2, Hq=8, Hkv=1, d=256, page=16, nlo=5, nhi=9, klo=90, khi=140, mix=3),
        # a serving batch, each sequence with a full tree of drafts
        dict(t, name="tree batch", B=32, Hq=32, Hkv=8, nlo=60, nhi=60, klo=1000, khi=8000, mix=1),
        # one very long context
        dict(t, name="tree long", B=1, Hq=16, Hkv=2, page=32, nlo=26, nhi=26, klo=131000, khi=131000, mix=2),
        # a serving step under a window with sinks: trees, single tokens and a few chunks of prompts
        dict(t, name="tree mixed window", dtype="fp16", B=33, Hq=16, Hkv=4, d=64, page=32, window=1000, sinks=4, nlo=1, nhi=40,
             long=3, chunk=500, klo=600, khi=4000, mix=4),
        # a layer of a training step: queries and keys turned, their gradients turned back
        dict(op="rope", name="rope train", dtype="bf16", packed=False, B=2, Hq=16, Hkv=4, N=8192, d=128, r=128, half=True, far=0,
             back=True),
        # one decoding step far into a long context, part of the head, out of one fused projection
        dict(op="rope", name="rope decode", dtype="fp16", packed=True, B=1, Hq=32, Hkv=8, N=65, d=128, r=64, half=False,
             far=100000, back=False),
        # the angles of a context that was extended by parts
        dict(op="table", name="table long", n=131072, r=128, kind="turns", factor=8.0, original=16384),
        # the new nodes of every tree of a batch: laid out, turned and written into the pages
        dict(op="append", name="append trees", dtype="bf16", B=32, Hq=32, Hkv=8, d=128, r=64, page=64, nlo=60, nhi=60, klo=1000,
             khi=4000, half=True, mix=5),
        # one step of a beam search: half of the beams are dropped and the others continued in their place
        dict(p, op="fork", name="fork beams", layers=8, G=4, W=8, klo=600, khi=1500, mix=6),
        # pages moved to another place
        dict(p, op="copy", name="copy pages", layers=8, pairs=160),
        # the accepted nodes of each tree move up behind the cached tokens
        dict(p, op="compact", name="compact accepted", layers=8, B=32, klo=200, khi=1500, nlo=60, nhi=60, keep=8, mix=7),
        # a cache that keeps a quarter of its tokens: the first ones, and chosen ones of the rest
        dict(p, op="compact", name="compact evicted", layers=2, B=8, klo=0, khi=0, nlo=12000, nhi=16000, keep=4000, mix=8),
    ]


def spread(rng, lo, hi):
    """A whole number in [lo, hi], even in its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "rope", "table", "append", "fork", "copy", "compact"])
    mix = rng.randrange(1 << 20)
    dtype = rng.choice(["bf16", "fp16"])
    d = rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 7, 8])
    r = rng.choice([x for x in (16, 32, 64, 96, 128, 192, 256) if x <= d])
    half = rng.random() < 0.5
    if op == "tree":
        windowed = rng.random() < 0.4
        c = dict(op=op, dtype=dtype, Hq=Hkv * g, Hkv=Hkv, d=d, page=page, mix=mix, window=spread(rng, 30, 5000) if windowed else NO_WINDOW,
                 sinks=rng.choice([0, 1, 4, 130]) if windowed else 0, long=0, chunk=0)
        kind = rng.choice(["one", "batch", "batch", "mixed"])
        nhi = spread(rng, 1, 200)
        c.update(nlo=rng.randint(1, nhi), nhi=nhi)
        if kind == "one":
            khi = spread(rng, 20, 60000)
            c.update(B=1, klo=khi, khi=khi)
        else:
            B = spread(rng, 2, 40)
            khi = spread(rng, 20, 5000)
            c.update(B=B, klo=khi // 4, khi=khi)
            if kind == "mixed" and B >= 4:
                c.update(long=2, chunk=32 * (-(-nhi // 32)) + spread(rng, 1, 300))
        most = max(c["nhi"], c["chunk"])
        while c["B"] * c["Hq"] * most * (c["khi"] + most) > 1 << 29:
            if c["B"] > 4:
                c["B"] //= 2
            elif c["Hkv"] > 1:
                c["Hkv"] //= 2
                c["Hq"] //= 2
            else:
                c["khi"] = c["khi"] // 2 + 1
                c["klo"] = min(c["klo"], c["khi"])
        return c
    if op == "rope":
        packed = rng.random() < 0.5
        B = 1 if packed else spread(rng, 1, 4)
        N = spread(rng, 1, 8000 // B)
        return dict(op=op, dtype=dtype, packed=packed, B=B, Hq=Hkv * g, Hkv=Hkv, N=N, d=min(d, 128) if Hkv * g > 32 else d,
                    r=min(r, 128) if Hkv * g > 32 else r, half=half, far=spread(rng, 1, 100000) if packed else 0,
                    back=rng.random() < 0.5)
    if op == "table":
        kind = rng.choice(["none", "linear", "base", "turns", "index"])
        return dict(op=op, n=spread(rng, 1, 131072), r=rng.choice([16, 32, 64, 96, 128]), kind=kind, factor=rng.choice([1.5, 4.0, 32.0]),
                    original=spread(rng, 512, 16384))
    if op == "append":
        B = spread(rng, 1, 32)
        nhi = spread(rng, 1, 100)
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * g, Hkv=Hkv, d=d, r=r, page=page, nlo=rng.randint(1, nhi), nhi=nhi, klo=0,
                    khi=spread(rng, 1, 3000), half=half, mix=mix)
    c = dict(op=op, dtype=dtype, Hkv=Hkv, d=d, page=page, layers=spread(rng, 1, 16))
    if op == "fork":
        c.update(G=spread(rng, 1, 4), W=rng.choice([2, 3, 5, 8]), klo=page, khi=page + spread(rng, 1, 1200), mix=mix)
        rows = c["G"] * c["W"] * (c["khi"] // 3 + 2 * page) + c["G"] * c["khi"]
    elif op == "copy":
        c.update(pairs=spread(rng, 1, 300))
        rows = 2 * c["pairs"] * page
    else:
        nhi = spread(rng, 8, 4000)
        c.update(B=spread(rng, 1, 32), klo=0, khi=spread(rng, 1, 1000), nlo=nhi // 2, nhi=nhi, keep=max(1, nhi // 8), mix=mix)
        rows = c["B"] * (c["khi"] + nhi + page)
    while c["layers"] > 1 and rows * c["layers"] * Hkv * d > 1 << 27:
        c["layers"] = (c["layers"] + 1) // 2
    return c


TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def lengths(c):
    """The sequences of a ragged case: (new tokens, keys in the cache with them) for each.  With ``long`` > 0 that many
    of them bring a chunk of a prompt, the others a tree."""
    rng = random.Random(c["mix"])
    got = []
    for b in range(c["B"]):
        n = rng.randint(c["nlo"], c["nhi"])
        if c.get("long", 0) and b % (c["B"] // c["long"]) == 0:
            n = c["chunk"]
        got.append((n, n + rng.randint(c["klo"], c["khi"])))
    return got


def forest(c):
    """The nodes' parents, sequence by sequence: -1 for the first (the last accepted token), else an earlier node; a
    chunk's tokens follow one another."""
    rng = random.Random(c["mix"] + 1)
    got = []
    for n, _ in lengths(c):
        width = rng.randint(1, 12)
        chunk = n > 32 * words(c)
        got.append([-1] + [i - 1 if chunk else rng.randrange(max(0, i - width), i) for i in range(1, n)])
    return got


def words(c):
    return -(-c["nhi"] // 32)


def depths(parents):
    got = []
    for p in parents:
        got.append(0 if p < 0 else got[p] + 1)
    return got


def frequencies(c, theta):
    """The angle per position of each pair of a table case, in 64 bits."""
    r, s, kind = c["r"], c["factor"], c["kind"]
    if kind == "base":
        theta = theta * s ** (r / (r - 2))
    f = [theta ** (-2.0 * i / r) for i in range(r // 2)]
    if kind == "linear":
        return [x / s for x in f]
    if kind == "turns":  # between one and four turns over the original length
        keep = [min(1.0, max(0.0, (c["original"] * x / (2 * math.pi) - 1.0) / 3.0)) for x in f]
        return [(1 - k) * x / s + k * x for x, k in zip(f, keep)]
    if kind == "index":  # between the pairs that make 32 turns and one over the original length
        at = [r * math.log(c["original"] / (w * 2 * math.pi)) / (2 * math.log(theta)) for w in (32.0, 1.0)]
        lo, hi = max(0, math.floor(at[0])), min(r - 1, math.ceil(at[1]))
        keep = [1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(r // 2)]
        return [(1 - k) * x / s + k * x for x, k in zip(f, keep)]
    return f


def scaling(c):
    """The same as a user states it."""
    amplitude = 0.1 * math.log(c["factor"]) + 1.0 if c["kind"] == "index" else 1.0
    if c["kind"] == "none":
        return None
    got = dict(kind=c["kind"], factor=c["factor"], amplitude=amplitude)
    if c["kind"] == "turns":
        got.update(original=c["original"], low=1.0, high=4.0)
    if c["kind"] == "index":
        got.update(original=c["original"], low=1.0, high=32.0)
    return got


# -------------------------------------------------------------- prepare --

def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TYPES.get(c.get("dtype"))

    def normal(*shape):
        x = torch.empty(shape, dtype=dt, device="cuda")
        return x.normal_(generator=gen)

    def scattered(need, pages):
        """Every sequence's pages lie scattered over the cache; table entries past its last page are not in use."""
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((len(need), max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        return table, order[at:]

    s = dict(c=c)
    op = c["op"]
    if op == "table":
        rng = random.Random(seed)
        s["theta"], s["start"] = rng.uniform(1e4, 1e6), rng.randrange(1 << 15)
        return s
    d = c["d"]
    if op == "rope":
        B, Hq, Hkv, N, r = (c[n] for n in ("B", "Hq", "Hkv", "N", "r"))
        if c["packed"]:
            s["q"], s["k"], _ = normal(N, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], dim=1)
            s["gq"], s["gk"] = normal(N, Hq, d), normal(N, Hkv, d)
            s["pos"] = torch.randint(0, c["far"], (N,), generator=gen, device="cuda", dtype=torch.int32)
        else:
            s["q"], s["k"], s["gq"], s["gk"] = normal(B, Hq, N, d), normal(B, Hkv, N, d), normal(B, Hq, N, d), normal(B, Hkv, N, d)
            s["pos"] = None
        s["cos"], s["sin"] = angles(max(N, c["far"]), r)
        return s
    if op == "copy":
        pages = 2 * c["pairs"] + 3
        s["k_pages"], s["v_pages"] = (normal(c["layers"], pages, c["Hkv"], c["page"], d) for _ in range(2))
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        s["src"], s["dst"] = order[:c["pairs"]].contiguous(), order[c["pairs"]:2 * c["pairs"]].contiguous()
        return s
    if op == "fork":
        return prepare_fork(c, s, normal, gen)
    lens, ps = lengths(c), c["page"]
    need = [-(-nk // ps) for _, nk in lens]
    s["seq_k"] = ints([nk for _, nk in lens])
    if op == "compact":
        pages = sum(need) + 1
        s["table"], s["spare"] = scattered(need, pages)
        s["k_pages"], s["v_pages"] = (normal(c["layers"], pages, c["Hkv"], ps, d) for _ in range(2))
        rng = random.Random(c["mix"] + seed)
        keep = torch.zeros(len(lens), c["keep"], dtype=torch.int32)
        count = []
        for b, (n, nk) in enumerate(lens):
            # the first of them stay where they are, the others come from behind all that is kept
            m = min(rng.randint((c["keep"] + 1) // 2, c["keep"]), (n + 1) // 2)
            same = rng.randint(1, max(1, m // 4))
            kept = list(range(same)) + sorted(rng.sample(range(m, n), m - same))
            keep[b, :m] = torch.tensor(kept, dtype=torch.int32) + (nk - n)
            count.append(m)
        s["first"], s["keep"], s["keep_n"] = ints([nk - n for n, nk in lens]), keep.cuda(), ints(count)
        return s
    pages = sum(need) + 3
    s["table"], _ = scattered(need, pages)
    s["k_pages"], s["v_pages"] = (normal(pages, c["Hkv"], ps, d) for _ in range(2))
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    T = cu[-1]
    trees = forest(c)
    s["cu_q"], s["parents"] = ints(cu), ints([p for t in trees for p in t])
    if op == "append":
        s["q"], s["k"], s["v"] = normal(T, c["Hq"] + 2 * c["Hkv"], d).split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        s["cos"], s["sin"] = angles(c["khi"] + c["nhi"], c["r"])
        return s
    # what the step has laid out for all of its layers
    s["q"] = normal(T, c["Hq"], d)
    s["max_q"], s["max_k"], s["scale"] = max(n for n, _ in lens), max(nk for _, nk in lens), d ** -0.5
    W = words(c)
    mask, pos = torch.zeros(T, W, dtype=torch.int64), []
    for b, (n, nk) in enumerate(lens):
        pos += [nk - n + x for x in depths(trees[b])]
        if n > 32 * W:
            continue
        rows = []
        for i, p in enumerate(trees[b]):
            rows.append((1 << i) | (rows[p] if p >= 0 else 0))
            for w in range(W):
                mask[cu[b] + i, w] = (rows[i] >> (32 * w)) & 0xffffffff
    s["mask"] = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32).cuda()
    s["positions"] = ints(pos)
    return s


def angles(n, r):
    pos = torch.arange(n, dtype=torch.float64, device="cuda")
    ang = pos[:, None] * 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64, device="cuda") / r)
    return ang.cos().float(), ang.sin().float()


def prepare_fork(c, s, normal, gen):
    """Groups of beams that share the full pages of a prompt and go on in pages of their own; in a step the odd beams are
    dropped and even ones of their group continued in their place."""
    rng = random.Random(c["mix"])
    ps, G, W = c["page"], c["G"], c["W"]
    group, fresh = [], 0
    for _ in range(G):
        n = rng.randint(c["klo"], c["khi"])
        group.append((n, 2 * n // 3 // ps))  # tokens of each beam, pages they share
        fresh += group[-1][1] + W * (-(-n // ps) - group[-1][1])
    pages = fresh + 5
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    table = torch.full((G * W, max(-(-n // ps) for n, _ in group)), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    src, dst = [], []
    for b, (n, shared) in enumerate(group):
        common = [order.pop() for _ in range(shared)]
        for w in range(W):
            row = common + [order.pop() for _ in range(-(-n // ps) - shared)]
            table[b * W + w, :len(row)] = torch.tensor(row, dtype=torch.int32)
            refs[row] += 1
            if w % 2 == 1:
                dst.append(b * W + w)
                src.append(b * W + 2 * rng.randrange((W + 1) // 2))
    s["table"], s["refs"], s["src"], s["dst"] = table.cuda(), refs.cuda(), ints(src), ints(dst)
    s["seq_k"] = ints([n for n, _ in group for _ in range(W)])
    s["want"] = s["seq_k"].clone()
    s["want"][s["dst"].long()] = 0
    s["k_pages"], s["v_pages"] = (normal(c["layers"], pages, c["Hkv"], ps, c["d"]) for _ in range(2))
    return s


# ---------------------------------------------------------- plain forms --

def rows_of(s):
    """For each new token: its sequence and its place among that sequence's new tokens."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    return b, t - s["cu_q"].long()[b]


def bits(mask):
    """[T, words] of 32 bits -> [T, 32 words] truth values."""
    return ((mask[:, :, None] >> torch.arange(32, device=mask.device, dtype=torch.int32)) & 1).flatten(1).bool()


def tree_plain(s):
    c = s["c"]
    Hq, Hkv, d, ps, B, T = c["Hq"], c["Hkv"], c["d"], c["page"], c["B"], s["q"].shape[0]
    g, mq, mk = Hq // Hkv, s["max_q"], s["max_k"]
    b, i = rows_of(s)
    j = torch.arange(mk, device="cuda")
    page = s["table"].long()[:, j // ps].clamp(min=0)
    k, v = (x[page, :, j % ps].permute(0, 2, 1, 3).float() for x in (s["k_pages"], s["v_pages"]))  # [B, Hkv, max_k, d]
    q = torch.zeros(B, mq, Hq, d, device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, mq, Hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * mq, d)
    nq, nk = (s["cu_q"][1:] - s["cu_q"][:-1]).long(), s["seq_k"].long()
    ctx = (nk - nq)[b][:, None]
    pos = s["positions"].long()[:, None]
    cached = (j < ctx) & ((j > pos - c["window"]) | (j < c["sinks"]))
    # a node sees its ancestors and itself; the tokens of a chunk, too long for the mask, those of their window
    node = j - ctx
    tree = bits(s["mask"]).gather(1, node.clamp(0, 32 * s["mask"].shape[1] - 1)) & (node >= 0) & (node <= i[:, None])
    chunk = (node >= 0) & (node <= i[:, None]) & ((j > pos - c["window"]) | (j < c["sinks"]))
    see = torch.zeros(B, mq, mk, dtype=torch.bool, device="cuda")
    see[b, i] = cached | torch.where(nq[b][:, None] > 32 * s["mask"].shape[1], chunk, tree)
    see = see.repeat(1, g, 1)[:, None]
    e = q @ k.transpose(-1, -2)
    e.mul_(s["scale"]).masked_fill_(~see, -math.inf)
    m = e.amax(-1, keepdim=True)
    e.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = e.sum(-1, keepdim=True)
    o = e @ v
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).view(B, Hkv, g, mq, d).permute(0, 3, 1, 2, 4)[b, i]
    lse = (m + l.log()).view(B, Hkv, g, mq).permute(0, 3, 1, 2)[b, i]
    return o.reshape(T, Hq, d).to(s["q"].dtype), lse.reshape(T, Hq)


def turned(x, cos, sin, half):
    """Rotary positions of the first columns: pairs (i, i + r/2) (half) or (2i, 2i + 1) of r, the others as they are."""
    r = 2 * cos.shape[-1]
    y = x[..., :r].float()
    a, b = y.chunk(2, -1) if half else (y[..., 0::2], y[..., 1::2])
    y, z = a * cos - b * sin, a * sin + b * cos
    y = torch.cat([y, z], -1) if half else torch.stack([y, z], -1).flatten(-2)
    return torch.cat([y.to(x.dtype), x[..., r:]], -1)


def rope_plain(s):
    c = s["c"]
    if c["packed"]:
        cos, sin = (t[s["pos"].long()][:, None] for t in (s["cos"], s["sin"]))
    else:
        cos, sin = s["cos"], s["sin"]
    out = [turned(s[n], cos, sin, c["half"]) for n in ("q", "k")]
    if c["back"]:
        out += [turned(s[n], cos, -sin, c["half"]) for n in ("gq", "gk")]
    return tuple(out)


def table_plain(s):
    c = s["c"]
    f = torch.tensor(frequencies(c, s["theta"]), dtype=torch.float64, device="cuda")
    pos = torch.arange(s["start"], s["start"] + c["n"], dtype=torch.float64, device="cuda")
    ang = pos[:, None] * f
    amplitude = (scaling(c) or {}).get("amplitude", 1.0)
    return (ang.cos() * amplitude).float(), (ang.sin() * amplitude).float()


def append_plain(s):
    c, dt = s["c"], s["q"].dtype
    b, i = rows_of(s)
    W = words(c)
    # ancestors, doubling the step: after k rounds those up to 2^k - 1 levels up are known
    base = s["cu_q"].long()[b]
    T = base.shape[0]
    up = torch.where(s["parents"] >= 0, s["parents"].long() + base, torch.full_like(base, T))
    up = torch.cat([up, up.new_full((1,), T)])
    seen = torch.zeros(T + 1, 32 * W, dtype=torch.bool, device="cuda")
    seen[torch.arange(T, device="cuda"), i] = True
    for _ in range(max(1, (32 * W - 1).bit_length())):
        seen = seen | seen[up]
        up = up[up]
    seen = seen[:T]
    value = (seen.view(T, W, 32).long() << torch.arange(32, device="cuda")).sum(-1)
    mask = torch.where(value >= 1 << 31, value - (1 << 32), value).to(torch.int32)
    at = s["seq_k"].long()[b] - (s["cu_q"][1:] - s["cu_q"][:-1]).long()[b]
    pos = at + seen.sum(-1) - 1
    at = at + i
    page, at = s["table"].long()[b, at // c["page"]], at % c["page"]
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    s["k_pages"][page, :, at] = turned(s["k"], cos, sin, c["half"])
    s["v_pages"][page, :, at] = s["v"]
    return mask, pos.to(torch.int32), turned(s["q"], cos, sin, c["half"]), s["k_pages"], s["v_pages"]


def free_pages(refs):
    """The free pages, lowest first, and how many they are."""
    free = refs == 0
    return torch.argsort((~free).to(torch.int32), stable=True), free.sum()


def resize_plain(refs, table, seq_k, want, ps):
    """Rows give back the pages that their new length does not need, then rows that grow get the lowest free ones."""
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    hold, goal = (seq_k.long() + ps - 1)[:, None] // ps, (want.long() + ps - 1)[:, None] // ps
    drop = (col >= goal) & (col < hold)
    refs.index_add_(0, table.long().clamp(min=0).flatten(), -drop.to(torch.int32).flatten())
    table.masked_fill_(drop, -1)
    more = (col >= hold) & (col < goal)
    rank = more.flatten().long().cumsum(0).view_as(more) - 1
    order, free = free_pages(refs)
    got = more & (rank < free)
    page = order[rank.clamp(0, refs.shape[0] - 1)]
    table.copy_(torch.where(got, page, torch.where(more, torch.full_like(page, -1), table.long())))
    refs.index_add_(0, torch.where(got, page, torch.zeros_like(page)).flatten(), got.to(torch.int32).flatten())
    room = (torch.minimum(hold[:, 0], goal[:, 0]) + got.sum(1)) * ps
    seq_k.copy_(torch.minimum(want.long(), room))


def fork_plain(s):
    ps, refs, table, seq_k = s["c"]["page"], s["refs"], s["table"], s["seq_k"]
    resize_plain(refs, table, seq_k, s["want"], ps)
    src, dst = s["src"].long(), s["dst"].long()
    n = seq_k.long()[src]
    full, rest = n // ps, n % ps
    old = table.long()[src]
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    share = col < full[:, None]
    refs.index_add_(0, old.clamp(min=0).flatten(), share.to(torch.int32).flatten())
    order, _ = free_pages(refs)
    new = order[((rest > 0).long().cumsum(0) - 1).clamp(min=0)]
    last = old.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    new, last = torch.where(rest > 0, new, old[:, 0]), torch.where(rest > 0, last, old[:, 0])
    refs.index_add_(0, new, (rest > 0).to(torch.int32))
    table[dst] = torch.where(share, old, torch.where((col == full[:, None]) & (rest > 0)[:, None], new[:, None], table.long()[dst])).to(torch.int32)
    seq_k[dst] = n.to(torch.int32)
    copied = (torch.arange(ps, device="cuda")[None, :] < rest[:, None])[None, :, None, :, None]
    for x in (s["k_pages"], s["v_pages"]):
        x[:, new] = torch.where(copied, x[:, last], x[:, new])
    return refs, table, seq_k, s["k_pages"], s["v_pages"]


def copy_plain(s):
    for x in (s["k_pages"], s["v_pages"]):
        x[:, s["dst"].long()] = x[:, s["src"].long()]
    return s["k_pages"], s["v_pages"]


def compact_plain(s):
    ps, table = s["c"]["page"], s["table"].long()
    i = torch.arange(s["keep"].shape[1], device="cuda")[None, :]
    real = i < s["keep_n"][:, None]
    a, z = s["keep"].long(), s["first"].long()[:, None] + i
    # places behind the kept ones: a row of a page that no sequence has, onto itself
    spare = s["spare"].long()[0]
    where = []
    for t in (a, z):
        t = torch.where(real, t, torch.zeros_like(t))
        where.append((torch.where(real, table.gather(1, t // ps), spare).flatten(), torch.where(real, t % ps, torch.zeros_like(t)).flatten()))
    (sp, sr), (dp, dr) = where
    for x in (s["k_pages"], s["v_pages"]):
        x[:, dp, :, dr] = x[:, sp, :, sr]
    return s["first"] + s["keep_n"], s["k_pages"], s["v_pages"]


PLAIN = dict(tree=tree_plain, rope=rope_plain, table=table_plain, append=append_plain, fork=fork_plain, copy=copy_plain,
             compact=compact_plain)


# ------------------------------------------------------------------ run --

def own_run(s):
    import exact_attention_forward_09_gb300 as fa
    c = s["c"]
    op = c["op"]
    if op == "tree":
        return fa.fwd_tree(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu_q"], s["seq_k"], s["mask"], s["positions"],
                           window=c["window"], sinks=c["sinks"], max_q=s["max_q"])
    if op == "table":
        return fa.rope_table(c["n"], c["r"], theta=s["theta"], scaling=scaling(c), start=s["start"])
    if op == "copy":
        fa.cache_copy(s["k_pages"], s["v_pages"], s["src"], s["dst"])
        return s["k_pages"], s["v_pages"]
    if op == "fork":
        fa.pages_resize(s["refs"], s["table"], s["seq_k"], s["want"], c["page"])
        fa.pages_fork(s["k_pages"], s["v_pages"], s["refs"], s["table"], s["seq_k"], s["src"], s["dst"])
        return s["refs"], s["table"], s["seq_k"], s["k_pages"], s["v_pages"]
    if op == "compact":
        n = fa.cache_compact(s["k_pages"], s["v_pages"], s["table"], s["first"], s["keep"], s["keep_n"])
        return n, s["k_pages"], s["v_pages"]
    rope = (s["cos"], s["sin"], fa.FA_ROPE_HALF if c["half"] else fa.FA_ROPE_INTERLEAVED)
    if op == "rope":
        out = fa.rope(s["q"], s["k"], rope, positions=s["pos"])
        return out + fa.rope(s["gq"], s["gk"], rope, positions=s["pos"], inverse=True) if c["back"] else out
    mask, pos = fa.tree_plan(s["parents"], s["cu_q"], s["seq_k"], c["nhi"])
    q = fa.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cu_q"], s["seq_k"], q=s["q"], rope=rope,
                        positions=pos)
    return mask, pos, q, s["k_pages"], s["v_pages"]


def run(s):
    return own_run(s) if own else PLAIN[s["c"]["op"]](s)


def work(c):
    op = c["op"]
    if op == "table":
        return {"bytes": 4 * c["n"] * c["r"], "flops": 2 * c["n"] * c["r"]}
    Hkv, d = c["Hkv"], c["d"]
    token = 2 * 2 * Hkv * d * c.get("layers", 1)  # a token's keys and values
    if op == "copy":
        return {"bytes": 2 * token * c["pairs"] * c["page"], "flops": 0}
    if op == "fork":
        rng = random.Random(c["mix"])
        n = [rng.randint(c["klo"], c["khi"]) for _ in range(c["G"])]
        beams = c["W"] // 2
        return {"bytes": sum(beams * (2 * token * (x % c["page"]) + 16 * (-(-x // c["page"]))) for x in n), "flops": 0}
    if op == "compact":
        # (about: how many of the kept ones move depends on the seed)
        rows = sum(min(3 * c["keep"] // 4, (n + 1) // 2) * 7 // 8 for n, _ in lengths(c))
        return {"bytes": 2 * token * rows + 4 * rows, "flops": 0}
    Hq = c["Hq"]
    if op == "rope":
        n = c["B"] * c["N"]
        passes = 2 if c["back"] else 1
        return {"bytes": passes * 2 * 2 * d * n * (Hq + Hkv) + 4 * c["N"] * c["r"], "flops": passes * 3 * c["r"] * n * (Hq + Hkv)}
    lens = lengths(c)
    T = sum(n for n, _ in lens)
    if op == "append":
        return {"bytes": 2 * d * T * (2 * Hq + 4 * Hkv) + 4 * T * (c["r"] + 2 + words(c)), "flops": 3 * c["r"] * T * (Hq + Hkv)}
    pairs, keys = 0, 0
    for (n, nk), parents in zip(lens, forest(c)):
        ctx = nk - n
        for x in depths(parents):
            lo = max(0, min(ctx, ctx + x - c["window"] + 1))
            pairs += min(x + 1, c["window"]) if n > 32 * words(c) else x + 1
            pairs += ctx - lo + min(c["sinks"], lo)
        lo = max(0, ctx - c["window"] + 1)
        keys += nk - lo + min(c["sinks"], lo)
    return {"bytes": 2 * d * (2 * T * Hq + 2 * keys * Hkv) + 4 * T * (Hq + words(c) + 1), "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------- exact --

def exact_turn(x, cos, sin, half, back=False):
    """Rows of x turned as complex numbers, in 64 bits."""
    r = 2 * cos.shape[-1]
    m = torch.arange(r // 2, device=x.device)
    lo, hi = (m, m + r // 2) if half else (2 * m, 2 * m + 1)
    turn = torch.complex(cos.double(), sin.double())
    x = x.double()
    z = torch.complex(x[..., lo], x[..., hi]) * (turn.conj() if back else turn)
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def exact(c, seed):
    op = c["op"]
    if op in ("fork", "copy", "compact"):
        return None  # copies and whole numbers
    s = prepare(c, seed)
    if op == "table":
        f = torch.tensor(frequencies(c, s["theta"]), dtype=torch.float64, device="cuda")
        p = torch.arange(c["n"], dtype=torch.float64, device="cuda") + s["start"]
        turns = torch.polar(torch.full((c["n"], c["r"] // 2), (scaling(c) or {}).get("amplitude", 1.0), dtype=torch.float64, device="cuda"),
                            torch.outer(p, f))
        return turns.real, turns.imag
    if op == "rope":
        at = s["pos"].long() if c["packed"] else torch.arange(c["N"], device="cuda")
        cos, sin = s["cos"][at], s["sin"][at]
        if c["packed"]:
            cos, sin = cos[:, None], sin[:, None]
        out = [exact_turn(s[n], cos, sin, c["half"]) for n in ("q", "k")]
        return tuple(out + [exact_turn(s[n], cos, sin, c["half"], True) for n in ("gq", "gk")] if c["back"] else out)
    lens, trees, Hq, Hkv, d, ps = lengths(c), forest(c), c["Hq"], c["Hkv"], c["d"], c["page"]
    if op == "append":
        kp, qs, at = s["k_pages"].double(), [], 0
        for b, (n, nk) in enumerate(lens):
            pos = torch.tensor(depths(trees[b]), device="cuda") + (nk - n)
            cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
            qs.append(exact_turn(s["q"][at:at + n], cos, sin, c["half"]))
            slot = torch.arange(nk - n, nk, device="cuda")
            kp[s["table"][b, slot // ps].long(), :, slot % ps] = exact_turn(s["k"][at:at + n], cos, sin, c["half"])
            at += n
        return None, None, torch.cat(qs), kp, None
    if work(c)["flops"] > 6e12:
        return None
    g, scale = Hq // Hkv, d ** -0.5
    T = s["q"].shape[0]
    O, L = torch.empty(T, Hq, d, dtype=torch.float64, device="cuda"), torch.empty(T, Hq, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, nk) in enumerate(lens):
        ctx, parents = nk - n, trees[b]
        depth = torch.tensor(depths(parents), device="cuda")[:, None]
        line = torch.zeros(n, n, dtype=torch.bool)  # what of the new tokens each one descends from
        for i, p in enumerate(parents):
            if p >= 0:
                line[i] = line[p]
            line[i, i] = True
        line = line.cuda()
        if n > 32 * words(c):
            far = (depth - torch.arange(n, device="cuda")[None, :] >= c["window"]) & (torch.arange(nk - n, nk, device="cuda") >= c["sinks"])
            line &= ~far
        j = torch.arange(ctx, device="cuda")[None, :]
        see = torch.cat([(ctx + depth - j < c["window"]) | (j < c["sinks"]), line], 1)
        ids = s["table"][b, :-(-nk // ps)].long()
        k, v = (x[ids].double().transpose(0, 1).reshape(Hkv, -1, d)[:, :nk] for x in (s["k_pages"], s["v_pages"]))
        for h in range(Hkv):
            a = torch.einsum("thd,jd->thj", s["q"][at:at + n, h * g:(h + 1) * g].double(), k[h]) * scale
            a = torch.where(see[:, None], a, torch.full_like(a, -math.inf))
            lse = torch.logsumexp(a, -1)
            w = torch.exp(a - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
            O[at:at + n, h * g:(h + 1) * g] = torch.einsum("thj,jd->thd", w, v[h])
            L[at:at + n, h * g:(h + 1) * g] = lse
        at += n
    return O, L
