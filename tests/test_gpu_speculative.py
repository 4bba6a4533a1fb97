"""Rounds of a serving loop that drafts trees: pages handed out, trees laid out,
keys turned and written, attention over them, the accepted path kept, pages given
back, and sequences forked -- all on the device, against a model in 64 bits that
holds each sequence as a plain list of tokens."""
import random

import pytest
import torch

import attn_inputs as gen
from rope_util import HALF, turn
from tree_util import layout, random_tree, reference, sees
from window_util import check_forward, ints

pytestmark = pytest.mark.gpu
ALL = 1 << 30


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


class Loop:
    def __init__(self, fa, rows, Hq, Hkv, d, r, dtype, page, pages, max_pages, layers, window, sinks, max_tree):
        self.fa, self.Hq, self.Hkv, self.d, self.r, self.dtype, self.page = fa, Hq, Hkv, d, r, dtype, page
        self.layers, self.window, self.sinks, self.max_tree = layers, window, sinks, max_tree
        self.k, self.v = (torch.full((layers, pages, Hkv, page, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        self.refs, self.table = ints([0] * pages), torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
        self.seq = ints([0] * rows)
        self.cos, self.sin = fa.rope_table(max_pages * page, r, 10000.0)
        # the model: for each layer and row the turned keys and the values as the cache holds them, [n, Hkv, d]
        empty = torch.zeros(0, Hkv, d, dtype=dtype, device="cuda")
        self.model = [[(empty, empty) for _ in range(rows)] for _ in range(layers)]
        self.seed = 0

    def step(self, trees, accept):
        """trees: parents for each row (may be empty; longer than max_tree: a chunk); accept(row, parents) -> kept nodes."""
        fa, rows = self.fa, len(trees)
        n = [len(t) for t in trees]
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        T = cu[-1]
        ctx = self.seq.clone()
        want = ctx + ints(n)
        fa.pages_resize(self.refs, self.table, self.seq, want, self.page)
        assert torch.equal(self.seq, want), "the pool is large enough"
        cu_q, parents = ints(cu), ints([p for t in trees for p in t])
        mask, pos = fa.tree_plan(parents, cu_q, self.seq, self.max_tree)
        rope = (self.cos, self.sin, HALF)
        words = -(-self.max_tree // 32)
        for layer in range(self.layers):
            self.seed += 1
            wide = torch.from_numpy(gen.normal((T, self.Hq + 2 * self.Hkv, self.d), self.seed, 0)).to(self.dtype).cuda()
            q, k, v = wide.split([self.Hq, self.Hkv, self.Hkv], dim=1)
            q = fa.cache_append(k, v, self.k[layer], self.v[layer], self.table, cu_q, self.seq, q=q, rope=rope, positions=pos)
            o, lse = fa.fwd_tree(q, self.k[layer], self.v[layer], self.table, cu_q, self.seq, mask, pos, window=self.window,
                                 sinks=self.sinks)
            fa.check_device_error()
            for b in range(rows):
                if n[b] == 0:
                    continue
                mk, mv = self.model[layer][b]
                c, r = mk.shape[0], slice(cu[b], cu[b + 1])
                seen, depth = layout(trees[b], words)
                # the same operator on plain tensors gives the turned keys' own bits
                at = [c + x for x in depth]
                kt, _ = fa.rope(k[r], None, rope, positions=ints(at))
                ref, _ = turn(k[r], self.cos[at][:, None], self.sin[at][:, None], HALF)
                assert float((kt.double() - ref).abs().max()) < 0.05
                mk, mv = torch.cat([mk, kt]), torch.cat([mv, v[r]])
                see = sees(n[b], c, seen, at, self.window, self.sinks, n[b] > 32 * words)
                want_ = reference(q[r], mk.transpose(0, 1), mv.transpose(0, 1), see, self.d ** -0.5)
                check_forward(o[r].transpose(0, 1), lse[r].transpose(0, 1), want_, self.dtype, self.d, mk.shape[0],
                              f"layer {layer} row {b}: {n[b]} over {c}")
                self.model[layer][b] = (mk, mv)
        # the accepted path moves up, and the rest's pages go back
        kept = [accept(b, t) for b, t in enumerate(trees)]
        most = max(len(x) for x in kept)
        first = ctx.tolist()
        keep = torch.zeros(rows, max(most, 1), dtype=torch.int32)
        for b, x in enumerate(kept):
            keep[b, :len(x)] = torch.tensor([first[b] + i for i in x], dtype=torch.int32)
        new = fa.cache_compact(self.k, self.v, self.table, ctx, keep.cuda(), ints([len(x) for x in kept]))
        fa.pages_resize(self.refs, self.table, self.seq, new, self.page)
        fa.check_device_error()
        for layer in range(self.layers):
            for b, x in enumerate(kept):
                mk, mv = self.model[layer][b]
                rows_ = torch.tensor(list(range(first[b])) + [first[b] + i for i in x], dtype=torch.long, device="cuda")
                self.model[layer][b] = (mk[rows_], mv[rows_])
        self.check()

    def fork(self, src, dst):
        want = self.seq.clone()
        want[ints(dst).long()] = 0
        self.fa.pages_resize(self.refs, self.table, self.seq, want, self.page)
        fresh = self.fa.pages_fork(self.k, self.v, self.refs, self.table, self.seq, ints(src), ints(dst))
        assert bool((fresh >= -1).all())
        for layer in range(self.layers):
            for a, b in zip(src, dst):
                self.model[layer][b] = self.model[layer][a]
        self.check()

    def check(self):
        """The cache holds the model's bits, and the counts are those of the table."""
        self.fa.check_device_error()
        seq, table = self.seq.tolist(), self.table.tolist()
        count = [0] * self.refs.shape[0]
        for b, n in enumerate(seq):
            pages = table[b][:-(-n // self.page)]
            assert all(p >= 0 for p in pages) and all(p == -1 for p in table[b][len(pages):])
            for p in pages:
                count[p] += 1
            ids = torch.tensor(pages, dtype=torch.long, device="cuda")
            for layer in range(self.layers):
                mk, mv = self.model[layer][b]
                assert mk.shape[0] == n
                for x, m in ((self.k[layer], mk), (self.v[layer], mv)):
                    got = x[ids].transpose(1, 2).reshape(-1, self.Hkv, self.d)[:n]
                    assert torch.equal(got.view(torch.int16), m.contiguous().view(torch.int16))
        assert self.refs.tolist() == count


def path_of(parents, rng):
    """A random accepted path: from a root down."""
    if not parents:
        return []
    node, path = rng.choice([i for i, p in enumerate(parents) if p < 0]), []
    while True:
        path.append(node)
        below = [i for i, p in enumerate(parents) if p == node]
        if not below or rng.random() < 0.2:
            return path
        node = rng.choice(below)


@pytest.mark.parametrize("d,r,Hq,Hkv,dtype,page,window,sinks", [(64, 64, 4, 2, torch.bfloat16, 16, ALL, 0), (128, 64, 8, 2, torch.float16, 32, 60, 3),
                                                               (256, 128, 2, 1, torch.bfloat16, 16, ALL, 0)])
def test_rounds(fa, d, r, Hq, Hkv, dtype, page, window, sinks):
    rng = random.Random(d)
    rows = 5
    loop = Loop(fa, rows, Hq, Hkv, d, r, dtype, page, pages=160, max_pages=60, layers=2, window=window, sinks=sinks, max_tree=40)
    # prompts as chunks (one of them short enough to be a line of nodes), one row empty
    prompts = [list(range(-1, n - 1)) for n in (70, 90, 33, 150, 0)]
    loop.step(prompts, lambda b, t: list(range(len(t))))
    for step in range(5):
        trees = [random_tree(rng.randint(1, 40), rng) if int(loop.seq[b]) else [] for b in range(rows)]
        if step == 2:
            trees[1] = list(range(-1, 99))  # a further chunk beside the trees
        loop.step(trees, lambda b, t: list(range(len(t))) if len(t) > 40 else path_of(t, rng))
        if step in (1, 3):
            loop.fork([0, 3] if step == 1 else [1, 1], [4, 2] if step == 1 else [0, 3])
    # eviction: sequence 0 keeps its first 4 and last 20 tokens, the others theirs
    n = loop.seq.tolist()
    kept = [list(range(4)) + list(range(max(4, x - 20), x)) if b == 0 else list(range(x)) for b, x in enumerate(n)]
    keep = torch.zeros(rows, max(n), dtype=torch.int32)
    for b, x in enumerate(kept):
        keep[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
    # (its pages are its own: after the forks above rows 0 and 3 continue row 1, so a copy of what is shared comes first)
    shared = [p for p in loop.table[0].tolist() if p >= 0 and int(loop.refs[p]) > 1]
    free = [p for p, c in enumerate(loop.refs.tolist()) if c == 0][:len(shared)]
    fa.cache_copy(loop.k, loop.v, ints(shared), ints(free))
    for a, b in zip(shared, free):
        loop.table[0][loop.table[0] == a] = b
        loop.refs[a] -= 1
        loop.refs[b] += 1
    loop.check()
    new = fa.cache_compact(loop.k, loop.v, loop.table, ints([0] * rows), keep.cuda(), ints([len(x) for x in kept]))
    fa.pages_resize(loop.refs, loop.table, loop.seq, new, page)
    for layer in range(2):
        loop.model[layer] = [tuple(t[torch.tensor(x, dtype=torch.long, device="cuda")] for t in m) for m, x in zip(loop.model[layer], kept)]
    loop.check()
    fa.pages_resize(loop.refs, loop.table, loop.seq, torch.zeros_like(loop.seq), page)
    assert int(loop.refs.sum()) == 0


def test_a_round_as_a_graph(fa):
    """One captured round, replayed with other trees and lengths, gives the bits of the calls made one by one."""
    rows, Hq, Hkv, d, page, T = 3, 4, 2, 128, 16, 24
    rng = random.Random(7)
    rope = (*fa.rope_table(400, 64), HALF)
    q, k, v = (torch.from_numpy(gen.normal((T, h, d), 3, i)).to(torch.bfloat16).cuda() for i, h in enumerate((Hq, Hkv, Hkv)))

    def state(lens):
        pages = torch.from_numpy(gen.normal((2, 40, Hkv, page, d), 5, 0)).to(torch.bfloat16).cuda()
        s = dict(k=pages[0].clone(), v=pages[1].clone(), refs=ints([0] * 40), table=torch.full((rows, 12), -1, dtype=torch.int32, device="cuda"),
                 seq=ints([0] * rows), want=ints(lens))
        fa.pages_resize(s["refs"], s["table"], s["seq"], s["want"], page)
        return s

    def round_(s, parents, cu, want, keep, keep_n, ws):
        ctx = s["seq"].clone()
        fa.pages_resize(s["refs"], s["table"], s["seq"], want, page)
        mask, pos = fa.tree_plan(parents, cu, s["seq"], 32)
        y = fa.cache_append(k, v, s["k"], s["v"], s["table"], cu, s["seq"], q=q, rope=rope, positions=pos)
        o, lse = fa.fwd_tree(y, s["k"], s["v"], s["table"], cu, s["seq"], mask, pos, window=90, sinks=1, workspace=ws)
        new = fa.cache_compact(s["k"], s["v"], s["table"], ctx, keep, keep_n)
        fa.pages_resize(s["refs"], s["table"], s["seq"], new, page)
        return o, lse

    def inputs(lens, sizes):
        trees = [random_tree(n, rng) for n in sizes]
        paths = [path_of(t, rng) for t in trees]
        keep = torch.zeros(rows, 12, dtype=torch.int32)
        for b, x in enumerate(paths):
            x = x[:12]
            keep[b, :len(x)] = torch.tensor([lens[b] + i for i in x], dtype=torch.int32)
        cu = [0, sizes[0], sizes[0] + sizes[1], sum(sizes)]
        return (ints([p for t in trees for p in t]), ints(cu), ints([a + b for a, b in zip(lens, sizes)]), keep.cuda(),
                ints([min(12, len(x)) for x in paths]))

    ws = torch.empty(fa.paged_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    first, second = ([20, 0, 133], [9, 8, 7]), ([3, 100, 47], [2, 20, 2])
    held, static = state(first[0]), inputs(*first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        round_(state(first[0]), *static, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = round_(held, *static, ws)
    torch.cuda.current_stream().wait_stream(side)
    for lens, sizes in (first, second):
        args, fresh, plain = inputs(lens, sizes), state(lens), state(lens)
        for name in fresh:
            held[name].copy_(fresh[name])
        for x, y in zip(static, args):
            x.copy_(y)
        g.replay()
        want = round_(plain, *args, ws)
        fa.check_device_error()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for name in ("k", "v", "refs", "table", "seq"):
            assert torch.equal(held[name].view(torch.int16) if held[name].dtype == torch.bfloat16 else held[name],
                               plain[name].view(torch.int16) if plain[name].dtype == torch.bfloat16 else plain[name]), name


def test_on_another_stream_while_the_default_one_works(fa):
    """Calls go to the current stream of the tensors' device, whatever else runs."""
    d = 128
    q = torch.from_numpy(gen.normal((2, 8, 3000, d), 1, 0)).to(torch.bfloat16).cuda()
    cos, sin = fa.rope_table(3000, d)
    want = fa.rope(q, None, (cos, sin, HALF))[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn(6000, 6000, device="cuda")
    for _ in range(20):
        busy = busy @ busy
        busy = busy / busy.norm()
    with torch.cuda.stream(side):
        c2, s2 = fa.rope_table(3000, d)
        got = fa.rope(q, None, (c2, s2, HALF))[0]
        side.synchronize()
        assert torch.equal(got, want)
    torch.cuda.synchronize()
