"""Trees of drafted tokens (fa_tree_plan, fa_fwd_tree) against plain models,
within bounds derived from the arithmetic.  Everything a cache holds beside the
sequences' own rows is NaN: nothing of it may reach a result."""
import math
import random

import pytest
import torch

import attn_inputs as gen
from tree_util import layout, mask_of, random_tree, reference, sees
from window_util import Paged, check_forward, ints

pytestmark = pytest.mark.gpu
ALL = 1 << 30


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _reported(fa):
    try:
        fa.check_device_error()
    except fa.FaError as e:
        assert e.status == fa.FA_ERR_INDEX
        fa.check_device_error()
        return True
    return False


def _normal(shape, seed, stream, dtype):
    return torch.from_numpy(gen.normal(shape, seed, stream)).to(dtype).cuda()


class Batch:
    """lens: [(new tokens, keys)], sequences of more than 32 * words tokens chunks."""

    def __init__(self, lens, Hq, Hkv, d, dtype, page, words, seed=1, trees=None, **kw):
        rng = random.Random(seed)
        self.lens, self.words = lens, words
        self.seqs = [tuple(_normal((Hkv, max(nk, 0), d), seed, 10 * b + i, dtype) for i in (1, 2)) for b, (_, nk) in enumerate(lens)]
        self.cache = Paged(self.seqs, page, seed=seed, **kw)
        cu = [0]
        for n, _ in lens:
            cu.append(cu[-1] + n)
        self.T = cu[-1]
        self.q = _normal((self.T, Hq, d), seed, 0, dtype)
        self.cu, self.sk = ints(cu), ints([nk for _, nk in lens])
        self.chunk = [n > 32 * words for n, _ in lens]
        self.parents = trees or [list(range(-1, n - 1)) if c else random_tree(n, rng) for (n, _), c in zip(lens, self.chunk)]
        self.rows, depths = zip(*[layout(p, words) for p in self.parents])
        self.pos = [[nk - n + x for x in dep] for (n, nk), dep in zip(lens, depths)]
        self.mask = torch.cat([mask_of(r, words) for r in self.rows]).cuda()
        self.positions = ints([p for x in self.pos for p in x])

    def run(self, fa, **kw):
        c = self.cache
        return fa.fwd_tree(self.q, c.k, c.v, c.table, self.cu, self.sk, kw.pop("mask", self.mask), kw.pop("positions", self.positions), **kw)

    def check(self, o, lse, what, window=ALL, sinks=0, scale=None, rows=None, pos=None):
        d, at = self.q.shape[2], 0
        for b, ((n, nk), (k, v)) in enumerate(zip(self.lens, self.seqs)):
            r = slice(at, at + n)
            if n:
                see = sees(n, nk - n, (rows or self.rows)[b], (pos or self.pos)[b], window, sinks, self.chunk[b])
                ref = reference(self.q[r], k, v, see, d ** -0.5 if scale is None else scale)
                check_forward(o[r].transpose(0, 1), lse[r].transpose(0, 1), ref, self.q.dtype, d, max(nk, 1), f"{what} sequence {b} ({n}, {nk})")
            at += n


def _run(fa, lens, Hq, Hkv, d, dtype, page, words=2, window=ALL, sinks=0, scale=None, max_q=0, **kw):
    x = Batch(lens, Hq, Hkv, d, dtype, page, words, **kw)
    o, lse = x.run(fa, window=window, sinks=sinks, scale=scale, max_q=max_q)
    fa.check_device_error()
    x.check(o, lse, f"Hq{Hq} Hkv{Hkv} d{d} page{page} w{window} s{sinks} max_q{max_q}", window, sinks, scale)
    return x, o, lse


# ------------------------------------------------------------------ plan --

@pytest.mark.parametrize("words,sizes", [(1, [1, 2, 32, 31, 0, 7]), (2, [64, 33, 1, 60, 65, 200]), (5, [160, 161, 3, 150]),
                                         (32, [1024, 1000, 500, 1025, 2048, 1])])
def test_plan(fa, words, sizes):
    lens = [(n, n + 13 * i) for i, n in enumerate(sizes)]
    rng = random.Random(words)
    trees = [list(range(-1, n - 1)) if n > 32 * words or n == 1000 else random_tree(n, rng) for n in sizes]  # (one tree is a line)
    cu = [0]
    for n in sizes:
        cu.append(cu[-1] + n)
    mask, pos = fa.tree_plan(ints([p for t in trees for p in t]), ints(cu), ints([nk for _, nk in lens]), 32 * words)
    assert not _reported(fa)
    rows, depths = zip(*[layout(t, words) for t in trees])
    assert torch.equal(mask.cpu(), torch.cat([mask_of(r, words) for r in rows]))
    assert pos.tolist() == [nk - n + x for (n, nk), dep in zip(lens, depths) for x in dep]


def test_plan_takes_max_tree_up_to_words(fa):
    p = ints([-1, 0, 0])
    for most, words in ((1, 1), (32, 1), (33, 2), (1024, 32)):
        assert fa.tree_plan(p, ints([0, 3]), ints([3]), most)[0].shape == (3, words)


def test_plan_leaves_rows_outside_and_reports_bad_parents(fa):
    parents = ints([9, 9, -1, 0, 2, -2, 1, 0, 5, -1, 0, 0, 7])
    # rows 0, 1 before the sequences, 12 behind them; sequence 0: nodes 2 (its own number) and 3 (-2) are bad
    cu, sk = ints([2, 6, 12]), ints([14, 6])
    mask, pos = torch.full((13, 1), 77, dtype=torch.int32, device="cuda"), torch.full((13,), 77, dtype=torch.int32, device="cuda")
    fa.tree_plan(parents, cu, sk, 32, mask=mask, positions=pos)
    assert _reported(fa)
    # sequence 1: parents 1 (bad: not before it), 0, 5 (bad), -1, 0, 0
    assert mask[:, 0].tolist() == [77, 77, 1, 3, 4, 8, 1, 3, 4, 8, 17, 33, 77]
    assert pos.tolist() == [77, 77, 10, 11, 10, 10, 0, 1, 0, 0, 1, 1, 77]
    # a chunk whose tokens do not follow one another
    long = list(range(-1, 39))
    fa.tree_plan(ints(long), ints([0, 40]), ints([40]), 32)
    assert not _reported(fa)
    long[20] = 3
    fa.tree_plan(ints(long), ints([0, 40]), ints([40]), 32)
    assert _reported(fa)


def test_plan_of_nothing(fa):
    mask, pos = fa.tree_plan(ints([]), ints([0, 0]), ints([5]), 64)
    assert mask.shape == (0, 2) and pos.shape == (0,)


# --------------------------------------------------------------- forward --

FEW = [(1, 1), (2, 2), (1, 130), (4, 129), (3, 128), (2, 1000), (4, 2500), (3, 67)]
TREES = [(1, 1), (5, 5), (33, 33), (60, 700), (64, 192), (17, 136), (31, 150), (2, 129), (0, 40), (64, 64 + 127), (50, 1500)]


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("max_q", [4, 0])
def test_few_nodes(fa, d, page, max_q):
    # up to 16 rows to a unit, and the same batch without the hint
    _run(fa, FEW, 8, 2, d, torch.bfloat16, page, words=1, max_q=max_q)


@pytest.mark.parametrize("page", [16, 64, 512])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2)])
def test_trees(fa, d, page, Hq, Hkv):
    _run(fa, TREES, Hq, Hkv, d, torch.float16 if page == 64 else torch.bfloat16, page)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (10, 2), (7, 1), (128, 1), (100, 1)])
@pytest.mark.parametrize("d", [64, 256])
def test_head_groups(fa, Hq, Hkv, d):
    _run(fa, [(1, 300), (9, 200), (40, 40), (64, 140)], Hq, Hkv, d, torch.float16, 32)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_where_the_nodes_begin_in_a_tile(fa, d):
    # one sequence for each place at which the nodes can begin, near the ends of tiles and words
    lens = [(37, 37 + c) for c in (*range(0, 4), *range(28, 36), *range(60, 66), *range(90, 98), *range(122, 134), 255, 256, 257)]
    _run(fa, lens, 2, 1, d, torch.bfloat16, 32, junk=float("nan"))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_trees(fa, d):
    _run(fa, [(1024, 1024 + 50), (300, 1300), (1000, 1000), (513, 900)], 4, 2, d, torch.bfloat16, 64, words=32)


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (100, 3), (128, 0), (129, 130), (500, 20), (ALL, 9), (50, 5000)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_window_and_sinks(fa, window, sinks, d):
    _run(fa, TREES + [(64, 2000), (3, 900), (200, 1300), (130, 130), (1, 2000)], 6, 2, d, torch.bfloat16, 32, window=window, sinks=sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows_that_end_among_the_nodes(fa, d):
    # longer than what is cached, shorter than where the last node lies: by its depth a node may see all of it
    for window in (30, 33, 34, 60, 69, 70):
        _run(fa, [(37, 70), (37, 70), (4, 36), (60, 61)], 4, 1, d, torch.float16, 32, window=window, sinks=1)
        _run(fa, [(4, 30), (3, 33), (4, 34)], 4, 1, d, torch.bfloat16, 16, words=1, window=min(window, 31), max_q=4)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [ALL, 300])
def test_few_nodes_under_a_window(fa, d, window):
    _run(fa, FEW + [(4, 3000)] * 3, 4, 1, d, torch.float16, 16, words=1, window=window, sinks=4, max_q=4)


@pytest.mark.parametrize("layout_", ["hnd", "nhd", "both"])
def test_cache_layouts(fa, layout_):
    _run(fa, TREES, 4, 2, 128, torch.float16, 16, window=300, sinks=4, layout=layout_)


@pytest.mark.parametrize("max_q", [0, 1, 3, 64, 1000])
def test_max_q_is_a_hint(fa, max_q):
    _run(fa, TREES, 8, 2, 128, torch.bfloat16, 64, max_q=max_q)


@pytest.mark.parametrize("scale", [0.0, -0.3, 0.6])
def test_scales(fa, scale):
    for d, lens in ((128, [(60, 400), (50, 200)]), (64, [(2, 300), (3, 3)]), (256, [(4, 129), (30, 300)])):
        _run(fa, lens, 4, 2, d, torch.bfloat16, 16, window=150, sinks=2, scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_long_context_is_cut(fa, d):
    _run(fa, [(26, 20000)], 4, 1, d, torch.bfloat16, 64, max_q=26)
    _run(fa, [(3, 9001), (64, 64), (1, 7000)], 4, 2, d, torch.bfloat16, 16)


def test_fewer_keys_than_nodes(fa):
    # the first nodes lie before the sequence: what they would hold is not there
    for d in (64, 128, 256):
        _run(fa, [(40, 25), (3, 0), (64, 1), (1, 1), (200, 150)], 4, 2, d, torch.bfloat16, 16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("words", [1, 3])
def test_any_mask(fa, d, words):
    # rows of random bits: some without their own, some without any (of which those
    # without cached keys see nothing), bits behind the node itself
    rng = random.Random(words)
    lens = [(32 * words, 32 * words), (20, 20), (30, 333), (5, 5), (32 * words, 140 + 32 * words), (7, 7)]
    x = Batch(lens, 4, 2, d, torch.bfloat16, 32, words)
    rows = [[frozenset(k for k in range(32 * words) if k < n + 40 and rng.random() < (0.4 if i % 3 else 0.0)) for i in range(n)] for n, _ in lens]
    mask = torch.cat([mask_of(r, words) for r in rows]).cuda()
    for max_q in (0, 32 * words):
        o, lse = x.run(fa, mask=mask, max_q=max_q)
        fa.check_device_error()
        x.check(o, lse, "any mask", rows=rows)
        assert bool((lse == -math.inf).any())
    few = Batch([(4, 4), (3, 3), (4, 133)], 4, 1, d, torch.bfloat16, 32, words)
    rows = [[frozenset({0}) if i == 2 else frozenset() for i in range(n)] for n, _ in few.lens]
    o, lse = few.run(fa, mask=torch.cat([mask_of(r, words) for r in rows]).cuda(), max_q=4)
    fa.check_device_error()
    few.check(o, lse, "any mask, few rows", rows=rows)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [3, 20, 60])
def test_a_line_of_nodes_sees_what_a_chunk_sees(fa, d, n):
    # fwd_paged on the same batch has the same reference, window included (no
    # window here ends among the nodes).  Not the same bits: the two cut the work at
    # other places and may take other forms, so the parts of a row are summed in
    # another order; each is held to the bound of its own arithmetic.
    x = Batch([(n, n), (n, 500), (n, 128 + n)], 2, 1, d, torch.bfloat16, 32, 2, trees=[list(range(-1, n - 1))] * 3)
    c = x.cache
    for window, sinks in ((ALL, 0), (70, 3)):
        for o, lse in (x.run(fa, window=window, sinks=sinks, max_q=n),
                       fa.fwd_paged(x.q, c.k, c.v, c.table, x.cu, x.sk, window=window, sinks=sinks, max_q=n)):
            fa.check_device_error()
            x.check(o, lse, f"a line of {n}", window, sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_chunks_ignore_their_mask_and_positions(fa, d):
    x = Batch([(40, 300), (500, 900), (2, 700), (33, 33)], 4, 2, d, torch.bfloat16, 32, 1)
    mask, pos = x.mask.clone(), x.positions.clone()
    mask[:40], pos[:40] = 0x55, -7
    mask[40:540], pos[40:540] = -1, 1 << 30
    mask[542:], pos[542:] = 0, 0
    o, lse = x.run(fa, mask=mask, positions=pos, window=100, sinks=2)
    fa.check_device_error()
    x.check(o, lse, "chunks", 100, 2)


def test_without_positions_nodes_sit_where_they_lie(fa):
    x = Batch([(20, 300), (5, 200)], 4, 2, 128, torch.bfloat16, 32, 1)
    pos = [list(range(nk - n, nk)) for n, nk in x.lens]
    o, lse = x.run(fa, positions=None, window=60, sinks=2)
    fa.check_device_error()
    x.check(o, lse, "no positions", 60, 2, pos=pos)
    assert torch.equal(x.run(fa)[0], x.run(fa, positions=None)[0])  # without a window they do not matter


def test_positions_out_of_range_are_cut_and_reported(fa):
    x = Batch([(20, 300), (5, 200)], 4, 2, 64, torch.bfloat16, 32, 1)
    p = x.positions.clone()
    p[3], p[7], p[22] = 279, 1 << 30, -5
    o, lse = x.run(fa, positions=p, window=60, sinks=2)
    assert _reported(fa)
    pos = [list(r) for r in x.pos]
    pos[0][3], pos[0][7], pos[1][2] = 280, 287, 195
    x.check(o, lse, "cut positions", 60, 2, pos=pos)


def test_pages_before_the_window_are_not_read(fa):
    x = Batch([(30, 1000), (3, 800)], 4, 2, 128, torch.float16, 32, 1)
    table = x.cache.table
    for b, (n, nk) in enumerate(x.lens):
        lo = nk - n - 200 + 1
        for j in range(1, lo // 32):  # (page 0 holds the sinks)
            page = int(table[b, j])
            x.cache.k[page] = x.cache.v[page] = math.nan
            table[b, j] = -9
    o, lse = x.run(fa, window=200, sinks=20)
    fa.check_device_error()
    x.check(o, lse, "freed pages", 200, 20)


def test_bad_pages_are_reported(fa):
    x = Batch([(10, 100), (10, 90)], 2, 1, 64, torch.bfloat16, 16, 1)
    x.cache.table[0, 2] = 1 << 20
    o, lse = x.run(fa)
    assert _reported(fa)
    k, v = x.seqs[0]
    k[:, 32:48], v[:, 32:48] = 0, 0  # (it reads as zeros)
    x.check(o, lse, "a bad page")


def test_rows_outside_the_sequences_are_left(fa):
    x = Batch([(5, 60), (9, 300)], 4, 2, 64, torch.bfloat16, 16, 1)
    c = x.cache
    q, mask, pos = (torch.cat([t[:3], t, t[:4]]) for t in (x.q, x.mask, x.positions))
    q[:3], q[17:] = math.nan, math.nan
    o = torch.full((21, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((21, 4), 5.0, device="cuda")
    fa.fwd_tree(q, c.k, c.v, c.table, x.cu + 3, x.sk, mask, pos, out=o, lse=lse)
    fa.check_device_error()
    x.check(o[3:17], lse[3:17], "inside")
    assert bool((o[:3] == 7).all()) and bool((o[17:] == 7).all()) and bool((lse[:3] == 5).all()) and bool((lse[17:] == 5).all())


def test_queries_out_of_a_projection_and_given_outputs(fa):
    x = Batch([(20, 60), (1, 300), (7, 7)], 4, 2, 128, torch.bfloat16, 16, 1)
    wide = torch.full((x.T, 9, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:6] = x.q
    c, ws = x.cache, torch.empty(fa.paged_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(x.q), torch.empty(x.T, 4, device="cuda")
    got = fa.fwd_tree(wide[:, 2:6], c.k, c.v, c.table, x.cu, x.sk, x.mask, x.positions, out=o, lse=lse, workspace=ws)
    fa.check_device_error()
    assert got[0] is o and got[1] is lse
    x.check(o, lse, "strided queries")
    for bad in (dict(out=o[:, :2]), dict(lse=lse[1:]), dict(mask=x.mask[1:]), dict(positions=x.positions[1:]), dict(positions=x.positions.long())):
        with pytest.raises(ValueError):
            x.run(fa, **bad)
    with pytest.raises(fa.FaError):
        x.run(fa, workspace=ws[:1000])


def test_nonfinite_values_of_masked_nodes(fa):
    # the scores of keys that a row does not see are replaced, NaN or not; LSE shows it alone
    x = Batch([(30, 200), (4, 50)], 4, 2, 128, torch.bfloat16, 32, 1, trees=[[-1] + [0] * 29, [-1, 0, 0, 0]])
    table = x.cache.table
    for b, at in ((0, 170 + 17), (1, 46 + 2)):
        x.cache.k[int(table[b, at // 32]), :, at % 32] = math.nan
    _, lse = x.run(fa)
    bad = torch.isnan(lse).any(1)
    assert bad.nonzero().flatten().tolist() == [17, 32]


@pytest.mark.parametrize("d", [64, 128, 256])
def test_random_batches(fa, d):
    for seed in range(8):
        rng = random.Random(100 * d + seed)
        B, Hkv, g = rng.randint(1, 12), rng.choice([1, 2, 3]), rng.choice([1, 2, 4, 7])
        most = rng.choice([4, 20, 64, 90])
        lens = []
        for _ in range(B):
            n = rng.randint(0, most)
            lens.append((n, n + rng.choice([0, rng.randint(0, 200), rng.randint(0, 1500)])))
        if sum(n for n, _ in lens) == 0:
            lens.append((1, 9))
        window, sinks = (ALL, 0) if rng.random() < 0.5 else (rng.randint(1, 700), rng.choice([0, 1, 4, 40, 200]))
        _run(fa, lens, Hkv * g, Hkv, d, rng.choice([torch.bfloat16, torch.float16]), rng.choice([16, 32, 128]), words=rng.choice([1, 2, 3]),
             window=window, sinks=sinks, max_q=rng.choice([0, most]), seed=seed + 1)


# -------------------------------------------------- graphs and streams --

def test_a_captured_graph_follows_masks_and_lengths(fa):
    x = Batch([(20, 300), (30, 500), (3, 40)], 4, 2, 128, torch.bfloat16, 32, 1)
    y = Batch([(3, 300), (20, 400), (30, 40)], 4, 2, 128, torch.bfloat16, 32, 1, seed=2)
    ws = torch.empty(fa.paged_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    c = x.cache
    mask, pos = torch.empty_like(x.mask), torch.empty_like(x.positions)
    parents = ints([p for t in x.parents for p in t])
    o, lse = torch.empty_like(x.q), torch.empty(x.T, 4, device="cuda")

    def step():
        fa.tree_plan(parents, x.cu, x.sk, 32, mask=mask, positions=pos)
        fa.fwd_tree(x.q, c.k, c.v, c.table, x.cu, x.sk, mask, pos, window=200, out=o, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    g.replay()
    fa.check_device_error()
    x.check(o, lse, "captured", 200)
    # other lengths and trees over the same pages
    x.lens, x.parents, x.rows = [(3, 250), (20, 400), (30, 39)], y.parents, y.rows
    x.pos = [[nk - n + q - (mk - n) for q in p] for (n, nk), (_, mk), p in zip(x.lens, y.lens, y.pos)]
    x.seqs = [(k[:, :nk], v[:, :nk]) for (k, v), (_, nk) in zip(x.seqs, x.lens)]
    parents.copy_(ints([p for t in y.parents for p in t]))
    x.cu.copy_(y.cu)
    x.sk.copy_(ints([nk for _, nk in x.lens]))
    g.replay()
    fa.check_device_error()
    x.check(o, lse, "replayed", 200)


def test_a_wait_that_runs_out_is_reported(fa):
    x = Batch([(20, 300)], 4, 2, 64, torch.bfloat16, 32, 1)
    assert fa.lib().fa_debug_inject(1) == fa.FA_OK
    x.run(fa)
    with pytest.raises(fa.FaError) as e:
        fa.check_device_error()
    assert e.value.status == fa.FA_ERR_TIMEOUT
    o, lse = x.run(fa)
    fa.check_device_error()
    x.check(o, lse, "after it")


# ------------------------------------------- windows among the nodes --

def _kept(rows, pos, n, window, sinks):
    """Of what a node sees of its own path, what its window and the sinks leave."""
    return [frozenset(k for k in row if k < n and (pos[k] > pos[i] - window or pos[k] < sinks)) for i, row in enumerate(rows)]


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (5, 0), (7, 40), (33, 1), (64, 70), (1000, 0), (ALL, 9), (1, 1 << 40)])
@pytest.mark.parametrize("words", [1, 3, 32])
def test_plan_under_a_window(fa, words, window, sinks):
    # trees, lines and chunks, behind no cached token, a few (within the sinks) and many
    rng = random.Random(words)
    lens, trees = [], []
    for ctx in (0, 1, 2, 30, 39, 70, 500):
        for n in (1, 7, 32 * words, 32 * words - 1, 32 * words + 1 + 5 * ctx):
            lens.append((n, ctx + n))
            trees.append(list(range(-1, n - 1)) if n > 32 * words or n % 2 else random_tree(n, rng))
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    args = ints([p for t in trees for p in t]), ints(cu), ints([nk for _, nk in lens]), 32 * words
    mask, pos = fa.tree_plan(*args, window=window, sinks=sinks)
    assert not _reported(fa)
    want = []
    for (n, nk), parents in zip(lens, trees):
        rows, depth = layout(parents, words)
        want.append(mask_of(rows if n > 32 * words else _kept(rows, [nk - n + x for x in depth], n, window, sinks), words))
    assert torch.equal(mask.cpu(), torch.cat(want))
    plain = fa.tree_plan(*args)
    assert torch.equal(pos, plain[1])
    if window == ALL:
        assert torch.equal(mask, plain[0])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [3, 20, 60])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (5, 0), (16, 4), (40, 25)])
def test_a_line_of_nodes_under_a_window_is_a_chunk(fa, d, n, window, sinks):
    # windows that end among the nodes: laid out under it, a line sees what the same tokens of a chunk see
    x = Batch([(n, n), (n, n + 2), (n, 128 + n), (n, 500)], 2, 1, d, torch.bfloat16, 32, 2, trees=[list(range(-1, n - 1))] * 4)
    mask, pos = fa.tree_plan(ints([p for t in x.parents for p in t]), x.cu, x.sk, 64, window=window, sinks=sinks)
    x.chunk = [True] * 4
    for max_q in (0, n):
        o, lse = x.run(fa, mask=mask, positions=pos, window=window, sinks=sinks, max_q=max_q)
        fa.check_device_error()
        x.check(o, lse, f"a line of {n}", window, sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(3, 0), (9, 2), (20, 50)])
def test_a_tree_under_a_window_sees_what_its_paths_see(fa, d, window, sinks):
    # each path of a tree decoded token by token: the cached tokens, then the nodes from the root on
    n, ctx = 40, 45
    parents = random_tree(n, random.Random(5), 4)
    x = Batch([(n, ctx + n)], 4, 2, d, torch.bfloat16, 32, 2, trees=[parents])
    mask, pos = fa.tree_plan(ints(parents), x.cu, x.sk, 64, window=window, sinks=sinks)
    o, lse = x.run(fa, mask=mask, positions=pos, window=window, sinks=sinks)
    fa.check_device_error()
    k, v = x.seqs[0]
    for i in range(n):
        path = [i]
        while parents[path[0]] >= 0:
            path.insert(0, parents[path[0]])
        at = list(range(ctx)) + [ctx + j for j in path]
        see = sees(1, len(at) - 1, None, None, window, sinks, chunk=True)
        ref = reference(x.q[i:i + 1], k[:, at], v[:, at], see, d ** -0.5)
        check_forward(o[i:i + 1].transpose(0, 1), lse[i:i + 1].transpose(0, 1), ref, x.q.dtype, d, len(at), f"node {i}")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_that_share_pages(fa, d):
    # beams: rows with the same full pages (neighbours or not), and the same batch with copies of them: the same bits
    page, full, n = 32, 9, [5, 1, 20, 7, 3, 60]
    group = [0, 0, 1, 1, 0, 1]
    lens = [(x, page * full + 3 + x) for x in n]
    x = Batch(lens, 4, 2, d, torch.bfloat16, page, 2)
    c = x.cache
    at = {0: 0, 1: 2}
    shared = c.table.clone()
    for b, g in enumerate(group):
        own, first = c.table[b, :full].long(), c.table[at[g], :full].long()
        c.k[own], c.v[own] = c.k[first], c.v[first]
        shared[b, :full] = shared[at[g], :full]
        x.seqs[b][0][:, :page * full], x.seqs[b][1][:, :page * full] = (t[:, :page * full] for t in x.seqs[at[g]])
    for window, sinks, max_q in ((ALL, 0, 0), (100, 40, 60), (ALL, 0, 3)):
        c.table, copies = shared, c.table
        o, lse = x.run(fa, window=window, sinks=sinks, max_q=max_q)
        c.table = copies
        p, mse = x.run(fa, window=window, sinks=sinks, max_q=max_q)
        fa.check_device_error()
        assert torch.equal(o, p) and torch.equal(lse, mse)
        x.check(o, lse, "shared pages", window, sinks)
