"""The operators on a cache's pages (fa_pages_resize, fa_pages_fork,
fa_cache_copy, fa_cache_compact) against a plain model on the host.  Everything
here is whole numbers and copies: results have to be equal, the bytes that are
not to be written included."""
import random
import threading

import pytest
import torch

from window_util import ints

pytestmark = pytest.mark.gpu


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


def _pages(layers, n, heads, page, d, layout="hnd", dtype=torch.bfloat16):
    """Keys and values of distinct random bits; layers None: a cache of one layer, 4-D."""
    L = 1 if layers is None else layers

    def bits(*shape):
        return torch.randint(-32768, 32767, shape, dtype=torch.int16, device="cuda").view(dtype)

    if layout == "hnd":
        k, v = (bits(L, n, heads, page, d) for _ in range(2))
    elif layout == "nhd":
        k, v = (bits(L, n, page, heads, d).transpose(2, 3) for _ in range(2))
    elif layout == "pages first":  # the layers of a page together
        k, v = (bits(n, L, heads, page, d).transpose(0, 1) for _ in range(2))
    else:  # keys and values interleaved, padding behind each token
        both = bits(L, n, page, 2, heads, d + 8)
        k, v = (both[:, :, :, i, :, :d].transpose(2, 3) for i in range(2))
    return (k[0], v[0]) if layers is None else (k, v)


def _raw(x):
    return x.contiguous().view(torch.int16)


LAYOUTS = ["hnd", "nhd", "pages first", "both"]


# ------------------------------------------------------------------ copy --

@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("layers,heads,page,d", [(None, 1, 16, 64), (1, 3, 32, 128), (3, 2, 64, 256), (2, 8, 256, 64), (5, 5, 16, 128)])
def test_copy(fa, layers, heads, page, d, layout):
    n = 23
    k, v = _pages(layers, n, heads, page, d, layout)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(1))
    src, dst = order[:9], order[9:18]
    want = [x.clone() for x in (k, v)]
    for x in want:
        x = x if layers is not None else x[None]
        x[:, dst.cuda()] = x[:, src.cuda()]
    fa.cache_copy(k, v, src.to(torch.int32).cuda(), dst.to(torch.int32).cuda())
    assert not _reported(fa)
    for x, w in zip((k, v), want):
        assert torch.equal(_raw(x), _raw(w))


def test_copy_edges(fa):
    k, v = _pages(2, 5, 2, 16, 64)
    before = k.clone()
    fa.cache_copy(k, v, ints([]), ints([]))
    fa.cache_copy(k, v, ints([3]), ints([3]))
    assert not _reported(fa)
    assert torch.equal(_raw(k), _raw(before))
    # pairs outside the cache are passed over, the others done
    fa.cache_copy(k, v, ints([0, 5, -1, 1]), ints([2, 1, 0, 1 << 30]))
    assert _reported(fa)
    before[:, 2] = before[:, 0]
    assert torch.equal(_raw(k), _raw(before))
    # a page given twice as a source
    fa.cache_copy(k, v, ints([0, 0]), ints([3, 4]))
    assert not _reported(fa)
    before[:, [3, 4]] = before[:, [0, 0]]
    assert torch.equal(_raw(k), _raw(before))


# --------------------------------------------------------------- compact --

def _tables(rng, rows, width, n):
    """Rows of distinct scattered pages (-1 behind them), and a spare page."""
    order = list(range(n))
    rng.shuffle(order)
    table = torch.full((rows, width), -1, dtype=torch.int32)
    for r in range(rows):
        for j in range(width):
            table[r, j] = order.pop()
    return table


def _compact_model(x, table, first, keep, keep_n, page):
    """As if everything were read before anything is written."""
    x = x if x.dim() == 5 else x[None]
    y = x.clone()
    for b in range(table.shape[0]):
        for i in range(keep_n[b]):
            a, z = keep[b][i], first[b] + i
            y[:, table[b, z // page], :, z % page] = x[:, table[b, a // page], :, a % page]
    return y


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("layers,heads,page,d,K", [(None, 1, 16, 64, 1), (2, 3, 16, 128, 7), (1, 8, 64, 256, 30), (3, 5, 32, 64, 200),
                                                   (1, 1, 128, 128, 333)])
def test_compact(fa, layers, heads, page, d, K, layout):
    rng = random.Random(K)
    B = 3
    width = -(-(2 * K + 50) // page)
    n = B * width + 2
    k, v = _pages(layers, n, heads, page, d, layout)
    table = _tables(rng, B, width, n)
    first, keep, keep_n = [], [], []
    for b in range(B):
        f = rng.randint(0, 40)
        m = (K, rng.randint(0, K), max(0, K - 1))[b]
        keep.append(sorted(rng.sample(range(f, 2 * K + 45), m)) + [-5] * (K - m))
        first.append(f)
        keep_n.append(m)
    want = [_compact_model(x, table, first, keep, keep_n, page) for x in (k, v)]
    got = fa.cache_compact(k, v, table.cuda(), ints(first), ints(keep), ints(keep_n))
    assert not _reported(fa)
    assert got.tolist() == [f + m for f, m in zip(first, keep_n)]
    for x, w in zip((k, v), want):
        assert torch.equal(_raw(x), _raw(w if layers is not None else w[0]))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_compact_long(fa, d):
    # many rounds, neighbouring moves (each slot is read by one row and written by a later one), one sequence
    page, N, K = 64, 6000, 5000
    k, v = _pages(1, N // page + 1, 2, page, d)
    table = torch.randperm(N // page + 1, generator=torch.Generator().manual_seed(2)).to(torch.int32)[None]
    for keep in (list(range(1, K + 1)), list(range(7, 7 + K)), sorted(random.Random(3).sample(range(N), K)), list(range(K))):
        want = [_rows_model(x, table[0], keep, page) for x in (k, v)]
        fa.cache_compact(k, v, table.cuda(), ints([0]), ints([keep]), ints([K]))
        assert not _reported(fa)
        for x, w in zip((k, v), want):
            assert torch.equal(_raw(x), _raw(w))


def _rows_model(x, pages, keep, page):
    a, z = torch.tensor(keep), torch.arange(len(keep))
    y = x.clone()
    y[:, pages[z // page].long().cuda(), :, (z % page).cuda()] = x[:, pages[a // page].long().cuda(), :, (a % page).cuda()]
    return y


def test_compact_any_list_behind_its_place(fa):
    # repeated and descending positions, each at or behind the place it goes to
    page, d = 16, 64
    k, v = _pages(2, 8, 2, page, d)
    table = torch.tensor([[3, 1, 4, 7, 5, 2, 6, 0]], dtype=torch.int32)
    keep = [9, 9, 40, 30, 20, 10, 50, 49, 8, 127]
    want = [_compact_model(x, table, [0], [keep], [len(keep)], page) for x in (k, v)]
    fa.cache_compact(k, v, table.cuda(), ints([0]), ints([keep]), ints([len(keep)]))
    assert not _reported(fa)
    for x, w in zip((k, v), want):
        assert torch.equal(_raw(x), _raw(w))


def test_compact_passes_over_what_leads_out_of_range(fa):
    page, d = 16, 64
    k, v = _pages(1, 4, 1, page, d)
    table = torch.tensor([[0, 99], [2, 3], [1, -1]], dtype=torch.int32)
    before = k.clone()
    # sequence 0: position 16 has a bad page, 32 is behind the table, 1 lies before its place, -4 before the sequence; only 9 -> 4 is done
    keep = [[16, 32, 1, -4, 9], [5, 6, 7, 0, 0], [3, 0, 0, 0, 0]]
    got = fa.cache_compact(k, v, table.cuda(), ints([0, 30, -2]), ints(keep), ints([5, 9, 1]))
    assert _reported(fa)
    assert got.tolist() == [5, 32, 0]  # the second is cut to 5 kept ones, and to the table's 32 tokens
    before[:, 0, :, 4] = before[:, 0, :, 9]
    assert torch.equal(_raw(k), _raw(before))


def test_compact_nothing(fa):
    k, v = _pages(None, 4, 1, 16, 64)
    before = k.clone()
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    assert fa.cache_compact(k, v, table, ints([3, 9]), torch.empty(2, 0, dtype=torch.int32, device="cuda"), ints([0, 0])).tolist() == [3, 9]
    assert fa.cache_compact(k, v, table[:0], ints([]), torch.empty(0, 3, dtype=torch.int32, device="cuda"), ints([])).shape == (0,)
    assert not _reported(fa)
    assert torch.equal(_raw(k), _raw(before))


# ------------------------------------------------------- resize and fork --

class Pool:
    """The plain model: a list of reference counts, of rows, and of lengths."""

    def __init__(self, num_pages, rows, max_pages, page):
        self.refs, self.page, self.max = [0] * num_pages, page, max_pages
        self.table, self.seq = [[-1] * max_pages for _ in range(rows)], [0] * rows
        self.low = 0  # no page below is free

    def count(self, n):
        return -(-n // self.page)

    def free(self):
        while self.low < len(self.refs) and self.refs[self.low] > 0:
            self.low += 1
        return self.low if self.low < len(self.refs) else None

    def resize(self, want):
        for r, w in enumerate(want):
            for j in range(self.count(w), self.count(self.seq[r])):
                self.refs[self.table[r][j]] -= 1
                self.low = min(self.low, self.table[r][j])
                self.table[r][j] = -1
        for r, w in enumerate(want):
            room = min(self.count(w), self.count(self.seq[r]))
            for j in range(self.count(self.seq[r]), self.count(w)):
                p = self.free()
                self.table[r][j] = -1 if p is None else p
                if p is not None:
                    self.refs[p] = 1
                    room = j + 1
            self.seq[r] = min(w, room * self.page)

    def fork(self, src, dst, k, v):
        """The forks that are right; copies in k and v [layers, pages, heads, page, d]."""
        fresh = []
        for a, b in zip(src, dst):
            full, rest = divmod(self.seq[a], self.page)
            p = -1
            if rest:
                p = self.free()
                if p is None:
                    fresh.append(-3)
                    continue
                self.refs[p] = 1
            fresh.append(p)
        for a, b, p in zip(src, dst, fresh):
            if p == -3:
                continue
            full, rest = divmod(self.seq[a], self.page)
            for j in range(full):
                self.table[b][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
            if rest:
                self.table[b][full] = p
                for x in (k, v):
                    x[:, p, :, :rest] = x[:, self.table[a][full], :, :rest]
            self.seq[b] = self.seq[a]
        return fresh

    def check(self, refs, table, seq):
        assert seq.tolist() == self.seq
        assert refs.tolist() == self.refs
        assert table.tolist() == self.table


@pytest.mark.parametrize("num_pages,rows,max_pages,page", [(40, 9, 12, 16), (7, 3, 5, 64), (300, 33, 40, 16), (1, 1, 1, 16), (17001, 5, 6000, 16),
                                                           (40000, 70, 1200, 32), (1003, 1500, 3, 16), (2000, 12288, 1, 16)])
def test_resize_follows_the_model(fa, num_pages, rows, max_pages, page):
    # (the last four: several rounds over the counts, long rows, more rows than threads, and as many as 48 KB hold ranks of)
    rng = random.Random(num_pages)
    pool = Pool(num_pages, rows, max_pages, page)
    refs, table, seq = ints(pool.refs), ints(pool.table), ints(pool.seq)
    for step in range(4 if num_pages > 1000 else 12):
        most = max(1, min(max_pages * page, 3 * num_pages * page // rows))
        want = [rng.choice([0, s, rng.randint(0, most), min(max_pages * page, s + rng.randint(0, 40))]) for s in pool.seq]
        if num_pages > 1000 and step < 2:
            want = [rng.randint(0, most) if step == 0 else max(0, s - rng.randint(0, 500)) for s in pool.seq]
        fa.pages_resize(refs, table, seq, ints(want), page)
        pool.resize(want)
        assert not _reported(fa)
        pool.check(refs, table, seq)
    fa.pages_resize(refs, table, seq, torch.zeros_like(seq), page)
    assert int(refs.abs().sum()) == 0 and int((table != -1).sum()) == 0


def test_resize_reports_bad_data(fa):
    refs, table = ints([1, 0, 0, 2]), ints([[3, 0], [1, 77], [3, -1]])
    seq = ints([32, 32, 5])
    # row 0 gives both back; row 1's page 1 was held by nobody and 77 is none; row 2 asks for more than its row holds
    fa.pages_resize(refs, table, seq, ints([0, -3, 1000]), 16)
    assert _reported(fa)
    assert seq.tolist() == [0, 0, 32]
    assert table.tolist() == [[-1, -1], [-1, -1], [3, 0]]
    assert refs.tolist() == [1, 0, 0, 1]


def test_resize_with_a_wide_table(fa):
    # rows further apart than they are wide, and entries behind the used ones untouched
    wide = torch.full((3, 10), 55, dtype=torch.int32, device="cuda")
    refs, seq = ints([0, 1, 0, 0, 0]), ints([0, 0, 0])
    fa.pages_resize(refs, wide[:, 2:6], seq, ints([20, 0, 16]), 16)
    assert not _reported(fa)
    assert wide[:, 2:6].tolist() == [[0, 2, 55, 55], [55] * 4, [3, 55, 55, 55]]
    assert bool((wide[:, :2] == 55).all()) and bool((wide[:, 6:] == 55).all())
    assert refs.tolist() == [1, 1, 1, 1, 0] and seq.tolist() == [20, 0, 16]


@pytest.mark.parametrize("layers,heads,page,d,layout", [(None, 2, 16, 64, "hnd"), (3, 1, 16, 128, "nhd"), (2, 3, 64, 64, "both"),
                                                        (2, 2, 32, 256, "pages first")])
def test_forks_and_resizes_follow_the_model(fa, layers, heads, page, d, layout):
    rng = random.Random(page + d)
    rows, max_pages, num_pages = 8, 6, 14  # (so few that forks and resizes run out of them)
    k, v = _pages(layers, num_pages, heads, page, d, layout)
    mk, mv = ((x if layers is not None else x[None]).clone() for x in (k, v))
    pool = Pool(num_pages, rows, max_pages, page)
    refs, table, seq = ints(pool.refs), ints(pool.table), ints(pool.seq)
    short = 0
    for step in range(14):
        want = [rng.choice([0, s, s, rng.randint(0, max_pages * page)]) for s in pool.seq]
        if step == 5:
            want = [s // page * page for s in pool.seq]  # all pages full: forks need none
        fa.pages_resize(refs, table, seq, ints(want), page)
        pool.resize(want)
        pool.check(refs, table, seq)
        empty, full = [r for r in range(rows) if pool.seq[r] == 0], [r for r in range(rows) if pool.seq[r] > 0]
        if not full:
            continue
        dst = rng.sample(empty, rng.randint(0, len(empty)))
        src = [rng.choice(full) for _ in dst]
        fresh = fa.pages_fork(k, v, refs, table, seq, ints(src), ints(dst))
        assert not _reported(fa)
        assert fresh.tolist() == pool.fork(src, dst, mk, mv)
        short += -3 in fresh.tolist()
        pool.check(refs, table, seq)
        for x, m in ((k, mk), (v, mv)):
            assert torch.equal(_raw(x if layers is not None else x[None]), _raw(m))
    assert short > 0, "no step ran out of pages"


def test_fork_refuses_rows_in_use_and_given_twice(fa):
    page, n = 16, 20
    k, v = _pages(1, n, 1, page, 64)
    pool = Pool(n, 8, 3, page)
    refs, table, seq = ints(pool.refs), ints(pool.table), ints(pool.seq)
    want = [20, 33, 16, 0, 0, 0, 0, 0]
    fa.pages_resize(refs, table, seq, ints(want), page)
    pool.resize(want)
    mk, mv = k.clone(), v.clone()
    #       right, given twice (both), in use, a source, no row, no row, right
    src = [0, 1, 1, 0, 3, -1, 0, 2]
    dst = [4, 5, 5, 1, 3, 6, 8, 7]
    fresh = fa.pages_fork(k, v, refs, table, seq, ints(src), ints(dst))
    assert _reported(fa)
    # (row 3 is empty, but given as its own source)
    assert fresh.tolist() == [6, -2, -2, -2, -2, -2, -2, -1]
    assert pool.fork([0, 2], [4, 7], mk, mv) == [6, -1]
    pool.check(refs, table, seq)
    assert torch.equal(_raw(k), _raw(mk)) and torch.equal(_raw(v), _raw(mv))


def test_fork_with_a_bad_source(fa):
    page = 16
    k, v = _pages(1, 6, 1, page, 64)
    before = k.clone()
    refs, seq = ints([1, 1, 1, 0, 0, 0]), ints([40, 20, 20, 0, 0, 0])
    table = ints([[0, -1], [1, 9], [9, 2], [-1, -1], [-1, -1], [-1, -1]])
    # a length that the row cannot hold; a last page that is none; a full page that is none (its entry becomes -1)
    fresh = fa.pages_fork(k, v, refs, table, seq, ints([0, 1, 2]), ints([3, 4, 5]))
    assert _reported(fa)
    assert fresh.tolist() == [-2, -2, 3]
    assert seq.tolist() == [40, 20, 20, 0, 0, 20] and refs.tolist() == [1, 1, 1, 1, 0, 0]
    assert table[3:].tolist() == [[-1, -1], [-1, -1], [-1, 3]]
    before[:, 3, :, :4] = before[:, 2, :, :4]
    assert torch.equal(_raw(k), _raw(before))


def test_many_forks_of_one(fa):
    page, n, rows = 16, 5000, 2100
    k, v = _pages(1, n, 1, page, 64)
    mk, mv = k.clone(), v.clone()
    pool = Pool(n, rows, 4, page)
    refs, table, seq = ints(pool.refs), ints(pool.table), ints(pool.seq)
    want = [60] + [0] * (rows - 1)
    fa.pages_resize(refs, table, seq, ints(want), page)
    pool.resize(want)
    src, dst = [0] * (rows - 1), list(range(rows - 1, 0, -1))
    fresh = fa.pages_fork(k, v, refs, table, seq, ints(src), ints(dst))
    assert not _reported(fa)
    # (the model looks for each page from the start: the order is theirs)
    assert fresh.tolist() == list(range(4, 4 + rows - 1))
    for b, p in zip(dst, fresh.tolist()):
        mk[:, p, :, :12], mv[:, p, :, :12] = mk[:, 3, :, :12], mv[:, 3, :, :12]
    assert refs[:4].tolist() == [rows, rows, rows, 1] and bool((refs[4:4 + rows - 1] == 1).all())
    assert torch.equal(_raw(k), _raw(mk)) and torch.equal(_raw(v), _raw(mv))
    assert bool((seq == 60).all())


def test_the_most_rows_and_forks(fa):
    # as many rows of a resize as it takes, and as many rows and forks of a fork
    rows, pages = 49152, 50000
    refs, table, seq = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((pages,), (rows, 1), (rows,)))
    table -= 1
    want = torch.full_like(seq, 16)
    fa.pages_resize(refs, table, seq, want, 16)
    assert not _reported(fa)
    number = torch.arange(rows, dtype=torch.int32, device="cuda")
    assert torch.equal(table[:, 0], number) and torch.equal(seq, want) and int(refs.sum()) == rows
    want[1::2] = 0
    fa.pages_resize(refs, table, seq, want, 16)
    assert torch.equal(table[:, 0], torch.where(number % 2 == 1, torch.full_like(number, -1), number)) and torch.equal(seq, want)
    assert int(refs.sum()) == rows // 2 and int(refs[1:rows:2].sum()) == 0
    with pytest.raises(fa.FaError):
        fa.pages_resize(refs, torch.zeros(rows + 1, 1, dtype=torch.int32, device="cuda"), *(torch.zeros(rows + 1, dtype=torch.int32, device="cuda"),) * 2, 16)
    rows, n, pages = 1 << 18, 16384, 20000
    k, v = _pages(1, pages, 1, 16, 64)
    refs, table, seq = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((pages,), (rows, 2), (rows,)))
    table[5], refs[[7, 9]], seq[5] = ints([7, 9]), 1, 21
    src, dst = ints([5]).repeat(n), torch.arange(rows - n, rows, dtype=torch.int32, device="cuda")
    fresh = fa.pages_fork(k, v, refs, table, seq, src, dst)
    assert not _reported(fa)
    free = torch.tensor([p for p in range(n + 2) if p not in (7, 9)], dtype=torch.int32, device="cuda")
    assert torch.equal(fresh, free) and bool((seq[rows - n:] == 21).all()) and int(refs[7]) == n + 1
    assert torch.equal(table[rows - n:, 1], free) and bool((table[rows - n:, 0] == 7).all())
    assert torch.equal(_raw(k[0, free.long(), :, :5]), _raw(k[0, 9:10, :, :5]).expand(n, -1, -1, -1))
    with pytest.raises(fa.FaError):
        fa.pages_fork(k, v, refs, table, seq, ints([5]).repeat(n + 1), ints([6]).repeat(n + 1))


# -------------------------------------------------------------- together --

def test_a_captured_graph_follows_the_arrays(fa):
    page, n = 16, 30
    k, v = _pages(2, n, 2, page, 64)
    mk, mv = k.clone(), v.clone()
    pool = Pool(n, 4, 5, page)
    refs, table, seq = ints(pool.refs), ints(pool.table), ints(pool.seq)
    want, src, dst = ints([30, 50, 0, 0]), ints([0, 1]), ints([2, 3])

    def step():
        fa.pages_resize(refs, table, seq, want, page)
        fa.pages_fork(k, v, refs, table, seq, src, dst)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for w, a, b in (([30, 50, 0, 0], [0, 1], [2, 3]), ([0, 70, 11, 0], [1, 2], [0, 3]), ([5, 0, 0, 64], [3, 3], [1, 2])):
        want.copy_(ints(w))
        src.copy_(ints(a))
        dst.copy_(ints(b))
        g.replay()
        pool.resize(w)
        pool.fork(a, b, mk, mv)
        assert not _reported(fa)
        pool.check(refs, table, seq)
        assert torch.equal(_raw(k), _raw(mk)) and torch.equal(_raw(v), _raw(mv))


def _at_once(*loops):
    """Runs the loops at once, each in a thread and on a stream of its own; what one raised is raised here."""
    failed = []

    def go(loop):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                loop()
                torch.cuda.current_stream().synchronize()
        except BaseException as e:  # noqa: B902 (raised again below)
            failed.append(e)

    torch.cuda.synchronize()  # what the loops use has been made
    threads = [threading.Thread(target=go, args=(loop,)) for loop in loops]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failed:
        raise failed[0]


def test_pools_of_several_threads(fa):
    # Calls of one kernel that take different amounts of shared memory, above what a launch may have unasked: what one
    # thread asks for must not be lost to another's call in between.  (Threads of a pool of their own each.)
    def pool(rows, steps):
        refs, table, seq = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((rows + 5,), (rows, 1), (rows,)))
        some, none = torch.full_like(seq, 16), torch.zeros_like(seq)

        def loop():
            for _ in range(steps):
                fa.pages_resize(refs, table, seq, some, 16)
                fa.pages_resize(refs, table, seq, none, 16)
            fa.pages_resize(refs, table, seq, some, 16)

        return loop, refs, table, seq

    pools = [pool(49152, 200), pool(12288, 600), pool(20000, 400)]
    _at_once(*(p[0] for p in pools))
    assert not _reported(fa)
    for _, refs, table, seq in pools:
        rows = len(seq)
        assert torch.equal(table[:, 0], torch.arange(rows, dtype=torch.int32, device="cuda")) and bool((seq == 16).all())
        assert bool((refs[:rows] == 1).all()) and bool((refs[rows:] == 0).all())


def test_forks_of_several_threads(fa):
    def forks(rows, n, steps):
        k, v = _pages(1, n + 3, 1, 16, 64)
        refs, table, seq = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((n + 3,), (rows, 2), (rows,)))
        table[5], refs[[0, 1]], seq[5] = ints([0, 1]), 1, 21
        src, dst = ints([5]).repeat(n), torch.arange(rows - n, rows, dtype=torch.int32, device="cuda")
        back = seq.clone()
        fresh = []

        def loop():
            for i in range(steps):
                if i:
                    fa.pages_resize(refs, table[rows - n:], seq[rows - n:], back[rows - n:], 16)
                fresh.append(fa.pages_fork(k, v, refs, table, seq, src, dst))

        return loop, fresh, n

    both = [forks(1 << 18, 16384, 60), forks(20000, 12000, 80)]
    _at_once(*(f[0] for f in both))
    assert not _reported(fa)
    for _, fresh, n in both:
        for got in (fresh[0], fresh[-1]):
            assert torch.equal(got, torch.arange(2, n + 2, dtype=torch.int32, device="cuda"))
