"""Paged attention of ragged batches (fa_fwd_paged) and the cache append
(fa_cache_append) against 64-bit references, within bounds derived from the
arithmetic.  Everything a cache holds beside the sequences' own rows is NaN
unless a test says otherwise: nothing of it may reach a result."""
import math

import pytest
import torch

import attn_inputs as gen
from window_util import HALF_STEP, Paged, check_forward, ints, reference

pytestmark = pytest.mark.gpu
ALL = 1 << 30


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _normal(shape, seed, stream, dtype):
    return torch.from_numpy(gen.normal(shape, seed, stream)).to(dtype).cuda()


def _batch(lens, Hq, Hkv, d, dtype, page, seed=1, layout="hnd", junk=float("nan"), **kw):
    """lens: [(new tokens, keys)].  Returns q [T, Hq, d], the cache, cu_q, seq_k, seqs."""
    seqs = [tuple(_normal((Hkv, nk, d), seed, 10 * b + i, dtype) for i in (1, 2)) for b, (_, nk) in enumerate(lens)]
    cache = Paged(seqs, page, layout, junk=junk, seed=seed, **kw)
    cu = [0]
    for nq, _ in lens:
        cu.append(cu[-1] + nq)
    q = _normal((max(cu[-1], 1), Hq, d), seed, 0, dtype)[:cu[-1]]
    return q, cache, ints(cu), ints([nk for _, nk in lens]), seqs


def _check(o, lse, q, lens, seqs, window, sinks, scale, what):
    at, d = 0, q.shape[2]
    for b, ((nq, nk), (k, v)) in enumerate(zip(lens, seqs)):
        if nq:
            r = slice(at, at + nq)
            ref = reference(q[r].transpose(0, 1), k, v, window, sinks, scale)
            check_forward(o[r].transpose(0, 1), lse[r].transpose(0, 1), ref, q.dtype, d, nk, f"{what} sequence {b} ({nq}, {nk})")
        at += nq


def _run(fa, lens, Hq, Hkv, d, dtype, page, window=ALL, sinks=0, scale=None, max_q=0, **kw):
    q, c, cu, sk, seqs = _batch(lens, Hq, Hkv, d, dtype, page, **kw)
    o, lse = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, window=window, sinks=sinks, scale=scale, max_q=max_q)
    fa.check_device_error()
    _check(o, lse, q, lens, seqs, window, sinks, d ** -0.5 if scale is None else scale,
           f"Hq{Hq} Hkv{Hkv} d{d} page{page} w{window} s{sinks} max_q{max_q}")


DECODE = [(1, n) for n in (1, 2, 15, 16, 17, 127, 128, 129, 1000, 2500, 64, 333)]
CHUNKS = [(5, 5), (1, 700), (300, 900), (0, 50), (77, 77), (130, 1300), (2, 129), (64, 64)]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode(fa, d, page):
    _run(fa, DECODE, 8, 2, d, torch.bfloat16, page, max_q=1)


@pytest.mark.parametrize("page", [16, 64, 512])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_chunks(fa, d, page):
    _run(fa, CHUNKS, 4, 2, d, torch.bfloat16, page)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (10, 2), (7, 1), (12, 2), (48, 3), (128, 1), (100, 1)])
@pytest.mark.parametrize("d", [64, 256])
def test_head_groups(fa, Hq, Hkv, d):
    _run(fa, [(1, 300), (9, 200), (40, 40)], Hq, Hkv, d, torch.float16, 32)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (100, 3), (128, 0), (129, 130), (500, 20), (ALL, 9), (50, 5000)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_window_and_sinks(fa, window, sinks, d):
    _run(fa, CHUNKS + [(1, 2000)], 6, 2, d, torch.bfloat16, 32, window=window, sinks=sinks)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "both"])
@pytest.mark.parametrize("d", [64, 128])
def test_cache_layouts(fa, layout, d):
    _run(fa, CHUNKS, 4, 2, d, torch.float16, 16, window=300, sinks=4, layout=layout)
    _run(fa, [(3, 40)], 2, 1, d, torch.float16, 64, layout=layout, spare=0)  # one page, one head


@pytest.mark.parametrize("max_q", [0, 1, 3, 64, 1000])
def test_max_q_is_a_hint(fa, max_q):
    _run(fa, CHUNKS, 8, 2, 128, torch.bfloat16, 64, max_q=max_q)


@pytest.mark.parametrize("scale", [0.0, -0.3, 0.6])
def test_scales(fa, scale):
    _run(fa, [(1, 400), (50, 200)], 4, 2, 128, torch.bfloat16, 16, window=150, sinks=2, scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_long_sequence_is_cut(fa, d):
    _run(fa, [(1, 20000)], 4, 1, d, torch.bfloat16, 64, max_q=1)
    _run(fa, [(3, 9001), (1, 5), (1, 7000)], 4, 2, d, torch.bfloat16, 16)


def test_many_sequences(fa):
    # more sequences than threads share the start of the line
    lens = [((b * 7) % 4, (b * 37) % 200 + 3) for b in range(900)]
    _run(fa, lens, 2, 1, 64, torch.bfloat16, 16, junk=0.0)


def test_queries_without_keys(fa):
    # fewer keys than new tokens: the first ones sit before the sequence
    _run(fa, [(40, 25), (3, 0), (200, 1), (1, 1)], 4, 2, 128, torch.bfloat16, 16)
    _run(fa, [(400, 130), (5, 0)], 4, 2, 256, torch.float16, 32, window=20, sinks=1)


def test_strided_queries(fa):
    lens = [(20, 60), (1, 300)]
    q, c, cu, sk, seqs = _batch(lens, 4, 2, 128, torch.bfloat16, 16)
    wide = torch.full((21, 9, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:6] = q
    o, lse = fa.fwd_paged(wide[:, 2:6], c.k, c.v, c.table, cu, sk)
    fa.check_device_error()
    _check(o, lse, q, lens, seqs, ALL, 0, 128 ** -0.5, "strided q")


def test_rows_outside_the_sequences_are_left(fa):
    lens = [(5, 60), (1, 300)]
    q, c, cu, sk, seqs = _batch(lens, 4, 2, 64, torch.bfloat16, 16)
    cu = cu + 3  # three rows before the first sequence, seven behind the last
    qq = torch.full((16, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    qq[3:9] = q
    o = torch.full((16, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((16, 4), 5.0, device="cuda")
    fa.fwd_paged(qq, c.k, c.v, c.table, cu, sk, out=o, lse=lse)
    fa.check_device_error()
    _check(o[3:9], lse[3:9], q, lens, seqs, ALL, 0, 64 ** -0.5, "inner rows")
    for x, fill in ((o, 7.0), (lse, 5.0)):
        assert bool((x[:3] == fill).all()) and bool((x[9:] == fill).all())


def test_pages_behind_the_window_may_be_gone(fa):
    lens, window, sinks = [(4, 2000), (130, 1500)], 200, 3
    for d in (64, 256):
        q, c, cu, sk, seqs = _batch(lens, 4, 2, d, torch.bfloat16, 16)
        for b, (nq, nk) in enumerate(lens):
            first = nk - nq - window + 1  # the first key a query sees beside the sinks
            for i in range(1, first // 16):
                c.k[int(c.table[b, i])] = float("nan")
                c.v[int(c.table[b, i])] = float("nan")
            c.table[b, 1:first // 16] = -1
        o, lse = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, window=window, sinks=sinks)
        fa.check_device_error()
        _check(o, lse, q, lens, seqs, window, sinks, d ** -0.5, f"freed pages d={d}")


def test_shared_pages(fa):
    # two sequences with the same prefix pages, and the same sequence twice
    q, c, cu, sk, seqs = _batch([(2, 200), (2, 200)], 4, 2, 128, torch.bfloat16, 16)
    c.table[1] = c.table[0]
    o, lse = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk)
    fa.check_device_error()
    _check(o, lse, q, [(2, 200), (2, 200)], [seqs[0], seqs[0]], ALL, 0, 128 ** -0.5, "shared")


def test_offsets_beyond_32_bits(fa):
    # pages past 2^32 bytes of the cache
    Hkv, page, d = 2, 64, 128
    n = (1 << 32) // (Hkv * page * d * 2) + 50
    k, v = (torch.empty((n, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    seq = tuple(_normal((Hkv, 1000, d), 3, i, torch.bfloat16) for i in (1, 2))
    ids = list(range(n - 16, n))
    for x, pages in zip(seq, (k, v)):
        for i, p in enumerate(ids):
            part = x[:, i * page:(i + 1) * page]
            pages[p].fill_(float("nan"))
            pages[p, :, :part.shape[1]] = part
    q = _normal((9, 4, d), 3, 0, torch.bfloat16)
    o, lse = fa.fwd_paged(q, k, v, ints([ids]), ints([0, 9]), ints([1000]))
    fa.check_device_error()
    _check(o, lse, q, [(9, 1000)], [seq], ALL, 0, d ** -0.5, "far pages")


def test_bad_indices_are_reported_and_contained(fa):
    lens = [(3, 200), (2, 100)]
    q, c, cu, sk, seqs = _batch(lens, 4, 2, 128, torch.bfloat16, 16, junk=0.0)
    good, _ = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk)
    fa.check_device_error()
    n = c.k.shape[0]
    for bad in (-1, n, 1 << 30, -(1 << 31)):
        t = c.table.clone()
        t[0, 5] = bad
        o, _ = fa.fwd_paged(q, c.k, c.v, t, cu, sk)
        with pytest.raises(fa.FaError) as e:
            fa.check_device_error()
        assert e.value.status == fa.FA_ERR_INDEX
        assert torch.equal(o[3:], good[3:])  # the other sequence is right
        fa.check_device_error()  # reported once
    # lengths beyond the table, negative lengths, token ranges beyond T or going back
    for cu2, sk2 in (([0, 3, 5], [200, 1 << 30]), ([0, 3, 5], [-5, 100]), ([0, 3, 900], [200, 100]),
                     ([0, 4, 2], [200, 100]), ([-2, 3, 5], [200, 100])):
        guard = torch.full((8, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        fa.fwd_paged(q, c.k, c.v, c.table, ints(cu2), ints(sk2), out=guard[:5])
        with pytest.raises(fa.FaError) as e:
            fa.check_device_error()
        assert e.value.status == fa.FA_ERR_INDEX
        assert bool((guard[5:] == 3.0).all())


def test_same_result_every_time_and_in_a_graph(fa):
    lens = [(1, 3000), (1, 17), (200, 700), (1, 5000)]
    q, c, cu, sk, seqs = _batch(lens, 8, 2, 128, torch.bfloat16, 32)
    ws = torch.empty((fa.paged_workspace_bytes(128),), dtype=torch.uint8, device="cuda")
    want = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, workspace=ws)
    for _ in range(3):
        got = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, out=o, lse=lse, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    # the lengths are device data: a replay follows them
    sk2 = [2990, 17, 650, 4000]
    sk.copy_(ints(sk2))
    g.replay()
    fa.check_device_error()
    shorter = [(k[:, :n], v[:, :n]) for (k, v), n in zip(seqs, sk2)]
    _check(o, lse, q, [(nq, n) for (nq, _), n in zip(lens, sk2)], shorter, ALL, 0, 128 ** -0.5, "replayed")


def test_two_calls_at_once(fa):
    lens = [(1, 3000), (60, 700), (1, 900)]
    q, c, cu, sk, seqs = _batch(lens, 8, 2, 128, torch.bfloat16, 32)
    want = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty((fa.paged_workspace_bytes(128),), dtype=torch.uint8, device="cuda") for _ in range(2)]
    got = []
    for _ in range(4):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                got.append(fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, workspace=w))
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_paged_refusals(fa):
    q, c, cu, sk, _ = _batch([(2, 40), (1, 20)], 4, 2, 128, torch.bfloat16, 16, junk=0.0)
    ok = lambda **kw: fa.fwd_paged(**{**dict(q=q, k_pages=c.k, v_pages=c.v, block_table=c.table, cu_q=cu, seq_k=sk), **kw})  # noqa: E731
    ok()
    for kw in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[:, :, :64]), dict(k_pages=c.k.half()), dict(cu_q=cu.long()),
               dict(cu_q=cu[:2]), dict(seq_k=sk.cpu()), dict(block_table=c.table[:1]), dict(q=q.transpose(0, 1)),
               dict(out=torch.empty((2, 4, 128), dtype=torch.bfloat16, device="cuda")),
               dict(lse=torch.empty((3, 4), dtype=torch.float64, device="cuda")),
               dict(workspace=torch.empty((1 << 28,), dtype=torch.uint8)),
               dict(workspace=torch.empty((1,), dtype=torch.uint8, device="cuda").expand(1 << 28))):
        with pytest.raises(ValueError):
            ok(**kw)
    for kw in (dict(window=0), dict(sinks=-1), dict(scale=math.nan), dict(max_q=-1),
               dict(workspace=torch.empty((1000,), dtype=torch.uint8, device="cuda")),
               dict(k_pages=c.k[:, :, :12], v_pages=c.v[:, :, :12]), dict(k_pages=c.k[..., :96], v_pages=c.v[..., :96], q=q[..., :96].contiguous())):
        with pytest.raises(fa.FaError):
            ok(**kw)
    assert ok(q=q[:0]).__class__ is tuple
    fa.check_device_error()


# ---------------------------------------------------------------- append --

def _turned(x, pos, d, half):
    """Rotation in 64 bits by the fp32 angle tables the call gets."""
    cos, sin = _tables(int(pos.max()) + 1 if pos.numel() else 1, d)
    c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
    x = x.double()
    a, b = (x[..., :d // 2], x[..., d // 2:]) if half else (x[..., 0::2], x[..., 1::2])
    y, z = a * c - b * s, a * s + b * c
    size = torch.maximum((a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs())
    if half:
        return torch.cat([y, z], -1), torch.cat([size, size], -1)
    return torch.stack([y, z], -1).flatten(-2), torch.stack([size, size], -1).flatten(-2)


def _tables(n, d):
    cos, sin = gen.rope_tables(n, d)
    return torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()


def _close(got, want, size, dtype, what):
    # two products and a sum in fp32 (2^-24 each of |a c| + |b s|), one rounding
    tol = HALF_STEP[dtype] * want.abs() + 2.0 ** -22 * size + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), f"{what}: off by {float((off - tol).max()):.3e} more than the bound"


@pytest.mark.parametrize("half", [False, True, None], ids=["interleaved", "half", "no rope"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["hnd", "both"])
def test_append(fa, d, dtype, half, layout):
    Hq, Hkv, page = 6, 2, 16
    lens = [(3, 40), (1, 1), (0, 9), (50, 129), (17, 17), (1, 300)]
    seqs = [tuple(_normal((Hkv, nk, d), 5, 10 * b + i, dtype) for i in (1, 2)) for b, (_, nk) in enumerate(lens)]
    c = Paged(seqs, page, layout, junk=9.0)
    before = c.k.clone(), c.v.clone()
    T = sum(nq for nq, _ in lens)
    qkv = _normal((T + 2, Hq + 2 * Hkv, d), 6, 0, dtype)   # two rows behind the last sequence
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    cu = [0]
    for nq, _ in lens:
        cu.append(cu[-1] + nq)
    rope = None if half is None else (*_tables(300, d), fa.FA_ROPE_HALF if half else fa.FA_ROPE_INTERLEAVED)
    q_out = torch.full((T + 2, Hq, d), 4.0, dtype=dtype, device="cuda")
    r = fa.cache_append(k, v, c.k, c.v, c.table, ints(cu), ints([nk for _, nk in lens]), q=q, rope=rope, q_out=q_out)
    fa.check_device_error()
    assert r is q_out and bool((q_out[T:] == 4.0).all())
    wk, wv = before
    for b, (nq, nk) in enumerate(lens):
        pos = torch.arange(nk - nq, nk, device="cuda")
        rows = slice(cu[b], cu[b] + nq)
        page_of, at = c.table[b].long()[pos // page], pos % page
        new_k = c.k[page_of, :, at]
        if half is None:
            assert torch.equal(new_k, k[rows]) and torch.equal(q_out[rows], q[rows])
        else:
            for got, x, what in ((new_k, k[rows], "k"), (q_out[rows], q[rows], "q")):
                want, size = _turned(x, pos, d, half)
                _close(got, want, size, dtype, f"{what} of sequence {b}")
        wk[page_of, :, at] = new_k
        wv[page_of, :, at] = v[rows]
    assert torch.equal(c.k, wk) and torch.equal(c.v, wv), "rows of other tokens changed"


def test_append_without_queries_and_in_place(fa):
    d, Hkv = 128, 2
    seqs = [tuple(_normal((Hkv, 30, d), 5, i, torch.bfloat16) for i in (1, 2))]
    c = Paged(seqs, 16, junk=0.0)
    k, v = _normal((4, Hkv, d), 6, 1, torch.bfloat16), _normal((4, Hkv, d), 6, 2, torch.bfloat16)
    rope = (*_tables(64, d), fa.FA_ROPE_HALF)
    assert fa.cache_append(k, v, c.k, c.v, c.table, ints([0, 4]), ints([30]), rope=rope) is None
    q = _normal((4, 8, d), 6, 0, torch.bfloat16)
    want = fa.cache_append(k, v, c.k, c.v, c.table, ints([0, 4]), ints([30]), q=q, rope=rope)
    got = fa.cache_append(k, v, c.k, c.v, c.table, ints([0, 4]), ints([30]), q=q, rope=rope, q_out=q)
    assert got is q and torch.equal(got, want)
    fa.check_device_error()


def test_append_bad_indices(fa):
    d, Hkv = 64, 1
    seqs = [tuple(_normal((Hkv, 30, d), 5, i + 3 * b, torch.bfloat16) for i in (1, 2)) for b in range(2)]
    c = Paged(seqs, 16, junk=0.0)
    k, v = _normal((4, Hkv, d), 6, 1, torch.bfloat16), _normal((4, Hkv, d), 6, 2, torch.bfloat16)
    rope = (*_tables(40, d), fa.FA_ROPE_HALF)
    keep = c.k.clone(), c.v.clone()
    cu = ints([0, 2, 4])

    def dropped(table, cu, sk, rope=rope):
        fa.cache_append(k, v, c.k, c.v, table, cu, ints(sk), rope=rope)
        with pytest.raises(fa.FaError) as e:
            fa.check_device_error()
        assert e.value.status == fa.FA_ERR_INDEX

    bad = c.table.clone()
    bad[:, 1] = c.k.shape[0]
    dropped(bad, cu, [30, 30])                    # page number out of range
    dropped(c.table, cu, [0, 1 << 30])            # positions before the sequence, and behind the table
    dropped(c.table, cu, [-40, 33])               # position 31 of the second sequence is a row of its page 1, 32 is behind it
    dropped(c.table, cu, [30, 30], (rope[0][:20], rope[1][:20], rope[2]))  # behind the angle tables
    page, row = int(c.table[1, 1]), 15
    assert torch.equal(c.v[page, :, row], v[2])
    want, size = _turned(k[2:3], ints([31]).long(), d, True)
    _close(c.k[page, :, row], want[0], size[0], torch.bfloat16, "the token at position 31")
    keep[0][page, :, row], keep[1][page, :, row] = c.k[page, :, row], c.v[page, :, row]
    assert torch.equal(c.k, keep[0]) and torch.equal(c.v, keep[1])


def test_append_then_attend_in_chunks_matches_dense(fa):
    """The operators as they are used: a sequence comes in chunks and then
    token by token, each step appended and attended to over the pages; the
    results are those of windowed attention over the whole sequence."""
    Hq, Hkv, d, page, window, sinks = 8, 2, 128, 16, 150, 4
    steps = [200, 1, 90, 1, 1, 130, 1]
    N = sum(steps)
    x = [_normal((2, N, h, d), 8, i, torch.bfloat16) for i, h in enumerate((Hq, Hkv, Hkv))]
    pages = -(-N // page)
    kp, vp = (torch.full((2 * pages, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.randperm(2 * pages, generator=torch.Generator().manual_seed(1)).view(2, pages).to(torch.int32).cuda()
    rope = (*_tables(N, d), fa.FA_ROPE_INTERLEAVED)
    outs, lses, rot = [], [], []
    at = 0
    for n in steps:
        q, k, v = (t[:, at:at + n].reshape(2 * n, -1, d) for t in x)
        at += n
        cu, sk = ints([0, n, 2 * n]), ints([at, at])
        qr = fa.cache_append(k, v, kp, vp, table, cu, sk, q=q, rope=rope)
        o, lse = fa.fwd_paged(qr, kp, vp, table, cu, sk, window=window, sinks=sinks, max_q=n)
        outs.append(o.view(2, n, Hq, d))
        lses.append(lse.view(2, n, Hq))
        rot.append(qr.view(2, n, Hq, d))
    fa.check_device_error()
    o, lse, q = torch.cat(outs, 1), torch.cat(lses, 1), torch.cat(rot, 1)
    keys = [kp[table[b].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :N] for b in range(2)]
    vals = [vp[table[b].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :N] for b in range(2)]
    qd = q.transpose(1, 2).contiguous()
    od, ld = fa.fwd_window(qd, torch.stack(keys), torch.stack(vals), window, sinks)
    fa.check_device_error()
    for b in range(2):
        ref = reference(qd[b], keys[b], vals[b], window, sinks, d ** -0.5)
        check_forward(o[b].transpose(0, 1), lse[b].transpose(0, 1), ref, torch.bfloat16, d, N, f"paged, sequence {b}")
        check_forward(od[b], ld[b], ref, torch.bfloat16, d, N, f"dense, sequence {b}")


@pytest.mark.parametrize("sinks", [1, 32, 33])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_few_sinks_far_from_the_window(fa, sinks, d):
    _run(fa, [(1, 1900), (70, 900), (3, 2500)], 4, 2, d, torch.bfloat16, 16, window=150, sinks=sinks)


@pytest.mark.parametrize("d", [64, 256])
def test_paged_wait_that_runs_out_is_reported(fa, d):
    lens = [(200, 900), (1, 3000)]
    q, c, cu, sk, seqs = _batch(lens, 4, 2, d, torch.bfloat16, 16)
    want = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk)
    fa.check_device_error()
    assert fa.lib().fa_debug_inject(1) == fa.FA_OK
    fa.fwd_paged(q, c.k, c.v, c.table, cu, sk)
    with pytest.raises(fa.FaError) as e:
        fa.check_device_error()
    assert e.value.status == fa.FA_ERR_TIMEOUT
    got = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk)
    fa.check_device_error()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
