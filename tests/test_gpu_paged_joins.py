"""Paged attention whose sequences are cut over many SMs: few or many rows per
unit, few or many parts, few or many units, and d = 64 batches on both sides
of the size at which the kernel takes one query tile per block or two."""
import pytest
import torch

import attn_inputs as gen
from window_util import Paged, check_forward, ints, reference

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


def _make(lens, Hq, Hkv, d, dtype, page, seed=3):
    seqs = [tuple(_normal((Hkv, nk, d), seed, 10 * b + i, dtype) for i in (1, 2)) for b, (_, nk) in enumerate(lens)]
    cu = [0]
    for nq, _ in lens:
        cu.append(cu[-1] + nq)
    q = _normal((cu[-1], Hq, d), seed, 0, dtype)
    return q, Paged(seqs, page, junk=float("nan"), seed=seed), ints(cu), ints([nk for _, nk in lens]), seqs


def _check(o, lse, q, lens, seqs, window, sinks, what):
    at, d = 0, q.shape[2]
    for b, ((nq, nk), (k, v)) in enumerate(zip(lens, seqs)):
        r = slice(at, at + nq)
        ref = reference(q[r].transpose(0, 1), k, v, window, sinks, d ** -0.5)
        check_forward(o[r].transpose(0, 1), lse[r].transpose(0, 1), ref, q.dtype, d, nk, f"{what} sequence {b} ({nq}, {nk})")
        at += nq


def _run(fa, lens, Hq, Hkv, d, dtype=torch.bfloat16, page=32, window=ALL, sinks=0, max_q=0):
    q, c, cu, sk, seqs = _make(lens, Hq, Hkv, d, dtype, page)
    o, lse = fa.fwd_paged(q, c.k, c.v, c.table, cu, sk, window=window, sinks=sinks, max_q=max_q)
    fa.check_device_error()
    _check(o, lse, q, lens, seqs, window, sinks, f"Hq{Hq} Hkv{Hkv} d{d} w{window} s{sinks} max_q{max_q}")


@pytest.mark.parametrize("nq", [1, 2, 7, 9, 31, 64, 100])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_sequence_rows_by_parts(fa, d, nq):
    # one head group: a unit of g * nq rows (or some units) in as many parts as there are key tiles
    for g, nk in ((1, 6000), (8, 9001), (3, 500)):
        _run(fa, [(nq, nk)], g, 1, d)
        _run(fa, [(nq, nk)], 2 * g, 2, d, max_q=nq, window=nk // 2, sinks=200)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_widest_group_over_a_long_sequence(fa, d):
    _run(fa, [(1, 20000)], 128, 1, d, max_q=1)
    _run(fa, [(2, 7001), (1, 30)], 128, 1, d, dtype=torch.float16)


@pytest.mark.parametrize("seqs", [2, 18, 19, 20, 38, 39])
@pytest.mark.parametrize("d", [64, 128])
def test_units_around_the_number_of_blocks(fa, d, seqs):
    # 8 heads: 19 sequences are 152 units, 38 are 304
    _run(fa, [(1 + b % 3, 100 + (b * 391) % 1500) for b in range(seqs)], 16, 8, d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_cut_units_with_rows_that_see_nothing(fa, d):
    _run(fa, [(120, 90), (7, 4000)], 2, 1, d)                        # the first rows sit before the sequence
    _run(fa, [(250, 200)], 1, 1, d, dtype=torch.float16, window=60)  # parts that some rows do not take part in
    _run(fa, [(60, 5000)], 4, 1, d, window=10)
    _run(fa, [(60, 5000)], 4, 1, d, window=130, sinks=3000)


@pytest.mark.parametrize("off", [-1, 0, 1])
def test_d64_around_the_choice_of_query_tiles(fa, off):
    # 4 heads share a key head; the sizes are rows per sequence on average: 32 rows are 8 tokens, 128 are 32
    for lens, max_q in (([(8, 900), (8, 40), (8 + off, 700), (8, 3000)], 0),
                        ([(8, 900), (8, 40), (8 + off, 700), (8, 3000)], 9),
                        ([(32, 900), (32, 40), (32 + off, 700), (32, 3000)], 33),
                        ([(61 + off, 2000), (1, 300), (1, 5), (1, 4000)], 64 + off),    # the longest at 4 times the average
                        ([(125 + off, 2000), (1, 300), (1, 5), (1, 4000)], 125 + off)):
        _run(fa, lens, 8, 2, 64, max_q=max_q)
        _run(fa, lens, 8, 2, 64, max_q=max_q, window=300, sinks=5, dtype=torch.float16)


@pytest.mark.parametrize("seqs,nq", [(75, 32), (76, 32), (76, 33), (77, 20)])
def test_d64_many_sequences_of_several_tokens(fa, seqs, nq):
    _run(fa, [(nq - b % 2, 33 + (b * 61) % 400) for b in range(seqs)], 16, 4, 64, max_q=nq)


def test_d64_forms_share_a_workspace(fa):
    """Calls of both forms on one workspace, in turn and replayed from a graph, give the bits of calls alone."""
    few = _make([(1, 3000), (1, 700), (2, 1500)], 8, 2, 64, torch.bfloat16, 16)
    many = _make([(200, 1000), (3, 2500)], 8, 2, 64, torch.bfloat16, 16)
    ws = torch.empty(fa.paged_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    call = lambda s: fa.fwd_paged(s[0], s[1].k, s[1].v, s[1].table, s[2], s[3], workspace=ws)  # noqa: E731
    want = []
    for s, lens in ((few, [(1, 3000), (1, 700), (2, 1500)]), (many, [(200, 1000), (3, 2500)])):
        ws.fill_(255)  # NaN
        o, lse = call(s)
        _check(o, lse, s[0], lens, s[4], ALL, 0, "alone")
        want.append((o, lse))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            got = [call(s) for s in (few, many, few, many, many, few)]
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    fa.check_device_error()
    for i, (o, lse) in zip((0, 1, 0, 1, 1, 0), got):
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
