"""Token ranges (cu_q) that do not fit the packed arrays, which only the kernels
can see: they are cut to what exists, the same by fa_cache_append and
fa_fwd_paged, and reported."""
import math

import pytest
import torch

import attn_inputs as gen
from window_util import check_forward, ints, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _index_error(fa):
    with pytest.raises(fa.FaError) as e:
        fa.check_device_error()
    assert e.value.status == fa.FA_ERR_INDEX
    fa.check_device_error()


RANGES = [
    # cu_q, seq_k, the rows that belong to a sequence: (first, number, sequence)
    ([0, 3, 11], [20, 30], [(0, 3, 0), (3, 5, 1)]),      # more tokens than the arrays hold
    ([-4, 3, 8], [20, 30], [(0, 3, 0), (3, 5, 1)]),      # a range that begins before them
    ([0, 8, 12], [20, 30], [(0, 8, 0)]),                 # a whole range behind them
    ([2, 5, 1 << 30], [20, 30], [(2, 3, 0), (5, 3, 1)]),
    ([0, 8, 5], [20, 30], [(0, 8, 0)]),                  # a range that goes back
]


@pytest.mark.parametrize("cu,sk,rows", RANGES)
def test_append_and_attention_cut_ranges_alike(fa, cu, sk, rows):
    T, Hq, Hkv, d, page = 8, 4, 2, 64, 16
    q, k, v = (torch.from_numpy(gen.normal((T, h, d), 71, i)).bfloat16().cuda() for i, h in enumerate((Hq, Hkv, Hkv)))
    old = [torch.from_numpy(gen.normal((4, Hkv, page, d), 72, i)).bfloat16().cuda() for i in range(2)]
    kp, vp = (x.clone() for x in old)
    table = ints([[2, 0], [1, 3]])
    fa.check_device_error()
    fa.cache_append(k, v, kp, vp, table, ints(cu), ints(sk))
    _index_error(fa)
    want = [x.clone() for x in old]
    for first, n, b in rows:  # a sequence's tokens are its last ones
        for i in range(n):
            pos = sk[b] - n + i
            for w, x in zip(want, (k, v)):
                w[int(table[b, pos // page]), :, pos % page] = x[first + i]
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    o = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    fa.fwd_paged(q, kp, vp, table, ints(cu), ints(sk), out=o, lse=lse)
    _index_error(fa)
    left = torch.ones(T, dtype=torch.bool, device="cuda")
    for first, n, b in rows:
        r = slice(first, first + n)
        left[r] = False
        ks, vs = (x[table[b].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :sk[b]] for x in (kp, vp))
        ref = reference(q[r].transpose(0, 1), ks, vs, 1 << 30, 0, d ** -0.5)
        check_forward(o[r].transpose(0, 1), lse[r].transpose(0, 1), ref, q.dtype, d, sk[b], f"{cu} sequence {b}")
    assert bool((o[left] == 7.0).all()) and bool((lse[left] == 7.0).all())


def test_append_of_good_ranges_reports_nothing(fa):
    # rows before, between the last sequence and the arrays' end, empty sequences
    k, v = (torch.from_numpy(gen.normal((300, 1, 64), 73, i)).bfloat16().cuda() for i in range(2))
    kp, vp = (torch.zeros((400, 1, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = 290
    cu = [3] * 40 + [3 + i for i in range(1, n + 1)] + [3 + n] * 300  # 629 sequences, one token or none
    B = len(cu) - 1
    table = torch.arange(B, dtype=torch.int32, device="cuda").remainder(400)[:, None].contiguous()
    fa.cache_append(k, v, kp, vp, table, ints(cu), ints([1] * B))
    fa.check_device_error()
    at = table[39:39 + n, 0].long()
    assert torch.equal(kp[at, 0, 0], k[3:3 + n, 0]) and torch.equal(vp[at, 0, 0], v[3:3 + n, 0])
    assert int((kp != 0).any(-1).sum()) == n


@pytest.mark.parametrize("B,T,Hkv,page,pages", [(64, 8192, 1, 16, 64), (20000, 65536, 8, 1024, 64)])
def test_more_work_than_ranges_without_overlap_can_have_is_not_run(fa, B, T, Hkv, page, pages):
    # every other sequence claims all tokens; the second batch's key tiles, 1.05e10, do not fit 32 bits
    d = 64
    q = torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device="cuda")
    kp = torch.zeros((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
    sk = torch.full((B,), page * pages, dtype=torch.int32, device="cuda")
    cu = ints([0, T] * (B // 2) + [0])
    o = torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hkv), 7.0, device="cuda")
    fa.check_device_error()
    fa.fwd_paged(q, kp, kp, table, cu, sk, out=o, lse=lse)
    _index_error(fa)
    assert bool((o == 7.0).all()) and bool((lse == 7.0).all())
    # the same arrays with ranges that fit: every row sees its window's 100 keys, of score 0
    cu = ints([i * T // B for i in range(B + 1)])
    fa.fwd_paged(q, kp, kp, table, cu, sk, window=100, out=o, lse=lse)
    fa.check_device_error()
    # (ln 100 in fp32, by a hardware logarithm within 2^-21 of it, as in window_util)
    assert bool((o == 0.0).all()) and float((lse.double() - math.log(100)).abs().max()) <= 2.0 ** -20 + 2.0 ** -21 * math.log(100)
