"""Trees, rotary positions and pages where offsets pass 32 bits, and calls that
run at the same time on two streams."""
import pytest
import torch

import attn_inputs as gen
from rope_util import HALF, check_turned
from tree_util import layout, mask_of, reference, sees
from window_util import check_forward, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _normal(shape, seed, dtype):
    return torch.from_numpy(gen.normal(shape, seed, 1)).to(dtype).cuda()


def test_pages_behind_two_to_the_31(fa):
    """Two layers of 40000 pages, 2.6 thousand million elements: an element of
    the second layer's last pages lies behind 2^31."""
    L, n, H, ps, d = 2, 40000, 8, 64, 64
    k, v = (torch.empty((L, n, H, ps, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k[1, -20:].storage_offset() > 1 << 31
    top = list(range(n - 12, n))
    fill = [_normal((L, 12, H, ps, d), 1 + i, torch.bfloat16) for i in range(2)]
    for x, f in ((k, fill[0]), (v, fill[1])):
        x[:, n - 12:] = f
    # copy
    fa.cache_copy(k, v, ints([n - 1, n - 2]), ints([n - 5, n - 6]))
    fa.check_device_error()
    for x, f in ((k, fill[0]), (v, fill[1])):
        f[:, 7], f[:, 6] = f[:, 11], f[:, 10]
        assert torch.equal(x[:, n - 12:], f)
    # compact: 100 of 192 tokens of pages n - 12, n - 9, n - 7
    pages, keep = [0, 3, 5], list(range(30, 60)) + list(range(100, 170))
    new = fa.cache_compact(k, v, ints([[top[p] for p in pages]]), ints([10]), ints([keep]), ints([100]))
    fa.check_device_error()
    assert new.tolist() == [110]
    at = lambda s: (torch.tensor([pages[x // ps] for x in s], device="cuda"), torch.tensor([x % ps for x in s], device="cuda"))  # noqa: E731
    (sp, sr), (dp, dr) = at(keep), at(list(range(10, 110)))
    for x, f in ((k, fill[0]), (v, fill[1])):
        f[:, dp, :, dr] = f[:, sp, :, sr]
        assert torch.equal(x[:, n - 12:], f)
    # fork: the only free pages are the last ones
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    refs[n - 3:] = 0
    table, seq = torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), ints([110, 0])
    table[0, :2] = ints([top[0], top[3]])
    fresh = fa.pages_fork(k, v, refs, table, seq, ints([0]), ints([1]))
    fa.check_device_error()
    assert fresh.tolist() == [n - 3] and table[1, :2].tolist() == [top[0], n - 3] and int(refs[top[0]]) == 2
    for x, f in ((k, fill[0]), (v, fill[1])):
        f[:, 9, :, :46] = f[:, 3, :, :46]
        assert torch.equal(x[:, n - 12:], f)
    # append and attention of the second row, in the second layer
    parents = [-1, 0, 0, 1, 2, 2, 5]
    cu, sk = ints([0, 0, 7]), ints([110, 117])
    mask, pos = fa.tree_plan(ints(parents), cu, sk, 7)
    q, knew, vnew = (_normal((7, h, d), 5 + h, torch.bfloat16) for h in (16, H, H))
    rope = (*fa.rope_table(200, 32), HALF)
    q = fa.cache_append(knew, vnew, k[1], v[1], table, cu, sk, q=q, rope=rope, positions=pos)
    o, lse = fa.fwd_tree(q, k[1], v[1], table, cu, sk, mask, pos)
    fa.check_device_error()
    rows, depth = layout(parents, 1)
    assert torch.equal(mask.cpu(), mask_of(rows, 1)) and pos.tolist() == [110 + x for x in depth]
    turned, _ = fa.rope(knew, None, rope, positions=pos)
    seqs = [torch.cat([f[1, [0, 9]].transpose(0, 1).reshape(H, -1, d)[:, :110], new_.transpose(0, 1)], 1)
            for f, new_ in ((fill[0], turned), (fill[1], vnew))]
    ref = reference(q, *seqs, sees(7, 110, rows, pos.tolist(), 1 << 30, 0), d ** -0.5)
    check_forward(o.transpose(0, 1), lse.t(), ref, torch.bfloat16, d, 117, "pages behind 2^31")


def test_rows_behind_two_to_the_31(fa):
    H, N, d = 40, 430000, 128
    x = torch.zeros((1, H, N, d), dtype=torch.bfloat16, device="cuda")
    some = _normal((3, 50, d), 9, torch.bfloat16)
    picks = ((0, 0), (20, 200000), (H - 1, N - 50))
    for (h, a), s in zip(picks, some):
        x[0, h, a:a + 50] = s
    cos, sin = fa.rope_table(N, 64)
    assert x[0, H - 1, N - 50].storage_offset() > 1 << 31
    y, _ = fa.rope(x, None, (cos, sin, HALF))
    fa.check_device_error()
    for (h, a), s in zip(picks, some):
        check_turned(y[0, h, a:a + 50], s, cos[a:a + 50], sin[a:a + 50], HALF, f"head {h} row {a}")


def test_two_streams_at_once(fa):
    """Calls with workspaces of their own may run side by side: the same bits as one after the other."""
    d, page, B = 128, 32, 6
    jobs = []
    for seed in (1, 2):
        lens = [(20, 1500 + 100 * b + seed) for b in range(B)]
        need = [-(-nk // page) for _, nk in lens]
        pages = torch.from_numpy(gen.normal((2, sum(need), 2, page, d), seed, 3)).to(torch.bfloat16).cuda()
        table = torch.zeros(B, max(need), dtype=torch.int32)
        at = 0
        for b, x in enumerate(need):
            table[b, :x] = torch.arange(at, at + x)
            at += x
        parents = ints([i // 2 - 1 if i % 2 else max(-1, i // 2 - 1) for _ in range(B) for i in range(20)])
        q = _normal((20 * B, 8, d), seed, torch.bfloat16)
        jobs.append((q, pages[0], pages[1], table.cuda(), ints([20 * b for b in range(B + 1)]), ints([nk for _, nk in lens]), parents))

    def run(q, k, v, table, cu, sk, parents):
        mask, pos = fa.tree_plan(parents, cu, sk, 20)
        return fa.fwd_tree(q, k, v, table, cu, sk, mask, pos, window=700, sinks=2)

    alone = [run(*j) for j in jobs]
    fa.check_device_error()
    streams, got = [torch.cuda.Stream() for _ in jobs], [[] for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (s, j) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(s):
                got[i].append(run(*j))
    torch.cuda.synchronize()
    fa.check_device_error()
    for want, many in zip(alone, got):
        for o, lse in many:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
