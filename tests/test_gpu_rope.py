"""Rotary positions (fa_rope, fa_rope_table, fa_cache_append_at) against 64-bit
references, within bounds derived from the arithmetic."""
import math

import pytest
import torch

import attn_inputs as gen
from rope_util import HALF, INTERLEAVED, check_turned, frequencies, turn
from window_util import Paged, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_forward_09_gb300 as fa
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa.lib()
    return fa


def _normal(shape, seed, dtype):
    return torch.from_numpy(gen.normal(shape, seed, 1)).to(dtype).cuda()


def _angles(n, r, seed=0):
    t = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)
    return t.cos().float().cuda(), t.sin().float().cuda()


# ---------------------------------------------------------------- dense --

@pytest.mark.parametrize("layout", [INTERLEAVED, HALF])
@pytest.mark.parametrize("d,r", [(64, 16), (64, 48), (64, 64), (128, 32), (128, 112), (128, 128), (256, 64), (256, 256)])
@pytest.mark.parametrize("B,Hq,Hkv,N", [(1, 1, 1, 1), (2, 6, 2, 77), (1, 5, 5, 129), (3, 9, 1, 16)])
def test_dense(fa, B, Hq, Hkv, N, d, r, layout):
    dtype = torch.bfloat16 if (Hq + r // 16) % 2 else torch.float16
    q, k = _normal((B, Hq, N, d), 1, dtype), _normal((B, Hkv, N, d), 2, dtype)
    cos, sin = _angles(N + 40, r)
    for inverse in (False, True):
        yq, yk = fa.rope(q, k, (cos, sin, layout), offset=33, inverse=inverse)
        fa.check_device_error()
        for x, y in ((q, yq), (k, yk)):
            check_turned(y, x, cos[33:33 + N], sin[33:33 + N], layout, f"dense {B, Hq, Hkv, N, d, r, layout, inverse}", inverse)


@pytest.mark.parametrize("layout", [INTERLEAVED, HALF])
@pytest.mark.parametrize("T,Hq,Hkv,d,r", [(1, 8, 1, 64, 32), (67, 32, 8, 128, 64), (500, 3, 1, 256, 256), (33, 40, 40, 64, 64)])
def test_packed_tokens_of_a_projection(fa, T, Hq, Hkv, d, r, layout):
    wide = _normal((T, Hq + 2 * Hkv, d), 3, torch.bfloat16)
    q, k, _ = wide.split([Hq, Hkv, Hkv], dim=1)
    cos, sin = _angles(1000, r)
    pos = torch.randint(0, 1000, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
    yq, yk = fa.rope(q, k, (cos, sin, layout), positions=pos)
    fa.check_device_error()
    at = pos.long()
    for x, y in ((q, yq), (k, yk)):
        assert y.is_contiguous()
        check_turned(y, x, cos[at][:, None], sin[at][:, None], layout, f"packed {T, Hq, Hkv, d, r}")


@pytest.mark.parametrize("shared", [True, False])
def test_positions_of_each_entry(fa, shared):
    B, H, N, d, r = 3, 4, 50, 128, 64
    q = _normal((B, H, N, d), 4, torch.float16)
    cos, sin = _angles(300, r)
    pos = torch.randint(0, 300, (N,) if shared else (B, N), generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    y, none = fa.rope(q, None, (cos, sin, HALF), positions=pos)
    fa.check_device_error()
    assert none is None
    at = pos.long().expand(B, N)
    check_turned(y, q, cos[at][:, None], sin[at][:, None], HALF, "positions of each entry")


@pytest.mark.parametrize("layout", [INTERLEAVED, HALF])
def test_in_place_and_strides(fa, layout):
    B, H, N, d, r = 2, 3, 40, 128, 96
    cos, sin = _angles(N, r)
    base = _normal((B, N, H, d + 8), 6, torch.bfloat16)
    x = base[..., :d].transpose(1, 2)          # [B, H, N, d] with the tokens' heads together and padding between rows
    want, _ = fa.rope(x, None, (cos, sin, layout))
    before = base.clone()
    got, _ = fa.rope(x, None, (cos, sin, layout), q_out=x)
    fa.check_device_error()
    assert got is x and torch.equal(x, want)
    check_turned(want, before[..., :d].transpose(1, 2), cos, sin, layout, "strided")
    assert torch.equal(base[..., d:], before[..., d:]), "padding was written"
    # an expanded input (stride 0) gives the rows of its copy
    one = _normal((1, 1, N, d), 7, torch.bfloat16)
    assert torch.equal(fa.rope(one.expand(B, H, N, d), None, (cos, sin, layout))[0],
                       fa.rope(one.expand(B, H, N, d).contiguous(), None, (cos, sin, layout))[0])


def test_long_sequences_and_many_heads(fa):
    for B, H, N, d in ((1, 2, 40001, 64), (1, 300, 9, 256), (5, 1, 5000, 128)):
        q = _normal((B, H, N, d), 8, torch.bfloat16)
        cos, sin = _angles(N, d)
        y, _ = fa.rope(q, None, (cos, sin, HALF))
        fa.check_device_error()
        check_turned(y, q, cos, sin, HALF, f"{B, H, N, d}")


def test_nothing_to_do(fa):
    cos, sin = _angles(4, 64)
    for shape in ((0, 2, 3, 64), (2, 0, 3, 64), (2, 2, 0, 64), (0, 2, 64), (3, 0, 64)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        y, z = fa.rope(x, x, (cos, sin, HALF))
        assert y.shape == x.shape and z.shape == x.shape
    some = _normal((3, 2, 64), 1, torch.bfloat16)
    y, z = fa.rope(some, some[:, :0], (cos, sin, HALF))
    check_turned(y, some, cos[:3, None], sin[:3, None], HALF, "one of two arrays empty")


def test_nonfinite_values_stay_in_their_pair(fa):
    q = _normal((1, 1, 4, 64), 9, torch.bfloat16)
    q[0, 0, 1, 3], q[0, 0, 2, 5] = math.nan, math.inf
    cos, sin = _angles(4, 32)
    y, _ = fa.rope(q, None, (cos, sin, HALF))
    bad = ~torch.isfinite(y)
    assert bad[0, 0, 1].nonzero().flatten().tolist() == [3, 19] and bad[0, 0, 2].nonzero().flatten().tolist() == [5, 21]
    assert not bad[0, 0, [0, 3]].any()


def test_positions_outside_the_tables_are_left_and_reported(fa):
    q = _normal((5, 2, 64), 10, torch.float16)
    cos, sin = _angles(20, 64)
    out = torch.full_like(q, 7.0)
    fa.rope(q, None, (cos, sin, HALF), positions=ints([3, -1, 20, 19, 1 << 30]), q_out=out)
    with pytest.raises(fa.FaError) as e:
        fa.check_device_error()
    assert e.value.status == fa.FA_ERR_INDEX
    fa.check_device_error()
    assert bool((out[[1, 2, 4]] == 7.0).all())
    at = torch.tensor([3, 19], device="cuda")
    check_turned(out[[0, 3]], q[[0, 3]], cos[at][:, None], sin[at][:, None], HALF, "rows inside")


# ------------------------------------------------------------- gradient --

@pytest.mark.parametrize("layout", [INTERLEAVED, HALF])
@pytest.mark.parametrize("amplitude", [1.0, 1.3])
def test_gradient(fa, layout, amplitude):
    """The inverse is the gradient of sum(dy * rope(x)): of the formula (autograd
    in 64 bits) and of differences (the map is linear, so a difference quotient of
    any width is exact but for rounding)."""
    B, H, N, d, r = 2, 2, 9, 64, 48
    x, dy = _normal((B, H, N, d), 11, torch.bfloat16), _normal((B, H, N, d), 12, torch.bfloat16)
    cos, sin = (amplitude * t for t in _angles(N, r))
    dx, _ = fa.rope(dy, None, (cos, sin, layout), inverse=True)
    fa.check_device_error()
    leaf = x.double().requires_grad_()
    i = torch.arange(r // 2, device="cuda")
    lo, hi = (i, i + r // 2) if layout == HALF else (2 * i, 2 * i + 1)
    a, b = leaf[..., lo], leaf[..., hi]
    c, s = cos.double(), sin.double()
    loss = (dy[..., lo].double() * (a * c - b * s)).sum() + (dy[..., hi].double() * (a * s + b * c)).sum() \
        + (dy[..., r:].double() * leaf[..., r:]).sum()
    loss.backward()
    ref, size = turn(dy, cos, sin, layout, inverse=True)
    assert float((ref - leaf.grad).abs().max()) < 1e-12
    check_turned(dx, dy, cos, sin, layout, "gradient", inverse=True)
    # differences of the kernel's own forward along random directions
    for seed in range(3):
        step = _normal((B, H, N, d), 20 + seed, torch.bfloat16)
        moved = [fa.rope(v, None, (cos, sin, layout))[0].double() for v in (step, -step)]
        diff = float((dy.double() * (moved[0] - moved[1])).sum() / 2)
        want = float((dx.double() * step.double()).sum())
        # each side is off by a rounding (2^-8 of bf16) of each of its elements
        y, _ = turn(step, cos, sin, layout)
        tol = 1.01 * 2.0 ** -8 * float((dy.double().abs() * y.abs()).sum() + (ref.abs() * step.double().abs()).sum())
        assert abs(diff - want) <= tol


def test_inverse_undoes(fa):
    q = _normal((1, 4, 100, 128), 13, torch.float16)
    cos, sin = _angles(100, 128)
    back, _ = fa.rope(fa.rope(q, None, (cos, sin, HALF))[0], None, (cos, sin, HALF), inverse=True)
    # two roundings of half a step of at most the pair's length, and of the tables
    i = torch.arange(64, device="cuda")
    length = (q[..., i].double() ** 2 + q[..., i + 64].double() ** 2).sqrt().repeat(1, 1, 1, 2)
    assert bool(((back - q).double().abs() <= 2.5 * 2.0 ** -11 * length + 2.0 ** -23).all())


# --------------------------------------------------------------- tables --

SCALINGS = [dict(kind="none"), dict(kind="linear", factor=4.0), dict(kind="base", factor=8.0),
            dict(kind="turns", factor=8.0, original=8192, low=1.0, high=4.0), dict(kind="turns", factor=2.0, original=300, low=0.0, high=32.0),
            dict(kind="index", factor=40.0, original=4096, low=1.0, high=32.0, amplitude=0.1 * math.log(40.0) + 1.0),
            dict(kind="index", factor=2.0, original=7, low=0.5, high=64.0), dict(kind="none", amplitude=-0.7)]


@pytest.mark.parametrize("sc", SCALINGS)
@pytest.mark.parametrize("n,r,theta,start", [(1, 16, 10000.0, 0), (333, 64, 500000.0, 5), (1000, 128, 10000.0, 1 << 20), (77, 256, 1.5, 0),
                                             (200, 96, 1e6, (1 << 30) - 200)])
def test_tables(fa, n, r, theta, start, sc):
    """A value is within two units of the last place (sincospif: one; its
    argument and the amplitude half each), beside the error of the frequency
    itself, which both sides take in 64 bits: a few 2^-53 of the angle."""
    cos, sin = fa.rope_table(n, r, theta, scaling=sc, start=start)
    assert cos.shape == sin.shape == (n, r // 2)
    f = torch.tensor(frequencies(r, theta, **sc), dtype=torch.float64)
    p = torch.arange(start, start + n, dtype=torch.float64)
    ang, amp = torch.outer(p, f), sc.get("amplitude", 1.0)
    for got, ref in ((cos, ang.cos() * amp), (sin, ang.sin() * amp)):
        tol = 2.0 ** -22 * ref.abs() + abs(amp) * (ang * 2.0 ** -49 + 2.0 ** -60 * (p[:, None] + 1))
        off = (got.cpu().double() - ref).abs()
        assert bool((off <= tol).all()), f"worst excess {float((off - tol).max()):.3e}"


def test_tables_into_given_ones_and_none(fa):
    out = (torch.empty(10, 32, device="cuda"), torch.empty(10, 32, device="cuda"))
    got = fa.rope_table(10, 64, out=out)
    assert got[0] is out[0] and torch.equal(got[1], fa.rope_table(12, 64)[1][:10])
    assert torch.equal(fa.rope_table(3, 64, start=7)[0], out[0][7:])
    assert fa.rope_table(0, 64)[0].shape == (0, 32)


# --------------------------------------------------------------- append --

@pytest.mark.parametrize("layout", [INTERLEAVED, HALF])
@pytest.mark.parametrize("d,r", [(64, 64), (64, 16), (128, 96), (256, 64)])
def test_append_part_of_the_head_at_given_positions(fa, d, r, layout):
    lens, Hq, Hkv, page = [(5, 40), (1, 17), (0, 3), (33, 33)], 4, 2, 16
    T = sum(n for n, _ in lens)
    dtype = torch.bfloat16
    wide = _normal((T, Hq + 2 * Hkv, d), 14, dtype)
    q, k, v = wide.split([Hq, Hkv, Hkv], dim=1)
    cos, sin = _angles(50, r)
    for given in (True, False):
        cache = Paged([(torch.zeros(Hkv, nk, d, dtype=dtype),) * 2 for _, nk in lens], page, junk=5.0)
        cu = [0]
        for n, _ in lens:
            cu.append(cu[-1] + n)
        at = torch.cat([torch.arange(nk - n, nk) for n, nk in lens])
        pos = torch.randint(0, 50, (T,), generator=torch.Generator().manual_seed(1)) if given else at
        out = fa.cache_append(k, v, cache.k, cache.v, cache.table, ints(cu), ints([nk for _, nk in lens]), q=q, rope=(cos, sin, layout),
                              positions=pos.to(torch.int32).cuda() if given else None)
        fa.check_device_error()
        c, s = cos[pos.cuda()][:, None], sin[pos.cuda()][:, None]
        check_turned(out, q, c, s, layout, "queries")
        b = torch.cat([torch.full((n,), i) for i, (n, _) in enumerate(lens)])
        pg = cache.table.cpu()[b, at // page].long().cuda()
        check_turned(cache.k[pg, :, (at % page).cuda()], k, c, s, layout, "keys")
        assert torch.equal(cache.v[pg, :, (at % page).cuda()], v)


def test_append_drops_positions_outside_the_tables(fa):
    cache = Paged([(torch.zeros(1, 4, 64, dtype=torch.bfloat16),) * 2], 16, junk=5.0)
    k = _normal((4, 1, 64), 15, torch.bfloat16)
    cos, sin = _angles(9, 64)
    fa.cache_append(k, k, cache.k, cache.v, cache.table, ints([0, 4]), ints([4]), rope=(cos, sin, HALF), positions=ints([8, 9, -1, 0]))
    with pytest.raises(fa.FaError) as e:
        fa.check_device_error()
    assert e.value.status == fa.FA_ERR_INDEX
    page = cache.table[0, 0].long()
    assert torch.equal(cache.v[page, :, [0, 3]].transpose(0, 1), k[[0, 3]])
    assert bool((cache.v[page, :, 1:3] == 0).all())


# -------------------------------------------------- graphs and streams --

def test_a_captured_graph_follows_the_positions(fa):
    q = _normal((7, 2, 128), 16, torch.bfloat16)
    cos, sin = _angles(100, 64)
    pos, out = ints([1] * 7), torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa.rope(q, None, (cos, sin, HALF), positions=pos, q_out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            fa.rope(q, None, (cos, sin, HALF), positions=pos, q_out=out)
    torch.cuda.current_stream().wait_stream(side)
    pos.copy_(ints([9, 0, 99, 5, 5, 41, 17]))
    g.replay()
    fa.check_device_error()
    check_turned(out, q, cos[pos.long()][:, None], sin[pos.long()][:, None], HALF, "replayed")


def test_tables_of_another_width_are_refused(fa):
    q = _normal((3, 2, 64), 17, torch.bfloat16)
    for half in (4, 12, 40, 0):
        cos = torch.zeros(8, half, device="cuda")
        with pytest.raises(ValueError):
            fa.rope(q, None, (cos, cos, HALF))
