"""GPU parity of hlta_rope_axes against the 64-bit form, and its inverse as the gradient."""
import pytest
import torch

from serving_util import grid_positions, rope_bound, rope_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def h():
    import linear_video_world_b200 as h
    assert torch.cuda.is_available()
    return h


def _x(*shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _check(got, x, ref, pairs, halves):
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= rope_bound(x, ref, pairs, halves)).all()), float(err.max())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("d,pairs,B,Hq,Hk,L", [
    (128, (22, 21, 21), 2, 5, 3, 77),     # every channel rotated, odd lengths
    (128, (8, 16, 16), 1, 1, 1, 1),       # one token, channels passing through
    (128, (0, 32, 32), 3, 9, 2, 300),     # images: no time axis
    (64, (4, 3, 5), 2, 2, 1, 33),         # 2P no multiple of a 16-byte chunk
    (13, (1, 2, 3), 2, 3, 2, 9),          # odd d
    (16, (0, 0, 0), 1, 2, 2, 5),          # nothing rotates: a copy
])
def test_grid_and_positions(h, dtype, halves, d, pairs, B, Hq, Hk, L):
    q, k = _x(B, Hq, L, d, dtype=dtype, seed=1), _x(B, Hk, L, d, dtype=dtype, seed=2)
    grid, t0 = (3, 4), torch.arange(B, dtype=torch.int32) * 11
    for shared, pos in ((False, None), (True, torch.randint(-50, 70000, (B, L, 3), generator=torch.Generator().manual_seed(3), dtype=torch.int32))):
        at = grid_positions(B, L, grid, t0) if pos is None else pos
        kw = dict(grid=grid, t0=t0.cuda()) if pos is None else dict(pos=pos.cuda())
        gq, gk = h.rope_axes(q.cuda(), k.cuda(), pairs, halves=halves, shared_freq=shared, **kw)
        for got, x in ((gq, q), (gk, k)):
            _check(got, x, rope_ref(x, pairs, at, halves=halves, shared=shared), pairs, halves)
    assert h.hlta_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_positions(h, dtype):
    """Positions up to the ends of int32: the angle is reduced in double precision. The product
    position * frequency is off by 2^-53 of 2^31 / (2 pi) turns, 2.4e-7 rad on top of the bound."""
    pos = torch.tensor([[[2 ** 31 - 1, -2 ** 31, 123456789], [0, 1, -1]]], dtype=torch.int32)
    x = _x(1, 2, 2, 128, dtype=dtype, seed=5)
    got, _ = h.rope_axes(x.cuda(), None, (22, 21, 21), pos=pos.cuda())
    ref = rope_ref(x, (22, 21, 21), pos)
    m = x.double().abs()
    pair = torch.repeat_interleave(m[..., 0::2] + m[..., 1::2], 2, -1)
    assert bool(((got.double().cpu() - ref).abs() <= rope_bound(x, ref, (22, 21, 21), False) + 2 * 2.4e-7 * pair).all())


@pytest.mark.parametrize("halves", [False, True])
def test_in_place_and_round_trip(h, halves):
    q = _x(2, 3, 50, 128, dtype=F32, seed=7)
    g = q.cuda()
    out = h.rope_axes(g, None, (22, 21, 21), grid=(5, 5), halves=halves, out=(g, None))
    assert out[0] is g
    _check(g, q, rope_ref(q, (22, 21, 21), grid_positions(2, 50, (5, 5)), halves=halves), (22, 21, 21), halves)
    h.rope_axes(g, None, (22, 21, 21), grid=(5, 5), halves=halves, inverse=True, out=(g, None))
    # two rotations: twice the bound of one on values of at most |x0| + |x1|
    assert float((g.cpu() - q).abs().max()) <= 2 * 8e-7 * 2 * float(q.abs().max())


def test_inverse_is_the_gradient(h):
    """<dy, R(x + e z) - R(x - e z)> / 2e = <R^-1 dy, z>, R linear: differences without a limit."""
    pairs, grid = (5, 4, 3), (2, 3)
    x, z, dy = (_x(1, 2, 7, 32, dtype=F32, seed=s).cuda() for s in (1, 2, 3))
    f = lambda t: h.rope_axes(t, None, pairs, grid=grid, halves=True)[0].double()   # noqa: E731
    num = float((dy.double() * (f(x + z) - f(x - z)) / 2).sum())
    ana = float((h.rope_axes(dy, None, pairs, grid=grid, halves=True, inverse=True)[0].double() * z.double()).sum())
    scale = float((dy.double().abs() * (x.double().abs() + z.double().abs())).sum())
    assert abs(num - ana) <= 8 * 8e-7 * scale


def test_equals_rope_of_one_axis(h):
    """With one axis of all pairs and a grid of one row the rotation is hlta_rope's (both forms
    round the same angle differently: twice the bound)."""
    q = _x(1, 2, 40, 128, dtype=F32, seed=9)
    a = q.cuda().clone()
    h.rope(a, None, N=40, pos_mode=0)
    b, _ = h.rope_axes(q.cuda(), None, (0, 0, 64), grid=(1, 40))
    assert float((a - b).abs().max()) <= 2 * 8e-7 * 2 * float(q.abs().max())
