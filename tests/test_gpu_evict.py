"""GPU parity of hlta_paged_evict: the kept positions, their keys, values and weights, bit for bit."""
import math

import pytest
import torch

from serving_util import Cache

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def h():
    import linear_video_world_b200 as h
    assert torch.cuda.is_available()
    return h


def _keep(w, n, budget, sink, recent):
    if n <= budget:
        return list(range(n))
    rank = lambda i: (math.inf if math.isnan(w[i]) else -w[i], i)   # noqa: E731
    mid = sorted(range(sink, n - recent), key=rank)[:budget - sink - recent]
    return list(range(sink)) + sorted(mid) + list(range(n - recent, n))


def _weights(kind, *shape):
    g = torch.Generator().manual_seed(11)
    u = torch.rand(shape, generator=g)
    if kind == "ties":
        return (u * 4).floor() / 4
    if kind == "equal":
        return torch.full(shape, 0.5)
    if kind == "odd":           # NaN, infinities, zeros of both signs, negative, denormal
        pool = torch.tensor([float("nan"), math.inf, -math.inf, 0.0, -0.0, -1.0, 1e-42, 2e-42, 1.0, -1e-42])
        return pool[(u * len(pool)).long().clamp(max=len(pool) - 1)]
    return u ** 6


@pytest.mark.parametrize("kind", ["skewed", "ties", "equal", "odd"])
@pytest.mark.parametrize("dtype,d,page,kv,budget,sink,recent", [
    (BF, 128, 16, [100, 33, 1, 0, 20], 33, 4, 8),       # above, at and below the budget
    (BF, 128, 64, [1500, 1025], 700, 0, 0),             # several scans of a block
    (F32, 128, 32, [90, 64], 64, 64, 0),                # the first ones alone
    (F32, 40, 16, [90, 65], 64, 0, 64),                 # the last ones alone
    (F32, 7, 128, [200, 130], 129, 1, 127),             # all but one
    (BF, 9, 16, [50], 1, 0, 0),                         # one
])
def test_evict(h, kind, dtype, d, page, kv, budget, sink, recent):
    H, B = 3, len(kv)
    c = Cache(kv, H, d, page, dtype, seed=budget)
    kp, vp, table, lens = c.cuda()
    w = _weights(kind, B, H, table.shape[1] * page)
    for b, n in enumerate(kv):
        w[b, :, n:] = math.inf              # behind the end: never read
    dw = -(-budget // page) + 1
    kd, vd = (torch.full((B * dw + 1, H, page, d), 5.0, device="cuda").to(dtype) for _ in range(2))
    dst = torch.randperm(B * dw, generator=torch.Generator().manual_seed(3)).to(torch.int32).view(B, dw).cuda()
    kept = torch.full((B, H, budget), -9, dtype=torch.int32, device="cuda")
    w_out = torch.full((B, H, dw * page), 6.0, device="cuda")
    new = h.paged_evict(w.cuda(), kp, vp, table, lens, budget, sink, recent, kd, vd, dst, kept=kept, w_out=w_out)
    assert h.hlta_device_status() == 0
    assert new.tolist() == [min(n, budget) for n in kv]
    K, V = torch.full_like(kd, 5.0).cpu(), torch.full_like(vd, 5.0).cpu()
    W = torch.full_like(w_out, 6.0).cpu()
    for b, n in enumerate(kv):
        for g in range(H):
            keep = _keep(w[b, g].tolist(), n, budget, sink, recent)
            assert kept[b, g].tolist() == keep + [-1] * (budget - len(keep))
            for r, i in enumerate(keep):
                pg = int(dst[b, r // page])
                K[pg, g, r % page], V[pg, g, r % page] = c.keys[b][g, i], c.vals[b][g, i]
                W[b, g, r] = w[b, g, i]
    assert torch.equal(kd.cpu(), K) and torch.equal(vd.cpu(), V)
    assert torch.equal(w_out.cpu().nan_to_num(1.25), W.nan_to_num(1.25))
    # without the optional outputs, into the pool itself (fresh pages at its end)
    kp2, vp2 = (torch.cat([p, torch.full_like(kd, 5.0)]) for p in (kp, vp))
    h.paged_evict(w.cuda(), kp2, vp2, table, lens, budget, sink, recent, kp2, vp2, dst + kp.shape[0])
    assert torch.equal(kp2[kp.shape[0]:].cpu(), K) and torch.equal(vp2[kp.shape[0]:].cpu(), V)
    assert torch.equal(kp2[:kp.shape[0]].nan_to_num(1.25), kp.nan_to_num(1.25))


@pytest.mark.parametrize("n,budget,H", [(120000, 50001, 1), (20000, 7001, 3), (20000, 7001, 80)])
def test_long_rows(h, n, budget, H):
    """Two blocks a row or one, more positions than they hold in shared memory, equal weights
    straddling the border."""
    page = 128
    width = -(-n // page)
    kp, vp = (torch.randn(width, H, page, 16, device="cuda") for _ in range(2))
    table = torch.randperm(width, device="cuda").to(torch.int32)[None].contiguous()
    w = (torch.rand(1, H, width * page, generator=torch.Generator().manual_seed(1)) * 1000).floor()
    dw = -(-budget // page)
    kd, vd = (torch.zeros(dw, H, page, 16, device="cuda") for _ in range(2))
    dst = torch.arange(dw, dtype=torch.int32, device="cuda")[None].contiguous()
    kept = torch.zeros((1, H, budget), dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    h.paged_evict(w.cuda(), kp, vp, table, lens, budget, 100, 1000, kd, vd, dst, kept=kept)
    assert h.hlta_device_status() == 0
    for x in {0, H - 1}:
        assert kept[0, x].tolist() == _keep(w[0, x].tolist(), n, budget, 100, 1000)
        at = kept[0, x].long()
        assert torch.equal(kd[:, x].reshape(-1, 16)[:budget], kp[table[0].long(), x].reshape(-1, 16)[at])
        assert torch.equal(vd[:, x].reshape(-1, 16)[:budget], vp[table[0].long(), x].reshape(-1, 16)[at])


def test_tables_out_of_range_are_reported(h):
    c = Cache([60, 50], 2, 128, 16, BF, seed=1)
    for what in ("src", "dst", "len"):
        kp, vp, table, lens = c.cuda()
        kp, vp = kp.nan_to_num(0.0), vp.nan_to_num(0.0)
        w = _weights("skewed", 2, 2, table.shape[1] * 16).cuda()
        kd, vd = (torch.zeros(5, 2, 16, 128, device="cuda", dtype=BF) for _ in range(2))
        dst = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
        if what == "src":
            table[0, 0] = kp.shape[0]
        elif what == "dst":
            dst[0, 1] = 5
        else:
            lens[0] = 10 ** 6
            table[0] = table[0].clamp(0, kp.shape[0] - 1)
        h.paged_evict(w, kp, vp, table, lens, 30, 2, 5, kd, vd, dst)
        st, word = h.hlta_device_status_code()
        assert st == h.HLTA_ERR_INVALID_ARG and word == h.HLTA_DEVERR_TABLE, what
        assert bool((kd[4] == 0).all())
