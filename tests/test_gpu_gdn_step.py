"""GPU parity of the recurrent gated delta rule over a pool of states (64-bit recurrence, and the
chunk form's oracle)."""
import pytest
import torch

from serving_util import EPS, gdn_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def h():
    import linear_video_world_b200 as h
    assert torch.cuda.is_available()
    return h


def _inputs(B, H, L, d, dtype, raw, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(B, H, L, d, generator=g) for _ in range(3))
    x, y = (torch.randn(B, H, L, generator=g) for _ in range(2))
    if not raw:
        q, k = (t / t.norm(dim=-1, keepdim=True) for t in (q, k))
        x, y = torch.exp(-torch.nn.functional.softplus(x)), torch.sigmoid(y)
    return q.to(dtype), k.to(dtype), v.to(dtype), x, y


def _check(o, S, q, k, v, a, b, S0, n, dtype, raw, c=0.7):
    if raw:
        q, k = (t.double() / t.double().norm(dim=-1, keepdim=True).clamp(min=1e-300) for t in (q, k))
        a, b = torch.exp(-c * torch.nn.functional.softplus(a.double())), torch.sigmoid(b.double())
    ro, rS, bound = gdn_ref(q, k, v, a, b, S0, n)
    if raw:                     # unit norms and gates: a few roundings more of factors of order one
        bound *= 2
    assert float((S.double() - rS).abs().max()) <= bound
    half = EPS[dtype] if dtype == BF else 0.0
    assert bool(((o[:, :n].double() - ro[:, :n]).abs() <= bound + half * (ro[:, :n].abs() + bound)).all())


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("dtype,d,B,H,L", [(BF, 128, 1, 1, 1), (BF, 128, 5, 3, 1), (BF, 128, 3, 2, 9), (F32, 128, 2, 8, 4), (F32, 64, 3, 2, 5),
                                           (F32, 1, 2, 1, 3), (F32, 37, 2, 3, 2)])
def test_step(h, raw, dtype, d, B, H, L):
    q, k, v, a, b = _inputs(B, H, L, d, dtype, raw, seed=L)
    if raw and L > 1:
        q[0, 0, 1], k[0, 0, 0] = 0.0, 0.0               # zero vectors stay zero
    slots_n = B + 3
    S = 0.3 * torch.randn(slots_n, H, d, d, generator=torch.Generator().manual_seed(5))
    slots = torch.randperm(slots_n, generator=torch.Generator().manual_seed(6))[:B].to(torch.int32)
    lens = torch.tensor([(L - i) % (L + 1) for i in range(B)], dtype=torch.int32)      # all tokens, one fewer, ..., none
    out, S_out = torch.full_like(q, 44.0).cuda(), torch.full_like(S, 22.0).cuda()
    args = [t.cuda() for t in (q, k, v, a, b)]
    call = (lambda **kw: h.gdn_step_raw(*args, 0.7, S.cuda(), **kw)) if raw else (lambda **kw: h.gdn_step(*args, S.cuda(), **kw))
    call(slots=slots.cuda(), lens=lens.cuda(), out=out, S_out=S_out)
    assert h.hlta_device_status() == 0
    out, S_out = out.cpu(), S_out.cpu()
    for r in range(B):
        n, s = int(lens[r]), int(slots[r])
        _check(out[r], S_out[s], q[r], k[r], v[r], a[r], b[r], S[s], n, dtype, raw)
        assert bool((out[r, :, n:] == 44).all())
        if n == 0:
            assert torch.equal(S_out[s], S[s])
    rest = sorted(set(range(slots_n)) - set(slots.tolist()))
    assert bool((S_out[rest] == 22).all())
    # in place, without tables
    pool = S[:B].clone().cuda()
    o = (h.gdn_step_raw(*args, 0.7, pool) if raw else h.gdn_step(*args, pool))[0].cpu()
    for r in range(B):
        _check(o[r], pool[r].cpu(), q[r], k[r], v[r], a[r], b[r], S[r], L, dtype, raw)


def test_token_by_token_equals_one_call(h):
    q, k, v, a, b = (t.cuda() for t in _inputs(2, 2, 6, 128, BF, False))
    S = 0.1 * torch.randn(2, 2, 128, 128, device="cuda")
    one, many = S.clone(), S.clone()
    o1, _ = h.gdn_step(q, k, v, a, b, one)
    o2 = torch.cat([h.gdn_step(*(t[:, :, i:i + 1].contiguous() for t in (q, k, v, a, b)), many)[0] for i in range(6)], 2)
    assert torch.equal(o1, o2) and torch.equal(one, many)


def test_against_the_chunk_form(h, orc):
    """The same recurrence as hlta_gdn_chunk_fwd: both against its oracle, at that test's tolerance."""
    q, k, v, a, b = _inputs(1, 2, 40, 128, BF, False, seed=3)
    S0 = 0.1 * torch.randn(1, 2, 128, 128, generator=torch.Generator().manual_seed(2))
    args = [t.cuda() for t in (q, k, v, a, b)]
    o, S = h.gdn_step(*args, S0.cuda(), S_out=torch.empty_like(S0).cuda())
    oc, Sc = h.gdn(*args, S0=S0.cuda())
    ro, rS = orc.gdn(q, k, v, a, b, S0.double().numpy())
    assert float((o.double().cpu() - torch.from_numpy(ro).view(o.shape)).abs().max()) <= 2e-2
    assert float((S.double().cpu() - torch.from_numpy(rS).view(S.shape)).abs().max()) <= 1e-4
    assert float((o - oc).abs().max()) <= 4e-2 and float((S - Sc).abs().max()) <= 4e-2


def test_padded_and_bad_slots(h):
    q, k, v, a, b = (t.cuda() for t in _inputs(5, 2, 2, 128, BF, False))
    S = torch.randn(4, 2, 128, 128, device="cuda")
    clean = S.clone()
    want, want_S = h.gdn_step(q[:1].contiguous(), k[:1].contiguous(), v[:1].contiguous(), a[:1].contiguous(), b[:1].contiguous(), S[2:3].clone())
    out = torch.full_like(q, 8.0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")      # noqa: E731
    # a padded batch: nothing to report
    pool = clean.clone()
    h.gdn_step(q, k, v, a, b, pool, slots=i32([2, -1, -1, -5, -1]), out=out)
    assert h.hlta_device_status() == 0
    assert torch.equal(out[0], want[0]) and torch.equal(pool[2], want_S[0]) and bool((out[1:] == 8).all())
    assert torch.equal(pool[[0, 1, 3]], clean[[0, 1, 3]])
    # a slot out of range, a slot twice (the first keeps it), a bad length: reported and skipped
    for slots, lens, ok in (([2, 4, 0, 1, 3], None, [0, 2, 3, 4]), ([2, 2, 0, 2, 3], None, [0, 2, 4]), ([2, 1, 0, 3, -1], [2, 3, 2, -1, 1], [0, 2])):
        pool, out = clean.clone(), torch.full_like(q, 8.0)
        h.gdn_step(q, k, v, a, b, pool, slots=i32(slots), lens=None if lens is None else i32(lens), out=out)
        st, word = h.hlta_device_status_code()
        assert st == h.HLTA_ERR_INVALID_ARG and word == h.HLTA_DEVERR_TABLE
        assert torch.equal(out[0], want[0]) and torch.equal(pool[2], want_S[0])
        for r in range(5):
            if r not in ok:
                assert bool((out[r] == 8).all())
        idle = sorted(set(range(4)) - {slots[r] for r in ok})
        assert torch.equal(pool[idle], clean[idle])


def test_captured_step_replayed(h):
    q, k, v, a, b = (t.cuda() for t in _inputs(3, 2, 1, 128, BF, False))
    S0 = torch.randn(3, 2, 128, 128, device="cuda")
    pool, out = S0.clone(), torch.zeros_like(q)
    h.gdn_step(q, k, v, a, b, S0.clone(), out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h.gdn_step(q, k, v, a, b, pool, out=out)
    ref = S0.clone()
    for seed in (1, 2, 3):
        for t, n in zip((q, k, v, a, b), _inputs(3, 2, 1, 128, BF, False, seed=seed)):
            t.copy_(n)
        g.replay()
        want, _ = h.gdn_step(q, k, v, a, b, ref)
        assert torch.equal(out, want) and torch.equal(pool, ref)


def test_empty_batch_and_empty_step(h):
    q, k, v, a, b = (t.cuda() for t in _inputs(2, 2, 3, 128, BF, False))
    S = torch.randn(2, 2, 128, 128, device="cuda")
    o, So = h.gdn_step(*(t[:0] for t in (q, k, v, a, b)), S.clone())
    assert o.shape[0] == 0 and torch.equal(So, S)
    o, So = h.gdn_step(*(t[:, :, :0].contiguous() for t in (q, k, v, a, b)), S, S_out=torch.zeros_like(S))
    assert o.numel() == 0 and torch.equal(So, S) and h.hlta_device_status() == 0
