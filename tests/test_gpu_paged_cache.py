"""The serving operators together, as a rollout server uses them: PagedCache with rotary axes, frame
windows and eviction, beside the recurrent gated delta rule, against a 64-bit form of the whole."""
import pytest
import torch

from serving_util import Cache, attn_ref, gdn_ref, grid_positions, rope_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
PAIRS = (22, 21, 21)


@pytest.fixture(scope="module")
def h():
    import linear_video_world_b200 as h
    assert torch.cuda.is_available()
    return h


class Twin:
    """What PagedCache should hold: each rollout's rounded keys and values by position."""

    def __init__(self, B, H, d, page, width, dtype):
        self.keys = [torch.zeros(H, 0, d).to(dtype) for _ in range(B)]
        self.vals = [torch.zeros(H, 0, d).to(dtype) for _ in range(B)]
        self.page, self.k, self.table = page, torch.zeros(1, H, page, d), torch.zeros(B, width)

    @property
    def kv(self):
        return [k.shape[1] for k in self.keys]


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rollouts_with_windows_and_eviction(h, dtype):
    """Frames of 6 tokens for three rollouts that start at different times, one padded; every step
    rotates, appends, attends (three frames back, weights kept) and runs the gated delta heads;
    after steps 3 and 5 the rollouts are cut to 20 tokens."""
    B, Hq, H, Hg, d, N, page = 3, 4, 2, 2, 128, 6, 16
    grid, gen = (2, 3), torch.Generator().manual_seed(5)
    cache = h.PagedCache(B, H, d, num_pages=24, max_len=64, page=page, dtype=dtype, weights=True, decay=0.75)
    twin = Twin(B, H, d, page, cache.width, dtype)
    weights = torch.zeros(B, H, cache.width * page).double()
    slack = torch.zeros_like(weights)
    pool = 0.1 * torch.randn(B + 1, Hg, d, d, generator=gen)
    slots = torch.tensor([3, 0, 1], dtype=torch.int32)
    state, states = pool.cuda(), [pool[s].clone() for s in slots]
    steps = [0] * B
    for step in range(6):
        new = [N, N if step >= 1 else 0, [N, N, 5, N, 1, N][step]]
        q, k, v = (torch.randn(B, n, N, d, generator=gen).to(dtype) for n in (Hq, H, H))
        t0 = torch.tensor(steps, dtype=torch.int32)
        rq, _ = h.rope_axes(q.cuda(), None, PAIRS, grid=grid, t0=t0.cuda())
        cache.append(k.cuda(), v.cuda(), new, rope=dict(pairs=PAIRS, grid=grid, t0=t0.cuda()))
        # the rotation itself is compared elsewhere; here its rounded result goes on
        rk = h.rope_axes(k.cuda(), None, PAIRS, grid=grid, t0=t0.cuda())[0].cpu()
        ref = rope_ref(k, PAIRS, grid_positions(B, N, grid, t0))
        assert float((rk.double() - ref).abs().max()) <= (2.0 ** -8 if dtype == BF else 2.0 ** -20) * float(ref.abs().max())
        for b in range(B):
            twin.keys[b] = torch.cat([twin.keys[b], rk[b, :, :new[b]]], 1)
            twin.vals[b] = torch.cat([twin.vals[b], v[b, :, :new[b]]], 1)
        assert cache.lens == twin.kv
        lse = torch.zeros(B, Hq, N, device="cuda")
        o = cache.attend(rq, N=N, w=3, lse=lse)
        ro, rl, rw, ob, lb, wb = attn_ref(rq.cpu(), twin, new, N, 3, weights, 0.75)
        for b, n in enumerate(new):
            assert bool(((o[b, :, :n].cpu().double() - ro[b, :, :n]).abs() <= ob[b, :, :n]).all())
            assert bool(((lse[b, :, :n].cpu().double() - rl[b, :, :n]).abs() <= lb[b, :, :n]).all())
            assert bool((o[b, :, n:] == 0).all())
            kv = cache.lens[b]
            slack[b, :, :kv] = 0.75 * slack[b, :, :kv] + wb[b, :, :kv] + 1e-30
            slack[b, :, kv - n:kv] = wb[b, :, kv - n:kv] + 1e-30
            got = cache.weights[b, :, :kv].cpu().double()
            assert bool(((got - rw[b, :, :kv]).abs() <= slack[b, :, :kv]).all())
            weights[b, :, :kv] = rw[b, :, :kv]
        # the gated delta heads of the same tokens
        gq, gk, gv = (torch.randn(B, Hg, N, d, generator=gen) for _ in range(3))
        gq, gk = (t / t.norm(dim=-1, keepdim=True) for t in (gq, gk))
        gq, gk, gv = gq.to(dtype), gk.to(dtype), gv.to(dtype)
        a, g = torch.rand(B, Hg, N, generator=gen), torch.rand(B, Hg, N, generator=gen)
        go, _ = h.gdn_step(gq.cuda(), gk.cuda(), gv.cuda(), a.cuda(), g.cuda(), state, slots.cuda(), torch.tensor(new, dtype=torch.int32).cuda())
        for b, n in enumerate(new):
            po, pS, bound = gdn_ref(gq[b], gk[b], gv[b], a[b], g[b], states[b], n)
            got = state[int(slots[b])].cpu()
            assert float((got.double() - pS).abs().max()) <= bound
            half = 2.0 ** -8 if dtype == BF else 0.0
            assert bool(((go[b, :, :n].cpu().double() - po[:, :n]).abs() <= bound + half * (po[:, :n].abs() + bound)).all())
            states[b] = got
            steps[b] += 1 if n else 0
        if step in (3, 5):
            kept_by = cache.weights.cpu()
            cut = cache.evict(20, sink=2, recent=N)
            assert cut == [b for b in range(B) if twin.kv[b] > 20] and cut
            # every page is free or one rollout's, no rollout has more than it needs
            assert sorted(cache._free + sum(cache._pages, [])) == list(range(24))
            assert [len(x) for x in cache._pages] == [-(-n // page) for n in cache.lens]
            for b in cut:
                n = twin.kv[b]
                K, V, W = [], [], []
                for g2 in range(H):
                    w = kept_by[b, g2]
                    mid = sorted(range(2, n - N), key=lambda i: (-float(w[i]), i))[:20 - 2 - N]
                    keep = list(range(2)) + sorted(mid) + list(range(n - N, n))
                    K.append(twin.keys[b][g2, keep])
                    V.append(twin.vals[b][g2, keep])
                    weights[b, g2, :20], slack[b, g2, :20] = weights[b, g2, keep].clone(), slack[b, g2, keep].clone()
                    W.append(w[keep])
                twin.keys[b], twin.vals[b] = torch.stack(K), torch.stack(V)
                assert torch.equal(cache.weights[b, :, :20].cpu(), torch.stack(W))
            assert cache.lens == twin.kv
            for b in range(B):                          # what the pages hold now
                for i in range(cache.lens[b]):
                    pg = int(cache.table[b, i // page])
                    assert torch.equal(cache.k_pages[pg, :, i % page].cpu(), twin.keys[b][:, i])
                    assert torch.equal(cache.v_pages[pg, :, i % page].cpu(), twin.vals[b][:, i])
    assert h.hlta_device_status() == 0


def test_pages_are_counted(h):
    cache = h.PagedCache(2, 1, 128, num_pages=5, max_len=80, page=16, weights=True)
    k = torch.zeros(2, 1, 40, 128, device="cuda", dtype=BF)
    cache.append(k, k, [40, 20])
    assert cache.lens == [40, 20] and len(cache._free) == 0
    for bad in (dict(new_lens=[1, 13]), dict(new_lens=[41, 0]), dict(new_lens=[1]), dict(new_lens=[-1, 0])):
        with pytest.raises(h.HltaError):
            cache.append(k, k, **bad)
        assert cache.lens == [40, 20]
    with pytest.raises(h.HltaError):
        cache.evict(16)                                 # no free page to copy to
    cache.append(k, k, [8, 12])
    cache.release(1)
    assert cache.lens == [48, 0] and len(cache._free) == 2
    assert cache.evict(16) == [0] and cache.lens == [16, 0] and len(cache._free) == 4
    cache.append(k, k, [40, 0])
    with pytest.raises(h.HltaError):
        cache.append(k, k, [25, 0])                     # past max_len
    q = torch.zeros(2, 2, 40, 128, device="cuda", dtype=BF)
    assert cache.attend(q).shape == q.shape and h.hlta_device_status() == 0
    with pytest.raises(h.HltaError):
        h.PagedCache(1, 1, 128, 4, 64, page=24)
    plain = h.PagedCache(1, 1, 128, 4, 64)
    with pytest.raises(h.HltaError):
        plain.evict(3)


def test_rollout_continues_as_one_call(h):
    """A clip token by token, in chunks, and at once: the same positions see the same keys, so the
    outputs agree within the roundings of P and the output of both."""
    H, L = 2, 90
    q, k, v = (torch.randn(1, H, L, 128, generator=torch.Generator().manual_seed(s)).to(BF).cuda() for s in (1, 2, 3))
    got = []
    for sizes in ([90], [1] * 90, [17, 1, 40, 16, 16]):
        c = h.PagedCache(1, H, 128, 8, 128, page=16)
        outs, at = [], 0
        for n in sizes:
            s = slice(at, at + n)
            c.append(k[:, :, s].contiguous(), v[:, :, s].contiguous())
            outs.append(c.attend(q[:, :, s].contiguous()))
            at += n
        got.append(torch.cat(outs, 2))
    bound = 4 * 2.0 ** -8 * float(v.abs().max())
    assert float((got[0] - got[1]).abs().max()) <= bound and float((got[0] - got[2]).abs().max()) <= bound
    assert h.hlta_device_status() == 0


def test_results_allocated_on_the_call_s_stream(h):
    """A call on another stream than the current one, which is busy: what the wrappers allocate and
    fill belongs to the call's stream."""
    c = Cache([70, 33], 2, 128, 16, torch.bfloat16, seed=5)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(2, 4, 3, 128, generator=g).to(torch.bfloat16).cuda()
    kp, vp, table, lens = c.cuda()
    new = torch.tensor([3, 2], dtype=torch.int32).cuda()
    S, a = torch.randn(2, 4, 128, 128, generator=g).cuda(), torch.rand(2, 4, 3, generator=g).cuda()
    u = torch.nn.functional.normalize(q.float(), dim=-1).to(torch.bfloat16)
    want = h.paged_attn(q, kp, vp, table, lens, new), h.gdn_step(u, u, q, a, a, S.clone(), lens=new)[0]
    So = torch.empty_like(S)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)              # the current stream is busy for about 0.1 s
    got = []
    for s in (side, side.cuda_stream):
        got += [h.paged_attn(q, kp, vp, table, lens, new, stream=s), h.gdn_step(u, u, q, a, a, S, S_out=So, lens=new, stream=s)[0]]
    torch.cuda.synchronize()
    for x, y in zip(got, want * 2):
        assert torch.equal(x, y)


def test_refused_append_changes_nothing(h):
    c = h.PagedCache(2, 2, 128, 8, 64, page=16)
    k = torch.randn(2, 2, 20, 128, device="cuda").to(torch.bfloat16)
    c.append(k, k, [20, 3])
    state = list(c.lens), [list(p) for p in c._pages], sorted(c._free), c.table.clone(), c.kv_lens.clone()
    for bad in (k.float(), k[..., :64], k[:, :1], k[:1], k.transpose(1, 2)):
        with pytest.raises(h.HltaError):
            c.append(bad, bad, [bad.shape[2], 20])
        with pytest.raises(h.HltaError):
            c.append(k, k, rope=dict(pairs=(60, 60, 0), grid=(1, 1)))
        assert (c.lens, c._pages, sorted(c._free)) == state[:3]
        assert torch.equal(c.kv_lens, state[4]) and torch.equal(c.table, state[3])
    c.append(k, k, [5, 20])
    assert c.lens == [25, 23] and h.hlta_device_status() == 0


def test_attending_after_a_rollout_was_cut_or_released(h):
    c = h.PagedCache(3, 2, 128, 20, 64, page=16, weights=True)
    k, q = (torch.randn(3, n, 40, 128, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda() for n in (2, 4))
    c.append(k, k, [40, 30, 20])
    o = c.attend(q, N=40)
    w = c.weights.clone()
    assert c.evict(33) == [0]
    c.release(1)
    again = c.attend(q, N=40)
    assert h.hlta_device_status() == 0
    assert torch.equal(again[2], o[2]) and bool((again[:2] == 0).all())
    # what the cut rollout kept has its weights, once
    assert torch.equal(c.weights[0, :, :33].sort(-1).values, w[0, :, :40].sort(-1).values[:, -33:])


@pytest.mark.parametrize("emptied_by", ["release", "evict"])
@pytest.mark.parametrize("Hq", [2, 4])
def test_weights_of_an_earlier_occupant_are_gone(h, emptied_by, Hq):
    """Chunks appended where a released or cut rollout's positions were, the last one alone attended:
    the weights of a call that starts those positions from zero."""
    gen = torch.Generator().manual_seed(3)
    k, q = (torch.randn(2, n, 20, 128, generator=gen).to(BF).cuda() for n in (2, Hq))
    c = h.PagedCache(2, 2, 128, 20, 64, page=16, weights=True, decay=0.5)
    c.append(k, k, [20, 13])
    c.attend(q)
    if emptied_by == "release":
        c.release(0)
        kept = 0
    else:
        kept = 6
        assert c.evict(kept, sink=1, recent=2) == [0, 1]
    for n in (9, 4):
        x = k[:, :, :n].contiguous()
        c.append(x, x)
    start = c.weights.clone()
    start[:, :, kept:] = 0.0
    if emptied_by == "release":
        start[1] = c.weights[1]                     # as it was: nothing was cut there
        assert bool((c.weights[1, :, :13] > 0).any())
    want = start.clone()
    x = q[:, :, :4].contiguous()
    o = h.paged_attn(x, c.k_pages, c.v_pages, c.table, c.kv_lens, w_in=start, w_out=want, decay=0.5)
    assert torch.equal(c.attend(x), o)
    for b, n in enumerate(c.lens):
        assert torch.equal(c.weights[b, :, :n], want[b, :, :n])
    # eviction goes by them: positions never attended have none
    if emptied_by == "release":
        c.release(0)
        c.append(k, k, [20, 0])
        assert c.evict(5)[:1] == [0] and torch.equal(c.k_pages[c._pages[0][0], :, :5], k[0, :, :5])
    assert h.hlta_device_status() == 0


def test_attending_after_a_refused_append(h):
    """A refused append leaves the chunk appended before it the one that is attended."""
    gen = torch.Generator().manual_seed(4)
    k, q = (torch.randn(2, n, 20, 128, generator=gen).to(BF).cuda() for n in (2, 4))
    c = h.PagedCache(2, 2, 128, 8, 64, page=16)
    c.append(k, k, [20, 3])
    new, want = c.new_lens.clone(), c.attend(q)
    with pytest.raises(h.HltaError):
        c.append(k.float(), k.float(), [1, 20])
    assert torch.equal(c.new_lens, new) and torch.equal(c.attend(q), want)
    assert h.hlta_device_status() == 0


def test_captured_attend_replayed_around_evictions(h):
    """An attend captured once serves chunks appended before and after an eviction and a release: the
    same bits, and the same weights, as the call made anew."""
    gen = torch.Generator().manual_seed(6)
    c = h.PagedCache(2, 2, 128, 20, 64, page=16, weights=True, decay=0.5)
    k, q = (torch.randn(2, n, 5, 128, generator=gen).to(BF).cuda() for n in (2, 4))
    out = torch.zeros_like(q)
    c.append(k, k)
    c.attend(q, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(q, out=out)
    for step in range(8):
        if step == 3:
            assert c.evict(9, sink=1, recent=3) == [0, 1]
        if step == 5:
            c.release(1)
        k.copy_(torch.randn(2, 2, 5, 128, generator=gen))
        q.copy_(torch.randn(2, 4, 5, 128, generator=gen))
        c.append(k, k, [5, 5 - step % 3])
        want_w = c.weights.clone()
        want = h.paged_attn(q, c.k_pages, c.v_pages, c.table, c.kv_lens, c.new_lens, out=out.clone(), w_in=want_w, w_out=want_w, decay=0.5)
        g.replay()
        assert torch.equal(out, want) and torch.equal(c.weights, want_w)
    assert h.hlta_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [1, 20])
def test_step_captured_and_replayed(h, dtype, L):
    """A whole step in one graph: rotation, append (rotated on the way), attention with weights kept in
    place, the gated delta rule, eviction into another pool. Replayed for other tokens and lengths, below
    and above the budget: the bits of the calls made one by one."""
    B, H, Hq, page, width, budget = 2, 2, 6, 16, 8, 40
    gen, lens_of = torch.Generator().manual_seed(L), [[30, 41], [100, 40], [128, 39 + L], [L, 127]]
    rand = lambda *s: torch.randn(*s, generator=gen).to(dtype)      # noqa: E731
    ins = dict(q=rand(B, Hq, L, 128).cuda(), k=rand(B, H, L, 128).cuda(), v=rand(B, H, L, 128).cuda(), a=torch.rand(B, Hq, L, generator=gen).cuda(),
               lens=torch.tensor(lens_of[0], dtype=torch.int32).cuda(), new=torch.tensor([L, L], dtype=torch.int32).cuda(), t0=torch.tensor([3, 5], dtype=torch.int32).cuda())
    table = torch.randperm(B * width, generator=gen).to(torch.int32).view(B, width).cuda()
    dst = torch.randperm(2 * 3, generator=gen).to(torch.int32).view(B, 3).cuda()
    start = dict(kp=rand(B * width, H, page, 128).cuda(), vp=rand(B * width, H, page, 128).cuda(), w=torch.rand(B, H, width * page, generator=gen).cuda(),
                 S=0.1 * torch.randn(B, Hq, 128, 128, generator=gen).cuda(), kd=torch.zeros(6, H, page, 128, dtype=dtype).cuda(),
                 vd=torch.zeros(6, H, page, 128, dtype=dtype).cuda(), rq=torch.zeros_like(ins["q"]), o=torch.zeros_like(ins["q"]), go=torch.zeros_like(ins["q"]),
                 lse=torch.zeros(B, Hq, L).cuda(), nl=torch.zeros(B, dtype=torch.int32).cuda(), kept=torch.zeros(B, H, budget, dtype=torch.int32).cuda(),
                 wo=torch.zeros(B, H, 3 * page).cuda())

    def step(s):
        rope = dict(pairs=PAIRS, grid=(2, 3), t0=ins["t0"])
        h.rope_axes(ins["q"], None, out=(s["rq"], None), **rope)
        h.paged_append(ins["k"], ins["v"], s["kp"], s["vp"], table, ins["lens"], ins["new"], rope=rope)
        h.paged_attn(s["rq"], s["kp"], s["vp"], table, ins["lens"], ins["new"], out=s["o"], lse=s["lse"], w_in=s["w"], w_out=s["w"], decay=0.5)
        h.gdn_step_raw(s["rq"], s["o"], ins["q"], ins["a"], ins["a"], 1.0, s["S"], lens=ins["new"], out=s["go"])
        h.paged_evict(s["w"], s["kp"], s["vp"], table, ins["lens"], budget, 4, 8, s["kd"], s["vd"], dst, new_lens=s["nl"], kept=s["kept"], w_out=s["wo"])

    mine, one_by_one = ({k: t.clone() for k, t in start.items()} for _ in range(2))
    step({k: t.clone() for k, t in start.items()})
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(mine)
    for i, lens in enumerate(lens_of + lens_of[:1]):
        for n in ("q", "k", "v"):
            ins[n].copy_(rand(*ins[n].shape))
        ins["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        ins["new"].copy_(torch.tensor([L, max(1, L - 3 * i)], dtype=torch.int32))
        g.replay()
        step(one_by_one)
        for n in start:
            assert torch.equal(mine[n], one_by_one[n]), (n, i)
        assert mine["nl"].tolist() == [min(n, budget) for n in lens] and bool(torch.isfinite(mine["go"].float()).all())
    assert h.hlta_device_status() == 0
