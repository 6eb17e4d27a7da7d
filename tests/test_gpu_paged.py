"""GPU parity of the paged cache's append and attention against the 64-bit forms (serving_util;
slots that no rollout holds are NaN there, table entries behind a rollout's pages out of range)."""
import math

import pytest
import torch

from serving_util import Cache, attn_ref, grid_positions, rope_bound, rope_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def h():
    import linear_video_world_b200 as h
    assert torch.cuda.is_available()
    return h


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


# ---- append ---------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,d,page", [(BF, 128, 16), (BF, 128, 128), (F32, 128, 32), (F32, 33, 64), (BF, 12, 16)])
@pytest.mark.parametrize("rotate", [None, "pairs", "halves"])
def test_append(h, dtype, d, page, rotate):
    B, H, L = 4, 3, 21
    new = [21, 1, 0, 20]                    # padded, one token, none
    kv = [21, 130, 40, page + 20]           # from empty; across pages; untouched; into the second page
    c = Cache(kv, H, d, page, dtype)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(B, H, L, d, generator=g).to(dtype) for _ in range(2))
    pairs = (2, 1, 2)
    t0 = _i32([0, 9, 3, 5])
    spec = None if rotate is None else dict(pairs=pairs, grid=(2, 3), t0=t0.cuda(), halves=rotate == "halves")
    kp, vp, table, lens = c.cuda()
    h.paged_append(k.cuda(), v.cuda(), kp, vp, table, lens, _i32(new).cuda(), rope=spec)
    assert h.hlta_device_status() == 0
    ref, bound = k.double(), torch.zeros_like(k).double()
    if rotate:
        ref = rope_ref(k, pairs, grid_positions(B, L, (2, 3), t0), halves=rotate == "halves")
        bound = rope_bound(k, ref, pairs, rotate == "halves")
    kp, vp, kw, vw = kp.cpu(), vp.cpu(), c.k.clone(), c.v.clone()
    for b in range(B):
        for i in range(new[b]):
            p = kv[b] - new[b] + i
            pg, s = int(c.table[b, p // page]), p % page
            assert bool(((kp[pg, :, s].double() - ref[b, :, i]).abs() <= bound[b, :, i]).all())
            assert torch.equal(vp[pg, :, s], v[b, :, i])
            kw[pg, :, s], vw[pg, :, s] = kp[pg, :, s], vp[pg, :, s]
    # every other slot as it was
    assert torch.equal(kp.nan_to_num(7.5), kw.nan_to_num(7.5)) and torch.equal(vp.nan_to_num(7.5), vw.nan_to_num(7.5))


def test_append_far_page(h):
    """A pool of more than 2^31 elements: slots behind that offset."""
    pages, H, page, d = 17000, 8, 128, 128
    kp, vp = (torch.empty((pages, H, page, d), dtype=BF, device="cuda") for _ in range(2))
    assert kp.numel() > 2 ** 31
    table, lens = _i32([[pages - 1, 3]]).cuda(), _i32([130]).cuda()
    k, v = (torch.randn(1, H, 4, d, device="cuda").to(BF) for _ in range(2))
    kp[pages - 1, :, :126], vp[pages - 1, :, :126] = 0.0, 1.0
    h.paged_append(k, v, kp, vp, table, lens)
    assert torch.equal(kp[pages - 1, :, 126:], k[0, :, :2]) and torch.equal(kp[3, :, :2], k[0, :, 2:])
    assert torch.equal(vp[pages - 1, :, 126:], v[0, :, :2]) and torch.equal(vp[3, :, :2], v[0, :, 2:])
    # queries of zero weigh every position alike: the mean of the values
    o = h.paged_attn(torch.zeros(1, H, 4, d, device="cuda", dtype=BF), kp, vp, table, lens, N=4)
    mean = (126 + v[0].double().sum(1)) / 130
    assert h.hlta_device_status() == 0
    # weights 1/130 round at most by half a step each, the output once
    assert bool(((o[0, :, 0].double() - mean).abs() <= 2.0 ** -8 * (126 + v[0].double().abs().sum(1)) / 130 + 2.0 ** -8 * mean.abs()).all())
    del kp, vp
    torch.cuda.empty_cache()


# ---- attention ------------------------------------------------------------------------------

# B rollouts of kv tokens, `new` of them in the chunk of up to L; heads, frame size, window, page
CASES = [
    dict(kv=[1], new=[1], Hq=1, Hkv=1, L=1, N=1, w=0, page=16),                          # the smallest
    dict(kv=[129, 1, 0, 64, 63, 65], new=[1, 1, 0, 1, 1, 1], Hq=4, Hkv=2, L=1, N=1, w=0, page=16),
    dict(kv=[700, 17], new=[1, 1], Hq=6, Hkv=2, L=1, N=1, w=100, page=32),               # one token, window
    dict(kv=[300, 40], new=[4, 3], Hq=8, Hkv=2, L=4, N=1, w=0, page=64),                 # drafted tokens, 16 rows
    dict(kv=[300, 40, 7], new=[5, 2, 5], Hq=9, Hkv=3, L=5, N=5, w=2, page=16),           # 15 rows, frames
    dict(kv=[257, 128], new=[17, 1], Hq=2, Hkv=2, L=17, N=1, w=0, page=128),             # 17 rows
    dict(kv=[200, 130, 127], new=[130, 130, 127], Hq=2, Hkv=1, L=130, N=1, w=0, page=32),  # chunk longer than history
    dict(kv=[333, 150], new=[150, 97], Hq=3, Hkv=3, L=150, N=50, w=0, page=16),          # frames, ragged last
    dict(kv=[500, 260], new=[150, 150], Hq=2, Hkv=2, L=150, N=50, w=2, page=64),         # frame window inside tiles
    dict(kv=[420], new=[270], Hq=2, Hkv=2, L=270, N=1, w=33, page=128),                  # short window, several row tiles
    dict(kv=[600, 300], new=[40, 33], Hq=16, Hkv=2, L=40, N=1, w=0, page=32),            # 320 packed rows of 8 heads
    dict(kv=[900, 300, 700], new=[150, 150, 149], Hq=8, Hkv=4, L=150, N=50, w=0, page=64),   # twelve heads of two row tiles, cut
    dict(kv=[900, 300, 700], new=[270, 100, 1], Hq=16, Hkv=16, L=270, N=90, w=0, page=64),   # more tiles than blocks take at least
]


def _run(h, c, q, new, cfg, lse=True, weights=True, decay=0.5):
    B, Hq, L, d = q.shape
    kp, vp, table, lens = c.cuda()
    cap = table.shape[1] * c.page
    o = torch.full_like(q, 77.0).cuda()
    ls = torch.full((B, Hq, L), 55.0, device="cuda") if lse else None
    w_in = torch.rand((B, cfg["Hkv"], cap), generator=torch.Generator().manual_seed(8)) if weights else None
    w_out = torch.full((B, cfg["Hkv"], cap), 33.0, device="cuda") if weights else None
    # what lies at and behind the chunk in w_in is never read
    if weights:
        for b in range(B):
            w_in[b, :, c.kv[b] - new[b]:] = float("nan")
    h.paged_attn(q.cuda(), kp, vp, table, lens, _i32(new).cuda(), N=cfg["N"], w=cfg["w"], out=o, lse=ls, w_in=w_in.cuda() if weights else None,
                 w_out=w_out, decay=decay)
    assert h.hlta_device_status() == 0
    return o.cpu(), None if ls is None else ls.cpu(), w_in, None if w_out is None else w_out.cpu()


@pytest.mark.parametrize("dtype,d", [(F32, 128), (F32, 40), (F32, 7), (BF, 128)])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(h, i, dtype, d):
    _against_64_bits(h, i, dtype, d, None)


@pytest.mark.parametrize("dtype,d", [(F32, 128), (F32, 30), (BF, 128)])
@pytest.mark.parametrize("i", [1, 4, 6, 8, 9, 10])
def test_attention_in_a_wide_table(h, i, dtype, d):
    """A table of far more pages than the rollouts have: the capacity decides about tiles and blocks."""
    _against_64_bits(h, i, dtype, d, 30000 // CASES[i]["page"])


def _against_64_bits(h, i, dtype, d, width):
    cfg = CASES[i]
    kv, new, L = cfg["kv"], cfg["new"], cfg["L"]
    c = Cache(kv, cfg["Hkv"], d, cfg["page"], dtype, seed=i, width=width)
    q = torch.randn(len(kv), cfg["Hq"], L, d, generator=torch.Generator().manual_seed(100 + i)).to(dtype)
    for b, n in enumerate(new):
        q[b, :, n:] = float("nan")          # padded rows hold anything
        if cfg["w"]:                        # so do slots before the window
            c.poison(b, 0, max(0, kv[b] - n - (cfg["w"] - 1) * cfg["N"]))
    o, lse, w_in, w_out = _run(h, c, q, new, cfg)
    ro, rl, rw, ob, lb, wb = attn_ref(q, c, new, cfg["N"], cfg["w"], w_in, 0.5)
    for b, n in enumerate(new):
        assert bool((o[b, :, n:] == 77).all()) and bool((lse[b, :, n:] == 55).all())
        assert bool((w_out[b, :, kv[b]:] == 33).all())
        e = (o[b, :, :n].double() - ro[b, :, :n]).abs()
        assert bool((e <= ob[b, :, :n]).all()), (b, float((e / ob[b, :, :n]).max()))
        e = (lse[b, :, :n].double() - rl[b, :, :n]).abs()
        assert bool((e <= lb[b, :, :n]).all()), (b, float((e / lb[b, :, :n]).max()))
        e = (w_out[b, :, :kv[b]].double() - rw[b, :, :kv[b]]).abs()
        assert bool((e <= wb[b, :, :kv[b]] + 1e-37).all()), (b, float(e.max()))
    # the same call again: the same bits; without lse and weights: the same output
    o2, lse2, _, w2 = _run(h, c, q, new, cfg)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(w_out, w2)
    o3, _, _, _ = _run(h, c, q, new, cfg, lse=False, weights=False)
    assert torch.equal(o, o3)


@pytest.mark.parametrize("L,Hq", [(1, 2), (20, 2), (300, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_unseen_keys_never_leak(h, dtype, L, Hq):
    """Keys that a row does not see but other rows of the chunk do hold values of 1e4 there: any
    weight on them, 2^-24 of the sum even, would show."""
    kv, N, w = 420, 3, 20
    c = Cache([kv], 1, 128, 16, dtype, seed=3)
    q = torch.randn(1, Hq, L, 128, generator=torch.Generator().manual_seed(1)).to(dtype)
    base = _run(h, c, q, [L], dict(Hkv=1, N=N, w=w), weights=False)[0]
    h0 = kv - L
    for i in sorted({0, L // 2, L - 1}):
        lo, hi = max(0, h0 + (i // N - w + 1) * N), min(kv, h0 + (i // N + 1) * N)
        d = Cache([kv], 1, 128, 16, dtype, seed=3)
        for a, b in ((0, lo), (hi, kv)):
            for p in range(a, b):
                d.v[int(d.table[0, p // 16]), :, p % 16] = 1e4
        got = _run(h, d, q, [L], dict(Hkv=1, N=N, w=w), weights=False)[0]
        rows = [j for j in range(L) if max(0, h0 + (j // N - w + 1) * N) >= lo and min(kv, h0 + (j // N + 1) * N) <= hi]
        assert i in rows and torch.equal(got[:, :, rows], base[:, :, rows])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [1, 40])
def test_large_scores_and_infinities(h, dtype, L):
    """Scores of +-1e3: one key takes all the weight. An infinite value reaches the row that sees it."""
    c = Cache([200], 1, 128, 32, dtype, seed=5)
    q = (torch.randn(1, 2, L, 128, generator=torch.Generator().manual_seed(2)) * 100).to(dtype)
    o, lse, _, w = _run(h, c, q, [L], dict(Hkv=1, N=1, w=0))
    ro, rl, _, ob, lb, _ = attn_ref(q, c, [L], 1, 0, None, 0.5)
    assert bool(torch.isfinite(o.double()).all())
    # scores this far apart decide by their largest: compare where the winner is clear of the bound
    for g in range(2):
        for i in range(L):
            x = torch.sort(c.keys[0][0, :200 - L + i + 1].double() @ q[0, g, i].double() * 128 ** -0.5, descending=True).values
            if float(x[0] - x[1]) > 40:
                assert bool(((o[0, g, i].double() - ro[0, g, i]).abs() <= 2.0 ** -8 * ro[0, g, i].abs() + 1e-15).all())
                assert abs(float(lse[0, g, i]) - float(rl[0, g, i])) <= float(lb[0, g, i])
    pg, s = int(c.table[0, 199 // 32]), 199 % 32
    c.v[pg, :, s] = float("inf")
    o, _, _, _ = _run(h, c, q / 100, [L], dict(Hkv=1, N=1, w=0), weights=False)
    assert not bool(torch.isfinite(o[0, :, L - 1].double()).any())


def test_scale_and_shared_pages(h):
    """Two rollouts that share their first pages; a softmax scale of one's own."""
    c = Cache([100, 90], 2, 128, 32, BF, seed=6)
    c.table[1, :2] = c.table[0, :2]
    c.keys[1][:, :64], c.vals[1][:, :64] = c.keys[0][:, :64], c.vals[0][:, :64]
    q = torch.randn(2, 2, 5, 128, generator=torch.Generator().manual_seed(7)).to(BF)
    kp, vp, table, lens = c.cuda()
    o = h.paged_attn(q.cuda(), kp, vp, table, lens, scale=0.3).cpu()
    ro, _, _, ob, _, _ = attn_ref(q, c, [5, 5], 1, 0, scale=0.3)
    assert bool(((o.double() - ro).abs() <= ob).all())


def test_against_window_attention(h):
    """A clip appended frame by frame equals hlta_swa_fwd over the clip: the same keys in the same
    order of tiles but for their borders, so within two roundings of P and two of the output."""
    T, N, w, H = 4, 70, 3, 2
    q, k, v = (torch.randn(1, H, T * N, 128, generator=torch.Generator().manual_seed(s)).to(BF).cuda() for s in (1, 2, 3))
    ref = h.swa(q, k, v, T, N, w)
    page, width = 64, 5
    kp, vp = (torch.full((width, H, page, 128), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    table = torch.arange(width, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    for f in range(T):
        s = slice(f * N, (f + 1) * N)
        lens = _i32([(f + 1) * N]).cuda()
        h.paged_append(k[:, :, s].contiguous(), v[:, :, s].contiguous(), kp, vp, table, lens)
        o = h.paged_attn(q[:, :, s].contiguous(), kp, vp, table, lens, N=N, w=w)
        assert float((o - ref[:, :, s]).abs().max()) <= 4 * 2.0 ** -8 * float(v.abs().max())
    assert h.hlta_device_status() == 0


def test_accumulating_in_place(h):
    """w_in = w_out: one buffer over several chunks; every row adds weights of sum one."""
    c = Cache([150, 80], 2, 128, 16, BF, seed=9)
    kp, vp, table, lens = c.cuda()
    w = torch.zeros((2, 2, table.shape[1] * 16), device="cuda")
    q = torch.randn(2, 6, 7, 128, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    for step in range(3):
        h.paged_attn(q, kp, vp, table, lens, w_in=w, w_out=w)
    for b, n in enumerate(c.kv):
        # rows 7, heads 3 a group; the chunk's own positions start over at every call
        total = w[b, :, :n].double().sum(-1).cpu()
        own = w[b, :, n - 7:n].double().sum(-1).cpu()
        assert bool(((total - own) <= 3 * 21 * (1 + 1e-4)).all())
        assert bool(((total - own) / 3 + own - 21).abs().max() <= 21 * 1e-4)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [1, 40])
def test_tables_out_of_range_are_reported(h, dtype, L):
    c = Cache([100, 90], 1, 128, 16, dtype, seed=2)
    q = torch.randn(2, 1, L, 128, generator=torch.Generator().manual_seed(7)).to(dtype).cuda()
    good = h.paged_attn(q, *c.cuda(), w=0)
    for what in ("page", "neg", "long", "minus", "short"):
        kp, vp, table, lens = c.cuda()
        kp, vp = kp.nan_to_num(0.0), vp.nan_to_num(0.0)
        if what == "page":
            table[0, 2] = kp.shape[0]
        elif what == "neg":
            table[0, 3] = -1
        elif what == "long":
            lens[0] = table.shape[1] * 16 + 1
        elif what == "minus":
            lens[0] = -5
        else:
            lens[0] = L - 1                 # fewer tokens cached than new
        if what == "long":
            table[0] = table[0].clamp(0, kp.shape[0] - 1)
        o = h.paged_attn(q, kp, vp, table, lens)
        st, word = h.hlta_device_status_code()
        assert st == h.HLTA_ERR_INVALID_ARG and word == h.HLTA_DEVERR_TABLE, what
        assert torch.equal(o[1], good[1]), what           # the other rollout's rows
        if what in ("minus", "short") and L == 1:
            assert bool((o[0] == 0).all())                # a row that sees nothing
        k, v = (torch.randn(2, 1, L, 128, device="cuda").to(dtype) for _ in range(2))
        before = kp.clone()
        if what in ("page", "neg"):
            lens[0] = 64                                  # the chunk's last tokens fall on the bad page
        h.paged_append(k, v, kp, vp, table, lens)
        st, word = h.hlta_device_status_code()
        assert st == h.HLTA_ERR_INVALID_ARG or what == "page", what
        pages = set(int(x) for x in c.table.flatten().tolist() if x >= 0)
        for pg in range(kp.shape[0]):
            if pg not in pages and what != "long":
                assert torch.equal(kp[pg], before[pg]), what
    assert h.hlta_device_status() == 0


@pytest.mark.parametrize("L,Hq", [(1, 8), (3, 4), (200, 4)])
def test_captured_and_replayed_with_new_lengths(h, L, Hq):
    """One captured call replayed for other lengths, on a side stream; a second graph that shares
    its workspace, replayed after it, changes nothing."""
    sizes = [[40 + L, 300], [500, L], [130 + L, 129 + L]]
    big = Cache([max(s[b] for s in sizes) for b in range(2)], 4, 128, 32, BF, seed=4)
    kp, vp, table, _ = big.cuda()
    lens = _i32(sizes[0]).cuda()
    q = torch.randn(2, Hq, L, 128, generator=torch.Generator().manual_seed(7)).to(BF).cuda()
    w_out, lse = torch.zeros(2, 4, table.shape[1] * 32, device="cuda"), torch.zeros(2, Hq, L, device="cuda")
    out, out2 = torch.zeros_like(q), torch.zeros_like(q)
    ws = torch.empty(h.hlta_paged_attn_workspace_bytes(2, Hq, 4, L, 128, 32, table.shape[1], True), dtype=torch.uint8, device="cuda")
    call = lambda o, x: h.paged_attn(x, kp, vp, table, lens, out=o, lse=lse, w_out=w_out, workspace=ws)   # noqa: E731
    call(out, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for o, x in ((out, q), (out2, q.flip(1).contiguous())):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(o, x)
        graphs.append((g, x))
    for s in sizes + sizes[:1]:
        lens.copy_(_i32(s))
        torch.cuda.synchronize()
        graphs[0][0].replay()
        graphs[1][0].replay()
        torch.cuda.synchronize()
        want = h.paged_attn(q, kp, vp, table, lens)
        assert torch.equal(out, want)
        want2 = h.paged_attn(graphs[1][1], kp, vp, table, lens)
        assert torch.equal(out2, want2)
    assert h.hlta_device_status() == 0


def test_two_streams_at_once(h):
    """Two calls of different rollouts on two streams, each with its own workspace."""
    cs = [Cache([700, 90], 2, 128, 64, BF, seed=s) for s in (1, 2)]
    qs = [torch.randn(2, 4, n, 128, generator=torch.Generator().manual_seed(n)).to(BF).cuda() for n in (1, 90)]
    dev = [c.cuda() for c in cs]
    want = [h.paged_attn(q, *d) for q, d in zip(qs, dev)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(h.paged_attn(qs[i], *dev[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o, want[i])


def test_many_rollouts_and_empty_batch(h):
    """More rollouts than threads of a block, lengths from one on; a batch of none."""
    B = 700
    kv = [1 + (37 * b) % 50 for b in range(B)]
    c = Cache(kv, 1, 128, 16, BF, seed=1)
    q = torch.randn(B, 1, 1, 128, generator=torch.Generator().manual_seed(7)).to(BF)
    kp, vp, table, lens = c.cuda()
    w = torch.zeros(B, 1, table.shape[1] * 16, device="cuda")
    o = h.paged_attn(q.cuda(), kp, vp, table, lens, w_out=w).cpu()
    ro, _, rw, ob, _, wb = attn_ref(q, c, [1] * B, 1, 0)
    assert bool(((o.double() - ro).abs() <= ob).all())
    assert bool(((w.cpu().double() - rw).abs() <= wb + 1e-37).all())
    e = h.paged_attn(q[:0].cuda(), kp, vp, table[:0], lens[:0])
    assert e.shape[0] == 0 and h.hlta_device_status() == 0


def test_no_new_token_decays_the_weights(h):
    c = Cache([50, 20], 2, 128, 16, BF, seed=1)
    kp, vp, table, lens = c.cuda()
    w = torch.rand(2, 2, table.shape[1] * 16, generator=torch.Generator().manual_seed(1))
    out = torch.full_like(w, 9.0).cuda()
    for q, new in ((torch.zeros(2, 4, 0, 128), None), (torch.zeros(2, 4, 3, 128), _i32([0, 0]).cuda())):
        o = torch.full_like(q.to(BF), 3.0).cuda()
        h.paged_attn(q.to(BF).cuda(), kp, vp, table, lens, new, out=o, w_in=w.cuda(), w_out=out, decay=0.25)
        assert h.hlta_device_status() == 0 and bool((o == 3).all())
        for b, n in enumerate(c.kv):
            assert torch.equal(out[b, :, :n].cpu(), 0.25 * w[b, :, :n]) and bool((out[b, :, n:] == 9).all())


def test_error_bound_would_show_a_lost_key():
    """The bounds used above are far below what one wrong key does (fp32, 64 keys)."""
    c = Cache([64], 1, 40, 16, F32, seed=1)
    q = torch.randn(1, 1, 1, 40, generator=torch.Generator().manual_seed(7))
    ro, _, _, ob, _, _ = attn_ref(q, c, [1], 1, 0)
    for drop in range(64):
        keep = [j for j in range(64) if j != drop]
        p = torch.softmax(c.keys[0][0, keep].double() @ q[0, 0, 0].double() / math.sqrt(40), 0)
        assert float(((p @ c.vals[0][0, keep].double() - ro[0, 0, 0]).abs() / ob[0, 0, 0]).max()) > 5


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weights_of_few_rows_over_a_huge_capacity(h, dtype):
    """Rows x capacity past what single tokens keep scores for: the weights then come from a second
    pass over the keys, the same within both paths' bounds."""
    page, kv = 128, 300
    c = Cache([kv], 1, 128, page, dtype, seed=4)
    q = torch.randn(1, 16, 1, 128, generator=torch.Generator().manual_seed(3)).to(dtype)
    kp, vp, table, lens = c.cuda()
    wide = torch.full((1, (1 << 24) // page + 64), -3, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    ro, _, rw, ob, _, wb = attn_ref(q, c, [1], 1, 0)
    for t in (table, wide):
        cap = t.shape[1] * page
        assert (h.hlta_paged_attn_workspace_bytes(1, 16, 1, 1, 128, page, t.shape[1], True, h._dt(q)) < 1 << 30) or t is table
        w = torch.full((1, 1, cap), 5.0, device="cuda")
        o = h.paged_attn(q.cuda(), kp, vp, t, lens, w_out=w).cpu()
        assert bool(((o.double() - ro).abs() <= ob).all())
        assert bool(((w[..., :kv].cpu().double() - rw[..., :kv]).abs() <= wb[..., :kv]).all())
        assert bool((w[..., kv:] == 5).all())
    assert h.hlta_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L,Hq", [(1, 2), (3, 4), (40, 4)])
def test_pages_before_the_window_may_be_gone(h, dtype, L, Hq):
    """The window starts inside a tile of keys: the pages before it, same tile or not, are no longer
    in the table."""
    kv, w, page = [331, 90], 70, 16
    c = Cache(kv, 2, 128, page, dtype, seed=L)
    for b, n in enumerate(kv):
        c.table[b, :max(0, n - L - w + 1) // page] = -1
    q = torch.randn(2, Hq, L, 128, generator=torch.Generator().manual_seed(3)).to(dtype)
    kp, vp, table, lens = c.cuda()
    wo = torch.zeros((2, 2, table.shape[1] * page), device="cuda")
    o = h.paged_attn(q.cuda(), kp, vp, table, lens, N=1, w=w, w_out=wo)
    assert h.hlta_device_status() == 0
    ro, _, rw, ob, _, wb = attn_ref(q, c, [L, L], 1, w)
    assert bool(((o.cpu().double() - ro).abs() <= ob).all())
    for b, n in enumerate(kv):
        assert bool(((wo[b, :, :n].cpu().double() - rw[b, :, :n]).abs() <= wb[b, :, :n]).all())


def test_append_of_tensors_side_by_side(h):
    """Chunk, pages and tables one behind the other in one buffer: nothing overlaps."""
    H, page, L, pages = 2, 16, 3, 4
    pool, chunk = pages * H * page * 128, H * L * 128
    buf = torch.zeros(2 * pool + 2 * chunk + 64, dtype=BF, device="cuda")
    k, kp, v, vp = (t.view(shape) for t, shape in zip(buf[:-64].split([chunk, pool, chunk, pool]),
                                                     ((1, H, L, 128), (pages, H, page, 128), (1, H, L, 128), (pages, H, page, 128))))
    tail = buf[-64:].view(torch.int32)
    table, lens = tail[:pages].view(1, pages), tail[pages:pages + 1]
    table.copy_(_i32([[2, 0, 3, 1]]))
    lens.copy_(_i32([18]))
    k.copy_(torch.randn(k.shape, generator=torch.Generator().manual_seed(1)))
    v.copy_(torch.randn(v.shape, generator=torch.Generator().manual_seed(2)))
    h.paged_append(k, v, kp, vp, table, lens)
    for x, p in ((k, kp), (v, vp)):
        assert torch.equal(p[2, :, 15], x[0, :, 0]) and torch.equal(p[0, :, :2], x[0, :, 1:])
    assert h.hlta_device_status() == 0
