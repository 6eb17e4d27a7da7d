"""Refusals of the serving operators' entry points, on the host before anything is enqueued (no
GPU: the pointers are never read)."""
import ctypes

import pytest

F = ctypes.c_float


@pytest.fixture(scope="module")
def h():
    import linear_video_world_b200 as h
    return h


def _p(i):
    return ctypes.c_void_p((1 << 32) * (i + 1))


ODD = ctypes.c_void_p((1 << 40) + 8)


def _refused(h, fn, good, cases, ok_is=None):
    names = list(good)
    for change, status in cases:
        args = dict(good)
        args.update(change)
        assert fn(*[args[n] for n in names]) == status, change


def _spec(h, **kw):
    a = dict(pairs=(22, 21, 21), layout=0, shared=0, gh=2, gw=2, base=1e4, pos=None, t0=None)
    a.update(kw)
    return ctypes.byref(h.hlta_rope_axes_t((ctypes.c_int * 3)(*a["pairs"]), a["layout"], a["shared"], a["gh"], a["gw"], a["base"], a["pos"], a["t0"]))


SPECS = [dict(pairs=(64, 1, 0)), dict(pairs=(-1, 2, 2)), dict(pairs=(65, 0, 0)), dict(layout=2), dict(shared=2), dict(gh=0), dict(gw=-1), dict(base=1.0),
         dict(base=float("nan")), dict(base=float("inf")), dict(pos=1 << 20 | 2), dict(t0=1 << 20 | 1)]


def test_rope_axes(h):
    BAD, ok = h.HLTA_ERR_INVALID_ARG, h.HLTA_OK
    good = dict(q=_p(0), k=_p(1), qo=_p(2), ko=_p(3), B=1, Hq=4, Hk=2, L=10, d=128, spec=_spec(h), inv=0, dt=h.HLTA_BF16, s=None)
    cases = [(dict(spec=_spec(h, **s)), BAD) for s in SPECS]
    cases += [(dict(spec=None), BAD), (dict(qo=None), BAD), (dict(ko=None), BAD), (dict(q=ODD), BAD), (dict(ko=ODD), BAD), (dict(dt=7), BAD),
              (dict(d=129), BAD), (dict(d=0), BAD), (dict(B=-1), BAD), (dict(Hq=-1), BAD), (dict(L=-1), BAD), (dict(L=1 << 31), BAD),
              (dict(qo=_p(1)), BAD), (dict(ko=_p(2)), BAD), (dict(qo=ctypes.c_void_p((1 << 32) + 64)), BAD),
              # nothing to do
              (dict(B=0), ok), (dict(L=0), ok), (dict(q=None, k=None), ok)]
    _refused(h, h._lib.hlta_rope_axes, good, cases)


CACHE = [dict(page=8), dict(page=48), dict(page=256), dict(num_pages=0), dict(num_pages=1 << 31), dict(max_pages=0), dict(max_pages=1 << 27),
         dict(table=None), dict(kv_lens=None), dict(table=ctypes.c_void_p((1 << 33) + 2)), dict(kv_lens=ctypes.c_void_p((1 << 33) + 1))]


def test_paged_append(h):
    BAD, ok = h.HLTA_ERR_INVALID_ARG, h.HLTA_OK
    good = dict(k=_p(0), v=_p(1), kp=_p(2), vp=_p(3), table=_p(4), kv_lens=_p(5), new=None, B=2, H=4, L=3, d=128, num_pages=9, page=16, max_pages=4,
                spec=None, dt=h.HLTA_BF16, s=None)
    cases = [(c, BAD) for c in CACHE] + [(dict(spec=_spec(h, **s)), BAD) for s in SPECS]
    cases += [(dict(k=None), BAD), (dict(v=None), BAD), (dict(kp=None), BAD), (dict(vp=None), BAD), (dict(vp=_p(2)), BAD), (dict(k=ODD), BAD),
              (dict(kp=ODD), BAD), (dict(new=ctypes.c_void_p(1 << 33 | 1)), BAD), (dict(dt=5), BAD), (dict(d=200), BAD), (dict(L=-1), BAD), (dict(B=-1), BAD),
              (dict(B=0), ok), (dict(H=0), ok), (dict(L=0), ok)]
    _refused(h, h._lib.hlta_paged_append, good, cases)


def test_paged_attn(h):
    BAD, NO, ok = h.HLTA_ERR_INVALID_ARG, h.HLTA_ERR_UNSUPPORTED, h.HLTA_OK
    ws = h.hlta_paged_attn_workspace_bytes(2, 8, 4, 3, 128, 16, 4, True)
    assert ws > 0
    good = dict(q=_p(0), kp=_p(1), vp=_p(2), table=_p(3), kv_lens=_p(4), new=None, o=_p(5), lse=None, w_in=_p(6), w_out=_p(7), decay=F(1.0), B=2, Hq=8,
                H=4, L=3, d=128, num_pages=9, page=16, max_pages=4, N=1, w=0, scale=F(0.0), ws=_p(8), wsb=ws, dt=h.HLTA_BF16, s=None)
    cases = [(c, BAD) for c in CACHE if c.get("max_pages") != 1 << 27] + [(dict(max_pages=1 << 27), BAD)]
    cases += [(dict(q=None), BAD), (dict(o=None), BAD), (dict(o=_p(0)), BAD), (dict(q=ODD), BAD), (dict(o=ODD), BAD), (dict(Hq=9), BAD), (dict(Hq=0), BAD),
              (dict(H=0), BAD), (dict(L=-1), BAD), (dict(N=0), BAD), (dict(w=-1), BAD), (dict(w_out=None), BAD), (dict(decay=F(float("nan"))), BAD),
              (dict(decay=F(float("inf"))), BAD), (dict(scale=F(float("inf"))), BAD), (dict(scale=F(float("nan"))), BAD), (dict(w_in=ctypes.c_void_p((1 << 32) * 8 + 16)), BAD), (dict(lse=ctypes.c_void_p(3)), BAD),
              (dict(w_out=ctypes.c_void_p(1 << 34 | 2)), BAD), (dict(new=ctypes.c_void_p(5)), BAD), (dict(ws=None), BAD), (dict(wsb=ws - 1), BAD),
              (dict(ws=ctypes.c_void_p((1 << 40) + 16)), BAD), (dict(dt=3), BAD), (dict(d=64), NO), (dict(d=0), BAD), (dict(Hq=4 * 129), NO),
              (dict(B=0), ok), (dict(L=0, w_in=None, w_out=None), ok)]
    _refused(h, h._lib.hlta_paged_attn_fwd, good, cases)
    big = dict(good, B=70000, H=1, Hq=1, ws=_p(8), wsb=1 << 60)
    # past what a launch can index (the shape is refused before anything is enqueued, if there is a device at all)
    assert h._lib.hlta_paged_attn_fwd(*[dict(big, w_in=None, w_out=None)[n] for n in good]) in (NO, h.HLTA_ERR_CUDA)
    wide = dict(good, B=1, L=1 << 24, page=128, max_pages=1 << 20, num_pages=9, o=ctypes.c_void_p(1 << 50), w_out=ctypes.c_void_p(1 << 51), w_in=None, ws=_p(8), wsb=1 << 60)
    assert h._lib.hlta_paged_attn_fwd(*[wide[n] for n in good]) in (NO, h.HLTA_ERR_CUDA)
    size = h.hlta_paged_attn_workspace_bytes
    assert size(2, 9, 4, 3, 128, 16, 4) == 0 and size(2, 8, 4, 3, 200, 16, 4) == 0 and size(-1, 8, 4, 3, 128, 16, 4) == 0
    assert size(2, 8, 4, 3, 128, 16, 4, False) < ws


def test_paged_evict(h):
    BAD, ok = h.HLTA_ERR_INVALID_ARG, h.HLTA_OK
    ws = h.hlta_paged_evict_workspace_bytes(2, 4, 20)
    assert ws > 0 and h.hlta_paged_evict_workspace_bytes(2, 4, 0) == 0
    good = dict(weights=_p(0), kp=_p(1), vp=_p(2), table=_p(3), kv_lens=_p(4), B=2, H=4, d=128, num_pages=9, page=16, max_pages=4, budget=20, sink=2,
                recent=5, kd=_p(5), vd=_p(6), dt_=_p(7), num_dst=5, max_dst=2, new=_p(8), kept=None, w_out=None, ws=_p(9), wsb=ws, dt=h.HLTA_BF16, s=None)
    cases = [(c, BAD) for c in CACHE]
    cases += [(dict(weights=None), BAD), (dict(new=None), BAD), (dict(new=_p(4)), BAD), (dict(budget=0), BAD), (dict(budget=33), BAD), (dict(sink=-1), BAD),
              (dict(recent=-1), BAD), (dict(sink=16), BAD), (dict(max_dst=1), BAD), (dict(num_dst=0), BAD), (dict(kd=None), BAD), (dict(vd=None), BAD),
              (dict(vd=_p(5)), BAD), (dict(dt_=None), BAD), (dict(kd=ODD), BAD), (dict(w_out=_p(0)), BAD), (dict(kept=ctypes.c_void_p(2)), BAD),
              (dict(ws=None), BAD), (dict(wsb=ws - 1), BAD), (dict(ws=ctypes.c_void_p((1 << 40) + 128)), BAD), (dict(dt=9), BAD), (dict(d=129), BAD),
              (dict(B=0), ok), (dict(H=0), ok), (dict(B=0, kept=_p(10), ws=None, wsb=0), ok), (dict(kept=_p(10), ws=ctypes.c_void_p((1 << 40) + 128)), BAD)]
    _refused(h, h._lib.hlta_paged_evict, good, cases)


def test_gdn_step(h):
    BAD, NO, ok = h.HLTA_ERR_INVALID_ARG, h.HLTA_ERR_UNSUPPORTED, h.HLTA_OK
    good = dict(q=_p(0), k=_p(1), v=_p(2), a=_p(3), b=_p(4), o=_p(5), S=_p(6), So=_p(7), slots=None, lens=None, B=2, H=4, L=3, d=128, num_slots=5,
                dt=h.HLTA_BF16, s=None)
    cases = [({n: None}, BAD) for n in ("q", "k", "v", "a", "b", "o", "S", "So")] + [({n: ODD}, BAD) for n in ("q", "k", "v", "o", "S", "So")]
    cases += [({n: ctypes.c_void_p(1 << 35 | 2)}, BAD) for n in ("a", "b", "slots", "lens")]
    cases += [(dict(B=-1), BAD), (dict(H=-1), BAD), (dict(L=-1), BAD), (dict(num_slots=0), BAD), (dict(num_slots=1), BAD), (dict(d=64), NO), (dict(dt=4), BAD),
              (dict(So=ctypes.c_void_p((1 << 32) * 7 + 64)), BAD), (dict(B=0), ok), (dict(H=0), ok)]
    cases += [(dict(o=good[n]), BAD) for n in ("q", "k", "v")]
    _refused(h, h._lib.hlta_gdn_step, good, cases)
    raw = dict(list(good.items())[:5] + [("c", F(1.0))] + list(good.items())[5:])
    _refused(h, h._lib.hlta_gdn_step_raw, raw, [(dict(c=F(-1.0)), BAD), (dict(c=F(float("nan"))), BAD), (dict(c=F(float("inf"))), BAD), (dict(B=0), ok)])


def test_wrappers_refuse_host_tensors_and_shapes(h):
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 2, 3, 128)
    with pytest.raises(h.HltaError):
        h.rope_axes(q, None, (22, 21, 21), grid=(1, 1))
    with pytest.raises(h.HltaError):
        h.rope_axes(q, torch.zeros(1, 2, 4, 128), (22, 21, 21), grid=(1, 1))
    with pytest.raises(h.HltaError):
        h.rope_axes(None, None, (22, 21, 21), grid=(1, 1))
    for bad in (dict(), dict(grid=(1, 1), pos=torch.zeros(1, 3, 3, dtype=torch.int32)), dict(pos=torch.zeros(1, 3, 3, dtype=torch.int32), t0=torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(h.HltaError):
            h.rope_axes_spec((1, 1, 1), **bad)
    pages, table, lens = torch.zeros(4, 2, 16, 128), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for k in (q, torch.zeros(1, 3, 3, 128)):
        with pytest.raises(h.HltaError):
            h.paged_append(k, k, pages, pages, table, lens)
    with pytest.raises(h.HltaError):
        h.paged_attn(q, pages, pages, table, lens, w_out=torch.zeros(1, 2, 33))
    with pytest.raises(h.HltaError):
        h.gdn_step(q, q, q, torch.zeros(1, 2, 4), torch.zeros(1, 2, 3), torch.zeros(3, 2, 128, 128))


def test_attention_of_too_many_heads_is_refused_before_anything_runs(h):
    """B * Hkv above 65535, few rows and many, with weights and without: refused on the host, where no
    device is asked for."""
    for dt, L, G in ((h.HLTA_BF16, 40, 1), (h.HLTA_BF16, 40, 4), (h.HLTA_BF16, 1, 1), (h.HLTA_FP32, 40, 1), (h.HLTA_FP32, 1, 1)):
        for w_out in (None, ctypes.c_void_p(1 << 52)):
            for B, H, status in ((65536, 1, h.HLTA_ERR_UNSUPPORTED), (256, 256, h.HLTA_ERR_UNSUPPORTED), (70000, 3, h.HLTA_ERR_UNSUPPORTED)):
                assert h._lib.hlta_paged_attn_fwd(ctypes.c_void_p(1 << 48), ctypes.c_void_p(1 << 44), ctypes.c_void_p(1 << 45), _p(3), _p(4), None,
                                                  ctypes.c_void_p(1 << 49), None, None, w_out, F(1.0), B, G * H, H, L, 128, 9, 16, 4, 1, 0, F(0.0),
                                                  ctypes.c_void_p(1 << 53), 1 << 50, dt, None) == status, (dt, L, G, w_out, B)


def test_attention_of_a_huge_pool_or_query_is_refused_before_anything_runs(h):
    """bf16: a pool or a query tensor of 2^31 rows."""
    for L, B, num_pages in ((40, 1, 1 << 27), (1, 1, 1 << 27), (1 << 28, 8, 9)):
        for w_out in (None, ctypes.c_void_p(1 << 53)):
            assert h._lib.hlta_paged_attn_fwd(ctypes.c_void_p(1 << 50), ctypes.c_void_p(1 << 44), ctypes.c_void_p(1 << 45), _p(3), _p(4), None,
                                              ctypes.c_void_p(1 << 51), None, None, w_out, F(1.0), B, 1, 1, L, 128, num_pages, 16, 4, 1, 0, F(0.0),
                                              ctypes.c_void_p(1 << 54), 1 << 60, h.HLTA_BF16, None) == h.HLTA_ERR_UNSUPPORTED, (L, B, num_pages, w_out)


def _at(p, off):
    return ctypes.c_void_p(p.value + off)


def test_append_over_its_own_inputs_is_refused(h):
    """The pool may not hold the chunk, the tables or the positions, nor the keys' pages the values'."""
    good = dict(k=_p(0), v=_p(1), kp=_p(2), vp=_p(3), table=_p(4), kv_lens=_p(5), new=None, B=2, H=4, L=3, d=128, num_pages=9, page=16, max_pages=4,
                spec=None, dt=h.HLTA_BF16, s=None)
    pool, chunk = 9 * 4 * 16 * 128 * 2, 2 * 4 * 3 * 128 * 2
    bad = [dict(vp=_at(_p(2), pool - 16)), dict(vp=_at(_p(2), 16 - pool)), dict(k=_at(_p(2), pool - 16)), dict(k=_at(_p(3), 16 - chunk)), dict(v=_at(_p(2), 256)),
           dict(v=_at(_p(3), 0)), dict(table=_at(_p(2), pool - 4)), dict(kv_lens=_at(_p(3), 4)), dict(new=_at(_p(3), 128)),
           dict(spec=_spec(h, pos=_p(3).value + pool - 4)), dict(spec=_spec(h, t0=_p(2).value))]
    _refused(h, h._lib.hlta_paged_append, good, [(c, h.HLTA_ERR_INVALID_ARG) for c in bad])


def test_attention_whose_outputs_overlap_other_tensors_is_refused(h):
    ws = h.hlta_paged_attn_workspace_bytes(2, 8, 4, 3, 128, 16, 4, True)
    good = dict(q=_p(0), kp=_p(1), vp=_p(2), table=_p(3), kv_lens=_p(4), new=None, o=_p(5), lse=None, w_in=_p(6), w_out=_p(7), decay=F(1.0), B=2, Hq=8,
                H=4, L=3, d=128, num_pages=9, page=16, max_pages=4, N=1, w=0, scale=F(0.0), ws=_p(8), wsb=ws, dt=h.HLTA_BF16, s=None)
    pool, rows, nw = 9 * 4 * 16 * 128 * 2, 2 * 8 * 3, 2 * 4 * 64 * 4
    bad = [dict(o=_at(_p(1), pool - 16)), dict(o=_at(_p(2), 16 - rows * 256)), dict(o=_at(_p(7), nw - 16)), dict(o=_at(_p(6), 0)), dict(o=_at(_p(8), 64)),
           dict(lse=_at(_p(5), 4)), dict(lse=_at(_p(0), rows * 256 - 4)), dict(lse=_at(_p(7), nw - 4)), dict(lse=_at(_p(6), 0)), dict(lse=_at(_p(8), ws - 256)), dict(lse=_at(_p(4), 4)),
           dict(w_out=_at(_p(1), 0)), dict(w_out=_at(_p(3), 28)), dict(w_out=_at(_p(0), 8)), dict(w_in=_p(8)),
           dict(ws=_p(0)), dict(ws=_at(_p(2), 256)), dict(ws=_p(3)), dict(ws=_p(5)), dict(ws=_p(7)), dict(new=_at(_p(8), 256)), dict(new=_at(_p(5), 4))]
    _refused(h, h._lib.hlta_paged_attn_fwd, good, [(c, h.HLTA_ERR_INVALID_ARG) for c in bad])


def test_eviction_whose_outputs_overlap_other_tensors_is_refused(h):
    ws = h.hlta_paged_evict_workspace_bytes(2, 4, 20)
    good = dict(weights=_p(0), kp=_p(1), vp=_p(2), table=_p(3), kv_lens=_p(4), B=2, H=4, d=128, num_pages=9, page=16, max_pages=4, budget=20, sink=2,
                recent=5, kd=_p(5), vd=_p(6), dt_=_p(7), num_dst=5, max_dst=2, new=_p(8), kept=None, w_out=None, ws=_p(9), wsb=ws, dt=h.HLTA_BF16, s=None)
    pool, dst, nw, no, nk = 9 * 4 * 16 * 128 * 2, 5 * 4 * 16 * 128 * 2, 2 * 4 * 64 * 4, 2 * 4 * 32 * 4, 2 * 4 * 20 * 4
    bad = [dict(vd=_at(_p(5), dst - 16)), dict(kd=_at(_p(0), nw - 16)), dict(vd=_at(_p(3), 16)), dict(kd=_at(_p(7), 0)), dict(new=_at(_p(4), 4)), dict(new=_at(_p(3), 28)),
           dict(new=_at(_p(0), 0)), dict(new=_at(_p(5), 8)), dict(kept=_at(_p(0), nw - 4)), dict(kept=_at(_p(1), 0)), dict(kept=_at(_p(8), 4 - nk)), dict(kept=_at(_p(7), 12)),
           dict(w_out=_at(_p(2), pool - 4)), dict(w_out=_at(_p(0), 4 - no)), dict(w_out=_p(9)), dict(w_out=_p(10), kept=_at(_p(10), no - 4)), dict(ws=_p(0)), dict(ws=_p(4)),
           dict(ws=_p(8)), dict(ws=_at(_p(6), 256))]
    _refused(h, h._lib.hlta_paged_evict, good, [(c, h.HLTA_ERR_INVALID_ARG) for c in bad])


def test_gated_delta_step_whose_outputs_overlap_other_tensors_is_refused(h):
    good = dict(q=_p(0), k=_p(1), v=_p(2), a=_p(3), b=_p(4), o=_p(5), S=_p(6), So=_p(7), slots=None, lens=None, B=2, H=4, L=3, d=128, num_slots=5,
                dt=h.HLTA_BF16, s=None)
    states, rows = 5 * 4 * 128 * 128 * 4, 2 * 4 * 3
    bad = [dict(o=_at(_p(3), 16)), dict(o=_at(_p(4), 16 - rows * 256)), dict(o=_at(_p(6), states - 16)), dict(o=_at(_p(7), 0)), dict(So=_at(_p(0), 16)), dict(So=_at(_p(2), 16 - states)),
           dict(So=_p(3)), dict(So=_p(5)), dict(slots=_at(_p(7), 8)), dict(lens=_at(_p(5), 4)), dict(S=_p(7), slots=_at(_p(7), states - 4))]
    _refused(h, h._lib.hlta_gdn_step, good, [(c, h.HLTA_ERR_INVALID_ARG) for c in bad])


def test_rotation_whose_outputs_overlap_the_positions_is_refused(h):
    good = dict(q=_p(0), k=_p(1), qo=_p(2), ko=_p(3), B=1, Hq=4, Hk=2, L=10, d=128, spec=_spec(h), inv=0, dt=h.HLTA_BF16, s=None)
    bad = [dict(spec=_spec(h, pos=_p(2).value + 4 * 10 * 256 - 4)), dict(spec=_spec(h, pos=_p(3).value - 116)), dict(spec=_spec(h, t0=_p(2).value)),
           dict(qo=_p(0), spec=_spec(h, t0=_p(0).value + 16)), dict(q=None, spec=_spec(h, pos=_p(3).value))]
    _refused(h, h._lib.hlta_rope_axes, good, [(c, h.HLTA_ERR_INVALID_ARG) for c in bad])
