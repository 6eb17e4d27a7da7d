"""PagedCache's host side on the CPU: lengths, pages, tables and weights, with plain stand-ins for the
three paged calls (what they compute is tested on the GPU)."""
import pytest
import torch

BF = torch.bfloat16


class _OnTheHost:
    """torch, with what is asked for on the GPU made on the CPU."""

    def __getattr__(self, name):
        return getattr(torch, name)

    def zeros(self, *a, device=None, **kw):
        return torch.zeros(*a, **kw)

    def empty(self, *a, device=None, **kw):
        return torch.empty(*a, **kw)


@pytest.fixture
def h(monkeypatch):
    import linear_video_world_b200 as h

    def append(k, v, k_pages, v_pages, table, kv_lens, new_lens=None, rope=None, stream=None):
        if k.dtype != k_pages.dtype:
            raise h.HltaError(h.HLTA_ERR_INVALID_ARG, "dtype")
        assert bool((new_lens <= kv_lens).all())

    def attn(q, k_pages, v_pages, table, kv_lens, new_lens=None, N=1, w=0, scale=0.0, out=None, lse=None, w_in=None, w_out=None, decay=1.0, **kw):
        # every live row gives each position of the rollout a weight of one
        for b, (kv, n) in enumerate(zip(kv_lens.tolist(), new_lens.tolist())):
            assert 0 <= n <= kv
            if w_out is not None:
                old = decay * w_in[b, :, :kv - n]
                w_out[b, :, kv - n:kv] = float(n)
                w_out[b, :, :kv - n] = old + float(n)
        return q

    def evict(weights, k_pages, v_pages, table, kv_lens, budget, sink, recent, k_dst, v_dst, dst_table, w_out=None, **kw):
        assert w_out.shape == (table.shape[0], weights.shape[1], dst_table.shape[1] * k_dst.shape[2])
        for b, n in enumerate(kv_lens.tolist()):
            for g in range(weights.shape[1]):
                mid = sorted(range(sink, n - recent), key=lambda i: (-float(weights[b, g, i]), i))[:max(0, budget - sink - recent)]
                keep = list(range(n)) if n <= budget else list(range(sink)) + sorted(mid) + list(range(n - recent, n))
                w_out[b, g, :len(keep)] = weights[b, g, keep]

    monkeypatch.setattr(h, "_th", lambda: _OnTheHost())
    monkeypatch.setattr(torch.Tensor, "cuda", lambda self, *a, **kw: self)
    for name, f in (("paged_append", append), ("paged_attn", attn), ("paged_evict", evict)):
        monkeypatch.setattr(h, name, f)
    return h


def _tokens(B, n):
    return torch.zeros(B, 2, n, 128, dtype=BF)


@pytest.mark.parametrize("emptied_by", ["release", "evict"])
def test_weights_of_an_earlier_occupant_are_gone(h, emptied_by):
    """Positions that a released or cut rollout had start without weight, however many chunks are
    appended before the next is attended."""
    c = h.PagedCache(2, 2, 128, 20, 64, page=16, weights=True, decay=0.5)
    c.append(_tokens(2, 40), _tokens(2, 40), [40, 30])
    c.attend(_tokens(2, 40))
    kept = 0
    if emptied_by == "release":
        c.release(0)
    else:
        kept = 8
        assert c.evict(kept) == [0, 1]
        c.release(1)
        c.append(_tokens(2, 30), _tokens(2, 30), [0, 30])
    for n in (10, 7):
        c.append(_tokens(2, n), _tokens(2, n), [n, 0])
    assert bool((c.weights[0, :, kept:] == 0).all())
    c.attend(_tokens(2, 7))
    assert bool((c.weights[0, :, :kept] == 0.5 * 40 + 7).all()) and bool((c.weights[0, :, kept:kept + 17] == 7).all())


def test_refused_append_leaves_the_last_chunk(h):
    c = h.PagedCache(2, 2, 128, 8, 64, page=16)
    c.append(_tokens(2, 20), _tokens(2, 20), [20, 3])
    state = list(c.lens), [list(p) for p in c._pages], sorted(c._free), c.table.clone(), c.kv_lens.clone(), c.new_lens.clone()
    assert c.new_lens.tolist() == [20, 3]
    with pytest.raises(h.HltaError):
        c.append(_tokens(2, 20).float(), _tokens(2, 20).float(), [1, 20])
    assert (c.lens, c._pages, sorted(c._free)) == state[:3]
    for t, u in zip((c.table, c.kv_lens, c.new_lens), state[3:]):
        assert torch.equal(t, u)
    c.attend(_tokens(2, 20))
    # a rollout that was released since the chunk stays so
    c.release(1)
    with pytest.raises(h.HltaError):
        c.append(_tokens(2, 20).float(), _tokens(2, 20).float(), [1, 20])
    assert c.new_lens.tolist() == [20, 0] and c.kv_lens.tolist() == [20, 0]
    # so does one whose tables cannot be copied
    tables, failed = c._tables, []

    def once(pages):
        if not failed:
            failed.append(pages)
            raise RuntimeError("no copy")
        tables(pages)
    c._tables = once
    with pytest.raises(RuntimeError):
        c.append(_tokens(2, 20), _tokens(2, 20))
    assert c.lens == [20, 0] and len(c._free) == 6 and c.new_lens.tolist() == [20, 0]
    c.append(_tokens(2, 20), _tokens(2, 20))
    assert c.lens == [40, 20] and c.new_lens.tolist() == [20, 20] and c.kv_lens.tolist() == [40, 20]


def test_the_cache_s_tensors_stay_the_same(h):
    """A captured attend reads and writes the tensors that the cache had then: no call puts others in
    their place."""
    c = h.PagedCache(2, 2, 128, 20, 64, page=16, weights=True)
    names = ("k_pages", "v_pages", "table", "kv_lens", "new_lens", "weights")
    at = [getattr(c, n).data_ptr() for n in names]
    c.append(_tokens(2, 20), _tokens(2, 20), [20, 7])
    c.attend(_tokens(2, 20))
    assert c.evict(8) == [0]
    assert bool((c.weights[0, :, :8] == 20).all()) and bool((c.weights[1, :, :7] == 7).all()) and bool((c.weights[0, :, 8:] == 0).all())
    c.release(1)
    c.append(_tokens(2, 3), _tokens(2, 3))
    assert [getattr(c, n).data_ptr() for n in names] == at
