"""Cases for measuring the serving operators beside the streaming cache: rotary positions over
several axes, append to and attention over a paged cache, eviction by accumulated attention
weight, and the gated delta rule's recurrent step over a pool of states.

`run` computes a case in plain torch operations, or through the framework's entry points when
`own` is set; `exact` gives the same outputs in 64 bits from the definitions.
"""
import math

import numpy as np
import torch

own = False

D = 128                    # head dim of every bf16 case (the framework's)
BASE = 10000.0


# ---- cases ---------------------------------------------------------------------------------

def _rope(name, **kw):
    c = dict(op="rope", name=name, dtype="bf16", B=1, Hq=16, Hk=16, L=1560, d=D, pt=22, ph=21, pw=21,
             halves=False, shared=False, gh=30, gw=52, explicit=False, inverse=False)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(op="append", name=name, dtype="bf16", B=8, H=8, L=1560, d=D, page=64, hist_min=0, hist_max=20280,
             ragged=False, pt=22, ph=21, pw=21, halves=False, shared=False, gh=30, gw=52, explicit=False)
    c.update(kw)
    return c


def _attn(name, **kw):
    c = dict(op="attn", name=name, dtype="bf16", B=1, Hq=8, Hkv=8, L=1, d=D, page=64, kv_min=1560, kv_max=1560,
             ragged=False, N=1, w=0, lse=False, weights=False)
    c.update(kw)
    return c


def _evict(name, **kw):
    c = dict(op="evict", name=name, dtype="bf16", B=1, H=8, d=D, page=64, n_min=2000, n_max=2000, budget=1024,
             sink=16, recent=256)
    c.update(kw)
    return c


def _gdn(name, **kw):
    c = dict(op="gdn", name=name, dtype="bf16", B=1, H=8, L=1, d=D, ragged=False, raw=False)
    c.update(kw)
    return c


def listed():
    return [
        # the 16 softmax heads of a 21-frame 480P clip (30 x 52 latent grid), q and k, one prologue call
        _rope("rope_clip", L=32760),
        # gradient map of fewer key heads at scattered positions (cropped or packed images), single precision
        _rope("rope_scattered_grad", dtype="fp32", B=3, Hq=8, Hk=2, L=777, pt=16, ph=24, pw=24, halves=True,
              shared=True, explicit=True, inverse=True),
        # one new 480P frame for each of eight rollouts of different ages
        _append("append_frame"),
        # one token for each rollout of a small batch: launch latency
        _append("append_token", B=16, L=1, hist_min=5, hist_max=9000, page=16, explicit=True),
        # the smallest call: one token of one rollout over one frame of history
        _attn("token_one", kv_min=1560, kv_max=1560, page=16),
        # tokens of a ragged batch, three query heads a key head, weights kept for eviction
        _attn("token_batch", B=32, Hq=24, kv_min=37, kv_max=32760, weights=True),
        # a new frame of each rollout over the whole history, up to a 480P clip
        _attn("frame_history", B=4, L=1560, N=1560, kv_min=7800, kv_max=32760, lse=True),
        # ragged token chunks in a sliding window, shared key heads, weights kept for eviction
        _attn("chunk_window", B=3, Hq=16, Hkv=4, L=517, kv_min=517, kv_max=9001, ragged=True, w=4096, page=32,
              lse=True, weights=True),
        # one young rollout cut to a small budget, single precision
        _evict("evict_one", dtype="fp32", H=4, n_min=1001, n_max=1001, budget=256, sink=4, recent=64, page=16),
        # eight rollouts of about a clip each cut to a quarter
        _evict("evict_rollouts", B=8, n_min=20000, n_max=32760, budget=8192, sink=64, recent=1560),
        # one token of one rollout, raw projections
        _gdn("gdn_token", raw=True),
        # a full batch of rollouts, up to four tokens each
        _gdn("gdn_batch", B=256, L=4, ragged=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "evict", "gdn"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    page = rng.choice([16, 32, 64, 128])
    pt, ph, pw = rng.choice([(22, 21, 21), (16, 24, 24), (8, 16, 16), (64, 0, 0), (0, 32, 32)])
    shape = dict(pt=pt, ph=ph, pw=pw, halves=rng.random() < 0.4, shared=rng.random() < 0.4, explicit=rng.random() < 0.5,
                 gh=rng.randint(1, 45), gw=rng.randint(1, 80))
    if op == "rope":
        Hq = rng.choice([1, 2, 4, 8, 16])
        c = _rope("", dtype=dtype, B=rng.randint(1, 4), Hq=Hq, Hk=rng.choice([h for h in (1, 2, 4, 8, 16) if h <= Hq]),
                  L=_log(rng, 1, 8000), inverse=rng.random() < 0.5, **shape)
    elif op == "append":
        lo = rng.randint(0, 3000)
        c = _append("", dtype=dtype, B=_log(rng, 1, 32), H=rng.choice([1, 2, 4, 8]), L=_log(rng, 1, 1560), page=page,
                    hist_min=lo, hist_max=lo + _log(rng, 1, 6000), ragged=rng.random() < 0.5, **shape)
    elif op == "attn":
        H, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        L = rng.choice([1, 1, 2, 4]) if rng.random() < 0.5 else _log(rng, 5, 1600)
        small = dtype == "fp32"
        L = min(L, 200) if small else L
        N = rng.choice([1, L, max(1, L // 3)])
        kv = _log(rng, 40, 3000 if small else 24000)
        B = _log(rng, 1, 4 if L > 64 else 24)
        kv = max(40, min(kv, 500_000_000 // (B * L * H * G)))
        c = _attn("", dtype=dtype, B=B, Hq=H * G, Hkv=H, L=L, page=page,
                  kv_min=L + kv // 7, kv_max=L + kv, ragged=rng.random() < 0.5, N=N,
                  w=rng.choice([0, 0, max(1, kv // (2 * N)), 3]), lse=rng.random() < 0.5, weights=rng.random() < 0.5)
    elif op == "evict":
        n = _log(rng, 30, 12000)
        budget = max(8, int(n * rng.uniform(0.1, 0.9)))
        c = _evict("", dtype=dtype, B=_log(rng, 1, 6), H=rng.choice([1, 2, 4, 8]), page=page, n_min=max(1, n // 3), n_max=n,
                   budget=budget, sink=rng.randint(0, budget // 4), recent=rng.randint(0, budget // 2))
    else:
        c = _gdn("", dtype=dtype, B=_log(rng, 1, 200), H=rng.choice([1, 3, 8]), L=_log(rng, 1, 8), ragged=rng.random() < 0.5,
                 raw=rng.random() < 0.5)
    del c["name"]
    return c


# ---- what a program has in hand --------------------------------------------------------------

def _type(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _size(c):
    return 2 if c["dtype"] == "bf16" else 4


def _spread(lo, hi, n):
    """n lengths from hi down to lo, in an order that mixes them."""
    v = [hi if n == 1 else hi - (hi - lo) * i // (n - 1) for i in range(n)]
    return v[::2] + v[1::2][::-1]


def _new_tokens(c):
    """Tokens of the chunk that each rollout really has."""
    return [max(1, c["L"] - i * c["L"] // (2 * c["B"])) for i in range(c["B"])] if c["ragged"] else [c["L"]] * c["B"]


def _ints(v, device="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=device)


def _table(lens, page, spare, gen):
    """A block table whose pages are scattered over the pool (-1: none), and the pool's pages."""
    need = [max(1, -(-n // page)) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=gen)[:sum(need)].tolist()
    width, rows = max(need), []
    for n in need:
        rows.append(order[:n] + [-1] * (width - n))
        order = order[n:]
    return _ints(rows), sum(need) + spare


def _positions(c, gen):
    if not c["explicit"]:
        return None
    hi = torch.tensor([c.get("hist_max", 20000) + c["L"], c["gh"], c["gw"]], dtype=torch.float64)
    u = torch.rand((c["B"], c["L"], 3), generator=gen, device="cuda", dtype=torch.float64)
    return (u * hi.cuda()).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    dt = _type(c)
    s = {"case": c}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    if c["op"] == "rope":
        s["q"], s["k"] = normal(c["B"], c["Hq"], c["L"], c["d"]), normal(c["B"], c["Hk"], c["L"], c["d"])
        s["pos"] = _positions(c, gen)
        s["t0"] = None if c["explicit"] else _ints([7 * b for b in range(c["B"])])
    elif c["op"] == "append":
        s["k"], s["v"] = normal(c["B"], c["H"], c["L"], c["d"]), normal(c["B"], c["H"], c["L"], c["d"])
        new = _new_tokens(c)
        lens = [h + n for h, n in zip(_spread(c["hist_min"], c["hist_max"], c["B"]), new)]
        s["table"], pages = _table(lens, c["page"], 3, host)
        s["new_lens"], s["kv_lens"] = _ints(new), _ints(lens)
        s["pos"] = _positions(c, gen)
        s["t0"] = None if c["explicit"] else _ints([5 * b for b in range(c["B"])])
        s["k_pages"] = torch.zeros((pages, c["H"], c["page"], c["d"]), dtype=dt, device="cuda")
        s["v_pages"] = torch.zeros_like(s["k_pages"])
    elif c["op"] == "attn":
        s["q"] = normal(c["B"], c["Hq"], c["L"], c["d"])
        lens, new = _spread(c["kv_min"], c["kv_max"], c["B"]), _new_tokens(c)
        s["table"], pages = _table(lens, c["page"], 3, host)
        s["q_lens"], s["kv_lens"] = _ints(new), _ints(lens)
        s["k_pages"], s["v_pages"] = (normal(pages, c["Hkv"], c["page"], c["d"]) for _ in range(2))
        # outputs keep what they hold behind a rollout's last row or key
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(s["q"].shape[:3], device="cuda") if c["lse"] else None
        if c["weights"]:
            cap = s["table"].shape[1] * c["page"]
            s["w_in"] = 4.0 * uniform(c["B"], c["Hkv"], cap) ** 4
            s["w_out"] = torch.zeros_like(s["w_in"])
    elif c["op"] == "evict":
        lens = _spread(c["n_min"], c["n_max"], c["B"])
        s["table"], pages = _table(lens, c["page"], 3, host)
        s["dst_table"], dst_pages = _table([min(n, c["budget"]) for n in lens], c["page"], 1, host)
        width = -(-c["budget"] // c["page"])
        s["dst_table"] = torch.nn.functional.pad(s["dst_table"], (0, width - s["dst_table"].shape[1]), value=-1)
        s["kv_lens"] = _ints(lens)
        s["k_pages"], s["v_pages"] = (normal(pages, c["H"], c["page"], c["d"]) for _ in range(2))
        # most of the weight on few keys, many keys never attended (equal weights)
        u = uniform(c["B"], c["H"], s["table"].shape[1] * c["page"])
        s["weights"] = torch.where(u < 0.1, torch.zeros_like(u), 4.0 * u ** 6)
        s["k_dst"], s["v_dst"] = (torch.zeros((dst_pages, c["H"], c["page"], c["d"]), dtype=dt, device="cuda") for _ in range(2))
        s["new_lens"] = torch.zeros(c["B"], dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros((c["B"], c["H"], c["budget"]), dtype=torch.int32, device="cuda")
        s["w_out"] = torch.zeros((c["B"], c["H"], width * c["page"]), device="cuda")
    else:
        B, H, L, d = c["B"], c["H"], c["L"], c["d"]
        q, k, s["v"] = (torch.randn((B, H, L, d), generator=gen, device="cuda") for _ in range(3))
        x, y = (torch.randn((B, H, L), generator=gen, device="cuda") for _ in range(2))
        if c["raw"]:
            s["a"], s["b"] = x, y
        else:
            q, k = (t * torch.rsqrt((t * t).sum(-1, keepdim=True)) for t in (q, k))
            s["a"], s["b"] = torch.exp(-torch.log1p(torch.exp(x))), torch.sigmoid(y)
        s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), s["v"].to(dt)
        slots = B + 2
        s["S"] = 0.1 * torch.randn((slots, H, d, d), generator=gen, device="cuda")
        s["S_out"] = torch.zeros_like(s["S"])
        s["slots"] = torch.randperm(slots, generator=host)[:B].to(torch.int32).cuda()
        s["lens"] = _ints(_new_tokens(c))
        s["o"] = torch.zeros_like(s["q"])
    return s


# ---- plain forms -------------------------------------------------------------------------------

def _rotate(x, c, pos, t0, inverse=False):
    """Rotation of the pairs of x [B, H, L, d] in 32 bits; the angles in 64 (far positions)."""
    B, _, L, d = x.shape
    n = torch.tensor([c["pt"], c["ph"], c["pw"]], device=x.device)
    P = c["pt"] + c["ph"] + c["pw"]
    if pos is None:
        i = torch.arange(L, device=x.device)
        plane = c["gh"] * c["gw"]
        at = torch.stack([i // plane, i % plane // c["gw"], i % c["gw"]], -1).expand(B, L, 3).clone()
        at[..., 0] += t0[:, None]
    else:
        at = pos
    axis = torch.repeat_interleave(torch.arange(3, device=x.device), n, output_size=P)
    j = torch.arange(P, device=x.device)
    first = torch.cumsum(n, 0) - n
    power = j.double() / P if c["shared"] else (j - first[axis]).double() / n[axis]
    ang = at.double()[..., axis] * torch.exp(power * -math.log(BASE))
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    sin = -sin if inverse else sin
    f = x.float()
    if c["halves"]:
        u, v = f[..., :P], f[..., P:2 * P]
        y = torch.cat([u * cos - v * sin, u * sin + v * cos, f[..., 2 * P:]], -1)
    else:
        u, v = f[..., 0:2 * P:2], f[..., 1:2 * P:2]
        y = torch.cat([torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2), f[..., 2 * P:]], -1)
    return y.to(x.dtype)


def _gather(pages, table):
    """[B, H, capacity, d] of a paged tensor [pages, H, page, d] (page 0 where there is none)."""
    t = pages[table.clamp(min=0).long()]
    return t.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_append(s):
    c = s["case"]
    k = _rotate(s["k"], c, s["pos"], s["t0"])
    i = torch.arange(c["L"], device="cuda")
    live = i < s["new_lens"][:, None]
    at = ((s["kv_lens"] - s["new_lens"])[:, None] + i).clamp(min=0, max=s["table"].shape[1] * c["page"] - 1).long()
    page = s["table"].gather(1, at // c["page"])[live].long()
    slot = (at % c["page"])[live]
    s["k_pages"][page, :, slot] = k.transpose(1, 2)[live]
    s["v_pages"][page, :, slot] = s["v"].transpose(1, 2)[live]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attn(s):
    c = s["case"]
    B, H, L, N, G = c["B"], c["Hkv"], c["L"], c["N"], c["Hq"] // c["Hkv"]
    k, v = _gather(s["k_pages"], s["table"]).float(), _gather(s["v_pages"], s["table"]).float()
    cap = k.shape[2]
    i = torch.arange(L, device="cuda")
    j = torch.arange(cap, device="cuda")
    hist = (s["kv_lens"] - s["q_lens"])[:, None]
    frame = i // N
    hi = torch.minimum(hist + (frame + 1) * N, s["kv_lens"][:, None])
    lo = hist + (frame - c["w"] + 1) * N if c["w"] else torch.zeros_like(hi)
    live = i < s["q_lens"][:, None]
    seen = (j < hi[..., None]) & (j >= lo[..., None]) & live[..., None]
    v = torch.where((j < s["kv_lens"][:, None])[:, None, :, None], v, 0.0)
    x = torch.matmul(s["q"].float().view(B, H, G * L, c["d"]), k.transpose(2, 3)) / math.sqrt(c["d"])
    x = x.view(B, H, G, L, cap).masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, G * L, cap), v).view(B, H, G, L, c["d"]) / torch.where(total > 0, total, 1.0)
    s["o"].copy_(o.view(B, c["Hq"], L, c["d"]))
    out = {"o": s["o"]}
    if c["lse"]:
        lse = (m + torch.log(total)).view(B, c["Hq"], L)
        s["lse"].copy_(torch.where(live[:, None], lse, 0.0))
        out["lse"] = s["lse"]
    if c["weights"]:
        got = (p / torch.where(total > 0, total, 1.0)).sum((2, 3))
        old = torch.where((j < hist)[:, None], s["w_in"], 0.0)
        s["w_out"].copy_(torch.where((j < s["kv_lens"][:, None])[:, None], 0.95 * old + got, 0.0))
        out["weights"] = s["w_out"]
    return out


def _plain_evict(s):
    c = s["case"]
    B, H, cap = s["weights"].shape
    n = s["kv_lens"][:, None, None].long()
    new = n.clamp(max=c["budget"])
    j = torch.arange(cap, device="cuda").expand(B, H, cap)
    rank = torch.where((j < c["sink"]) | (j >= n - c["recent"]), math.inf, s["weights"])
    rank = torch.where(j < n, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :c["budget"]]
    i = torch.arange(order.shape[-1], device="cuda")
    kept = torch.sort(torch.where(i < new, order, cap), dim=-1).values
    full = torch.full((B, H, c["budget"]), cap, device="cuda")
    full[..., :kept.shape[-1]] = kept
    live = full < cap
    at = torch.where(live, full, 0)
    i = torch.arange(c["budget"], device="cuda")
    b, h, r = torch.where(live)
    src = at[live]
    page, slot = s["table"][b, src // c["page"]].long(), src % c["page"]
    dpage, dslot = s["dst_table"][b, i[r] // c["page"]].long(), i[r] % c["page"]
    s["k_dst"][dpage, h, dslot] = s["k_pages"][page, h, slot]
    s["v_dst"][dpage, h, dslot] = s["v_pages"][page, h, slot]
    s["kept"].copy_(torch.where(live, full, -1))
    s["new_lens"].copy_(new[:, 0, 0])
    s["w_out"][..., :c["budget"]] = torch.where(live, s["weights"].gather(2, at), 0.0)
    return {k: s[k] for k in ("k_dst", "v_dst", "kept", "new_lens", "w_out")}


def _plain_gdn(s):
    c = s["case"]
    q, k, v, a, b = (s[n].float() for n in ("q", "k", "v", "a", "b"))
    if c["raw"]:
        q, k = (t * torch.rsqrt((t * t).sum(-1, keepdim=True)) for t in (q, k))
        a, b = torch.exp(-(torch.relu(a) + torch.log1p(torch.exp(-a.abs())))), torch.sigmoid(b)
    at = s["slots"].long()
    S = s["S"][at]
    for t in range(c["L"]):                 # the recurrence itself
        live = (t < s["lens"])[:, None, None, None]
        kt, bt = k[:, :, t], b[:, :, t, None, None]
        u = v[:, :, t] - a[:, :, t, None] * torch.matmul(S, kt[..., None])[..., 0]
        S = torch.where(live, a[:, :, t, None, None] * S + bt * u[..., None] * kt[..., None, :], S)
        o = torch.matmul(S, q[:, :, t, :, None])[..., 0]
        s["o"][:, :, t] = torch.where(live[..., 0], o, 0.0).to(s["o"].dtype)
    s["S_out"][at] = S
    return {"o": s["o"], "S": s["S_out"]}


def run(state):
    s, c = state, state["case"]
    if own:
        import linear_video_world_b200 as h
        if c["op"] in ("rope", "append"):
            spec = dict(pairs=(c["pt"], c["ph"], c["pw"]), grid=None if c["explicit"] else (c["gh"], c["gw"]), pos=s["pos"], t0=s["t0"],
                        base=BASE, halves=c["halves"], shared_freq=c["shared"])
            if c["op"] == "rope":
                q, k = h.rope_axes(s["q"], s["k"], inverse=c["inverse"], **spec)
                return {"q": q, "k": k}
            h.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"], s["new_lens"], rope=spec)
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if c["op"] == "attn":
            h.paged_attn(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"], s["q_lens"], N=c["N"], w=c["w"],
                         out=s["o"], lse=s["lse"], w_in=s.get("w_in"), w_out=s.get("w_out"), decay=0.95)
            out = {"o": s["o"]}
            if c["lse"]:
                out["lse"] = s["lse"]
            if c["weights"]:
                out["weights"] = s["w_out"]
            return out
        if c["op"] == "evict":
            h.paged_evict(s["weights"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"], c["budget"], c["sink"],
                          c["recent"], s["k_dst"], s["v_dst"], s["dst_table"], new_lens=s["new_lens"], kept=s["kept"],
                          w_out=s["w_out"])
            return {k: s[k] for k in ("k_dst", "v_dst", "kept", "new_lens", "w_out")}
        if c["raw"]:
            h.gdn_step_raw(s["q"], s["k"], s["v"], s["a"], s["b"], 1.0, s["S"], slots=s["slots"], lens=s["lens"],
                           out=s["o"], S_out=s["S_out"])
        else:
            h.gdn_step(s["q"], s["k"], s["v"], s["a"], s["b"], s["S"], slots=s["slots"], lens=s["lens"], out=s["o"],
                       S_out=s["S_out"])
        return {"o": s["o"], "S": s["S_out"]}
    if c["op"] == "rope":
        return {"q": _rotate(s["q"], c, s["pos"], s["t0"], c["inverse"]), "k": _rotate(s["k"], c, s["pos"], s["t0"], c["inverse"])}
    return {"append": _plain_append, "attn": _plain_attn, "evict": _plain_evict, "gdn": _plain_gdn}[c["op"]](s)


# ---- what a pass has to move and compute -------------------------------------------------------

def work(case):
    c, e = case, _size(case)
    if c["op"] == "rope":
        n = c["B"] * (c["Hq"] + c["Hk"]) * c["L"] * c["d"]
        return {"bytes": 2 * e * n + (12 * c["B"] * c["L"] if c["explicit"] else 4 * c["B"]), "flops": 3 * n}
    if c["op"] == "append":
        n = sum(_new_tokens(c)) * c["H"] * c["d"]
        return {"bytes": 4 * e * n + (12 * sum(_new_tokens(c)) if c["explicit"] else 4 * c["B"]), "flops": 3 * n}
    if c["op"] == "attn":
        pairs = keys = 0
        for kv, n in zip(_spread(c["kv_min"], c["kv_max"], c["B"]), _new_tokens(c)):
            f = np.arange(n) // c["N"]
            hi = np.minimum(kv - n + (f + 1) * c["N"], kv)
            lo = np.maximum(kv - n + (f - c["w"] + 1) * c["N"], 0) if c["w"] else 0 * hi
            pairs += int((hi - lo).sum())
            keys += int(hi.max() - lo.min())
        rows = sum(_new_tokens(c)) * c["Hq"]
        bytes_ = 2 * e * rows * c["d"] + 2 * e * keys * c["Hkv"] * c["d"] + (4 * rows if c["lse"] else 0)
        if c["weights"]:
            bytes_ += 8 * c["Hkv"] * sum(_spread(c["kv_min"], c["kv_max"], c["B"]))
        return {"bytes": bytes_, "flops": 4 * c["d"] * pairs * c["Hq"]}
    if c["op"] == "evict":
        lens = _spread(c["n_min"], c["n_max"], c["B"])
        kept = sum(min(n, c["budget"]) for n in lens) * c["H"]
        return {"bytes": 4 * sum(lens) * c["H"] + 4 * e * kept * c["d"] + 4 * kept + 4 * c["B"] * c["H"] * c["budget"],
                "flops": sum(lens) * c["H"]}
    toks = sum(_new_tokens(c)) * c["H"]
    return {"bytes": 8 * c["B"] * c["H"] * c["d"] ** 2 + 4 * e * toks * c["d"] + 8 * toks, "flops": 8 * toks * c["d"] ** 2}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _exact_turn(x, c, pos, t0, sign):
    """x's pairs as complex numbers, each times exp(i angle)."""
    B, H, L, d = x.shape
    n = [c["pt"], c["ph"], c["pw"]]
    P = sum(n)
    ang = np.zeros((B, L, P))
    j = 0
    for a in range(3):
        for i in range(n[a]):
            freq = BASE ** -((j / P) if c["shared"] else (i / n[a]))
            if pos is not None:
                p = pos[:, :, a].astype(np.float64)
            else:
                l = np.arange(L)
                p = [l // (c["gh"] * c["gw"]), (l // c["gw"]) % c["gh"], l % c["gw"]][a][None].astype(np.float64)
                p = p + t0[:, None] if a == 0 else np.broadcast_to(p, (B, L))
            ang[:, :, j] = p * freq
            j += 1
    turn = torch.from_numpy(np.exp(1j * sign * ang)).cuda()[:, None]
    y = x.double().clone()
    if c["halves"]:
        z = torch.complex(y[..., :P], y[..., P:2 * P]) * turn
        y[..., :P], y[..., P:2 * P] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:2 * P:2], y[..., 1:2 * P:2]) * turn
        y[..., 0:2 * P:2], y[..., 1:2 * P:2] = z.real, z.imag
    return y


def _exact_attn(s, c):
    G, N, page = c["Hq"] // c["Hkv"], c["N"], c["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device="cuda")
    wo = torch.zeros((c["B"], c["Hkv"], s["table"].shape[1] * page), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        kv, n = int(s["kv_lens"][b]), int(s["q_lens"][b])
        pages = s["table"][b, :-(-kv // page)].long()
        i = torch.arange(n, device="cuda")
        j = torch.arange(kv, device="cuda")
        f, jf = i // N, torch.where(j < kv - n, torch.div(j - (kv - n), N, rounding_mode="floor"), (j - (kv - n)) // N)
        seen = jf[None] <= f[:, None]
        if c["w"]:
            seen &= jf[None] > f[:, None] - c["w"]
        for h in range(c["Hkv"]):
            K = s["k_pages"][pages, h].reshape(-1, c["d"])[:kv].double()
            V = s["v_pages"][pages, h].reshape(-1, c["d"])[:kv].double()
            for g in range(h * G, h * G + G):
                x = s["q"][b, g, :n].double() @ K.T * c["d"] ** -0.5
                x = x.masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, 1)
                p = torch.exp(x - z[:, None])
                o[b, g, :n], lse[b, g, :n] = p @ V, z
                wo[b, h, :kv] += p.sum(0)
        if c["weights"]:
            wo[b, :, :kv - n] += 0.95 * s["w_in"][b, :, :kv - n].double()
    out = {"o": o}
    if c["lse"]:
        out["lse"] = lse
    if c["weights"]:
        out["weights"] = wo
    return out


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    pos = s["pos"].cpu().numpy() if s.get("pos") is not None else None
    t0 = s["t0"].cpu().numpy() if s.get("t0") is not None else None
    if c["op"] == "rope":
        sign = -1 if c["inverse"] else 1
        return {"q": _exact_turn(s["q"], c, pos, t0, sign), "k": _exact_turn(s["k"], c, pos, t0, sign)}
    if c["op"] == "append":
        k, v = _exact_turn(s["k"], c, pos, t0, 1), s["v"].double()
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        table = s["table"].cpu().numpy()
        for b, (n, kv) in enumerate(zip(s["new_lens"].tolist(), s["kv_lens"].tolist())):
            at = np.arange(kv - n, kv)
            pg, sl = torch.from_numpy(table[b, at // c["page"]]).long().cuda(), torch.from_numpy(at % c["page"]).cuda()
            kp[pg, :, sl], vp[pg, :, sl] = k[b, :, :n].transpose(0, 1), v[b, :, :n].transpose(0, 1)
        return {"k_pages": kp, "v_pages": vp}
    if c["op"] == "attn":
        return _exact_attn(s, c)
    if c["op"] == "evict":
        kd, vd, wo = s["k_dst"].double(), s["v_dst"].double(), s["w_out"].double()
        kept = np.full(s["kept"].shape, -1, dtype=np.int32)
        w, table, dst = s["weights"].cpu().numpy(), s["table"].cpu().numpy(), s["dst_table"].cpu().numpy()
        lens = s["kv_lens"].tolist()
        for b, n in enumerate(lens):
            for h in range(c["H"]):
                if n <= c["budget"]:
                    idx = np.arange(n)
                else:
                    mid = np.arange(c["sink"], n - c["recent"])
                    best = np.lexsort((mid, -w[b, h, mid]))[:c["budget"] - c["sink"] - c["recent"]]
                    idx = np.concatenate([np.arange(c["sink"]), np.sort(mid[best]), np.arange(n - c["recent"], n)])
                kept[b, h, :len(idx)] = idx
                r = np.arange(len(idx))
                at = [torch.from_numpy(x).long().cuda() for x in (table[b, idx // c["page"]], idx % c["page"], dst[b, r // c["page"]], r % c["page"])]
                kd[at[2], h, at[3]] = s["k_pages"][at[0], h, at[1]].double()
                vd[at[2], h, at[3]] = s["v_pages"][at[0], h, at[1]].double()
                wo[b, h, :len(idx)] = s["weights"][b, h, torch.from_numpy(idx).cuda()].double()
        return {"k_dst": kd, "v_dst": vd, "kept": torch.from_numpy(kept),
                "new_lens": torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32), "w_out": wo}
    q, k, v, a, b = (s[n].double() for n in ("q", "k", "v", "a", "b"))
    if c["raw"]:
        q, k = (t / torch.linalg.vector_norm(t, dim=-1, keepdim=True) for t in (q, k))
        a, b = torch.exp(-torch.nn.functional.softplus(a)), torch.sigmoid(b)
    o, S_out = s["o"].double(), s["S_out"].double()
    eye = torch.eye(c["d"], dtype=torch.float64, device="cuda")
    for r, (slot, n) in enumerate(zip(s["slots"].tolist(), s["lens"].tolist())):
        S = s["S"][slot].double()
        for t in range(n):
            kt, vt = k[r, :, t], v[r, :, t]
            bt = b[r, :, t, None, None]
            S = a[r, :, t, None, None] * S @ (eye - bt * kt[:, :, None] * kt[:, None, :]) + bt * vt[:, :, None] * kt[:, None, :]
            o[r, :, t] = torch.einsum("hij,hj->hi", S, q[r, :, t])
        S_out[slot] = S
    return {"o": o, "S": S_out}
