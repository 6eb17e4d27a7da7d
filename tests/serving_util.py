"""Plain 64-bit forms of the serving operators and error bounds for them (CPU, small sizes)."""
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}    # half a step, relative


def rope_ref(x, pairs, at, base=10000.0, halves=False, shared=False, inverse=False):
    """x [B, H, L, d], at [B, L, 3]: pairs as complex numbers times exp(i angle)."""
    P = sum(pairs)
    ang = torch.zeros(at.shape[:2] + (P,), dtype=torch.float64)
    j = 0
    for a, n in enumerate(pairs):
        for i in range(n):
            ang[..., j] = at[..., a].double() * base ** -(j / P if shared else i / n)
            j += 1
    z = torch.polar(torch.ones_like(ang), -ang if inverse else ang)[:, None]
    y = x.double().clone()
    if halves:
        w = torch.complex(y[..., :P], y[..., P:2 * P]) * z
        y[..., :P], y[..., P:2 * P] = w.real, w.imag
    else:
        w = torch.complex(y[..., 0:2 * P:2], y[..., 1:2 * P:2]) * z
        y[..., 0:2 * P:2], y[..., 1:2 * P:2] = w.real, w.imag
    return y


def rope_bound(x, ref, pairs, halves):
    """One rounding to the type, plus in fp32: the reduced turn's rounding (2^-26 turns of 2 pi),
    two units in the last place of sine and cosine, three roundings of products and sums."""
    P = sum(pairs)
    s = x.double().abs()
    if halves:
        t = s[..., :P] + s[..., P:2 * P]
        m = torch.cat([t, t, torch.zeros_like(s[..., 2 * P:])], -1)
    else:
        t = s[..., 0:2 * P:2] + s[..., 1:2 * P:2]
        m = torch.cat([torch.repeat_interleave(t, 2, -1), torch.zeros_like(s[..., 2 * P:])], -1)
    f32 = (2 * math.pi * 2.0 ** -26 + 2 * 2.0 ** -23 + 3 * 2.0 ** -24) * m
    half = EPS[x.dtype] if x.dtype == torch.bfloat16 else 0.0
    return half * (ref.abs() + f32) + f32


def grid_positions(B, L, grid, t0=None):
    l = torch.arange(L)
    at = torch.stack([l // (grid[0] * grid[1]), l // grid[1] % grid[0], l % grid[1]], -1).expand(B, L, 3).clone()
    if t0 is not None:
        at[..., 0] += t0[:, None]
    return at


class Cache:
    """A paged cache on the CPU with the rollouts' keys and values scattered over its pages. Slots
    that no rollout holds are NaN, table entries behind a rollout's pages out of range."""

    def __init__(self, kv, H, d, page, dtype, seed=0, spare=2, width=None, share=None):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.page = kv, page
        need = [-(-n // page) for n in kv]
        width = width or max(1, max(need))
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        self.k, self.v = (torch.full((pages, H, page, d), float("nan")).to(dtype) for _ in range(2))
        self.table = torch.full((len(kv), width), -7, dtype=torch.int32)
        self.keys, self.vals = [], []
        for b, n in enumerate(kv):
            K, V = (torch.randn(H, n, d, generator=g).to(dtype) for _ in range(2))
            for i in range(need[b]):
                pg = order.pop()
                self.table[b, i] = pg
                m = min(page, n - i * page)
                self.k[pg, :, :m] = K[:, i * page:i * page + m]
                self.v[pg, :, :m] = V[:, i * page:i * page + m]
            self.keys.append(K)
            self.vals.append(V)
        self.lens = torch.tensor(kv, dtype=torch.int32)

    def poison(self, b, lo, hi, value=float("nan")):
        """Overwrites positions [lo, hi) of rollout b in the pages (not in the reference)."""
        for p in range(lo, hi):
            pg = int(self.table[b, p // self.page])
            self.k[pg, :, p % self.page] = value
            self.v[pg, :, p % self.page] = value

    def cuda(self):
        return self.k.cuda(), self.v.cuda(), self.table.cuda(), self.lens.cuda()


def attn_ref(q, cache, new, N, w, w_in=None, decay=1.0, scale=None):
    """Per rollout and head: o, lse, weights and their error bounds, in 64 bits.

    Bounds, with u = 2^-24 (fp32) or 2^-23 (bf16, whose tensor-core sums may truncate): a score of d
    products is off by at most (d + 8) u sum |q k| scale (sum, scale, base of the exponential); call
    the largest of a row e. Every weight is then off by a factor 1 +- (2 e + 4 u), numerator and
    sum; a sum of n terms adds n u. bf16 rounds each weight once before the product with the values
    (half a step) and the output once."""
    B, Hq, L, d = q.shape
    H = cache.k.shape[1]
    cap = cache.table.shape[1] * cache.page
    bf = q.dtype == torch.bfloat16
    u = 2.0 ** -23 if bf else 2.0 ** -24
    half = 2.0 ** -8 if bf else u
    scale = d ** -0.5 if scale is None else scale
    o, lse = torch.zeros(B, Hq, L, d).double(), torch.full((B, Hq, L), -math.inf).double()
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
    wt, wb = torch.zeros(B, H, cap).double(), torch.zeros(B, H, cap).double()
    for b in range(B):
        n, kv = new[b], cache.kv[b]
        h0 = kv - n
        if w_in is not None:
            wt[b, :, :h0] = decay * w_in[b, :, :h0].double()
            wb[b, :, :h0] = 2 * 2.0 ** -24 * wt[b, :, :h0].abs()
        for i in range(n):
            lo = max(0, h0 + (i // N - w + 1) * N) if w else 0
            hi = min(kv, h0 + (i // N + 1) * N)
            for g in range(Hq):
                h = g // (Hq // H)
                K, V = cache.keys[b][h, lo:hi].double(), cache.vals[b][h, lo:hi].double()
                x = K @ q[b, g, i].double() * scale
                e = (d + 8) * u * float((K.abs() @ q[b, g, i].double().abs()).max()) * abs(scale)
                z = torch.logsumexp(x, 0)
                p = torch.exp(x - z)
                o[b, g, i], lse[b, g, i] = p @ V, z
                rel = 2 * e + (hi - lo + 4) * u
                mass = p @ V.abs()
                ob[b, g, i] = (rel + (half if bf else 0)) * mass + half * (p @ V).abs()
                lb[b, g, i] = e + (hi - lo + 4) * u + 2 * 2.0 ** -24 * abs(float(z))
                wt[b, h, lo:hi] += p
                wb[b, h, lo:hi] += p * (2 * e + (hi - lo + 4 + n * Hq // H) * u + 2 * 2.0 ** -24 * abs(float(z)))
    return o, lse, wt, ob, lb, wb


def gdn_ref(q, k, v, a, b, S0, n):
    """One rollout, [H, L, d]: outputs of the first n tokens and the state after them."""
    S = S0.double().clone()
    o = torch.zeros(v.shape).double()
    big = float(S.abs().sum(-1).max())
    for t in range(n):
        kt, vt = k[:, t].double(), v[:, t].double()
        at, bt = a[:, t, None, None].double(), b[:, t, None, None].double()
        eye = torch.eye(S.shape[-1], dtype=torch.float64)
        S = at * S @ (eye - bt * kt[:, :, None] * kt[:, None, :]) + bt * vt[:, :, None] * kt[:, None, :]
        o[:, t] = torch.einsum("hij,hj->hi", S, q[:, t].double())
        big = max(big, float(S.abs().sum(-1).max()), float(vt.abs().max()))
    # per token: two products of d terms and three roundings, on rows of absolute sum at most `big`
    # with |q|, |k| channels at most `c`; errors of earlier tokens are carried, not amplified
    # (contraction) beyond the factor 2 of |I - b k k^T| in the row sum norm
    c = max(1.0, float(q.abs().max()), float(k.abs().max()))
    return o, S, 2 * max(1, n) * (S.shape[-1] + 8) * 2.0 ** -24 * big * c * c
