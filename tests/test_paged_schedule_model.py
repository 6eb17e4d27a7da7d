"""Host models of the paged kernels (no GPU): the division of the line of key tiles among gangs and
the join's view of it, the invariant division, and the barrier protocols of the chunk attention and
weights kernels under random interleavings."""
import random

import pytest


# ---- the line (csrc/paged.cuh) ---------------------------------------------------------------

def _pieces(T, H, passes, ngang, steps, least, extra=0):
    """What each gang takes, as place_of / next_piece do it: {(pass, b, h): [(from, to, gang, slot, whole)]}
    (in places; `extra` of them lie in front of a head's tiles when the gangs have enough to do)."""
    T = [t * steps for t in T]
    if sum(T) * H * passes > least * ngang:
        T = [t + extra if t else 0 for t in T]
    per = sum(T) * H
    W = per * passes
    ng = min(W if W <= len(T) * H * passes else -(-W // least), ngang)
    got = {}
    for g in range(ng):
        a = W * g // ng
        left = W * (g + 1) // ng - a
        ps, x, b = a // per, a % per, 0
        while x >= T[b] * H:
            x -= T[b] * H
            b += 1
        h, t, index = x // T[b], x % T[b], 0
        assert left > 0
        while left > 0:
            while T[b] == 0:
                b += 1
                if b == len(T):
                    b, ps = 0, ps + 1
            take = min(left, T[b] - t)
            got.setdefault((ps, b, h), []).append((t, t + take, g, 0 if index == 0 else 1, take == T[b]))
            # a cut piece is the first or the last of its gang: two slots hold them
            assert take == T[b] or index == 0 or left == take
            left, t, index, h = left - take, 0, index + 1, h + 1
            if h == H:
                h, b = 0, b + 1
                if b == len(T):
                    b, ps = 0, ps + 1
    return T, per, W, ng, got


def _holders(W, ng, a, n):
    """holders_at of csrc/paged.cuh."""
    g0, g1 = ((a + 1) * ng - 1) // W, ((a + n) * ng - 1) // W
    return g0, g1, 0 if W * g0 // ng == a else 1


@pytest.mark.parametrize("seed", range(8))
def test_line_division_and_join_agree(seed):
    r = random.Random(seed)
    for _ in range(300):
        B, H, passes, steps = r.randint(1, 9), r.randint(1, 5), r.choice([1, 1, 2, 3]), r.choice([1, 1, 5])
        T = [r.choice([0, 1, 2, r.randint(1, 300)]) for _ in range(B)]
        if not sum(T):
            continue
        if steps > 1:
            passes = 1
        T, per, W, ng, got = _pieces(T, H, passes, r.choice([1, 2, 3, 21, 148, 296, r.randint(1, 148)]), steps, r.choice([1, 1, 2, 3]),
                                     r.choice([0, 0, 3, 4]) if steps == 1 else 0)
        sizes = [sum(p[1] - p[0] for c in got.values() for p in c if p[2] == g) for g in range(ng)]
        assert max(sizes) - min(sizes) <= 1 and sum(sizes) == W
        for ps in range(passes):
            for b in range(B):
                for h in range(H):
                    if not T[b]:
                        assert (ps, b, h) not in got
                        continue
                    c = got[ps, b, h]
                    assert c[0][0] == 0 and c[-1][1] == T[b] and all(x[1] == y[0] for x, y in zip(c, c[1:]))
                    g0, g1, slot0 = _holders(W, ng, per * ps + sum(T[:b]) * H + h * T[b], T[b])
                    assert [x[2] for x in c] == list(range(g0, g1 + 1))
                    if g0 == g1:
                        assert c[0][4]
                    else:
                        assert all(not x[4] and x[3] == (slot0 if x[2] == g0 else 0) for x in c)


def test_division_by_a_launch_constant():
    """fast_div / fdiv of csrc/paged.cuh in exact arithmetic: m fits 32 bits, the sum does not
    overflow, the quotient is right, for divisors below 2^30 and dividends below 2^31."""
    r = random.Random(1)
    for _ in range(100000):
        d = r.choice([1, 2, 3, 5, 7, 64, 1560, 2 ** 30 - 1, r.randint(1, 2 ** 30 - 1), 2 ** r.randint(0, 29)])
        x = min(2 ** 31 - 1, r.choice([0, 1, d - 1, d, d + 1, 2 ** 31 - 1, r.randint(0, 2 ** 31 - 1)]))
        s = 0
        while (1 << s) < d:
            s += 1
        m = ((((1 << s) - d) << 32) // d) + 1
        hi = m * x >> 32
        assert m < 2 ** 32 and hi + x < 2 ** 32 and (hi + x) >> s == x // d


# ---- barrier protocols -------------------------------------------------------------------------

class Bar:
    """An mbarrier: `count` arrivals complete a phase; a wait names the parity of the phase it wants."""

    def __init__(self, count):
        self.count, self.n, self.phase = count, 0, 0

    def arrive(self):
        self.n += 1
        assert self.n <= self.count
        if self.n == self.count:
            self.n, self.phase = 0, self.phase + 1

    def done(self, parity):
        return (self.phase - 1) & 1 == parity


def _wait(bar, parity):
    while not bar.done(parity):
        yield


def _run(roles, bars, r):
    """Random interleaving of the roles until all have ended."""
    idle = 0
    while roles:
        g = r.choice(roles)
        before = sum(b.phase * 1000 + b.n for b in bars.values())
        try:
            next(g)
        except StopIteration:
            roles.remove(g)
            idle = 0
            continue
        idle = idle + 1 if before == sum(b.phase * 1000 + b.n for b in bars.values()) else 0
        assert idle < 5000, "no role can go on"


def _attention(seed):
    r = random.Random(seed)
    slots = 3
    shares = []
    for _ in range(r.randint(1, 6)):                    # (first tile, end, [a, b) per sub-tile, edge tiles)
        n = r.randint(1, 6)
        sub = []
        for _q in range(2):
            a = r.randint(0, n)
            sub.append((a, r.randint(a, n)))
        need = [s for s in sub if s[1] > s[0]]
        shares.append((min([s[0] for s in need], default=0), max([s[1] for s in need], default=0), sub, {t for t in range(n) if r.random() < 0.4}))
    B = {"qfull": Bar(1), "qfree": Bar(2)}
    for i in range(slots):
        B["full", i], B["empty", i] = Bar(1), Bar(2)
    for q in range(2):
        for n in ("sfull", "sfree", "pfull", "pvdone", "odone", "ofree"):
            B[n, q] = Bar(1)
    slot, Q, S, P, O = [None] * slots, [None], [None, None], [None, None], [None, None]
    o_read, rescaling, zeroed = [True, True], [False, False], set()

    def producer():
        it = units = 0
        for u, (lo, hi, _sub, _edge) in enumerate(shares):
            if hi <= lo:
                continue

            def load(what):
                nonlocal it
                if it >= slots:
                    yield from _wait(B["empty", it % slots], (it // slots + 1) & 1)
                slot[it % slots] = what
                B["full", it % slots].arrive()
                it += 1
                yield
            if units:
                yield from _wait(B["qfree"], (units - 1) & 1)
            Q[0] = u
            B["qfull"].arrive()
            units += 1
            yield from load(("K", u, lo))
            for t in range(lo, hi):
                if t + 1 < hi:
                    yield from load(("K", u, t + 1))
                yield from load(("V", u, t))

    def issuer(q):
        it = units = ns = npv = 0
        for u, (lo, hi, sub, edge) in enumerate(shares):
            if hi <= lo:
                continue
            a, b = sub[q]
            yield from _wait(B["qfull"], units & 1)

            def do_s(t):
                nonlocal it, ns
                yield from _wait(B["full", it % slots], (it // slots) & 1)
                assert slot[it % slots] == ("K", u, t)
                if a <= t < b:
                    if ns:
                        yield from _wait(B["sfree", q], (ns - 1) & 1)
                    assert Q[0] == u and S[q] is None
                    S[q] = (u, t)
                    yield
                    B["sfull", q].arrive()
                    ns += 1
                B["empty", it % slots].arrive()
                it += 1
                if t + 1 == hi:
                    B["qfree"].arrive()
                yield

            def do_pv(t):
                nonlocal it, npv
                yield from _wait(B["full", it % slots], (it // slots) & 1)
                assert slot[it % slots] == ("V", u, t)
                if a <= t < b:
                    yield from _wait(B["pfull", q], npv & 1)
                    if t == a and units:
                        yield from _wait(B["ofree", q], (units - 1) & 1)
                    assert P[q] == (u, t) and (t > a or o_read[q]) and not rescaling[q]
                    assert t not in edge or (u, t, q) in zeroed
                    yield
                    assert P[q] == (u, t)
                    P[q], O[q], o_read[q] = None, (u, t), False
                    B["pvdone", q].arrive()
                    npv += 1
                B["empty", it % slots].arrive()
                it += 1
                yield
            yield from do_s(lo)
            for t in range(lo, hi):
                if t + 1 < hi:
                    yield from do_s(t + 1)
                yield from do_pv(t)
            if a >= b and units:
                yield from _wait(B["ofree", q], (units - 1) & 1)
            B["odone", q].arrive()
            units += 1
            yield

    def softmax(q):
        k = units = items = 0
        for u, (lo, hi, sub, edge) in enumerate(shares):
            a, b = sub[q]
            for t in range(a, b):
                yield from _wait(B["sfull", q], k & 1)
                assert S[q] == (u, t)
                S[q] = None
                B["sfree", q].arrive()
                yield
                if k:
                    yield from _wait(B["pvdone", q], (k - 1) & 1)
                assert P[q] is None
                P[q] = (u, t)
                yield
                if t > a and r.random() < 0.4:          # O rescaled
                    assert O[q] == (u, t - 1)
                    rescaling[q] = True
                    yield
                    rescaling[q] = False
                if t in edge:                           # values outside the span zeroed in the slot
                    item = items + (2 * (t - lo) + 2 if t + 1 < hi else 2 * (t - lo) + 1)
                    yield from _wait(B["full", item % slots], (item // slots) & 1)
                    assert slot[item % slots] == ("V", u, t)
                    zeroed.add((u, t, q))
                B["pfull", q].arrive()
                k += 1
                yield
            items += 2 * (hi - lo)
            if hi > lo:
                yield from _wait(B["odone", q], units & 1)
                units += 1
                assert b <= a or O[q] == (u, b - 1)
                yield
                o_read[q] = True
                B["ofree", q].arrive()
            yield
    _run([producer(), issuer(0), issuer(1), softmax(0), softmax(1)], B, r)


def _weights(seed):
    r = random.Random(seed)
    nk_, nq_ = 2, 4
    tiles = [[rt for rt in range(r.randint(0, 7)) if r.random() < 0.8] for _ in range(r.randint(1, 7))]
    B = {}
    for i in range(nk_):
        B["kfull", i], B["kempty", i] = Bar(1), Bar(1)
    for i in range(nq_):
        B["qfull", i], B["qempty", i], B["sfull", i], B["sfree", i] = Bar(1), Bar(1), Bar(1), Bar(1)
    K, Q, Z, S = [None] * nk_, [None] * nq_, [None] * nq_, [None] * nq_

    def producer():
        nq = 0
        for nk, rows in enumerate(tiles):
            if nk >= nk_:
                yield from _wait(B["kempty", nk % nk_], (nk // nk_ + 1) & 1)
            K[nk % nk_] = nk
            B["kfull", nk % nk_].arrive()
            for rt in rows:
                s = nq % nq_
                if nq >= nq_:
                    yield from _wait(B["qempty", s], (nq // nq_ + 1) & 1)
                    yield from _wait(B["sfree", s], (nq // nq_ + 1) & 1)
                Q[s] = Z[s] = (nk, rt)
                B["qfull", s].arrive()
                nq += 1
                yield

    def issuer():
        nq = 0
        for nk, rows in enumerate(tiles):
            yield from _wait(B["kfull", nk % nk_], (nk // nk_) & 1)
            for rt in rows:
                s = nq % nq_
                yield from _wait(B["qfull", s], (nq // nq_) & 1)
                if nq >= nq_:
                    yield from _wait(B["sfree", s], (nq // nq_ + 1) & 1)
                assert Q[s] == (nk, rt) and K[nk % nk_] == nk and S[s] is None
                S[s] = (nk, rt)
                yield
                B["sfull", s].arrive()
                B["qempty", s].arrive()
                nq += 1
                yield
            B["kempty", nk % nk_].arrive()
            yield

    def group(g):
        nq = 0
        for nk, rows in enumerate(tiles):
            for rt in rows:
                s, par, mine = nq % nq_, (nq // nq_) & 1, nq & 1 == g
                nq += 1
                if not mine:
                    continue
                yield from _wait(B["qfull", s], par)
                yield from _wait(B["sfull", s], par)
                assert S[s] == (nk, rt) and Z[s] == (nk, rt)
                yield
                assert Z[s] == (nk, rt)
                S[s] = None
                B["sfree", s].arrive()
                yield
    _run([producer(), issuer(), group(0), group(1)], B, r)


@pytest.mark.parametrize("protocol", [_attention, _weights])
def test_protocol_under_random_interleavings(protocol):
    for seed in range(400):
        protocol(seed)
