// Shared by the kernels over a paged cache: a rollout's lengths, the keys a row of the chunk
// sees, and page lookup.
#pragma once

#include "hlta_internal.cuh"

namespace hlta {
namespace paged {

// Division by a number fixed for the launch (of non-negative numbers below 2^31): quotient
// (umulhi(m, x) + x) >> s with s the bits of d - 1 and m = floor(2^32 (2^s - d) / d) + 1 (the
// invariant division of Granlund and Montgomery).
struct FastDiv {
    unsigned d, m, s;
};
__host__ inline FastDiv fast_div(unsigned d)
{
    FastDiv f;
    f.d = d;
    f.s = 0;
    while ((1ull << f.s) < d) ++f.s;
    f.m = (unsigned)((((1ull << f.s) - d) << 32) / d + 1);
    return f;
}
__device__ __forceinline__ int fdiv(int x, const FastDiv &f)
{
    return (int)((__umulhi(f.m, (unsigned)x) + (unsigned)x) >> f.s);
}
__device__ __forceinline__ int frem(int x, const FastDiv &f) { return x - fdiv(x, f) * (int)f.d; }

// A rollout of the batch: kv tokens cached, n of them new (the chunk), h before the chunk.
// Lengths that do not fit are clamped (h may be negative: the chunk's first rows then lie before
// position 0).
struct Roll {
    int kv, n, h;
    bool bad;
};
__device__ __forceinline__ Roll roll_of(const int *kv_lens, const int *new_lens, int b, int L, int cap)
{
    Roll r;
    const int kv = kv_lens[b], n = new_lens ? new_lens[b] : L;
    r.kv = max(0, min(kv, cap));
    r.n = max(0, min(n, L));
    r.h = r.kv - r.n;
    r.bad = r.kv != kv || r.n != n || r.h < 0;
    return r;
}

// Positions [lo, hi) that token i of the chunk sees (empty: hi <= lo, both clamped to [0, kv]).
struct Span {
    int lo, hi;
};
// (w frames of N tokens back; `back` = (w - 1) N, clamped to 2^30, or 2^30 for no window).
struct Mask {
    FastDiv N;
    int back;
};
__host__ inline Mask mask_of(int N, int w)
{
    // frames longer than any chunk (2^29 tokens) are all alike
    const long long n = N < (1 << 30) ? N : (1 << 30) - 1, b = w > 0 ? (long long)(w - 1) * n : 1LL << 30;
    return Mask{fast_div((unsigned)n), (int)(b < (1LL << 30) ? b : 1LL << 30)};
}
__device__ __forceinline__ Span span_of(const Roll &r, int i, const Mask &m)
{
    // h + start is a position, at most 2^30, and N below that: the sums stay inside 32 bits
    const int start = fdiv(i, m.N) * (int)m.N.d, hi = r.h + start + (int)m.N.d, lo = r.h + start - m.back;
    Span s;
    s.hi = max(0, min(hi, r.kv));
    s.lo = max(0, min(lo, r.kv));
    return s;
}

// The page of position p of rollout b; page 0, recorded, when the table's entry is out of range.
__device__ __forceinline__ int page_of(const PagedKV &c, int b, int p)
{
    const int pg = c.table[(long)b * c.max_pages + (p >> c.page_log2)];
    if (pg >= 0 && pg < c.num_pages) return pg;
    atomicOr(c.err, DEVERR_TABLE);
    return 0;
}

// ---------------------------------------------------------------------------------------
// Division of the work over the GPU (the attention and weights kernels).
//
// A key head's packed rows come in row tiles. The keys that a rollout's chunk sees come in tiles of
// TK keys (aligned to multiples of TK in the cache); rollout b has T_b of them per key head. A gang
// of `gs` consecutive blocks takes the row tiles pass * gs .. pass * gs + gs - 1 of a key head
// together, a block each, over the same key tiles, so that they meet in L2. The line of all
// (pass, rollout, key head, key tile) is cut into equal lengths, one per gang (the start and end of a head
// count as `extra` tiles, if they cost as much): no gang has more than one place more than another,
// whatever the rollouts' lengths, no counter is shared, and the division depends on the lengths and the
// grid alone. Places are not work: those of `extra` hold no tile, and of the tiles, which are those that
// the whole chunk sees, a block walks only what its own row tile sees. With a long history that is nearly
// all of them; of a chunk without history the first row tiles see few and the last all, and so do blocks
// of row tiles far apart under a short window (8192 tokens of 8 heads, each seeing those before it:
// 222 us, 0.62 PFLOP/s, where a frame over 32760 keys reaches 0.94).
// A gang's cut ends fall inside a head's keys; that head's pieces are joined by a second kernel from
// (maximum, sum, unnormalised output) in the workspace, at most two per block: slot 0 for the first piece
// of its range, slot 1 for the last.
struct Line {
    int B, H, L, cap, gs, ngang, passes;
    int least;                      // places a gang takes at least (while there are gangs to spare)
    int steps;                      // places on the line per key tile (1; more where a tile's work is cut too)
    int extra;                      // places in front of each head's tiles: what its start and end cost
    FastDiv byL;
    Mask mask;
    const int *kv_lens, *new_lens;
};
__host__ inline Line line_of(const PagedAttnArgs &a, int gs, int ngang, int passes, int least = 1, int steps = 1, int extra = 0)
{
    Line p;
    p.B = a.B; p.H = a.c.H; p.L = (int)a.L;
    p.cap = a.c.max_pages << a.c.page_log2;
    p.gs = gs; p.ngang = ngang; p.passes = passes; p.least = least; p.steps = steps; p.extra = extra;
    p.byL = fast_div((unsigned)(a.L > 0 ? a.L : 1));
    p.mask = mask_of(a.N, a.w);
    p.kv_lens = a.c.kv_lens; p.new_lens = a.new_lens;
    return p;
}
// Gangs that take part: none with less than `least` places (one where there are no more places than
// heads: such cuts fall between them), and no cut is empty.
__device__ __forceinline__ long long gangs(const Line &p, long long W)
{
    const long long n = W <= (long long)p.B * p.H * p.passes ? W : (W + p.least - 1) / p.least;
    return n < p.ngang ? n : p.ngang;
}
// 64-bit quotient; in 32 bits where both fit (a third of the time)
__device__ __forceinline__ long long quot(long long a, long long b)
{
    return (unsigned long long)a >> 32 || (unsigned long long)b >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

template <int TK>
struct Tiles {
    Roll r;
    int t0, T;                      // first key tile; places (tiles x steps)
};
template <int TK>
__device__ __forceinline__ Tiles<TK> tiles_of(const Line &p, int b)
{
    Tiles<TK> x;
    x.r = roll_of(p.kv_lens, p.new_lens, b, p.L, p.cap);
    x.t0 = x.T = 0;
    if (x.r.n > 0) {
        const int lo = span_of(x.r, 0, p.mask).lo, hi = span_of(x.r, x.r.n - 1, p.mask).hi;
        if (hi > lo) {
            x.t0 = lo / TK;
            x.T = ((hi + TK - 1) / TK - x.t0) * p.steps;
        }
    }
    return x;
}

// Places per key head and pass of rollouts [0, b) and of all, and rollout b's own, by one warp (all
// lanes get them). A head's start and end count only where there are more tiles than the gangs take
// at least: then a gang has several heads, or few tiles beside one's start.
struct Sums {
    long long before, all;
    int own, extra;
};
template <int TK>
__device__ __forceinline__ Sums tile_sums(const Line &p, int b)
{
    Sums s{0, 0, 0, 0};
    int n_all = 0, n_before = 0;                    // rollouts with tiles
    for (int i = threadIdx.x & 31; i < p.B; i += 32) {
        const int T = tiles_of<TK>(p, i).T;
        s.all += T;
        n_all += T > 0;
        if (i < b) {
            s.before += T;
            n_before += T > 0;
        }
        s.own = i == b ? T : s.own;
    }
    for (int o = 16; o; o >>= 1) {
        s.all += __shfl_xor_sync(0xffffffffu, s.all, o);
        s.before += __shfl_xor_sync(0xffffffffu, s.before, o);
    }
    s.own = __shfl_sync(0xffffffffu, s.own, b & 31);
    if (p.extra && s.all * p.H * p.passes > (long long)p.least * p.ngang) {
        s.extra = p.extra;
        s.all += (long long)p.extra * __reduce_add_sync(0xffffffffu, n_all);
        s.before += (long long)p.extra * __reduce_add_sync(0xffffffffu, n_before);
        s.own += s.own > 0 ? p.extra : 0;
    }
    return s;
}

// A place on the line: the next key tile `t` of key head h of rollout b in pass `pass`.
struct Place {
    int pass, b, h, t;
    int left;                       // places left of the range
    int extra;
};

// Start of gang g's range (one warp; all lanes get it).
template <int TK>
__device__ __forceinline__ Place place_of(const Line &p, int g)
{
    const int lane = threadIdx.x & 31;
    const Sums sums = tile_sums<TK>(p, 0);
    const long long per = sums.all * p.H, W = per * p.passes;
    const long long ng = gangs(p, W);
    Place c;
    c.left = 0;
    c.extra = sums.extra;
    c.pass = c.b = c.h = c.t = 0;
    if (g >= ng) return c;
    const long long a = quot(W * g, ng);
    c.left = (int)(quot(W * (g + 1), ng) - a);
    c.pass = p.passes > 1 ? (int)quot(a, per) : 0;
    long long x = a - per * c.pass;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int own = b0 + lane < p.B ? tiles_of<TK>(p, b0 + lane).T : 0;
        const long long n = own ? (long long)(own + c.extra) * p.H : 0;
        long long s = n;                                    // inclusive scan
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        const unsigned in = __ballot_sync(0xffffffffu, x < s);
        if (in) {
            const int f = __ffs(in) - 1;
            const long long before = __shfl_sync(0xffffffffu, s - n, f);
            const int T = tiles_of<TK>(p, b0 + f).T + c.extra;
            c.b = b0 + f;
            x -= before;
            c.h = (int)quot(x, T);
            c.t = (int)(x - (long long)c.h * T);
            return c;
        }
        x -= __shfl_sync(0xffffffffu, s, 31);
    }
    c.left = 0;                     // not reached
    return c;
}

// The piece at c (key tiles, or steps, [ta, tb) of its head, `whole` when that is all of them), and c moved
// behind it. False at the end of the range.
template <int TK>
struct Piece {
    Tiles<TK> x;
    int pass, b, h, ta, tb;
    bool whole;
};
template <int TK>
__device__ __forceinline__ bool next_piece(const Line &p, Place &c, Piece<TK> &o)
{
    if (c.left <= 0) return false;
    o.x = tiles_of<TK>(p, c.b);
    // rollouts without tiles have no place on the line (bounded, like `take` below, in case the lengths
    // are changed under the kernel)
    for (int seen = 0; o.x.T == 0; ++seen) {
        if (seen > p.B) return false;
        if (++c.b == p.B) {
            c.b = 0;
            ++c.pass;
        }
        o.x = tiles_of<TK>(p, c.b);
    }
    o.pass = c.pass;
    o.b = c.b;
    o.h = c.h;
    const int T = o.x.T + c.extra, take = min(c.left, T - c.t);
    if (take <= 0) return false;
    // the places in front of the tiles hold none: a piece of them alone is empty
    o.ta = o.x.t0 * p.steps + max(0, c.t - c.extra);
    o.tb = o.x.t0 * p.steps + max(0, c.t + take - c.extra);
    o.whole = take == T;
    c.left -= take;
    c.t = 0;
    if (++c.h == p.H) {
        c.h = 0;
        if (++c.b == p.B) {
            c.b = 0;
            ++c.pass;
        }
    }
    return true;
}

// The gangs that hold pieces of places [a, a + n) of the line (one warp): g0 .. g1.
struct Holders {
    int g0, g1, slot0, T;           // slot of g0's piece (the others lie in slot 0); places
};
__device__ __forceinline__ Holders holders_at(const Line &p, long long W, long long a, int n)
{
    Holders o;
    o.T = n;
    o.g0 = o.g1 = o.slot0 = 0;
    if (n == 0) return o;
    // gang g holds [W g / ng, W (g + 1) / ng), rounded down
    const long long ng = gangs(p, W);
    o.g0 = (int)quot((a + 1) * ng - 1, W);
    o.g1 = (int)quot((a + n) * ng - 1, W);
    o.slot0 = quot(W * o.g0, ng) == a ? 0 : 1;
    return o;
}
// ... of one head's keys in one pass.
template <int TK>
__device__ __forceinline__ Holders holders_of(const Line &p, int pass, int b, int h)
{
    const Sums s = tile_sums<TK>(p, b);
    const long long per = s.all * p.H;
    return holders_at(p, per * p.passes, per * pass + s.before * p.H + (long long)h * s.own, s.own);
}

}  // namespace paged
}  // namespace hlta
