// Shared by the kernels over a paged cache: a rollout's lengths, the keys a row of the chunk
// sees, and page lookup.
#pragma once

#include "hlta_internal.cuh"

namespace hlta {
namespace paged {

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
__device__ __forceinline__ Span span_of(const Roll &r, int i, int N, int w)
{
    const long long f = i / N;
    const long long hi = (long long)r.h + (f + 1) * N;
    const long long lo = w > 0 ? (long long)r.h + (f - w + 1) * N : 0;
    Span s;
    s.hi = (int)(hi < 0 ? 0 : hi < r.kv ? hi : r.kv);
    s.lo = (int)(lo < 0 ? 0 : lo < r.kv ? lo : r.kv);
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
// Division of the work over the GPU (bf16 kernels).
//
// A key head's packed rows come in row tiles. The keys that a rollout's chunk sees come in tiles of
// TK keys (aligned to multiples of TK in the cache); rollout b has T_b of them per key head. A gang
// of `gs` consecutive blocks takes the row tiles pass * gs .. pass * gs + gs - 1 of a key head
// together, a block each, over the same key tiles, so that they meet in L2. The line of all
// (pass, rollout, key head, key tile) is cut into equal lengths, one per gang: no gang has more
// than one tile more than another, whatever the rollouts' lengths, no counter is shared, and the
// division depends on the lengths and the grid alone. A gang's cut ends fall inside a head's
// keys; that head's pieces are joined by a second kernel from (maximum, sum, unnormalised output)
// in the workspace, at most two per block: slot 0 for the first piece of its range, slot 1 for the
// last.
struct Line {
    int B, H, L, N, w, cap, gs, ngang, passes;
    const int *kv_lens, *new_lens;
};
template <int TK>
struct Tiles {
    Roll r;
    int t0, T;                      // first key tile; tiles
};
template <int TK>
__device__ __forceinline__ Tiles<TK> tiles_of(const Line &p, int b)
{
    Tiles<TK> x;
    x.r = roll_of(p.kv_lens, p.new_lens, b, p.L, p.cap);
    x.t0 = x.T = 0;
    if (x.r.n > 0) {
        const int lo = span_of(x.r, 0, p.N, p.w).lo, hi = span_of(x.r, x.r.n - 1, p.N, p.w).hi;
        if (hi > lo) {
            x.t0 = lo / TK;
            x.T = (hi + TK - 1) / TK - x.t0;
        }
    }
    return x;
}

// Sum of T over rollouts [0, b) by one warp (all lanes get it).
template <int TK>
__device__ __forceinline__ long long tiles_before(const Line &p, int b)
{
    long long s = 0;
    for (int i = threadIdx.x & 31; i < b; i += 32) s += tiles_of<TK>(p, i).T;
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// A place on the line: the next key tile `t` of key head h of rollout b in pass `pass`.
struct Place {
    int pass, b, h, t;
    int left;                       // tiles left of the range
};

// Start of gang g's range (one warp; all lanes get it).
template <int TK>
__device__ __forceinline__ Place place_of(const Line &p, int g)
{
    const int lane = threadIdx.x & 31;
    const long long per = tiles_before<TK>(p, p.B) * p.H, W = per * p.passes;
    const long long ng = W < p.ngang ? W : p.ngang;         // no gang's cut is empty
    Place c;
    c.left = 0;
    c.pass = c.b = c.h = c.t = 0;
    if (g >= ng) return c;
    const long long a = W * g / ng;
    c.left = (int)(W * (g + 1) / ng - a);
    c.pass = (int)(a / per);
    long long x = a - per * c.pass;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const long long n = b0 + lane < p.B ? (long long)tiles_of<TK>(p, b0 + lane).T * p.H : 0;
        long long s = n;                                    // inclusive scan
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        const unsigned in = __ballot_sync(0xffffffffu, x < s);
        if (in) {
            const int f = __ffs(in) - 1;
            const long long before = __shfl_sync(0xffffffffu, s - n, f);
            const int T = (int)(__shfl_sync(0xffffffffu, n, f) / p.H);
            c.b = b0 + f;
            x -= before;
            c.h = (int)(x / T);
            c.t = (int)(x - (long long)c.h * T);
            return c;
        }
        x -= __shfl_sync(0xffffffffu, s, 31);
    }
    c.left = 0;                     // not reached
    return c;
}

// The piece at c (key tiles [ta, tb) of its head, `whole` when that is all of them), and c moved
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
    while (o.x.T == 0) {            // rollouts without tiles have no place on the line
        if (++c.b == p.B) {
            c.b = 0;
            ++c.pass;
        }
        o.x = tiles_of<TK>(p, c.b);
    }
    o.pass = c.pass;
    o.b = c.b;
    o.h = c.h;
    const int take = min(c.left, o.x.T - c.t);
    o.ta = o.x.t0 + c.t;
    o.tb = o.ta + take;
    o.whole = take == o.x.T;
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

// The gangs that hold pieces of one head's keys in one pass: g0 .. g1 (one warp).
struct Holders {
    int g0, g1, slot0, T;           // slot of g0's piece; the others lie in slot 0
};
template <int TK>
__device__ __forceinline__ Holders holders_of(const Line &p, int pass, int b, int h)
{
    const long long per = tiles_before<TK>(p, p.B) * p.H, W = per * p.passes;
    Holders o;
    o.T = tiles_of<TK>(p, b).T;
    o.g0 = o.g1 = o.slot0 = 0;
    const long long a = per * pass + tiles_before<TK>(p, b) * p.H + (long long)h * o.T;
    if (o.T == 0) return o;
    // gang g holds [W g / ng, W (g + 1) / ng), rounded down
    const long long ng = W < p.ngang ? W : p.ngang;
    o.g0 = (int)(((a + 1) * ng - 1) / W);
    o.g1 = (int)(((a + o.T) * ng - 1) / W);
    o.slot0 = W * o.g0 / ng == a ? 0 : 1;
    return o;
}

}  // namespace paged
}  // namespace hlta
