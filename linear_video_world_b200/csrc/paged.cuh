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

}  // namespace paged
}  // namespace hlta
