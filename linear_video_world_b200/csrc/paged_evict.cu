// Eviction from a paged cache by accumulated attention weight: choose the positions to keep, then
// copy their keys, values and weights to the destination's pages.
//
// Choice, one block per (rollout, key head): of the middle positions the `take` largest weights,
// found by a radix select over order-preserving 32-bit keys of the weights (four passes of 8 bits,
// from the top: each pass counts the digits of the keys that still match the threshold's prefix);
// then one pass in order of position numbers the kept ones with a block scan of two counts
// (above the threshold; equal to it, of which the first `ties` stay).
// Copy: a warp per kept position, 16 bytes a lane, K and V in flight together. HBM bound.
#include "hlta_internal.cuh"
#include "paged.cuh"

#include <algorithm>
#include <math.h>

namespace hlta {
namespace {

using namespace paged;

constexpr int ST = 1024;                // threads of the choice

// rises with the weight; equal weights (0 and -0 too) give equal keys, NaN the least
__device__ __forceinline__ uint32_t key_of(float w)
{
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int2 block_scan(int2 v, int2 *warp_s, int2 &total)
{
    // exclusive scan over the block's threads in thread order
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 x = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
        if (lane >= o) {
            x.x += a;
            x.y += b;
        }
    }
    __syncthreads();
    if (lane == 31) warp_s[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int2 y = lane < ST / 32 ? warp_s[lane] : make_int2(0, 0);
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, y.x, o), b = __shfl_up_sync(0xffffffffu, y.y, o);
            if (lane >= o) {
                y.x += a;
                y.y += b;
            }
        }
        warp_s[lane] = y;
    }
    __syncthreads();
    total = warp_s[ST / 32 - 1];
    const int2 before = warp ? warp_s[warp - 1] : make_int2(0, 0);
    return make_int2(before.x + x.x - v.x, before.y + x.y - v.y);
}

__global__ void __launch_bounds__(ST) evict_choose_kernel(PagedEvictArgs a, int *kept)
{
    __shared__ int hist[256];
    __shared__ int2 warp_s[32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    const int h = blockIdx.x % a.c.H, b = blockIdx.x / a.c.H;
    const int cap = a.c.max_pages << a.c.page_log2;
    const int kv = a.c.kv_lens[b];
    const int n = max(0, min(kv, cap));
    if (n != kv && threadIdx.x == 0) atomicOr(a.c.err, DEVERR_TABLE);
    int *out = kept + (long)blockIdx.x * a.budget;
    if (h == 0 && threadIdx.x == 0) a.new_lens[b] = min(n, a.budget);
    if (n <= a.budget) {
        for (int i = threadIdx.x; i < a.budget; i += ST) out[i] = i < n ? i : -1;
        return;
    }
    const float *w = a.weights + (long)blockIdx.x * cap;
    const int lo = a.sink, hi = n - a.recent, take = a.budget - a.sink - a.recent;
    // the take-th largest key of [lo, hi) (take < hi - lo since n > budget)
    uint32_t prefix = 0, mask = 0;
    int left = take;
    if (take > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = threadIdx.x; i < 256; i += ST) hist[i] = 0;
            __syncthreads();
            for (int i = lo + threadIdx.x; i < hi; i += ST) {
                const uint32_t k = key_of(w[i]);
                if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                int d = 255, acc = 0;
                while (d > 0 && acc + hist[d] < left) acc += hist[d--];
                s_prefix = prefix | ((uint32_t)d << shift);
                s_left = left - acc;
            }
            __syncthreads();
            prefix = s_prefix;
            left = s_left;
            mask |= 255u << shift;
            __syncthreads();
        }
    } else {
        prefix = 0xffffffffu;       // nothing is above it
        left = 0;
    }
    // number the kept positions in order
    int2 base = make_int2(0, 0);    // kept so far; equal to the threshold so far
    for (int i0 = 0; i0 < n; i0 += ST) {
        const int i = i0 + threadIdx.x;
        bool sure = false, equal = false;
        if (i < n) {
            if (i < lo || i >= hi) sure = true;
            else {
                const uint32_t k = key_of(w[i]);
                sure = k > prefix;
                equal = k == prefix && left > 0;
            }
        }
        int2 total;
        const int2 at = block_scan(make_int2(sure ? 1 : 0, equal ? 1 : 0), warp_s, total);
        // of the equal ones before this position, those among the first `left` are kept
        const int eq = base.y + at.y;
        const int rank = base.x + at.x + min(eq, left);
        if (sure || (equal && eq < left)) out[rank] = i;
        base.x += total.x;
        base.y += total.y;
    }
}

template <int ROW16>
__device__ __forceinline__ void copy_row(const char *s, char *d, int bytes, int lane)
{
    if constexpr (ROW16) {
        for (int x = lane * 16; x < bytes; x += 512) *(uint4 *)(d + x) = *(const uint4 *)(s + x);
    } else {
        for (int x = lane * 2; x < bytes; x += 64) *(uint16_t *)(d + x) = *(const uint16_t *)(s + x);
    }
}

template <int ROW16>
__global__ void __launch_bounds__(256) evict_copy_kernel(PagedEvictArgs a, const int *kept, int row_bytes)
{
    const int lane = threadIdx.x & 31;
    const long item = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long bh = item / a.budget;
    if (bh >= (long)a.B * a.c.H) return;
    const int r = (int)(item - bh * a.budget);
    const int h = (int)(bh % a.c.H), b = (int)(bh / a.c.H);
    const int src = kept[item];
    if (src < 0) return;
    const int psz = 1 << a.c.page_log2;
    const int dpg = a.dst_table[(long)b * a.max_dst + (r >> a.c.page_log2)];
    if (dpg < 0 || dpg >= a.num_dst) {
        if (lane == 0) atomicOr(a.c.err, DEVERR_TABLE);
        return;
    }
    const long s = (((long)page_of(a.c, b, src) * a.c.H + h) * psz + (src & (psz - 1))) * row_bytes;
    const long d = (((long)dpg * a.c.H + h) * psz + (r & (psz - 1))) * row_bytes;
    copy_row<ROW16>((const char *)a.c.k + s, (char *)a.k_dst + d, row_bytes, lane);
    copy_row<ROW16>((const char *)a.c.v + s, (char *)a.v_dst + d, row_bytes, lane);
    if (a.w_out && lane == 0)
        a.w_out[bh * ((long)a.max_dst << a.c.page_log2) + r] = a.weights[bh * ((long)a.c.max_pages << a.c.page_log2) + src];
}

}  // namespace

size_t paged_evict_bytes(int B, int H, int budget) { return (size_t)B * H * budget * sizeof(int); }

cudaError_t launch_paged_evict(const PagedEvictArgs &a, bool bf16, cudaStream_t s)
{
    const long bh = (long)a.B * a.c.H;
    if (bh == 0) return cudaSuccess;
    const long blocks = (bh * a.budget + 7) / 8;
    if (bh > 0x7fffffffL || blocks > 0x7fffffffL) return cudaErrorNotSupported;
    int *kept = a.kept ? a.kept : (int *)a.ws;
    evict_choose_kernel<<<(unsigned)bh, ST, 0, s>>>(a, kept), note_launch();
    const int row = a.c.d * (bf16 ? 2 : 4);
    if (row % 16 == 0) evict_copy_kernel<1><<<(unsigned)blocks, 256, 0, s>>>(a, kept, row), note_launch();
    else evict_copy_kernel<0><<<(unsigned)blocks, 256, 0, s>>>(a, kept, row), note_launch();
    return cudaGetLastError();
}

}  // namespace hlta
