// Eviction from a paged cache by accumulated attention weight: choose the positions to keep, then
// copy their keys, values and weights to the destination's pages.
//
// Choice, one block per (rollout, key head), or a cluster of two for long rows that fit the GPU
// together (64 rows of 20000 to 32760 positions: the choice 38 us with one block each, 24 us
// with two; the whole call, 16 rows of 9231: 20.8 and 20.7 us; 16 of 900: 10.8 and 13.9 us; clusters of four and
// eight were never the faster: 23 and 53 us at 9231): of the
// middle positions the `take` largest weights, found by a radix select over order-preserving 32-bit
// keys of the weights (three passes of 11, 11 and 10 bits, from the top: each counts the digits of
// the keys that still match the threshold's prefix; the blocks read one another's counts). Each
// block has a run of the positions; it reads their keys from memory once and keeps them in shared
// memory (up to KEEP; longer runs are read again). A warp whose keys share a digit adds them with one
// atomic: unused positions have equal weights. Then each warp takes a run of its block's positions
// and numbers the kept ones by ballots, after a scan over the blocks' and warps' counts (above the
// threshold; equal to it, of which the first `left` stay).
// Copy: a warp takes eight kept positions, all their 16-byte words of K and V in flight together.
// Bound by HBM.
#include "hlta_internal.cuh"
#include "paged.cuh"

#include <algorithm>
#include <cooperative_groups.h>
#include <math.h>

namespace hlta {
namespace {

using namespace paged;

constexpr int ST = 1024, SW = ST / 32;                  // threads and warps of the choice
constexpr int BINS = 2048, KEEP = 49152;
constexpr size_t CHOOSE_SMEM = (size_t)(KEEP + 2 * BINS) * 4;
std::atomic<unsigned long long> g_shared{0};

// rises with the weight; equal weights (0 and -0 too) give equal keys, NaN the least
__device__ __forceinline__ uint32_t key_of(float w)
{
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(ST) evict_choose_kernel(PagedEvictArgs a, int *kept)
{
    extern __shared__ uint32_t sm[];
    uint32_t *keys = sm + 2 * BINS;             // behind two sets of counts, used in turn
    __shared__ int warp_n[SW], warp_e[SW], block_n[2];
    __shared__ uint32_t s_digit;
    __shared__ int s_left;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int nblk = (int)cluster.num_blocks(), blk = (int)cluster.block_rank();
    auto sync = [&] {
        if (nblk > 1) cluster.sync();
        else __syncthreads();
    };
    // sum of the warps' numbers before this one
    auto before_warp = [&](const int *v) {
        int x = lane < warp ? v[lane] : 0;
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    };
    const long bh = blockIdx.x / nblk;
    const int h = (int)(bh % a.c.H), b = (int)(bh / a.c.H), tid = blk * ST + (int)threadIdx.x;
    const int cap = a.c.max_pages << a.c.page_log2;
    const int kv = a.c.kv_lens[b];
    const int n = max(0, min(kv, cap));
    if (n != kv && tid == 0) atomicOr(a.c.err, DEVERR_TABLE);
    int *out = kept + bh * a.budget;
    if (h == 0 && tid == 0) a.new_lens[b] = min(n, a.budget);
    if (n <= a.budget) {                    // the whole cluster alike
        for (int i = tid; i < a.budget; i += nblk * ST) out[i] = i < n ? i : -1;
        return;
    }
    const int middle = n - a.recent - a.sink, take = a.budget - a.sink - a.recent;
    // this block's run of the middle positions: [lo, lo + m)
    const int first = (int)((long)middle * blk / nblk), m = (int)((long)middle * (blk + 1) / nblk) - first, lo = a.sink + first;
    const float *w = a.weights + bh * cap;
    const bool held = m <= KEEP;
    if (held && take > 0) {
#pragma unroll 8
        for (int i = threadIdx.x; i < m; i += ST) keys[i] = key_of(w[lo + i]);
    }
    auto key = [&](int i) { return held ? keys[i] : key_of(w[lo + i]); };
    // the take-th largest key of the middle ones (take < middle since n > budget)
    uint32_t prefix = 0, mask = 0;
    int left = take;
    if (take > 0) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
            uint32_t *hist = sm + (pass & 1) * BINS;
            for (int i = threadIdx.x; i < BINS; i += ST) hist[i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int i0 = 0; i0 < m; i0 += ST) {
                const int i = i0 + threadIdx.x;
                const uint32_t k = i < m ? key(i) : 0u;
                const bool in = i < m && (k & mask) == prefix;
                const uint32_t d = in ? (k >> shift) & ((1u << width) - 1u) : 0xffffffffu;
                if (__all_sync(0xffffffffu, d == __shfl_sync(0xffffffffu, d, 0))) {
                    if (lane == 0 && in) atomicAdd(&hist[d], 32u);
                } else if (in) {
                    atomicAdd(&hist[d], 1u);
                }
            }
            sync();
            // the digit at which the count from the top reaches `left`: thread t owns digits
            // BINS - 1 - 2 t and BINS - 2 - 2 t
            int c0 = 0, c1 = 0;
            for (int v = 0; v < nblk; ++v) {
                const uint32_t *theirs = cluster.map_shared_rank(hist, v);
                c0 += (int)theirs[BINS - 1 - 2 * threadIdx.x];
                c1 += (int)theirs[BINS - 2 - 2 * threadIdx.x];
            }
            int x = c0 + c1;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) warp_n[warp] = x;
            __syncthreads();
            const int before = before_warp(warp_n) + x - c0 - c1;
            if (before < left && before + c0 + c1 >= left) {
                const bool second = before + c0 < left;
                s_digit = (uint32_t)(BINS - 1 - 2 * (int)threadIdx.x - (second ? 1 : 0));
                s_left = left - before - (second ? c0 : 0);
            }
            __syncthreads();
            prefix |= s_digit << shift;
            mask |= ((1u << width) - 1u) << shift;
            left = s_left;
        }
    } else {
        prefix = 0xffffffffu;       // nothing is above it, and none of its equals stay
        left = 0;
    }
    for (int i = tid; i < a.sink; i += nblk * ST) out[i] = i;
    for (int i = tid; i < a.recent; i += nblk * ST) out[a.sink + take + i] = n - a.recent + i;
    if (take == 0) return;
    // number the kept middle positions in order: each warp a run of them
    const int run = ((m + SW - 1) / SW + 31) & ~31, i_lo = min(m, warp * run), i_hi = min(m, i_lo + run);
    int above = 0, equal = 0;
#pragma unroll 4
    for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < i_hi ? key(i) : 0u;
        above += __popc(__ballot_sync(0xffffffffu, i < i_hi && k > prefix));
        equal += __popc(__ballot_sync(0xffffffffu, i < i_hi && k == prefix));
    }
    if (lane == 0) {
        warp_n[warp] = above;
        warp_e[warp] = equal;
    }
    __syncthreads();
    above = before_warp(warp_n);
    equal = before_warp(warp_e);
    if (threadIdx.x == ST - 1) {
        block_n[0] = above + warp_n[SW - 1];
        block_n[1] = equal + warp_e[SW - 1];
    }
    sync();
    for (int v = 0; v < blk; ++v) {
        const int *theirs = cluster.map_shared_rank(block_n, v);
        above += theirs[0];
        equal += theirs[1];
    }
    sync();                                     // no block ends while another reads its counts
#pragma unroll 4
    for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < i_hi ? key(i) : 0u;
        const unsigned is_above = __ballot_sync(0xffffffffu, i < i_hi && k > prefix), is_equal = __ballot_sync(0xffffffffu, i < i_hi && k == prefix);
        const unsigned below = (1u << lane) - 1u;
        const int eq = equal + __popc(is_equal & below), rank = above + __popc(is_above & below) + min(eq, left);
        if ((is_above >> lane & 1u) || ((is_equal >> lane & 1u) && eq < left)) out[a.sink + rank] = lo + i;
        above += __popc(is_above);
        equal += __popc(is_equal);
    }
}

constexpr int CPW = 8;                                  // kept positions per warp of the copy

// WORD: bytes per access (16, or 2 for rows of another length)
template <typename WORD>
__global__ void __launch_bounds__(256) evict_copy_kernel(PagedEvictArgs a, const int *kept, int words)
{
    const int lane = threadIdx.x & 31;
    const int per = (a.budget + CPW - 1) / CPW;         // warps per head
    const long item = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long bh = item / per;
    if (bh >= (long)a.B * a.c.H) return;
    const int r0 = (int)(item - bh * per) * CPW, h = (int)(bh % a.c.H), b = (int)(bh / a.c.H);
    const int psz = 1 << a.c.page_log2;
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the choice (set up at its end: blocks that
                                                            // wait from its start on cost it 15 us)
    // lanes 0-7: where the eight positions come from and go, in words
    long s = 0, d = -1;
    if (lane < CPW && r0 + lane < a.budget) {
        const int r = r0 + lane, src = kept[bh * a.budget + r];
        if (src >= 0) {
            const int dpg = a.dst_table[(long)b * a.max_dst + (r >> a.c.page_log2)];
            if (dpg < 0 || dpg >= a.num_dst) {
                atomicOr(a.c.err, DEVERR_TABLE);
            } else {
                s = (((long)page_of(a.c, b, src) * a.c.H + h) * psz + (src & (psz - 1))) * words;
                d = (((long)dpg * a.c.H + h) * psz + (r & (psz - 1))) * words;
                if (a.w_out)
                    a.w_out[bh * ((long)a.max_dst << a.c.page_log2) + r] = a.weights[bh * ((long)a.c.max_pages << a.c.page_log2) + src];
            }
        }
    }
    // a lane's words of K and V of all eight: the row of K, then that of V
    for (int x0 = 0; x0 < 2 * words; x0 += 32) {
        const int x = x0 + lane;
        const bool in = x < 2 * words, in_k = x < words;
        const WORD *src = (const WORD *)(in_k ? a.c.k : a.c.v) + (in_k ? x : x - words);
        WORD *dst = (WORD *)(in_k ? a.k_dst : a.v_dst) + (in_k ? x : x - words);
        WORD v[CPW];
#pragma unroll
        for (int j = 0; j < CPW; ++j) {
            const long at = __shfl_sync(0xffffffffu, s, j);
            const bool go = __shfl_sync(0xffffffffu, d, j) >= 0;
            if (in && go) v[j] = src[at];
        }
#pragma unroll
        for (int j = 0; j < CPW; ++j) {
            const long at = __shfl_sync(0xffffffffu, d, j);
            if (in && at >= 0) dst[at] = v[j];
        }
    }
}

}  // namespace

size_t paged_evict_bytes(int B, int H, int budget) { return (size_t)B * H * budget * sizeof(int); }

cudaError_t launch_paged_evict(const PagedEvictArgs &a, bool bf16, cudaStream_t s)
{
    const long bh = (long)a.B * a.c.H;
    if (bh == 0) return cudaSuccess;
    const long blocks = (bh * ((a.budget + CPW - 1) / CPW) + 7) / 8;
    if (bh > 0x0fffffffL || blocks > 0x7fffffffL) return cudaErrorNotSupported;
    int *kept = a.kept ? a.kept : (int *)a.ws;
    cudaError_t e = allow_shared((const void *)evict_choose_kernel, CHOOSE_SMEM, g_shared);
    if (e != cudaSuccess) return e;
    const int cap = a.c.max_pages << a.c.page_log2;
    const int nblk = cap > 8 * ST && bh * 2 <= device_sms() ? 2 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(bh * nblk));
    cfg.blockDim = dim3(ST);
    cfg.dynamicSmemBytes = (size_t)(std::min((cap + nblk - 1) / nblk, KEEP) + 2 * BINS) * 4;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)nblk;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, evict_choose_kernel, a, kept)) != cudaSuccess) return e;
    note_launch();
    const int row = a.c.d * (bf16 ? 2 : 4);
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    e = row % 16 == 0 ? cudaLaunchKernelEx(&cfg, evict_copy_kernel<uint4>, a, (const int *)kept, row / 16)
                      : cudaLaunchKernelEx(&cfg, evict_copy_kernel<uint16_t>, a, (const int *)kept, row / 2);
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace hlta
