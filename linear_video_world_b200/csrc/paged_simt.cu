// Attention of a chunk over a paged cache on the CUDA cores: the HLTA_FP32 element type's path
// (full single precision throughout), with the accumulated attention weights.
//
// Exact softmax by tiles with a running maximum and sum (log2 domain). A block of four warps owns
// 16 packed rows of one key head and walks the 64-key tiles of a share of the keys those rows see
// (grid z); with more than one share, each leaves (maximum, sum, unnormalised output) in the
// workspace and a second kernel joins them in the order of the shares. Scores: a lane owns two
// keys and four rows, K rows padded by one 16-byte word so that the lanes' vector reads fall in
// different banks: six 16-byte shared reads per 32 multiply-adds. Output: a lane owns four
// channels, two reads per 16 multiply-adds.
// Positions outside the keys that the block's rows see are staged as zeros and masked, whatever
// the cache holds there.
#include "hlta_internal.cuh"
#include "paged.cuh"

#include <algorithm>
#include <math.h>

namespace hlta {
namespace {

using namespace paged;

constexpr int QB = 16, KT = 64, THREADS = 128, RPW = 4;   // rows, keys, threads, rows per warp

__device__ __forceinline__ float warp_max(float x)
{
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float warp_sum(float x)
{
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// [rows][d] of the cache from position p0 on into shared memory, row stride `st` floats, channels
// from d to dp and positions outside [lo, hi) as zeros
template <typename E>
__device__ __forceinline__ void stage(const PagedKV &c, const void *pages, int b, int h, int p0, int lo, int hi,
                                      float *dst, int st, int dp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int j = warp; j < KT; j += THREADS / 32) {
        const int p = p0 + j;
        const bool in = p >= lo && p < hi;
        const E *src = nullptr;
        if (in) {
            const int psz = 1 << c.page_log2;
            src = (const E *)pages + (((long)page_of(c, b, p) * c.H + h) * psz + (p & (psz - 1))) * c.d;
        }
        for (int x = lane; x < dp; x += 32) dst[j * st + x] = in && x < c.d ? to_f(src[x]) : 0.f;
    }
}

template <typename E>
__global__ void __launch_bounds__(THREADS) paged_attn_kernel(PagedAttnArgs a, Mask mask, int nsplit, float *ws_m, float *ws_l, float *ws_o)
{
    extern __shared__ float smem[];
    const int d = a.c.d, dp = (d + 3) & ~3, kst = dp + 4;
    float *Qs = smem;                       // [QB][dp]
    float *Ks = Qs + QB * dp;               // [KT][dp + 4]
    float *Vs = Ks + KT * kst;              // [KT][dp]
    float *Ps = Vs + KT * dp;               // per warp [KT][RPW]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.y % a.c.H, b = blockIdx.y / a.c.H;
    const int R = a.G * (int)a.L;
    const int r0 = blockIdx.x * QB;
    const long row0 = (long)blockIdx.y * R + r0;
    const Roll ro = roll_of(a.c.kv_lens, a.new_lens, b, (int)a.L, a.c.max_pages << a.c.page_log2);
    if (ro.bad && threadIdx.x == 0) atomicOr(a.c.err, DEVERR_TABLE);

    // the block's rows, and the keys that any of them sees
    Span sp[RPW];
    bool live[RPW];
    int lo = 0x7fffffff, hi = 0;
    for (int r = 0; r < QB; ++r) {
        const int i = (r0 + r) % (int)a.L;
        if (r0 + r >= R || i >= ro.n) continue;
        const Span s = span_of(ro, i, mask);
        if (s.hi > s.lo) {
            lo = min(lo, s.lo);
            hi = max(hi, s.hi);
        }
    }
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        const int rr = r0 + warp * RPW + r, i = rr % (int)a.L;
        live[r] = rr < R && i < ro.n;
        sp[r] = live[r] ? span_of(ro, i, mask) : Span{0, 0};
    }
    const int t_lo = hi > lo ? lo / KT : 0, nt = hi > lo ? (hi + KT - 1) / KT - t_lo : 0;
    const int ta = t_lo + (int)((long)nt * blockIdx.z / nsplit), tb = t_lo + (int)((long)nt * (blockIdx.z + 1) / nsplit);

    for (int e = threadIdx.x; e < QB * dp; e += THREADS) {
        const int r = e / dp, x = e % dp;
        Qs[e] = r0 + r < R && x < d ? to_f(((const E *)a.q)[(row0 + r) * d + x]) * a.sl2 : 0.f;
    }
    float m[RPW], l[RPW], acc[RPW][4];
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        for (int x = 0; x < 4; ++x) acc[r][x] = 0.f;
    }
    float *P = Ps + warp * KT * RPW;
    for (int t = ta; t < tb; ++t) {
        const int p0 = t * KT;
        __syncthreads();
        stage<E>(a.c, a.c.k, b, h, p0, lo, hi, Ks, kst, dp);
        stage<E>(a.c, a.c.v, b, h, p0, lo, hi, Vs, dp, dp);
        __syncthreads();
        float s[RPW][2];
#pragma unroll
        for (int r = 0; r < RPW; ++r) s[r][0] = s[r][1] = 0.f;
        const float *k0 = Ks + lane * kst, *k1 = Ks + (lane + 32) * kst, *q = Qs + warp * RPW * dp;
        for (int x = 0; x < dp; x += 4) {
            const float4 a0 = *(const float4 *)(k0 + x), a1 = *(const float4 *)(k1 + x);
#pragma unroll
            for (int r = 0; r < RPW; ++r) {
                const float4 v = *(const float4 *)(q + r * dp + x);
                s[r][0] = fmaf(v.x, a0.x, fmaf(v.y, a0.y, fmaf(v.z, a0.z, fmaf(v.w, a0.w, s[r][0]))));
                s[r][1] = fmaf(v.x, a1.x, fmaf(v.y, a1.y, fmaf(v.z, a1.z, fmaf(v.w, a1.w, s[r][1]))));
            }
        }
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
            const int pa = p0 + lane, pb = pa + 32;
            if (pa < sp[r].lo || pa >= sp[r].hi) s[r][0] = -INFINITY;
            if (pb < sp[r].lo || pb >= sp[r].hi) s[r][1] = -INFINITY;
            const float mn = fmaxf(m[r], warp_max(fmaxf(s[r][0], s[r][1])));
            const float base = mn == -INFINITY ? 0.f : mn;
            const float p_a = exp2f(s[r][0] - base), p_b = exp2f(s[r][1] - base), f = exp2f(m[r] - base);
            l[r] = l[r] * f + warp_sum(p_a + p_b);
            m[r] = mn;
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[r][x] *= f;
            P[lane * RPW + r] = p_a;
            P[(lane + 32) * RPW + r] = p_b;
        }
        __syncwarp();
        if (lane * 4 < dp) {
#pragma unroll 4
            for (int j = 0; j < KT; ++j) {
                const float4 p = *(const float4 *)(P + j * RPW);
                const float4 v = *(const float4 *)(Vs + j * dp + lane * 4);
                const float pr[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int r = 0; r < RPW; ++r) {
                    acc[r][0] = fmaf(pr[r], v.x, acc[r][0]);
                    acc[r][1] = fmaf(pr[r], v.y, acc[r][1]);
                    acc[r][2] = fmaf(pr[r], v.z, acc[r][2]);
                    acc[r][3] = fmaf(pr[r], v.w, acc[r][3]);
                }
            }
        }
        __syncwarp();
    }
    const long rows = (long)a.B * a.c.H * R;
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        if (!live[r]) continue;
        const long row = row0 + warp * RPW + r;
        if (nsplit == 1) {
            const float inv = l[r] > 0.f ? 1.f / l[r] : l[r] == l[r] ? 0.f : l[r];
            for (int x = 0; x < 4; ++x)
                if (lane * 4 + x < d) put((E *)a.o + row * d + lane * 4 + x, acc[r][x] * inv);
            if (a.lse && lane == 0) a.lse[row] = (m[r] + log2f(l[r])) * 0.69314718055994531f;
        } else {
            const long at = blockIdx.z * rows + row;
            for (int x = 0; x < 4; ++x)
                if (lane * 4 + x < d) ws_o[at * d + lane * 4 + x] = acc[r][x];
            if (lane == 0) {
                ws_m[at] = m[r];
                ws_l[at] = l[r];
            }
        }
    }
}

// Joins the shares of a row, one warp per row.
template <typename E>
__global__ void __launch_bounds__(THREADS) paged_join_kernel(PagedAttnArgs a, int nsplit, const float *ws_m, const float *ws_l, const float *ws_o)
{
    const int lane = threadIdx.x & 31;
    const long rows = (long)a.B * a.c.H * a.G * a.L;
    const long row = (long)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int b = (int)(row / ((long)a.c.H * a.G * a.L)), i = (int)(row % a.L), d = a.c.d;
    const Roll ro = roll_of(a.c.kv_lens, a.new_lens, b, (int)a.L, a.c.max_pages << a.c.page_log2);
    if (i >= ro.n) return;
    float m = -INFINITY;
    for (int s = 0; s < nsplit; ++s) m = fmaxf(m, ws_m[s * rows + row]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < nsplit; ++s) {
        const long at = s * rows + row;
        const float f = exp2f(ws_m[at] - base);
        l = fmaf(ws_l[at], f, l);
        for (int x = 0; x < 4; ++x)
            if (lane + 32 * x < d) acc[x] = fmaf(ws_o[at * d + lane + 32 * x], f, acc[x]);
    }
    const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;
    for (int x = 0; x < 4; ++x)
        if (lane + 32 * x < d) put((E *)a.o + row * d + lane + 32 * x, acc[x] * inv);
    if (a.lse && lane == 0) a.lse[row] = (m + log2f(l)) * 0.69314718055994531f;
}

// Accumulated attention weights: a block owns 64 keys of one key head and sums, over every row of
// the head group that sees them, 2^(score - lse) in the order of the rows; each warp takes every
// fourth group of four rows, and the four partial sums are joined at the end.
template <typename E>
__global__ void __launch_bounds__(THREADS) paged_weights_kernel(PagedAttnArgs a, Mask mask)
{
    extern __shared__ float smem[];
    const int d = a.c.d, dp = (d + 3) & ~3, kst = dp + 4;
    float *Ks = smem;                       // [KT][dp + 4]
    float *Qs = Ks + KT * kst;              // [QB][dp]
    float *Sum = Qs + QB * dp;              // [warps][KT]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.y % a.c.H, b = blockIdx.y / a.c.H;
    const int cap = a.c.max_pages << a.c.page_log2;
    const Roll ro = roll_of(a.c.kv_lens, a.new_lens, b, (int)a.L, cap);
    const int p0 = blockIdx.x * KT;
    if (p0 >= ro.kv) return;
    const int R = a.G * (int)a.L;
    const long row0 = (long)blockIdx.y * R;
    stage<E>(a.c, a.c.k, b, h, p0, 0, ro.n > 0 ? ro.kv : 0, Ks, kst, dp);
    float sum[2] = {0.f, 0.f};
    for (int rb = 0; rb < R; rb += QB) {
        // a block of rows that sees none of these keys is skipped by all threads
        bool any = false;
        for (int r = rb; r < min(R, rb + QB); ++r) {
            const int i = r % (int)a.L;
            const Span s = i < ro.n ? span_of(ro, i, mask) : Span{0, 0};
            any = any || (s.lo < p0 + KT && s.hi > p0 && s.hi > s.lo);
        }
        if (!any) continue;
        __syncthreads();
        for (int e = threadIdx.x; e < QB * dp; e += THREADS) {
            const int r = e / dp, x = e % dp;
            Qs[e] = rb + r < R && x < d ? to_f(((const E *)a.q)[(row0 + rb + r) * d + x]) * a.sl2 : 0.f;
        }
        __syncthreads();
        float s[RPW][2];
#pragma unroll
        for (int r = 0; r < RPW; ++r) s[r][0] = s[r][1] = 0.f;
        const float *k0 = Ks + lane * kst, *k1 = Ks + (lane + 32) * kst, *q = Qs + warp * RPW * dp;
        for (int x = 0; x < dp; x += 4) {
            const float4 a0 = *(const float4 *)(k0 + x), a1 = *(const float4 *)(k1 + x);
#pragma unroll
            for (int r = 0; r < RPW; ++r) {
                const float4 v = *(const float4 *)(q + r * dp + x);
                s[r][0] = fmaf(v.x, a0.x, fmaf(v.y, a0.y, fmaf(v.z, a0.z, fmaf(v.w, a0.w, s[r][0]))));
                s[r][1] = fmaf(v.x, a1.x, fmaf(v.y, a1.y, fmaf(v.z, a1.z, fmaf(v.w, a1.w, s[r][1]))));
            }
        }
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
            const int rr = rb + warp * RPW + r, i = rr % (int)a.L;
            if (rr >= R || i >= ro.n) continue;
            const Span v = span_of(ro, i, mask);
            if (v.hi <= v.lo) continue;
            const float z = a.lse[row0 + rr] * 1.4426950408889634f;
            const int pa = p0 + lane, pb = pa + 32;
            if (pa >= v.lo && pa < v.hi) sum[0] += exp2f(s[r][0] - z);
            if (pb >= v.lo && pb < v.hi) sum[1] += exp2f(s[r][1] - z);
        }
    }
    Sum[warp * KT + lane] = sum[0];
    Sum[warp * KT + lane + 32] = sum[1];
    __syncthreads();
    const int p = p0 + threadIdx.x;
    if (threadIdx.x < KT && p < ro.kv) {
        float t = 0.f;
        for (int w = 0; w < THREADS / 32; ++w) t += Sum[w * KT + threadIdx.x];
        const long at = (long)blockIdx.y * cap + p;
        if (a.w_in && p < ro.h) t = fmaf(a.decay, a.w_in[at], t);
        a.w_out[at] = t;
    }
}

// shares of the keys: enough blocks for four per SM, no share under two tiles
int splits_of(int B, int Hkv, long R, int max_keys)
{
    const long blocks = (long)B * Hkv * ((R + QB - 1) / QB);
    const long want = (148L * 4 + blocks - 1) / std::max(blocks, 1L);
    return (int)std::max(1L, std::min({want, (long)(max_keys + 2 * KT - 1) / (2 * KT), 64L}));
}

template <typename E>
cudaError_t run(const PagedAttnArgs &a, cudaStream_t s)
{
    const long R = a.G * a.L, rows = (long)a.B * a.c.H * R;
    const int keys = a.c.max_pages << a.c.page_log2;
    const int ns = splits_of(a.B, a.c.H, R, keys);
    const int dp = (a.c.d + 3) & ~3;
    if (R > (1L << 30) || (long)a.B * a.c.H > 65535) return cudaErrorNotSupported;
    float *m = (float *)a.ws, *l = m + ns * rows, *o = l + ns * rows;
    const size_t sm = (size_t)(QB * dp + KT * (dp + 4) + KT * dp + THREADS / 32 * KT * RPW) * 4;
    cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    if (e != cudaSuccess) return e;
    if (R > 0) {
        const dim3 grid((unsigned)((R + QB - 1) / QB), (unsigned)(a.B * a.c.H), (unsigned)ns);
        paged_attn_kernel<E><<<grid, THREADS, sm, s>>>(a, mask_of(a.N, a.w), ns, m, l, o), note_launch();
    }
    if (R > 0 && ns > 1) {
        const long blocks = (rows + THREADS / 32 - 1) / (THREADS / 32);
        if (blocks > 0x7fffffffL) return cudaErrorNotSupported;
        paged_join_kernel<E><<<(unsigned)blocks, THREADS, 0, s>>>(a, ns, m, l, o), note_launch();
    }
    return cudaGetLastError();
}

template <typename E>
cudaError_t run_weights(const PagedAttnArgs &a, cudaStream_t s)
{
    const int dp = (a.c.d + 3) & ~3, keys = a.c.max_pages << a.c.page_log2;
    if ((long)a.B * a.c.H > 65535) return cudaErrorNotSupported;
    const size_t sw = (size_t)(KT * (dp + 4) + QB * dp + THREADS / 32 * KT) * 4;
    cudaError_t e = cudaFuncSetAttribute(paged_weights_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sw);
    if (e != cudaSuccess) return e;
    paged_weights_kernel<E><<<dim3((unsigned)((keys + KT - 1) / KT), (unsigned)(a.B * a.c.H)), THREADS, sw, s>>>(a, mask_of(a.N, a.w)), note_launch();
    return cudaGetLastError();
}

}  // namespace

size_t paged_attn_simt_bytes(int B, int Hq, int Hkv, long L, int d, int max_keys)
{
    const long rows = (long)B * Hq * L;
    const int ns = splits_of(B, Hkv, (Hq / Hkv) * L, max_keys);
    return ns > 1 ? (size_t)ns * rows * (d + 2) * 4 : 0;
}

cudaError_t launch_paged_attn_simt(const PagedAttnArgs &a, cudaStream_t s) { return run<float>(a, s); }

cudaError_t launch_paged_weights_simt(const PagedAttnArgs &a, cudaStream_t s) { return run_weights<float>(a, s); }

}  // namespace hlta
