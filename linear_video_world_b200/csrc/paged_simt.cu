// Attention of a chunk over a paged cache on the CUDA cores: the HLTA_FP32 element type's path for
// more than a few rows (full single precision throughout), and its accumulated attention weights.
//
// Exact softmax by 64-key tiles with a running maximum and sum (log2 domain). A block of 256 threads
// owns 64 packed rows of one key head and walks the key tiles of a share of the keys those rows see
// (grid z); with more than one share, each leaves (maximum, sum, unnormalised output) in the
// workspace and a second kernel joins them in the order of the shares.
// Bound by shared-memory reads: a thread forms 4 rows x 4 keys of scores (eight 16-byte reads
// per 64 multiply-adds) and 4 rows x 8 channels of output (twelve per 128), 12000 wavefronts a tile of
// 64 x 64 against 8192 cycles of multiply-adds; 16 threads share a row,
// so its maximum and sum stay inside half a warp and P inside a warp. Tiles are copied
// asynchronously into two stages, one ahead. (A first form, 16 rows a block with tiles copied
// between two barriers, took 590 us where this takes 159: 2 x 200 rows of 8 heads over 700
// and 3000 keys of 2.)
// Positions outside the keys that the block's rows see are staged as zeros and masked, whatever
// the cache holds there.
#include "hlta_internal.cuh"
#include "paged.cuh"
#include "paged_f32.cuh"

#include <algorithm>
#include <cooperative_groups.h>
#include <math.h>

namespace hlta {
namespace {

using namespace paged;
using namespace f32;

constexpr int TM = 64, TN = 64, THREADS = 256;          // rows, keys, threads
constexpr int PST = TN + 4;                             // row stride of P
std::atomic<unsigned long long> g_shared{0}, g_shared_w{0};

__device__ __forceinline__ float half_max(float x)
{
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float half_sum(float x)
{
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 pa, pb, pc, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
        "mov.b64 pc, {%6, %7};\n\tfma.rn.f32x2 pd, pa, pb, pc;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// s[i][j] = row (4 rg + i) . key (kg + 16 j): even and odd pairs of channels in the two halves of a
// two-wide multiply-add
__device__ __forceinline__ void scores(const float *Q, const float *K, int st, int dp, int rg, int kg, float (&s)[4][4])
{
    float2 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int x = 0; x < dp; x += 4) {
        float4 q[4], k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = *(const float4 *)(Q + (4 * rg + i) * st + x);
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = *(const float4 *)(K + (kg + 16 * j) * st + x);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = ffma2(make_float2(q[i].x, q[i].y), make_float2(k[j].x, k[j].y), acc[i][j]);
                acc[i][j] = ffma2(make_float2(q[i].z, q[i].w), make_float2(k[j].z, k[j].w), acc[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = acc[i][j].x + acc[i][j].y;
}

// rows [r0, r0 + TM) of the head group's queries, asynchronously; rows that are none, and channels from d to dp, as zeros
__device__ __forceinline__ void copy_q(const PagedAttnArgs &a, const FastDiv &byL, const Roll &ro, long head, int R, int r0, float *Q, int st, int dp)
{
    const int per = dp >> 2, d = a.c.d;
    const bool words = (d & 3) == 0;
#pragma unroll 4
    for (int e = threadIdx.x; e < TM * per; e += THREADS) {
        const int r = e / per, x = 4 * (e - r * per);
        const bool in = r0 + r < R && frem(r0 + r, byL) < ro.n;
        const float *src = (const float *)a.q + (in ? (head * R + r0 + r) * d + x : 0);
        float *dst = Q + r * st + x;
        if (words) {
            copy16(dst, src, in);
        } else {
            for (int y = 0; y < 4; ++y) {
                const bool ch = in && x + y < d;
                copy4(dst + y, ch ? src + y : (const float *)a.q, ch);
            }
        }
    }
}

// the span of the live rows among packed rows [r0, r0 + TM): see the chunk kernel
__device__ __forceinline__ Span rows_span(const Roll &ro, const FastDiv &byL, const Mask &mask, int r0, int R)
{
    const int L = (int)byL.d, r1 = min(r0 + TM, R);
    int i0 = frem(r0, byL), i1 = i0 + (r1 - 1 - r0);
    if (i1 >= L) {
        i0 = 0;
        i1 = L - 1;
    }
    if (i0 >= ro.n) return Span{0, 0};
    const Span s{span_of(ro, i0, mask).lo, span_of(ro, min(i1, ro.n - 1), mask).hi};
    return s.hi > s.lo ? s : Span{0, 0};
}

__global__ void __launch_bounds__(THREADS) paged_attn_f32_kernel(PagedAttnArgs a, FastDiv byL, Mask mask, int nsplit, float *ws_m, float *ws_l, float *ws_o)
{
    extern __shared__ __align__(16) float smem[];
    const int d = a.c.d, dp = (d + 3) & ~3, st = dp + 4;
    float *Q = smem, *KV = Q + TM * st, *P = KV + 4 * TN * st;          // K and V of two stages
    const int rg = threadIdx.x >> 4, kg = threadIdx.x & 15;
    const int h = blockIdx.y % a.c.H, b = blockIdx.y / a.c.H, R = a.G * (int)a.L, r0 = blockIdx.x * TM;
    const Roll ro = roll_of(a.c.kv_lens, a.new_lens, b, (int)a.L, a.c.max_pages << a.c.page_log2);
    if (ro.bad && threadIdx.x == 0) atomicOr(a.c.err, DEVERR_TABLE);
    const Span u = rows_span(ro, byL, mask, r0, R);
    const int t_lo = u.lo / TN, nt = u.hi > u.lo ? (u.hi + TN - 1) / TN - t_lo : 0;
    const int ta = t_lo + (int)((long)nt * blockIdx.z / nsplit), tb = t_lo + (int)((long)nt * (blockIdx.z + 1) / nsplit);
    Span sp[4];
    bool live[4];
    float m[4], l[4];
    float2 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * rg + i, tok = frem(r, byL);
        live[i] = r < R && tok < ro.n;
        sp[i] = live[i] ? span_of(ro, tok, mask) : Span{0, 0};
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[i][x] = make_float2(0.f, 0.f);
    }
    auto load = [&](int t) {
        float *k = KV + (t & 1) * 2 * TN * st;
        copy_tile<TN, THREADS>(a.c, b, h, t * TN, u, k, k + TN * st, st, dp);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (tb > ta) {
        copy_q(a, byL, ro, blockIdx.y, R, r0, Q, st, dp);
        load(ta);
    }
    for (int t = ta; t < tb; ++t) {
        if (t + 1 < tb) {
            load(t + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const float *K = KV + (t & 1) * 2 * TN * st, *V = K + TN * st;
        float s[4][4];
        scores(Q, K, st, dp, rg, kg, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = t * TN + kg + 16 * j;
                s[i][j] = p < sp[i].lo || p >= sp[i].hi ? -INFINITY : s[i][j] * a.sl2;
            }
            const float mn = fmaxf(m[i], half_max(fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]))));
            const float base = mn == -INFINITY ? 0.f : mn, f = exp2f(m[i] - base);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - base);
                sum += p;
                P[(4 * rg + i) * PST + kg + 16 * j] = p;
            }
            l[i] = fmaf(l[i], f, sum);              // this thread's keys; joined at the end
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                acc[i][x].x *= f;
                acc[i][x].y *= f;
            }
        }
        __syncwarp();
        if (4 * kg < dp) {
            const bool second = 64 + 4 * kg < dp;
#pragma unroll 2
            for (int k = 0; k < TN; k += 4) {
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = *(const float4 *)(P + (4 * rg + i) * PST + k);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const float4 v0 = *(const float4 *)(V + (k + kk) * st + 4 * kg);
                    const float4 v1 = second ? *(const float4 *)(V + (k + kk) * st + 64 + 4 * kg) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                        const float2 ww = make_float2(w, w);
                        acc[i][0] = ffma2(ww, make_float2(v0.x, v0.y), acc[i][0]);
                        acc[i][1] = ffma2(ww, make_float2(v0.z, v0.w), acc[i][1]);
                        acc[i][2] = ffma2(ww, make_float2(v1.x, v1.y), acc[i][2]);
                        acc[i][3] = ffma2(ww, make_float2(v1.z, v1.w), acc[i][3]);
                    }
                }
            }
        }
        __syncthreads();
    }
    const long rows = (long)a.B * a.c.H * R;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float sum = half_sum(l[i]);
        if (!live[i]) continue;
        const long row = (long)blockIdx.y * R + r0 + 4 * rg + i;
        const float inv = nsplit > 1 ? 1.f : sum > 0.f ? 1.f / sum : sum == sum ? 0.f : sum;
        float *dst = nsplit > 1 ? ws_o + (blockIdx.z * rows + row) * d : (float *)a.o + row * d;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int ch = (x >> 2) * 64 + 4 * kg + (x & 3);
            if (ch < d) dst[ch] = ((x & 1) ? acc[i][x >> 1].y : acc[i][x >> 1].x) * inv;
        }
        if (kg == 0) {
            if (nsplit > 1) {
                ws_m[blockIdx.z * rows + row] = m[i];
                ws_l[blockIdx.z * rows + row] = sum;
            } else if (a.lse) {
                a.lse[row] = (m[i] + log2f(sum)) * 0.69314718055994531f;
            }
        }
    }
}

// Joins the shares of a row, one warp per row.
__global__ void __launch_bounds__(128) paged_join_f32_kernel(PagedAttnArgs a, FastDiv byL, int nsplit, const float *ws_m, const float *ws_l, const float *ws_o)
{
    const int lane = threadIdx.x & 31;
    const long R = a.G * a.L, rows = (long)a.B * a.c.H * R;
    const long row = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int b = (int)(row / (a.c.H * R)), i = frem((int)(row % R), byL), d = a.c.d;
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
        if (lane + 32 * x < d) ((float *)a.o)[row * d + lane + 32 * x] = acc[x] * inv;
    if (a.lse && lane == 0) a.lse[row] = (m + log2f(l)) * 0.69314718055994531f;
}

// Accumulated attention weights: 64 keys of one key head, and over every row of the head group that
// sees them the sum of 2^(score - lse). A cluster of one to eight blocks (grid z) shares those keys, each
// with every nz-th block of 64 rows, copied asynchronously one ahead; a thread sums its four keys over
// its four rows of each, and the 16 threads of a key and the blocks are joined at the end in a fixed
// order. (One block for all rows, copied word by word between two barriers: 1600 rows over 381 keys, the
// whole call, 287 us for 56.)
__global__ void __launch_bounds__(THREADS) paged_weights_f32_kernel(PagedAttnArgs a, FastDiv byL, Mask mask)
{
    extern __shared__ __align__(16) float smem[];
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int nz = (int)gridDim.z, z = (int)blockIdx.z;
    const int d = a.c.d, dp = (d + 3) & ~3, st = dp + 4;
    float *K = smem, *Qs = K + TN * st, *Sum = Qs + 2 * TM * st;        // Q of two stages; Sum: [16 row groups][64 keys]
    __shared__ float total[TN];
    const int rg = threadIdx.x >> 4, kg = threadIdx.x & 15;
    const int h = blockIdx.y % a.c.H, b = blockIdx.y / a.c.H, cap = a.c.max_pages << a.c.page_log2, p0 = blockIdx.x * TN;
    const Roll ro = roll_of(a.c.kv_lens, a.new_lens, b, (int)a.L, cap);
    if (p0 >= ro.kv) return;                    // the whole cluster alike
    const int R = a.G * (int)a.L, nrb = (R + TM - 1) / TM;
    // this block's next block of rows from rb that sees some of the keys: all threads alike
    auto seen = [&](int rb) {
        for (; rb < nrb; rb += nz) {
            const Span u = rows_span(ro, byL, mask, rb * TM, R);
            if (u.lo < p0 + TN && u.hi > p0) break;
        }
        return rb;
    };
    int rb = seen(z), stage = 0;
    if (rb < nrb) {
        // no position outside what the chunk's rows see: their pages may be gone
        const Span u{span_of(ro, 0, mask).lo, span_of(ro, ro.n - 1, mask).hi};
        copy_tile<TN, THREADS>(a.c, b, h, p0, u, K, nullptr, st, dp);
        copy_q(a, byL, ro, blockIdx.y, R, rb * TM, Qs, st, dp);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    while (rb < nrb) {
        const int next = seen(rb + nz);
        if (next < nrb) {
            copy_q(a, byL, ro, blockIdx.y, R, next * TM, Qs + (stage ^ 1) * TM * st, st, dp);
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        float lse[4];
        Span v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = rb * TM + 4 * rg + i, tok = frem(r, byL);
            const bool in = r < R && tok < ro.n;
            v[i] = in ? span_of(ro, tok, mask) : Span{0, 0};
            lse[i] = in ? a.lse[(long)blockIdx.y * R + r] * 1.4426950408889634f : 0.f;
        }
        __syncthreads();
        float s[4][4];
        scores(Qs + stage * TM * st, K, st, dp, rg, kg, s);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = p0 + kg + 16 * j;
                if (p >= v[i].lo && p < v[i].hi) sum[j] += exp2f(fmaf(s[i][j], a.sl2, -lse[i]));
            }
        __syncthreads();
        rb = next;
        stage ^= 1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) Sum[rg * TN + kg + 16 * j] = sum[j];
    __syncthreads();
    if (threadIdx.x < TN) {
        float t = 0.f;
        for (int g = 0; g < 16; ++g) t += Sum[g * TN + threadIdx.x];
        total[threadIdx.x] = t;
    }
    if (nz > 1) cluster.sync();
    const int p = p0 + threadIdx.x;
    if (z == 0 && threadIdx.x < TN && p < ro.kv) {
        float t = total[threadIdx.x];
        for (int o = 1; o < nz; ++o) t += cluster.map_shared_rank(total, o)[threadIdx.x];
        const long at = (long)blockIdx.y * cap + p;
        if (a.w_in && p < ro.h) t = fmaf(a.decay, a.w_in[at], t);
        a.w_out[at] = t;
    }
    if (nz > 1) cluster.sync();                 // no block ends while its sums are read
}

// shares of the keys: enough blocks for two rounds of the SMs, no share under two tiles
int splits_of(int B, int Hkv, long R, int max_keys)
{
    const long blocks = (long)B * Hkv * ((R + TM - 1) / TM);
    const long want = (148L * 2 + blocks - 1) / std::max(blocks, 1L);
    return (int)std::max(1L, std::min({want, (long)(max_keys + 2 * TN - 1) / (2 * TN), 64L}));
}

}  // namespace

size_t paged_attn_simt_bytes(int B, int Hq, int Hkv, long L, int d, int max_keys)
{
    const long rows = (long)B * Hq * L;
    const int ns = splits_of(B, Hkv, (Hq / Hkv) * L, max_keys);
    return ns > 1 ? (size_t)ns * rows * (d + 2) * 4 : 0;
}

cudaError_t launch_paged_attn_simt(const PagedAttnArgs &a, cudaStream_t s)
{
    const long R = a.G * a.L, rows = (long)a.B * a.c.H * R;
    const int ns = splits_of(a.B, a.c.H, R, a.c.max_pages << a.c.page_log2), st = ((a.c.d + 3) & ~3) + 4;
    if (R < 1) return cudaSuccess;
    if (R > (1L << 30) || (long)a.B * a.c.H > 65535 || (rows + 3) / 4 > 0x7fffffffL) return cudaErrorNotSupported;
    float *m = (float *)a.ws, *l = m + ns * rows, *o = l + ns * rows;
    cudaError_t e = allow_shared((const void *)paged_attn_f32_kernel, (size_t)((TM + 4 * TN) * 132 + TM * PST) * 4, g_shared);
    if (e != cudaSuccess) return e;
    const FastDiv byL = fast_div((unsigned)a.L);
    const dim3 grid((unsigned)((R + TM - 1) / TM), (unsigned)(a.B * a.c.H), (unsigned)ns);
    paged_attn_f32_kernel<<<grid, THREADS, (size_t)((TM + 4 * TN) * st + TM * PST) * 4, s>>>(a, byL, mask_of(a.N, a.w), ns, m, l, o), note_launch();
    if (ns > 1) paged_join_f32_kernel<<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(a, byL, ns, m, l, o), note_launch();
    return cudaGetLastError();
}

cudaError_t launch_paged_weights_simt(const PagedAttnArgs &a, cudaStream_t s)
{
    const int keys = a.c.max_pages << a.c.page_log2, st = ((a.c.d + 3) & ~3) + 4;
    const long heads = (long)a.B * a.c.H, nrb = (a.G * a.L + TM - 1) / TM;
    if (heads > 65535) return cudaErrorNotSupported;
    cudaError_t e = allow_shared((const void *)paged_weights_f32_kernel, (size_t)((2 * TM + TN) * 132 + 16 * TN) * 4, g_shared_w);
    if (e != cudaSuccess) return e;
    // blocks per key tile: while the SMs have room (two fit one) and each has two blocks of rows
    const long tiles = heads * ((keys + TN - 1) / TN);
    unsigned nz = 1;
    while (nz < 8 && tiles * nz * 2 <= 2L * device_sms() && nrb >= 4L * nz) nz *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((keys + TN - 1) / TN), (unsigned)heads, nz);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = (size_t)((2 * TM + TN) * st + 16 * TN) * 4;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = nz;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, paged_weights_f32_kernel, a, fast_div((unsigned)std::max(a.L, 1L)), mask_of(a.N, a.w));
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace hlta
