// Attention of a chunk over a paged cache on the CUDA cores: the HLTA_FP32 element type's path for
// more than a few rows (full single precision throughout), and its accumulated attention weights.
//
// Exact softmax by 64-key tiles with a running maximum and sum (log2 domain). The division of the
// work is that of paged.cuh with single blocks as gangs: a block of 256 threads takes 32, 64 or 128
// packed rows of a key head past its share of the key tiles; pieces of a head leave (maximum, sum,
// unnormalised output) in the workspace and a second kernel joins them.
// Bound by the multiply-adds and the shared-memory reads that feed them: eight lanes share a row (its
// maximum and sum stay inside the warp, and P too), four rows a warp at a time, so that every 16-byte
// read of a half-warp is one or two addresses of Q or P, or eight of K or V side by side. With four rows a thread
// 12 reads feed 128 multiply-adds of a score step and 20 feed 256 of an output step. Tiles are copied
// asynchronously, K one tile ahead (V too, where shared memory has room).
// Measured, 2 x 200 rows of 8 heads over 700 and 3000 keys of 2: 117 us (16 rows a block with tiles
// copied between two barriers 590; 4 rows x 4 keys a thread and equal shares of every head's keys 156).
// Positions outside the keys that the block's rows see are staged as zeros and masked, whatever
// the cache holds there.
#include "hlta_internal.cuh"
#include "paged.cuh"
#include "paged_f32.cuh"

#include <algorithm>
#include <cooperative_groups.h>
#include <math.h>
#include <type_traits>

namespace hlta {
namespace {

using namespace paged;
using namespace f32;

// A thread forms RW rows x 8 keys of scores and RW rows x 16 channels of output; a block has 32 RW rows.
constexpr int TN = 64, THREADS = 256, D = 128;          // keys, threads, channels at most
constexpr int PST = TN + 8;                             // row stride of P
constexpr int rows_of(int rw) { return 32 * rw; }
constexpr int v_stages(int rw) { return rw > 2 ? 1 : 2; }       // of V: two where shared memory has room
std::atomic<unsigned long long> g_shared[5], g_shared_w[5];

// over the eight lanes that share a row
__device__ __forceinline__ float row_max(float x)
{
    for (int o = 4; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum(float x)
{
    for (int o = 4; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
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

// s[i][j] = row 4 i of Q . key 8 j of K (both from this thread's first): even and odd pairs of channels in
// the two halves of a two-wide multiply-add
template <int RW>
__device__ __forceinline__ void scores(const float *Q, const float *K, int st, int dp, float (&s)[RW][8])
{
    float2 acc[RW][8];
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int x = 0; x < dp; x += 4) {
        float4 q[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) q[i] = *(const float4 *)(Q + 4 * i * st + x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 k = *(const float4 *)(K + 8 * j * st + x);
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                acc[i][j] = ffma2(make_float2(q[i].x, q[i].y), make_float2(k.x, k.y), acc[i][j]);
                acc[i][j] = ffma2(make_float2(q[i].z, q[i].w), make_float2(k.z, k.w), acc[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] = acc[i][j].x + acc[i][j].y;
}

// rows [r0, r0 + N) of the head group's queries, asynchronously; rows that are none, and channels from d to dp, as zeros
template <int N>
__device__ __forceinline__ void copy_q(const PagedAttnArgs &a, const FastDiv &byL, const Roll &ro, long head, int R, int r0, float *Q, int st, int dp)
{
    const int d = a.c.d, x = 4 * (threadIdx.x & 31);
    if (x >= dp) return;
    const bool words = (d & 3) == 0;
#pragma unroll 4
    for (int r = threadIdx.x >> 5; r < N; r += THREADS / 32) {
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

// the span of the live rows among packed rows [r0, r0 + n): see the chunk kernel
__device__ __forceinline__ Span rows_span(const Roll &ro, const FastDiv &byL, const Mask &mask, int r0, int n, int R)
{
    const int L = (int)byL.d, r1 = min(r0 + n, R);
    int i0 = frem(r0, byL), i1 = i0 + (r1 - 1 - r0);
    if (i1 >= L) {
        i0 = 0;
        i1 = L - 1;
    }
    if (i0 >= ro.n) return Span{0, 0};
    const Span s{span_of(ro, i0, mask).lo, span_of(ro, min(i1, ro.n - 1), mask).hi};
    return s.hi > s.lo ? s : Span{0, 0};
}

template <int RW>
__global__ void __launch_bounds__(THREADS) paged_attn_f32_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ Line line, float2 *ml, float *part)
{
    extern __shared__ __align__(16) float smem[];
    constexpr int TM = rows_of(RW);
    const int d = a.c.d, dp = (d + 3) & ~3, st = dp + 4;
    constexpr int VS = v_stages(RW);
    float *Q = smem, *Ks = Q + TM * st, *Vs = Ks + 2 * TN * st, *P = Vs + VS * TN * st;         // K of two stages
    const int warp = threadIdx.x >> 5, rl = (threadIdx.x & 31) >> 3, kl = threadIdx.x & 7;
    const int row0 = warp * 4 * RW + rl;                // this thread's rows: row0 + 4 i; its keys: kl + 8 j
    const int R = a.G * (int)a.L;
    __shared__ Place s_place;
    if (warp == 0) {
        const Place c = place_of<TN>(line, blockIdx.x);
        if ((threadIdx.x & 31) == 0) s_place = c;
    }
    __syncthreads();
    Place at = s_place;
    Piece<TN> x;
    for (int piece = 0; next_piece<TN>(line, at, x); ++piece) {
        const Roll &ro = x.x.r;
        const int b = x.b, h = x.h, r0 = x.pass * TM;
        const long head = (long)b * a.c.H + h;
        if (ro.bad && threadIdx.x == 0) atomicOr(a.c.err, DEVERR_TABLE);
        const Span u = rows_span(ro, line.byL, line.mask, r0, TM, R);
        const bool any = u.hi > u.lo;
        const int ta = any ? max(x.ta, u.lo / TN) : 0, tb = any ? min(x.tb, (u.hi + TN - 1) / TN) : 0;
        Span sp[RW];
        bool live[RW];
        float m[RW], l[RW];
        float2 acc[RW][8];                                  // channels 4 kl + 32 y + (0, 1), (2, 3)
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int r = r0 + row0 + 4 * i, tok = frem(r, line.byL);
            live[i] = r < R && tok < ro.n;
            sp[i] = live[i] ? span_of(ro, tok, line.mask) : Span{0, 0};
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int y = 0; y < 8; ++y) acc[i][y] = make_float2(0.f, 0.f);
        }
        PagedKV values = a.c;
        values.k = a.c.v;
        auto load_k = [&](int t) {                          // (and V, of two stages)
            float *k = Ks + (t & 1) * TN * st;
            if (t < tb) copy_tile<TN, THREADS>(a.c, b, h, t * TN, u, k, VS == 2 ? k + 2 * TN * st : nullptr, st, dp);
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto load_v = [&](int t) {                          // V of one stage
            if constexpr (VS == 1) {
                if (t < tb) copy_tile<TN, THREADS>(values, b, h, t * TN, u, Vs, nullptr, st, dp);
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
        };
        if (tb > ta) {
            copy_q<TM>(a, line.byL, ro, head, R, r0, Q, st, dp);
            load_k(ta);
            load_v(ta);
        }
        for (int t = ta; t < tb; ++t) {
            load_k(t + 1);                                  // its stage has been read
            asm volatile("cp.async.wait_group %0;" ::"n"(VS == 1 ? 2 : 1) : "memory");
            __syncthreads();
            float s[RW][8];
            scores<RW>(Q + row0 * st, Ks + (t & 1) * TN * st + kl * st, st, dp, s);
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int p = t * TN + kl + 8 * j;
                    s[i][j] = p < sp[i].lo || p >= sp[i].hi ? -INFINITY : s[i][j] * a.sl2;
                    mx = fmaxf(mx, s[i][j]);
                }
                const float mn = fmaxf(m[i], row_max(mx));
                const float base = mn == -INFINITY ? 0.f : mn, f = exp2f(m[i] - base);
                m[i] = mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = exp2f(s[i][j] - base);
                    sum += p;
                    P[(row0 + 4 * i) * PST + kl + 8 * j] = p;
                }
                l[i] = fmaf(l[i], f, sum);                  // this thread's keys; joined at the end
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    acc[i][x].x *= f;
                    acc[i][x].y *= f;
                }
            }
            if constexpr (VS == 1) {
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                __syncthreads();
            } else {
                __syncwarp();
            }
            const float *V = VS == 1 ? Vs : Vs + (t & 1) * TN * st;
            auto outputs = [&](auto full) {
#pragma unroll 2
                for (int k = 0; k < TN; k += 4) {
                    float4 p[RW];
#pragma unroll
                    for (int i = 0; i < RW; ++i) p[i] = *(const float4 *)(P + (row0 + 4 * i) * PST + k);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            if (!decltype(full)::value && 32 * y + 4 * kl >= dp) continue;
                            const float4 v = *(const float4 *)(V + (k + kk) * st + 32 * y + 4 * kl);
#pragma unroll
                            for (int i = 0; i < RW; ++i) {
                                const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                                acc[i][2 * y] = ffma2(make_float2(w, w), make_float2(v.x, v.y), acc[i][2 * y]);
                                acc[i][2 * y + 1] = ffma2(make_float2(w, w), make_float2(v.z, v.w), acc[i][2 * y + 1]);
                            }
                        }
                }
            };
            if (dp == 128) outputs(std::true_type{});
            else outputs(std::false_type{});
            __syncthreads();
            load_v(t + 1);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        const long slot = (long)blockIdx.x * 2 + (piece == 0 ? 0 : 1);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const float sum = row_sum(l[i]);
            if (!live[i]) continue;
            const int rr = row0 + 4 * i;
            const long row = head * R + r0 + rr;
            const float inv = !x.whole ? 1.f : sum > 0.f ? 1.f / sum : sum == sum ? 0.f : sum;
            float *dst = x.whole ? (float *)a.o + row * d : part + (slot * TM + rr) * D;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int ch = 32 * y + 4 * kl;
                const float o[4] = {acc[i][2 * y].x * inv, acc[i][2 * y].y * inv, acc[i][2 * y + 1].x * inv, acc[i][2 * y + 1].y * inv};
                if ((d & 3) == 0) {
                    if (ch < d) *(float4 *)(dst + ch) = make_float4(o[0], o[1], o[2], o[3]);
                } else {
                    for (int z = 0; z < 4; ++z)
                        if (ch + z < d) dst[ch + z] = o[z];
                }
            }
            if (kl == 0) {
                if (!x.whole) ml[slot * TM + rr] = make_float2(m[i], sum);
                else if (a.lse) a.lse[row] = (m[i] + log2f(sum)) * 0.69314718055994531f;
            }
        }
    }
}

// Joins the pieces of heads whose keys were cut, in the order of the blocks, one warp per row; rows that
// see no key get zeros here.
__global__ void __launch_bounds__(128) paged_join_f32_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ Line line, int TM, const float2 *ml, const float *part)
{
    const int lane = threadIdx.x & 31, d = a.c.d;
    const long R = a.G * a.L, rows = (long)a.B * a.c.H * R, row = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int head = (int)(row / R), r = (int)(row % R), b = head / a.c.H, h = head % a.c.H, rr = r % TM;
    const Holders g = holders_of<TN>(line, r / TM, b, h);
    if (g.T > 0 && g.g0 == g.g1) return;
    const Roll ro = roll_of(a.c.kv_lens, a.new_lens, b, (int)a.L, line.cap);
    if (ro.bad && lane == 0) atomicOr(a.c.err, DEVERR_TABLE);
    if (frem(r, line.byL) >= ro.n) return;
    const int np = g.T > 0 ? g.g1 - g.g0 + 1 : 0;
    auto at = [&](int i) { return ((long)(g.g0 + i) * 2 + (i == 0 ? g.slot0 : 0)) * TM + rr; };
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = lane; i < np; i += 32) m = fmaxf(m, ml[at(i)].x);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    for (int i0 = 0; i0 < np; i0 += 32) {
        const float2 y = i0 + lane < np ? ml[at(i0 + lane)] : make_float2(-INFINITY, 0.f);
        const float f = exp2f(y.x - base);
        l = fmaf(y.y, f, l);
#pragma unroll 4
        for (int i = 0; i < min(32, np - i0); ++i) {
            const float w = __shfl_sync(0xffffffffu, f, i);
            const float *src = part + at(i0 + i) * D;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (lane + 32 * x < d) acc[x] = fmaf(src[lane + 32 * x], w, acc[x]);
        }
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;
    for (int x = 0; x < 4; ++x)
        if (lane + 32 * x < d) ((float *)a.o)[row * d + lane + 32 * x] = acc[x] * inv;
    if (a.lse && lane == 0) a.lse[row] = (m + log2f(l)) * 0.69314718055994531f;
}

// Accumulated attention weights: 64 keys of one key head, and over every row of the head group that
// sees them the sum of 2^(score - lse). A cluster of one to eight blocks (grid z) shares those keys, each
// with every nz-th block of 32 WRW rows (64 or 128), copied asynchronously one ahead; a thread sums eight
// keys over its WRW (two or four) rows of each, and the 32 threads of a key and the blocks are joined at
// the end in a fixed order. Bound like the attention by the multiply-adds of the scores, which are formed a
// second time, and the shared-memory reads that feed them. (One block for all rows, copied word by word
// between two barriers: 1600 rows over 381 keys, the whole call, 287 us for 56. 2 x 800 rows over 562 and
// 2736 keys of 4 heads: 299 us with the weights, 180 without.)
template <int WRW>
__global__ void __launch_bounds__(THREADS) paged_weights_f32_kernel(PagedAttnArgs a, FastDiv byL, Mask mask)
{
    extern __shared__ __align__(16) float smem[];
    constexpr int WTM = rows_of(WRW);
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int nz = (int)gridDim.z, z = (int)blockIdx.z;
    const int d = a.c.d, dp = (d + 3) & ~3, st = dp + 4;
    float *K = smem, *Qs = K + TN * st, *Sum = Qs + 2 * WTM * st;        // Q of two stages; Sum: [32 row groups][64 keys]
    __shared__ float total[TN];
    const int warp = threadIdx.x >> 5, rl = (threadIdx.x & 31) >> 3, kl = threadIdx.x & 7, row0 = warp * 4 * WRW + rl;
    const int h = blockIdx.y % a.c.H, b = blockIdx.y / a.c.H, cap = a.c.max_pages << a.c.page_log2, p0 = blockIdx.x * TN;
    const Roll ro = roll_of(a.c.kv_lens, a.new_lens, b, (int)a.L, cap);
    if (p0 >= ro.kv) return;                    // the whole cluster alike
    const int R = a.G * (int)a.L, nrb = (R + WTM - 1) / WTM;
    // this block's next block of rows from rb that sees some of the keys: all threads alike
    auto seen = [&](int rb) {
        for (; rb < nrb; rb += nz) {
            const Span u = rows_span(ro, byL, mask, rb * WTM, WTM, R);
            if (u.lo < p0 + TN && u.hi > p0) break;
        }
        return rb;
    };
    int rb = seen(z), stage = 0;
    if (rb < nrb) {
        // no position outside what the chunk's rows see: their pages may be gone
        const Span u{span_of(ro, 0, mask).lo, span_of(ro, ro.n - 1, mask).hi};
        copy_tile<TN, THREADS>(a.c, b, h, p0, u, K, nullptr, st, dp);
        copy_q<WTM>(a, byL, ro, blockIdx.y, R, rb * WTM, Qs, st, dp);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float sum[8] = {};
    while (rb < nrb) {
        const int next = seen(rb + nz);
        if (next < nrb) {
            copy_q<WTM>(a, byL, ro, blockIdx.y, R, next * WTM, Qs + (stage ^ 1) * WTM * st, st, dp);
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        float lse[WRW];
        Span v[WRW];
#pragma unroll
        for (int i = 0; i < WRW; ++i) {
            const int r = rb * WTM + row0 + 4 * i, tok = frem(r, byL);
            const bool in = r < R && tok < ro.n;
            v[i] = in ? span_of(ro, tok, mask) : Span{0, 0};
            lse[i] = in ? a.lse[(long)blockIdx.y * R + r] * 1.4426950408889634f : 0.f;
        }
        __syncthreads();
        float s[WRW][8];
        scores<WRW>(Qs + (stage * WTM + row0) * st, K + kl * st, st, dp, s);
#pragma unroll
        for (int i = 0; i < WRW; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int p = p0 + kl + 8 * j;
                if (p >= v[i].lo && p < v[i].hi) sum[j] += exp2f(fmaf(s[i][j], a.sl2, -lse[i]));
            }
        __syncthreads();
        rb = next;
        stage ^= 1;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) Sum[(4 * warp + rl) * TN + kl + 8 * j] = sum[j];
    __syncthreads();
    if (threadIdx.x < TN) {
        float t = 0.f;
        for (int g = 0; g < 32; ++g) t += Sum[g * TN + threadIdx.x];
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

// Rows of a thread: four (12 shared reads feed 128 multiply-adds) where that leaves three tiles a block,
// else two, or one for at most 32 rows, which divide small work more finely. 2 x 800 rows over 562 and 2736
// keys of 4 heads: 440, 261 and 181 us with one, two and four; 2 x 404 rows over 236 keys of 8 heads: 75, 55 and
// 52; 23 x 23 rows over 201 to 1271 keys of 2 heads: 60, 65 and 81.
int rw_of(int B, int Hkv, long R, int cap)
{
    const double tiles = (double)B * Hkv * ((cap + TN - 1) / TN) * ((R + 127) / 128);
    return R <= 32 ? 1 : tiles >= 3.0 * device_sms() ? 4 : 2;
}

size_t attn_smem(int rw, int st) { return (size_t)((rows_of(rw) + (2 + v_stages(rw)) * TN) * st + rows_of(rw) * PST) * 4; }
size_t weights_smem(int rw, int st) { return (size_t)((2 * rows_of(rw) + TN) * st + 32 * TN) * 4; }

}  // namespace

size_t paged_attn_simt_bytes(int B, int Hq, int Hkv, long L, int cap)
{
    return (size_t)device_sms() * 2 * rows_of(rw_of(B, Hkv, (Hq / Hkv) * L, cap)) * (D * 4 + 8);
}

cudaError_t launch_paged_attn_simt(const PagedAttnArgs &a, cudaStream_t s)
{
    const long R = a.G * a.L, rows = (long)a.B * a.c.H * R;
    const int rw = rw_of(a.B, a.c.H, R, a.c.max_pages << a.c.page_log2), tm = rows_of(rw), st = ((a.c.d + 3) & ~3) + 4, sms = device_sms();
    if (R < 1) return cudaSuccess;
    if (R > (1L << 30) || (long)a.B * a.c.H > 65535 || (rows + 3) / 4 > 0x7fffffffL) return cudaErrorNotSupported;
    float *part = (float *)a.ws;
    float2 *ml = (float2 *)(part + (size_t)sms * 2 * tm * D);
    auto *kernel = rw == 1 ? paged_attn_f32_kernel<1> : rw == 2 ? paged_attn_f32_kernel<2> : paged_attn_f32_kernel<4>;
    cudaError_t e = allow_shared((const void *)kernel, attn_smem(rw, 132), g_shared[rw]);
    if (e != cudaSuccess) return e;
    const Line line = line_of(a, 1, sms, (int)((R + tm - 1) / tm));
    kernel<<<sms, THREADS, attn_smem(rw, st), s>>>(a, line, ml, part), note_launch();
    paged_join_f32_kernel<<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(a, line, tm, ml, part), note_launch();
    return cudaGetLastError();
}

cudaError_t launch_paged_weights_simt(const PagedAttnArgs &a, cudaStream_t s)
{
    const int keys = a.c.max_pages << a.c.page_log2, st = ((a.c.d + 3) & ~3) + 4;
    const int rw = rw_of(a.B, a.c.H, a.G * a.L, keys) == 4 ? 4 : 2;
    const long heads = (long)a.B * a.c.H, nrb = (a.G * a.L + rows_of(rw) - 1) / rows_of(rw);
    if (heads > 65535) return cudaErrorNotSupported;
    auto *kernel = rw == 4 ? paged_weights_f32_kernel<4> : paged_weights_f32_kernel<2>;
    cudaError_t e = allow_shared((const void *)kernel, weights_smem(rw, 132), g_shared_w[rw]);
    if (e != cudaSuccess) return e;
    // blocks per key tile: while the SMs have room (two fit one) and each has two blocks of rows
    const long tiles = heads * ((keys + TN - 1) / TN);
    unsigned nz = 1;
    while (nz < 8 && tiles * nz * 2 <= 2L * device_sms() && nrb >= 4L * nz) nz *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((keys + TN - 1) / TN), (unsigned)heads, nz);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = weights_smem(rw, st);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = nz;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a, fast_div((unsigned)std::max(a.L, 1L)), mask_of(a.N, a.w));
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace hlta
