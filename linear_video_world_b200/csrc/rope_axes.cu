// Rotary positions over several axes, and the append to a paged cache that applies them.
//
// A head's first 2P channels are P pairs; pair j belongs to one axis (time, height, width) and
// turns by position-on-that-axis times its frequency. Angles are kept in turns: the frequencies
// come from the host in double precision (f / 2 pi), position * frequency is reduced to
// [-1/2, 1/2] turns in double precision, and sine and cosine of pi times twice that are taken once
// per (token, pair) in single precision (the reduced turn rounds by 2^-26 turns, 1e-7 rad) and
// used for every head.
//
// Bound by HBM: every element is read and written once. A thread owns one 16-byte chunk of a
// token's row (layout 1: the two chunks that its pairs join) and walks heads in groups of eight,
// all eight loads in flight before the first store (groups of four: 3 % slower at 21 frames of 16 heads,
// 5 % at one frame of 8); the heads are split over blockIdx.y until the
// grid fills the GPU, so a call of few tokens has one group of heads per thread and pays one
// round trip. Measured: q and k of 32760 tokens, 16 heads, 84.9 us (6.3 TB/s); 8 x 1560 tokens of 8
// heads appended 19.8 us; 16 tokens 4.7 us. Rows whose d or 2P is no multiple of the chunk take one pair or channel per thread.
#include "hlta_internal.cuh"

#include <algorithm>
#include <math.h>
#include <string.h>

namespace hlta {
namespace {

constexpr int THREADS = 256;
constexpr int MAXP = 64;

struct Turns {
    double f[MAXP];             // turns per position
    unsigned char axis[MAXP];
    int P, layout, gh, gw, inverse;
    const int *pos, *t0;
};

struct Job {
    // rope: x0 = q, x1 = k with H0, H1 heads; append: x0 = k, x1 = v with H0 = H1 heads
    const void *x0, *x1;
    void *y0, *y1;
    int H0, H1, d, per;         // per: heads (of both tensors together) per thread
    long L, units;              // units: threads' items per token
    long total;                 // B * L * units
    // append
    const int *table, *kv_lens, *new_lens;
    long num_pages;
    int page_log2, max_pages, rotate;
    unsigned int *err;
};

// positions of token l of rollout b on the three axes
__device__ __forceinline__ void positions(const Turns &t, long b, long l, long L, int (&p)[3])
{
    if (t.pos) {
        const int *s = t.pos + (b * L + l) * 3;
        p[0] = s[0];
        p[1] = s[1];
        p[2] = s[2];
        return;
    }
    const long row = l / t.gw;
    p[2] = (int)(l - row * t.gw);
    const long f = row / t.gh;
    p[1] = (int)(row - f * t.gh);
    p[0] = (int)f + (t.t0 ? t.t0[b] : 0);
}

__device__ __forceinline__ void turn(const double *f, const unsigned char *axis, int j, const int (&p)[3],
                                     int inverse, float &c, float &s)
{
    const int a = axis[j];
    const double x = f[j] * (double)(a == 0 ? p[0] : a == 1 ? p[1] : p[2]);
    sincospif(2.f * (float)(x - rint(x)), &s, &c);
    if (inverse) s = -s;
}

// Where a token goes: row index in a [rows][d] view of the output for head 0, and the stride
// between heads in rows. False: no such token, or a page out of range (recorded).
__device__ __forceinline__ bool paged_row(const Job &w, long b, long l, long &row0, long &hstride)
{
    const int cap = w.max_pages << w.page_log2;
    int n = w.new_lens ? w.new_lens[b] : (int)w.L;
    const int kv = w.kv_lens[b];
    const bool bad = n < 0 || n > w.L || kv < 0 || kv > cap || kv < n;
    if (bad) {
        if (l == 0) atomicOr(w.err, DEVERR_TABLE);
        n = max(0, min(n, (int)w.L));
    }
    if (l >= n) return false;
    const long at = (long)kv - n + l;
    if (at < 0 || at >= cap) return false;
    const int pg = w.table[b * w.max_pages + (at >> w.page_log2)];
    if (pg < 0 || pg >= w.num_pages) {
        atomicOr(w.err, DEVERR_TABLE);
        return false;
    }
    const int psz = 1 << w.page_log2;
    row0 = (long)pg * w.H0 * psz + (at & (psz - 1));
    hstride = psz;
    return true;
}

template <typename E> struct Two;
template <> struct Two<__nv_bfloat16> {
    static __device__ __forceinline__ float ld(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void st(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
};
template <> struct Two<float> {
    static __device__ __forceinline__ float ld(const float *p) { return *p; }
    static __device__ __forceinline__ void st(float *p, float v) { *p = v; }
};

// the channel values of a 16-byte chunk as fp32, and back with one rounding each
template <typename E, int V>
__device__ __forceinline__ void unpack(const uint4 &u, float (&x)[V])
{
    if constexpr (sizeof(E) == 2) {
        const __nv_bfloat162 *h2 = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 v = __bfloat1622float2(h2[i]);
            x[2 * i] = v.x;
            x[2 * i + 1] = v.y;
        }
    } else {
        const float *f = reinterpret_cast<const float *>(&u);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = f[i];
    }
}
template <typename E, int V>
__device__ __forceinline__ uint4 pack(const float (&x)[V])
{
    uint4 u;
    if constexpr (sizeof(E) == 2) {
        __nv_bfloat162 *h2 = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) h2[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    } else {
        float *f = reinterpret_cast<float *>(&u);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = x[i];
    }
    return u;
}

// One 16-byte chunk per thread (d and 2P multiples of the chunk; layout 1: P too).
template <typename E, int LAYOUT, bool PAGED>
__global__ void __launch_bounds__(THREADS) turn_kernel_v(const __grid_constant__ Turns t, const __grid_constant__ Job w)
{
    constexpr int V = 16 / (int)sizeof(E);
    constexpr int NC = LAYOUT ? 2 : 1;           // chunks a rotating thread owns
    constexpr int NP = LAYOUT ? V : V / 2;       // pairs in them
    constexpr int NB = 8;                        // heads in flight
    __shared__ double f_s[MAXP];
    __shared__ unsigned char a_s[MAXP];
    for (int i = threadIdx.x; i < MAXP; i += THREADS) {
        f_s[i] = t.f[i];
        a_s[i] = t.axis[i];
    }
    __syncthreads();
    const long gid = (long)blockIdx.x * THREADS + threadIdx.x;
    if (gid >= w.total) return;
    const long bl = gid / w.units;
    const int u = (int)(gid - bl * w.units);
    const long b = bl / w.L, l = bl - b * w.L;
    const int Htot = w.H0 + w.H1;
    const int h_lo = blockIdx.y * w.per, h_hi = min(Htot, h_lo + w.per);
    long prow = 0, phs = 0;
    if (PAGED && !paged_row(w, b, l, prow, phs)) return;

    const int rot_units = LAYOUT ? t.P / V : (2 * t.P) / V;
    const bool rot = u < rot_units;
    // element offset of the thread's chunk(s) in a row
    const int c0 = LAYOUT && !rot ? 2 * t.P + (u - rot_units) * V : u * V;
    const bool two = LAYOUT && rot;
    float cs[NP], sn[NP];
    if (rot && (!PAGED || (w.rotate && h_lo < w.H0))) {
        int p[3];
        positions(t, b, l, w.L, p);
#pragma unroll
        for (int i = 0; i < NP; ++i) turn(f_s, a_s, u * NP + i, p, t.inverse, cs[i], sn[i]);
    }
    for (int h = h_lo; h < h_hi; h += NB) {
        uint4 x[NB][NC];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int hh = h + i;
            if (hh >= h_hi) break;
            const E *s = hh < w.H0 ? (const E *)w.x0 + ((b * w.H0 + hh) * w.L + l) * w.d
                                   : (const E *)w.x1 + ((b * w.H1 + (hh - w.H0)) * w.L + l) * w.d;
            x[i][0] = *reinterpret_cast<const uint4 *>(s + c0);
            if (LAYOUT && two) x[i][NC - 1] = *reinterpret_cast<const uint4 *>(s + c0 + t.P);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int hh = h + i;
            if (hh >= h_hi) break;
            const bool first = hh < w.H0;
            if (rot && (!PAGED || (w.rotate && first))) {
                float a[V];
                unpack<E, V>(x[i][0], a);
                if constexpr (LAYOUT) {
                    float c[V];
                    unpack<E, V>(x[i][1], c);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float u0 = a[j], u1 = c[j];
                        a[j] = u0 * cs[j] - u1 * sn[j];
                        c[j] = u0 * sn[j] + u1 * cs[j];
                    }
                    x[i][1] = pack<E, V>(c);
                } else {
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        const float u0 = a[2 * j], u1 = a[2 * j + 1];
                        a[2 * j] = u0 * cs[j] - u1 * sn[j];
                        a[2 * j + 1] = u0 * sn[j] + u1 * cs[j];
                    }
                }
                x[i][0] = pack<E, V>(a);
            }
            const int hl = first ? hh : hh - w.H0;
            E *y = (E *)(first ? w.y0 : w.y1);
            y += PAGED ? (prow + hl * phs) * w.d : ((b * (first ? w.H0 : w.H1) + hl) * w.L + l) * w.d;
            *reinterpret_cast<uint4 *>(y + c0) = x[i][0];
            if (LAYOUT && two) *reinterpret_cast<uint4 *>(y + c0 + t.P) = x[i][NC - 1];
        }
    }
}

// One pair, or one channel behind them, per thread: any d and P.
template <typename E, bool PAGED>
__global__ void __launch_bounds__(THREADS) turn_kernel(const __grid_constant__ Turns t, const __grid_constant__ Job w)
{
    const long gid = (long)blockIdx.x * THREADS + threadIdx.x;
    if (gid >= w.total) return;
    const long bl = gid / w.units;
    const int u = (int)(gid - bl * w.units);
    const long b = bl / w.L, l = bl - b * w.L;
    const int Htot = w.H0 + w.H1;
    const int h_lo = blockIdx.y * w.per, h_hi = min(Htot, h_lo + w.per);
    long prow = 0, phs = 0;
    if (PAGED && !paged_row(w, b, l, prow, phs)) return;
    const bool pair = u < t.P;
    const int c0 = !pair ? t.P + u : t.layout ? u : 2 * u;
    const int c1 = t.layout ? u + t.P : 2 * u + 1;
    float c = 1.f, s = 0.f;
    if (pair && (!PAGED || w.rotate)) {
        int p[3];
        positions(t, b, l, w.L, p);
        turn(t.f, t.axis, u, p, t.inverse, c, s);
    }
    for (int hh = h_lo; hh < h_hi; ++hh) {
        const bool first = hh < w.H0;
        const int hl = first ? hh : hh - w.H0, H = first ? w.H0 : w.H1;
        const E *x = (const E *)(first ? w.x0 : w.x1) + ((b * H + hl) * w.L + l) * w.d;
        E *y = (E *)(first ? w.y0 : w.y1) + (PAGED ? (prow + hl * phs) * w.d : ((b * H + hl) * w.L + l) * w.d);
        if (!pair) {
            y[c0] = x[c0];
        } else if (!PAGED || (w.rotate && first)) {
            const float u0 = Two<E>::ld(x + c0), u1 = Two<E>::ld(x + c1);
            Two<E>::st(y + c0, u0 * c - u1 * s);
            Two<E>::st(y + c1, u0 * s + u1 * c);
        } else {
            const E u0 = x[c0], u1 = x[c1];
            y[c0] = u0;
            y[c1] = u1;
        }
    }
}

template <bool PAGED>
cudaError_t launch(const Turns &t, Job w, int B, bool bf16, cudaStream_t s)
{
    const int Htot = w.H0 + w.H1;
    if (B == 0 || w.L == 0 || Htot == 0) return cudaSuccess;
    const int V = bf16 ? 8 : 4;
    const bool vec = w.d % V == 0 && (t.layout ? t.P % V == 0 : (2 * t.P) % V == 0);
    w.units = vec ? (t.layout ? (w.d - t.P) / V : w.d / V) : w.d - t.P;
    w.total = (long)B * w.L * w.units;
    const long blocks = (w.total + THREADS - 1) / THREADS;
    if (blocks > 0x7fffffffL) return cudaErrorNotSupported;
    // heads per thread: all of them once the tokens alone fill the GPU twice (148 SMs of 8 blocks),
    // fewer for fewer tokens, down to one group in flight
    const long want = (148L * 16 + blocks - 1) / blocks;
    const int groups = (int)std::min<long>(std::max<long>(want, 1), (Htot + 7) / 8);
    w.per = (((Htot + groups - 1) / groups) + 7) & ~7;
    const dim3 grid((unsigned)blocks, (unsigned)((Htot + w.per - 1) / w.per));
    if (!vec) {
        if (bf16) turn_kernel<__nv_bfloat16, PAGED><<<grid, THREADS, 0, s>>>(t, w), note_launch();
        else turn_kernel<float, PAGED><<<grid, THREADS, 0, s>>>(t, w), note_launch();
    } else if (t.layout) {
        if (bf16) turn_kernel_v<__nv_bfloat16, 1, PAGED><<<grid, THREADS, 0, s>>>(t, w), note_launch();
        else turn_kernel_v<float, 1, PAGED><<<grid, THREADS, 0, s>>>(t, w), note_launch();
    } else {
        if (bf16) turn_kernel_v<__nv_bfloat16, 0, PAGED><<<grid, THREADS, 0, s>>>(t, w), note_launch();
        else turn_kernel_v<float, 0, PAGED><<<grid, THREADS, 0, s>>>(t, w), note_launch();
    }
    return cudaGetLastError();
}

Turns turns_of(const hlta_rope_axes_t *sp, int inverse)
{
    Turns t;
    memset(&t, 0, sizeof t);
    t.gh = t.gw = 1;
    if (!sp) return t;
    int j = 0;
    const int P = sp->pairs[0] + sp->pairs[1] + sp->pairs[2];
    // a ladder by repeated products in extended precision: 64 roundings of 2^-64 stay below the one
    // to double, and cost a fraction of as many powers
    long double f = 1.L;
    for (int a = 0; a < 3; ++a) {
        if (!sp->pairs[a]) continue;
        const long double step = powl((long double)sp->base, -1.L / (sp->shared_freq ? P : sp->pairs[a]));
        if (!sp->shared_freq) f = 1.L;
        for (int i = 0; i < sp->pairs[a]; ++i, ++j, f *= step) {
            t.f[j] = (double)(f / 6.283185307179586476925287L);
            t.axis[j] = (unsigned char)a;
        }
    }
    t.P = P;
    t.layout = sp->layout;
    t.gh = sp->pos ? 1 : sp->grid_h;
    t.gw = sp->pos ? 1 : sp->grid_w;
    t.inverse = inverse;
    t.pos = sp->pos;
    t.t0 = sp->t0;
    return t;
}

}  // namespace

cudaError_t launch_rope_axes(const void *q, const void *k, void *q_out, void *k_out, int B, int Hq, int Hk,
                             long L, int d, const hlta_rope_axes_t *sp, int inverse, bool bf16, cudaStream_t s)
{
    Job w;
    memset(&w, 0, sizeof w);
    w.x0 = q; w.x1 = k;
    w.y0 = q_out; w.y1 = k_out;
    w.H0 = q ? Hq : 0; w.H1 = k ? Hk : 0;
    w.d = d; w.L = L;
    return launch<false>(turns_of(sp, inverse), w, B, bf16, s);
}

cudaError_t launch_paged_append(const PagedKV &c, const void *k, const void *v, const int *new_lens, int B, long L,
                                const hlta_rope_axes_t *sp, bool bf16, cudaStream_t s)
{
    Job w;
    memset(&w, 0, sizeof w);
    w.x0 = k; w.x1 = v;
    w.y0 = c.k; w.y1 = c.v;
    w.H0 = w.H1 = c.H;
    w.d = c.d; w.L = L;
    w.table = c.table; w.kv_lens = c.kv_lens; w.new_lens = new_lens;
    w.num_pages = c.num_pages; w.page_log2 = c.page_log2; w.max_pages = c.max_pages;
    w.rotate = sp != nullptr;
    w.err = c.err;
    return launch<true>(turns_of(sp, 0), w, B, bf16, s);
}

}  // namespace hlta
