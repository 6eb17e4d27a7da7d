// Gated delta rule token by token over a pool of states: the recurrent form, for steps of one or
// a few tokens.
//
// Row i of the state only meets itself: with u = S_i . k and the old row,
//   S_i' = a S_i + (b v_i - a b u) k,     o_i = S_i' . q = a (S_i . q) + (b v_i - a b u) (k . q),
// so both products of a token read the same old row and are reduced together, and k . q is one
// number per token. Bound by HBM: 4 d^2 bytes in and as many out per state, against 8 d^2
// operations per token.
// d = 128: eight lanes share a row (16 channels each, as four 16-byte words 128 bytes apart, so
// that a warp's load covers whole 128-byte lines of four rows); a thread keeps the rows' channels
// in registers for all of the step's tokens, so the state moves once however many tokens there are.
// Two rows a thread, 32 a block, six blocks per SM: 256 rollouts of 8 heads, up to four tokens each,
// take 59.7 us (4.6 TB/s of states in and out; one row a thread 81, four rows 70); one token of 8 heads
// 3.3 us.
// Other d (fp32 tensors): a warp walks a row.
#include "hlta_internal.cuh"

#include <math.h>

namespace hlta {
namespace {

__device__ __forceinline__ float ldf(const float *p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float *p, float v) { *p = v; }
__device__ __forceinline__ void stf(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float x)
{
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The rollout's state slot and token count as the tables say.
__device__ __forceinline__ void rollout(const GdnStepArgs &p, int b, long &slot, int &n)
{
    slot = p.slots ? p.slots[b] : b;
    n = p.lens ? p.lens[b] : (int)p.L;
}
// Whether to skip it: out of range, or its slot taken by an earlier rollout. Every thread of the block.
__device__ __forceinline__ bool refused(const GdnStepArgs &p, int b, long slot, int n)
{
    int bad = slot >= p.num_slots || n < 0 || n > p.L;
    if (p.slots)
        for (int i = threadIdx.x; i < b; i += blockDim.x) bad |= p.slots[i] == slot;
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) atomicOr(p.err, DEVERR_TABLE);
    return bad;
}

// gates of a token: given, or a = exp(-c softplus(x)), b = sigmoid(y)
__device__ __forceinline__ void gates(const GdnStepArgs &p, long at, float &a, float &b)
{
    a = p.a[at];
    b = p.b[at];
    if (p.raw) {
        a = expf(-p.raw_c * (fmaxf(a, 0.f) + log1pf(expf(-fabsf(a)))));
        b = 1.f / (1.f + expf(-b));
    }
}

// scale to unit norm; a zero vector stays zero
__device__ __forceinline__ float unit(float sumsq) { return sumsq > 0.f ? rsqrtf(sumsq) : 0.f; }

constexpr int D = 128, TOK = 4, RPT = 2, NT = 128;      // staged tokens, rows per thread, threads
constexpr int ROWS = NT / 8 * RPT;                      // rows per block (32)

template <typename E>
__global__ void __launch_bounds__(NT, 6) gdn_step_kernel(const GdnStepArgs p)
{
    __shared__ __align__(16) float qs[TOK][D], ks[TOK][D], vs[TOK][ROWS];
    __shared__ float as[TOK], bs[TOK], kq[TOK];
    const int b = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long slot;
    int n;
    rollout(p, b, slot, n);
    if (slot < 0) return;
    const int sub = threadIdx.x & 7, row0 = blockIdx.x * ROWS, row = threadIdx.x >> 3;
    const long bh = (long)b * p.H + h;
    const float *S = p.S + (min(slot, p.num_slots - 1) * p.H + h) * D * D + (long)(row0 + row) * D + sub * 4;
    // the state's loads are in flight while the tables are looked through and the tokens staged
    float s[RPT][16];
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float4 v = *(const float4 *)(S + r * (NT / 8) * D + x * 32);
            s[r][4 * x] = v.x; s[r][4 * x + 1] = v.y; s[r][4 * x + 2] = v.z; s[r][4 * x + 3] = v.w;
        }
    if (refused(p, b, slot, n)) return;
    for (int t0 = 0; t0 < n; t0 += TOK) {
        if (t0) __syncthreads();
        if (t0 + warp < n) {            // one warp stages a token
            const long tok = bh * p.L + t0 + warp, at = tok * D;
            float q[4], k[4], qq = 0.f, kk = 0.f, qk = 0.f;
            for (int x = lane; x < ROWS; x += 32) vs[warp][x] = ldf((const E *)p.v + at + row0 + x);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                q[x] = ldf((const E *)p.q + at + x * 32 + lane);
                k[x] = ldf((const E *)p.k + at + x * 32 + lane);
            }
            if (lane == 0) gates(p, tok, as[warp], bs[warp]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                qq = fmaf(q[x], q[x], qq);
                kk = fmaf(k[x], k[x], kk);
                qk = fmaf(q[x], k[x], qk);
            }
            qk = warp_sum(qk);
            float fq = 1.f, fk = 1.f;
            if (p.raw) {
                fq = unit(warp_sum(qq));
                fk = unit(warp_sum(kk));
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                qs[warp][x * 32 + lane] = q[x] * fq;
                ks[warp][x * 32 + lane] = k[x] * fk;
            }
            if (lane == 0) kq[warp] = qk * fq * fk;
        }
        __syncthreads();
        for (int j = 0; j < min(TOK, n - t0); ++j) {
            float u[RPT] = {}, w[RPT] = {};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float4 q = *(const float4 *)&qs[j][x * 32 + sub * 4], k = *(const float4 *)&ks[j][x * 32 + sub * 4];
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    u[r] = fmaf(s[r][4 * x], k.x, fmaf(s[r][4 * x + 1], k.y, fmaf(s[r][4 * x + 2], k.z, fmaf(s[r][4 * x + 3], k.w, u[r]))));
                    w[r] = fmaf(s[r][4 * x], q.x, fmaf(s[r][4 * x + 1], q.y, fmaf(s[r][4 * x + 2], q.z, fmaf(s[r][4 * x + 3], q.w, w[r]))));
                }
            }
#pragma unroll
            for (int o = 4; o; o >>= 1)
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    u[r] += __shfl_xor_sync(0xffffffffu, u[r], o);
                    w[r] += __shfl_xor_sync(0xffffffffu, w[r], o);
                }
            const float a = as[j], bb = bs[j], qk = kq[j];
            float g[RPT];
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                g[r] = bb * (vs[j][row + r * (NT / 8)] - a * u[r]);
                if (sub == 0) stf((E *)p.o + (bh * p.L + t0 + j) * D + row0 + row + r * (NT / 8), fmaf(a, w[r], g[r] * qk));
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float4 k = *(const float4 *)&ks[j][x * 32 + sub * 4];
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    s[r][4 * x] = fmaf(a, s[r][4 * x], g[r] * k.x);
                    s[r][4 * x + 1] = fmaf(a, s[r][4 * x + 1], g[r] * k.y);
                    s[r][4 * x + 2] = fmaf(a, s[r][4 * x + 2], g[r] * k.z);
                    s[r][4 * x + 3] = fmaf(a, s[r][4 * x + 3], g[r] * k.w);
                }
            }
        }
    }
    float *So = p.S_out + (slot * p.H + h) * D * D + (long)(row0 + row) * D + sub * 4;
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            *(float4 *)(So + r * (NT / 8) * D + x * 32) = make_float4(s[r][4 * x], s[r][4 * x + 1], s[r][4 * x + 2], s[r][4 * x + 3]);
}

// fp32 tensors of any d <= 128: a warp per state row, up to four channels a lane.
__global__ void __launch_bounds__(NT) gdn_step_any_kernel(const GdnStepArgs p)
{
    const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31, d = p.d;
    long slot;
    int n;
    rollout(p, b, slot, n);
    if (slot < 0 || refused(p, b, slot, n)) return;
    const int row = blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    if (row >= d) return;
    const long bh = (long)b * p.H + h, base = (slot * p.H + h) * d * d + (long)row * d;
    float s[4];
    for (int x = 0; x < 4; ++x) s[x] = x * 32 + lane < d ? p.S[base + x * 32 + lane] : 0.f;
    for (int t = 0; t < n; ++t) {
        const long at = (bh * p.L + t) * d;
        float q[4], k[4], qq = 0.f, kk = 0.f, qk = 0.f, u = 0.f, w = 0.f;
        for (int x = 0; x < 4; ++x) {
            const bool in = x * 32 + lane < d;
            q[x] = in ? ((const float *)p.q)[at + x * 32 + lane] : 0.f;
            k[x] = in ? ((const float *)p.k)[at + x * 32 + lane] : 0.f;
            qq = fmaf(q[x], q[x], qq);
            kk = fmaf(k[x], k[x], kk);
            qk = fmaf(q[x], k[x], qk);
            u = fmaf(s[x], k[x], u);
            w = fmaf(s[x], q[x], w);
        }
        float fq = 1.f, fk = 1.f, a, bb;
        if (p.raw) {
            fq = unit(warp_sum(qq));
            fk = unit(warp_sum(kk));
        }
        u = warp_sum(u) * fk;
        w = warp_sum(w) * fq;
        qk = warp_sum(qk) * fq * fk;
        gates(p, bh * p.L + t, a, bb);
        const float g = bb * (((const float *)p.v)[at + row] - a * u);
        for (int x = 0; x < 4; ++x) s[x] = fmaf(a, s[x], g * (k[x] * fk));
        if (lane == 0) ((float *)p.o)[at + row] = fmaf(a, w, g * qk);
    }
    for (int x = 0; x < 4; ++x)
        if (x * 32 + lane < d) p.S_out[base + x * 32 + lane] = s[x];
}

}  // namespace

cudaError_t launch_gdn_step(const GdnStepArgs &a, bool bf16, cudaStream_t s)
{
    if (a.B == 0 || a.H == 0) return cudaSuccess;
    if (a.B > 65535 || a.H > 65535) return cudaErrorNotSupported;
    if (a.d == D) {
        const dim3 grid(D / ROWS, (unsigned)a.H, (unsigned)a.B);
        if (bf16) gdn_step_kernel<__nv_bfloat16><<<grid, NT, 0, s>>>(a), note_launch();
        else gdn_step_kernel<float><<<grid, NT, 0, s>>>(a), note_launch();
    } else {
        gdn_step_any_kernel<<<dim3((unsigned)((a.d + NT / 32 - 1) / (NT / 32)), (unsigned)a.H, (unsigned)a.B), NT, 0, s>>>(a), note_launch();
    }
    return cudaGetLastError();
}

}  // namespace hlta
