// Accumulated attention weights of a chunk over a paged cache, bf16, head dim 128: the second pass,
// once the chunk's log-sum-exp is known.
//
// w_out[j] = decay w_in[j] + sum over the head group's rows of 2^(score - lse): a sum over rows, so
// the products are taken the other way round, S^T = K Q^T with keys on tensor memory's lanes and 128
// rows on its columns: a key's sum is a thread's own, in the order of the rows, with no atomics and no
// exchange between lanes. A block owns a key tile of 128 and streams the rows past it.
// Bound by the exponentials: 1024 cycles (16 a cycle) per 128 x 128 scores against 512 of products.
// Roles: warps 0-3 and 4-7 sum every other row tile; warp 8 copies K tiles (two buffers; a lane per
// page) and row tiles (a ring of four) by TMA and lays the rows' log-sum-exp and spans beside them;
// warp 9 issues the products into four buffers of tensor memory. Equal shares of the line of (key
// tile, row tile) steps (paged.cuh, one block a gang): the sums of a key tile that is cut between
// blocks go to the workspace and a second kernel joins them in the order of the blocks. (Whole key
// tiles per block: 312 of them on 148 SMs took three rounds for two; with the log-sum-exp fetched by
// the summing warps themselves 61 us, now 44: 3 chunks of 517 tokens of 16 heads, window 4096, 312 key tiles.)
#include "hlta_internal.cuh"
#include "paged.cuh"
#include "sm100_ptx.cuh"
#include "tc_ptx.cuh"

#include <algorithm>

namespace hlta {
namespace {

using namespace ptx;
using namespace paged;

constexpr int BN = 128, RT = 128, D = 128;              // keys per tile, rows per row tile
constexpr int THREADS = 320, WARP_TMA = 8, WARP_MMA = 9;
constexpr uint32_t HALF = 128 * 128, TILE = 2 * HALF;
constexpr int NQ = 4, NK = 2, NS = 4;
static_assert(NQ == NS, "a row tile's ring slot and its buffer of products have the same number");
constexpr uint32_t SM_K = 0, SM_Q = NK * TILE, SM_Z = SM_Q + NQ * TILE;         // z: [slot][128 rows]
constexpr uint32_t SM_SPAN = SM_Z + NQ * RT * 4, SM_SUM = SM_SPAN + NQ * RT * 8;    // spans; sums of group 1
constexpr uint32_t SM_BAR = SM_SUM + BN * 4;
enum { B_KFULL, B_KEMPTY = B_KFULL + NK, B_QFULL = B_KEMPTY + NK, B_QEMPTY = B_QFULL + NQ, B_SFULL = B_QEMPTY + NQ, B_SFREE = B_SFULL + NS, NBARS = B_SFREE + NS };
constexpr uint32_t SM_PLACE = SM_BAR + 8 * NBARS, SM_OK = SM_PLACE + 32, SM_TMEM = SM_OK + 32, SM_ABORT = SM_TMEM + 4;
std::atomic<unsigned long long> g_shared{0};
constexpr size_t SMEM_BYTES = SM_ABORT + 4;
static_assert(SMEM_BYTES <= 232448 && SM_BAR % 8 == 0, "shared memory of one block");

struct Params {
    Line line;
    PagedKV c;
    int R;
    float sl2;
    const float *lse, *w_in;
    float *w_out, decay;
    float *part;                    // [block][2][128 keys]
};

// the keys that row tile rt's live rows see, and whether all of its rows are live and see [p0, p0 + BN)
struct RowTile {
    bool any, full;
};
__device__ __forceinline__ RowTile row_tile(const Params &p, const Roll &ro, int rt, int p0)
{
    const int L = p.line.L, r0 = rt * RT, r1 = min(r0 + RT, p.R);
    int i0 = frem(r0, p.line.byL), i1 = i0 + (r1 - 1 - r0);
    if (i1 >= L) {                  // runs into the next head
        i0 = 0;
        i1 = L - 1;
    }
    RowTile o{false, false};
    if (i0 >= ro.n) return o;
    const int last = min(i1, ro.n - 1);
    const Span a = span_of(ro, i0, p.line.mask), b = span_of(ro, last, p.line.mask);
    o.any = a.lo < p0 + BN && b.hi > p0 && b.hi > a.lo;
    // spans move with the token: the first row's end and the last row's start bound them all
    o.full = r1 - r0 == RT && i1 < ro.n && a.hi >= p0 + BN && b.lo <= p0;
    return o;
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

__global__ void __launch_bounds__(THREADS, 1)
paged_weights_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    auto BAR = [&](int i) { return sbase + SM_BAR + 8u * (uint32_t)i; };
    volatile int *abort_flag = (volatile int *)(smem + SM_ABORT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;");      // the second kernel may be set up meanwhile
    if (sbase & 1023u) {                    // not seen: the attribute asks for it
        if (threadIdx.x == 0) atomicOr(p.c.err, DEVERR_ATTN_WAIT);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(BAR(B_KFULL + i), 1);
            mbar_init(BAR(B_KEMPTY + i), 1);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(BAR(B_QFULL + i), 1);
            mbar_init(BAR(B_QEMPTY + i), 1);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(BAR(B_SFULL + i), 1);
            mbar_init(BAR(B_SFREE + i), 128);
        }
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == WARP_TMA) {
        const Place c = place_of<BN>(p.line, blockIdx.x);
        if (lane == 0) *(Place *)(smem + SM_PLACE) = c;
    }
    if (warp == WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + SM_TMEM), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *(uint32_t *)(smem + SM_TMEM);
    Place at = *(Place *)(smem + SM_PLACE);
    Piece<BN> x;
    const int nrt = p.line.steps;
    auto wait_bar = [&](uint32_t bar, uint32_t parity) -> bool {
        return mbar_try(bar, parity) || mbar_wait(bar, parity, abort_flag, p.c.err, DEVERR_ATTN_WAIT);
    };

    if (warp == WARP_TMA) {
        const int psz = 1 << p.c.page_log2, npg = BN >> p.c.page_log2;
        long nk = 0, nq = 0;
        bool ok = true;
        while (ok && next_piece<BN>(p.line, at, x)) {
            const Roll &ro = x.x.r;
            const Span u{span_of(ro, 0, p.line.mask).lo, span_of(ro, ro.n - 1, p.line.mask).hi};
            const long row0 = (long)(x.b * p.c.H + x.h) * p.R;
            for (int st = x.ta; ok && st < x.tb;) {
                const int t = st / nrt, rt0 = st - t * nrt, rt1 = min(nrt, rt0 + x.tb - st);
                st += rt1 - rt0;
                const int p0 = t * BN + lane * psz;
                const int pg = lane < npg && p0 < u.hi && p0 + psz > u.lo ? page_of(p.c, x.b, max(p0, u.lo)) : -1;
                const int ks = (int)(nk % NK);
                bool w = true;
                if (lane == 0 && nk >= NK) w = wait_bar(BAR(B_KEMPTY + ks), (uint32_t)(nk / NK + 1) & 1u);
                if (!(ok = __shfl_sync(0xffffffffu, w, 0))) break;
                const unsigned have = __ballot_sync(0xffffffffu, pg >= 0);
                if (lane == 0) mbar_expect_tx(BAR(B_KFULL + ks), (uint32_t)__popc(have) * (uint32_t)psz * 256u);
                __syncwarp();
                if (pg >= 0) {
                    const int row = (pg * p.c.H + x.h) << p.c.page_log2;
                    const uint32_t dst = sbase + SM_K + (uint32_t)ks * TILE + (uint32_t)(lane * psz) * 128u;
                    tma_load_2d(dst, &tk, 0, row, BAR(B_KFULL + ks));
                    tma_load_2d(dst + HALF, &tk, 64, row, BAR(B_KFULL + ks));
                }
                ++nk;
                for (int rt = rt0; rt < rt1; ++rt) {
                    const RowTile k = row_tile(p, ro, rt, t * BN);
                    if (!k.any) continue;
                    // the rows' log-sum-exp (log2, negative) and spans; rows that are none see nothing
                    float z[4];
                    Span v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = rt * RT + 4 * lane + j, i = frem(r, p.line.byL);
                        const bool live = r < p.R && i < ro.n;
                        z[j] = live ? p.lse[row0 + r] * -1.4426950408889634f : 0.f;
                        v[j] = live && !k.full ? span_of(ro, i, p.line.mask) : Span{0, 0};
                    }
                    const int qs = (int)(nq % NQ);
                    // the slot's product is done, and its scores, log-sum-exp and spans were read
                    if (lane == 0 && nq >= NQ)
                        w = wait_bar(BAR(B_QEMPTY + qs), (uint32_t)(nq / NQ + 1) & 1u) && wait_bar(BAR(B_SFREE + qs), (uint32_t)(nq / NQ + 1) & 1u);
                    if (!(ok = __shfl_sync(0xffffffffu, w, 0))) break;
                    *(float4 *)(smem + SM_Z + (qs * RT + 4 * lane) * 4) = make_float4(z[0], z[1], z[2], z[3]);
                    if (!k.full) {
                        int4 *d = (int4 *)(smem + SM_SPAN + (qs * RT + 4 * lane) * 8);
                        // (first position, number of positions)
                        d[0] = make_int4(v[0].lo, max(0, v[0].hi - v[0].lo), v[1].lo, max(0, v[1].hi - v[1].lo));
                        d[1] = make_int4(v[2].lo, max(0, v[2].hi - v[2].lo), v[3].lo, max(0, v[3].hi - v[3].lo));
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_expect_tx(BAR(B_QFULL + qs), TILE);
                        const int row = (int)(row0 + rt * RT);
                        tma_load_2d(sbase + SM_Q + (uint32_t)qs * TILE, &tq, 0, row, BAR(B_QFULL + qs));
                        tma_load_2d(sbase + SM_Q + (uint32_t)qs * TILE + HALF, &tq, 64, row, BAR(B_QFULL + qs));
                    }
                    ++nq;
                }
            }
        }
        if (lane == 0 && *abort_flag) {
            // a bounded wait expired: let the copies this block issued land
            const long long t0 = clock64();
            for (long i = nk - 1; i >= 0 && i >= nk - NK; --i)
                while (!mbar_try(BAR(B_KFULL + (int)(i % NK)), (uint32_t)(i / NK) & 1u) && clock64() - t0 < (1LL << 31)) {}
            for (long i = nq - 1; i >= 0 && i >= nq - NQ; --i)
                while (!mbar_try(BAR(B_QFULL + (int)(i % NQ)), (uint32_t)(i / NQ) & 1u) && clock64() - t0 < (1LL << 31)) {}
        }
    } else if (warp == WARP_MMA) {
        if (lane == 0) {
            constexpr uint32_t IDESC = tc::idesc_bf16(BN, RT, false, false);
            const uint64_t dk0 = tc::sw128_desc(sbase + SM_K, 16, 1024), dq0 = tc::sw128_desc(sbase + SM_Q, 16, 1024);
            uint32_t nk = 0, nq = 0;
            bool ok = true;
            while (ok && next_piece<BN>(p.line, at, x)) {
                for (int st = x.ta; ok && st < x.tb;) {
                    const int t = st / nrt, rt0 = st - t * nrt, rt1 = min(nrt, rt0 + x.tb - st);
                    st += rt1 - rt0;
                    const uint32_t ks = nk % NK;
                    if (!(ok = wait_bar(BAR(B_KFULL + ks), (nk / NK) & 1u))) break;
                    for (int rt = rt0; rt < rt1; ++rt) {
                        if (!row_tile(p, x.x.r, rt, t * BN).any) continue;
                        const uint32_t qs = nq % NQ, sb = nq % NS;
                        if (!(ok = wait_bar(BAR(B_QFULL + qs), (nq / NQ) & 1u))) break;
                        if (nq >= NS && !(ok = wait_bar(BAR(B_SFREE + sb), (nq / NS + 1) & 1u))) break;
                        tc::fence_after_sync();
                        const uint64_t dk = dk0 + (uint64_t)(ks * (TILE >> 4)), dq = dq0 + (uint64_t)(qs * (TILE >> 4));
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t off = (uint64_t)((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
                            tc::umma_bf16(tmem + 128u * sb, dk + off, dq + off, IDESC, kk > 0 ? 1u : 0u);
                        }
                        tc::umma_commit(BAR(B_SFULL + sb));
                        tc::umma_commit(BAR(B_QEMPTY + qs));
                        ++nq;
                    }
                    if (!ok) break;
                    tc::umma_commit(BAR(B_KEMPTY + ks));
                    ++nk;
                }
            }
        }
    } else {
        const int grp = warp >> 2, row = (warp & 3) * 32 + lane;        // the group; this thread's key
        const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float *sums = (float *)(smem + SM_SUM);
        volatile int *sok = (volatile int *)(smem + SM_OK);
        uint32_t nq = 0;
        int tiles = 0;                      // key tiles so far: a cut one is the first or the last
        bool ok = true;
        while (next_piece<BN>(p.line, at, x)) {
            const Roll ro = x.x.r;
            const long head = (long)x.b * p.c.H + x.h;
            for (int st = x.ta; ok && st < x.tb;) {
                const int t = st / nrt, rt0 = st - t * nrt, rt1 = min(nrt, rt0 + x.tb - st);
                st += rt1 - rt0;
                const int p0 = t * BN, key = p0 + row;
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                for (int rt = rt0; rt < rt1; ++rt) {
                    const RowTile k = row_tile(p, ro, rt, p0);
                    if (!k.any) continue;
                    const uint32_t sb = nq % NS, par = (nq / NS) & 1u;
                    const bool mine = (int)(nq & 1) == grp;
                    ++nq;
                    if (!mine) continue;
                    ok = __all_sync(0xffffffffu, ok && wait_bar(BAR(B_QFULL + sb), par) && wait_bar(BAR(B_SFULL + sb), par));
                    tc::fence_after_sync();
                    const float *z = (const float *)(smem + SM_Z) + sb * RT;
                    const int4 *spans = (const int4 *)(smem + SM_SPAN) + sb * (RT / 2);
                    const float2 sl = make_float2(p.sl2, p.sl2);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t sv[64];
                        tc::tmem_ld64(tlane + 128u * sb + 64u * h, sv);
                        if (k.full) {
#pragma unroll
                            for (int c = 0; c < 64; c += 4) {
                                const float4 zz = *(const float4 *)(z + 64 * h + c);
                                const float2 a = ffma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sl, make_float2(zz.x, zz.y));
                                const float2 b = ffma2(make_float2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), sl, make_float2(zz.z, zz.w));
                                acc[0].x += tc::ex2(a.x);
                                acc[0].y += tc::ex2(a.y);
                                acc[1].x += tc::ex2(b.x);
                                acc[1].y += tc::ex2(b.y);
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < 64; c += 4) {
                                const float4 zz = *(const float4 *)(z + 64 * h + c);
                                const int4 v = spans[32 * h + c / 2], w = spans[32 * h + c / 2 + 1];
                                const float2 a = ffma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sl, make_float2(zz.x, zz.y));
                                const float2 b = ffma2(make_float2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), sl, make_float2(zz.z, zz.w));
                                const float e[4] = {tc::ex2(a.x), tc::ex2(a.y), tc::ex2(b.x), tc::ex2(b.y)};
                                acc[0].x += (unsigned)(key - v.x) < (unsigned)v.y ? e[0] : 0.f;
                                acc[0].y += (unsigned)(key - v.z) < (unsigned)v.w ? e[1] : 0.f;
                                acc[1].x += (unsigned)(key - w.x) < (unsigned)w.y ? e[2] : 0.f;
                                acc[1].y += (unsigned)(key - w.z) < (unsigned)w.w ? e[3] : 0.f;
                            }
                        }
                    }
                    tc::fence_before_sync();
                    mbar_arrive(BAR(B_SFREE + sb));
                }
                // group 1's sums join group 0's; both groups give up together
                const float sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                if (grp == 1) sums[row] = sum;
                if (lane == 0) sok[warp] = ok;
                asm volatile("bar.sync 3, 256;" ::: "memory");
                for (int w = 0; w < 8; ++w) ok = ok && sok[w];
                const bool whole = rt0 == 0 && rt1 == nrt;
                if (ok && grp == 0) {
                    float s = sum + sums[row];
                    if (!whole) {
                        p.part[((long)blockIdx.x * 2 + (tiles == 0 ? 0 : 1)) * BN + row] = s;
                    } else if (key < ro.kv) {
                        const long o = head * p.line.cap + key;
                        if (p.w_in && key < ro.h) s = fmaf(p.decay, p.w_in[o], s);
                        p.w_out[o] = s;
                    }
                }
                ++tiles;
                asm volatile("bar.sync 3, 256;" ::: "memory");
            }
            if (!ok) break;
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == WARP_MMA) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Joins the sums of key tiles that were cut between blocks, in the order of the blocks, and gives the
// positions of no key tile (before the window; every position of a rollout without new tokens)
// decay w_in. A block per 128 positions.
__global__ void __launch_bounds__(BN) paged_weights_join_kernel(const __grid_constant__ Params p)
{
    const int h = blockIdx.y % p.c.H, b = blockIdx.y / p.c.H;
    const Roll ro = roll_of(p.line.kv_lens, p.line.new_lens, b, p.line.L, p.line.cap);
    const int t = blockIdx.x, k = t * BN + threadIdx.x;
    // one block waits whatever there is to do, so that this kernel never ends before the first one
    // (what is captured behind it depends on this kernel alone)
    if (t == 0 && blockIdx.y == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t * BN >= ro.kv) return;
    const Tiles<BN> x = tiles_of<BN>(p.line, b);
    const int nt = x.T / p.line.steps;
    float s = 0.f;
    if (t >= x.t0 && t < x.t0 + nt) {
        const Sums sums = tile_sums<BN>(p.line, b);
        const long long W = sums.all * p.line.H;
        const Holders g = holders_at(p.line, W, sums.before * p.line.H + (long long)h * x.T + (long long)(t - x.t0) * p.line.steps, p.line.steps);
        if (g.g0 == g.g1) return;
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the first kernel's results from here on
        for (int i = g.g0; i <= g.g1; ++i) s += p.part[((long)i * 2 + (i == g.g0 ? g.slot0 : 0)) * BN + threadIdx.x];
    } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    if (k >= ro.kv) return;
    const long at = (long)blockIdx.y * p.line.cap + k;
    if (p.w_in && k < ro.h) s = fmaf(p.decay, p.w_in[at], s);
    p.w_out[at] = s;
}

}  // namespace

bool paged_weights_fit(long R, int cap) { return (cap / BN + 2L) * ((R + RT - 1) / RT) < (1L << 30); }

cudaError_t launch_paged_weights_tc(const PagedAttnArgs &a, cudaStream_t s)
{
    const long R = a.G * a.L, q_rows = (long)a.B * a.c.H * R, kv_rows = a.c.num_pages * a.c.H << a.c.page_log2;
    if (R < 1 || q_rows + RT >= (1L << 31) || kv_rows + BN >= (1L << 31) || (long)a.B * a.c.H > 65535) return cudaErrorNotSupported;
    CUtensorMap mq, mk;
    cudaError_t e;
    if ((e = make_tmap_2d_bf16(&mq, a.q, q_rows, D, 64, RT, true)) != cudaSuccess) return e;
    if ((e = make_tmap_2d_bf16(&mk, a.c.k, kv_rows, D, 64, 1u << a.c.page_log2, true)) != cudaSuccess) return e;
    const int sms = device_sms();
    Params p;
    p.c = a.c;
    p.R = (int)R;
    const int nrt = (int)((R + RT - 1) / RT);
    p.line = line_of(a, 1, sms, 1, 1, nrt);
    p.part = (float *)a.ws;         // the attention's pieces are joined by now
    p.sl2 = a.sl2;
    p.lse = a.lse; p.w_in = a.w_in; p.w_out = a.w_out; p.decay = a.decay;
    if ((e = allow_shared((const void *)paged_weights_tc_kernel, SMEM_BYTES, g_shared)) != cudaSuccess) return e;
    paged_weights_tc_kernel<<<sms, THREADS, SMEM_BYTES, s>>>(mq, mk, p), note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.line.cap + BN - 1) / BN), (unsigned)(a.B * a.c.H));
    cfg.blockDim = dim3(BN);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, paged_weights_join_kernel, p)) == cudaSuccess) note_launch();
    return e;
}

}  // namespace hlta
