// Attention of a few tokens over a paged cache (at most 16 packed rows of a key head), with the
// accumulated attention weights. bf16, head dim 128, on the tensor cores; fp32 on the CUDA cores.
//
// Bound by HBM: every key and value is read once, 512 bytes for at most 16 rows. The division of
// the work is that of paged.cuh with single blocks as gangs, two blocks per SM: equal shares of the
// 64-key tiles whatever the rollouts' lengths (a head's start and end counted as two of them where blocks
// have several). One warp of a block copies tiles (K and V of 64 keys, 32 KB) into a ring of three by TMA,
// a lane per page; 192 KB in flight per SM cover the latency several times. Four warps take 16 keys of a tile each and never wait for one
// another: S = Q K^T of 16 x 16 by warp-level products (the rows fill one m16 tile, a tcgen05 product
// would be 7/8 padding), running maximum and sum per warp, O += P V with V's fragments through
// transposing loads. At the end of a piece the warps' results are joined through shared memory; a
// piece that is a whole head is stored, others go to the workspace.
// Weights: their scale is known only at the end, so the scaled scores are stored (4 bytes per row
// and key next to the 512 that are read) and a second kernel turns them into weights while it joins
// the pieces; reading K again instead would add half of the traffic. Measured: 32 tokens of 24 query
// heads over 37 to 32760 keys of 8 heads, 2.2 GB: 351 us (6.1 TB/s), and 33 us for the second kernel; one token over
// 1560 keys of 8 heads 11.5 us in all.
//
// What the cache holds where no row looks: as in the chunk kernel, scores are masked before use and
// values outside the span of the rows are zeroed in shared memory.
//
// fp32 tensors (any d <= 128): the same division and the same second kernel; 32-key tiles copied
// asynchronously into three stages, four warps of eight keys each. A score is summed by four lanes
// (32 channels each), a lane owns four channels of the output; built for 1, 2, 4, 8 and 16 rows, so that
// few rows do not pay for 16 (8 tokens over 500 to 3000 keys of 8 heads: 42 us, 62 with no form below
// four rows; 32 query heads over 4: 44 us, 66 with 16 rows for eight). Bound by the instructions of a tile
// (a warp's copies, score sums over lanes, softmax), for 16 rows by shared-memory reads.
#include "hlta_internal.cuh"
#include "paged.cuh"
#include "paged_f32.cuh"
#include "sm100_ptx.cuh"
#include "tc_ptx.cuh"

#include <algorithm>
#include <math.h>

namespace hlta {
namespace {

using namespace ptx;
using namespace paged;

constexpr int MROWS = 16, BN = 64, D = 128;
constexpr int CW = 4, THREADS = 32 * (CW + 1);          // consumer warps; and the producer
constexpr int NSLOT = 3;
constexpr uint32_t HALF = BN * 128, KT = 2 * HALF, TILE = 2 * KT;    // [64 keys][64 columns]; K; K and V
constexpr uint32_t SM_MERGE = NSLOT * TILE;                          // two warps' O in fragment order
constexpr uint32_t SM_ML = SM_MERGE + 2 * 64 * 32 * 4;               // [warp][row] (maximum, sum)
constexpr uint32_t SM_OK = SM_ML + CW * MROWS * 8, SM_BAR = SM_OK + 16, SM_PLACE = SM_BAR + 16 * NSLOT;
constexpr uint32_t SM_ABORT = SM_PLACE + 32;
std::atomic<unsigned long long> g_shared{0};
constexpr size_t SMEM_BYTES = SM_ABORT + 16;
static_assert(2 * (SMEM_BYTES + 1024) <= 233472, "two blocks per SM");

struct Params {
    Line line;
    PagedKV c;
    int G, R;
    float sl2;
    const void *q;
    void *o;
    float *lse;
    float *part;                    // bf16: [block][2][64 registers][32 lanes]; fp32: [block][2][16 rows][128]
    float2 *ml;                     // [block][2][16 rows]
    float *scores;                  // [b][h][R][cap], log2 units; null without weights
    float2 *whole;                  // [b][h][16 rows] (maximum, sum) of heads that one block had whole
    const float *w_in;
    float *w_out, decay;
    int nj, keys;                   // second kernel: blocks of a head that join; keys per block of the weights
    int early;                      // whether its blocks may take their places while the first kernel runs
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// factors that bring two (maximum, unnormalised) pairs to the larger maximum
__device__ __forceinline__ float2 rebase(float m0, float m1, float &m)
{
    m = fmaxf(m0, m1);
    const float base = m == -INFINITY ? 0.f : m;
    return make_float2(tc::ex2(m0 - base), tc::ex2(m1 - base));
}

__global__ void __launch_bounds__(THREADS, 2)
paged_token_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    volatile int *abort_flag = (volatile int *)(smem + SM_ABORT);
    auto FULL = [&](int i) { return sbase + SM_BAR + 16u * (uint32_t)i; };
    auto EMPTY = [&](int i) { return sbase + SM_BAR + 16u * (uint32_t)i + 8u; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.early) asm volatile("griddepcontrol.launch_dependents;");     // the second kernel may be set up meanwhile
    if (sbase & 1023u) {                    // not seen: the attribute asks for it
        if (threadIdx.x == 0) atomicOr(p.c.err, DEVERR_ATTN_WAIT);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NSLOT; ++i) {
            mbar_init(FULL(i), 1);
            mbar_init(EMPTY(i), CW);
        }
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (threadIdx.x < 2) asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)(threadIdx.x ? &tv : &tk)) : "memory");
    if (warp == CW) {
        const Place c = place_of<BN>(p.line, blockIdx.x);
        if (lane == 0) *(Place *)(smem + SM_PLACE) = c;
    }
    __syncthreads();
    Place at = *(Place *)(smem + SM_PLACE);
    auto wait_bar = [&](uint32_t bar, uint32_t parity) -> bool {
        return mbar_try(bar, parity) || mbar_wait(bar, parity, abort_flag, p.c.err, DEVERR_ATTN_WAIT);
    };
    Piece<BN> x;
    int slot = 0;
    uint32_t lap = 0;
    auto next_slot = [&] {
        if (++slot == NSLOT) {
            slot = 0;
            lap ^= 1u;
        }
    };
    // the span of the chunk's live rows: every tile of the line lies in it
    auto span_all = [&](const Roll &r) {
        return Span{span_of(r, 0, p.line.mask).lo, span_of(r, r.n - 1, p.line.mask).hi};
    };

    if (warp == CW) {
        const int psz = 1 << p.c.page_log2, box = min(psz, BN), nbox = BN / box;
        bool ok = true;
        long issued = 0;
        while (ok && next_piece<BN>(p.line, at, x)) {
            if (x.x.r.bad && lane == 0) atomicOr(p.c.err, DEVERR_TABLE);
            const Span u = span_all(x.x.r);
            // the first row of this lane's part of tile t, or -1 when none of its positions is seen
            auto row_at = [&](int t) -> int {
                const int p0 = t * BN + lane * box;
                if (lane >= nbox || t >= x.tb || p0 >= u.hi || p0 + box <= u.lo) return -1;
                return ((page_of(p.c, x.b, max(p0, u.lo)) * p.c.H + x.h) << p.c.page_log2) + (p0 & (psz - 1));
            };
            int row = row_at(x.ta);
            for (int t = x.ta; t < x.tb; ++t) {
                const int next = row_at(t + 1);             // looked up ahead of the wait
                bool w = true;
                if (lane == 0 && issued >= NSLOT) w = wait_bar(EMPTY(slot), lap ^ 1u);
                if (!(ok = __shfl_sync(0xffffffffu, w, 0))) break;
                const unsigned have = __ballot_sync(0xffffffffu, row >= 0);
                if (lane == 0) mbar_expect_tx(FULL(slot), (uint32_t)__popc(have) * (uint32_t)box * 512u);
                __syncwarp();
                if (row >= 0) {
                    const uint32_t dst = sbase + (uint32_t)slot * TILE + (uint32_t)(lane * box) * 128u;
                    tma_load_2d(dst, &tk, 0, row, FULL(slot));
                    tma_load_2d(dst + HALF, &tk, 64, row, FULL(slot));
                    tma_load_2d(dst + KT, &tv, 0, row, FULL(slot));
                    tma_load_2d(dst + KT + HALF, &tv, 64, row, FULL(slot));
                }
                ++issued;
                next_slot();
                row = next;
            }
        }
        if (lane == 0 && *abort_flag) {
            // a bounded wait expired: let the copies this block issued land
            const long long t0 = clock64();
            for (long i = issued - 1; i >= 0 && i >= issued - NSLOT; --i)
                while (!mbar_try(FULL((int)(i % NSLOT)), (uint32_t)(i / NSLOT) & 1u) && clock64() - t0 < (1LL << 31)) {}
        }
        return;
    }

    // ------------------------------- consumers -------------------------------------------------
    const int g = lane >> 2, c = lane & 3;
    const int key0 = warp * 16;             // this warp's keys of a tile
    float *merge = (float *)(smem + SM_MERGE);
    float2 *sml = (float2 *)(smem + SM_ML);
    volatile int *sok = (volatile int *)(smem + SM_OK);
    // addresses of the fragments inside a tile: K as [key][channel] (no transposition), V transposed
    const int km = lane >> 3, kr = lane & 7;
    const int kkey = key0 + (km >> 1) * 8 + kr, vkey = key0 + (km & 1) * 8 + kr;
    auto k_addr = [&](uint32_t base, int kk) {
        const int col = 16 * kk + (km & 1) * 8;
        return base + (uint32_t)(col >> 6) * HALF + (uint32_t)kkey * 128u + ((((uint32_t)(col & 63) >> 3) ^ (uint32_t)(kkey & 7)) << 4);
    };
    auto v_addr = [&](uint32_t base, int n2) {
        const int col = 16 * n2 + (km >> 1) * 8;
        return base + KT + (uint32_t)(col >> 6) * HALF + (uint32_t)vkey * 128u + ((((uint32_t)(col & 63) >> 3) ^ (uint32_t)(vkey & 7)) << 4);
    };
    bool ok = true;
    for (int piece = 0; next_piece<BN>(p.line, at, x); ++piece) {
        const Span u = span_all(x.x.r);
        Span v[2];
        bool live[2];
        const long row0 = (long)(x.b * p.c.H + x.h) * p.R;
        uint32_t qa[8][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = g + 8 * j, i = frem(r, p.line.byL);
            live[j] = r < p.R && i < x.x.r.n;
            v[j] = live[j] ? span_of(x.x.r, i, p.line.mask) : Span{0, 0};
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint32_t *s = reinterpret_cast<const uint32_t *>((const __nv_bfloat16 *)p.q + (row0 + r) * D + 16 * kk + 2 * c);
                qa[kk][j] = live[j] ? s[0] : 0u;
                qa[kk][2 + j] = live[j] ? s[4] : 0u;
            }
        }
        float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][j] = 0.f;
        for (int t = x.ta; ok && t < x.tb; ++t) {
            if (!(ok = __all_sync(0xffffffffu, wait_bar(FULL(slot), lap)))) break;
            const uint32_t base = sbase + (uint32_t)slot * TILE;
            float s[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                uint32_t b[4];
                ldsm4(k_addr(base, kk), b);
                mma16816(s[0], qa[kk], b[0], b[1]);
                mma16816(s[1], qa[kk], b[2], b[3]);
            }
            const int p0 = t * BN + key0;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int pos = p0 + 8 * n + 2 * c;
                    float &a = s[n][2 * j], &d = s[n][2 * j + 1];
                    a = pos >= v[j].lo && pos < v[j].hi ? a * p.sl2 : -INFINITY;
                    d = pos + 1 >= v[j].lo && pos + 1 < v[j].hi ? d * p.sl2 : -INFINITY;
                    // positions are even and the rows' capacity too, so a pair stays in its row
                    if (p.scores && live[j] && pos < x.x.r.kv)
                        *reinterpret_cast<float2 *>(p.scores + (row0 + g + 8 * j) * p.line.cap + pos) = make_float2(a, d);
                }
            float f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float mn = fmaxf(m[j], quad_max(fmaxf(fmaxf(s[0][2 * j], s[0][2 * j + 1]), fmaxf(s[1][2 * j], s[1][2 * j + 1]))));
                const float mb = mn == -INFINITY ? 0.f : mn;
                f[j] = tc::ex2(m[j] - mb);
                m[j] = mn;
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    s[n][2 * j] = tc::ex2(s[n][2 * j] - mb);
                    s[n][2 * j + 1] = tc::ex2(s[n][2 * j + 1] - mb);
                    sum += s[n][2 * j] + s[n][2 * j + 1];
                }
                l[j] = fmaf(l[j], f[j], sum);
            }
            if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
                for (int n = 0; n < 16; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[n][j] *= f[j >> 1];
            }
            const bool edge = u.lo > p0 || u.hi < p0 + 16;
            if (edge) {
                // values outside the span: zeros (16 rows of 256 bytes, 128 bytes a lane)
                const int key = key0 + (lane & 15), pos = t * BN + key;
                if (pos < u.lo || pos >= u.hi) {
                    const uint32_t a = base + KT + (uint32_t)(lane >> 4) * HALF + (uint32_t)key * 128u;
#pragma unroll
                    for (int y = 0; y < 8; ++y) asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a + 16 * y), "r"(0) : "memory");
                }
                __syncwarp();
            }
            // P as the left operand: the scores' layout is already that of its fragment. Two bf16 numbers a
            // weight, the second what the first's rounding left (2^-16 of the weight is lost, not 2^-8): the
            // products it costs are hidden behind the copies
            uint32_t pa[4], pb[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float e0 = s[y >> 1][2 * (y & 1)], e1 = s[y >> 1][2 * (y & 1) + 1];
                pa[y] = tc::pack_bf16(e0, e1);
                pb[y] = tc::pack_bf16(e0 - __uint_as_float(pa[y] << 16), e1 - __uint_as_float(pa[y] & 0xffff0000u));
            }
#pragma unroll
            for (int n2 = 0; n2 < 8; ++n2) {
                uint32_t b[4];
                ldsm4t(v_addr(base, n2), b);
                mma16816(o[2 * n2], pa, b[0], b[1]);
                mma16816(o[2 * n2 + 1], pa, b[2], b[3]);
                mma16816(o[2 * n2], pb, b[0], b[1]);
                mma16816(o[2 * n2 + 1], pb, b[2], b[3]);
            }
            if (edge) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(EMPTY(slot));
            next_slot();
        }
        // join the four warps: 2 and 3 into 0 and 1, then 1 into 0
        l[0] = quad_sum(l[0]);
        l[1] = quad_sum(l[1]);
        auto put = [&](int buf) {
#pragma unroll
            for (int n = 0; n < 16; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) merge[(buf * 64 + n * 4 + j) * 32 + lane] = o[n][j];
            if (c == 0) {
                sml[warp * MROWS + g] = make_float2(m[0], l[0]);
                sml[warp * MROWS + g + 8] = make_float2(m[1], l[1]);
            }
        };
        auto take = [&](int buf, int from) {
            float2 f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 y = sml[from * MROWS + g + 8 * j];
                float mm;
                f[j] = rebase(m[j], y.x, mm);
                m[j] = mm;
                l[j] = l[j] * f[j].x + y.y * f[j].y;
            }
#pragma unroll
            for (int n = 0; n < 16; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][j] = o[n][j] * f[j >> 1].x + merge[(buf * 64 + n * 4 + j) * 32 + lane] * f[j >> 1].y;
        };
        if (warp >= 2) put(warp - 2);
        if (lane == 0) sok[warp] = ok;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        ok = sok[0] && sok[1] && sok[2] && sok[3];
        if (!ok) break;                     // all four together
        if (warp < 2) take(warp, warp + 2);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (warp == 1) put(0);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (warp == 0) {
            take(0, 1);
            if (x.whole) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (!live[j]) continue;
                    const long row = row0 + g + 8 * j;
                    const float inv = l[j] > 0.f ? 1.f / l[j] : l[j] == l[j] ? 0.f : l[j];
#pragma unroll
                    for (int n = 0; n < 16; ++n)
                        *reinterpret_cast<uint32_t *>((__nv_bfloat16 *)p.o + row * D + 8 * n + 2 * c) = tc::pack_bf16(o[n][2 * j] * inv, o[n][2 * j + 1] * inv);
                    if (p.lse && c == 0) p.lse[row] = (m[j] + log2f(l[j])) * 0.69314718055994531f;
                    if (p.scores && c == 0) p.whole[(long)(x.b * p.c.H + x.h) * MROWS + g + 8 * j] = make_float2(m[j], l[j]);
                }
            } else {
                const long sl = (long)blockIdx.x * 2 + (piece == 0 ? 0 : 1);
#pragma unroll
                for (int n = 0; n < 16; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) p.part[(sl * 64 + n * 4 + j) * 32 + lane] = o[n][j];
                if (c == 0) {
                    p.ml[sl * MROWS + g] = make_float2(m[0], l[0]);
                    p.ml[sl * MROWS + g + 8] = make_float2(m[1], l[1]);
                }
            }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
    }
}

// fp32: at most RB rows.
constexpr int FN = 32, FSTAGES = 3, FT = 128;           // keys per tile, stages, threads
std::atomic<unsigned long long> g_shared_f1{0}, g_shared_f2{0}, g_shared_f4{0}, g_shared_f8{0}, g_shared_f16{0};
constexpr size_t f32_floats(int rb, int st) { return (size_t)FSTAGES * 2 * FN * st + (size_t)rb * st + 4 * 8 * rb; }

template <int RB>
__global__ void __launch_bounds__(FT) paged_token_f32_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(16) float fs[];
    __shared__ Place s_place;
    __shared__ float2 s_ml[4][RB];
    const int d = p.c.d, dp = (d + 3) & ~3, st = dp + 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *KV = fs, *Q = KV + FSTAGES * 2 * FN * st, *P = Q + RB * st + warp * 8 * RB;     // P: this warp's [8 keys][RB]
    if (p.early) asm volatile("griddepcontrol.launch_dependents;");
    if (warp == 0) {
        const Place c = place_of<FN>(p.line, blockIdx.x);
        if (lane == 0) s_place = c;
    }
    __syncthreads();
    Place at = s_place;
    Piece<FN> x;
    const int key = 8 * warp + (lane >> 2), dq = 4 * (lane & 3);            // this lane's key of a tile, first channel
    for (int piece = 0; next_piece<FN>(p.line, at, x); ++piece) {
        if (x.x.r.bad && threadIdx.x == 0) atomicOr(p.c.err, DEVERR_TABLE);
        const Span u{span_of(x.x.r, 0, p.line.mask).lo, span_of(x.x.r, x.x.r.n - 1, p.line.mask).hi};
        const long row0 = (long)(x.b * p.c.H + x.h) * p.R;
        auto load = [&](int t) {
            if (t < x.tb) {
                float *k = KV + (t % FSTAGES) * 2 * FN * st;
                f32::copy_tile<FN, FT>(p.c, x.b, x.h, t * FN, u, k, k + FN * st, st, dp);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        __syncthreads();                    // the piece before this one was read
        load(x.ta);
        load(x.ta + 1);
        for (int e = threadIdx.x; e < RB * dp; e += FT) {
            const int r = e / dp, y = e - r * dp;
            const bool in = r < p.R && y < d && frem(r, p.line.byL) < x.x.r.n;
            Q[r * st + y] = in ? ((const float *)p.q)[(row0 + r) * d + y] * p.sl2 : 0.f;
        }
        float m[RB], l[RB], acc[RB][4];
        // the rows' spans (empty for rows that are none), kept where there are registers for them
        constexpr bool KEPT = RB <= 8;
        auto row_span = [&](int r) {
            const int i = frem(r, p.line.byL);
            return r < p.R && i < x.x.r.n ? span_of(x.x.r, i, p.line.mask) : Span{0, -1};
        };
        Span kept[KEPT ? RB : 1];
        if constexpr (KEPT) {
#pragma unroll
            for (int r = 0; r < RB; ++r) kept[r] = row_span(r);
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) acc[r][y] = 0.f;
        }
        for (int t = x.ta; t < x.tb; ++t) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            load(t + 2);                    // into the stage of tile t - 1, which all have read
            const float *K = KV + (t % FSTAGES) * 2 * FN * st, *V = K + FN * st;
            float s[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) s[r] = 0.f;
#pragma unroll 2
            for (int y = dq; y < dp; y += 16) {
                const float4 k = *(const float4 *)(K + key * st + y);
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const float4 q = *(const float4 *)(Q + r * st + y);
                    s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
                }
            }
            const int pos = t * FN + key;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                s[r] += __shfl_xor_sync(0xffffffffu, s[r], 1);
                s[r] += __shfl_xor_sync(0xffffffffu, s[r], 2);
                const Span v = KEPT ? kept[KEPT ? r : 0] : row_span(r);
                if (pos < v.lo || pos >= v.hi) s[r] = -INFINITY;
                if (p.scores && v.hi >= 0 && pos < x.x.r.kv && (lane & 3) == 0) p.scores[(row0 + r) * p.line.cap + pos] = s[r];
                float mx = s[r];
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn, f = exp2f(m[r] - base);
                m[r] = mn;
                s[r] = exp2f(s[r] - base);
                l[r] = fmaf(l[r], f, s[r]);         // this lane's key; joined at the end
#pragma unroll
                for (int y = 0; y < 4; ++y) acc[r][y] *= f;
                if ((lane & 3) == 0) P[(lane >> 2) * RB + r] = s[r];
            }
            __syncwarp();
            if (4 * lane < dp) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float4 v = *(const float4 *)(V + (8 * warp + k) * st + 4 * lane);
                    constexpr int W = RB < 4 ? RB : 4;
#pragma unroll
                    for (int r = 0; r < RB; r += W) {
                        float ws[4];
                        if constexpr (W == 4) *(float4 *)ws = *(const float4 *)(P + k * RB + r);
                        else if constexpr (W == 2) *(float2 *)ws = *(const float2 *)(P + k * RB + r);
                        else ws[0] = P[k];
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            acc[r + j][0] = fmaf(ws[j], v.x, acc[r + j][0]);
                            acc[r + j][1] = fmaf(ws[j], v.y, acc[r + j][1]);
                            acc[r + j][2] = fmaf(ws[j], v.z, acc[r + j][2]);
                            acc[r + j][3] = fmaf(ws[j], v.w, acc[r + j][3]);
                        }
                    }
                }
            }
            __syncwarp();
        }
        // join the four warps through the stages' memory, in their order
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        float *M = KV;                      // [warp][RB][128]
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 4);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 8);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
            if (lane == 0) s_ml[warp][r] = make_float2(m[r], l[r]);
            if (4 * lane < dp) *(float4 *)(M + (warp * RB + r) * D + 4 * lane) = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
        }
        __syncthreads();
        const long sl = (long)blockIdx.x * 2 + (piece == 0 ? 0 : 1);
        for (int r = 0; r < min(RB, p.R); ++r) {
            if (frem(r, p.line.byL) >= x.x.r.n) continue;
            const float mm = fmaxf(fmaxf(s_ml[0][r].x, s_ml[1][r].x), fmaxf(s_ml[2][r].x, s_ml[3][r].x)), base = mm == -INFINITY ? 0.f : mm;
            float o = 0.f, ll = 0.f;
            for (int w = 0; w < 4; ++w) {
                const float f = exp2f(s_ml[w][r].x - base);
                ll = fmaf(s_ml[w][r].y, f, ll);
                if (threadIdx.x < d) o = fmaf(M[(w * RB + r) * D + threadIdx.x], f, o);
            }
            if (x.whole) {
                const float inv = ll > 0.f ? 1.f / ll : ll == ll ? 0.f : ll;
                if (threadIdx.x < d) ((float *)p.o)[(row0 + r) * d + threadIdx.x] = o * inv;
                if (threadIdx.x == 0) {
                    if (p.lse) p.lse[row0 + r] = (mm + log2f(ll)) * 0.69314718055994531f;
                    if (p.scores) p.whole[(long)(x.b * p.c.H + x.h) * MROWS + r] = make_float2(mm, ll);
                }
            } else {
                p.part[(sl * MROWS + r) * D + threadIdx.x] = o;
                if (threadIdx.x == 0) p.ml[sl * MROWS + r] = make_float2(mm, ll);
            }
        }
    }
}

// Joins the pieces of heads whose keys were cut, in the order of the blocks, and turns the scores
// into weights. Block (x, b * H + h): x < nj joins 32 of that head's items (eight channels of a row; 16 for a
// single row), x - nj = i the weights of its keys from i * keys on. The pieces' factors come first, a
// lane per piece, so that the sums over pieces wait for no chain of loads. (One joining block a head took
// 57 us for 8 rows over 19781 keys of 2 heads, 148 pieces each.)
constexpr int JT = 256, MAXP = 512;                     // threads; pieces of a head (blocks of the first kernel)
template <typename E, int TK>
__global__ void __launch_bounds__(JT) paged_token_join_kernel(const __grid_constant__ Params p)
{
    __shared__ float s_f[MAXP][MROWS];      // factor of a piece's row
    __shared__ float2 s_ml[MROWS];          // a row's maximum, and one over its sum
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y % p.c.H, b = blockIdx.y / p.c.H;
    const Roll ro = roll_of(p.line.kv_lens, p.line.new_lens, b, p.line.L, p.line.cap);
    const bool joins = (int)blockIdx.x < p.nj;
    const int k0 = ((int)blockIdx.x - p.nj) * p.keys;
    if (!joins && k0 >= ro.kv) return;
    const Holders hd = holders_of<TK>(p.line, 0, b, h);
    const bool cut = hd.T > 0 && hd.g0 != hd.g1;
    if (blockIdx.x == 0 && ro.bad && threadIdx.x == 0) atomicOr(p.c.err, DEVERR_TABLE);
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the first kernel's results from here on
    const long row0 = (long)blockIdx.y * p.R;
    const int np = cut ? hd.g1 - hd.g0 + 1 : 0;
    auto slot = [&](int i) { return (long)(hd.g0 + i) * 2 + (i == 0 ? hd.slot0 : 0); };
    if (hd.T == 0 || cut) {
        for (int r = warp; r < p.R; r += JT / 32) {
            float m = -INFINITY, l = 0.f;
            for (int i = lane; i < np; i += 32) m = fmaxf(m, p.ml[slot(i) * MROWS + r].x);
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            for (int i = lane; i < np; i += 32) {
                const float2 y = p.ml[slot(i) * MROWS + r];
                const float f = tc::ex2(y.x - (m == -INFINITY ? 0.f : m));
                s_f[i][r] = f;
                l = fmaf(y.y, f, l);
            }
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) {
                s_ml[r] = make_float2(m, l > 0.f ? 1.f / l : l == l ? 0.f : l);
                if (p.lse && blockIdx.x == 0 && frem(r, p.line.byL) < ro.n) p.lse[row0 + r] = (m + log2f(l)) * 0.69314718055994531f;
            }
        }
    } else if (p.w_out && threadIdx.x < p.R) {
        const float2 y = p.whole[(long)blockIdx.y * MROWS + threadIdx.x];
        s_ml[threadIdx.x] = make_float2(y.x, 1.f / y.y);
    }
    __syncthreads();
    if (joins && (hd.T == 0 || cut)) {
        // An item is eight channels of a row, 16 items a row (bf16: a pair of registers of the fragment
        // in four lanes); the lanes that share it take its pieces in turn.
        const int share = p.R > 1 ? 8 : 16;
        const int item = blockIdx.x * (JT / share) + threadIdx.x / share, r = item >> 4, n = item & 15;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), d = a;
        if (r < p.R) {
            // bf16: row r of the fragment is lanes 4 (r & 7) .., registers 4 n + 2 (r >> 3) and the next
            // (even and odd channels); fp32: the two words of the row's channels
            constexpr int next = sizeof(E) == 2 ? 8 : 1;
            const float4 *src = reinterpret_cast<const float4 *>(p.part) + (sizeof(E) == 2 ? (4 * n + 2 * (r >> 3)) * 8 + (r & 7) : r * 32 + 2 * n);
#pragma unroll 8
            for (int i = threadIdx.x % share; i < np; i += share) {
                const float4 u = src[slot(i) * 512], v = src[slot(i) * 512 + next];
                const float f = s_f[i][r];
                a.x = fmaf(u.x, f, a.x); a.y = fmaf(u.y, f, a.y); a.z = fmaf(u.z, f, a.z); a.w = fmaf(u.w, f, a.w);
                d.x = fmaf(v.x, f, d.x); d.y = fmaf(v.y, f, d.y); d.z = fmaf(v.z, f, d.z); d.w = fmaf(v.w, f, d.w);
            }
        }
        for (int o = share >> 1; o; o >>= 1) {
            a.x += __shfl_xor_sync(0xffffffffu, a.x, o); a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
            a.z += __shfl_xor_sync(0xffffffffu, a.z, o); a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
            d.x += __shfl_xor_sync(0xffffffffu, d.x, o); d.y += __shfl_xor_sync(0xffffffffu, d.y, o);
            d.z += __shfl_xor_sync(0xffffffffu, d.z, o); d.w += __shfl_xor_sync(0xffffffffu, d.w, o);
        }
        if (threadIdx.x % share == 0 && r < p.R && frem(r, p.line.byL) < ro.n) {
            const float inv = s_ml[r].y;
            if constexpr (sizeof(E) == 4) {
                const float y[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
                for (int x = 0; x < 8; ++x)
                    if (8 * n + x < p.c.d) ((float *)p.o)[(row0 + r) * p.c.d + 8 * n + x] = y[x] * inv;
            } else
                *reinterpret_cast<uint4 *>((__nv_bfloat16 *)p.o + (row0 + r) * D + 8 * n) = make_uint4(tc::pack_bf16(a.x * inv, d.x * inv), tc::pack_bf16(a.y * inv, d.y * inv), tc::pack_bf16(a.z * inv, d.z * inv), tc::pack_bf16(a.w * inv, d.w * inv));
        }
    }
    if (joins) return;
    const Span u = ro.n > 0 ? Span{span_of(ro, 0, p.line.mask).lo, span_of(ro, ro.n - 1, p.line.mask).hi} : Span{0, 0};
    // four keys a thread: the capacity is a multiple of 16, so neither rows nor words straddle
    const long head = (long)blockIdx.y * p.line.cap;
#pragma unroll 2
    for (int k = k0 + 4 * threadIdx.x; k < min(k0 + p.keys, ro.kv); k += 4 * JT) {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
        if (k + 3 >= u.lo && k < u.hi) {
#pragma unroll 4
            for (int r = 0; r < p.R; ++r) {
                if (frem(r, p.line.byL) >= ro.n) continue;
                const float4 y = *reinterpret_cast<const float4 *>(p.scores + (row0 + r) * p.line.cap + k);
                const float s[4] = {y.x, y.y, y.z, y.w};
                // what no row of the chunk sees was not stored; a key that this row does not see is
                // -inf (a row that sees none: no NaN from -inf + inf)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (k + j >= u.lo && k + j < u.hi && s[j] != -INFINITY) t[j] = fmaf(tc::ex2(s[j] - s_ml[r].x), s_ml[r].y, t[j]);
            }
        }
        float old[4] = {0.f, 0.f, 0.f, 0.f};
        if (p.w_in && k < ro.h) {
            if (k + 3 < ro.h && !((uintptr_t)p.w_in & 15u)) {
                const float4 y = *reinterpret_cast<const float4 *>(p.w_in + head + k);
                old[0] = y.x; old[1] = y.y; old[2] = y.z; old[3] = y.w;
            } else {
                for (int j = 0; j < 4; ++j)
                    if (k + j < ro.h) old[j] = p.w_in[head + k + j];
            }
        }
        for (int j = 0; j < 4; ++j)
            if (p.w_in && k + j < ro.h) t[j] = fmaf(p.decay, old[j], t[j]);
        if (k + 3 < ro.kv && !((uintptr_t)p.w_out & 15u)) {
            *reinterpret_cast<float4 *>(p.w_out + head + k) = make_float4(t[0], t[1], t[2], t[3]);
        } else {
            for (int j = 0; j < 4; ++j)
                if (k + j < ro.kv) p.w_out[head + k + j] = t[j];
        }
    }
}

size_t part_bytes() { return (size_t)device_sms() * 4 * (64 * 32 * 4 + MROWS * 8); }

}  // namespace

// The scores kept for the weights grow with rollouts x rows x capacity: past 1 GiB the chunk kernel
// and a second pass over K serve instead.
bool paged_token_fits(int B, int H, int G, long L, int cap, bool weights)
{
    return G * L <= MROWS && (!weights || (double)B * H * G * L * cap * 4 <= (double)(1L << 30));
}

size_t paged_token_bytes(int B, int H, int G, long L, int cap, bool weights)
{
    return part_bytes() + (weights ? (size_t)B * H * (G * L * (size_t)cap * 4 + MROWS * 8) : 0);
}

cudaError_t launch_paged_token(const PagedAttnArgs &a, bool bf16, cudaStream_t s)
{
    const long kv_rows = a.c.num_pages * a.c.H << a.c.page_log2;
    if ((bf16 && kv_rows + BN >= (1L << 31)) || (long)a.B * a.c.H > 65535) return cudaErrorNotSupported;
    cudaError_t e = cudaSuccess;
    const int sms = device_sms(), tile = bf16 ? BN : FN;
    Params p;
    p.c = a.c;
    p.G = a.G;
    p.R = (int)(a.G * a.L);
    // no more blocks than the longest rollouts have tiles
    const long most = (long)a.B * a.c.H * (((a.c.max_pages << a.c.page_log2) + tile - 1) / tile);
    // bf16: a head's start and end cost about two tiles (64 tokens over 10 to 500 keys of 8 heads 32.8 us with none, 27.0
    // with one, 26.0 with two, 27.3 with four; 24 x 2 over 100 to 4000 55.1, 47.5, 44.7, 44.7); fp32: tiles
    // cost as much as they do (32 over 50 to 1000 keys 50.6, 49.4, 50.8, 55.4)
    p.line = line_of(a, 1, (int)std::min<long>(std::min<long>(2L * sms, MAXP), most), 1, 1, 1, bf16 ? 2 : 0);
    p.sl2 = a.sl2;
    p.q = a.q;
    p.o = a.o;
    p.lse = a.lse;
    p.part = (float *)a.ws;
    p.ml = (float2 *)((char *)a.ws + (size_t)sms * 4 * 64 * 32 * 4);
    p.whole = (float2 *)((char *)a.ws + part_bytes());
    p.scores = a.w_out ? (float *)(p.whole + (size_t)a.B * a.c.H * MROWS) : nullptr;
    p.w_in = a.w_in; p.w_out = a.w_out; p.decay = a.decay;
    p.nj = std::max(1, (p.R + 1) / 2);
    // Early blocks gather on the SMs that the first kernel leaves first: 1 us won where they have little to
    // read (one token over 1560 keys of 8 heads 11.3 us, 12.1 late), lost where they have much (8 rows over
    // 19781 keys of 2 heads 42 us, 22 late; 16 rows over 6861 keys of 10 heads 27 and 21).
    p.early = p.R <= 3;
    // long runs of keys a block, unless there are too few to fill the SMs twice
    p.keys = 4096;
    while (p.keys > 1024 && (long)a.B * a.c.H * ((p.line.cap + p.keys - 1) / p.keys) < 2L * sms) p.keys /= 2;
    if (bf16) {
        const uint32_t box = (uint32_t)std::min(1 << a.c.page_log2, BN);
        CUtensorMap mk, mv;
        if ((e = make_tmap_2d_bf16(&mk, a.c.k, kv_rows, D, 64, box, true)) != cudaSuccess) return e;
        if ((e = make_tmap_2d_bf16(&mv, a.c.v, kv_rows, D, 64, box, true)) != cudaSuccess) return e;
        if ((e = allow_shared((const void *)paged_token_kernel, SMEM_BYTES, g_shared)) != cudaSuccess) return e;
        paged_token_kernel<<<p.line.ngang, THREADS, SMEM_BYTES, s>>>(mk, mv, p), note_launch();
    } else {
        const int st = ((a.c.d + 3) & ~3) + 4;
        // the stages also hold the four warps' outputs at the end of a piece
        const int rb = p.R <= 1 ? 1 : p.R <= 2 ? 2 : p.R <= 4 ? 4 : p.R <= 8 ? 8 : 16;
        const size_t need = std::max(f32_floats(rb, st), (size_t)4 * rb * D) * 4;
        auto go = [&](void (*kernel)(Params), std::atomic<unsigned long long> &done) {
            if ((e = allow_shared((const void *)kernel, f32_floats(rb, 132) * 4, done)) != cudaSuccess) return;
            kernel<<<p.line.ngang, FT, need, s>>>(p), note_launch();
        };
        if (rb == 1) go(paged_token_f32_kernel<1>, g_shared_f1);
        else if (rb == 2) go(paged_token_f32_kernel<2>, g_shared_f2);
        else if (rb == 4) go(paged_token_f32_kernel<4>, g_shared_f4);
        else if (rb == 8) go(paged_token_f32_kernel<8>, g_shared_f8);
        else go(paged_token_f32_kernel<16>, g_shared_f16);
        if (e != cudaSuccess) return e;
    }
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.nj + (a.w_out ? (p.line.cap + p.keys - 1) / p.keys : 0)), (unsigned)(a.B * a.c.H));
    cfg.blockDim = dim3(JT);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = bf16 ? cudaLaunchKernelEx(&cfg, paged_token_join_kernel<__nv_bfloat16, BN>, p) : cudaLaunchKernelEx(&cfg, paged_token_join_kernel<float, FN>, p);
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace hlta
