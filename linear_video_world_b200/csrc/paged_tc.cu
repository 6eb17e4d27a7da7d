// Attention of a chunk over a paged cache, bf16, head dim 128, on the sm_100a tensor cores.
//
// Exact softmax by 128-key tiles with a running maximum and sum. The division of the work over the
// GPU (gangs over a line of key tiles, pieces joined by a second kernel) is in paged.cuh; a row
// tile is 256 packed rows (two sub-tiles of 128) of one key head, so the query heads that share a
// key head share its tiles too.
// Roles of a block's 12 warps (one block per SM):
//   warps 0-3 / 4-7  softmax of sub-tile 0 / 1, one thread per row (its tensor-memory lane)
//   warp 8           producer: per share Q, then K and V tiles through one ring of three 32 KB slots
//                    in the order K0, K1, V0, K2, V1, ...; a lane per page of the tile looks the
//                    page up and copies it by TMA to its rows of the swizzled tile (a page holds
//                    whole groups of eight rows, so page and tile swizzle alike)
//   warps 9, 10      issuers of the products of sub-tile 0 / 1 (one thread for both left the tensor
//                    cores idle between its groups of products: 1.09 PFLOP/s in place of 1.17)
//   warp 11          completes the warpgroup that gives registers to the softmax warps
// S = Q K^T goes to tensor memory, the softmax reads a row's 128 scores into registers and frees it
// at once, so S of the next tile is done while P of this one is formed; P goes to shared memory, once
// the previous P V has read it (half of this tile's exponentials are done by then).
// What bounds it: per tile of 2 x 128 rows the products take 2051 cycles (64 per 128 x 128 x 16,
// measured, from shared or tensor memory alike; a product of 64 keys takes 62, so tiles are not
// halved), the exponentials 2048 (16 a cycle). So neither may wait for the other. Measured: 3260
// cycles a tile, 1.17 PFLOP/s on full row tiles; a frame of 1560 rows, six row tiles and 24 rows of a
// seventh, over 4 x 7800-32760 keys of 8 heads runs into the 1000 W power cap (1.38 GHz) at 606 us, 0.86
// PFLOP/s. Part of the exponentials on the FMA pipe (one pair in eight to three) was slower by 3 to 9 %.
// The softmax has to stay in registers: 168 a thread (what 384 threads may have) spilled, and with
// all of the SM's memory given to shared memory a spilled register comes back from L2. The last
// warpgroup gives its registers to the other two (96 / 200), and the share's bookkeeping is worked
// out twice instead of being kept across the tiles.
// O is rescaled only when a row's maximum grew by more than 2^8 (numerator and denominator share
// the stale maximum). P is rounded to bf16 for the tensor cores (half a step, 2^-8 of each weight),
// the sums are taken in fp32 before that rounding.
//
// What the cache holds where no row looks: pages without a visible key are not copied; keys that a
// row does not see are masked to -inf before the maximum, whatever their score (NaN too), and the
// values of keys outside the row tile's span are zeroed in shared memory before P V, since a weight
// of zero times NaN is NaN.
//
// Every mbarrier wait is bounded; on expiry the kernel records DEVERR_ATTN_WAIT, every role
// stops, and the tensor memory is released.
#include "hlta_internal.cuh"
#include "paged.cuh"
#include "sm100_ptx.cuh"
#include "tc_ptx.cuh"

#include <algorithm>
#include <math.h>

namespace hlta {
namespace {

using namespace ptx;
using namespace paged;

constexpr int BM = 128, QT = 2, ROWS = BM * QT;     // rows per sub-tile, sub-tiles, rows per block
constexpr int BN = 128, D = 128;                    // keys per tile, head dim
constexpr int THREADS = 384;
constexpr int WARP_TMA = 8, WARP_MMA = 9;
constexpr uint32_t HALF = 128 * 128;                // [128 rows][64 columns] bf16
constexpr uint32_t TILE = 2 * HALF;
constexpr int NSLOT = 3;
constexpr uint32_t SM_Q = 0, SM_SLOT = QT * TILE, SM_P = SM_SLOT + NSLOT * TILE, SM_BAR = SM_P + QT * TILE;
constexpr uint32_t TMEM_COLS = 512;                 // S of sub-tile q at 128 q, O at 256 + 128 q
enum {
    B_QFULL, B_QFREE,
    B_FULL, B_EMPTY = B_FULL + NSLOT,               // per slot
    B_SFULL = B_EMPTY + NSLOT,                      // per sub-tile from here
    B_SFREE = B_SFULL + QT, B_PFULL = B_SFREE + QT,
    B_PVDONE = B_PFULL + QT, B_ODONE = B_PVDONE + QT, B_OFREE = B_ODONE + QT, NBARS = B_OFREE + QT
};
constexpr uint32_t SM_PLACE = SM_BAR + 8 * NBARS;   // the block's start on the line; the softmax warps' places
constexpr uint32_t SM_TMEM = SM_PLACE + 9 * 32, SM_ABORT = SM_TMEM + 4;
std::atomic<unsigned long long> g_shared{0};
constexpr size_t SMEM_BYTES = SM_ABORT + 4;
static_assert(SMEM_BYTES <= 232448, "shared memory of one block");
static_assert(sizeof(Place) <= 32, "place");

struct Params {
    Line line;
    PagedKV c;
    int G, R, nr;                   // query heads a key head; packed rows; row tiles
    float sl2;
    __nv_bfloat16 *o;
    float *lse;
    float *part;                    // [block][2][32 column quads][256 rows] float4
    float2 *ml;                     // [block][2][256 rows] (maximum, sum)
};

__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 pa, pb, pc, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
        "mov.b64 pc, {%6, %7};\n\tfma.rn.f32x2 pd, pa, pb, pc;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 pa, pb, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
        "add.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// 128 consecutive fp32 columns: both loads in flight before the wait
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, uint32_t (&x)[128])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%128];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
        "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
        "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
        "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%129];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : TC_REGS32(x), TC_REGS32((x + 32)), TC_REGS32((x + 64)), TC_REGS32((x + 96))
        : "r"(taddr), "r"(taddr + 64u)
        : "memory");
}

// The bounded wait of sm100_ptx.cuh, inlined: a kernel that moves registers between its warpgroups
// may not call functions.
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, volatile int *abort_flag, unsigned int *err)
{
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try(bar, parity)) return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > (1LL << 32)) {
            *abort_flag = 1;
            atomicOr(err, DEVERR_ATTN_WAIT);
            return false;
        }
    }
}

// The span of the live rows among packed rows [r0, r1): tokens of a range that stays inside one
// head are consecutive, one that runs into the next head covers the first or every token.
__device__ __forceinline__ Span rows_span(const Params &p, const Roll &ro, int r0, int r1)
{
    const int L = p.line.L;
    r1 = min(r1, p.R);
    if (r0 >= r1) return Span{0, 0};
    int i0 = frem(r0, p.line.byL), i1 = i0 + (r1 - 1 - r0);
    if (i1 >= L) {
        // the range holds the head's last tokens and the next head's first ones
        i0 = 0;
        i1 = L - 1;
    }
    if (i0 >= ro.n) return Span{0, 0};
    Span s;
    s.lo = span_of(ro, i0, p.line.mask).lo;
    s.hi = span_of(ro, min(i1, ro.n - 1), p.line.mask).hi;
    if (s.hi <= s.lo) s.lo = s.hi = 0;
    return s;
}

// A block's share of a piece: its row tile, the span of its rows, the key tiles of each sub-tile.
struct Share {
    Piece<BN> x;
    int rt;
    Span u;                         // span of the row tile
    int ta, tb;                     // key tiles of the piece that the span touches
    int a0, b0, a1, b1;             // of which sub-tile 0 / 1 needs [a, b)
};
__device__ __forceinline__ bool next_share(const Params &p, Place &c, int member, Share &s)
{
    if (!next_piece<BN>(p.line, c, s.x)) return false;
    s.rt = s.x.pass * p.line.gs + member;
    const int r0 = s.rt * ROWS;
    auto clip = [&](const Span &v, int &a, int &b) {
        a = max(s.x.ta, v.lo / BN);
        b = min(s.x.tb, (v.hi + BN - 1) / BN);
        if (v.hi <= v.lo || b < a) a = b = s.x.ta;
    };
    const Span v0 = rows_span(p, s.x.x.r, r0, r0 + BM), v1 = rows_span(p, s.x.x.r, r0 + BM, r0 + ROWS);
    clip(v0, s.a0, s.b0);
    clip(v1, s.a1, s.b1);
    const bool e0 = v0.hi > v0.lo, e1 = v1.hi > v1.lo;
    s.u.lo = e0 && e1 ? min(v0.lo, v1.lo) : e0 ? v0.lo : v1.lo;
    s.u.hi = max(v0.hi, v1.hi);
    // the tiles walked: from the first to the last that either sub-tile needs
    const bool n0 = s.b0 > s.a0, n1 = s.b1 > s.a1;
    s.ta = n0 && n1 ? min(s.a0, s.a1) : n0 ? s.a0 : s.a1;
    s.tb = max(n0 ? s.b0 : s.ta, n1 ? s.b1 : s.ta);
    return true;
}

__global__ void __launch_bounds__(THREADS, 1)
paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t smem[];   // the swizzled tiles repeat every 1024 bytes
    const uint32_t sbase = smem_u32(smem);
    auto BAR = [&](int i) { return sbase + SM_BAR + 8u * (uint32_t)i; };
    volatile int *abort_flag = (volatile int *)(smem + SM_ABORT);
    uint32_t *tmem_slot = (uint32_t *)(smem + SM_TMEM);
    auto place = [&](int i) { return (Place *)(smem + SM_PLACE + 32 * i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gang = blockIdx.x / p.line.gs, member = blockIdx.x % p.line.gs;

    asm volatile("griddepcontrol.launch_dependents;");      // the second kernel may be set up meanwhile
    if (sbase & 1023u) {                    // not seen: the attribute asks for it
        if (threadIdx.x == 0) atomicOr(p.c.err, DEVERR_ATTN_WAIT);
        return;
    }
    if (threadIdx.x == 0) {
        mbar_init(BAR(B_QFULL), 1);
        mbar_init(BAR(B_QFREE), 2);
        for (int i = 0; i < NSLOT; ++i) {
            mbar_init(BAR(B_FULL + i), 1);
            mbar_init(BAR(B_EMPTY + i), 2);
        }
        for (int q = 0; q < QT; ++q) {
            mbar_init(BAR(B_SFULL + q), 1);
            mbar_init(BAR(B_SFREE + q), BM);
            mbar_init(BAR(B_PFULL + q), BM);
            mbar_init(BAR(B_PVDONE + q), 1);
            mbar_init(BAR(B_ODONE + q), 1);
            mbar_init(BAR(B_OFREE + q), BM);
        }
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == WARP_TMA && lane < 3)
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)(lane == 0 ? &tq : lane == 1 ? &tk : &tv)) : "memory");
    if (warp == WARP_TMA) {
        const Place c = place_of<BN>(p.line, gang);
        if (lane < 9) *place(lane) = c;
    }
    if (warp == WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto wait_bar = [&](uint32_t bar, uint32_t parity) -> bool {
        return wait_inline(bar, parity, abort_flag, p.c.err);
    };
    // A share's ring items: K of its first tile, then K of tile j + 1 and V of tile j in turn. With n
    // tiles, K(j) is item 2j - 1 (j >= 1), V(j) item 2j + 2, the last V item 2n - 1.

    if (warp >= WARP_TMA) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == WARP_TMA) {
            Place at = *place(0);
            Share s;
            int it = 0, units = 0;
            bool ok = true;
            const int psz = 1 << p.c.page_log2, npg = BN >> p.c.page_log2;
            while (ok && next_share(p, at, member, s)) {
                if (s.tb <= s.ta) continue;
                if (s.x.x.r.bad && lane == 0) atomicOr(p.c.err, DEVERR_TABLE);
                // the page of this lane's part of tile t, or -1 when none of its positions is seen
                auto page_at = [&](int t) -> int {
                    const int p0 = t * BN + lane * psz;
                    return lane < npg && p0 < s.u.hi && p0 + psz > s.u.lo ? page_of(p.c, s.x.b, max(p0, s.u.lo)) : -1;
                };
                auto load = [&](const CUtensorMap *map, int pg) -> bool {
                    const int sl = it % NSLOT;
                    bool w = true;
                    if (lane == 0 && it >= NSLOT) w = wait_bar(BAR(B_EMPTY + sl), (uint32_t)((it / NSLOT) + 1) & 1u);
                    if (!__shfl_sync(0xffffffffu, w, 0)) return false;
                    const unsigned have = __ballot_sync(0xffffffffu, pg >= 0);
                    if (lane == 0) mbar_expect_tx(BAR(B_FULL + sl), (uint32_t)__popc(have) * (uint32_t)psz * 256u);
                    __syncwarp();
                    if (pg >= 0) {
                        const int row = (pg * p.c.H + s.x.h) << p.c.page_log2;
                        const uint32_t dst = sbase + SM_SLOT + (uint32_t)sl * TILE + (uint32_t)(lane * psz) * 128u;
                        tma_load_2d(dst, map, 0, row, BAR(B_FULL + sl));
                        tma_load_2d(dst + HALF, map, 64, row, BAR(B_FULL + sl));
                    }
                    ++it;
                    return true;
                };
                int pg = page_at(s.ta);
                if (units > 0) {
                    bool w = true;
                    if (lane == 0) w = wait_bar(BAR(B_QFREE), (uint32_t)(units - 1) & 1u);
                    if (!(ok = __shfl_sync(0xffffffffu, w, 0))) break;
                }
                if (lane == 0) {
                    const int row = (s.x.b * p.c.H + s.x.h) * p.R + s.rt * ROWS;
                    mbar_expect_tx(BAR(B_QFULL), QT * TILE);
                    for (int q = 0; q < QT; ++q)
                        for (int x = 0; x < 2; ++x)
                            tma_load_2d(sbase + SM_Q + q * TILE + x * HALF, &tq, 64 * x, row + q * BM, BAR(B_QFULL));
                }
                ++units;
                ok = load(&tk, pg);
                for (int t = s.ta; ok && t < s.tb; ++t) {
                    const int v_pg = pg;                          // K and V share pages
                    if (t + 1 < s.tb) {
                        pg = page_at(t + 1);
                        if (!(ok = load(&tk, pg))) break;
                    }
                    ok = load(&tv, v_pg);
                }
            }
            if (lane == 0 && *abort_flag) {
                // a bounded wait expired somewhere: let the copies this block issued land
                const long long t0 = clock64();
                for (int i = it - 1; i >= 0 && i >= it - NSLOT; --i)
                    while (!mbar_try(BAR(B_FULL + i % NSLOT), (uint32_t)(i / NSLOT) & 1u) && clock64() - t0 < (1LL << 31)) {}
                if (units > 0)
                    while (!mbar_try(BAR(B_QFULL), (uint32_t)(units - 1) & 1u) && clock64() - t0 < (1LL << 31)) {}
            }
        } else if (warp < WARP_MMA + QT) {
            if (lane == 0) {
                const int q = warp - WARP_MMA;
                constexpr uint32_t IDESC_S = tc::idesc_bf16(BM, BN, false, false), IDESC_O = tc::idesc_bf16(BM, D, false, true);
                const uint64_t dq = tc::sw128_desc(sbase + SM_Q + q * TILE, 16, 1024);
                const uint64_t dk0 = tc::sw128_desc(sbase + SM_SLOT, 16, 1024);       // K-major (K)
                const uint64_t dv0 = tc::sw128_desc(sbase + SM_SLOT, HALF, 1024);     // MN-major (V)
                const uint64_t dp = tc::sw128_desc(sbase + SM_P + q * TILE, 16, 1024);
                const uint32_t s_tm = tmem + 128u * q, o_tm = tmem + 256u + 128u * q;
                const uint32_t sfull = BAR(B_SFULL + q), sfree = BAR(B_SFREE + q), pfull = BAR(B_PFULL + q), pvdone = BAR(B_PVDONE + q), ofree = BAR(B_OFREE + q);
                Place at = *place(0);
                uint32_t slot = 0, lap = 0;                           // the next ring item, the parity of its lap
                uint32_t s_par = 0, p_par = 0;                        // parities of the next S, the next P
                bool any_s = false;                                   // an S was issued before
                int units = 0;
                bool ok = true;
                auto item = [&]() -> bool { return wait_bar(BAR(B_FULL) + 8u * slot, lap); };
                auto next_item = [&] {
                    if (++slot == NSLOT) {
                        slot = 0;
                        lap ^= 1u;
                    }
                };
                while (ok) {
                    int a, b, ta, tb;
                    {
                        Share s;
                        if (!next_share(p, at, member, s)) break;
                        a = q ? s.a1 : s.a0;
                        b = q ? s.b1 : s.b0;
                        ta = s.ta;
                        tb = s.tb;
                    }
                    if (tb <= ta) continue;
                    if (!(ok = wait_bar(BAR(B_QFULL), (uint32_t)units & 1u))) break;
                    // S of tile t, once the softmax has read the previous S
                    auto do_s = [&](int t) -> bool {
                        if (!item()) return false;
                        if (t >= a && t < b) {
                            if (any_s && !wait_bar(sfree, s_par ^ 1u)) return false;
                            tc::fence_after_sync();
                            const uint64_t dk = dk0 + (uint64_t)(slot * (TILE >> 4));
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint64_t off = (uint64_t)((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
                                tc::umma_bf16(s_tm, dq + off, dk + off, IDESC_S, kk > 0 ? 1u : 0u);
                            }
                            tc::umma_commit(sfull);
                            tc::umma_commit(BAR(B_EMPTY) + 8u * slot);
                            any_s = true;
                            s_par ^= 1u;
                        } else {
                            mbar_arrive(BAR(B_EMPTY) + 8u * slot);
                        }
                        next_item();
                        if (t + 1 == tb) tc::umma_commit(BAR(B_QFREE));               // the share's last S was issued
                        return true;
                    };
                    // O += P V of tile t
                    auto do_pv = [&](int t) -> bool {
                        if (!item()) return false;
                        if (t >= a && t < b) {
                            if (!wait_bar(pfull, p_par)) return false;
                            // the share's first P V overwrites O: the previous epilogue must have read it
                            if (t == a && units > 0 && !wait_bar(ofree, (uint32_t)(units - 1) & 1u)) return false;
                            tc::fence_after_sync();
                            const uint64_t dv = dv0 + (uint64_t)(slot * (TILE >> 4));
                            const uint32_t acc = t > a ? 1u : 0u;
#pragma unroll
                            for (int kk = 0; kk < BN / 16; ++kk) {
                                tc::umma_bf16(o_tm, dp + ((uint64_t)((kk >> 2) * HALF + (kk & 3) * 32) >> 4), dv + (uint64_t)((kk * 2048) >> 4), IDESC_O,
                                              kk > 0 ? 1u : acc);
                            }
                            tc::umma_commit(pvdone);
                            tc::umma_commit(BAR(B_EMPTY) + 8u * slot);
                            p_par ^= 1u;
                        } else {
                            mbar_arrive(BAR(B_EMPTY) + 8u * slot);
                        }
                        next_item();
                        return true;
                    };
                    ok = do_s(ta);
                    for (int t = ta; ok && t < tb; ++t) ok = (t + 1 >= tb || do_s(t + 1)) && do_pv(t);
                    if (!ok) break;
                    // a share without a P V of this sub-tile still waits for its previous epilogue, so that
                    // its completion never runs two shares ahead of the softmax
                    if (a >= b && units > 0 && !(ok = wait_bar(ofree, (uint32_t)(units - 1) & 1u))) break;
                    tc::umma_commit(BAR(B_ODONE + q));
                    ++units;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int q = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_tm = tlane + 128u * q, o_tm = tlane + 256u + 128u * q;
        const uint32_t prow = sbase + SM_P + (uint32_t)q * TILE + (uint32_t)row * 128u;
        const uint32_t rx = (uint32_t)(row & 7);
        constexpr float LAZY = 8.f;
        bool ok = true;
        int k = 0, units = 0, items = 0;
        for (int piece = 0;; ++piece) {
            int a, b, ta, tb, ulo, uhi, vlo, vhi;
            {
                Place at = *place(1 + warp);
                Share s;
                if (!next_share(p, at, member, s)) break;
                const int r = s.rt * ROWS + q * BM + row, i = frem(r, p.line.byL);
                // a row that is none takes the row tile's span: it computes what nobody reads, and
                // its warp keeps to the unmasked path
                const Span v = r < p.R && i < s.x.x.r.n ? span_of(s.x.x.r, i, p.line.mask) : s.u;
                a = q ? s.a1 : s.a0;
                b = q ? s.b1 : s.b0;
                ta = s.ta;
                tb = s.tb;
                ulo = s.u.lo; uhi = s.u.hi;
                vlo = v.lo; vhi = v.hi;
            }
            __syncwarp();
            float m = -INFINITY, lsum = 0.f;
            const int k0 = k;
            for (int t = a; t < b; ++t, ++k) {
                if (!(ok = __all_sync(0xffffffffu, wait_bar(BAR(B_SFULL + q), (uint32_t)k & 1u)))) break;
                tc::fence_after_sync();
                uint32_t sv[128];
                tmem_ld128(s_tm, sv);
                tc::fence_before_sync();
                mbar_arrive(BAR(B_SFREE + q));
                const int p0 = t * BN;
                if (__any_sync(0xffffffffu, vlo > p0 || vhi < p0 + BN)) {
                    const int lo = vlo - p0, hi = vhi - p0;
#pragma unroll
                    for (int x = 0; x < BN; ++x)
                        if (x < lo || x >= hi) sv[x] = __float_as_uint(-INFINITY);
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int x = 0; x < BN / 2; ++x)
                    asm("max.f32 %0, %0, %1, %2;" : "+f"(mx[x & 3]) : "f"(__uint_as_float(sv[2 * x])), "f"(__uint_as_float(sv[2 * x + 1])));
                const float mnew = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.sl2);
                const bool need = mnew > m + LAZY;
                const float alpha = (need && m != -INFINITY) ? tc::ex2(m - mnew) : 1.f;
                const bool resc = __any_sync(0xffffffffu, need && m != -INFINITY);
                if (need) m = mnew;
                const float negm = m == -INFINITY ? 0.f : -m;
                const float2 sl = make_float2(p.sl2, p.sl2), nm = make_float2(negm, negm);
                float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t pk[32];
                // P of 64 keys into registers; stored when the previous P V is done
                auto half = [&](int h) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        const float2 e = ffma2(make_float2(__uint_as_float(sv[64 * h + 2 * x]), __uint_as_float(sv[64 * h + 2 * x + 1])), sl, nm);
                        const float2 w = make_float2(tc::ex2(e.x), tc::ex2(e.y));
                        ps[x & 1] = fadd2(ps[x & 1], w);
                        pk[x] = tc::pack_bf16(w.x, w.y);
                    }
                };
                auto store = [&](int h) {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(prow + (uint32_t)h * HALF + ((((uint32_t)c) ^ rx) << 4)),
                                     "r"(pk[c * 4]), "r"(pk[c * 4 + 1]), "r"(pk[c * 4 + 2]), "r"(pk[c * 4 + 3])
                                     : "memory");
                };
                half(0);
                if (k >= 1 && !(ok = __all_sync(0xffffffffu, wait_bar(BAR(B_PVDONE + q), (uint32_t)(k - 1) & 1u)))) break;
                store(0);
                half(1);
                store(1);
                if (resc) {
                    tc::fence_after_sync();
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t orow[32];
                        tc::tmem_ld32(o_tm + cc * 32, orow);
#pragma unroll
                        for (int x = 0; x < 32; ++x) orow[x] = __float_as_uint(__uint_as_float(orow[x]) * alpha);
                        tc::tmem_st32(o_tm + cc * 32, orow);
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                }
                if (ulo > p0 || uhi < p0 + BN) {
                    // values outside the row tile's span: zeros (each sub-tile that reads the tile
                    // writes them before its own P V)
                    const int item = items + (t + 1 < tb ? 2 * (t - ta) + 2 : 2 * (t - ta) + 1), vs = item % NSLOT;
                    if (!(ok = __all_sync(0xffffffffu, wait_bar(BAR(B_FULL + vs), (uint32_t)(item / NSLOT) & 1u)))) break;
                    if (p0 + row < ulo || p0 + row >= uhi) {
                        const uint32_t vrow = sbase + SM_SLOT + (uint32_t)vs * TILE + (uint32_t)row * 128u;
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vrow + (c >> 3) * HALF + (c & 7) * 16), "r"(0) : "memory");
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(BAR(B_PFULL + q));
                lsum = lsum * alpha + ((ps[0].x + ps[0].y) + (ps[1].x + ps[1].y));
            }
            if (!ok) break;
            Place at = *place(1 + warp);
            Share s;
            next_share(p, at, member, s);
            const int n = s.tb - s.ta;
            __syncwarp();
            if (lane == 0) *place(1 + warp) = at;
            __syncwarp();
            if (n > 0) {
                if (!(ok = __all_sync(0xffffffffu, wait_bar(BAR(B_ODONE + q), (uint32_t)units & 1u)))) break;
                tc::fence_after_sync();
                ++units;
            }
            items += 2 * n;
            const bool have = k > k0;
            const int r = s.rt * ROWS + q * BM + row;
            const bool live = r < p.R && frem(r, p.line.byL) < s.x.x.r.n;
            const long grow = (long)(s.x.b * p.c.H + s.x.h) * p.R + r;
            const int rr = q * BM + row;
            const long slot = (long)blockIdx.x * 2 + (piece == 0 ? 0 : 1);
            float inv = 1.f;
            if (s.x.whole) {
                inv = lsum > 0.f ? 1.f / lsum : lsum == lsum ? 0.f : lsum;
                if (p.lse && live) p.lse[grow] = (m + log2f(lsum)) * 0.69314718055994531f;
            } else if (live) {
                p.ml[slot * ROWS + rr] = make_float2(m, lsum);
            }
            // (a whole piece's rows go through this warp's rows of P, whose last product is done: stored
            // from the accumulators, 16 bytes of 32 rows an access, they took 1 us more)
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t ov[32];
                __syncwarp();
                if (have) tc::tmem_ld32(o_tm + cc * 32, ov);
                if (s.x.whole) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            w[y] = have ? tc::pack_bf16(__uint_as_float(ov[8 * x + 2 * y]) * inv, __uint_as_float(ov[8 * x + 2 * y + 1]) * inv) : 0u;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(prow + (uint32_t)(cc >> 1) * HALF + ((((uint32_t)(cc & 1) * 4u + x) ^ rx) << 4)),
                                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                } else if (have && live) {
                    float4 *dst = reinterpret_cast<float4 *>(p.part) + (slot * (D / 4) + 8 * cc) * ROWS + rr;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        dst[x * ROWS] = make_float4(__uint_as_float(ov[4 * x]), __uint_as_float(ov[4 * x + 1]), __uint_as_float(ov[4 * x + 2]), __uint_as_float(ov[4 * x + 3]));
                }
            }
            if (s.x.whole) {
                // two rows an access, half a warp each
                const unsigned rows_live = __ballot_sync(0xffffffffu, live);
                uint4 *dst = reinterpret_cast<uint4 *>(p.o + (grow - lane) * D) + (lane & 15);
#pragma unroll 2
                for (int i = lane >> 4; i < 32; i += 2) {
                    const uint32_t from = prow - (uint32_t)lane * 128u + (uint32_t)i * 128u + (uint32_t)((lane >> 3) & 1) * HALF + (uint32_t)(((lane & 7) ^ (i & 7)) << 4);
                    uint4 w;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(from) : "memory");
                    if (rows_live >> i & 1u) dst[i * (D / 8)] = w;
                }
                __syncwarp();
            }
            if (n > 0) {
                tc::fence_before_sync();
                mbar_arrive(BAR(B_OFREE + q));
            }
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == WARP_MMA) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

// Joins the pieces of heads whose keys were cut, in the order of the gangs; rows that see no key
// get zeros here. A block takes 32 rows (a lane each): the pieces' factors first, the warps taking
// them in turn, then 4 W channels a warp, the loads of four pieces in flight (128 rows over 5000 keys
// of 2 heads, 40 pieces each: the call took 42 us with a chain of loads, 32 so). W = 4, a block for all
// channels; W = 1, four blocks, where the rows are too few to fill half of the SMs (the same 27.8 and 23.8;
// 224 blocks of W = 4, whole pieces: 17.2 and 21.1).
constexpr int MAXG = 160;               // pieces whose factors are kept; there are no more gangs
template <int W>
__global__ void __launch_bounds__(256) paged_join_tc_kernel(const __grid_constant__ Params p)
{
    __shared__ float s_f[MAXG][32];
    __shared__ float s_m[8][32], s_l[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nb = (p.R + 31) / 32, quad = (blockIdx.y * 8 + warp) * W;         // this warp's first four channels
    const int bh = blockIdx.x / nb, r = (blockIdx.x % nb) * 32 + lane;
    const int b = bh / p.c.H, h = bh % p.c.H;
    const int rt = r / ROWS, pass = rt / p.line.gs, member = rt % p.line.gs, rr = r % ROWS;
    const Holders g = holders_of<BN>(p.line, pass, b, h);
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the first kernel's results from here on
    if (g.T > 0 && g.g0 == g.g1) return;
    const Roll ro = roll_of(p.line.kv_lens, p.line.new_lens, b, p.line.L, p.line.cap);
    if (ro.bad && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.c.err, DEVERR_TABLE);
    const bool live = r < p.R && frem(r, p.line.byL) < ro.n;
    const int np = g.T > 0 ? g.g1 - g.g0 + 1 : 0;
    auto slot = [&](int i) { return ((long)(g.g0 + i) * p.line.gs + member) * 2 + (i == 0 ? g.slot0 : 0); };
    float m = -INFINITY;
    for (int i = warp; i < np; i += 8)
        if (live) m = fmaxf(m, p.ml[slot(i) * ROWS + rr].x);
    s_m[warp][lane] = m;
    __syncthreads();
    for (int w = 0; w < 8; ++w) m = fmaxf(m, s_m[w][lane]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int i = warp; i < np; i += 8) {
        const float2 y = live ? p.ml[slot(i) * ROWS + rr] : make_float2(-INFINITY, 0.f);
        // none of the piece's keys: no output was written
        const float f = y.x == -INFINITY && y.y == 0.f ? 0.f : exp2f(y.x - base);
        s_f[i][lane] = f;
        l = fmaf(y.y, f, l);
    }
    s_l[warp][lane] = l;
    __syncthreads();
    l = 0.f;
    for (int w = 0; w < 8; ++w) l += s_l[w][lane];
    if (!live) return;
    float4 acc[W];
#pragma unroll
    for (int x = 0; x < W; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < np; ++i) {
        const float f = s_f[i][lane];
        const float4 *src = reinterpret_cast<const float4 *>(p.part) + slot(i) * (D / 4) * ROWS + rr;
#pragma unroll
        for (int x = 0; x < W; ++x) {
            const float4 v = f != 0.f ? src[(quad + x) * ROWS] : make_float4(0.f, 0.f, 0.f, 0.f);
            acc[x].x = fmaf(v.x, f, acc[x].x);
            acc[x].y = fmaf(v.y, f, acc[x].y);
            acc[x].z = fmaf(v.z, f, acc[x].z);
            acc[x].w = fmaf(v.w, f, acc[x].w);
        }
    }
    const long row = (long)bh * p.R + r;
    const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;
    uint2 *dst = reinterpret_cast<uint2 *>(p.o + row * D + quad * 4);
#pragma unroll
    for (int x = 0; x < W; ++x) dst[x] = make_uint2(tc::pack_bf16(acc[x].x * inv, acc[x].y * inv), tc::pack_bf16(acc[x].z * inv, acc[x].w * inv));
    if (p.lse && quad == 0) p.lse[row] = (m + log2f(l)) * 0.69314718055994531f;
}

// Blocks per gang for nr row tiles on `sms` SMs: as many as waste the fewest block-passes, the
// largest of equals (more blocks that meet in L2).
int gang_size(int nr, int sms)
{
    int best = 1;
    double top = 0;
    for (int g = 1; g <= std::min(nr, sms); ++g) {
        const int passes = (nr + g - 1) / g;
        const double use = (double)nr / ((double)passes * g) * ((double)(sms / g) * g / sms);
        if (use >= top - 1e-9) {
            top = std::max(top, use);
            best = g;
        }
    }
    return best;
}

}  // namespace

size_t paged_attn_tc_bytes() { return (size_t)device_sms() * 2 * ROWS * (D * 4 + 8); }

cudaError_t launch_paged_attn_tc(const PagedAttnArgs &a, cudaStream_t s)
{
    const long R = a.G * a.L;
    const long q_rows = (long)a.B * a.c.H * R, kv_rows = a.c.num_pages * a.c.H << a.c.page_log2;
    if (R == 0 || a.B == 0) return cudaSuccess;
    const long blocks = (long)a.B * a.c.H * ((R + 31) / 32);            // of the join
    if (q_rows + ROWS >= (1L << 31) || kv_rows + BN >= (1L << 31) || blocks > 0x7fffffffL) return cudaErrorNotSupported;
    const int psz = 1 << a.c.page_log2;
    CUtensorMap mq, mk, mv;
    cudaError_t e;
    if ((e = make_tmap_2d_bf16(&mq, a.q, q_rows, D, 64, BM, true)) != cudaSuccess) return e;
    if ((e = make_tmap_2d_bf16(&mk, a.c.k, kv_rows, D, 64, (uint32_t)psz, true)) != cudaSuccess) return e;
    if ((e = make_tmap_2d_bf16(&mv, a.c.v, kv_rows, D, 64, (uint32_t)psz, true)) != cudaSuccess) return e;
    const int sms = device_sms();
    Params p;
    p.c = a.c;
    p.G = a.G;
    p.R = (int)R;
    p.nr = (int)((R + ROWS - 1) / ROWS);
    const int gs = gang_size(p.nr, sms);
    // two tiles a gang at least (unless the heads have but one each): a block's start and end cost as
    // much as several tiles, and the join grows with the pieces (128 rows over 5000 keys of 2 heads: 32 us with one, 25 to 28 with two)
    // a head's start and end count as four tiles where blocks have several (three chunks of 517 tokens, window
    // 4096, 108 heads of 5 to 37 tiles: 122 us in all with none, 115 with two, 107 with four; heads of many
    // tiles the same)
    p.line = line_of(a, gs, std::min(sms / gs, MAXG), (p.nr + gs - 1) / gs, 2, 1, 4);
    p.sl2 = a.sl2;
    p.o = (__nv_bfloat16 *)a.o;
    p.lse = a.lse;
    p.part = (float *)a.ws;
    p.ml = (float2 *)((char *)a.ws + (size_t)sms * 2 * ROWS * D * 4);
    if ((e = allow_shared((const void *)paged_attn_tc_kernel, SMEM_BYTES, g_shared)) != cudaSuccess) return e;
    paged_attn_tc_kernel<<<p.line.gs * p.line.ngang, THREADS, SMEM_BYTES, s>>>(mq, mk, mv, p), note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const bool split = 2 * blocks <= sms;
    cfg.gridDim = dim3((unsigned)blocks, split ? 4 : 1);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, split ? paged_join_tc_kernel<1> : paged_join_tc_kernel<4>, p)) == cudaSuccess) note_launch();
    return e;
}

}  // namespace hlta
