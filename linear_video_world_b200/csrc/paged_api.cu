// C ABI of the serving operators beside the streaming cache: rotary positions over several axes,
// the paged cache (append, attention, eviction) and the recurrent gated delta rule. Argument
// checks and dispatch; the contract of every entry point is in include/hlta.h.
#include "hlta_internal.cuh"

#include <math.h>

namespace hlta {
namespace {

#define FAIL(...) record_error(HLTA_ERR_INVALID_ARG, __VA_ARGS__)

bool misaligned(const void *p) { return ((uintptr_t)p & 15u) != 0; }
bool misaligned4(const void *p) { return ((uintptr_t)p & 3u) != 0; }

hlta_status check_type(hlta_dtype dt, int d, bool bf16_128)
{
    if (dt != HLTA_BF16 && dt != HLTA_FP32) return FAIL("unknown dtype %d", (int)dt);
    if (d < 1 || d > 128) return FAIL("d must be in [1, 128] (got %d)", d);
    if (bf16_128 && dt == HLTA_BF16 && d != 128)
        return record_error(HLTA_ERR_UNSUPPORTED, "bf16 path supports d = 128 only (got %d)", d);
    return HLTA_OK;
}

// two ranges of bytes that share some (the same range too)
bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// a tensor of n bytes (none: null or empty)
struct Bytes {
    const void *p;
    size_t n;
};
// whether a tensor that is written shares bytes with another one that is written, or with one that is read
template <size_t NO, size_t NI>
bool outputs_overlap(const Bytes (&out)[NO], const Bytes (&in)[NI])
{
    auto hit = [](const Bytes &a, const Bytes &b) { return a.p && b.p && a.n && b.n && overlap(a.p, a.n, b.p, b.n); };
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = i + 1; j < NO; ++j)
            if (hit(out[i], out[j])) return true;
        for (size_t j = 0; j < NI; ++j)
            if (hit(out[i], in[j])) return true;
    }
    return false;
}
size_t bytes_of(hlta_dtype dt) { return dt == HLTA_BF16 ? 2 : 4; }
size_t pool_bytes(long num_pages, int H, int page, int d, hlta_dtype dt) { return (size_t)num_pages * H * page * d * bytes_of(dt); }

hlta_status check_spec(const hlta_rope_axes_t *sp, int d)
{
    long pairs = 0;
    for (int a = 0; a < 3; ++a) {
        if (sp->pairs[a] < 0 || sp->pairs[a] > 64) return FAIL("pairs[%d] must be in [0, 64] (got %d)", a, sp->pairs[a]);
        pairs += sp->pairs[a];
    }
    if (2 * pairs > d) return FAIL("%ld pairs do not fit d = %d", pairs, d);
    if (sp->layout != 0 && sp->layout != 1) return FAIL("layout must be 0 or 1 (got %d)", sp->layout);
    if (sp->shared_freq != 0 && sp->shared_freq != 1) return FAIL("shared_freq must be 0 or 1 (got %d)", sp->shared_freq);
    if (!(sp->base > 1.f) || !(sp->base <= 3.0e38f)) return FAIL("base must be finite and > 1 (got %g)", (double)sp->base);
    if (!sp->pos && (sp->grid_h < 1 || sp->grid_w < 1)) return FAIL("grid must be at least 1 x 1 (got %d x %d)", sp->grid_h, sp->grid_w);
    if (misaligned4(sp->pos) || misaligned4(sp->t0)) return FAIL("positions must be 4-byte aligned");
    return HLTA_OK;
}

hlta_status check_cache(const void *k_pages, const void *v_pages, const int *table, const int *kv_lens, int B, int Hkv,
                        long num_pages, int page, int max_pages)
{
    if (B < 0 || Hkv < 0) return FAIL("bad shape B=%d Hkv=%d", B, Hkv);
    if (page != 16 && page != 32 && page != 64 && page != 128) return FAIL("page must be 16, 32, 64 or 128 (got %d)", page);
    if (num_pages < 1 || max_pages < 1) return FAIL("num_pages and max_pages must be >= 1 (got %ld, %d)", num_pages, max_pages);
    if ((long)max_pages * page > (1L << 30)) return FAIL("max_pages * page must be at most 2^30");
    if (num_pages > 0x7fffffffL) return FAIL("num_pages must fit 31 bits");
    if (B > 0 && (!k_pages || !v_pages || !table || !kv_lens)) return FAIL("null cache pointer");
    if (misaligned(k_pages) || misaligned(v_pages)) return FAIL("tensor pointers must be 16-byte aligned");
    if (misaligned4(table) || misaligned4(kv_lens)) return FAIL("tables must be 4-byte aligned");
    return HLTA_OK;
}

PagedKV cache_of(const void *k, const void *v, const int *table, const int *kv_lens, int H, int d, long num_pages, int page,
                 int max_pages, unsigned int *err)
{
    PagedKV c;
    c.k = const_cast<void *>(k); c.v = const_cast<void *>(v);
    c.table = table; c.kv_lens = kv_lens;
    c.num_pages = num_pages;
    c.H = H; c.d = d; c.max_pages = max_pages;
    c.page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    c.err = err;
    return c;
}

hlta_status done(cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return HLTA_OK;
    if (e == cudaErrorNotSupported) return record_error(HLTA_ERR_UNSUPPORTED, "%s: unsupported shape", what);
    return record_error(HLTA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

#define ERR_WORD(err)                                       \
    unsigned int *err = device_error_word();                \
    if (!err) return HLTA_ERR_CUDA

size_t pad(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

int device_sms()
{
    static std::atomic<int> sms[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 148;
    }
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return 148;
    }
    sms[dev].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t allow_shared(const void *kernel, size_t bytes, std::atomic<unsigned long long> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)) != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
}

}  // namespace hlta

using namespace hlta;

extern "C" {

hlta_status hlta_rope_axes(const void *q, const void *k, void *q_out, void *k_out, int B, int Hq, int Hk, long L, int d,
                           const hlta_rope_axes_t *spec, int inverse, hlta_dtype dt, void *stream)
{
    hlta_status st;
    if (!spec) return FAIL("null spec");
    if (B < 0 || Hq < 0 || Hk < 0 || L < 0 || L > (1L << 30)) return FAIL("bad shape B=%d Hq=%d Hk=%d L=%ld", B, Hq, Hk, L);
    if ((st = check_type(dt, d, false)) != HLTA_OK) return st;
    if ((st = check_spec(spec, d)) != HLTA_OK) return st;
    if ((q && !q_out) || (k && !k_out)) return FAIL("null tensor pointer");
    if (misaligned(q) || misaligned(k) || misaligned(q_out) || misaligned(k_out)) return FAIL("tensor pointers must be 16-byte aligned");
    const size_t el = dt == HLTA_BF16 ? 2 : 4;
    const size_t nq = q ? (size_t)B * Hq * L * d * el : 0, nk = k ? (size_t)B * Hk * L * d * el : 0;
    if ((nq && q != q_out && overlap(q, nq, q_out, nq)) || (nk && k != k_out && overlap(k, nk, k_out, nk)) ||
        (nq && nk && (overlap(q_out, nq, k, nk) || overlap(q_out, nq, k_out, nk) || overlap(q, nq, k_out, nk))))
        return FAIL("an output overlaps another tensor");
    if (outputs_overlap({{q_out, nq}, {k_out, nk}}, {{spec->pos, (size_t)B * L * 12}, {spec->t0, (size_t)B * 4}}))
        return FAIL("an output overlaps the positions");
    if (nq + nk == 0) return HLTA_OK;
    return done(launch_rope_axes(q, k, q_out, k_out, B, Hq, Hk, L, d, spec, inverse != 0, dt == HLTA_BF16, (cudaStream_t)stream),
                "rotary axes");
}

hlta_status hlta_paged_append(const void *k, const void *v, void *k_pages, void *v_pages, const int *table, const int *kv_lens,
                              const int *new_lens, int B, int Hkv, long L, int d, long num_pages, int page, int max_pages,
                              const hlta_rope_axes_t *spec, hlta_dtype dt, void *stream)
{
    hlta_status st;
    if ((!k || !v) && B > 0 && Hkv > 0 && L > 0) return FAIL("null tensor pointer");
    if (L < 0 || L > (1L << 30)) return FAIL("bad shape L=%ld", L);
    if ((st = check_type(dt, d, false)) != HLTA_OK) return st;
    if ((st = check_cache(k_pages, v_pages, table, kv_lens, B, Hkv, num_pages, page, max_pages)) != HLTA_OK) return st;
    if (spec && (st = check_spec(spec, d)) != HLTA_OK) return st;
    if (misaligned(k) || misaligned(v)) return FAIL("tensor pointers must be 16-byte aligned");
    if (misaligned4(new_lens)) return FAIL("tables must be 4-byte aligned");
    if (B == 0 || Hkv == 0 || L == 0) {
        if (B > 0 && k_pages == v_pages) return FAIL("k_pages and v_pages must be different buffers");
        return HLTA_OK;
    }
    const size_t np = pool_bytes(num_pages, Hkv, page, d, dt), nk = (size_t)B * Hkv * L * d * bytes_of(dt), nb = (size_t)B * 4;
    if (outputs_overlap({{k_pages, np}, {v_pages, np}},
                        {{k, nk}, {v, nk}, {table, nb * max_pages}, {kv_lens, nb}, {new_lens, nb},
                         {spec ? spec->pos : nullptr, nb * L * 3}, {spec ? spec->t0 : nullptr, nb}}))
        return FAIL("the pages of the keys or of the values overlap another tensor");
    ERR_WORD(err);
    return done(launch_paged_append(cache_of(k_pages, v_pages, table, kv_lens, Hkv, d, num_pages, page, max_pages, err), k, v,
                                    new_lens, B, L, spec, dt == HLTA_BF16, (cudaStream_t)stream), "paged append");
}

size_t hlta_paged_attn_workspace_bytes(int B, int Hq, int Hkv, long L, int d, int page, int max_pages, int weights, hlta_dtype dt)
{
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || L < 0 || L > (1L << 29) || d < 1 || d > 128 || max_pages < 1 || page < 1 ||
        (long)max_pages * page > (1L << 30) || (dt != HLTA_BF16 && dt != HLTA_FP32))
        return 0;
    if (paged_token_fits(B, Hkv, Hq / Hkv, L, max_pages * page, weights != 0))
        return pad(paged_token_bytes(B, Hkv, Hq / Hkv, L, max_pages * page, weights != 0)) + 256;
    const size_t lse = weights ? pad((size_t)B * Hq * L * 4) : 0;
    return lse + pad(dt == HLTA_BF16 ? paged_attn_tc_bytes() : paged_attn_simt_bytes(B, Hq, Hkv, L, max_pages * page)) + 256;
}

hlta_status hlta_paged_attn_fwd(const void *q, const void *k_pages, const void *v_pages, const int *table, const int *kv_lens,
                                const int *new_lens, void *o, float *lse, const float *w_in, float *w_out, float decay, int B,
                                int Hq, int Hkv, long L, int d, long num_pages, int page, int max_pages, int N, int w,
                                float scale, void *workspace, size_t ws_bytes, hlta_dtype dt, void *stream)
{
    hlta_status st;
    if ((!q || !o) && B > 0 && L > 0) return FAIL("null tensor pointer");
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || L < 0 || L > (1L << 29))
        return FAIL("bad shape B=%d Hq=%d Hkv=%d L=%ld (Hq must be a multiple of Hkv)", B, Hq, Hkv, L);
    if ((st = check_type(dt, d, true)) != HLTA_OK) return st;
    if ((st = check_cache(k_pages, v_pages, table, kv_lens, B, Hkv, num_pages, page, max_pages)) != HLTA_OK) return st;
    if (N < 1 || w < 0) return FAIL("N must be >= 1 and w >= 0 (got %d, %d)", N, w);
    if (Hq / Hkv > 128) return record_error(HLTA_ERR_UNSUPPORTED, "at most 128 query heads a key head (got %d)", Hq / Hkv);
    if (misaligned(q) || misaligned(o)) return FAIL("tensor pointers must be 16-byte aligned");
    if (misaligned4(new_lens) || misaligned4(lse) || misaligned4(w_in) || misaligned4(w_out))
        return FAIL("lengths, lse and weights must be 4-byte aligned");
    if (w_in && !w_out) return FAIL("w_in without w_out");
    if (!isfinite(scale)) return FAIL("scale must be finite (got %g)", (double)scale);
    if (w_out && !isfinite(decay)) return FAIL("decay must be finite (got %g)", (double)decay);
    const size_t need = hlta_paged_attn_workspace_bytes(B, Hq, Hkv, L, d, page, max_pages, w_out != nullptr, dt);
    if (!workspace || ws_bytes < need) return FAIL("workspace too small: need %zu bytes, got %zu", need, workspace ? ws_bytes : 0);
    if ((uintptr_t)workspace & 255u) return FAIL("workspace must be 256-byte aligned");
    const size_t nw = (size_t)B * Hkv * max_pages * page * 4, nl = (size_t)B * Hq * L * 4, nq = nl / 4 * d * bytes_of(dt), nb = (size_t)B * 4,
                 np = pool_bytes(num_pages, Hkv, page, d, dt);
    if (outputs_overlap({{o, nq}, {lse, nl}, {w_out, nw}, {workspace, B > 0 ? need : 0}},
                        {{q, nq}, {k_pages, np}, {v_pages, np}, {table, nb * max_pages}, {kv_lens, nb}, {new_lens, nb}, {w_in == w_out ? nullptr : w_in, nw}}))
        return FAIL("an output or the workspace overlaps another tensor");
    if (B == 0 || (L == 0 && !w_out)) return HLTA_OK;
    // what one of the call's kernels could not be launched for is refused before the first is
    const bool few = paged_token_fits(B, Hkv, Hq / Hkv, L, max_pages * page, w_out != nullptr);
    const long R = (Hq / Hkv) * L, heads = (long)B * Hkv;
    if (heads > 65535) return record_error(HLTA_ERR_UNSUPPORTED, "at most 65535 key heads of rollouts (got %d x %d)", B, Hkv);
    if (dt == HLTA_BF16 ? heads * R + 256 >= (1L << 31) || num_pages * Hkv * page + 128 >= (1L << 31)
                        : R > (1L << 30) || (heads * R + 3) / 4 > 0x7fffffffL)
        return record_error(HLTA_ERR_UNSUPPORTED, "too many rows of queries (%ld) or of the pool (%ld)", heads * R, num_pages * Hkv * page);
    if (w_out && !few && dt == HLTA_BF16 && !paged_weights_fit(R, max_pages * page))
        return record_error(HLTA_ERR_UNSUPPORTED, "weights of %ld rows over a capacity of %d", R, max_pages * page);
    ERR_WORD(err);
    PagedAttnArgs a;
    a.c = cache_of(k_pages, v_pages, table, kv_lens, Hkv, d, num_pages, page, max_pages, err);
    a.q = q; a.o = o;
    char *ws = (char *)workspace;
    a.lse = lse;
    a.w_in = w_in; a.w_out = w_out; a.decay = decay;
    a.new_lens = new_lens;
    a.B = B; a.G = Hq / Hkv; a.L = L;
    a.N = N; a.w = w;
    a.sl2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)d)) * 1.4426950408889634f;
    a.ws = ws;
    if (few)
        return done(launch_paged_token(a, dt == HLTA_BF16, (cudaStream_t)stream), "paged attention");
    if (w_out) {
        // the weights are taken in a second pass, from the log-sum-exp
        if (!lse) a.lse = (float *)ws;
        a.ws = ws + pad((size_t)B * Hq * L * 4);
    }
    cudaError_t e = dt == HLTA_BF16 ? launch_paged_attn_tc(a, (cudaStream_t)stream) : launch_paged_attn_simt(a, (cudaStream_t)stream);
    if (e == cudaSuccess && w_out)
        e = dt == HLTA_BF16 ? launch_paged_weights_tc(a, (cudaStream_t)stream) : launch_paged_weights_simt(a, (cudaStream_t)stream);
    return done(e, "paged attention");
}

size_t hlta_paged_evict_workspace_bytes(int B, int Hkv, int budget)
{
    return B < 0 || Hkv < 0 || budget < 1 ? 0 : pad(paged_evict_bytes(B, Hkv, budget)) + 256;
}

hlta_status hlta_paged_evict(const float *weights, const void *k_pages, const void *v_pages, const int *table, const int *kv_lens,
                             int B, int Hkv, int d, long num_pages, int page, int max_pages, int budget, int sink, int recent,
                             void *k_dst, void *v_dst, const int *dst_table, long num_dst, int max_dst, int *new_lens, int *kept,
                             float *w_out, void *workspace, size_t ws_bytes, hlta_dtype dt, void *stream)
{
    hlta_status st;
    if ((!weights || !new_lens) && B > 0) return FAIL("null tensor pointer");
    if ((st = check_type(dt, d, false)) != HLTA_OK) return st;
    if ((st = check_cache(k_pages, v_pages, table, kv_lens, B, Hkv, num_pages, page, max_pages)) != HLTA_OK) return st;
    if ((st = check_cache(k_dst, v_dst, dst_table, kv_lens, B, Hkv, num_dst, page, max_dst)) != HLTA_OK) return st;
    if (B > 0 && k_dst == v_dst) return FAIL("k_dst and v_dst must be different buffers");
    if (budget < 1 || sink < 0 || recent < 0 || (long)sink + recent > budget)
        return FAIL("budget >= 1, sink, recent >= 0, sink + recent <= budget (got %d, %d, %d)", budget, sink, recent);
    if (budget > (long)max_dst * page) return FAIL("budget %d does not fit %d pages of %d", budget, max_dst, page);
    if (misaligned4(weights) || misaligned4(new_lens) || misaligned4(kept) || misaligned4(w_out))
        return FAIL("weights, lengths and positions must be 4-byte aligned");
    const size_t need = hlta_paged_evict_workspace_bytes(B, Hkv, budget);
    if (!kept && (!workspace || ws_bytes < need)) return FAIL("workspace too small: need %zu bytes, got %zu", need, workspace ? ws_bytes : 0);
    if ((uintptr_t)workspace & 255u) return FAIL("workspace must be 256-byte aligned");
    const size_t bh = (size_t)B * Hkv, nw = bh * max_pages * page * 4, no = bh * max_dst * page * 4, nb = (size_t)B * 4;
    const size_t np = pool_bytes(num_pages, Hkv, page, d, dt), nd = pool_bytes(num_dst, Hkv, page, d, dt);
    const Bytes w = {weights, nw}, t = {table, nb * max_pages}, td = {dst_table, nb * max_dst}, kl = {kv_lens, nb};
    // (the destination may lie in the pool that is read, in other pages)
    if (B > 0 && (outputs_overlap({{k_dst, nd}, {v_dst, nd}}, {w, t, td, kl}) ||
                  outputs_overlap({{new_lens, nb}, {kept, bh * budget * 4}, {w_out, no}, {kept ? nullptr : workspace, need}},
                                  {w, t, td, kl, {k_pages, np}, {v_pages, np}, {k_dst, nd}, {v_dst, nd}})))
        return FAIL("an output or the workspace overlaps another tensor");
    if (B == 0 || Hkv == 0) return HLTA_OK;
    ERR_WORD(err);
    PagedEvictArgs a;
    a.c = cache_of(k_pages, v_pages, table, kv_lens, Hkv, d, num_pages, page, max_pages, err);
    a.weights = weights;
    a.B = B; a.budget = budget; a.sink = sink; a.recent = recent;
    a.k_dst = k_dst; a.v_dst = v_dst; a.dst_table = dst_table; a.num_dst = num_dst; a.max_dst = max_dst;
    a.new_lens = new_lens; a.kept = kept; a.w_out = w_out;
    a.ws = workspace;
    return done(launch_paged_evict(a, dt == HLTA_BF16, (cudaStream_t)stream), "paged eviction");
}

static hlta_status gdn_step(const void *q, const void *k, const void *v, const float *a, const float *b, int raw, float c, void *o,
                            const float *S, float *S_out, const int *slots, const int *lens, int B, int H, long L, int d,
                            long num_slots, hlta_dtype dt, void *stream)
{
    hlta_status st;
    if (B > 0 && H > 0 && (!S || !S_out || (L > 0 && (!q || !k || !v || !a || !b || !o)))) return FAIL("null tensor pointer");
    if (B < 0 || H < 0 || L < 0 || L > (1L << 30) || num_slots < 1 || num_slots > 0x7fffffffL)
        return FAIL("bad shape B=%d H=%d L=%ld num_slots=%ld", B, H, L, num_slots);
    if ((st = check_type(dt, d, true)) != HLTA_OK) return st;
    if (raw && (!(c >= 0.f) || !(c <= 1e30f))) return FAIL("decay constant c must be finite and >= 0 (got %g)", (double)c);
    if (!slots && B > num_slots) return FAIL("%d rollouts do not fit %ld slots", B, num_slots);
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(o) || misaligned(S) || misaligned(S_out))
        return FAIL("tensor pointers must be 16-byte aligned");
    if (misaligned4(a) || misaligned4(b) || misaligned4(slots) || misaligned4(lens)) return FAIL("gates and tables must be 4-byte aligned");
    // (blocks of different state rows read the whole of q and k; a block reads and writes its own rows of S)
    const size_t ns = (size_t)num_slots * H * d * d * 4, ng = (size_t)B * H * L * 4, no = ng / 4 * d * bytes_of(dt), nb = (size_t)B * 4;
    if (outputs_overlap({{o, no}, {S_out, ns}}, {{q, no}, {k, no}, {v, no}, {a, ng}, {b, ng}, {slots, nb}, {lens, nb}, {S == S_out ? nullptr : S, ns}}))
        return FAIL("an output overlaps another tensor");
    if (B == 0 || H == 0) return HLTA_OK;
    ERR_WORD(err);
    GdnStepArgs g;
    g.q = q; g.k = k; g.v = v; g.a = a; g.b = b;
    g.raw = raw; g.raw_c = c;
    g.o = o; g.S = S; g.S_out = S_out; g.slots = slots; g.lens = lens;
    g.B = B; g.H = H; g.d = d; g.L = L; g.num_slots = num_slots;
    g.err = err;
    return done(launch_gdn_step(g, dt == HLTA_BF16, (cudaStream_t)stream), "gated delta step");
}

hlta_status hlta_gdn_step(const void *q, const void *k, const void *v, const float *a, const float *b, void *o, const float *S,
                          float *S_out, const int *slots, const int *lens, int B, int H, long L, int d, long num_slots,
                          hlta_dtype dt, void *stream)
{
    return gdn_step(q, k, v, a, b, 0, 0.f, o, S, S_out, slots, lens, B, H, L, d, num_slots, dt, stream);
}

hlta_status hlta_gdn_step_raw(const void *q, const void *k, const void *v, const float *x, const float *y, float c, void *o,
                              const float *S, float *S_out, const int *slots, const int *lens, int B, int H, long L, int d,
                              long num_slots, hlta_dtype dt, void *stream)
{
    return gdn_step(q, k, v, x, y, 1, c, o, S, S_out, slots, lens, B, H, L, d, num_slots, dt, stream);
}

}  // extern "C"
