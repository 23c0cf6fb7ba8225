// q8_api.cu -- host side of the calls over 8-bit pages: checks, scratch and the
// choice of kernel.
#include <algorithm>
#include <cmath>

#include "q8.cuh"

namespace skv {
namespace q8 {

// Makes the handle's device current for a call.
struct OnDevice {
    int prev = -1;
    bool moved = false;
    explicit OnDevice(int want)
    {
        if (cudaGetDevice(&prev) == cudaSuccess && prev != want) moved = cudaSetDevice(want) == cudaSuccess;
    }
    ~OnDevice()
    {
        if (moved) cudaSetDevice(prev);
    }
};

// Query rows of a KV head from which the tensor-core kernel serves: it computes 256
// rows whatever is there, the decode kernel passes over the keys again for each 16.
// Eight KV heads of D = 128, decode against tensor cores: 32768 keys of one sequence
// 39.9 / 44.2 us at 32 rows and 49.8 / 44.0 at 36 with fp16 results (fp32: 44.4 / 60.5,
// 57.3 / 60.3, and 74.5 / 60.4 at 64); 8000 keys of eight sequences 66.5 / 65.5 us at 32 rows
// and 91.5 / 65.7 at 36 (fp32: 75 / 109, 104 / 108 and 132 / 108 at 64).  So the border is
// fp16's; fp32 results of 33 to 48 rows lose 2 to 5 % by it.  Over short contexts it costs
// both types a few us up to 128 rows (2000 keys of one sequence: 16.2 / 20.6 us at 36 rows and
// 20.8 / 21.0 at 128, fp32 16.7 / 22.6 and 22.1 / 22.9): lengths are not known to the host.
constexpr int kTcRows = 33;
// Scratch for the pages' log sums or the selection's keys of one launch (one token's
// at least).
constexpr int64_t kPageScratch = int64_t(256) << 20;
// Pages that the units of a decode launch pass by: positions on their line, and those with
// the units rounded up to whole pieces (a CTA's fraction of a page and 8 pages more for each
// CTA), are counted in 32 bits.
constexpr int64_t kMaxVisits = 0xffff0000ll;
// Entries of a selection: the kernels index them, and the log sums of their halves,
// in 32 bits.
constexpr int32_t kMaxSel = 1 << 30;

static bool misaligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

static int check_pool(skv_handle *h, const skv_q8_pool *p)
{
    if (!p) return fail(h, SKV_EINVAL, "pool is NULL");
    if (p->D != 64 && p->D != 128) return fail(h, SKV_EUNSUPPORTED, "head dim %d (supported: 64, 128)", p->D);
    if (p->n_pages < 1 || p->n_pages > INT32_MAX) return fail(h, SKV_EINVAL, "pool of %lld pages", (long long)p->n_pages);
    if (!p->k || !p->v || !p->k_scale || !p->v_scale || !p->k_min || !p->k_max)
        return fail(h, SKV_EINVAL, "a pool pointer is NULL");
    if (misaligned(p->k, 16) || misaligned(p->v, 16) || misaligned(p->k_min, 16) || misaligned(p->k_max, 16) ||
        misaligned(p->k_scale, 4) || misaligned(p->v_scale, 4))
        return fail(h, SKV_EUNSUPPORTED, "pool codes must be 16-byte and scales 4-byte aligned");
    return SKV_OK;
}

static int check_lists(skv_handle *h, int32_t S, int32_t Hk, const int32_t *ids, int64_t cap, const int32_t *kv_len)
{
    if (S < 1 || Hk < 1) return fail(h, SKV_EINVAL, "bad sizes S=%d Hk=%d", S, Hk);
    if (S > 65535 || Hk > 65535) return fail(h, SKV_EUNSUPPORTED, "S and Hk are limited to 65535");
    // lengths and list indices are int32
    if (cap < 1 || cap > INT32_MAX / kPage) return fail(h, SKV_EINVAL, "pages_per_list = %lld", (long long)cap);
    if (!ids || !kv_len) return fail(h, SKV_EINVAL, "page_ids or kv_len is NULL");
    return SKV_OK;
}

static int check_query(skv_handle *h, const skv_q8_pool *pool, const skv_shape *sh, const void *q)
{
    if (!sh) return fail(h, SKV_EINVAL, "shape is NULL");
    if (sh->nq < 1 || sh->H < 1 || sh->Hk < 1 || sh->S < 1 || sh->H % sh->Hk)
        return fail(h, SKV_EINVAL, "bad shape S=%d nq=%d H=%d Hk=%d", sh->S, sh->nq, sh->H, sh->Hk);
    if (sh->D != pool->D) return fail(h, SKV_EINVAL, "head dim %d over pages of head dim %d", sh->D, pool->D);
    if (!std::isfinite(sh->scale)) return fail(h, SKV_EINVAL, "scale is not finite");
    if (!q) return fail(h, SKV_EINVAL, "q is NULL");
    if (misaligned(q, 16)) return fail(h, SKV_EUNSUPPORTED, "q must be 16-byte aligned");
    if (static_cast<int64_t>(sh->S) * sh->nq > INT32_MAX || static_cast<int64_t>(sh->nq) * (sh->H / sh->Hk) > INT32_MAX)
        return fail(h, SKV_EUNSUPPORTED, "S*nq or nq*H/Hk exceeds 2^31 - 1");
    return SKV_OK;
}

static Lists lists_of(skv_handle *h, int64_t n_pages, int32_t S, int32_t Hk, const int32_t *ids, int64_t cap,
                      const int32_t *kv_len)
{
    return Lists{ids, kv_len, cap, n_pages, S, Hk, h->status};
}

// How a call is served: which kernel, rows of its units (the tensor-core kernel takes 256
// at a time, the decode kernel 8 or 16), and the tokens of one launch: as many as the
// kernels' counters have units for, as keep their lines of pages or key tiles within
// 32 bits, and as keep the pages' log sums within kPageScratch (but one at least).
struct AttnSplit {
    bool tc;
    int nc;
    int64_t unit_rows;
    int64_t tokens;                // 0: not even one
};

static AttnSplit attn_split(const skv_shape &sh, int64_t cap, int32_t n_sel, bool mass)
{
    const bool sel = n_sel > 0;
    const int64_t heads = static_cast<int64_t>(sh.S) * sh.Hk, G = sh.H / sh.Hk;
    constexpr int64_t max_units = kMaxUnits - 1;          // (a grid's y)
    AttnSplit x;
    x.tc = !sel && sh.nq * G >= kTcRows;
    x.nc = (sel ? G : sh.nq * G) <= 8 ? 1 : 2;
    x.unit_rows = x.tc ? 256 : 8 * x.nc;
    const int64_t groups = (G + x.unit_rows - 1) / x.unit_rows;   // units of a token's rows
    x.tokens = std::min<int64_t>(sh.nq, sel ? max_units / (heads * groups) : (max_units / heads) * x.unit_rows / G);
    if (x.tokens < 1) return x;
    // (a token's units fit a launch: heads * G is below 2^24 from here on)
    if (sel) {
        x.tokens = std::min(x.tokens, kMaxVisits / (heads * groups * n_sel));
    } else {
        const int64_t line = x.tc ? (int64_t(1) << 31) / (heads * ((cap + 1) / 2)) : kMaxVisits / (heads * cap);
        x.tokens = std::min(x.tokens, std::min<int64_t>(INT32_MAX, line) * x.unit_rows / G);
    }
    if (x.tokens >= 1 && mass)
        x.tokens = std::min(x.tokens, std::max<int64_t>(1, kPageScratch / (heads * G * (sel ? n_sel : cap) * 8)));
    return x;
}

static size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace q8
}  // namespace skv

using namespace skv;
using namespace skv::q8;

extern "C" {

int skv_q8_append(skv_handle *h, const skv_q8_pool *pool, int32_t S, int32_t Hk, int32_t n_max, int32_t x_type,
                  const void *k_new, const void *v_new, const int32_t *page_ids, int64_t pages_per_list,
                  const int32_t *kv_len, const int32_t *n_new, void *stream)
{
    if (!h) return SKV_EINVAL;
    h->err[0] = 0;
    int rc = check_pool(h, pool);
    if (rc || (rc = check_lists(h, S, Hk, page_ids, pages_per_list, kv_len))) return rc;
    if (n_max < 0) return fail(h, SKV_EINVAL, "n_max = %d", n_max);
    if (x_type != SKV_F32 && x_type != SKV_F16) return fail(h, SKV_EINVAL, "rows to append are SKV_F32 or SKV_F16");
    if (n_max == 0) return SKV_OK;
    if (!k_new || !v_new) return fail(h, SKV_EINVAL, "k_new or v_new is NULL");
    if (misaligned(k_new, 16) || misaligned(v_new, 16))
        return fail(h, SKV_EUNSUPPORTED, "k_new and v_new must be 16-byte aligned");
    OnDevice on(h->device);
    return launch_append(h, *pool, lists_of(h, pool->n_pages, S, Hk, page_ids, pages_per_list, kv_len), n_max, x_type,
                         k_new, v_new, n_new, static_cast<cudaStream_t>(stream));
}

int skv_q8_attn(skv_handle *h, const skv_q8_pool *pool, const skv_shape *shape, const void *q,
                const int32_t *page_ids, int64_t pages_per_list, const int32_t *kv_len, const int32_t *q_pos,
                const int32_t *sel, int32_t n_sel, float *mass, int32_t o_type, void *o, float *lse, void *stream)
{
    if (!h) return SKV_EINVAL;
    h->err[0] = 0;
    int rc = check_pool(h, pool);
    if (rc || (rc = check_query(h, pool, shape, q)) ||
        (rc = check_lists(h, shape->S, shape->Hk, page_ids, pages_per_list, kv_len)))
        return rc;
    if (sel && n_sel < 1) return fail(h, SKV_EINVAL, "n_sel = %d", n_sel);
    if (sel && n_sel >= kMaxSel) return fail(h, SKV_EUNSUPPORTED, "n_sel = %d (below 2^30 is supported)", n_sel);
    if (o_type != SKV_F32 && o_type != SKV_F16) return fail(h, SKV_EINVAL, "o_type is SKV_F32 or SKV_F16");
    if (!o || !lse) return fail(h, SKV_EINVAL, "o or lse is NULL");
    if (misaligned(o, 16) || misaligned(lse, 4)) return fail(h, SKV_EUNSUPPORTED, "o must be 16-byte aligned");
    OnDevice on(h->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int D = shape->D;
    AttnArgs a = {};
    a.L = lists_of(h, pool->n_pages, shape->S, shape->Hk, page_ids, pages_per_list, kv_len);
    a.k = pool->k;
    a.v = pool->v;
    a.k_scale = pool->k_scale;
    a.v_scale = pool->v_scale;
    a.q = static_cast<const __half *>(q);
    a.q_pos = q_pos;
    a.sel = sel;
    a.n_sel = sel ? n_sel : 0;
    a.nq_ld = shape->nq;
    a.H = shape->H;
    a.G = shape->H / shape->Hk;
    a.scale_log2 = shape->scale * 1.4426950408889634f;
    a.o = o;
    a.lse = lse;
    a.counters = h->counters;
    const bool f16 = o_type == SKV_F16;
    const int64_t heads = static_cast<int64_t>(shape->S) * shape->Hk;
    const int64_t per_list = sel ? n_sel : pages_per_list;
    const AttnSplit split = attn_split(*shape, pages_per_list, a.n_sel, mass != nullptr);
    const bool tc = split.tc;
    const int nc = split.nc;
    const int64_t unit_rows = split.unit_rows, nq_max = split.tokens;
    if (nq_max < 1)
        return fail(h, SKV_EUNSUPPORTED, "S*Hk = %lld lists of %lld pages with %d query heads each are too many for one launch",
                    (long long)heads, (long long)per_list, a.G);
    a.nq = static_cast<int>(nq_max);
    a.rows = sel ? a.G : a.nq * a.G;
    a.row_groups = static_cast<int>((a.rows + unit_rows - 1) / unit_rows);
    const int64_t units = (sel ? heads * a.nq : heads) * a.row_groups;
    // one CTA a SM, but no more than pieces of kPieceMin pages
    const int64_t pieces = tc ? (units * per_list + 1) / 2 : (units * per_list + kPieceMin - 1) / kPieceMin;
    const int grid = static_cast<int>(std::min<int64_t>(h->sm_count, pieces));
    // two partials for each CTA's piece
    const size_t po = round256(static_cast<size_t>(2) * grid * unit_rows * D * sizeof(float));
    const size_t pm = round256(static_cast<size_t>(2) * grid * unit_rows * 2 * sizeof(float));
    const size_t pp = tc ? round256((static_cast<size_t>(shape->S) * a.row_groups + 2) * sizeof(uint32_t)) : 0;
    const size_t pl = mass ? static_cast<size_t>(heads) * a.nq * a.G * per_list * (tc ? 4 : 8) : 0;
    if ((rc = ensure_workspace(h, po + pm + pp + pl, st))) return rc;
    uint8_t *ws = static_cast<uint8_t *>(h->workspace);
    a.part_o = reinterpret_cast<float *>(ws);
    a.part_ml = reinterpret_cast<float *>(ws + po);
    a.page_ld = 2 * per_list;
    a.page_lse = mass ? reinterpret_cast<float *>(ws + po + pm + pp) : nullptr;
    for (int t = 0; t < shape->nq; t += static_cast<int>(nq_max)) {
        a.tok0 = t;
        a.nq = static_cast<int>(std::min<int64_t>(nq_max, shape->nq - t));
        if (!sel) a.rows = a.nq * a.G;
        a.row_groups = static_cast<int>((a.rows + unit_rows - 1) / unit_rows);
        if (tc) {
            rc = launch_prefill(h, a, D, f16, reinterpret_cast<uint32_t *>(ws + po + pm), a.row_groups, mass, grid, st);
        } else {
            rc = launch_decode(h, a, pool->n_pages, D, f16, grid, nc, st);
            if (!rc && mass) rc = launch_mass(h, a, mass, st);
        }
        if (rc) return rc;
    }
    return SKV_OK;
}

int skv_plan_q8_tokens(const skv_shape *shape, int64_t pages_per_list, int32_t n_sel, int32_t mass, int32_t *tokens)
{
    if (!shape || !tokens || shape->S < 1 || shape->S > 65535 || shape->nq < 1 || shape->Hk < 1 || shape->Hk > 65535 ||
        shape->H < shape->Hk || shape->H % shape->Hk || pages_per_list < 1 || pages_per_list > INT32_MAX / kPage || n_sel < 0 ||
        n_sel >= kMaxSel || static_cast<int64_t>(shape->nq) * (shape->H / shape->Hk) > INT32_MAX)
        return SKV_EINVAL;
    const int64_t n = attn_split(*shape, pages_per_list, n_sel, mass != 0).tokens;
    if (n < 1) return SKV_EUNSUPPORTED;
    *tokens = static_cast<int32_t>(n);
    return SKV_OK;
}

int skv_q8_select(skv_handle *h, const skv_q8_pool *pool, const skv_shape *shape, const void *q,
                  const int32_t *page_ids, int64_t pages_per_list, const int32_t *kv_len, const int32_t *q_pos,
                  int32_t n_sel, int32_t n_first, int32_t n_last, int32_t *sel, void *stream)
{
    if (!h) return SKV_EINVAL;
    h->err[0] = 0;
    int rc = check_pool(h, pool);
    if (rc || (rc = check_query(h, pool, shape, q)) ||
        (rc = check_lists(h, shape->S, shape->Hk, page_ids, pages_per_list, kv_len)))
        return rc;
    if (n_sel < 1 || n_first < 0 || n_last < 0 || static_cast<int64_t>(n_first) + n_last > n_sel)
        return fail(h, SKV_EINVAL, "n_sel = %d with n_first = %d, n_last = %d", n_sel, n_first, n_last);
    if (n_sel >= kMaxSel) return fail(h, SKV_EUNSUPPORTED, "n_sel = %d (below 2^30 is supported)", n_sel);
    if (!sel) return fail(h, SKV_EINVAL, "sel is NULL");
    const int64_t rows = static_cast<int64_t>(shape->S) * shape->nq * shape->Hk;
    if (rows > INT32_MAX) return fail(h, SKV_EUNSUPPORTED, "S*nq*Hk exceeds 2^31 - 1");
    OnDevice on(h->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    SelectArgs a = {};
    a.L = lists_of(h, pool->n_pages, shape->S, shape->Hk, page_ids, pages_per_list, kv_len);
    a.k_min = pool->k_min;
    a.k_max = pool->k_max;
    a.k_scale = pool->k_scale;
    a.q = static_cast<const __half *>(q);
    a.q_pos = q_pos;
    a.nq_ld = shape->nq;
    a.H = shape->H;
    a.G = shape->H / shape->Hk;
    a.n_sel = n_sel;
    a.n_first = n_first;
    a.n_last = n_last;
    a.sel = sel;
    const int64_t per_token = static_cast<int64_t>(shape->S) * shape->Hk * pages_per_list * sizeof(uint32_t);
    const int nq_max = static_cast<int>(std::min<int64_t>(shape->nq, std::max<int64_t>(1, kPageScratch / per_token)));
    if ((rc = ensure_workspace(h, static_cast<size_t>(per_token) * nq_max, st))) return rc;
    a.keys = static_cast<uint32_t *>(h->workspace);
    a.counters = h->counters;
    for (int t = 0; t < shape->nq; t += nq_max) {
        a.tok0 = t;
        a.nq = std::min(nq_max, shape->nq - t);
        if ((rc = launch_select(h, a, shape->D, st))) return rc;
    }
    return SKV_OK;
}

int skv_q8_evict(skv_handle *h, int32_t S, int32_t Hk, int64_t pages_per_list, const int32_t *page_ids,
                 const float *mass, const int32_t *kv_len, int32_t n_keep, int32_t n_first, int32_t n_last,
                 int32_t *page_ids_out, float *mass_out, int32_t *kv_len_out, int32_t *freed_out, void *stream)
{
    if (!h) return SKV_EINVAL;
    h->err[0] = 0;
    int rc = check_lists(h, S, Hk, page_ids, pages_per_list, kv_len);
    if (rc) return rc;
    if (n_keep < 1 || n_first < 0 || n_last < 1 || static_cast<int64_t>(n_first) + n_last > n_keep)
        return fail(h, SKV_EINVAL, "n_keep = %d with n_first = %d, n_last = %d (at least 1)", n_keep, n_first, n_last);
    if (!mass || !page_ids_out || !mass_out || !kv_len_out || !freed_out) return fail(h, SKV_EINVAL, "NULL pointer");
    struct Span {
        uintptr_t at, bytes;
    };
    const uintptr_t lists = static_cast<uintptr_t>(S) * Hk * pages_per_list * 4, lens = static_cast<uintptr_t>(S) * 4;
    const Span spans[7] = {{reinterpret_cast<uintptr_t>(page_ids_out), lists}, {reinterpret_cast<uintptr_t>(mass_out), lists},
                           {reinterpret_cast<uintptr_t>(freed_out), lists},    {reinterpret_cast<uintptr_t>(kv_len_out), lens},
                           {reinterpret_cast<uintptr_t>(page_ids), lists},     {reinterpret_cast<uintptr_t>(mass), lists},
                           {reinterpret_cast<uintptr_t>(kv_len), lens}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 7; ++j)
            if (spans[i].at < spans[j].at + spans[j].bytes && spans[j].at < spans[i].at + spans[i].bytes)
                return fail(h, SKV_EINVAL, "an output overlaps an input or another output");
    OnDevice on(h->device);
    return launch_evict(h, lists_of(h, INT32_MAX, S, Hk, page_ids, pages_per_list, kv_len), mass, n_keep, n_first,
                        n_last, page_ids_out, mass_out, kv_len_out, freed_out, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
