// bwd_api.cu -- host side of skv_attn_backward: checks, geometry, scratch, launches.
#include <string.h>

#include <algorithm>
#include <cmath>

#include "bwd.cuh"

namespace skv {
namespace bwd {

static bool misaligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }
static size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Costs in tiles of 128 x 128 of dq (1.1 us): a tile of dk and dv, a CTA's fixed part (tensor memory,
// barriers, row statistics, pipeline fill, result), the launch that adds up pieces.  Measured with D = 128 and used for
// D = 64 too, whose products are half as long but whose CTAs take nearly as much time (996 and 1230 us for 16384 causal
// tokens, 8 heads on 2): pieces were not timed there.
constexpr double kKvTile = 1.5, kFixed = 6, kJoin = 2.5;
// Tiles of an SM up to which p and ds, or dq's ds alone, come in two fp16 parts.
constexpr double kTwoTiles = 2, kTwoDqTiles = 8;
// fp32 bytes that the adding up moves in a tile's time.
constexpr double kJoinBytes = 9e6;

// The CTAs of one launch: those of the kind whose CTAs take longer go out first, the others fill the
// SMs.  So the launch ends when the longest CTA does, or when all SMs' work is done and about half a CTA of
// the second kind later; a unit's tiles are cut into pieces (their sums added up by a further launch)
// where that ends sooner.  Positions are taken to be those of a causal mask whose last token sees
// all keys (what they hold is known on the device only): the share of tiles seen.
//   16384 tokens, causal, 8 heads on 2: no pieces 1233 us, dk and dv in two 1273; on one KV head (128 CTAs
//   of up to 1024 tiles) none 1642, two 1265; 8192 tokens on 2 none 428, two 369.
//   512 tokens over 32768 keys: dq's 128 CTAs of 256 tiles first, dk and dv's 2048 of 16 after them 749 us,
//   the other way round 769.  128 tokens over 4096 keys: none 57, dq in two 63.
// Of 32 shapes (1 to 16384 tokens) the plan took the best pieces or came within 6 % of them, but for 16384 tokens
// that all see 16384 keys, 8 heads on 2: none 2850 to 2913, dk and dv in six 2548.  There dq's CTAs, beside a second
// wave of dk's and dv's long ones, slow these down by half; why was not found.
struct Plan {
    int kv_pieces, q_pieces;
    bool q_first;
};
static Plan plan_of(const Geo &g, int64_t units, int sms, bool kv, bool q, double share)
{
    static const int steps[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128};
    const double kv_bytes = 8.0 * units * g.KT * kTile * g.D, q_bytes = 4.0 * units * g.QT * kTile * g.D;
    Plan best{1, 1, false};
    double least = -1;
    for (int pk : steps) {
        if (pk > 1 && (!kv || pk > g.QT)) break;
        for (int pq : steps) {
            if (pq > 1 && (!q || pq > g.KT)) break;
            const double kv_one = kv ? kKvTile * ((g.QT + pk - 1) / pk) + kFixed : 0, q_one = q ? (g.KT + pq - 1) / pq + kFixed : 0;
            const double kv_all = kv ? units * g.KT * (kKvTile * share * g.QT + kFixed * pk) : 0;
            const double q_all = q ? units * g.QT * (share * g.KT + kFixed * pq) : 0;
            const double last = !kv ? q_one : !q ? kv_one : std::min(kv_one, q_one);
            double cost = std::max(std::max(kv_one, q_one), (kv_all + q_all) / sms + 0.5 * last);
            if (pk > 1) cost += kJoin + kv_bytes * (pk + 0.5) / kJoinBytes;
            if (pq > 1) cost += kJoin + q_bytes * (pq + 0.5) / kJoinBytes;
            if (least < 0 || cost < least - 1e-9) {
                least = cost;
                best = Plan{pk, pq, q_one > kv_one};
            }
        }
    }
    return best;
}

// p and ds as one fp16 number leave results an error like that of their own rounding to fp16: 3.0e-4 in the 2-norm where
// that is 2.1e-4.  Over few rows or keys single roundings show: over 3.1e-4 in 3 % of 2086 shapes of up to 2e11 pairs x channels,
// 4.1e-4 at most.  Two parts leave 2.1e-4.  Where an SM has few tiles, the CTAs' fixed parts hide what they cost:
//   all in two: 26.6 us both ways (64 rows over 256 keys), 30.7 -> 34.8 (0.6 tiles an SM), 45 -> 47 (1.7); beyond, 50 -> 55 (3.4),
//   67.6 -> 73.7 (6.7).  dq's ds in two: 49.2 -> 47.5 (2.5), 67.6 -> 64.5 (6.7), beyond 88 -> 98 (13.5), 166 -> 174 (27).
// Where a KV head has one query tile, dq has few rows to even roundings out whatever the keys, and CTAs of dk and dv with
// one tile each take the time: 398 -> 391 us (one token over 65536 keys).
static int parts_of(const Geo &g, int64_t units, int sms)
{
    const double tiles = static_cast<double>(units) * g.QT * g.KT;
    if (tiles <= kTwoTiles * sms) return kTwoParts;
    return tiles <= kTwoDqTiles * sms || g.QT == 1 ? kTwoOfDq : kOnePart;
}

// Tokens x heads of a query tile: the fewest tiles, then the fewest heads (a tile of
// one head has consecutive tokens, which see about the same keys).
static void choose_tiles(Geo &g)
{
    int64_t best = INT64_MAX;
    for (int gb = 1; gb <= std::min(g.G, kTile); ++gb) {
        const int64_t tb = std::min<int64_t>(kTile / gb, g.T);
        const int64_t tiles = (g.T + tb - 1) / tb * ((g.G + gb - 1) / gb);
        if (tiles < best) {
            best = tiles;
            g.Gb = gb;
            g.Tb = static_cast<int>(tb);
        }
    }
    g.TT = static_cast<int>(std::min<int64_t>((g.T + g.Tb - 1) / g.Tb, INT32_MAX));
    g.GG = (g.G + g.Gb - 1) / g.Gb;
    g.QT = static_cast<int>(std::min<int64_t>(best, INT32_MAX));
}

// 5-D map over [groups][T][Hk][G][D] fp16 rows: a box is 64 values x Gb heads x Tb tokens.
static int map_q(skv_handle *h, CUtensorMap *map, const void *base, const Geo &g)
{
    tc::EncodeTiledFn fn = tc::encode_fn();
    if (!fn) return fail(h, SKV_ECUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t d = static_cast<cuuint64_t>(g.D);
    cuuint64_t dims[5] = {d, static_cast<cuuint64_t>(g.G), static_cast<cuuint64_t>(g.Hk), static_cast<cuuint64_t>(g.T),
                          static_cast<cuuint64_t>(g.groups)};
    cuuint64_t strides[4] = {2 * d, 2 * d * g.G, 2 * d * g.H, g.groups > 1 ? 2 * d * g.H * g.T : 2 * d * g.H};
    cuuint32_t box[5] = {64, static_cast<cuuint32_t>(g.Gb), 1, static_cast<cuuint32_t>(g.Tb), 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(h, SKV_EUNSUPPORTED, "tensor map encoding failed (%d)", static_cast<int>(r));
    return SKV_OK;
}

// 3-D map over [groups][n][Hk * D] fp16 rows: a box is 64 values x 128 keys.
static int map_k(skv_handle *h, CUtensorMap *map, const void *base, const Geo &g, int64_t row_bytes)
{
    tc::EncodeTiledFn fn = tc::encode_fn();
    if (!fn) return fail(h, SKV_ECUDA, "cuTensorMapEncodeTiled is not available");
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(g.Hk) * g.D, static_cast<cuuint64_t>(g.n), static_cast<cuuint64_t>(g.groups)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(row_bytes * (g.groups > 1 ? g.n : 1))};
    cuuint32_t box[3] = {64, kTile, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(h, SKV_EUNSUPPORTED, "tensor map encoding failed (%d)", static_cast<int>(r));
    return SKV_OK;
}

static int check(skv_handle *h, const skv_shape *sh, const void *q, const void *k, const void *v, const int32_t *q_pos,
                 const int32_t *kv_rows, int64_t kv_rows_ld, int64_t kv_begin, int64_t kv_end, const float *o, const float *lse,
                 int32_t do_type, const void *d_o, const float *d_lse, int32_t g_type, void *dq, void *dk, void *dv)
{
    if (!sh) return fail(h, SKV_EINVAL, "shape is NULL");
    if (sh->S < 1 || sh->nq < 1 || sh->H < 1 || sh->Hk < 1 || sh->H % sh->Hk)
        return fail(h, SKV_EINVAL, "bad shape S=%d nq=%d H=%d Hk=%d", sh->S, sh->nq, sh->H, sh->Hk);
    if (sh->D != 64 && sh->D != 128) return fail(h, SKV_EUNSUPPORTED, "head dim %d (supported: 64, 128)", sh->D);
    if (sh->k_type != SKV_F16 || sh->v_type != SKV_F16) return fail(h, SKV_EUNSUPPORTED, "gradients are of fp16 rows");
    if (!std::isfinite(sh->scale)) return fail(h, SKV_EINVAL, "scale is not finite");
    if (kv_begin < 0 || kv_end < kv_begin)
        return fail(h, SKV_EINVAL, "bad key range [%lld, %lld)", (long long)kv_begin, (long long)kv_end);
    if (kv_rows && kv_rows_ld < kv_end) return fail(h, SKV_EINVAL, "kv_rows_ld smaller than kv_end");
    if (static_cast<int64_t>(sh->S) * sh->nq > INT32_MAX - 256 || kv_end > INT32_MAX - 256)
        return fail(h, SKV_EUNSUPPORTED, "S*nq or kv_end exceeds 2^31 - 256");
    if (!q || !k || !v || !o || !lse || !d_o) return fail(h, SKV_EINVAL, "NULL pointer");
    if (!dk != !dv) return fail(h, SKV_EINVAL, "dk and dv go together");
    if (do_type != SKV_F16 && do_type != SKV_F32) return fail(h, SKV_EINVAL, "d_o: type %d (fp16 or fp32 is wanted)", do_type);
    if (g_type != SKV_F16 && g_type != SKV_F32) return fail(h, SKV_EINVAL, "results: type %d (fp16 or fp32 is wanted)", g_type);
    const int64_t seg = static_cast<int64_t>(sh->Hk) * sh->D * 2;
    if (sh->k_row_bytes < seg || sh->v_row_bytes < seg) return fail(h, SKV_EINVAL, "row stride smaller than Hk head segments");
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) || misaligned(d_o, 16) ||
        misaligned(dq, 16) || misaligned(dk, 16) || misaligned(dv, 16) || sh->k_row_bytes % 16 || sh->v_row_bytes % 16)
        return fail(h, SKV_EUNSUPPORTED, "q, k, v, o, d_o, results and row strides must be multiples of 16 bytes");
    if (misaligned(lse, 4) || misaligned(d_lse, 4) || misaligned(q_pos, 4) || misaligned(kv_rows, 4))
        return fail(h, SKV_EUNSUPPORTED, "lse, d_lse, q_pos and kv_rows must be 4-byte aligned");
    // strides of a tensor map are below 2^40
    if (sh->k_row_bytes >= int64_t(1) << 39 || sh->v_row_bytes >= int64_t(1) << 39)
        return fail(h, SKV_EUNSUPPORTED, "row stride exceeds 2^39 bytes");
    return SKV_OK;
}

}  // namespace bwd
}  // namespace skv

using namespace skv;

extern "C" int skv_attn_backward(skv_handle *h, const skv_shape *shape, const void *q, const void *k, const void *v,
                                 const int32_t *q_pos, int64_t key_pos0, const int32_t *kv_rows, int64_t kv_rows_ld,
                                 int32_t kv_rows_per_head, int64_t kv_begin, int64_t kv_end, const float *o,
                                 const float *lse, int32_t do_type, const void *d_o, const float *d_lse, int32_t g_type,
                                 void *dq, void *dk, void *dv, void *stream)
{
    using namespace bwd;
    if (!h) return SKV_EINVAL;
    h->err[0] = 0;
    int rc = check(h, shape, q, k, v, q_pos, kv_rows, kv_rows_ld, kv_begin, kv_end, o, lse, do_type, d_o, d_lse, g_type, dq, dk, dv);
    if (rc) return rc;
    if (!dq && !dk) return SKV_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    Geo g{};
    g.groups = kv_rows ? shape->S : 1;
    g.T = kv_rows ? shape->nq : static_cast<int64_t>(shape->S) * shape->nq;
    g.Hk = shape->Hk;
    g.H = shape->H;
    g.G = shape->H / shape->Hk;
    g.D = shape->D;
    g.n = kv_end - kv_begin;
    g.KT = static_cast<int>((g.n + kTile - 1) / kTile);
    choose_tiles(g);
    const int64_t units = static_cast<int64_t>(g.groups) * g.Hk;
    if (g.QT > kMaxQTiles) return fail(h, SKV_EUNSUPPORTED, "%d tiles of query rows of a KV head (at most %d)", g.QT, kMaxQTiles);
    // (units first: the product of all stays within 64 bits, and so do the sizes below, of at most 128 rows a tile)
    if (units > INT32_MAX || units * (g.KT + static_cast<int64_t>(g.QT)) > INT32_MAX) return fail(h, SKV_EUNSUPPORTED, "too many tiles for one launch");
    if (g.groups > 1 && (2 * static_cast<int64_t>(g.H) * g.D * g.T >= int64_t(1) << 39 ||
                         2 * static_cast<int64_t>(g.Hk) * g.D * g.n >= int64_t(1) << 39))
        return fail(h, SKV_EUNSUPPORTED, "a sequence's rows exceed 2^39 bytes");
    OnDevice on(h->device);
    const size_t gs = g_type == SKV_F32 ? 4 : 2;
    const int64_t q_vals = static_cast<int64_t>(g.groups) * g.T * g.H * g.D, k_vals = static_cast<int64_t>(g.groups) * g.n * g.Hk * g.D;
    if (g.n == 0) {
        if (dq) return cuda_fail(h, cudaMemsetAsync(dq, 0, static_cast<size_t>(q_vals) * gs, st), "clearing dq");
        return SKV_OK;
    }
    // Pieces of a unit's tiles for grids that would leave SMs idle.
    const double nq = static_cast<double>(shape->nq), keys = static_cast<double>(g.n);
    const double share = !q_pos ? 1.0 : nq <= keys ? 1.0 - 0.5 * nq / keys : 0.5 * keys / nq;
    const Plan plan = plan_of(g, units, h->sm_count, dk != nullptr, dq != nullptr, share);
    const int parts = parts_of(g, units, h->sm_count);
    const int kv_pieces = plan.kv_pieces, q_pieces = plan.q_pieces;
    const bool kv_slot = dk && (kv_pieces > 1 || g.QT > kStretch), q_slot = dq && (q_pieces > 1 || g.KT > kStretch);

    // Scratch: row statistics, tile sums, exponents of the keys, rows gathered or converted, fp32 sums.
    size_t need = 0;
    auto take = [&](size_t bytes) {
        const size_t at = need;
        need += up(bytes);
        return at;
    };
    const size_t q_tiles = static_cast<size_t>(units) * g.QT, k_tiles = static_cast<size_t>(units) * g.KT;
    const size_t at_info = take(q_tiles * kInfoRows * kTile * 4);
    const size_t at_sum = take(q_tiles * sizeof(TileSum));
    const size_t at_ew = take(k_tiles * kTile);
    const size_t at_do = take(do_type == SKV_F32 ? static_cast<size_t>(q_vals) * 2 : 0);
    const size_t at_k = take(kv_rows ? static_cast<size_t>(k_vals) * 2 : 0);
    const size_t at_v = take(kv_rows ? static_cast<size_t>(k_vals) * 2 : 0);
    const size_t at_kv = take(kv_slot ? static_cast<size_t>(k_vals) * 2 * kv_pieces * 4 : 0);
    const size_t at_q = take(q_slot ? static_cast<size_t>(q_vals) * q_pieces * 4 : 0);
    if ((rc = ensure_workspace(h, need, st))) return rc;
    uint8_t *ws = static_cast<uint8_t *>(h->workspace);

    PrepArgs p{};
    p.g = g;
    p.d_o = d_o;
    p.o = o;
    p.lse = lse;
    p.d_lse = d_lse;
    p.q_pos = q_pos;
    p.pos0 = key_pos0 + kv_begin;
    p.doh = reinterpret_cast<__half *>(ws + at_do);
    p.info = reinterpret_cast<float *>(ws + at_info);
    p.sum = reinterpret_cast<TileSum *>(ws + at_sum);
    p.k = static_cast<const uint8_t *>(k) + (kv_rows ? 0 : kv_begin * shape->k_row_bytes);
    p.v = static_cast<const uint8_t *>(v) + (kv_rows ? 0 : kv_begin * shape->v_row_bytes);
    p.k_row_bytes = shape->k_row_bytes;
    p.v_row_bytes = shape->v_row_bytes;
    p.rows = kv_rows ? kv_rows + kv_begin : nullptr;
    p.rows_ld = kv_rows_ld;
    p.rows_per_head = kv_rows_per_head ? 1 : 0;
    p.kg = reinterpret_cast<__half *>(ws + at_k);
    p.vg = reinterpret_cast<__half *>(ws + at_v);
    p.ew = reinterpret_cast<int8_t *>(ws + at_ew);

    const int64_t packed = static_cast<int64_t>(g.Hk) * g.D * 2;
    CUtensorMap mq, mo, mk, mv;
    rc = map_q(h, &mq, q, g);
    if (!rc) rc = map_q(h, &mo, do_type == SKV_F32 ? static_cast<const void *>(p.doh) : d_o, g);
    if (!rc) rc = map_k(h, &mk, kv_rows ? static_cast<const void *>(p.kg) : p.k, g, kv_rows ? packed : shape->k_row_bytes);
    if (!rc) rc = map_k(h, &mv, kv_rows ? static_cast<const void *>(p.vg) : p.v, g, kv_rows ? packed : shape->v_row_bytes);
    if (rc) return rc;
    if ((rc = launch_prep(h, p, do_type, st))) return rc;

    MainArgs a{};
    a.g = g;
    a.scale = shape->scale;
    a.info = p.info;
    a.sum = p.sum;
    a.ew = p.ew;
    a.g_type = g_type;
    a.status = h->status;
    MainArgs b = a;
    a.pieces = kv_pieces;
    a.slot = kv_slot ? reinterpret_cast<float *>(ws + at_kv) : nullptr;
    a.out0 = dk;
    a.out1 = dv;
    b.pieces = q_pieces;
    b.slot = q_slot ? reinterpret_cast<float *>(ws + at_q) : nullptr;
    b.out0 = dq;
    if ((rc = launch_main(h, mq, mo, mk, mv, a, b, plan.q_first, parts, st))) return rc;
    if (kv_pieces > 1 && (rc = launch_join(h, a.slot, kv_pieces, k_vals, 2, g_type, dk, dv, st))) return rc;
    if (q_pieces > 1 && (rc = launch_join(h, b.slot, q_pieces, q_vals, 1, g_type, dq, nullptr, st))) return rc;
    return SKV_OK;
}
