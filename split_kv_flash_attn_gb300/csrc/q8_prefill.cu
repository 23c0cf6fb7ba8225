// q8_prefill.cu -- attention of many query rows per KV head over 8-bit pages, on
// the tensor cores (tcgen05).
//
// The mathematics.  Over a page the score of key j is (scale * d_k) (q . c_j) and
// its value d_v c_vj, with int8 codes c that are exact in fp16.  So a tile of 128
// keys (two pages) is decoded once into fp16 codes and used as it is: d_k enters
// as the factor of the exponent, d_v (its logarithm) as a summand of it:
//   w_j = 2^(d_k s_j - m + log2 d_v - r + 8),   O = sum w_j c_vj,
//   l = sum w_j 2^(r - log2 d_v),               o = 2^r O / l,
// m the row's reference (an integer, moved when a score passes it by 2^5), r the
// pages' (moved when a scale passes it by 2^2), both by exact powers of two.
// w stays below 2^15 and goes into the product as one fp16 number for fp16
// results, as two (itself rounded, and what that left) for fp32 ones.
//
// A CTA owns two 128-row query tiles of one KV head at a time (rows = tokens x
// the head's query heads), so each decoded tile serves both:
//   producers  : four warps, 32 key rows of every tile each; a row's 128 code
//                bytes lie 16 to a lane and are held in registers a tile ahead.
//   MMA thread : for tile g = 0, 1 in turn, O_g += W_g(j-1) V(j-1), then
//                S_g(j) = Q_g K(j)^T into the same tensor-memory columns.
//   softmax g  : four warps, one thread per query row, 64 keys (a page) at a time;
//                a half's weights are stored over its own consumed scores.
// While one tile's softmax runs, the tensor core works for the other.
//
// Work split.  All key tiles of all (sequence, KV head, tile pair) units form one
// line (its prefix sums come from a one-CTA plan kernel, which reads lengths and
// query positions on the device), cut into one equal piece for each CTA; units that several
// pieces share are merged by the last CTA to finish, in piece order.
//
// Tensor memory: S_0/W_0 in columns 0-127, S_1/W_1 128-255, O_0 256-383, O_1
// 384-511.  Every mbarrier wait is bounded; one that gives up sets the handle's
// device status word, the CTA drains what it issued and frees its tensor memory.
#include "q8.cuh"

namespace skv {
namespace q8 {

constexpr int kPM = 128;                        // query rows of a tile
constexpr int kPN = 128;                        // keys of a tile
constexpr int kSoftWarps = 8;                   // warps 0-3: tile 0, warps 4-7: tile 1
constexpr int kProdWarps = 4;                   // warps 8-11
constexpr int kMmaWarp = kSoftWarps + kProdWarps;
constexpr int kPfThreads = (kMmaWarp + 1) * 32;
constexpr int kPlanSmem = 1024;                 // plan entries kept in shared memory
constexpr float kPfShift = 8.f, kPfGrow = 5.f, kPfScaleGrow = 2.f;
constexpr float kNoScale = -100.f;              // log2 d_v - r of a zero scale (fp16 0, while l stays right)

template <int D>
struct PfSmem {
    static constexpr int kHalf = kPN * 128;     // 128 rows of 64 fp16
    static constexpr int kTile = D / 64 * kHalf;
    static constexpr int kQ = 0;                // two query tiles
    static constexpr int kK = kQ + 2 * kTile;   // two stages
    static constexpr int kV = kK + 2 * kTile;   // two stages
    static constexpr int kPlan = kV + 2 * kTile;
    static constexpr int kTotal = kPlan + (kPlanSmem + 1) * 8 + 1024;   // + alignment slack
};
static_assert(PfSmem<128>::kTotal <= 226 * 1024, "shared memory per CTA");

// Barriers (+ stage or query tile g).  Key tile j of the CTA is phase j / 2 of its
// K and V stages' barriers and j / 4 of its meta slot.  The t-th tile that query
// tile g takes part in (not every unit has a second one) is phase t of its S full,
// P full and PV done, the u-th such unit phase u of its Q full.  No waiter is ever
// two phases behind: each side needs the other's next step before it can complete
// another phase, and the softmax groups enter every unit together, so that a
// meta slot is rewritten (four tiles on) only after both have read it.
enum { PB_KFULL = 0, PB_KEMPTY = 2, PB_VFULL = 4, PB_VEMPTY = 6, PB_QFULL = 8, PB_SFULL = 10, PB_PFULL = 12,
       PB_PDONE = 14, PB_META = 16, PB_COUNT = 20 };

struct PrefillArgs {
    AttnArgs a;
    const int64_t *plan;                        // [S * n_pairs + 1] tiles before each (sequence, pair)
    int n_pairs;
    int out_f16;
};

// Tiles of each (sequence, pair of query tiles): up to its last visible key; prefix
// sums over all of them.
__global__ void __launch_bounds__(1024) prefill_plan_kernel(const AttnArgs a, int n_pairs, int64_t *plan)
{
    __shared__ int64_t s_sum[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n = static_cast<int64_t>(a.L.S) * n_pairs;
    const int64_t share = (n + 1023) / 1024, lo = min(n, tid * share), hi = min(n, lo + share);
    auto tiles = [&](int64_t e) {
        const int s = static_cast<int>(e / n_pairs), pr = static_cast<int>(e % n_pairs);
        int64_t keys = list_len(a.L, s);
        if (a.q_pos) {
            const int t0 = 2 * kPM * static_cast<int64_t>(pr) / a.G;
            const int t1 = static_cast<int>(min(int64_t(a.nq - 1), (2 * kPM * (static_cast<int64_t>(pr) + 1) - 1) / a.G));
            int top = -1;
            for (int t = t0; t <= t1; ++t) top = max(top, __ldg(a.q_pos + a.token(s, t)));
            keys = max(int64_t(0), min(keys, static_cast<int64_t>(top) + 1));
        }
        return (keys + kPN - 1) / kPN;
    };
    int64_t sum = 0;
    for (int64_t e = lo; e < hi; ++e) {
        const int64_t x = tiles(e);
        plan[e] = x;                            // (made a prefix sum below, by the same thread)
        sum += x;
    }
    for (int s = tid; s < a.L.S; s += 1024)
        if (list_len(a.L, s) < max(0, a.L.kv_len[s])) atomicOr(a.L.status, kStatusList);
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    int64_t before = inc - sum;
    for (int w = 0; w < warp; ++w) before += s_sum[w];
    for (int64_t e = lo; e < hi; ++e) {
        const int64_t x = plan[e];
        plan[e] = before;
        before += x;
    }
    if (tid == 1023) plan[n] = before;
}

template <int D, bool HILO>
__global__ void __launch_bounds__(kPfThreads, 1) prefill_kernel(const PrefillArgs pa)
{
    using SM = PfSmem<D>;
    const AttnArgs &a = pa.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_addr(sm);
    struct Meta {
        float ks, lv;                           // |d_k| scale log2(e); log2 |d_v|, -inf for 0
        int on;
    };
    __shared__ alignas(8) uint64_t s_bar[PB_COUNT];
    __shared__ Meta s_meta[4][2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_last;
    int64_t *s_plan = reinterpret_cast<int64_t *>(sm + SM::kPlan);
    const uint32_t bar0 = smem_addr(s_bar);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    constexpr uint32_t kIdescS = tc::idesc_f16(kPM, kPN, false);
    constexpr uint32_t kIdescPV = tc::idesc_f16(kPM, D, true);
    constexpr int kOCol = 2 * kPN;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int np = pa.n_pairs;
    const int64_t n_entries = static_cast<int64_t>(a.L.S) * np;
    const bool plan_here = n_entries <= kPlanSmem;
    if (plan_here)
        for (int i = tid; i <= n_entries; i += kPfThreads) s_plan[i] = __ldcg(pa.plan + i);
    auto plan = [&](int64_t e) { return plan_here ? s_plan[e] : __ldcg(pa.plan + e); };
    if (tid == 0) s_abort = 0;
    if (warp == 0) {
        tc::tmem_alloc<512>(smem_addr(&s_tmem));
        tc::tmem_relinquish();
    }
    if (tid == kMmaWarp * 32) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(PB_KFULL + i), kProdWarps * 32);
            tc::mbar_init(bar(PB_KEMPTY + i), 1);
            tc::mbar_init(bar(PB_VFULL + i), kProdWarps * 32);
            tc::mbar_init(bar(PB_VEMPTY + i), 1);
            tc::mbar_init(bar(PB_QFULL + i), kPM);
            tc::mbar_init(bar(PB_SFULL + i), 1);
            tc::mbar_init(bar(PB_PFULL + i), kPM);
            tc::mbar_init(bar(PB_PDONE + i), 1);
        }
        for (int i = 0; i < 4; ++i) tc::mbar_init(bar(PB_META + i), 2);
        tc::fence_barrier_init();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem;

    const int64_t total = plan(n_entries) * a.L.Hk;
    const int64_t chunk = max(int64_t(1), (total + gridDim.x - 1) / gridDim.x);
    const int64_t pos0 = min(total, blockIdx.x * chunk), pos_end = min(total, pos0 + chunk);

    // The units of the piece in turn, for every role.
    struct Unit {
        int s, kh, pr;
        int64_t unit0;                          // the line's position of its tile 0
        int t0, t1, n;                          // its tiles [t0, t1) are this CTA's, of n
    };
    auto unit_at = [&](int64_t pos) {
        Unit x;
        int lo = 0, hi = a.L.S;                 // the last sequence that begins at or before pos
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (plan(static_cast<int64_t>(mid) * np) * a.L.Hk <= pos) lo = mid;
            else hi = mid;
        }
        x.s = lo;
        const int64_t e0 = static_cast<int64_t>(lo) * np, p0 = plan(e0), T = plan(e0 + np) - p0;
        const int64_t r = pos - p0 * a.L.Hk;
        x.kh = static_cast<int>(r / T);
        const int64_t rr = r - x.kh * T + p0;   // within one head's pairs
        int64_t el = e0, eh = e0 + np;
        while (eh - el > 1) {
            const int64_t mid = (el + eh) >> 1;
            if (plan(mid) <= rr) el = mid;
            else eh = mid;
        }
        x.pr = static_cast<int>(el - e0);
        x.n = static_cast<int>(plan(el + 1) - plan(el));
        x.unit0 = pos - (rr - plan(el));
        x.t0 = static_cast<int>(pos - x.unit0);
        x.t1 = static_cast<int>(min(int64_t(x.n), pos_end - x.unit0));
        return x;
    };
    auto two_tiles = [&](const Unit &x) { return (2 * static_cast<int64_t>(x.pr) + 1) * kPM < a.rows; };

    // A phase already complete is taken at once; the abort flag is read only
    // when the barrier is not ready.
    auto wait = [&](int b, uint32_t parity) -> bool {
        if (tc::mbar_try_wait(bar(b), parity)) return true;
        if (*reinterpret_cast<volatile int *>(&s_abort)) return false;
        if (tc::mbar_wait(bar(b), parity, &s_abort)) return true;
        s_abort = 1;
        atomicOr(a.L.status, 1);
        return false;
    };
    auto store_o = [&](int64_t r, int c, const float (&v)[4]) {
        if (pa.out_f16)
            *reinterpret_cast<uint2 *>(static_cast<__half *>(a.o) + r * D + c) =
                make_uint2(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + r * D + c) = make_float4(v[0], v[1], v[2], v[3]);
    };

    // rows of pairs without a visible key: written here
    for (int64_t e = blockIdx.x; e < n_entries; e += gridDim.x) {
        if (plan(e + 1) != plan(e)) continue;
        const int s = static_cast<int>(e / np), pr = static_cast<int>(e % np);
        const int64_t r0 = 2 * kPM * static_cast<int64_t>(pr), nr = min(int64_t(2 * kPM), a.rows - r0);
        for (int64_t i = tid; i < nr * a.L.Hk; i += kPfThreads) {
            const int kh = static_cast<int>(i / nr), row = static_cast<int>(r0 + i % nr);
            const int64_t r = a.token(s, row / a.G) * a.H + kh * a.G + row % a.G;
            const float z[4] = {0.f, 0.f, 0.f, 0.f};
            for (int c = 0; c < D; c += 4) store_o(r, c, z);
            a.lse[r] = -INFINITY;
        }
    }

    if (warp >= kSoftWarps && warp < kMmaWarp) {
        // ---------------- producers ----------------------------------------------
        const int pw = warp - kSoftWarps;       // rows 32 pw .. of every tile: page pw / 2 of it
        constexpr int LPR = D / 16;             // lanes a row
        constexpr int RPI = 32 / LPR;           // rows an instruction
        constexpr int NI = 32 / RPI;            // instructions a warp's 32 rows
        const int c16 = lane % LPR, r0 = pw * 32 + lane / LPR;
        int64_t j = 0;                          // key tiles so far
        bool ok = true;
        auto convert = [&](const uint4 (&w)[NI], bool on, uint32_t neg, uint8_t *tile) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int r = r0 + i * RPI;
                const uint32_t in[4] = {w[i].x ^ 0x80808080u, w[i].y ^ 0x80808080u, w[i].z ^ 0x80808080u,
                                        w[i].w ^ 0x80808080u};
                uint32_t v[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[2 * e] = on ? codes_lo(in[e]) ^ neg : 0u;
                    v[2 * e + 1] = on ? codes_hi(in[e]) ^ neg : 0u;
                }
                // 16-byte chunks 2 c16 and 2 c16 + 1 of the row; lanes of the two
                // 64-channel halves write them in opposite order, so that a row's
                // writes spread over all banks
                uint8_t *dst = tile + (c16 >> 2) * SM::kHalf + r * 128;
                const int ch = 2 * (c16 & 3);
                const int a0 = ((ch + (c16 >> 2)) ^ (r & 7)) << 4, a1 = ((ch + 1 - (c16 >> 2)) ^ (r & 7)) << 4;
                const uint4 lo = make_uint4(v[0], v[1], v[2], v[3]), hi = make_uint4(v[4], v[5], v[6], v[7]);
                *reinterpret_cast<uint4 *>(dst + a0) = (c16 >> 2) ? hi : lo;
                *reinterpret_cast<uint4 *>(dst + a1) = (c16 >> 2) ? lo : hi;
            }
        };
        for (int64_t pos = pos0; ok && pos < pos_end;) {
            const Unit x = unit_at(pos);
            const int64_t len = list_len(a.L, x.s);
            const int32_t *ids = a.L.ids + (static_cast<int64_t>(x.s) * a.L.Hk + x.kh) * a.L.cap;
            auto page_id = [&](int tile) {
                const int64_t b = 2 * static_cast<int64_t>(tile) + (pw >> 1);
                return tile < x.t1 && b * kPage < len ? max(-1, checked_page(a.L, __ldg(ids + b))) : -1;
            };
            uint4 kr[NI], vr[NI];
            auto load = [&](uint4 (&w)[NI], const int8_t *codes, int id) {
                if (id < 0) return;
                const int8_t *p = codes + (static_cast<int64_t>(id) * kPage + (r0 & 63)) * D + c16 * 16;
#pragma unroll
                for (int i = 0; i < NI; ++i) w[i] = ld_stream16(p + i * RPI * D);
            };
            int id = page_id(x.t0), id1 = page_id(x.t0 + 1);
            float dk = id >= 0 ? __ldg(a.k_scale + id) : 0.f, dv = id >= 0 ? __ldg(a.v_scale + id) : 0.f;
            load(kr, a.k, id);
            load(vr, a.v, id);
            for (int tl = x.t0; tl < x.t1; ++tl, ++j) {
                const int b = static_cast<int>(j & 1);
                const uint32_t ph = static_cast<uint32_t>(j >> 1);
                const int id2 = page_id(tl + 2);
                const float dk1 = id1 >= 0 ? __ldg(a.k_scale + id1) : 0.f, dv1 = id1 >= 0 ? __ldg(a.v_scale + id1) : 0.f;
                const float ks = dk * a.scale_log2;
                if (!__all_sync(0xffffffffu, j < 2 || wait(PB_KEMPTY + b, (ph - 1) & 1))) { ok = false; break; }
                // (the slot's last reader is four tiles back: see the barriers)
                if ((pw & 1) == 0 && lane == 0) {
                    s_meta[j & 3][pw >> 1] = Meta{fmaxf(fabsf(ks), 1e-30f), dv != 0.f ? log2f(fabsf(dv)) : -INFINITY, id >= 0};
                    tc::mbar_arrive(bar(PB_META + static_cast<int>(j & 3)));
                }
                convert(kr, id >= 0, ks < 0.f ? 0x80008000u : 0u, sm + SM::kK + b * SM::kTile);
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(bar(PB_KFULL + b));
                load(kr, a.k, id1);
                if (!__all_sync(0xffffffffu, j < 2 || wait(PB_VEMPTY + b, (ph - 1) & 1))) { ok = false; break; }
                convert(vr, id >= 0, dv < 0.f ? 0x80008000u : 0u, sm + SM::kV + b * SM::kTile);
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(bar(PB_VFULL + b));
                load(vr, a.v, id1);
                id = id1;
                id1 = id2;
                dk = dk1;
                dv = dv1;
            }
            pos = x.unit0 + x.t1;
        }
    } else if (warp == kMmaWarp) {
        // ---------------- MMA issuer ---------------------------------------------
        if (lane == 0) {
            bool ok = true;
            int64_t j0 = 0;                     // the CTA's tiles before this unit
            uint32_t units[2] = {0, 0}, tiles[2] = {0, 0};   // of each query tile g so far
            int last_bar = -1;
            uint32_t last_par = 0;
            const uint64_t dq0 = tc::smem_desc(sbase + SM::kQ, 16, 1024);
            const uint64_t dk0 = tc::smem_desc(sbase + SM::kK, 16, 1024);
            const uint64_t dv0 = tc::smem_desc(sbase + SM::kV, SM::kHalf, 1024);
            for (int64_t pos = pos0; ok && pos < pos_end;) {
                const Unit x = unit_at(pos);
                const int ng = two_tiles(x) ? 2 : 1;
                const int n = x.t1 - x.t0;
                for (int g = 0; g < ng && ok; ++g) ok = wait(PB_QFULL + g, units[g]++ & 1);
                tc::tc_fence_after();
                for (int jj = 0; ok && jj <= n; ++jj) {
                    for (int g = 0; g < ng; ++g) {
                        const uint32_t d_s = tmem + static_cast<uint32_t>(g * kPN);
                        if (jj >= 1) {
                            // O_g += W_g V
                            const int64_t j = j0 + jj - 1;
                            const int b = static_cast<int>(j & 1);
                            const uint32_t par = (tiles[g] - 1) & 1;
                            if (!wait(PB_PFULL + g, par)) { ok = false; break; }
                            if (g == 0 && !wait(PB_VFULL + b, (j >> 1) & 1)) { ok = false; break; }
                            tc::tc_fence_after();
                            const uint32_t d_o = tmem + static_cast<uint32_t>(kOCol + g * D);
#pragma unroll
                            for (int kk = 0; kk < kPN / 16; ++kk) {
                                const uint64_t bd = tc::desc_add(dv0, b * SM::kTile + kk * 2048);
                                const uint32_t at = d_s + static_cast<uint32_t>((kk >> 2) * 64 + (kk & 3) * 8);
                                tc::mma_f16_ts(d_o, at, bd, kIdescPV, (jj > 1 || kk > 0) ? 1u : 0u);
                                if (HILO) tc::mma_f16_ts(d_o, at + 32, bd, kIdescPV, 1u);
                            }
                            tc::mma_commit(bar(PB_PDONE + g));
                            last_bar = PB_PDONE + g;
                            last_par = par;
                            if (g == ng - 1) tc::mma_commit(bar(PB_VEMPTY + b));
                        }
                        if (jj < n) {
                            // S_g = Q_g K^T, once PV_g of the tile before has read W_g
                            const int64_t j = j0 + jj;
                            const int b = static_cast<int>(j & 1);
                            if (g == 0 && !wait(PB_KFULL + b, (j >> 1) & 1)) { ok = false; break; }
                            if (tiles[g] >= 1 && !wait(PB_PDONE + g, (tiles[g] - 1) & 1)) { ok = false; break; }
                            tc::tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = (kk >> 2) * SM::kHalf + (kk & 3) * 32;
                                tc::mma_f16_ss(d_s, tc::desc_add(dq0, g * SM::kTile + off),
                                               tc::desc_add(dk0, b * SM::kTile + off), kIdescS, kk > 0 ? 1u : 0u);
                            }
                            tc::mma_commit(bar(PB_SFULL + g));
                            last_bar = PB_SFULL + g;
                            last_par = tiles[g]++ & 1;
                            if (g == ng - 1) tc::mma_commit(bar(PB_KEMPTY + b));
                        }
                    }
                }
                j0 += n;
                pos = x.unit0 + x.t1;
            }
            if (*reinterpret_cast<volatile int *>(&s_abort)) {
                // drain issued MMAs: the last commit covers every MMA issued before it
                if (last_bar >= 0) tc::mbar_wait(bar(last_bar), last_par, nullptr, 100000000ull);
            } else {
                // nobody waits for the last commits on the stages' free barriers;
                // they are awaited here, so that none is in flight at exit
                for (int64_t j = max(int64_t(0), j0 - 2); j < j0; ++j) {
                    wait(PB_KEMPTY + static_cast<int>(j & 1), (j >> 1) & 1);
                    wait(PB_VEMPTY + static_cast<int>(j & 1), (j >> 1) & 1);
                }
            }
        }
    } else {
        // ---------------- softmax: one thread per query row -----------------------
        const int g = warp >> 2;
        const int m = (warp & 3) * 32 + lane;   // row of the tile = lane of tensor memory
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_col = lane_base + static_cast<uint32_t>(g * kPN);
        const uint32_t o_col = lane_base + static_cast<uint32_t>(kOCol + g * D);
        auto put_q = [&](const Unit &x) {       // this thread's query row into shared memory
            const int64_t row = (2 * static_cast<int64_t>(x.pr) + g) * kPM + m;
            const bool on = row < a.rows;
            const int64_t r = on ? a.token(x.s, static_cast<int>(row / a.G)) * a.H + x.kh * a.G + row % a.G : 0;
            const __half *qp = a.q + r * D;
            uint8_t *qt = sm + SM::kQ + g * SM::kTile + m * 128;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint4 v = on ? __ldg(reinterpret_cast<const uint4 *>(qp) + c) : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(qt + (c >> 3) * SM::kHalf + (((c & 7) ^ (m & 7)) << 4)) = v;
            }
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(bar(PB_QFULL + g));
        };
        int64_t j = 0;                          // key tiles so far
        uint32_t tiles = 0;                     // of them with this group's query tile
        auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory"); };
        auto active = [&](const Unit &y) { return g == 0 || two_tiles(y); };
        Unit x = {};
        if (pos0 < pos_end) {
            x = unit_at(pos0);
            if (active(x)) put_q(x);
        }
        for (int64_t pos = pos0; pos < pos_end;) {
            meet();
            const int64_t row = (2 * static_cast<int64_t>(x.pr) + g) * kPM + m;
            const bool row_on = row < a.rows;
            const bool tile_on = active(x);
            const int64_t len = list_len(a.L, x.s);
            int64_t lim = len;                  // keys that this row sees
            const int64_t tok = a.token(x.s, row_on ? static_cast<int>(row / a.G) : 0);
            if (a.q_pos) lim = max(int64_t(0), min(len, static_cast<int64_t>(__ldg(a.q_pos + tok)) + 1));
            float m_ref = -INFINITY, r_ref = -INFINITY, l_run = 0.f;
            const int n = x.t1 - x.t0;
            if (tile_on) {
                // No early exit from this loop: after a wait gives up, every later
                // wait returns at once and the warp runs through (the outputs are
                // then invalid and the status word says so).
                for (int jj = 0; jj < n; ++jj, ++j, ++tiles) {
                    const int64_t key0 = static_cast<int64_t>(x.t0 + jj) * kPN;
                    __all_sync(0xffffffffu, wait(PB_SFULL + g, tiles & 1));
                    __all_sync(0xffffffffu, wait(PB_META + static_cast<int>(j & 3), (j >> 2) & 1));
                    tc::tc_fence_after();
                    const Meta m0 = s_meta[j & 3][0], m1 = s_meta[j & 3][1];
                    // the pages' reference
                    const float r_old = r_ref;
                    const float lv_max = fmaxf(m0.on ? m0.lv : -INFINITY, m1.on ? m1.lv : -INFINITY);
                    if (lv_max > r_ref + kPfScaleGrow) r_ref = ceilf(lv_max);
                    float ref = m_ref, beta = 1.f, ls0 = 0.f, ls1 = 0.f;
                    const int64_t lim_t = lim - key0;               // columns at or past it are masked
                    const bool masked = __any_sync(0xffffffffu, lim_t < kPN);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const Meta mt = h == 0 ? m0 : m1;
                        uint32_t xr[2][32];
#pragma unroll
                        for (int c = 0; c < 2; ++c) tc::tmem_ld32(s_col + h * 64 + c * 32, xr[c]);
#pragma unroll
                        for (int c = 0; c < 2; ++c) tc::tmem_wait_ld(xr[c]);
                        auto X = [&](int i) -> uint32_t & { return xr[i >> 5][i & 31]; };
                        if (masked || !mt.on) {
                            const int64_t lh = mt.on ? lim_t - h * 64 : 0;
#pragma unroll
                            for (int i = 0; i < 64; ++i)
                                if (i >= lh) X(i) = 0xff800000u;
                        }
                        float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < 64; ++i) mq[i & 3] = fmaxf(mq[i & 3], __uint_as_float(X(i)));
                        const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * mt.ks;
                        const float prev = ref;
                        if (mx > ref + kPfGrow) ref = ceilf(mx);    // true on the first finite maximum
                        const float dl = mt.lv == -INFINITY ? kNoScale : fmaxf(mt.lv - r_ref, kNoScale);
                        const float off = ref == -INFINITY ? 0.f : kPfShift + dl - ref;
                        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            // 32 keys: weights over their own consumed scores
                            uint32_t hi[16], lo[16];
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float w0 = fast_exp2(fmaf(__uint_as_float(xr[c][i]), mt.ks, off));
                                const float w1 = fast_exp2(fmaf(__uint_as_float(xr[c][i + 1]), mt.ks, off));
                                ls[i & 2] += w0;
                                ls[(i & 2) + 1] += w1;
                                hi[i >> 1] = pack_half2(w0, w1);
                                if (HILO) {
                                    const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hi[i >> 1]));
                                    lo[i >> 1] = pack_half2(w0 - back.x, w1 - back.y);
                                }
                            }
                            tc::tmem_st16u(s_col + h * 64 + c * 16, hi);
                            if (HILO) tc::tmem_st16u(s_col + h * 64 + 32 + c * 16, lo);
                        }
                        const float lh = ((ls[0] + ls[1]) + (ls[2] + ls[3])) * fast_exp2(-dl);
                        if (a.page_lse && row_on && key0 + h * 64 < len)
                            a.page_lse[((static_cast<int64_t>(x.s) * a.L.Hk + x.kh) * a.L.cap + 2 * (x.t0 + jj) + h) * a.rows + row] =
                                lh > 0.f ? ref - kPfShift + log2f(lh) : -INFINITY;
                        if (h == 0) {
                            ls0 = lh;
                        } else {
                            ls1 = lh;
                            if (ref != prev) beta = prev == -INFINITY ? 0.f : fast_exp2(prev - ref);
                            if (__any_sync(0xffffffffu, beta != 1.f)) {
                                // the first half's weights, stored above, to the moved reference
                                tc::tmem_wait_st();
                                // (two exact factors, as fp16 has none below 2^-24)
                                const float e = prev == -INFINITY ? -28.f : fmaxf(prev - ref, -28.f);
                                const __half2 b0 = __float2half2_rn(fast_exp2(fmaxf(e, -14.f)));
                                const __half2 b1 = __float2half2_rn(fast_exp2(fminf(e + 14.f, 0.f)));
#pragma unroll
                                for (int c = 0; c < (HILO ? 2 : 1); ++c) {
                                    uint32_t pr[32];
                                    tc::tmem_ld32(s_col + c * 32, pr);
                                    tc::tmem_wait_ld(pr);
#pragma unroll
                                    for (int i = 0; i < 32; ++i) {
                                        const __half2 v = __hmul2(__hmul2(*reinterpret_cast<const __half2 *>(&pr[i]), b0), b1);
                                        pr[i] = *reinterpret_cast<const uint32_t *>(&v);
                                    }
                                    tc::tmem_st32u(s_col + c * 32, pr);
                                }
                            }
                        }
                    }
                    const float alpha = ref == m_ref ? 1.f : (m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - ref));
                    const float alpha_o = r_ref == r_old ? alpha : (r_old == -INFINITY ? 0.f : alpha * fast_exp2(r_old - r_ref));
                    // O_g holds every PV up to the last tile (S_g was issued after
                    // it was done) and none of this tile before W_g is full
                    if (jj > 0 && __any_sync(0xffffffffu, alpha_o != 1.f)) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t rr[32];
                            tc::tmem_ld32(o_col + c * 32, rr);
                            tc::tmem_wait_ld(rr);
                            float v[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(rr[i]) * alpha_o;
                            tc::tmem_st32(o_col + c * 32, v);
                        }
                    }
                    l_run = l_run * alpha + (ls0 * beta + ls1);
                    m_ref = ref;
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                    tc::mbar_arrive(bar(PB_PFULL + g));
                }
            }
            // the next unit's queries go in while this one's last product runs: S_g of
            // the last tile is done, and nothing else reads Q_g
            const Unit cur = x;
            const int64_t here = pos;
            pos = x.unit0 + x.t1;
            if (!tile_on) j += n;
            if (pos < pos_end) {
                x = unit_at(pos);
                if (active(x)) put_q(x);
            }
            // ---------------- O / l, lse: result or piece ------------------------------
            const bool whole = cur.t0 == 0 && cur.t1 == cur.n;
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (here == pos0 ? 0 : 1);
            if (tile_on) {
                bool have = !*reinterpret_cast<volatile int *>(&s_abort) && wait(PB_PDONE + g, (tiles - 1) & 1);
                have = __all_sync(0xffffffffu, have);
                if (have) tc::tc_fence_after();
                const bool empty = !have || !(l_run > 0.f);
                const float inv = empty ? 0.f : fast_exp2(r_ref == -INFINITY ? 0.f : r_ref) / l_run;
                const int64_t r = tok * a.H + cur.kh * a.G + row % a.G;
                const float lse2 = empty ? -INFINITY : m_ref - kPfShift + log2f(l_run);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t orr[32];
                    if (have) {
                        tc::tmem_ld32(o_col + c * 32, orr);         // warp-wide: every lane takes part
                        tc::tmem_wait_ld(orr);
                    }
                    if (row_on) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            float v[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] = empty ? 0.f : __uint_as_float(orr[i + e]) * inv;
                            if (whole)
                                store_o(r, c * 32 + i, v);
                            else
                                *reinterpret_cast<float4 *>(a.part_o + ((slot * 2 + g) * kPM + m) * D + c * 32 + i) =
                                    make_float4(v[0], v[1], v[2], v[3]);
                        }
                    }
                }
                if (row_on) {
                    if (whole) a.lse[r] = lse2 * 0.6931471805599453f;
                    else a.part_ml[(slot * 2 + g) * kPM + m] = lse2;
                }
                tc::tc_fence_before();          // O_g is read before W_g of the next unit is announced
            }
            if (!whole) {
                // the last CTA of the unit puts the pieces together, in order
                const int64_t unit = (static_cast<int64_t>(cur.s) * a.L.Hk + cur.kh) * np + cur.pr;
                const int64_t c_lo = cur.unit0 / chunk, c_hi = (cur.unit0 + cur.n - 1) / chunk;
                __threadfence();
                meet();
                if (tid == 0) s_last = atomicAdd(a.counters + unit, 1) == static_cast<int>(c_hi - c_lo);
                meet();
                if (s_last) {
                    __threadfence();
                    const int64_t first = 2 * kPM * static_cast<int64_t>(cur.pr);
                    const int nr = static_cast<int>(min(int64_t(2 * kPM), a.rows - first));
                    auto slot_of = [&](int64_t c) { return 2 * c + (c == c_lo && cur.unit0 > c * chunk ? 1 : 0); };
                    constexpr int V = D / 4;    // float4 of a row
                    for (int i = tid; i < nr * V; i += kSoftWarps * 32) {
                        const int rr = i / V, c4 = i % V;
                        float M = -INFINITY;
                        for (int64_t c = c_lo; c <= c_hi; ++c) M = fmaxf(M, __ldcg(a.part_ml + slot_of(c) * 2 * kPM + rr));
                        float W = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
                        if (M != -INFINITY) {
#pragma unroll 4
                            for (int64_t c = c_lo; c <= c_hi; ++c) {
                                const int64_t at = slot_of(c) * 2 * kPM + rr;
                                const float w = fast_exp2(__ldcg(a.part_ml + at) - M);
                                const float4 y = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * D) + c4);
                                W += w;
                                v[0] = fmaf(w, y.x, v[0]);
                                v[1] = fmaf(w, y.y, v[1]);
                                v[2] = fmaf(w, y.z, v[2]);
                                v[3] = fmaf(w, y.w, v[3]);
                            }
                            const float q = 1.f / W;
                            for (int e = 0; e < 4; ++e) v[e] *= q;
                        }
                        const int64_t prow = first + rr;
                        const int64_t r = a.token(cur.s, static_cast<int>(prow / a.G)) * a.H + cur.kh * a.G + prow % a.G;
                        store_o(r, c4 * 4, v);
                        if (c4 == 0) a.lse[r] = M == -INFINITY ? -INFINITY : (M + log2f(W)) * 0.6931471805599453f;
                    }
                    if (tid == 0) a.counters[unit] = 0;
                }
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after();
        tc::tmem_dealloc<512>(tmem);
    }
}

// Attention weight of each page from the log sums of its rows: one warp a page,
// rows in the lanes' order.
__global__ void __launch_bounds__(256) prefill_mass_kernel(const AttnArgs a, float *mass)
{
    const int kh = blockIdx.y, s = blockIdx.z;
    const int64_t unit = static_cast<int64_t>(s) * a.L.Hk + kh;
    const int64_t p = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (p * kPage >= list_len(a.L, s)) return;
    const float *pl = a.page_lse + (unit * a.L.cap + p) * a.rows;
    float sum = 0.f;
    for (int r = lane; r < a.rows; r += 32) {
        const int64_t tok = a.token(s, r / a.G);
        // a tile past the row's last visible key was not walked: nothing was written
        if (a.q_pos && p * kPage > __ldg(a.q_pos + tok)) continue;
        const float z = a.lse[tok * a.H + kh * a.G + r % a.G] * 1.4426950408889634f;
        sum += z == -INFINITY ? 0.f : fast_exp2(__ldcg(pl + r) - z);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) mass[unit * a.L.cap + p] += sum;
}

template <int D, bool HILO>
static int launch_one(skv_handle *h, const PrefillArgs &pa, int grid, cudaStream_t st)
{
    static KernelAttrCache cache;
    constexpr int smem = PfSmem<D>::kTotal;
    const cudaError_t e = kernel_smem_optin(cache, reinterpret_cast<const void *>(prefill_kernel<D, HILO>), smem, kPfThreads, nullptr);
    if (e != cudaSuccess) return cuda_fail(h, e, "cudaFuncSetAttribute(8-bit prefill)");
    if (h->prof_before) cudaEventRecord(h->prof_before, st);
    prefill_kernel<D, HILO><<<grid, kPfThreads, smem, st>>>(pa);
    const cudaError_t l = cudaGetLastError();
    if (h->prof_after) cudaEventRecord(h->prof_after, st);
    return cuda_fail(h, l, "8-bit prefill launch");
}

int launch_prefill(skv_handle *h, const AttnArgs &a, int D, bool f16, int64_t *plan, int n_pairs, float *mass, int grid,
                   cudaStream_t st)
{
    prefill_plan_kernel<<<1, 1024, 0, st>>>(a, n_pairs, plan);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(h, e, "8-bit prefill plan launch");
    const PrefillArgs pa{a, plan, n_pairs, f16};
    int rc;
    if (D == 128) rc = f16 ? launch_one<128, false>(h, pa, grid, st) : launch_one<128, true>(h, pa, grid, st);
    else rc = f16 ? launch_one<64, false>(h, pa, grid, st) : launch_one<64, true>(h, pa, grid, st);
    if (rc || !mass) return rc;
    prefill_mass_kernel<<<dim3(static_cast<unsigned>((a.L.cap + 7) / 8), a.L.Hk, a.L.S), 256, 0, st>>>(a, mass);
    return cuda_fail(h, cudaGetLastError(), "page weight launch");
}

}  // namespace q8
}  // namespace skv
