// q8_select.cu -- picking pages: bounds of the pages' scores for each query,
// the choice of the best n, and the same choice by accumulated weight for
// eviction.
//
// The bound.  A page keeps the smallest and largest K code of each channel,
// so sum_d max(cq_d min_d, cq_d max_d) bounds the product of the coded query with
// every key of the page (where its scale is negative, sum_d max(-cq_d min_d, -cq_d max_d) the
// negated product).  It is cq+ . max + cq- . min, the positive and the
// negative part of the query against the two extremes, which change places (and the
// sign) for a negative scale: one product of length
// 2D of whole numbers of at most 127, whose sums stay below 2^21, so the tensor
// cores' fp32 sums are exact and the picks do not depend on the order of
// anything.  A warp takes 16 pages (the M side; bytes straight from global
// memory into fragments, as in the decode kernel) against the queries of a KV
// head, 8 columns at a time.
//
// The choice.  Scores become 32-bit keys whose order as unsigned numbers is the
// scores' order; one CTA for each list (a kernel of its own, or the last to score a
// page of it) finds the n-th largest key two bits at a
// time, counting keys in registers, and writes the picked indices in order by
// prefix sums over the warps' equal shares.  Ties at the n-th key go to the lowest
// indices.
//
// Bound (select and attend over 16 of 128 pages: 18.5 us, of which 9 here; 512 of 4096
// pages of 16 lists: 53 and 18): the scores by latency (lengths, ids, extremes and
// queries are read one after the other, 2D + 8 bytes a page and head in all); the
// choice by its counting rounds, each one pass over registers and one barrier, three or four until
// few keys are left to each warp alone (cutting 64 lists of up to 2048 pages to 512 took
// 13.4 us with 12 rounds, 10.3 so, and 9.0 since a warp ends a round at its last key).
#include <algorithm>
#include <type_traits>

#include "q8.cuh"

namespace skv {
namespace q8 {

constexpr uint32_t kNever = 0u;               // no candidate
constexpr uint32_t kAlways = 0xfffffffeu;     // picked whatever its score

// Order of floats as unsigned numbers within [1, 0xfffffffd]; -0 as +0, NaN as +inf.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (!(x == x)) x = INFINITY;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;      // -inf: 0x007fffff, +inf: 0xff800000
}

// ---------------------------------------------------------------- the bounds

constexpr int kScoreWarps = 8;
constexpr int kScoreCols = 64;                // query columns in shared memory at a time

// The codes of 16 pages as fragments: rows g, g + 8; [largest | smallest].
template <int D>
struct Extremes {
    static constexpr int CH = D / 64;
    uint4 x[2][2][CH];
    int id[2];
    float scale[2];

    __device__ void ids_of(const SelectArgs &a, const int32_t *ids, int64_t first, int64_t nb, int g)
    {
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
            const int64_t b = first + g + 8 * rr;
            id[rr] = b < nb ? checked_page(a.L, __ldg(ids + b)) : -1;
        }
    }
    __device__ void load(const SelectArgs &a, int t)
    {
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
            scale[rr] = id[rr] >= 0 ? __ldg(a.k_scale + id[rr]) : 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int64_t off = static_cast<int64_t>(max(id[rr], 0)) * D + 64 * c + 16 * t;
                x[0][rr][c] = id[rr] >= 0 ? ld_stream16(a.k_max + off) : make_uint4(0, 0, 0, 0);
                x[1][rr][c] = id[rr] >= 0 ? ld_stream16(a.k_min + off) : make_uint4(0, 0, 0, 0);
            }
        }
    }
    // Where a scale is negative, the two change places.
    __device__ void turn()
    {
#pragma unroll
        for (int rr = 0; rr < 2; ++rr)
            if (scale[rr] < 0.f) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint4 y = x[0][rr][c];
                    x[0][rr][c] = x[1][rr][c];
                    x[1][rr][c] = y;
                }
            }
    }
};

// ---------------------------------------------------------------- the choice

// The keys of one list for a CTA of THREADS: each warp takes an equal run of
// indices, 32 at a time.  KPT > 0: in registers, KPT a thread; 0: where `at` says.
template <int THREADS, int KPT>
struct Keys {
    static constexpr int W = THREADS / 32;
    uint32_t k[KPT > 0 ? KPT : 1];
    const uint32_t *at;
    int n, lo, hi;                                        // the warp's run

    __device__ Keys(int n_, const uint32_t *at_) : at(at_), n(n_)
    {
        const int share = (n + THREADS - 1) / THREADS * 32, warp = threadIdx.x >> 5;
        lo = min(n, warp * share);
        hi = min(n, lo + share);
    }
    // f(i, key of i or 0, whether there is an i) for the lane's index of every step
    template <typename F>
    __device__ __forceinline__ void each(F f) const
    {
        const int lane = threadIdx.x & 31;
        if constexpr (KPT > 0) {
#pragma unroll
            for (int e = 0; e < KPT; ++e) {
                if (lo + 32 * e >= hi) break;
                f(lo + 32 * e + lane, k[e], lo + 32 * e + lane < hi);
            }
        } else {
            for (int i = lo; i < hi; i += 32) f(i + lane, i + lane < hi ? at[i + lane] : 0u, i + lane < hi);
        }
    }
    template <typename F>
    __device__ __forceinline__ void fill(F f)             // k of index i = f(i), 0 past the end
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int e = 0; e < KPT; ++e) {
            const int i = lo + 32 * e + lane;
            k[e] = i < hi ? f(i) : 0u;
        }
    }
};

constexpr int kFew = 256;                     // keys that a warp looks through by itself

template <int THREADS>
struct PickScratch {
    static constexpr int W = THREADS / 32;
    int cnt[2][3][W];
    uint32_t lo[W], hi[W];
    int always[W], ranked[W];
    int n[3][W];
    uint32_t few[kFew];
    int n_few;
};

// A value T such that the `count` largest keys are those above T and some equal to
// it (n > count >= 1, no more than `count` of them kAlways): the count-th largest key,
// or, once a prefix of it tells the largest `count` from the others, anything between
// the two.  Two bits a round; when few keys share the prefix found so far, every warp
// goes on with those alone.
template <int THREADS, int KPT>
__device__ uint32_t threshold(const Keys<THREADS, KPT> &keys, int count, PickScratch<THREADS> &sc)
{
    constexpr int W = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // keys between kNever and kAlways: bits that all share need no rounds
    uint32_t both = 0xffffffffu, any = 0u;
    int na = 0, nr = 0;
    keys.each([&](int, uint32_t x, bool in) {
        const bool ranked = in && x - 1u < kAlways - 1u;
        both &= ranked ? x : 0xffffffffu;
        any |= ranked ? x : 0u;
        na += in && x == kAlways;
        nr += ranked;
    });
    both = __reduce_and_sync(0xffffffffu, both);
    any = __reduce_or_sync(0xffffffffu, any);
    na = __reduce_add_sync(0xffffffffu, na);
    nr = __reduce_add_sync(0xffffffffu, nr);
    if (lane == 0) {
        sc.lo[warp] = both;
        sc.hi[warp] = any;
        sc.always[warp] = na;
        sc.ranked[warp] = nr;
    }
    if (threadIdx.x == 0) sc.n_few = 0;
    __syncthreads();
    both = __reduce_and_sync(0xffffffffu, lane < W ? sc.lo[lane] : 0xffffffffu);
    any = __reduce_or_sync(0xffffffffu, lane < W ? sc.hi[lane] : 0u);
    na = __reduce_add_sync(0xffffffffu, lane < W ? sc.always[lane] : 0);
    nr = __reduce_add_sync(0xffffffffu, lane < W ? sc.ranked[lane] : 0);
    if (na >= count) return kAlways - 1u;
    if (na + nr <= count) return kNever;
    const uint32_t diff = both ^ any;
    if (diff == 0) return both;
    int b = (31 - __clz(diff)) & ~1;                      // the highest pair of bits in which keys differ
    uint32_t found = both & ~((4u << b) - 1u);            // (b = 30: none)
    int reach = na + nr, beyond = na;                     // keys from `found` up, and behind those that share its prefix
    // how many keys reach found + 1, 2, 3 units of 2^b; whether that decides
    auto decides = [&](int c1, int c2, int c3) {
        const uint32_t t1 = found | (1u << b), t2 = found | (2u << b), t3 = found | (3u << b);
        if (c3 == count || c2 == count || c1 == count) {
            found = (c3 == count ? t3 : c2 == count ? t2 : t1) - 1u;
            return true;
        }
        if (c3 > count) {
            found = t3;
            reach = c3;
        } else if (c2 > count) {
            found = t2;
            reach = c2;
            beyond = c3;
        } else if (c1 > count) {
            found = t1;
            reach = c1;
            beyond = c2;
        } else {
            beyond = c1;
        }
        return false;
    };
    for (int round = 0; reach - beyond > kFew; round ^= 1) {
        const uint32_t t1 = found | (1u << b), t2 = found | (2u << b), t3 = found | (3u << b);
        int c1 = 0, c2 = 0, c3 = 0;
        keys.each([&](int, uint32_t x, bool) {
            c1 += x >= t1;
            c2 += x >= t2;
            c3 += x >= t3;
        });
        c1 = __reduce_add_sync(0xffffffffu, c1);
        c2 = __reduce_add_sync(0xffffffffu, c2);
        c3 = __reduce_add_sync(0xffffffffu, c3);
        if (lane < 3) sc.cnt[round][lane][warp] = lane == 0 ? c1 : lane == 1 ? c2 : c3;
        __syncthreads();
        c1 = __reduce_add_sync(0xffffffffu, lane < W ? sc.cnt[round][0][lane] : 0);
        c2 = __reduce_add_sync(0xffffffffu, lane < W ? sc.cnt[round][1][lane] : 0);
        c3 = __reduce_add_sync(0xffffffffu, lane < W ? sc.cnt[round][2][lane] : 0);
        if (decides(c1, c2, c3)) return found;
        b -= 2;
        if (b < 0) return found;
    }
    // the keys that share the prefix: in [found, found + 4 units), all of them ranked
    const uint32_t width = (4u << b) - 1u;
    keys.each([&](int, uint32_t x, bool in) {
        if (in && x - 1u < kAlways - 1u && x - found <= width) sc.few[atomicAdd(&sc.n_few, 1)] = x;
    });
    __syncthreads();
    uint32_t x[kFew / 32];
#pragma unroll
    for (int i = 0; i < kFew / 32; ++i) x[i] = lane + 32 * i < reach - beyond ? sc.few[lane + 32 * i] : 0u;
    const int above = beyond;
    for (; b >= 0; b -= 2) {
        const uint32_t t1 = found | (1u << b), t2 = found | (2u << b), t3 = found | (3u << b);
        int c1 = 0, c2 = 0, c3 = 0;
#pragma unroll
        for (int i = 0; i < kFew / 32; ++i) {
            c1 += x[i] >= t1;
            c2 += x[i] >= t2;
            c3 += x[i] >= t3;
        }
        c1 = __reduce_add_sync(0xffffffffu, c1);
        c2 = __reduce_add_sync(0xffffffffu, c2);
        c3 = __reduce_add_sync(0xffffffffu, c3);
        if (decides(above + c1, above + c2, above + c3)) return found;
    }
    return found;
}

// In the order of indices, calls emit(i, key, above, ties, nevers) for every i in [0, n):
// how many earlier keys are above T, equal to it, and kNever.  `totals` receives the
// counts over all keys before any emit.
template <int THREADS, int KPT, typename B, typename E>
__device__ void in_order(const Keys<THREADS, KPT> &keys, uint32_t T, PickScratch<THREADS> &sc, B totals, E emit)
{
    constexpr int W = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int c0 = 0, c1 = 0, c2 = 0;
    keys.each([&](int, uint32_t k, bool in) {
        c0 += in && k > T;
        c1 += in && k == T;
        c2 += in && k == kNever;
    });
    c0 = __reduce_add_sync(0xffffffffu, c0);
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    if (lane < 3) sc.n[lane][warp] = lane == 0 ? c0 : lane == 1 ? c1 : c2;
    __syncthreads();
    int at[3], all[3];
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        const int x = lane < W ? sc.n[e][lane] : 0;
        at[e] = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
        all[e] = __reduce_add_sync(0xffffffffu, x);
    }
    totals(all[0], all[1], all[2]);
    const unsigned before = (1u << lane) - 1u;
    keys.each([&](int i, uint32_t k, bool in) {
        const unsigned m0 = __ballot_sync(0xffffffffu, in && k > T), m1 = __ballot_sync(0xffffffffu, in && k == T),
                       m2 = __ballot_sync(0xffffffffu, in && k == kNever);
        if (in) emit(i, k, at[0] + __popc(m0 & before), at[1] + __popc(m1 & before), at[2] + __popc(m2 & before));
        at[0] += __popc(m0);
        at[1] += __popc(m1);
        at[2] += __popc(m2);
    });
}

// Threads and keys a thread for lists of up to `cap` pages: few threads meet sooner
// and count in registers (choosing from 4096 pages took 14 us with 1024 threads over
// shared memory, 11 so).
template <typename F>
auto for_cap(int64_t cap, F f)
{
    if (cap <= 1024) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
    if (cap <= 6144) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 12>());
    if (cap <= 16384) return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 0>());
}

// The choice for one row (sequence, token, KV head) of n candidate pages.
template <int THREADS, int KPT>
__device__ void pick_row(const uint32_t *src, int n, int n_sel, int32_t *out, PickScratch<THREADS> &sc)
{
    Keys<THREADS, KPT> keys(n, src);
    if constexpr (KPT > 0) keys.fill([&](int i) { return __ldcg(src + i); });
    // no more pages than places: all candidates; else the keys above the n-th and the
    // first ties with it
    const uint32_t T = n > n_sel ? threshold(keys, n_sel, sc) : kNever;
    int need = 0, picked = 0;
    in_order(
        keys, T, sc,
        [&](int above, int, int) {
            need = T == kNever ? 0 : n_sel - above;
            picked = above + need;
        },
        [&](int i, uint32_t k, int above, int ties, int) {
            if (k > T || (k == T && ties < need)) out[above + min(ties, need)] = i;
        });
    for (int i = picked + threadIdx.x; i < n_sel; i += THREADS) out[i] = -1;
}

// One CTA a row.
template <int THREADS, int KPT>
__global__ void __launch_bounds__(THREADS) pick_kernel(const SelectArgs a)
{
    start();
    __shared__ PickScratch<THREADS> sc;
    const int64_t row = blockIdx.x;
    const int64_t st = row / a.L.Hk;
    const int s = static_cast<int>(st / a.nq);
    const int64_t tok = a.token(s, static_cast<int>(st % a.nq));
    int64_t seen = list_len(a.L, s);
    if (a.q_pos) seen = max(int64_t(0), min(seen, static_cast<int64_t>(__ldg(a.q_pos + tok)) + 1));
    pick_row<THREADS, KPT>(a.keys + row * a.L.cap, static_cast<int>((seen + kPage - 1) / kPage), a.n_sel,
                           a.sel + (tok * a.L.Hk + row % a.L.Hk) * a.n_sel, sc);
}

// ------------------------------------------------------- the bounds of all pages

// Grid: x pieces of a list's pages, `tg` tokens at a time dealt to `parts` CTAs, y KV
// heads, z sequences.  The warps of a CTA take groups of 16 of its pages in turn, a
// group's bytes a turn ahead.  KPT > 0 (one token a sequence, lists of up to KPT pages a
// thread): the last CTA of a list makes its choice.
template <int D, int KPT>
__global__ void __launch_bounds__(kScoreWarps * 32) score_kernel(const SelectArgs a, int tg, int parts)
{
    constexpr int KS = D / 16, CH = D / 64;
    __shared__ uint2 s_q[kScoreCols / 8][KS][32];         // coded queries in fragment order
    __shared__ float s_dq[kScoreCols];
    __shared__ int s_nb[kScoreCols];
    __shared__ float s_f[kScoreWarps][16][kScoreCols + 1];
    start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int kh = blockIdx.y, s = blockIdx.z;
    const int64_t len = list_len(a.L, s);
    if (blockIdx.x == 0 && kh == 0 && tid == 0 && len < max(0, __ldg(a.L.kv_len + s))) atomicOr(a.L.status, kStatusList);
    const int64_t nb = (len + kPage - 1) / kPage;
    const int piece = blockIdx.x / parts, part = blockIdx.x - piece * parts;
    const int64_t groups = (nb + 15) / 16, stride = static_cast<int64_t>(gridDim.x / parts) * kScoreWarps;
    const int64_t group0 = static_cast<int64_t>(piece) * kScoreWarps + warp;
    if (static_cast<int64_t>(piece) * kScoreWarps >= groups && (KPT == 0 || piece > 0)) return;
    const int32_t *ids = a.L.ids + (static_cast<int64_t>(s) * a.L.Hk + kh) * a.L.cap;

    // tokens in rounds whose columns fit; a token of more query heads than that
    // takes several rounds
    const int hg = min(a.G, kScoreCols);                  // heads a round
    for (int t0 = part * tg; t0 < a.nq; t0 += parts * tg) {
        const int nt = min(tg, a.nq - t0);
        for (int h0 = 0; h0 < a.G; h0 += hg) {
            const int nh = min(hg, a.G - h0);
            const int cols = nt * nh, ncg = (cols + 7) / 8;
            Extremes<D> nxt;
            nxt.ids_of(a, ids, group0 * 16, group0 < groups ? nb : 0, g);
            __syncthreads();                              // the last round's columns are read
            // coded queries: a warp takes up to eight columns, their values requested together
            constexpr int N = D / 32, CPW = kScoreCols / kScoreWarps;
            uint2 raw[CPW];
#pragma unroll
            for (int e = 0; e < CPW; ++e) {
                const int c = warp + e * kScoreWarps;
                raw[e] = make_uint2(0, 0);
                if (c < cols) {
                    const int tok = t0 + c / nh, head = kh * a.G + h0 + c % nh;
                    const __half *qp = a.q + (a.token(s, tok) * a.H + head) * D + lane * N;
                    if constexpr (N == 4) raw[e] = __ldg(reinterpret_cast<const uint2 *>(qp));
                    else raw[e].x = __ldg(reinterpret_cast<const uint32_t *>(qp));
                }
            }
            if (tid < nt) {
                // pages that hold a key the token sees
                int64_t seen = len;
                if (a.q_pos)
                    seen = max(int64_t(0), min(len, static_cast<int64_t>(__ldg(a.q_pos + a.token(s, t0 + tid))) + 1));
                s_nb[tid] = static_cast<int>((seen + kPage - 1) / kPage);
            }
#pragma unroll
            for (int e = 0; e < CPW; ++e) {
                const int c = warp + e * kScoreWarps;
                if (c >= ncg * 8) break;
                float v[N];
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const uint32_t w = i == 0 ? raw[e].x : raw[e].y;
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                    v[i] = f.x;
                    v[i + 1] = f.y;
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float m = fabsf(v[i]);
                    top = fmaxf(top, m <= 65504.f ? m : 0.f);
                }
                // (magnitudes: their order is that of their bits)
                top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
                const float dq = over_127(top);
                if (lane == 0) s_dq[c] = dq;
                // the integer nearest v / dq: by the approximate reciprocal unless that
                // comes within 2^-13 of a half-integer (its error is below 2^-14)
                float rd;
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rd) : "f"(dq));
                bool sure = dq > 0.f;
                float r[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float x = v[i] * rd;
                    r[i] = rintf(x);
                    sure = sure && fabsf(x - r[i]) < 0.5f - 0x1p-13f;
                }
                if (!sure) {
#pragma unroll
                    for (int i = 0; i < N; ++i) r[i] = dq > 0.f ? static_cast<float>(nearest_code(v[i], dq)) : 0.f;
                }
                __half hc[N];
#pragma unroll
                for (int i = 0; i < N; ++i) hc[i] = __float2half_rn(r[i]);
                // channel d of column c: chunk d/64, t = d/16 % 4, word d/4 % 4, place d % 4
                const int d = lane * N;
                __half *dst = reinterpret_cast<__half *>(&s_q[c >> 3][(d >> 6) * 4 + ((d >> 2) & 3)][(c & 7) * 4 + ((d >> 4) & 3)]) + (d & 3);
#pragma unroll
                for (int i = 0; i < N; ++i) dst[i] = hc[i];
            }
            nxt.load(a, t);
            __syncthreads();
            for (int64_t gr = group0; gr < groups; gr += stride) {
                Extremes<D> cur = nxt;
                // lane l finishes page l % 16
                const int id0 = __shfl_sync(0xffffffffu, cur.id[0], (lane & 7) * 4);
                const int id1 = __shfl_sync(0xffffffffu, cur.id[1], (lane & 7) * 4);
                const float ks0 = __shfl_sync(0xffffffffu, cur.scale[0], (lane & 7) * 4);
                const float ks1 = __shfl_sync(0xffffffffu, cur.scale[1], (lane & 7) * 4);
                const int page_id = (lane & 8) ? id1 : id0;
                const float page_scale = (lane & 8) ? ks1 : ks0;
                if (__any_sync(0xffffffffu, page_scale < 0.f)) cur.turn();
                if (gr + stride < groups) {
                    nxt.ids_of(a, ids, (gr + stride) * 16, nb, g);
                    nxt.load(a, t);
                }
                float acc[kScoreCols / 8][4];
#pragma unroll
                for (int j = 0; j < kScoreCols / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint4 &lo = cur.x[part][0][c], &hi = cur.x[part][1][c];
                            const uint32_t x = (w == 0 ? lo.x : w == 1 ? lo.y : w == 2 ? lo.z : lo.w) ^ 0x80808080u;
                            const uint32_t y = (w == 0 ? hi.x : w == 1 ? hi.y : w == 2 ? hi.z : hi.w) ^ 0x80808080u;
                            const uint32_t a0 = codes_lo(x), a1 = codes_lo(y), a2 = codes_hi(x), a3 = codes_hi(y);
                            const __half2 z = __half2half2(__ushort_as_half(0));
#pragma unroll
                            for (int j = 0; j < kScoreCols / 8; ++j) {
                                if (j >= ncg) break;
                                uint2 q = s_q[j][c * 4 + w][lane];
                                __half2 q0 = *reinterpret_cast<__half2 *>(&q.x), q1 = *reinterpret_cast<__half2 *>(&q.y);
                                q0 = part == 0 ? __hmax2(q0, z) : __hmin2(q0, z);
                                q1 = part == 0 ? __hmax2(q1, z) : __hmin2(q1, z);
                                mma_16816(acc[j], a0, a1, a2, a3, *reinterpret_cast<uint32_t *>(&q0),
                                          *reinterpret_cast<uint32_t *>(&q1));
                            }
                        }
#pragma unroll
                for (int j = 0; j < kScoreCols / 8; ++j) {
                    if (j >= ncg) break;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = j * 8 + 2 * t + (e & 1);
                        s_f[warp][g + 8 * (e >> 1)][c] = __fmul_rn(acc[j][e], cur.scale[e >> 1] < 0.f ? -s_dq[c] : s_dq[c]);
                    }
                }
                __syncwarp();
                // (page, token): the largest of its heads
                for (int x = lane; x < 16 * nt; x += 32) {
                    const int b = x & 15, tok = x >> 4;   // b = lane & 15: the lane's own page
                    float m = -INFINITY;
                    for (int i = 0; i < nh; ++i) m = fmaxf(m, s_f[warp][b][tok * nh + i]);
                    const int64_t blk = gr * 16 + b;
                    if (blk >= nb) continue;
                    const int64_t row = (static_cast<int64_t>(s) * a.nq + t0 + tok) * a.L.Hk + kh;
                    uint32_t *out = a.keys + row * a.L.cap + blk;
                    const int nbq = s_nb[tok];
                    uint32_t key = kNever;
                    if (page_id >= 0 && blk < nbq) {
                        key = blk < a.n_first || blk >= nbq - a.n_last ? kAlways : order_key(__fmul_rn(m, fabsf(page_scale)));
                        if (h0 > 0) key = max(key, *out);
                    }
                    *out = key;
                }
                __syncwarp();
            }
        }
    }
    if constexpr (KPT > 0) {
        constexpr int kThreads = kScoreWarps * 32;
        static_assert(sizeof(PickScratch<kThreads>) <= sizeof(s_f), "in the place of the scores");
        const int list = s * a.L.Hk + kh;
        const int pieces = static_cast<int>(max(int64_t(1), min(static_cast<int64_t>(gridDim.x), (groups + kScoreWarps - 1) / kScoreWarps)));
        __threadfence();
        __syncthreads();
        if (!__syncthreads_or(tid == 0 && atomicAdd(a.counters + list, 1) == pieces - 1)) return;
        if (tid == 0) a.counters[list] = 0;
        __threadfence();
        pick_row<kThreads, KPT>(a.keys + static_cast<int64_t>(list) * a.L.cap, s_nb[0], a.n_sel,
                                a.sel + (a.token(s, 0) * a.L.Hk + kh) * a.n_sel,
                                *reinterpret_cast<PickScratch<kThreads> *>(&s_f));
    }
}

int launch_select(skv_handle *h, const SelectArgs &a, int D, cudaStream_t st)
{
    // Two CTAs a SM in all, no more than groups of 16 pages for their warps.  Where those
    // are fewer, the tokens are dealt to several CTAs (two sequences of 16 tokens over
    // 512 pages, 32 heads: 63 us with the attention over the picked pages, against 69).
    const int64_t lists = static_cast<int64_t>(a.L.S) * a.L.Hk;
    const int64_t most = (a.L.cap + kScoreWarps * 16 - 1) / (kScoreWarps * 16);
    const int64_t want = std::max<int64_t>(1, (2 * h->sm_count + lists - 1) / lists);
    const int64_t pieces = std::min(most, want);
    int tg = std::min(a.nq, std::max(1, kScoreCols / a.G));
    const int64_t deal = std::min<int64_t>(a.nq, std::max<int64_t>(1, 2 * h->sm_count / (lists * pieces)));
    tg = std::min(tg, static_cast<int>((a.nq + deal - 1) / deal));
    const int parts = static_cast<int>(std::min<int64_t>(deal, (a.nq + tg - 1) / tg));
    const dim3 grid(static_cast<unsigned>(pieces * parts), a.L.Hk, a.L.S);
    // One token a sequence and short lists: the choice by the last CTA of a list's scores.
    // As fast on the GPU (16 of 128 pages, with the attention: 18.6 against 18.4 us), and
    // one launch less on the host (25 against 30 us a step on one box; 27 to 38 us as fused
    // over several).  By one CTA of 256 threads
    // longer lists take longer (512 of 4096 pages: 67 us with the attention, 52 by a kernel of 512 threads).
    constexpr int kFused = 4;
    const bool fused = a.nq == 1 && a.L.cap <= kFused * kScoreWarps * 32 && lists <= kMaxUnits;
    const auto kernel = D == 128 ? (fused ? score_kernel<128, kFused> : score_kernel<128, 0>)
                                 : (fused ? score_kernel<64, kFused> : score_kernel<64, 0>);
    cudaError_t e = launch(kernel, grid, kScoreWarps * 32, 0, st, a, tg, parts);
    if (e != cudaSuccess) return cuda_fail(h, e, "page score launch");
    if (fused) return SKV_OK;
    const dim3 rows(static_cast<unsigned>(static_cast<int64_t>(a.L.S) * a.nq * a.L.Hk));
    e = for_cap(a.L.cap, [&](auto threads, auto kpt) {
        return launch(pick_kernel<threads.value, kpt.value>, rows, threads.value, 0, st, a);
    });
    return cuda_fail(h, e, "page choice launch");
}

// ------------------------------------------------------------------ eviction

// One CTA a list.  With KPT = 0 the keys lie in the list's part of mass_out, which is
// written last.
template <int THREADS, int KPT>
__global__ void __launch_bounds__(THREADS) evict_kernel(const Lists L, const float *mass, int n_keep, int n_first,
                                                       int n_last, int32_t *ids_out, float *mass_out,
                                                       int32_t *kv_len_out, int32_t *freed_out)
{
    start();
    __shared__ PickScratch<THREADS> sc;
    const int kh = blockIdx.x, s = blockIdx.y;
    const int64_t list = static_cast<int64_t>(s) * L.Hk + kh;
    const int64_t len = list_len(L, s);
    const int cap = static_cast<int>(L.cap);
    const int n = static_cast<int>((len + kPage - 1) / kPage);
    const int32_t *ids = L.ids + list * L.cap;
    const float *m = mass + list * L.cap;
    int32_t *oi = ids_out + list * L.cap;
    float *om = mass_out + list * L.cap;
    int32_t *of = freed_out + list * L.cap;
    const int out_n = max(0, n - n_keep);                 // pages taken out
    if (kh == 0 && threadIdx.x == 0) {
        if (len < max(0, L.kv_len[s])) atomicOr(L.status, kStatusList);
        kv_len_out[s] = static_cast<int32_t>(len - static_cast<int64_t>(out_n) * kPage);
    }
    if (out_n == 0) {
        for (int i = threadIdx.x; i < cap; i += THREADS) {
            oi[i] = ids[i];
            om[i] = i < n ? m[i] : 0.f;
            of[i] = -1;
        }
        return;
    }
    // an absent page ranks below every weight, the kept ends above
    auto key_of = [&](int i) {
        const int id = __ldg(ids + i);
        const float x = __ldg(m + i);
        return i < n_first || i >= n - n_last ? kAlways : id < 0 ? kNever : order_key(x);
    };
    uint32_t *in_om = reinterpret_cast<uint32_t *>(om);
    Keys<THREADS, KPT> keys(n, in_om);
    if constexpr (KPT > 0) {
        keys.fill(key_of);
    } else {
        for (int i = threadIdx.x; i < n; i += THREADS) in_om[i] = key_of(i);
        __syncthreads();
    }
    // what lies behind the last token follows the kept pages
    for (int i = n + threadIdx.x; i < cap; i += THREADS) oi[i - out_n] = ids[i];
    for (int i = cap - out_n + threadIdx.x; i < cap; i += THREADS) oi[i] = -1;
    const uint32_t T = threshold(keys, n_keep, sc);
    // (T can be kNever: absent pages are then kept for want of others, and none is freed)
    int need = 0, freed = 0;
    in_order(
        keys, T, sc,
        [&](int above, int, int nevers) {
            need = n_keep - above;
            freed = T == kNever ? 0 : out_n - nevers;
        },
        [&](int i, uint32_t k, int above, int ties, int nevers) {
            const int at = above + min(ties, need);       // kept pages before i
            if (k > T || (k == T && ties < need)) {
                oi[at] = __ldg(ids + i);
                if constexpr (KPT > 0) om[at] = __ldg(m + i);
            } else if (k != kNever) {
                of[i - at - nevers] = __ldg(ids + i);     // taken out before i, absent ones apart
            }
        });
    for (int i = freed + threadIdx.x; i < cap; i += THREADS) of[i] = -1;
    if constexpr (KPT == 0) {
        // a kept page's weight moves to a lower place, whose key has been used by
        // then, one run of THREADS indices at a time
        __syncthreads();
        constexpr int W = THREADS / 32;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int above = 0, ties = 0;
        for (int b = 0; b < n; b += THREADS) {
            const int i = b + static_cast<int>(threadIdx.x);
            const uint32_t k = i < n ? in_om[i] : 0u;
            const unsigned m0 = __ballot_sync(0xffffffffu, i < n && k > T), m1 = __ballot_sync(0xffffffffu, i < n && k == T);
            __syncthreads();
            if (lane == 0) {
                sc.n[0][warp] = __popc(m0);
                sc.n[1][warp] = __popc(m1);
            }
            __syncthreads();
            const int x0 = lane < W ? sc.n[0][lane] : 0, x1 = lane < W ? sc.n[1][lane] : 0;
            const unsigned before = (1u << lane) - 1u;
            const int a0 = above + __reduce_add_sync(0xffffffffu, lane < warp ? x0 : 0) + __popc(m0 & before);
            const int a1 = ties + __reduce_add_sync(0xffffffffu, lane < warp ? x1 : 0) + __popc(m1 & before);
            above += __reduce_add_sync(0xffffffffu, x0);
            ties += __reduce_add_sync(0xffffffffu, x1);
            if (i < n && (k > T || (k == T && a1 < need))) om[a0 + min(a1, need)] = m[i];
            __syncthreads();
        }
    }
    for (int i = n_keep + threadIdx.x; i < cap; i += THREADS) om[i] = 0.f;
}

int launch_evict(skv_handle *h, const Lists &L, const float *mass, int n_keep, int n_first, int n_last,
                 int32_t *ids_out, float *mass_out, int32_t *kv_len_out, int32_t *freed_out, cudaStream_t st)
{
    const cudaError_t e = for_cap(L.cap, [&](auto threads, auto kpt) {
        return launch(evict_kernel<threads.value, kpt.value>, dim3(L.Hk, L.S), threads.value, 0, st, L, mass, n_keep, n_first,
                      n_last, ids_out, mass_out, kv_len_out, freed_out);
    });
    return cuda_fail(h, e, "eviction launch");
}

}  // namespace q8
}  // namespace skv
