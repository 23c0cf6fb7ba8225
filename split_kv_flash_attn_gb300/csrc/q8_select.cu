// q8_select.cu -- picking pages: bounds of the pages' scores for each query,
// the choice of the best n, and the same choice by accumulated weight for
// eviction.
//
// The bound.  A page keeps the smallest and largest K code of each channel,
// so sum_d max(cq_d min_d, cq_d max_d) bounds the product of the coded query with
// every key of the page.  It is cq+ . max + cq- . min, the positive and the
// negative part of the query against the two extremes: one product of length
// 2D of whole numbers of at most 127, whose sums stay below 2^21, so the tensor
// cores' fp32 sums are exact and the picks do not depend on the order of
// anything.  A warp takes 16 pages (the M side; bytes straight from global
// memory into fragments, as in the decode kernel) against the queries of a KV
// head, 8 columns at a time.
//
// The choice.  Scores become 32-bit keys whose order as unsigned numbers is the scores'
// order; one CTA for each list finds the n-th largest key two bits at a time,
// counting keys in shared memory, and writes the picked indices in order by
// prefix sums over the warps' equal shares.  Ties at the n-th key go to the lowest indices.
//
// Bound: 2D + 8 bytes a page and head for the scores; the choice is latency
// (about 15 counting rounds, each one pass over shared memory and one barrier).
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

constexpr int kScoreWarps = 4;
constexpr int kScoreCols = 64;                // query columns in shared memory at a time

template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) score_kernel(const SelectArgs a)
{
    constexpr int KS = D / 16, CH = D / 64;
    __shared__ uint2 s_q[kScoreCols / 8][KS][32];         // coded queries in fragment order
    __shared__ float s_dq[kScoreCols];
    __shared__ float s_f[kScoreWarps][16][kScoreCols + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int kh = blockIdx.y, s = blockIdx.z;
    const int64_t len = list_len(a.L, s);
    const int64_t nb = (len + kPage - 1) / kPage;
    const int64_t b0 = (static_cast<int64_t>(blockIdx.x) * kScoreWarps) * 16;      // the CTA's first page
    if (b0 >= nb) return;
    const int64_t bw = b0 + warp * 16;                                             // the warp's
    const int32_t *ids = a.L.ids + (static_cast<int64_t>(s) * a.L.Hk + kh) * a.L.cap;

    // rows g, g + 8 of the warp's 16 pages: [largest | smallest] codes
    int id[2];
    uint4 kr[2][2][CH];
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
        const int64_t b = bw + g + 8 * rr;
        id[rr] = b < nb ? checked_page(a.L, __ldg(ids + b)) : -1;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int64_t off = static_cast<int64_t>(max(id[rr], 0)) * D + 64 * c + 16 * t;
            kr[0][rr][c] = id[rr] >= 0 ? ld_stream16(a.k_max + off) : make_uint4(0, 0, 0, 0);
            kr[1][rr][c] = id[rr] >= 0 ? ld_stream16(a.k_min + off) : make_uint4(0, 0, 0, 0);
        }
    }
    // lane l finishes page l % 16
    const int id0 = __shfl_sync(0xffffffffu, id[0], (lane & 7) * 4);
    const int id1 = __shfl_sync(0xffffffffu, id[1], (lane & 7) * 4);
    const int page_id = (lane & 8) ? id1 : id0;
    const float page_scale = page_id >= 0 ? __ldg(a.k_scale + page_id) : 0.f;

    // tokens in groups whose columns fit; a token of more query heads than that
    // takes several rounds
    const int tg = max(1, kScoreCols / a.G);              // tokens a round
    const int hg = min(a.G, kScoreCols);                  // heads a round
    for (int t0 = 0; t0 < a.nq; t0 += tg) {
        const int nt = min(tg, a.nq - t0);
        for (int h0 = 0; h0 < a.G; h0 += hg) {
            const int nh = min(hg, a.G - h0);
            const int cols = nt * nh;
            __syncthreads();
            // coded queries: one warp a column
            for (int c = warp; c < (cols + 7) / 8 * 8; c += kScoreWarps) {
                float v[D / 32];
                float top = 0.f;
                const int tok = t0 + c / nh, head = kh * a.G + h0 + c % nh;
                const __half *qp = a.q + ((static_cast<int64_t>(s) * a.nq + tok) * a.H + head) * D + lane * (D / 32);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    v[i] = c < cols ? __half2float(qp[i]) : 0.f;
                    const float m = fabsf(v[i]);
                    top = fmaxf(top, m <= 65504.f ? m : 0.f);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float dq = __fdiv_rn(top, 127.f);
                if (lane == 0) s_dq[c] = dq;
                __half hc[4];
#pragma unroll
                for (int i = 0; i < D / 32; ++i) hc[i] = __int2half_rn(dq > 0.f ? nearest_code(v[i], dq) : 0);
                // channel d of column c: chunk d/64, t = d/16 % 4, word d/4 % 4, place d % 4
                const int d = lane * (D / 32);
                __half *dst = reinterpret_cast<__half *>(&s_q[c >> 3][(d >> 6) * 4 + ((d >> 2) & 3)][(c & 7) * 4 + ((d >> 4) & 3)]) + (d & 3);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) dst[i] = hc[i];
            }
            __syncthreads();
            if (bw < nb) {
                for (int j = 0; j < (cols + 7) / 8; ++j) {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int c = 0; c < CH; ++c)
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                const uint4 &lo = kr[part][0][c], &hi = kr[part][1][c];
                                const uint32_t x = (w == 0 ? lo.x : w == 1 ? lo.y : w == 2 ? lo.z : lo.w) ^ 0x80808080u;
                                const uint32_t y = (w == 0 ? hi.x : w == 1 ? hi.y : w == 2 ? hi.z : hi.w) ^ 0x80808080u;
                                uint2 q = s_q[j][c * 4 + w][lane];
                                const __half2 z = __half2half2(__ushort_as_half(0));
                                __half2 q0 = *reinterpret_cast<__half2 *>(&q.x), q1 = *reinterpret_cast<__half2 *>(&q.y);
                                q0 = part == 0 ? __hmax2(q0, z) : __hmin2(q0, z);
                                q1 = part == 0 ? __hmax2(q1, z) : __hmin2(q1, z);
                                mma_16816(acc, codes_lo(x), codes_lo(y), codes_hi(x), codes_hi(y),
                                          *reinterpret_cast<uint32_t *>(&q0), *reinterpret_cast<uint32_t *>(&q1));
                            }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = j * 8 + 2 * t + (e & 1);
                        s_f[warp][g + 8 * (e >> 1)][c] = __fmul_rn(acc[e], s_dq[c]);
                    }
                }
                __syncwarp();
                // (page, token): the largest of its heads
                for (int x = lane; x < 16 * nt; x += 32) {
                    const int b = x & 15, tok = x >> 4;   // b = lane & 15: the lane's own page
                    float m = -INFINITY;
                    for (int i = 0; i < nh; ++i) m = fmaxf(m, s_f[warp][b][tok * nh + i]);
                    const int64_t blk = bw + b;
                    if (blk >= nb) continue;
                    const int64_t row = (static_cast<int64_t>(s) * a.nq + t0 + tok) * a.L.Hk + kh;
                    uint32_t *out = a.keys + row * a.L.cap + blk;
                    int64_t seen = len;
                    if (a.q_pos) seen = max(int64_t(0), min(len, static_cast<int64_t>(a.q_pos[static_cast<int64_t>(s) * a.nq + t0 + tok]) + 1));
                    const int64_t nbq = (seen + kPage - 1) / kPage;
                    uint32_t key = kNever;
                    if (page_id >= 0 && blk < nbq) {
                        key = blk < a.n_first || blk >= nbq - a.n_last ? kAlways : order_key(__fmul_rn(m, page_scale));
                        if (h0 > 0) key = page_scale >= 0.f ? max(key, *out) : min(key, *out);
                    }
                    *out = key;
                }
                __syncwarp();
            }
        }
    }
}

// ---------------------------------------------------------------- the choice

constexpr int kPickThreads = 1024;
constexpr int kPickWarps = kPickThreads / 32;

struct PickScratch {
    int cnt[2][kPickWarps][3];
    uint32_t lo[kPickWarps], hi[kPickWarps];
    int warp_n[kPickWarps];
    int warp_m[kPickWarps];
};

// The k-th largest of keys[0, n) (n >= k >= 1).
__device__ uint32_t kth_largest(const uint32_t *keys, int n, int k, PickScratch &sc)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // bits that all keys share need no rounds
    uint32_t both = 0xffffffffu, any = 0u;
    for (int i = tid; i < n; i += kPickThreads) {
        const uint32_t x = keys[i];
        both &= x;
        any |= x;
    }
    both = __reduce_and_sync(0xffffffffu, both);
    any = __reduce_or_sync(0xffffffffu, any);
    if (lane == 0) {
        sc.lo[warp] = both;
        sc.hi[warp] = any;
    }
    __syncthreads();
    both = __reduce_and_sync(0xffffffffu, sc.lo[lane]);
    any = __reduce_or_sync(0xffffffffu, sc.hi[lane]);
    const uint32_t diff = both ^ any;
    uint32_t found = both;
    if (diff) {
        const int top = 31 - __clz(diff);                 // highest bit in which keys differ
        found = top == 31 ? 0u : both & ~((2u << top) - 1u);
        int round = 0;
        for (int b = top & ~1; b >= 0; b -= 2, round ^= 1) {
            // how many keys reach found + 1, 2, 3 units of 2^b
            const uint32_t t1 = found | (1u << b), t2 = found | (2u << b), t3 = found | (3u << b);
            int c1 = 0, c2 = 0, c3 = 0;
            for (int i = tid; i < n; i += kPickThreads) {
                const uint32_t x = keys[i];
                c1 += x >= t1;
                c2 += x >= t2;
                c3 += x >= t3;
            }
            c1 = __reduce_add_sync(0xffffffffu, c1);
            c2 = __reduce_add_sync(0xffffffffu, c2);
            c3 = __reduce_add_sync(0xffffffffu, c3);
            if (lane == 0) {
                sc.cnt[round][warp][0] = c1;
                sc.cnt[round][warp][1] = c2;
                sc.cnt[round][warp][2] = c3;
            }
            __syncthreads();
            c1 = __reduce_add_sync(0xffffffffu, sc.cnt[round][lane][0]);
            c2 = __reduce_add_sync(0xffffffffu, sc.cnt[round][lane][1]);
            c3 = __reduce_add_sync(0xffffffffu, sc.cnt[round][lane][2]);
            found = c3 >= k ? t3 : c2 >= k ? t2 : c1 >= k ? t1 : found;
        }
    }
    return found;
}

// Calls emit(i, rank) for the i in [0, n) for which pred(i) holds, rank counting
// them from 0 in the order of i.  Each warp takes an equal run of indices.
template <typename P, typename E>
__device__ int ordered(int n, int *warp_n, P pred, E emit)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int share = (n + kPickThreads - 1) / kPickThreads * 32;
    const int lo = min(n, warp * share), hi = min(n, lo + share);
    int c = 0;
    for (int i = lo; i < hi; i += 32) c += __popc(__ballot_sync(0xffffffffu, i + lane < hi && pred(i + lane)));
    __syncthreads();                                      // warp_n of an earlier call is read
    if (lane == 0) warp_n[warp] = c;
    __syncthreads();
    const int x = warp_n[lane];
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    const int all = __shfl_sync(0xffffffffu, inc, 31);
    int at = __shfl_sync(0xffffffffu, inc - x, warp);
    for (int i = lo; i < hi; i += 32) {
        const bool on = i + lane < hi && pred(i + lane);
        const unsigned m = __ballot_sync(0xffffffffu, on);
        if (on) emit(i + lane, at + __popc(m & ((1u << lane) - 1u)));
        at += __popc(m);
    }
    return all;
}

constexpr int kPickSmemKeys = 48 * 1024;                  // 192 KB of keys

// One CTA a row (sequence, token, KV head).
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const SelectArgs a, bool in_smem)
{
    extern __shared__ uint32_t s_keys[];
    __shared__ PickScratch sc;
    const int64_t row = blockIdx.x;
    const int64_t tok = row / a.L.Hk;
    const int s = static_cast<int>(tok / a.nq);
    int64_t seen = list_len(a.L, s);
    if (a.q_pos) seen = max(int64_t(0), min(seen, static_cast<int64_t>(a.q_pos[tok]) + 1));
    const int n = static_cast<int>((seen + kPage - 1) / kPage);
    const uint32_t *keys = a.keys + row * a.L.cap;
    int32_t *out = a.sel + row * a.n_sel;
    if (in_smem) {
        for (int i = threadIdx.x; i < n; i += kPickThreads) s_keys[i] = __ldcg(keys + i);
        __syncthreads();
        keys = s_keys;
    }
    // no more candidates than places: all of them
    uint32_t T = kNever;
    int need = 0;                                         // of the keys equal to T
    if (n > a.n_sel) {
        T = kth_largest(keys, n, a.n_sel, sc);
        __syncthreads();
        const int above = ordered(n, sc.warp_n, [&](int i) { return keys[i] > T; }, [](int, int) {});
        need = T == kNever ? 0 : a.n_sel - above;
    }
    // keys above T, and the first `need` of those equal to it.  A key's place is
    // the number of picked ones before it: those above plus at most `need` ties.
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int share = (n + kPickThreads - 1) / kPickThreads * 32;
    const int lo = min(n, warp * share), hi = min(n, lo + share);
    int ca = 0, ce = 0;
    for (int i = lo; i < hi; i += 32) {
        const uint32_t k = i + lane < hi ? keys[i + lane] : kNever;
        ca += __popc(__ballot_sync(0xffffffffu, k > T));
        ce += __popc(__ballot_sync(0xffffffffu, i + lane < hi && k == T && need > 0));
    }
    __syncthreads();
    if (lane == 0) {
        sc.warp_n[warp] = ca;
        sc.warp_m[warp] = ce;
    }
    __syncthreads();
    int ia = sc.warp_n[lane], ie = sc.warp_m[lane];
    const int xa = ia, xe = ie;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, ia, o), z = __shfl_up_sync(0xffffffffu, ie, o);
        if (lane >= o) {
            ia += y;
            ie += z;
        }
    }
    const int total = __shfl_sync(0xffffffffu, ia, 31) + min(need, __shfl_sync(0xffffffffu, ie, 31));
    int at_a = __shfl_sync(0xffffffffu, ia - xa, warp), at_e = __shfl_sync(0xffffffffu, ie - xe, warp);
    for (int i = lo; i < hi; i += 32) {
        const uint32_t k = i + lane < hi ? keys[i + lane] : kNever;
        const bool above = k > T, tie = i + lane < hi && k == T && need > 0;
        const unsigned ma = __ballot_sync(0xffffffffu, above), me = __ballot_sync(0xffffffffu, tie);
        const unsigned before = (1u << lane) - 1u;
        const int ra = at_a + __popc(ma & before), re = at_e + __popc(me & before);
        if (above || (tie && re < need)) out[ra + min(re, need)] = i + lane;
        at_a += __popc(ma);
        at_e += __popc(me);
    }
    for (int i = total + threadIdx.x; i < a.n_sel; i += kPickThreads) out[i] = -1;
}

int launch_select(skv_handle *h, const SelectArgs &a, int D, cudaStream_t st)
{
    const dim3 grid(static_cast<unsigned>((a.L.cap + kScoreWarps * 16 - 1) / (kScoreWarps * 16)), a.L.Hk, a.L.S);
    if (D == 128) score_kernel<128><<<grid, kScoreWarps * 32, 0, st>>>(a);
    else score_kernel<64><<<grid, kScoreWarps * 32, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(h, e, "page score launch");
    static KernelAttrCache cache;
    const bool in_smem = a.L.cap <= kPickSmemKeys;
    const int smem = in_smem ? static_cast<int>(a.L.cap) * 4 : 0;
    if (smem > 32 * 1024) {
        e = kernel_smem_optin(cache, reinterpret_cast<const void *>(pick_kernel), smem, kPickThreads, nullptr);
        if (e != cudaSuccess) return cuda_fail(h, e, "cudaFuncSetAttribute(page choice)");
    }
    pick_kernel<<<static_cast<unsigned>(static_cast<int64_t>(a.L.S) * a.nq * a.L.Hk), kPickThreads, smem, st>>>(a, in_smem);
    return cuda_fail(h, cudaGetLastError(), "page choice launch");
}

// ------------------------------------------------------------------ eviction

// One CTA a list.  `keys` is shared memory, or the list's part of mass_out, which
// is written last and holds its keys until then.
__global__ void __launch_bounds__(kPickThreads) evict_kernel(const Lists L, const float *mass, int n_keep, int n_first,
                                                            int n_last, int32_t *ids_out, float *mass_out,
                                                            int32_t *kv_len_out, int32_t *freed_out, bool in_smem)
{
    extern __shared__ uint32_t s_keys[];
    __shared__ PickScratch sc;
    const int kh = blockIdx.x, s = blockIdx.y;
    const int64_t list = static_cast<int64_t>(s) * L.Hk + kh;
    const int64_t len = list_len(L, s);
    if (kh == 0 && threadIdx.x == 0 && len < max(0, L.kv_len[s])) atomicOr(L.status, kStatusList);
    const int cap = static_cast<int>(L.cap);
    const int n = static_cast<int>((len + kPage - 1) / kPage);
    const int32_t *ids = L.ids + list * L.cap;
    const float *m = mass + list * L.cap;
    int32_t *oi = ids_out + list * L.cap;
    float *om = mass_out + list * L.cap;
    int32_t *of = freed_out + list * L.cap;
    const int out_n = max(0, n - n_keep);                 // pages taken out
    if (kh == 0 && threadIdx.x == 0) kv_len_out[s] = static_cast<int32_t>(len - static_cast<int64_t>(out_n) * kPage);
    if (out_n == 0) {
        for (int i = threadIdx.x; i < cap; i += kPickThreads) {
            oi[i] = ids[i];
            om[i] = i < n ? m[i] : 0.f;
            of[i] = -1;
        }
        return;
    }
    // an absent page ranks below every weight, the kept ends above
    uint32_t *keys = in_smem ? s_keys : reinterpret_cast<uint32_t *>(om);
    for (int i = threadIdx.x; i < n; i += kPickThreads)
        keys[i] = i < n_first || i >= n - n_last ? kAlways : ids[i] < 0 ? kNever : order_key(m[i]);
    __syncthreads();
    const uint32_t T = kth_largest(keys, n, n_keep, sc);
    __syncthreads();
    const int above = ordered(n, sc.warp_n, [&](int i) { return keys[i] > T; }, [](int, int) {});
    const int need = n_keep - above;
    // ties beyond the first `need` go: marked by key 0, the others by T + 1.  (T
    // can be kNever: absent pages are then kept for want of others, lowest index first.)
    const int ties = ordered(n, sc.warp_n, [&](int i) { return keys[i] == T; },
                             [&](int i, int rank) { of[rank] = i; });
    __syncthreads();
    for (int r = threadIdx.x; r < ties; r += kPickThreads) keys[of[r]] = r < need ? 0xffffffffu : 0u;
    __syncthreads();
    auto kept = [&](int i) { return keys[i] > T; };
    ordered(n, sc.warp_n, kept, [&](int i, int rank) { oi[rank] = ids[i]; });
    const int freed = ordered(n, sc.warp_n, [&](int i) { return !kept(i) && ids[i] >= 0; },
                              [&](int i, int rank) { of[rank] = ids[i]; });
    for (int i = n + threadIdx.x; i < cap; i += kPickThreads) oi[i - out_n] = ids[i];
    for (int i = cap - out_n + threadIdx.x; i < cap; i += kPickThreads) oi[i] = -1;
    for (int i = freed + threadIdx.x; i < cap; i += kPickThreads) of[i] = -1;
    if (in_smem) {
        ordered(n, sc.warp_n, kept, [&](int i, int rank) { om[rank] = m[i]; });
    } else {
        // the keys lie in om: a kept page's weight moves to a lower place, whose key
        // has been used by then, one run of kPickThreads indices at a time
        int at = 0;
        for (int b = 0; b < n; b += kPickThreads) {
            const int i = b + static_cast<int>(threadIdx.x);
            const bool on = i < n && kept(i);
            const unsigned ball = __ballot_sync(0xffffffffu, on);
            __syncthreads();
            if ((threadIdx.x & 31) == 0) sc.warp_n[threadIdx.x >> 5] = __popc(ball);
            __syncthreads();
            int before = at, all = 0;
            for (int w = 0; w < kPickWarps; ++w) {
                if (w < static_cast<int>(threadIdx.x >> 5)) before += sc.warp_n[w];
                all += sc.warp_n[w];
            }
            if (on) om[before + __popc(ball & ((1u << (threadIdx.x & 31)) - 1u))] = m[i];
            at += all;
            __syncthreads();
        }
    }
    __syncthreads();
    for (int i = n_keep + threadIdx.x; i < cap; i += kPickThreads) om[i] = 0.f;
}

int launch_evict(skv_handle *h, const Lists &L, const float *mass, int n_keep, int n_first, int n_last,
                 int32_t *ids_out, float *mass_out, int32_t *kv_len_out, int32_t *freed_out, cudaStream_t st)
{
    static KernelAttrCache cache;
    const bool in_smem = L.cap <= kPickSmemKeys;
    const int smem = in_smem ? static_cast<int>(L.cap) * 4 : 0;
    if (smem > 32 * 1024) {
        const cudaError_t e = kernel_smem_optin(cache, reinterpret_cast<const void *>(evict_kernel), smem, kPickThreads, nullptr);
        if (e != cudaSuccess) return cuda_fail(h, e, "cudaFuncSetAttribute(eviction)");
    }
    evict_kernel<<<dim3(L.Hk, L.S), kPickThreads, smem, st>>>(L, mass, n_keep, n_first, n_last, ids_out, mass_out,
                                                             kv_len_out, freed_out, in_smem);
    return cuda_fail(h, cudaGetLastError(), "eviction launch");
}

}  // namespace q8
}  // namespace skv
