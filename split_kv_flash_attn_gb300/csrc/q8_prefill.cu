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
// results, as two (itself rounded, and what that left) for fp32 ones.  One is off by up to
// 2^-11 as the result's own rounding is, and both together by 1.4 times that rounding: 512 tokens over
// 32768 keys 2.9e-4 of the result in the 2-norm, with two parts 2.1e-4 (the rounding
// alone) at 291 us instead of 229.
//
// A CTA owns two 128-row query tiles of one KV head at a time (rows = tokens x
// the head's query heads), so each decoded tile serves both:
//   producers  : four warps, 32 key rows of every tile each; a row's 128 code
//                bytes lie 16 to a lane and are held in registers a tile ahead.
//   MMA warps  : one issues S_g(j) = Q_g K(j)^T for tile g = 0, 1 in turn, the
//                other O_g += W_g(j) V(j), W_g in the columns of S_g (one warp for
//                both was bound by its issue, 130 cycles a product).
//   softmax g  : four warps, one thread per query row, 64 keys (a page) at a time;
//                a half's weights are stored over its own consumed scores.
// While one tile's softmax runs, the tensor core works for the other.
//
// Bound: the chain of S, softmax and product through the tensor-memory columns that
// scores and weights share (512 tokens of 32 heads over 32768 keys, fp16: 229 us, 1190
// TFLOP/s; the tensor pipe is busy 62 % of the cycles); with few tiles a CTA, its start
// (about 8 us: plan, first queries, first tile) and the merge (8 to 10 us).
//
// Work split.  All key tiles of all (sequence, KV head, tile pair) units form one
// line (its prefix sums are taken from the lengths and query positions on the
// device, by a one-CTA kernel where they are many), cut into one piece for each CTA:
// equal ones, or slightly longer ones that end with their units.  Units that several
// pieces share are merged by a kernel of a warp a row, in piece order (by the last
// CTA of each unit that took 60 to 100 us).
//
// Tensor memory: S_0/W_0 in columns 0-127, S_1/W_1 128-255, O_0 256-383, O_1
// 384-511.  Every mbarrier wait is bounded; one that gives up sets the handle's
// device status word, the CTA drains what it issued and frees its tensor memory.
#include <algorithm>

#include "q8.cuh"

namespace skv {
namespace q8 {

constexpr int kPM = 128;                        // query rows of a tile
constexpr int kPN = 128;                        // keys of a tile
constexpr int kSoftWarps = 8;                   // warps 0-3: tile 0, warps 4-7: tile 1
constexpr int kProdWarps = 4;                   // warps 8-11
constexpr int kMmaWarp = kSoftWarps + kProdWarps;   // S; the next warp O; two more fill their warpgroup
constexpr int kPfThreads = (kMmaWarp + 4) * 32;
// Registers of a thread by role: 16 warps launch with 128 each, the softmax groups
// take what the others can spare (spilled, they would go to an L1 of 20 KB:
// such loads had been most of the waiting).
constexpr int kRegSoft = 176, kRegProd = 112, kRegMma = 48;
static_assert(2 * kRegSoft + kRegProd + kRegMma <= 4 * 128, "no more than the launch has");
static_assert(kRegSoft >= 128 && kRegProd <= 128 && kRegMma <= 128, "the first is an increase, the others decreases");
template <int N>
__device__ __forceinline__ void more_regs()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr uint32_t kPieceTiles = 3;                // fewest key tiles of a piece: each costs set-up and merge
constexpr int kStraddleTiles = 3;               // tiles that a second start and result of a CTA cost
constexpr int kPlanHere = 256;                  // plan entries that the prefill kernel counts itself
constexpr int kPlanSmem = 1024;                 // plan entries kept in shared memory
constexpr float kPfShift = 8.f, kPfGrow = 5.f, kPfScaleGrow = 2.f;
constexpr uint32_t kSpins = 1u << 20;           // polls of a barrier before a wait gives up (tens of ms at least)
// The tensor core rounds its sums toward zero, so O loses with every addition, in proportion
// to the tiles (rows of like weights over values of one sign 5e-7 a tile with both parts
// of the weights): fp32 results take about kExactTiles at a time, put together in fp32.
// What a stretch loses is given back by taking the row's sum of weights the same way:
// each product's 16 keys added to w_cut toward zero, once for the first parts and once more
// for the second (kLowPart of the first), and O multiplied by the true sum over it.
// Weights of zero then count for nothing (a fixed share for each tile made a row of one key
// 2.4e-6 too large).  Ten tiles of like weights, relative to the results: values of one sign
// 3.0e-6 too small without, 5e-7 off with it; of both signs 2.1e-6 and 1.2e-6; few keys
// that decide the row, values of one sign 6e-6 and 4e-6.  Time: 48.8 -> 49.5 us (64 tokens of
// eight ragged sequences of up to 4096 keys); stretches of at most seven tiles without
// it 61 us and 1.5e-6 to 4e-6, of five 73 us and 1.2e-6 to 3.2e-6.
constexpr int kExactTiles = 8, kExactMore = 2;    // (up to that many more rather than another stretch)
constexpr float kLowPart = 0x1p-12f;
// fp16 results (single weights, nothing given back) take more: values of one sign lose 1.6e-6
// of the whole sum a tile, which over lists of 1048576 keys in one stretch made results
// 6.7e-3 too small (262144 keys: 1.7e-3); at kLongTiles it is 9e-5, a fifth of half a
// step of fp16.  512 tokens of eight sequences over 65536 keys 3.25 -> 3.37 ms (64
// tiles: 3.50 ms, 4e-5); CTAs of fewer tiles, as for one sequence over 32768, as before.
constexpr int kLongTiles = 128;
constexpr float kNoScale = -100.f;              // log2 d_v - r of a zero scale (fp16 0, while l stays right)

template <int D>
struct PfSmem {
    static constexpr int kHalf = kPN * 128;     // 128 rows of 64 fp16
    static constexpr int kTile = D / 64 * kHalf;
    static constexpr int kQ = 0;                // two query tiles
    static constexpr int kK = kQ + 2 * kTile;   // two stages
    static constexpr int kV = kK + 2 * kTile;   // two stages
    static constexpr int kStage = kV + 2 * kTile;               // results on their way out: 32 rows of 16 for each softmax warp
    static constexpr int kStageLd = 20;                         // (floats a row: free of bank conflicts)
    static constexpr int kPlan = kStage + kSoftWarps * 32 * kStageLd * 4;
    static constexpr int kTiles = kPlan + (kPlanSmem + 2) * 4;          // tiles of each entry, where they are counted here
    static constexpr int kTotal = kTiles + kPlanHere * 4 + 1024;        // + alignment slack
};
static_assert(PfSmem<128>::kTotal <= 226 * 1024, "shared memory per CTA");

// Barriers (+ stage or query tile g).  Key tile j of the CTA is phase j / 2 of its
// K and V stages' barriers and j / 4 of its meta slot.  The t-th tile that query
// tile g takes part in (not every unit has a second one) is phase t of its S full,
// P half, P full and PV done, the u-th such unit phase u of its Q full.  No waiter is ever
// two phases behind: each side needs the other's next step before it can complete
// another phase, and the softmax groups enter every unit together, so that a
// meta slot is rewritten (four tiles on) only after both have read it.
enum { PB_KFULL = 0, PB_KEMPTY = 2, PB_VFULL = 4, PB_VEMPTY = 6, PB_QFULL = 8, PB_SFULL = 10, PB_PFULL = 12,
       PB_PDONE = 14, PB_META = 16, PB_PHALF = 20, PB_COUNT = 22 };

struct PrefillArgs {
    AttnArgs a;
    uint32_t *plan;                             // [S * n_pairs + 1] the line's length before each (sequence, pair) of one
                                                // head, then the tiles of a piece
    int n_pairs;
    int out_f16;
};

// Tiles of a CTA's piece.
__host__ __device__ inline uint32_t piece_tiles(uint32_t total, uint32_t ctas)
{
    const uint32_t c = (total + ctas - 1) / ctas;
    return c < kPieceTiles ? kPieceTiles : c;
}

// Key tiles of (sequence, pair of query tiles) e: up to its last visible key.  For
// a whole warp.
__device__ __forceinline__ uint32_t entry_tiles(const AttnArgs &a, int n_pairs, int64_t e)
{
    const int lane = threadIdx.x & 31;
    const int s = static_cast<int>(e / n_pairs), pr = static_cast<int>(e % n_pairs);
    int keys = static_cast<int>(list_len(a.L, s));
    if (a.q_pos) {
        const int t0 = static_cast<int>(2 * kPM * static_cast<int64_t>(pr) / a.G);
        const int t1 = static_cast<int>(min(int64_t(a.nq - 1), (2 * kPM * (static_cast<int64_t>(pr) + 1) - 1) / a.G));
        int top = -1;
        for (int t = t0 + lane; t <= t1; t += 32) top = max(top, __ldg(a.q_pos + a.token(s, t)));
        top = __reduce_max_sync(0xffffffffu, top);
        keys = top < 0 ? 0 : (top < keys ? top + 1 : keys);
    }
    return (static_cast<uint32_t>(keys) + kPN - 1) / kPN;
}

// Sets the status bit of lengths beyond their lists; `t` of `n` threads.
__device__ __forceinline__ void check_lengths(const AttnArgs &a, int t, int n)
{
    for (int s = t; s < a.L.S; s += n)
        if (list_len(a.L, s) < max(0, a.L.kv_len[s])) atomicOr(a.L.status, kStatusList);
}

// The plan of many entries: prefix sums of their tiles.
__global__ void __launch_bounds__(1024) prefill_plan_kernel(const AttnArgs a, int n_pairs, uint32_t *plan, int ctas)
{
    start();
    __shared__ uint32_t s_sum[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n = static_cast<int64_t>(a.L.S) * n_pairs;
    for (int64_t e = warp; e < n; e += 32) {
        const uint32_t x = entry_tiles(a, n_pairs, e);
        if (lane == 0) plan[e] = x;
    }
    check_lengths(a, tid, 1024);
    __syncthreads();
    const int64_t share = (n + 1023) / 1024, lo = min(n, tid * share), hi = min(n, lo + share);
    uint32_t sum = 0;
    for (int64_t e = lo; e < hi; ++e) sum += plan[e];
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    uint32_t before = inc - sum;
    for (int w = 0; w < warp; ++w) before += s_sum[w];
    for (int64_t e = lo; e < hi; ++e) {
        const uint32_t x = plan[e];
        plan[e] = before;
        before += x;
    }
    if (tid == 1023) {
        plan[n] = before;
        plan[n + 1] = piece_tiles(before * a.L.Hk, ctas);
    }
}

// The units of a CTA's piece of the line in turn, as every role walks them.
struct Unit {
    int s, kh, pr;
    uint32_t unit0;                             // the line's position of its tile 0
    int n;                                      // its tiles
    int p0, p1;                                 // [p0, p1) of them are this CTA's part
    int t0, t1, sub;                            // [t0, t1) of the part are at hand, sub tiles at a time
};
struct Walk {
    const uint32_t *plan;                       // shared or global memory
    int np, S, Hk;
    int most;                                   // tiles at a time
    uint32_t end;                               // of the piece
    uint32_t whole;                             // tiles of a piece where pieces end with their units, else 0
    const uint32_t *of;                         // with whole: the entries' tiles (the line holds them rounded up to pieces)

    __device__ void cut(Unit &x, uint32_t pos) const
    {
        if (whole) {                            // the unit's tiles in as many equal parts as it has pieces
            const uint32_t T = of[x.s * np + x.pr];   // (below 2^24, and k and i below 2^8)
            const uint32_t k = x.n / whole, i = (pos - x.unit0) / whole;
            x.n = static_cast<int>(T);
            x.p0 = static_cast<int>(i * T / k);
            x.p1 = static_cast<int>((i + 1) * T / k);
            x.unit0 = pos - x.p0;
        } else {
            x.p0 = static_cast<int>(pos - x.unit0);
            x.p1 = static_cast<int>(min(static_cast<uint32_t>(x.n), end - x.unit0));
        }
        const int len = x.p1 - x.p0, k = max(1, (len + most - 1 - kExactMore) / most);
        x.sub = (len + k - 1) / k;
        x.t0 = x.p0;
        x.t1 = x.p0 + x.sub;
    }
    __device__ int tiles(const Unit &x) const
    {
        const int64_t e = static_cast<int64_t>(x.s) * np + x.pr;
        return static_cast<int>(plan[e + 1] - plan[e]);
    }
    __device__ Unit first(uint32_t pos) const
    {
        Unit x;
        int lo = 0, hi = S;                     // the last sequence that begins at or before pos
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (plan[static_cast<int64_t>(mid) * np] * Hk <= pos) lo = mid;
            else hi = mid;
        }
        x.s = lo;
        const int64_t e0 = static_cast<int64_t>(lo) * np;
        const uint32_t p0 = plan[e0], T = plan[e0 + np] - p0, r = pos - p0 * Hk;
        x.kh = static_cast<int>(r / T);
        const uint32_t rr = r - x.kh * T + p0;  // within one head's pairs
        int el = 0, eh = np;
        while (eh - el > 1) {
            const int mid = (el + eh) >> 1;
            if (plan[e0 + mid] <= rr) el = mid;
            else eh = mid;
        }
        x.pr = el;
        x.n = tiles(x);
        x.unit0 = pos - (rr - plan[e0 + el]);
        cut(x, pos);
        return x;
    }
    __device__ bool next(Unit &x) const         // false at the end of the piece
    {
        if (x.t1 < x.p1) {                      // the part goes on
            x.t0 = x.t1;
            x.t1 = min(x.p1, x.t0 + x.sub);
            return true;
        }
        const uint32_t pos = x.unit0 + x.p1;
        if (whole || pos >= end) return false;
        do {
            if (++x.pr == np) {
                x.pr = 0;
                const int64_t e0 = static_cast<int64_t>(x.s) * np;
                if (++x.kh == Hk || plan[e0 + np] == plan[e0]) {
                    x.kh = 0;
                    ++x.s;
                }
            }
            x.n = tiles(x);
        } while (x.n == 0);
        x.unit0 = pos;
        cut(x, pos);
        return true;
    }
};

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
    __shared__ int s_abort, s_whole;
    __shared__ Unit s_unit[kSoftWarps][2];      // the softmax warps' units: kept out of their registers
    const uint32_t bar0 = smem_addr(s_bar);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    constexpr uint32_t kIdescS = tc::idesc_f16(kPM, kPN, false);
    constexpr uint32_t kIdescPV = tc::idesc_f16(kPM, D, true);
    constexpr int kOCol = 2 * kPN;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
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
            tc::mbar_init(bar(PB_PHALF + i), kPM);
            tc::mbar_init(bar(PB_PDONE + i), 1);
        }
        for (int i = 0; i < 4; ++i) tc::mbar_init(bar(PB_META + i), 2);
        tc::fence_barrier_init();
    }
    start();
    const int np = pa.n_pairs;
    const int64_t n_entries = static_cast<int64_t>(a.L.S) * np;
    uint32_t *s_plan = reinterpret_cast<uint32_t *>(sm + SM::kPlan), *s_tiles = reinterpret_cast<uint32_t *>(sm + SM::kTiles);
    Walk walk{pa.plan, np, a.L.S, a.L.Hk, HILO ? kExactTiles : kLongTiles, 0, 0, s_tiles};
    if (n_entries <= kPlanHere) {               // few entries: every CTA counts them itself
        for (int e = warp; e < n_entries; e += kPfThreads / 32) {
            const uint32_t x = entry_tiles(a, np, e);
            if (lane == 0) s_tiles[e] = x;
        }
        if (blockIdx.x == 0) check_lengths(a, tid, kPfThreads);
        walk.plan = s_plan;
    } else if (n_entries <= kPlanSmem) {
        for (int i = tid; i <= n_entries + 1; i += kPfThreads) s_plan[i] = __ldcg(pa.plan + i);
        walk.plan = s_plan;
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem;
    if (n_entries <= kPlanHere) {               // pieces and prefix sums; the merge reads CTA 0's
        if (warp == 0) {
            // Pieces that end with their units spare the CTAs a second start and result:
            // taken when the least piece with which the grid covers units one by one is
            // at most kStraddleTiles longer than even shares (64 tokens of eight ragged
            // sequences over up to 4096 keys, fp32: 48 us, against 56).
            uint32_t sum = 0, n[kStraddleTiles + 1] = {};
            for (int e = lane; e < n_entries; e += 32) sum += s_tiles[e];
            const uint32_t even = piece_tiles(__reduce_add_sync(0xffffffffu, sum) * a.L.Hk, gridDim.x);
            for (int e = lane; e < n_entries; e += 32)
#pragma unroll
                for (int i = 0; i <= kStraddleTiles; ++i) n[i] += (s_tiles[e] + even + i - 1) / (even + i);
            uint32_t chunk = even;
            bool fits = false;
#pragma unroll
            for (int i = kStraddleTiles; i >= 0; --i)
                if (__reduce_add_sync(0xffffffffu, n[i]) * a.L.Hk <= gridDim.x) {
                    chunk = even + i;
                    fits = true;
                }
            uint32_t before = 0;
            for (int b = 0; b < n_entries; b += 32) {
                uint32_t x = b + lane < n_entries ? s_tiles[b + lane] : 0u;
                if (fits) x = (x + chunk - 1) / chunk * chunk;
                uint32_t inc = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                if (b + lane < n_entries) s_plan[b + lane] = before + inc - x;
                before += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0) {
                s_plan[n_entries] = before;
                s_plan[n_entries + 1] = chunk;
                s_whole = fits;
            }
        }
        __syncthreads();
        if (s_whole) walk.whole = s_plan[n_entries + 1];
        if (blockIdx.x == 0)
            for (int i = tid; i <= n_entries + 1; i += kPfThreads) pa.plan[i] = s_plan[i];
    }

    const uint32_t total = walk.plan[n_entries] * a.L.Hk;
    const uint32_t chunk = walk.plan[n_entries + 1];
    const uint32_t pos0 = min(total, blockIdx.x * chunk);
    walk.end = min(total, pos0 + chunk);
    const bool any = pos0 < walk.end;
    auto two_tiles = [&](const Unit &x) { return (2 * x.pr + 1) * kPM < a.rows; };

    // Bounded: gives up after kSpins polls, or when another role has.
    auto wait = [&](int b, uint32_t parity) -> bool {
#pragma unroll 1
        for (uint32_t i = 0; i < kSpins; ++i) {
            if (tc::mbar_try_wait(bar(b), parity)) return true;
            if (*reinterpret_cast<volatile int *>(&s_abort)) return false;
        }
        s_abort = 1;
        atomicOr(a.L.status, 1);
        return false;
    };

    if (warp >= kSoftWarps && warp < kMmaWarp) {
        // ---------------- producers ----------------------------------------------
        fewer_regs<kRegProd>();
        const int pw = warp - kSoftWarps;       // rows 32 pw .. of every tile: page pw / 2 of it
        // 16 code bytes a lane.  Eight lanes that write together cover the same 64
        // channels of two rows, whose swizzled pieces fall on different banks.
        constexpr int NI = D / 16;              // loads for a warp's 32 rows
        constexpr int RPI = 32 / NI;            // rows of one
        const int c16 = (lane & 3) | (D == 128 ? (lane >> 4) << 2 : 0);
        const int r0 = pw * 32 + ((lane >> 2) & (RPI - 1));
        const int ch = 2 * (c16 & 3);
        auto convert = [&](const uint4 (&w)[NI], bool on, bool neg, uint8_t *tile) {
            uint8_t *dst = tile + (c16 >> 2) * SM::kHalf + r0 * 128;
            if (!on) {
#pragma unroll 1
                for (int i = 0; i < NI; ++i) {
                    const int x7 = (r0 + i * RPI) & 7;
                    *reinterpret_cast<uint4 *>(dst + i * RPI * 128 + ((ch ^ x7) << 4)) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(dst + i * RPI * 128 + (((ch + 1) ^ x7) << 4)) = make_uint4(0, 0, 0, 0);
                }
                return;
            }
            // 1024 + u in fp16, then +-(that - 1152)
            const __half2 sg = neg ? __half2half2(__ushort_as_half(0xbc00)) : __half2half2(__ushort_as_half(0x3c00));
            const __half2 bias = neg ? __half2half2(__ushort_as_half(0x6480)) : __half2half2(__ushort_as_half(0xe480));
            auto pair = [&](uint32_t x, uint32_t sel) -> uint32_t {
                const uint32_t h = __byte_perm(x, 0x64646464u, sel);
                const __half2 v = __hfma2(*reinterpret_cast<const __half2 *>(&h), sg, bias);
                return *reinterpret_cast<const uint32_t *>(&v);
            };
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int x7 = (r0 + i * RPI) & 7;
                const uint32_t a0 = w[i].x ^ 0x80808080u, a1 = w[i].y ^ 0x80808080u;
                const uint32_t a2 = w[i].z ^ 0x80808080u, a3 = w[i].w ^ 0x80808080u;
                *reinterpret_cast<uint4 *>(dst + i * RPI * 128 + ((ch ^ x7) << 4)) =
                    make_uint4(pair(a0, 0x4140), pair(a0, 0x4342), pair(a1, 0x4140), pair(a1, 0x4342));
                *reinterpret_cast<uint4 *>(dst + i * RPI * 128 + (((ch + 1) ^ x7) << 4)) =
                    make_uint4(pair(a2, 0x4140), pair(a2, 0x4342), pair(a3, 0x4140), pair(a3, 0x4342));
            }
        };
        uint4 kr[NI], vr[NI];
        auto load = [&](uint4 (&w)[NI], const int8_t *codes, int id) {
            if (id < 0) return;
            const int8_t *p = codes + (static_cast<int64_t>(id) * kPage + (r0 & 63)) * D + c16 * 16;
#pragma unroll
            for (int i = 0; i < NI; ++i) w[i] = ld_stream16(p + i * RPI * D);
        };
        uint32_t j = 0;                         // key tiles so far
        bool ok = any;
        if (any) {
            Unit x = walk.first(pos0);
            do {
                const int pages = static_cast<int>((list_len(a.L, x.s) + kPage - 1) / kPage);
                const int32_t *ids = a.L.ids + (static_cast<int64_t>(x.s) * a.L.Hk + x.kh) * a.L.cap;
                auto page_id = [&](int tile) {
                    const int b = 2 * tile + (pw >> 1);
                    return tile < x.t1 && b < pages ? max(-1, checked_page(a.L, __ldg(ids + b))) : -1;
                };
                int id = page_id(x.t0), id1 = page_id(x.t0 + 1);
                load(kr, a.k, id);
                load(vr, a.v, id);
                float dk = id >= 0 ? __ldg(a.k_scale + id) : 0.f, dv = id >= 0 ? __ldg(a.v_scale + id) : 0.f;
#pragma unroll 1
                for (int tl = x.t0; tl < x.t1; ++tl, ++j) {
                    const int b = static_cast<int>(j & 1);
                    const uint32_t before = ((j >> 1) - 1) & 1;
                    const int id2 = page_id(tl + 2);
                    const float dk1 = id1 >= 0 ? __ldg(a.k_scale + id1) : 0.f, dv1 = id1 >= 0 ? __ldg(a.v_scale + id1) : 0.f;
                    const float ks = dk * a.scale_log2;
                    if (!__all_sync(0xffffffffu, j < 2 || wait(PB_KEMPTY + b, before))) { ok = false; break; }
                    if ((pw & 1) == 0 && lane == 0) {
                        s_meta[j & 3][pw >> 1] = Meta{fmaxf(fabsf(ks), 1e-30f), dv != 0.f ? log2f(fabsf(dv)) : -INFINITY, id >= 0};
                        tc::mbar_arrive(bar(PB_META + static_cast<int>(j & 3)));
                    }
                    convert(kr, id >= 0, ks < 0.f, sm + SM::kK + b * SM::kTile);
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(bar(PB_KFULL + b));
                    load(kr, a.k, id1);
                    if (!__all_sync(0xffffffffu, j < 2 || wait(PB_VEMPTY + b, before))) { ok = false; break; }
                    convert(vr, id >= 0, dv < 0.f, sm + SM::kV + b * SM::kTile);
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(bar(PB_VFULL + b));
                    load(vr, a.v, id1);
                    id = id1;
                    id1 = id2;
                    dk = dk1;
                    dv = dv1;
                }
            } while (ok && walk.next(x));
        }
    } else if (warp >= kMmaWarp) {
        // ---------------- MMA issuers --------------------------------------------
        fewer_regs<kRegMma>();
        auto all = [](bool p) { return __all_sync(0xffffffffu, p) != 0; };
        uint32_t j = 0, units0 = 0, units1 = 0, tiles0 = 0, tiles1 = 0;   // key tiles, and of each query tile, so far
        bool ok = any;
        if (warp == kMmaWarp && any) {
            // S_g = Q_g K^T, once PV_g of the tile before has read W_g
            const uint64_t dq0 = tc::smem_desc(sbase + SM::kQ, 16, 1024);
            const uint64_t dk0 = tc::smem_desc(sbase + SM::kK, 16, 1024);
            Unit x = walk.first(pos0);
            do {
                const bool two = two_tiles(x);
                // (a part that goes on keeps its queries)
                if (x.t0 == x.p0) ok = all(wait(PB_QFULL, units0++ & 1)) && (!two || all(wait(PB_QFULL + 1, units1++ & 1)));
#pragma unroll 1
                for (int tl = x.t0; ok && tl < x.t1; ++tl, ++j) {
                    const int b = static_cast<int>(j & 1);
                    if (!(ok = all(wait(PB_KFULL + b, (j >> 1) & 1)))) break;
#pragma unroll 1
                    for (int g = 0; g < (two ? 2 : 1); ++g) {
                        const uint32_t t = g ? tiles1++ : tiles0++;
                        if (!(ok = t == 0 || all(wait(PB_PDONE + g, (t - 1) & 1)))) break;
                        tc::tc_fence_after();
                        const uint64_t ad = tc::desc_add(dq0, g * SM::kTile), bd = tc::desc_add(dk0, b * SM::kTile);
                        const uint32_t d_s = tmem + static_cast<uint32_t>(g * kPN);
                        if (tc::elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = (kk >> 2) * SM::kHalf + (kk & 3) * 32;
                                tc::mma_f16_ss(d_s, tc::desc_add(ad, off), tc::desc_add(bd, off), kIdescS, kk > 0 ? 1u : 0u);
                            }
                            tc::mma_commit(bar(PB_SFULL + g));
                            if (g == 1 || !two) tc::mma_commit(bar(PB_KEMPTY + b));
                        }
                        __syncwarp();
                    }
                }
            } while (ok && walk.next(x));
            // nobody waits for the last commits on the stages' free barriers: they
            // are awaited here, so that none is in flight at exit (after a wait gave
            // up: with a limit, as for all that was issued)
            for (uint32_t i = j > 2 ? j - 2 : 0; i < j; ++i) tc::mbar_wait(bar(PB_KEMPTY + static_cast<int>(i & 1)), (i >> 1) & 1, nullptr, 100000000ull);
            if (!ok) {
                if (tiles0) tc::mbar_wait(bar(PB_SFULL), (tiles0 - 1) & 1, nullptr, 100000000ull);
                if (tiles1) tc::mbar_wait(bar(PB_SFULL + 1), (tiles1 - 1) & 1, nullptr, 100000000ull);
            }
        } else if (warp == kMmaWarp + 1 && any) {
            // O_g += W_g V
            const uint64_t dv0 = tc::smem_desc(sbase + SM::kV, SM::kHalf, 1024);
            Unit x = walk.first(pos0);
            do {
                const bool two = two_tiles(x);
#pragma unroll 1
                for (int tl = x.t0; ok && tl < x.t1; ++tl, ++j) {
                    const int b = static_cast<int>(j & 1);
                    if (!(ok = all(wait(PB_VFULL + b, (j >> 1) & 1)))) break;
#pragma unroll 1
                    for (int g = 0; g < (two ? 2 : 1); ++g) {
                        const uint32_t t = g ? tiles1++ : tiles0++;
                        // the second 64 keys first, as the softmax does
                        if (!(ok = all(wait(PB_PHALF + g, t & 1)))) break;
                        tc::tc_fence_after();
                        const uint64_t bd = tc::desc_add(dv0, b * SM::kTile);
                        const uint32_t d_w = tmem + static_cast<uint32_t>(g * kPN);
                        const uint32_t d_o = tmem + static_cast<uint32_t>(kOCol + g * D);
                        auto products = [&](int k0, bool from0) {
#pragma unroll
                            for (int i = 0; i < kPN / 32; ++i) {
                                const int kk = k0 + i;
                                const uint32_t at = d_w + static_cast<uint32_t>((kk >> 1) * 32 + (kk & 1) * 8);
                                tc::mma_f16_ts(d_o, at, tc::desc_add(bd, kk * 2048), kIdescPV, (from0 && i == 0) ? 0u : 1u);
                                if (HILO) tc::mma_f16_ts(d_o, at + 16, tc::desc_add(bd, kk * 2048), kIdescPV, 1u);
                            }
                        };
                        if (tc::elect_one()) products(kPN / 32, tl == x.t0);
                        __syncwarp();
                        if (!(ok = all(wait(PB_PFULL + g, t & 1)))) break;
                        tc::tc_fence_after();
                        if (tc::elect_one()) {
                            products(0, false);
                            tc::mma_commit(bar(PB_PDONE + g));
                            if (g == 1 || !two) tc::mma_commit(bar(PB_VEMPTY + b));
                        }
                        __syncwarp();
                    }
                }
            } while (ok && walk.next(x));
            for (uint32_t i = j > 2 ? j - 2 : 0; i < j; ++i) tc::mbar_wait(bar(PB_VEMPTY + static_cast<int>(i & 1)), (i >> 1) & 1, nullptr, 100000000ull);
            if (!ok) {
                if (tiles0) tc::mbar_wait(bar(PB_PDONE), (tiles0 - 1) & 1, nullptr, 100000000ull);
                if (tiles1) tc::mbar_wait(bar(PB_PDONE + 1), (tiles1 - 1) & 1, nullptr, 100000000ull);
            }
        } else if (warp == kMmaWarp + 2) {
            // rows of pairs without a visible key: written here, by all CTAs' spare warps
            for (int64_t e = 0; e < n_entries; ++e) {
                if (walk.plan[e + 1] != walk.plan[e]) continue;
                const int s = static_cast<int>(e / np), pr = static_cast<int>(e % np);
                const int r0 = 2 * kPM * pr;
                const int64_t nr = min(2 * kPM, a.rows - r0), n = nr * a.L.Hk * (D / 4);
                for (int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane; i < n; i += static_cast<int64_t>(gridDim.x) * 32) {
                    const int c = static_cast<int>(i % (D / 4)), kh = static_cast<int>(i / (D / 4) / nr);
                    const int row = r0 + static_cast<int>(i / (D / 4) % nr);
                    const int64_t r = a.token(s, row / a.G) * a.H + kh * a.G + row % a.G;
                    if (pa.out_f16) *reinterpret_cast<uint2 *>(static_cast<__half *>(a.o) + r * D + 4 * c) = make_uint2(0, 0);
                    else *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + r * D + 4 * c) = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (c == 0) a.lse[r] = -INFINITY;
                }
            }
        }
    } else {
        // ---------------- softmax: one thread per query row -----------------------
        more_regs<kRegSoft>();
        const int g = warp >> 2;
        const int m = (warp & 3) * 32 + lane;   // row of the tile = lane of tensor memory
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_col = lane_base + static_cast<uint32_t>(g * kPN);
        const uint32_t o_col = lane_base + static_cast<uint32_t>(kOCol + g * D);
        auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory"); };
        auto active = [&](const Unit &y) { return g == 0 || two_tiles(y); };
        // index of this thread's row in q and o (-1: past the last)
        auto row_index = [&](const Unit &x) -> int64_t {
            const int row = (2 * x.pr + g) * kPM + m;
            return row < a.rows ? a.token(x.s, row / a.G) * a.H + x.kh * a.G + row % a.G : -1;
        };
        // the warp's 32 query rows into shared memory, D / 8 lanes a row
        auto put_q = [&](int64_t index) {
            constexpr int LPR = D / 8;
            const int c = lane % LPR;
            uint8_t *qt = sm + SM::kQ + g * SM::kTile + (c >> 3) * SM::kHalf;
#pragma unroll
            for (int i = 0; i < LPR; ++i) {
                const int rl = i * (32 / LPR) + lane / LPR;         // row of the warp
                const int64_t r = __shfl_sync(0xffffffffu, index, rl);
                const uint4 v = r >= 0 ? __ldg(reinterpret_cast<const uint4 *>(a.q + r * D) + c) : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(qt + ((warp & 3) * 32 + rl) * 128 + (((c & 7) ^ (rl & 7)) << 4)) = v;
            }
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(bar(PB_QFULL + g));
        };
        uint32_t j = 0, tiles = 0;              // key tiles so far, and those with this query tile
        if (any) {
            if (lane == 0) s_unit[warp][0] = walk.first(pos0);
            __syncwarp();
            if (active(s_unit[warp][0])) put_q(row_index(s_unit[warp][0]));
        }
        bool more = any;
#pragma unroll 1
        for (int u = 0; more; u ^= 1) {
            const Unit &x = s_unit[warp][u];
            meet();
            const bool tile_on = active(x);
            const int n = x.t1 - x.t0;
            float m_ref = -INFINITY, r_ref = -INFINITY, l_run = 0.f;
            float w_sum = 0.f, w_cut = 0.f;     // of the weights in O: their sum, and one as the tensor core takes it
            if (tile_on) {
                const int row = (2 * x.pr + g) * kPM + m;
                const int len = static_cast<int>(list_len(a.L, x.s));
                int lim = len;                  // keys that this row sees
                if (a.q_pos) {
                    const int qp = __ldg(a.q_pos + a.token(x.s, min(row / a.G, a.nq - 1)));
                    lim = qp < 0 ? 0 : (qp < len ? qp + 1 : len);
                }
                lim -= x.t0 * kPN;              // counted from the tile at hand
                int pages = (len + kPage - 1) / kPage - 2 * x.t0;
                float *pl = nullptr;
                if (a.page_lse && row < a.rows)
                    pl = a.page_lse + ((static_cast<int64_t>(x.s) * a.L.Hk + x.kh) * a.L.cap + 2 * x.t0) * a.rows + row;
                // No early exit from this loop: after a wait gives up, every later
                // wait returns at once and the warp runs through (the outputs are
                // then invalid and the status word says so).
#pragma unroll 1
                for (int jj = 0; jj < n; ++jj, ++j, ++tiles, lim -= kPN, pages -= 2) {
                    // what does not depend on the scores first: the pages' factors and reference
                    __all_sync(0xffffffffu, wait(PB_META + static_cast<int>(j & 3), (j >> 2) & 1));
                    const Meta mt0 = s_meta[j & 3][0], mt1 = s_meta[j & 3][1];
                    const int lim0 = mt0.on ? lim : 0, lim1 = mt1.on ? lim - kPage : 0;
                    // (-inf where there is no page, or none that the row sees: a page it does not
                    // see must not push its own values out of fp16)
                    const float lv0 = lim0 > 0 ? mt0.lv : -INFINITY, lv1 = lim1 > 0 ? mt1.lv : -INFINITY;
                    const float r_old = r_ref;
                    const float lv_max = fmaxf(lv0, lv1);
                    if (lv_max > r_ref + kPfScaleGrow) r_ref = ceilf(lv_max);
                    const float dl0 = lv0 == -INFINITY ? kNoScale : fmaxf(lv0 - r_ref, kNoScale);
                    const float dl1 = lv1 == -INFINITY ? kNoScale : fmaxf(lv1 - r_ref, kNoScale);
                    const float un0 = fast_exp2(-dl0), un1 = fast_exp2(-dl1);
                    const bool masked = __any_sync(0xffffffffu, lim0 < kPage || lim1 < kPage);
                    __all_sync(0xffffffffu, wait(PB_SFULL + g, tiles & 1));
                    tc::tc_fence_after();
                    // The row's largest score, which the loads bring along; masked ones go
                    // back as -inf first.
                    uint32_t xr[2][32];
                    float top[4];
                    if (masked) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            const int lc = (c < 2 ? lim0 : lim1) - (c & 1) * 32;
                            tc::tmem_ld32(s_col + c * 32, xr[0]);
                            tc::tmem_wait_ld(xr[0]);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i >= lc) xr[0][i] = 0xff800000u;
                            tc::tmem_st32u(s_col + c * 32, xr[0]);
                        }
                        tc::tmem_wait_st();
                    }
                    tc::tmem_ld32_max(s_col, xr[0], top[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tc::tmem_wait_ld_max(xr[c & 1], top[c]);
                        if (c < 3) tc::tmem_ld32_max(s_col + (c + 1) * 32, xr[(c + 1) & 1], top[c + 1]);
                    }
                    float ref = m_ref;
                    const float mx = fmaxf(fmaxf(top[0], top[1]) * mt0.ks, fmaxf(top[2], top[3]) * mt1.ks);
                    if (mx > ref + kPfGrow) ref = ceilf(mx);        // true on the first finite maximum
                    const float off = ref == -INFINITY ? 0.f : kPfShift - ref;
                    const float alpha = ref == m_ref ? 1.f : (m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - ref));
                    const float alpha_o = r_ref == r_old ? alpha : (r_old == -INFINITY ? 0.f : alpha * fast_exp2(r_old - r_ref));
                    // O_g holds every PV up to the last tile (S_g was issued after
                    // it was done) and none of this tile before its weights are announced
                    if (jj > 0 && __any_sync(0xffffffffu, alpha_o != 1.f)) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t rr[16];
                            tc::tmem_ld16(o_col + c * 16, rr);
                            tc::tmem_wait_ld16(rr);
#pragma unroll
                            for (int i = 0; i < 16; ++i) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha_o);
                            tc::tmem_st16u(o_col + c * 16, rr);
                        }
                    }
                    // The weights, stored over their own scores (keys 32c .. in columns 32c ..,
                    // what rounding left 16 further on): the second page's, which are in
                    // registers, then the first's; each half is announced by itself.
                    float lq[2][4];
                    if (HILO) w_cut *= alpha_o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = i ^ 2;
                        uint32_t(&xc)[32] = xr[c & 1];
                        const float ks = c < 2 ? mt0.ks : mt1.ks, of = off + (c < 2 ? dl0 : dl1);
                        if (i >= 2) tc::tmem_wait_ld(xc);
                        float(&l4)[4] = lq[c >> 1];
                        if ((c & 1) == 0) l4[0] = l4[1] = l4[2] = l4[3] = 0.f;
                        uint32_t hi[16], lo[16];
                        float s16[2];                   // of a product's 16 keys
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float w0, w1;
                            fma2(w0, w1, __uint_as_float(xc[e]), __uint_as_float(xc[e + 1]), ks, of);
                            w0 = fast_exp2(w0);
                            w1 = fast_exp2(w1);
                            if (HILO) {
                                if ((e & 15) == 0) s16[0] = s16[1] = 0.f;
                                add2(s16[0], s16[1], w0, w1);
                                if ((e & 15) == 14) {
                                    const float h = s16[0] + s16[1];
                                    l4[e >> 4] += h;
                                    w_cut = __fmaf_rz(kLowPart, h, __fadd_rz(w_cut, h));
                                }
                            } else {
                                add2(l4[e & 2], l4[(e & 2) + 1], w0, w1);
                            }
                            hi[e >> 1] = pack_half2(w0, w1);
                            if (HILO) {
                                const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hi[e >> 1]));
                                lo[e >> 1] = pack_half2(w0 - back.x, w1 - back.y);
                            }
                        }
                        if (i < 2) tc::tmem_ld32(s_col + i * 32, xc);
                        tc::tmem_st16u(s_col + c * 32, hi);
                        if (HILO) tc::tmem_st16u(s_col + c * 32 + 16, lo);
                        if (i == 1) {
                            tc::tmem_wait_st();
                            tc::tc_fence_before();
                            tc::mbar_arrive(bar(PB_PHALF + g));
                        }
                    }
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                    tc::mbar_arrive(bar(PB_PFULL + g));
                    const float ws0 = (lq[0][0] + lq[0][1]) + (lq[0][2] + lq[0][3]);
                    const float ws1 = (lq[1][0] + lq[1][1]) + (lq[1][2] + lq[1][3]);
                    const float ls0 = ws0 * un0, ls1 = ws1 * un1;
                    if (HILO) w_sum = w_sum * alpha_o + (ws0 + ws1);
                    if (pl) {
                        if (pages > 0) pl[0] = ls0 > 0.f ? ref - kPfShift + log2f(ls0) : -INFINITY;
                        if (pages > 1) pl[a.rows] = ls1 > 0.f ? ref - kPfShift + log2f(ls1) : -INFINITY;
                        pl += 2 * static_cast<int64_t>(a.rows);
                    }
                    l_run = l_run * alpha + (ls0 + ls1);
                    m_ref = ref;
                }
            } else {
                j += n;
            }
            // the next unit's queries go in while this one's last product runs: S_g of
            // the last tile is done, and nothing else reads Q_g
            {
                int again = 0;
                if (lane == 0) {
                    Unit y = x;
                    again = walk.next(y);
                    s_unit[warp][u ^ 1] = y;
                }
                more = __shfl_sync(0xffffffffu, again, 0) != 0;
                __syncwarp();
                const Unit &y = s_unit[warp][u ^ 1];
                if (more && y.t0 == y.p0 && active(y)) put_q(row_index(y));
            }
            if (!tile_on) continue;
            const int64_t out = row_index(x);
            const bool whole = x.p0 == 0 && x.p1 == x.n && x.t1 == x.p1;      // the result, not a piece
            const bool joins = x.t0 > x.p0;                                   // an earlier stretch of the part is in the slot
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (x.unit0 + x.p0 == pos0 ? 0 : 1);
            // ---------------- O / l, lse: result or piece ------------------------------
            bool have = wait(PB_PDONE + g, (tiles - 1) & 1) && !*reinterpret_cast<volatile int *>(&s_abort);
            have = __all_sync(0xffffffffu, have);
            if (have) tc::tc_fence_after();
            const bool empty = !have || l_run == 0.f;
            float inv = empty ? 0.f : fast_exp2(r_ref == -INFINITY ? 0.f : r_ref) / l_run;
            float lse2 = empty ? -INFINITY : m_ref - kPfShift + log2f(l_run);
            float *const ml = a.part_ml + (slot * 2 + g) * kPM + m;
            float w_old = 0.f;                  // weight of the stretches before
            if (HILO && w_cut > 0.f) inv *= w_sum * (1.f + kLowPart) / w_cut;
            if (joins && out >= 0) {
                const float z = __ldcg(ml), top = fmaxf(z, lse2);
                if (z != -INFINITY || lse2 != -INFINITY) {
                    const float e_old = fast_exp2(z - top), e_new = fast_exp2(lse2 - top);
                    w_old = e_old / (e_old + e_new);
                    inv *= e_new / (e_old + e_new);
                    lse2 = top + log2f(e_old + e_new);
                }
            }
            // 16 columns of the warp's rows through shared memory, so that four lanes
            // write 64 (fp16: 32) bytes of a row
            float *stage = reinterpret_cast<float *>(sm + SM::kStage) + warp * 32 * SM::kStageLd;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                uint32_t orr[16];
                if (have) {
                    tc::tmem_ld16(o_col + c * 16, orr);             // warp-wide: every lane takes part
                    tc::tmem_wait_ld16(orr);
                }
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = empty ? 0.f : __uint_as_float(orr[i + e]) * inv;
                    *reinterpret_cast<float4 *>(stage + lane * SM::kStageLd + i) = make_float4(v[0], v[1], v[2], v[3]);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rl = i * 8 + (lane >> 2), col = c * 16 + (lane & 3) * 4;
                    float4 v = *reinterpret_cast<const float4 *>(stage + rl * SM::kStageLd + (lane & 3) * 4);
                    const int64_t r = __shfl_sync(0xffffffffu, out, rl);
                    const float w = __shfl_sync(0xffffffffu, w_old, rl);
                    if (r < 0) continue;
                    if (joins) {                // (the same thread wrote it)
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(a.part_o + ((slot * 2 + g) * kPM + (warp & 3) * 32 + rl) * D + col));
                        v.x = fmaf(w, y.x, v.x);
                        v.y = fmaf(w, y.y, v.y);
                        v.z = fmaf(w, y.z, v.z);
                        v.w = fmaf(w, y.w, v.w);
                    }
                    if (!whole)
                        *reinterpret_cast<float4 *>(a.part_o + ((slot * 2 + g) * kPM + (warp & 3) * 32 + rl) * D + col) = v;
                    else if (pa.out_f16)
                        *reinterpret_cast<uint2 *>(static_cast<__half *>(a.o) + r * D + col) =
                            make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
                    else
                        *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + r * D + col) = v;
                }
                __syncwarp();
            }
            if (out >= 0) {
                if (whole) a.lse[out] = lse2 * 0.6931471805599453f;
                else *ml = lse2;
            }
            tc::tc_fence_before();              // O_g is read before W_g of the next unit is announced
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after();
        tc::tmem_dealloc<512>(tmem);
    }
}

// Rows of units that several CTAs share: their pieces together.  D / 4 lanes a row,
// kMergeRows rows a thread.  DEEP = false: all pieces in order; true: every warp of a CTA
// the same rows and batches of four pieces in turn, then the warps' sums in order.
constexpr int kMergeRows = 4;
template <int D, bool DEEP>
__global__ void __launch_bounds__(256, 2) prefill_merge_kernel(const PrefillArgs pa)
{
    start();
    const AttnArgs &a = pa.a;
    constexpr int LPR = D / 4, RPP = (DEEP ? 32 : 256) / LPR;
    constexpr int kWarps = 8;
    const int np = pa.n_pairs;
    const int unit = blockIdx.y, list = unit / np, pr = unit - list * np;
    const int s = list / a.L.Hk, kh = list - s * a.L.Hk;
    const int64_t e0 = static_cast<int64_t>(s) * np;
    const uint32_t chunk = __ldcg(pa.plan + static_cast<int64_t>(a.L.S) * np + 1);
    const uint32_t p0 = __ldcg(pa.plan + e0), pe = __ldcg(pa.plan + e0 + pr), pe1 = __ldcg(pa.plan + e0 + pr + 1);
    const uint32_t T = __ldcg(pa.plan + e0 + np) - p0;
    if (pe1 == pe) return;
    const uint32_t unit0 = p0 * a.L.Hk + kh * T + (pe - p0);
    const uint32_t c_lo = unit0 / chunk, c_hi = (unit0 + (pe1 - pe) - 1) / chunk;
    if (c_lo == c_hi) return;
    const int lane = threadIdx.x % LPR;
    float M[kMergeRows], W[kMergeRows], v[kMergeRows][4];
    int rr[kMergeRows];                         // rows of the unit
#pragma unroll
    for (int i = 0; i < kMergeRows; ++i) {
        rr[i] = (blockIdx.x * kMergeRows + i) * RPP + (DEEP ? threadIdx.x & 31 : threadIdx.x) / LPR;
        M[i] = -INFINITY;
        W[i] = v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
    }
    // pieces four at a time, all their loads before any use
#pragma unroll 1
    for (uint32_t c0 = c_lo + (DEEP ? threadIdx.x / 32 * 4 : 0); c0 <= c_hi; c0 += DEEP ? kWarps * 4 : 4) {
        float z[kMergeRows][4];
        float4 y[kMergeRows][4];
#pragma unroll
        for (int i = 0; i < kMergeRows; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t c = c0 + e;
                // piece c of the unit is slot 2c, or 2c + 1 when an earlier unit begins CTA c's piece
                const int64_t at = (2 * static_cast<int64_t>(c) + (c == c_lo && unit0 > c * chunk ? 1 : 0)) * 2 * kPM + rr[i];
                const bool on = c <= c_hi && pr * 2 * kPM + rr[i] < a.rows && rr[i] < 2 * kPM;
                z[i][e] = on ? __ldcg(a.part_ml + at) : -INFINITY;
                y[i][e] = on ? __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * D) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
        for (int i = 0; i < kMergeRows; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float m = fmaxf(M[i], z[i][e]);
                const float bo = M[i] == -INFINITY ? 0.f : fast_exp2(M[i] - m);
                const float bn = z[i][e] == -INFINITY ? 0.f : fast_exp2(z[i][e] - m);
                M[i] = m;
                W[i] = fmaf(W[i], bo, bn);
                v[i][0] = fmaf(v[i][0], bo, bn * y[i][e].x);
                v[i][1] = fmaf(v[i][1], bo, bn * y[i][e].y);
                v[i][2] = fmaf(v[i][2], bo, bn * y[i][e].z);
                v[i][3] = fmaf(v[i][3], bo, bn * y[i][e].w);
            }
    }
    auto write = [&](int r_unit, float Mr, float Wr, const float (&vr)[4]) {
        const int row = pr * 2 * kPM + r_unit;
        if (row >= a.rows || r_unit >= 2 * kPM) return;
        const float q = Wr == 0.f ? 0.f : 1.f / Wr;
        const int64_t r = a.token(s, row / a.G) * a.H + kh * a.G + row % a.G;
        if (pa.out_f16)
            *reinterpret_cast<uint2 *>(static_cast<__half *>(a.o) + r * D + lane * 4) =
                make_uint2(pack_half2(vr[0] * q, vr[1] * q), pack_half2(vr[2] * q, vr[3] * q));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + r * D + lane * 4) =
                make_float4(vr[0] * q, vr[1] * q, vr[2] * q, vr[3] * q);
        if (lane == 0) a.lse[r] = Wr == 0.f ? -INFINITY : (Mr + log2f(Wr)) * 0.6931471805599453f;
    };
    if constexpr (!DEEP) {
#pragma unroll
        for (int i = 0; i < kMergeRows; ++i) write(rr[i], M[i], W[i], v[i]);
    } else {
        constexpr int kRows = kMergeRows * RPP; // of the CTA
        __shared__ float s_m[kWarps][kRows], s_w[kWarps][kRows];
        __shared__ float4 s_v[kWarps][kRows][LPR];
        const int warp = threadIdx.x / 32, sub = (threadIdx.x & 31) / LPR;
#pragma unroll
        for (int i = 0; i < kMergeRows; ++i) {
            if (lane == 0) {
                s_m[warp][i * RPP + sub] = M[i];
                s_w[warp][i * RPP + sub] = W[i];
            }
            s_v[warp][i * RPP + sub][lane] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        }
        __syncthreads();
        const int rl = threadIdx.x / LPR;
        if (rl >= kRows) return;
        float Mr = -INFINITY, Wr = 0.f, vr[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) Mr = fmaxf(Mr, s_m[w][rl]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float b = s_m[w][rl] == -INFINITY ? 0.f : fast_exp2(s_m[w][rl] - Mr);
            const float4 y = s_v[w][rl][lane];
            Wr = fmaf(s_w[w][rl], b, Wr);
            vr[0] = fmaf(y.x, b, vr[0]);
            vr[1] = fmaf(y.y, b, vr[1]);
            vr[2] = fmaf(y.z, b, vr[2]);
            vr[3] = fmaf(y.w, b, vr[3]);
        }
        write(blockIdx.x * kRows + rl, Mr, Wr, vr);
    }
}

// Attention weight of each page from the log sums of its rows: one warp a page,
// rows in the lanes' order.
__global__ void __launch_bounds__(256) prefill_mass_kernel(const AttnArgs a, float *mass)
{
    start();
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
    const cudaError_t l = launch(prefill_kernel<D, HILO>, dim3(grid), kPfThreads, smem, st, pa);
    if (h->prof_after) cudaEventRecord(h->prof_after, st);
    if (l != cudaSuccess) return cuda_fail(h, l, "8-bit prefill launch");
    const int units = pa.a.L.S * pa.a.L.Hk * pa.n_pairs;
    const int rows = std::min(2 * kPM, pa.a.rows);
    // Pieces of a unit, flat against deep: one unit of 108 rows and 140669 keys (138 pieces)
    // 61 / 34 us the call, four over 100000 keys (38) 61 / 53, eight over 32768 (19)
    // 48.4 / 49.1, sixteen (10) 73 / 80.
    const bool deep = grid > 24 * units;
    const int per_cta = (deep ? 32 : 256) * kMergeRows;
    const dim3 ctas((rows * (D / 4) + per_cta - 1) / per_cta, units);
    return cuda_fail(h, deep ? launch(prefill_merge_kernel<D, true>, ctas, 256, 0, st, pa)
                             : launch(prefill_merge_kernel<D, false>, ctas, 256, 0, st, pa), "8-bit prefill merge launch");
}

int launch_prefill(skv_handle *h, const AttnArgs &a, int D, bool f16, uint32_t *plan, int n_pairs, float *mass, int grid,
                   cudaStream_t st)
{
    if (static_cast<int64_t>(a.L.S) * n_pairs > kPlanHere) {
        const cudaError_t e = launch(prefill_plan_kernel, dim3(1), 1024, 0, st, a, n_pairs, plan, grid);
        if (e != cudaSuccess) return cuda_fail(h, e, "8-bit prefill plan launch");
    }
    const PrefillArgs pa{a, plan, n_pairs, f16};
    int rc;
    if (D == 128) rc = f16 ? launch_one<128, false>(h, pa, grid, st) : launch_one<128, true>(h, pa, grid, st);
    else rc = f16 ? launch_one<64, false>(h, pa, grid, st) : launch_one<64, true>(h, pa, grid, st);
    if (rc || !mass) return rc;
    return cuda_fail(h, launch(prefill_mass_kernel, dim3(static_cast<unsigned>((a.L.cap + 7) / 8), a.L.Hk, a.L.S), 256, 0, st, a, mass),
                     "page weight launch");
}

}  // namespace q8
}  // namespace skv
