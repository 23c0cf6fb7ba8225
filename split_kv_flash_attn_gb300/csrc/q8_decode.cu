// q8_decode.cu -- attention of a few query rows per KV head over 8-bit pages.
//
// The mathematics.  Over a page the score of key j is (scale * d_k) * (q . c_j)
// and its value d_v * c_vj, so the codes go into the products as they are
// (int8 is exact in fp16) and the page's scales multiply fp32 numbers.  With m
// the running reference of a query row,
//   p_j = 2^(s_j - m + 10),  l = sum p_j,  O = sum over pages d_v sum p_j c_vj,
// and o = O / l.  The weights p_j stay below 2^14, and each enters the product as
// two fp16 numbers (itself rounded, and what the rounding left), which keeps it
// to 2^-22 of its value down to 2^-24.  The tensor core adds to its accumulator
// with truncation, so products of 32 keys are summed from zero and joined to O
// by an fp32 FMA, which also applies d_v (one accumulator over all pages was
// off by 1.5e-6 after 11 pages a warp, growing with them).
//
// Work split.  All pages of all (sequence, KV head, row group) units form one
// line, of which every CTA takes an equal piece; a piece that covers several
// units works through them, and a unit that several pieces share is put
// together by the last CTA to finish with it, in piece order (so results do not
// depend on timing).  (Equal pieces end up to 15 % apart, as some SMs see less
// bandwidth; short pieces handed out at the end cost more than that: each begins
// with a chain of look-ups and ends with a join, 72 against 64 us.)  Lengths are read
// on the device: a call costs its keys, not its lists' capacity, and ragged batches
// stay balanced.
//
// A CTA is one warp that fetches and W that compute.  The first walks the CTA's
// pages, looks their ids and scales up 32 at a time and keeps a ring of pages (K
// and V, one TMA box each) in flight.  The others take half pages (32 keys) in
// turn, each on its own with a state of its own; twice the slots are a
// multiple of W, so that the same two warps own every turn of a slot (a
// barrier's parity tells a warp only whether the turn after its last one has
// come).  A ring of half pages was bound by the fetching warp (300 ns a slot).
//
// Fragments.  The order of channels inside q . c and of keys inside p . c is free,
// so a thread (g, t) of the mma layout takes 16-byte pieces: of key rows r(g), r(g) + 8
// the channels 16t .. and 64 + 16t .., of four value rows the channels 16 p(g) ..
// (pairs of rows are interleaved by byte permutes).  r and p swap the low bit of g
// to the top, which with the 128-byte swizzle makes these reads free of bank conflicts.
// Keys are the M side of S = K Q^T and channels that of O^T = V^T P^T, so
// the eight query columns of a product carry a KV head's query heads.
//
// Bound: the pages' bytes at long lengths (one sequence over 1048576 keys, eight KV
// heads of D = 128: 321 us, 6.7 TB/s; eight sequences of up to 32768: 60.8 us, 5.2 TB/s,
// DRAM reads 316 MB, which is the pages); launch, look-ups and joins at short ones
// (256 keys: 5.7 us); fetching and decoding the pages once for each 16 rows from 17 on
// (8 sequences of 16000 keys: 68 us with 16 rows a KV head, 110 with 32).
#include "q8.cuh"

namespace skv {
namespace q8 {

constexpr float kShift = 10.f;      // weights are kept times 2^10 ...
constexpr float kGrow = 4.f;        // ... and their reference moves when a score passes it by 2^4
constexpr int kStep = 32;           // keys a warp takes at a time
constexpr uint32_t kStraddle = 8;   // pages that a second start and join of a CTA cost

// Computing warps and as many ring slots.  One column group, D = 128: eight sequences of
// up to 32768 keys took 60 us with 11 and 11, 63 with 7 and 7 or 8 and 8, 68 with 6 and
// 12 (one of 1048576: 316, 334, 340 and 367; before the warps voted on their waits, which
// costs 1 %); D = 64: 38.5 us with 15, 44 with 11.  Two
// groups need the registers of 7 warps with D = 128; with D = 64 (four tokens of
// eight sequences over 16000 keys) 47.8 us with 10, 51.7 with 7.
__host__ __device__ constexpr int warps_of(int D, int nc) { return nc == 1 ? (D == 64 ? 15 : 11) : (D == 64 ? 10 : 7); }
// Pages that the fetching warp requests at a time: a ring of 7 would stand still.
__host__ __device__ constexpr int batch_of(int D, int nc) { return nc == 2 && D == 128 ? 2 : 4; }
template <int D, int NC>
__host__ __device__ constexpr int decode_smem()
{
    return 1024 + warps_of(D, NC) * 2 * kPage * D               // the ring, aligned for the swizzle
           + warps_of(D, NC) * 8 * (D + 4) * 4                  // the warps' results
           + NC * (D / 16) * 32 * 8;                         // query fragments
}
static_assert(decode_smem<128, 1>() < 226 * 1024 && decode_smem<128, 2>() < 226 * 1024, "shared memory per CTA");

// A list on the line of pages.
struct Place {
    int list;                       // sequence, or sequence x token with a selection
    uint32_t np;                    // its pages, rounded up to whole pieces where units are
    uint32_t base;                  // the line's position of its first page
};

__device__ __forceinline__ uint32_t pages_of(const AttnArgs &a, int list)
{
    if (a.sel) return a.n_sel;
    return static_cast<uint32_t>((list_len(a.L, list) + kPage - 1) / kPage);
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

template <int D, int NC, bool HILO, bool F16>
__global__ void __launch_bounds__(warps_of(D, NC) * 32 + 32, 1)
    decode_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const AttnArgs a)
{
    constexpr int KS = D / 16;                      // k-steps of S
    constexpr int CH = D / 64;                      // 16-byte chunks of a key row per thread
    constexpr int MT = D / 16;                      // m-tiles of O^T
    constexpr int VW = D / 32;                      // words of a value row per thread
    constexpr int LDO = D + 4;
    constexpr int W = warps_of(D, NC);                 // computing warps; the last warp fetches
    constexpr int kConsumers = W * 32, kThreads = kConsumers + 32;
    constexpr int NS = warps_of(D, NC);
    static_assert(2 * NS % W == 0, "the same warps own a slot's halves at every turn");
    constexpr int kBatch = batch_of(D, NC);
    constexpr int BYTES = kPage * D;                // of a slot's K or V
    struct Meta {
        int id, blk;
        float ks, vs;
    };
    extern __shared__ uint8_t smem_raw[];
    __shared__ alignas(8) uint64_t s_bar[2 * NS];   // full, empty
    __shared__ Meta s_meta[64];                     // of page n of the CTA: s_meta[n % 64]
    __shared__ float s_ml[W][8][2];
    __shared__ int s_last, s_abort;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float(*s_o)[8][LDO] = reinterpret_cast<float(*)[8][LDO]>(ring + NS * 2 * BYTES);
    uint2 *s_q = reinterpret_cast<uint2 *>(ring + NS * 2 * BYTES + W * 8 * LDO * 4);
    const uint32_t bar0 = smem_addr(s_bar);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_lists = a.sel ? a.L.S * a.nq : a.L.S;
    const uint32_t mult = a.L.Hk * a.row_groups;    // units per list
    if (tid == kConsumers) {
        tc::prefetch_tmap(&map_k);
        tc::prefetch_tmap(&map_v);
    }
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 2 * NS; ++i) tc::mbar_init(bar0 + 8 * i, i < NS ? 1 : 2);
        tc::fence_barrier_init();
    }
    start();

    // ---- the plan: total pages, this CTA's piece, the list that it starts in --
    uint32_t sum = 0;                               // (the host gives a launch no more than kMaxVisits)
    uint32_t np_lane = 0;                           // pages of list `lane`
    if (a.sel) {
        sum = static_cast<uint32_t>(n_lists) * a.n_sel;
        if (blockIdx.x == 0)
            for (int i = tid; i < a.L.S; i += kThreads)
                if (list_len(a.L, i) < max(0, a.L.kv_len[i])) atomicOr(a.L.status, kStatusList);
    } else {
        for (int i = lane; i < n_lists; i += 32) {
            const uint32_t n = pages_of(a, i);
            if (i == lane) np_lane = n;
            sum += n;
            if (blockIdx.x == 0 && static_cast<int64_t>(n) * kPage < max(0, a.L.kv_len[i])) atomicOr(a.L.status, kStatusList);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    sum *= mult;
    uint32_t total = sum;
    const uint32_t even = max(static_cast<uint32_t>(kPieceMin), (total + gridDim.x - 1) / gridDim.x);
    // Pieces that end with their units spare the CTAs a second start and join: taken
    // when the least piece with which the grid covers units one by one is at most
    // kStraddle pages longer than even shares (8 lists of 256 pages on 152 CTAs: 15
    // against 18 us).  The line then holds every unit rounded up to whole pieces.
    uint32_t chunk = even;
    bool whole_pieces = false;
    if (sum != 0 && (n_lists <= 32 || a.sel)) {
        auto count = [&](uint32_t c) -> uint32_t {        // pieces of c pages
            if (a.sel) return static_cast<uint32_t>(min(static_cast<uint64_t>(n_lists) * mult * ((a.n_sel + c - 1) / c), uint64_t(0x7fffffff)));
            return __reduce_add_sync(0xffffffffu, (np_lane + c - 1) / c) * mult;
        };
        uint32_t n = count(even);
        if (n > gridDim.x && count(even + kStraddle) <= gridDim.x) {
            uint32_t lo = even + 1, hi = even + kStraddle;
            while (lo < hi) {
                const uint32_t mid = (lo + hi) / 2;
                if (count(mid) <= gridDim.x) hi = mid;
                else lo = mid + 1;
            }
            chunk = hi;
            n = count(chunk);
        }
        whole_pieces = n <= gridDim.x;
        if (whole_pieces) total = n * chunk;
    }
    // a list's units on the line
    auto padded = [&](uint32_t np) { return whole_pieces ? (np + chunk - 1) / chunk * chunk : np; };
    const uint32_t pos0 = blockIdx.x * chunk, pos_end = min(total, pos0 + chunk);

    // lists without a page: their rows are written here
    if (!a.sel) {
        for (int i = blockIdx.x; i < n_lists; i += gridDim.x) {
            if ((n_lists <= 32 ? __shfl_sync(0xffffffffu, np_lane, i) : pages_of(a, i)) != 0) continue;
            const int64_t r0 = a.token(i, 0) * a.H, nr = static_cast<int64_t>(a.nq) * a.H;
            for (int64_t e = tid; e < nr * D; e += kThreads) {
                if (F16) static_cast<__half *>(a.o)[r0 * D + e] = __float2half(0.f);
                else static_cast<float *>(a.o)[r0 * D + e] = 0.f;
            }
            for (int64_t e = tid; e < nr; e += kThreads) a.lse[r0 + e] = -INFINITY;
        }
    }
    __syncthreads();                                // the barriers are ready
    if (pos0 >= pos_end) return;

    Place at = {0, 0, 0};
    if (a.sel) {
        at.np = padded(a.n_sel);
        at.list = static_cast<int>(pos0 / (at.np * mult));
        at.base = at.list * (at.np * mult);
    } else {
        uint32_t before = 0;
        for (int c0 = 0; c0 < n_lists; c0 += 32) {
            const uint32_t n = padded(c0 == 0 ? np_lane : c0 + lane < n_lists ? pages_of(a, c0 + lane) : 0u);
            uint32_t inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, (before + inc) * mult > pos0);
            if (hit) {
                const int f = __ffs(hit) - 1;
                at.list = c0 + f;
                at.np = __shfl_sync(0xffffffffu, n, f);
                at.base = (before + __shfl_sync(0xffffffffu, inc, f)) * mult - at.np * mult;
                break;
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
    }

    // The units of the piece in turn, for both roles: pages [pg0, pg1) of one unit.
    struct Unit {
        uint32_t u_in, unit0;                       // its number within the list; the line's position of its page 0
        uint32_t next;                              // the line's position behind what of it is in the piece
        int np, pg0, pg1, kh, rg, seq;              // np: its pages
        int64_t tok0;                               // token of its row 0
    };
    auto unit_at = [&](uint32_t pos) {
        while (pos >= at.base + at.np * mult) {     // the next list with pages
            at.base += at.np * mult;
            ++at.list;
            at.np = padded(pages_of(a, at.list));
        }
        Unit x;
        x.u_in = (pos - at.base) / at.np;
        x.unit0 = at.base + x.u_in * at.np;
        x.pg0 = static_cast<int>(pos - x.unit0);
        const uint32_t to = min(at.np, pos_end - x.unit0);
        x.next = x.unit0 + to;
        x.np = static_cast<int>(pages_of(a, at.list));
        x.pg1 = min(static_cast<int>(to), x.np);
        x.kh = static_cast<int>(x.u_in / a.row_groups);
        x.rg = static_cast<int>(x.u_in - x.kh * a.row_groups);
        x.seq = a.sel ? at.list / a.nq : at.list;
        x.tok0 = a.sel ? a.token(x.seq, at.list % a.nq) : a.token(at.list, 0);
        return x;
    };
    // A phase already complete is taken at once; the abort flag is read only
    // when the barrier is not ready.
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if (*reinterpret_cast<volatile int *>(&s_abort)) return false;
        if (tc::mbar_wait(bar, parity, &s_abort)) return true;
        s_abort = 1;
        atomicOr(a.L.status, 1);
        return false;
    };
    // keys that a row sees
    auto seen_by = [&](const Unit &x, int row, int len) {
        if (!a.q_pos) return len;
        const int qp = a.q_pos[x.tok0 + row / a.G];
        return qp < 0 ? 0 : (qp < len ? qp + 1 : len);
    };

    if (warp == W) {
        // ---------------- the fetching warp -----------------------------------
        uint32_t n_put = 0;                         // pages put into the ring so far
        bool ok = true;
        for (uint32_t pos = pos0; ok && pos < pos_end;) {
            const Unit x = unit_at(pos);
            const int len = static_cast<int>(list_len(a.L, x.seq));
            const int32_t *ids = a.L.ids + (static_cast<int64_t>(x.seq) * a.L.Hk + x.kh) * a.L.cap;
            const int32_t *sel = a.sel ? a.sel + (x.tok0 * a.L.Hk + x.kh) * a.n_sel : nullptr;
            int lim = len;                          // keys that any row of the unit sees
            if (a.q_pos) {
                const int row = x.rg * 8 * NC + lane;
                lim = lane < 8 * NC && row < a.rows ? seen_by(x, row, len) : 0;
                lim = __reduce_max_sync(0xffffffffu, lim);
            }
            auto load_meta = [&](int first) {
                Meta m = {-1, 0, 0.f, 0.f};
                const int p = first + lane;
                if (p < x.pg1) {
                    const int64_t blk = sel ? __ldg(sel + p) : p;
                    if (blk >= 0 && blk * kPage < lim) m.id = max(-1, checked_page(a.L, __ldg(ids + blk)));
                    m.blk = static_cast<int>(blk);
                    if (m.id >= 0) {
                        m.ks = __ldg(a.k_scale + m.id);
                        m.vs = __ldg(a.v_scale + m.id);
                    }
                }
                return m;
            };
            Meta nxt = load_meta(x.pg0);
            for (int first = x.pg0; ok && first < x.pg1; first += 32) {
                const Meta cur = nxt;
                if (first + 32 < x.pg1) nxt = load_meta(first + 32);
                const int n = min(32, x.pg1 - first);
                // the CTA's first pages go out before their scales are there, K and V by
                // neighbouring lanes (one lane took 60 ns a copy); they are announced below
                const int early = n_put == 0 ? min(n, NS) : 0;
                if (early) {                        // lanes 2i and 2i + 1: K and V of page i
                    static_assert(2 * NS <= 32, "a lane for each copy");
                    const int id = __shfl_sync(0xffffffffu, cur.id, lane >> 1);
                    if (lane < 2 * early && id >= 0) {
                        const uint32_t full = bar0 + 8 * (lane >> 1);
                        if ((lane & 1) == 0) tc::mbar_expect_tx_only(full, 2 * BYTES);
                        tc::tma_load_3d(smem_addr(ring + lane * BYTES), (lane & 1) ? &map_v : &map_k, 0, 0, id, full);
                    }
                }
                // (64 entries: those of the 32 pages before are still in use, at
                // most NS of them not taken yet)
                if (lane < n) s_meta[(n_put + lane) % 64] = Meta{cur.id, cur.blk, cur.ks * a.scale_log2, cur.vs};
                __syncwarp();
                // kBatch pages at a time, a lane for each copy (by one lane a page took 300 ns,
                // D = 64 more than its bytes: 50 us where two at a time take 44 and four 41)
                int done = 0;
                for (; done < n; done += kBatch) {
                    const int i = done + (lane >> 1);
                    const bool mine = lane < 2 * kBatch && i < n;
                    const uint32_t m = n_put + i, slot = m % NS, turn = m / NS;
                    const uint32_t full = bar0 + 8 * slot, empty = bar0 + 8 * (NS + slot);
                    ok = __all_sync(0xffffffffu, !mine || turn == 0 || wait(empty, (turn - 1) & 1));
                    if (!ok) break;
                    if (mine) {
                        const int id = s_meta[m % 64].id;
                        const bool copy = id >= 0 && i >= early;
                        if ((lane & 1) == 0) {
                            if (copy) tc::mbar_expect_tx(full, 2 * BYTES);
                            else tc::mbar_arrive(full);
                        }
                        if (copy)
                            tc::tma_load_3d(smem_addr(ring + (2 * slot + (lane & 1)) * BYTES), (lane & 1) ? &map_v : &map_k, 0, 0, id, full);
                    }
                    __syncwarp();
                }
                n_put += min(done, n);
            }
            pos = x.next;
        }
        if (!ok && lane == 0) {
            // copies in flight land before the CTA ends (bounded)
            for (uint32_t i = n_put > NS ? n_put - NS : 0; i < n_put; ++i)
                tc::mbar_wait(bar0 + 8 * (i % NS), (i / NS) & 1, nullptr, 100000000ull);
        }
        return;
    }

    // ---------------- the computing warps --------------------------------------
    const int g = lane >> 2, t = lane & 3;
    const int rg_ = D == 128 ? (g >> 1) | ((g & 1) << 2) : g;       // r(g), p(g)
    auto sync_all = [] { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); };
    // byte offsets of the thread's pieces in a page (see the header)
    uint32_t k_off[CH], v_off[2];
    if constexpr (D == 128) {
#pragma unroll
        for (int c = 0; c < CH; ++c) k_off[c] = rg_ * 128 + (((t + 4 * c) ^ rg_) << 4);
#pragma unroll
        for (int e = 0; e < 2; ++e) v_off[e] = (t + 4 * e) * 128 + ((rg_ ^ (t + 4 * e)) << 4);
    } else {
        k_off[0] = g * 64 + ((t ^ (g >> 1)) << 4);
#pragma unroll
        for (int e = 0; e < 2; ++e) v_off[e] = (2 * t + e) * 64 + (((g >> 1) ^ t) << 4) + (g & 1) * 8;
    }
    uint32_t n_taken = 0;                           // half pages of the CTA's earlier units
    for (uint32_t pos = pos0; pos < pos_end;) {
        const Unit x = unit_at(pos);
        const int row0 = x.rg * 8 * NC;
        const int len = static_cast<int>(list_len(a.L, x.seq));
        auto out_row = [&](int row) { return (x.tok0 + row / a.G) * a.H + x.kh * a.G + row % a.G; };
        auto page_lse = [&](int row) {              // log sums of a row's pages
            const int64_t r = a.sel ? (at.list % a.nq) * static_cast<int64_t>(a.G) + row : row;
            return a.page_lse + ((static_cast<int64_t>(x.seq) * a.L.Hk + x.kh) * a.nq * a.G + r) * a.page_ld;
        };
        // query fragments into shared memory: lane (g, t) of k-step (c, w) holds
        // channels 64c + 16t + 4w .. + 3 of column g
        for (int i = tid; i < NC * KS * 32; i += kConsumers) {
            const int row = row0 + i / (KS * 32) * 8 + ((i & 31) >> 2);
            const int ks = i / 32 % KS;
            uint2 v = make_uint2(0, 0);
            if (row < a.rows)
                v = __ldg(reinterpret_cast<const uint2 *>(a.q + out_row(row) * D + 64 * (ks >> 2) + 16 * (i & 3) + 4 * (ks & 3)));
            s_q[i] = v;
        }
        int lim[NC][2];                             // keys that columns 2t, 2t+1 see
        int lim_min = len;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = row0 + j * 8 + 2 * t + e;
                lim[j][e] = r < a.rows ? seen_by(x, r, len) : len;
                lim_min = min(lim_min, lim[j][e]);
            }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));
        sync_all();                                 // s_q is written

        float m_ref[NC][2], l_sum[NC][2], acc[NC][MT][4];
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            m_ref[j][0] = m_ref[j][1] = -INFINITY;
            l_sum[j][0] = l_sum[j][1] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][i][e] = 0.f;
        }

        const uint32_t n_end = n_taken + 2 * (x.pg1 - x.pg0);
        for (uint32_t n = n_taken + (warp + W - n_taken % W) % W; n < n_end; n += W) {
            const uint32_t m = n >> 1, slot = m % NS;   // (units begin at even n)
            const int p = x.pg0 + static_cast<int>((n - n_taken) >> 1), h = n & 1;
            // (the warp goes one way: what follows are its products and shuffles)
            const uint32_t full = bar0 + 8 * slot, turn = (m / NS) & 1;
            bool there = __all_sync(0xffffffffu, tc::mbar_try_wait(full, turn));
            if (!there) there = __all_sync(0xffffffffu, wait(full, turn));
            const Meta meta = s_meta[m % 64];
            if (!there || meta.id < 0) {
                if (a.page_lse && lane < 8 * NC && row0 + lane < a.rows) page_lse(row0 + lane)[2 * p + h] = -INFINITY;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar0 + 8 * (NS + slot));
                continue;
            }
            const uint8_t *pk = ring + slot * 2 * BYTES + h * (kStep * D), *pv = pk + BYTES;
            const int key0 = meta.blk * kPage + h * kStep;   // (blk * 64 is below len)
            // (a zero scale as a tiny one, so that its product with a masked -inf stays one)
            const float ks = fmaxf(fabsf(meta.ks), 1e-30f), vs = meta.vs;
            const bool masked = lim_min - key0 < kStep;
            {
                // S = K Q^T of 32 keys
                float s[NC][2][4];
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    uint4 kr[2][2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr)
                            kr[i][rr] = *reinterpret_cast<const uint4 *>(pk + (16 * i + 8 * rr) * D + k_off[c]);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint2 qf[NC];
#pragma unroll
                        for (int j = 0; j < NC; ++j) qf[j] = s_q[(j * KS + c * 4 + w) * 32 + lane];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t lo = word(kr[i][0], w) ^ 0x80808080u, hi = word(kr[i][1], w) ^ 0x80808080u;
                            const uint32_t a0 = codes_lo(lo), a1 = codes_lo(hi), a2 = codes_hi(lo), a3 = codes_hi(hi);
#pragma unroll
                            for (int j = 0; j < NC; ++j) {
                                if (c == 0 && w == 0) mma_16816_from0(s[j][i], a0, a1, a2, a3, qf[j].x, qf[j].y);
                                else mma_16816(s[j][i], a0, a1, a2, a3, qf[j].x, qf[j].y);
                            }
                        }
                    }
                }
                if (meta.ks < 0.f || masked) {
#pragma unroll
                    for (int j = 0; j < NC; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (meta.ks < 0.f) s[j][i][e] = -s[j][i][e];
                                if (16 * i + 8 * (e >> 1) + rg_ >= lim[j][e & 1] - key0) s[j][i][e] = -INFINITY;
                            }
                }
                float l_step[NC][2];
                uint32_t bh[NC][2][2], bl[NC][2][2];
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    // largest scores, in log2 units
                    float top[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        top[e] = fmaxf(fmaxf(s[j][0][e], s[j][0][e + 2]), fmaxf(s[j][1][e], s[j][1][e + 2])) * ks;
                    // m_ref + kGrow is -inf at first, and then any score moves it
                    if (__any_sync(0xffffffffu, top[0] > m_ref[j][0] + kGrow || top[1] > m_ref[j][1] + kGrow)) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float y = top[e];
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
                            if (y > m_ref[j][e] + kGrow) {
                                const float b = fast_exp2(m_ref[j][e] - y);
                                m_ref[j][e] = y;
                                l_sum[j][e] *= b;
#pragma unroll
                                for (int i = 0; i < MT; ++i) {
                                    acc[j][i][e] *= b;
                                    acc[j][i][e + 2] *= b;
                                }
                            }
                        }
                    }
                    float off[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        off[e] = m_ref[j][e] == -INFINITY ? 0.f : kShift - m_ref[j][e];
                        l_step[j][e] = 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float w[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                w[e] = fast_exp2(fmaf(s[j][i][half * 2 + e], ks, off[e]));
                                l_step[j][e] += w[e];
                            }
                            const uint32_t hw = pack_half2(w[0], w[1]);
                            bh[j][i][half] = movmatrix_trans(hw);
                            if (HILO) {
                                const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hw));
                                bl[j][i][half] = movmatrix_trans(pack_half2(w[0] - back.x, w[1] - back.y));
                            }
                        }
                    l_sum[j][0] += l_step[j][0];
                    l_sum[j][1] += l_step[j][1];
                }
                if (a.page_lse) {
#pragma unroll
                    for (int j = 0; j < NC; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float y = l_step[j][e];
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                            const int row = row0 + j * 8 + 2 * t + e;
                            if (g == 0 && row < a.rows)
                                page_lse(row)[2 * p + h] = y > 0.f ? m_ref[j][e] - kShift + log2f(y) : -INFINITY;
                        }
                }
                // O^T += d_v V^T P^T: 32 keys' sums from zero, then one fp32 addition.
                // B's rows 2t, 2t+1 (+ 8) are keys r(2t), r(2t+1) (+ 8).
                uint32_t vr[2][4][VW];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int rr = 0; rr < 4; ++rr) {
                        const uint8_t *src = pv + (16 * i + 8 * (rr >> 1)) * D + v_off[rr & 1];
                        if constexpr (VW == 4) {
                            const uint4 y = *reinterpret_cast<const uint4 *>(src);
                            vr[i][rr][0] = y.x;
                            vr[i][rr][1] = y.y;
                            vr[i][rr][2] = y.z;
                            vr[i][rr][3] = y.w;
                        } else {
                            const uint2 y = *reinterpret_cast<const uint2 *>(src);
                            vr[i][rr][0] = y.x;
                            vr[i][rr][1] = y.y;
                        }
                    }
                __syncwarp();                       // the slot is read
                if (lane == 0) tc::mbar_arrive(bar0 + 8 * (NS + slot));
#pragma unroll
                for (int w = 0; w < VW; ++w)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // channels (D/8) p(g) + 4w + 2e (m = g) and + 1 (m = g + 8)
                        float y[NC][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t p01 = __byte_perm(vr[i][0][w], vr[i][1][w], e ? 0x7362 : 0x5140) ^ 0x80808080u;
                            const uint32_t p89 = __byte_perm(vr[i][2][w], vr[i][3][w], e ? 0x7362 : 0x5140) ^ 0x80808080u;
                            const uint32_t a0 = codes_lo(p01), a1 = codes_hi(p01);
                            const uint32_t a2 = codes_lo(p89), a3 = codes_hi(p89);
#pragma unroll
                            for (int j = 0; j < NC; ++j) {
                                if (i == 0) mma_16816_from0(y[j], a0, a1, a2, a3, bh[j][i][0], bh[j][i][1]);
                                else mma_16816(y[j], a0, a1, a2, a3, bh[j][i][0], bh[j][i][1]);
                                if (HILO) mma_16816(y[j], a0, a1, a2, a3, bl[j][i][0], bl[j][i][1]);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < NC; ++j)
#pragma unroll
                            for (int c = 0; c < 4; ++c) acc[j][2 * w + e][c] = fmaf(vs, y[j][c], acc[j][2 * w + e][c]);
                    }
            }
        }
        n_taken = n_end;

        // The warps' results for column group j, as they stand in shared memory, to the
        // result or to a piece's slot.
        auto join = [&](int j, bool final, int64_t slot) {
            for (int i = tid; i < 8 * D; i += kConsumers) {
                const int c = i / D, d = i % D;
                const int row = row0 + j * 8 + c;
                if (row >= a.rows) continue;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < W; ++w) M = fmaxf(M, s_ml[w][c][0]);
                float Lw = 0.f, O = 0.f;
                if (M != -INFINITY) {
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float b = fast_exp2(s_ml[w][c][0] - M);
                        Lw = fmaf(b, s_ml[w][c][1], Lw);
                        O = fmaf(b, s_o[w][c][d], O);
                    }
                }
                if (final) {
                    const int64_t r = out_row(row);
                    const float v = Lw == 0.f ? 0.f : O / Lw;
                    if (F16) static_cast<__half *>(a.o)[r * D + d] = __float2half_rn(v);
                    else static_cast<float *>(a.o)[r * D + d] = v;
                    if (d == 0) a.lse[r] = Lw == 0.f ? -INFINITY : (M - kShift + log2f(Lw)) * 0.6931471805599453f;
                } else {
                    a.part_o[(slot * (8 * NC) + j * 8 + c) * D + d] = O;
                    if (d == 0) {
                        a.part_ml[(slot * (8 * NC) + j * 8 + c) * 2] = M;
                        a.part_ml[(slot * (8 * NC) + j * 8 + c) * 2 + 1] = Lw;
                    }
                }
            }
        };
        // ---- the warps' results together, eight columns at a time ---------------
        const bool whole = x.pg0 == 0 && x.pg1 == x.np;
        const int64_t slot_out = 2 * static_cast<int64_t>(blockIdx.x) + (pos == pos0 ? 0 : 1);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            if (j > 0) sync_all();                  // the buffers of the last round are read
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float y = l_sum[j][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if (g == 0) {
                    s_ml[warp][2 * t + e][0] = y == y ? m_ref[j][e] : INFINITY;   // (a NaN stays one in every sum)
                    s_ml[warp][2 * t + e][1] = y;
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)        // channels (D/8) p(g) + 2i, + 1
                    *reinterpret_cast<float2 *>(&s_o[warp][2 * t + e][(D / 8) * rg_ + 2 * i]) =
                        make_float2(acc[j][i][e], acc[j][i][e + 2]);
            }
            sync_all();
            join(j, whole, slot_out);
        }
        if (!whole) {
            // ---- the last CTA of the unit puts the pieces together, in order: each
            // warp some of them, then the warps' results as above
            const uint32_t u = at.list * mult + x.u_in;
            const uint32_t c_lo = x.unit0 / chunk, c_hi = (x.unit0 + at.np - 1) / chunk;
            __threadfence();
            sync_all();
            if (tid == 0) s_last = atomicAdd(a.counters + u, 1) == static_cast<int>(c_hi - c_lo);
            sync_all();
            if (s_last) {
                __threadfence();
                constexpr int CPI = 128 / D;        // columns a warp reads at once
                const int sub = lane / (D / 4), d4 = lane % (D / 4);
#pragma unroll 1
                for (int j = 0; j < NC; ++j) {
                    float M[8 / CPI], L[8 / CPI], O[8 / CPI][4];
#pragma unroll
                    for (int c = 0; c < 8 / CPI; ++c) {
                        M[c] = -INFINITY;
                        L[c] = O[c][0] = O[c][1] = O[c][2] = O[c][3] = 0.f;
                    }
#pragma unroll 1
                    for (uint32_t y = c_lo + warp; y <= c_hi; y += W) {
                        const int64_t sl = 2 * static_cast<int64_t>(y) + (y == c_lo && x.unit0 > c_lo * chunk ? 1 : 0);
                        float2 ml[8 / CPI];
                        float4 v[8 / CPI];
#pragma unroll
                        for (int c = 0; c < 8 / CPI; ++c) {
                            const int64_t at_c = sl * (8 * NC) + j * 8 + c * CPI + sub;
                            const bool on = row0 + j * 8 + c * CPI + sub < a.rows;
                            ml[c] = on ? __ldcg(reinterpret_cast<const float2 *>(a.part_ml) + at_c) : make_float2(-INFINITY, 0.f);
                            v[c] = on ? __ldcg(reinterpret_cast<const float4 *>(a.part_o + at_c * D) + d4) : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
#pragma unroll
                        for (int c = 0; c < 8 / CPI; ++c) {
                            const float m = fmaxf(M[c], ml[c].x);
                            const float bo = M[c] == -INFINITY ? 0.f : fast_exp2(M[c] - m);
                            const float bn = ml[c].x == -INFINITY ? 0.f : fast_exp2(ml[c].x - m);
                            M[c] = m;
                            L[c] = L[c] * bo + bn * ml[c].y;
                            O[c][0] = O[c][0] * bo + bn * v[c].x;
                            O[c][1] = O[c][1] * bo + bn * v[c].y;
                            O[c][2] = O[c][2] * bo + bn * v[c].z;
                            O[c][3] = O[c][3] * bo + bn * v[c].w;
                        }
                    }
                    if (j > 0) sync_all();
#pragma unroll
                    for (int c = 0; c < 8 / CPI; ++c) {
                        const int col = c * CPI + sub;
                        if (d4 == 0) {
                            s_ml[warp][col][0] = M[c];
                            s_ml[warp][col][1] = L[c];
                        }
                        *reinterpret_cast<float4 *>(&s_o[warp][col][d4 * 4]) = make_float4(O[c][0], O[c][1], O[c][2], O[c][3]);
                    }
                    sync_all();
                    join(j, true, 0);
                }
                if (tid == 0) a.counters[u] = 0;
            }
        }
        pos = x.next;
    }
}

// Attention weight of each page from its halves' log sums: mass += sum over rows
// of 2^(half page - row).  Rows are added in their order.
__global__ void __launch_bounds__(128) mass_kernel(const AttnArgs a, float *mass)
{
    start();
    const int kh = blockIdx.y, s = blockIdx.z;
    const int64_t unit = static_cast<int64_t>(s) * a.L.Hk + kh;
    const int rows = a.nq * a.G;
    const int64_t len = list_len(a.L, s);
    const float *pl = a.page_lse + unit * rows * a.page_ld;
    float *out = mass + unit * a.L.cap;
    auto lse2 = [&](int r) {
        return a.lse[a.token(s, r / a.G) * a.H + kh * a.G + r % a.G] * 1.4426950408889634f;
    };
    if (!a.sel) {
        const int64_t p = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
        if (p * kPage >= len) return;
        float sum = 0.f;
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
            const float z = lse2(r);
            const float2 x = __ldcg(reinterpret_cast<const float2 *>(pl + r * a.page_ld) + p);
            sum += z == -INFINITY ? 0.f : fast_exp2(x.x - z) + fast_exp2(x.y - z);
        }
        out[p] += sum;
        return;
    }
    // with a selection: token by token (a token's pages are different ones, or
    // the same page with the same weight: the order of their additions is free)
    for (int t = 0; t < a.nq; ++t) {
        const int32_t *sel = a.sel + (a.token(s, t) * a.L.Hk + kh) * a.n_sel;
        for (int i = threadIdx.x; i < a.n_sel; i += 128) {
            const int64_t blk = sel[i];
            if (blk < 0 || blk * kPage >= len) continue;
            float sum = 0.f;
            for (int g = 0; g < a.G; ++g) {
                const float z = lse2(t * a.G + g);
                const float2 x = __ldcg(reinterpret_cast<const float2 *>(pl + (t * a.G + g) * a.page_ld) + i);
                sum += z == -INFINITY ? 0.f : fast_exp2(x.x - z) + fast_exp2(x.y - z);
            }
            if (sum != 0.f) atomicAdd(out + blk, sum);
        }
        __syncthreads();
    }
}

int launch_mass(skv_handle *h, const AttnArgs &a, float *mass, cudaStream_t st)
{
    const unsigned bx = a.sel ? 1u : static_cast<unsigned>((a.L.cap + 127) / 128);
    return cuda_fail(h, launch(mass_kernel, dim3(bx, a.L.Hk, a.L.S), 128, 0, st, a, mass), "page weight launch");
}

int page_map(skv_handle *h, CUtensorMap *map, const int8_t *pages, int64_t n_pages, int D, int rows)
{
    tc::EncodeTiledFn fn = tc::encode_fn();
    if (!fn) return fail(h, SKV_ECUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), kPage, static_cast<cuuint64_t>(n_pages)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(D) * kPage};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t *>(pages), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(h, SKV_EUNSUPPORTED, "tensor map encoding failed (%d)", static_cast<int>(r));
    return SKV_OK;
}

template <int D, int NC, bool HILO, bool F16>
static int launch_one(skv_handle *h, const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int grid,
                      cudaStream_t st)
{
    static KernelAttrCache cache;
    constexpr int smem = decode_smem<D, NC>();
    const cudaError_t e = kernel_smem_optin(cache, reinterpret_cast<const void *>(decode_kernel<D, NC, HILO, F16>), smem,
                                            warps_of(D, NC) * 32 + 32, nullptr);
    if (e != cudaSuccess) return cuda_fail(h, e, "cudaFuncSetAttribute(8-bit decode)");
    if (h->prof_before) cudaEventRecord(h->prof_before, st);
    const cudaError_t l = launch(decode_kernel<D, NC, HILO, F16>, dim3(grid), warps_of(D, NC) * 32 + 32, smem, st, mk, mv, a);
    if (h->prof_after) cudaEventRecord(h->prof_after, st);
    return cuda_fail(h, l, "8-bit decode launch");
}

template <int D>
static int launch_d(skv_handle *h, const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, bool f16, int grid,
                    int nc, cudaStream_t st)
{
    // One column group always takes both parts of the weights (its products are
    // a small part of a page's time); two of them only when o is fp32.  For fp16 results the
    // second part would cost 7 to 13 % (four tokens of eight sequences over 16000 keys, D = 128:
    // 68.1 -> 75.1 us, D = 64: 46.1 -> 49.3; eight tokens over 32768: 39.5 -> 44.6) to take away an
    // error as large as the result's own rounding.
    if (nc == 1)
        return f16 ? launch_one<D, 1, true, true>(h, mk, mv, a, grid, st)
                   : launch_one<D, 1, true, false>(h, mk, mv, a, grid, st);
    return f16 ? launch_one<D, 2, false, true>(h, mk, mv, a, grid, st)
               : launch_one<D, 2, true, false>(h, mk, mv, a, grid, st);
}

int launch_decode(skv_handle *h, const AttnArgs &a, int64_t n_pages, int D, bool f16, int grid, int nc, cudaStream_t st)
{
    CUtensorMap mk, mv;
    int rc = page_map(h, &mk, a.k, n_pages, D, kPage);
    if (rc || (rc = page_map(h, &mv, a.v, n_pages, D, kPage))) return rc;
    return D == 128 ? launch_d<128>(h, mk, mv, a, f16, grid, nc, st) : launch_d<64>(h, mk, mv, a, f16, grid, nc, st);
}

}  // namespace q8
}  // namespace skv
