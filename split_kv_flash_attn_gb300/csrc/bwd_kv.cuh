// bwd_kv.cuh -- dk and dv: a CTA owns 128 keys of a KV head (TMEM lanes) and walks over
// the query tiles that see one of them.
//
//   S^T  = K Q^T        [128 keys x 128 rows]   dP^T = V dO^T
//   P^T  = 2^(S c - L)  over S in tensor memory, dS^T = P^T (dP^T sigma - D) over dP
//   dV  += P^T dO       dK  += dS^T Q           (A from tensor memory)
// Q and dO tiles are each the K-major B operand of one product and the MN-major one of the
// other: one TMA load serves both.  Tensor memory is full: S, dP, dV, dK of 128 columns
// (D = 64: two of 64).  So S and dP have one buffer each, and the tensor core turns
// from one to the other: while the compute warps form P(j) it runs dK(j-1), dP(j), and
// while they form dS(j) it runs dV(j), S(j+1).
//
// Warps: 0-15 compute (32 rows of the tile and 32 keys each), 16 TMA, 17 issues dV(j) and
// S(j+1), 18 dK(j) and dP(j+1), in turns, so that S(j+1), which the compute warps wait
// for, does not stand behind dP; a thread's products run in order, so that their buffers
// need no further wait.  The turn passes before a thread's last two products go out, and
// its waits for operands fall into the other's turn; the compute warps' arrival is waited for last, since
// a wait costs some hundred clocks even for what is there.  A whole warp runs this code and one lane issues by a
// predicate, so that descriptors stay in uniform registers.  19 looks each tile over when it has landed: it
// folds the powers of two into -L and -D, tells whether the tile needs a mask, and clears rows of
// tokens that see nothing, whatever they hold.
//
// Measured, dk and dv of 16384 x 16384, 8 heads on 2, no mask: 1588 us, 1385 TFLOP/s of the four products (70 % of
// the measured fp16 rate); the compute warps waited for first 1715, and no turns besides 1828.  Bound by the chain
// S -> P -> dV, S and dP -> dS -> dK, dP: each half of it is about as long as the two products that run beside it.
// Halves of a tile (products of 64 columns), which would shorten the links, took 8 % more.
//
// Every mbarrier wait is bounded, as in the prefill kernel.  Whoever gives up, and when: at the end of a stretch all loads
// asked for and all products issued are waited for before the CTA leaves, by waits that look at no status word; what they
// wait for ends by itself.
#pragma once

#include "bwd.cuh"

namespace skv {
namespace bwd {
namespace kv {

constexpr int kStages = 2;
constexpr int kHalf = kTile * 128;                           // a 64-column block of a tile

template <int D>
struct Lay {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kTileBytes;
    static constexpr int kOffQ = 2 * kTileBytes;
    static constexpr int kOffO = kOffQ + kStages * kTileBytes;
    static constexpr int kOffInfo = kOffO + kStages * kTileBytes;
    static constexpr int kOffBits = kOffInfo + kStages * kInfoBytes;      // bitmap of visited query tiles
    static constexpr int kOffList = kOffBits + kMaxQTiles / 8;
    static constexpr int kOffBar = kOffList + kStretch * 4;
    static constexpr int kBytes = kOffBar + 256 + 1024;                   // + alignment
};
static_assert(Lay<128>::kBytes <= 226 * 1024, "shared memory per CTA");

enum { B_KV, B_QLAND, B_QFULL = B_QLAND + kStages, B_QEMPTY = B_QFULL + kStages, B_OLAND = B_QEMPTY + kStages,
       B_OFULL = B_OLAND + kStages, B_OEMPTY = B_OFULL + kStages, B_S = B_OEMPTY + kStages, B_P, B_DP, B_DS, B_TURN,
       B_ACC = B_TURN + 2, B_COUNT = B_ACC + 2 };
static_assert(B_COUNT * 8 <= 256, "barrier area");

// Tensor memory columns.
constexpr int kColS = 0, kColP = 128, kColV = 256;

// TWO: p and ds in two fp16 parts each (bwd.cuh).
template <int D, bool TWO>
__device__ __forceinline__ void run(const CUtensorMap &tq, const CUtensorMap &to, const CUtensorMap &tk, const CUtensorMap &tv,
                                    const MainArgs &a, int unit, int piece, uint8_t *smem_raw)
{
    using L = Lay<D>;
    constexpr int kColK = kColV + D;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_addr(sm);
    auto bar = [&](int i) { return sbase + L::kOffBar + 8u * static_cast<uint32_t>(i); };
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_count, s_lim, s_eN, s_eD, s_c, s_ew;
    __shared__ int s_need[kStages], s_loads[2];
    uint32_t *bits = reinterpret_cast<uint32_t *>(sm + L::kOffBits);
    int *s_list = reinterpret_cast<int *>(sm + L::kOffList);       // a stretch's query tiles

    const Geo &g = a.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // key tile slowest: under causal positions the first keys have the most rows
    const int heads = g.Hk * g.groups;
    const int kt = unit / heads, gh = unit - kt * heads;
    const int group = gh / g.Hk, hk = gh - group * g.Hk;
    const int64_t j0 = static_cast<int64_t>(kt) * kTile;
    const int64_t tile0 = static_cast<int64_t>(gh) * g.QT;
    const int box_rows = g.Gb * g.Tb;

    if (tid == 0) {
        s_abort = 0;
        s_count = 0;
        s_lim = 0;
        s_eN = s_eD = kNoExp;
        s_c = -1000;
        s_ew = -100;
    }
    if (warp == 0) {
        tc::tmem_alloc<512>(smem_addr(&s_tmem));
        tc::tmem_relinquish();
    }
    if (tid == kCompute) {
        tc::mbar_init(bar(B_KV), 1);
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(bar(B_QLAND + i), 1);
            tc::mbar_init(bar(B_QFULL + i), 32);
            tc::mbar_init(bar(B_QEMPTY + i), 1);
            tc::mbar_init(bar(B_OLAND + i), 1);
            tc::mbar_init(bar(B_OFULL + i), 32);
            tc::mbar_init(bar(B_OEMPTY + i), 2);             // dP and dV of the tile
        }
        tc::mbar_init(bar(B_S), 1);
        tc::mbar_init(bar(B_P), kCompute);
        tc::mbar_init(bar(B_DP), 1);
        tc::mbar_init(bar(B_DS), kCompute);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(B_TURN + i), 1);
            tc::mbar_init(bar(B_ACC + i), 1);
        }
        tc::fence_barrier_init();
        // the keys' tiles, while the query tiles are looked through
        tc::mbar_expect_tx(bar(B_KV), 2 * L::kTileBytes);
        for (int b = 0; b < D / 64; ++b) {
            tc::tma_load_3d(sbase + L::kOffK + b * kHalf, &tk, hk * D + 64 * b, static_cast<int>(j0), group, bar(B_KV));
            tc::tma_load_3d(sbase + L::kOffV + b * kHalf, &tv, hk * D + 64 * b, static_cast<int>(j0), group, bar(B_KV));
        }
        tc::prefetch_tmap(&tq);
        tc::prefetch_tmap(&to);
    }
    const int key_lane = (warp & 3) * 32 + lane;             // compute threads: their key
    const int64_t key = j0 + key_lane;
    const int key_exp = warp < kCompute / 32 ? a.ew[(static_cast<int64_t>(gh) * g.KT + kt) * kTile + key_lane] : kAbsent;
    __syncthreads();
    // ---- the query tiles that see one of these keys, and their sizes ----
    {
        int n = 0, lim = 0, eN = kNoExp, eD = kNoExp, c = -1000;
        for (int b = 0; b < g.QT; b += kThreads) {
            const int i = b + tid;
            int4 s = make_int4(0, 0, 0, 0);
            if (i < g.QT) s = __ldg(reinterpret_cast<const int4 *>(a.sum + tile0 + i));
            const bool seen = i < g.QT && s.x > j0;
            const uint32_t w = __ballot_sync(0xffffffffu, seen);
            if (lane == 0 && b + warp * 32 < g.QT) bits[(b >> 5) + warp] = w;
            if (seen) {
                ++n;
                lim = max(lim, s.x);
                eN = max(eN, s.y);
                eD = max(eD, s.z);
                c = max(c, s.w);
            }
        }
        n = __reduce_add_sync(0xffffffffu, n);
        lim = __reduce_max_sync(0xffffffffu, lim);
        eN = __reduce_max_sync(0xffffffffu, eN);
        eD = __reduce_max_sync(0xffffffffu, eD);
        c = __reduce_max_sync(0xffffffffu, c);
        if (lane == 0) {
            atomicAdd(&s_count, n);
            atomicMax(&s_lim, lim);
            atomicMax(&s_eN, eN);
            atomicMax(&s_eD, eD);
            atomicMax(&s_c, c);
        }
        // rows that no TMA box writes
        for (int i = tid; i < (kTile - box_rows) * (D / 8) * 2 * kStages; i += kThreads) {
            const int per = (kTile - box_rows) * (D / 8);
            const int buf = i / per, x = i - buf * per, r = box_rows + x / (D / 8), ch = x % (D / 8);
            *reinterpret_cast<uint4 *>(sm + L::kOffQ + buf * L::kTileBytes + (ch >> 3) * kHalf + r * 128 + (ch & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem;
    const bool there = key < min(g.n, static_cast<int64_t>(s_lim)) && key_exp != kAbsent;
    if (there && warp < 4) atomicMax(&s_ew, key_exp);
    const int any = __syncthreads_or(there);
    const int cmax = s_c > -1000 ? s_c : 0;
    // 2^E bounds |d_o.v - delta| of these rows and keys
    const int E = max(max(s_eN + s_ew, s_eD) + 1, cmax - 100);
    const int sig_e = max(-100, min(100, cmax - E));
    const float sigma = pow2(sig_e);
    const int count = any ? s_count : 0;
    const int o_lo = static_cast<int>(static_cast<int64_t>(count) * piece / a.pieces);
    const int o_hi = static_cast<int>(static_cast<int64_t>(count) * (piece + 1) / a.pieces);

    auto wait = [&](int b, uint32_t parity) -> bool {
        if (tc::mbar_try_wait(bar(b), parity)) return true;
        if (*reinterpret_cast<volatile int *>(&s_abort)) return false;
        if (bounded_wait(bar(b), parity, a.status)) return true;
        s_abort = 1;
        atomicOr(a.status, 1);
        return false;
    };

    constexpr int NC = D / kParts;                           // result columns of a compute thread
    const int part = warp >> 2;                              // its part of a tile's rows, and of the results' columns
    // (where this thread's results go; worked out where they are stored: registers are short in between)
    auto out_at = [&]() { return ((group * g.n + key) * g.Hk + hk) * D + part * NC; };
    auto slot_of = [&](int which) {                          // dk's fp32 sums, then dv's
        return a.slot + (static_cast<int64_t>(piece) * 2 + which) * (static_cast<int64_t>(g.groups) * g.n * g.Hk * D) + out_at();
    };

    if (o_lo >= o_hi && tid == kCompute) tc::mbar_wait(bar(B_KV), 0, nullptr, kDrainNs);   // the loads land before the CTA leaves
    if (o_lo >= o_hi && warp < kCompute / 32 && key < g.n) {             // nobody sees these keys
        float z[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) z[i] = 0.f;
        if (a.pieces > 1) {
            store_row<NC>(slot_of(0), 0, SKV_F32, z);
            store_row<NC>(slot_of(1), 0, SKV_F32, z);
        } else {
            store_row<NC>(a.out0, out_at(), a.g_type, z);
            store_row<NC>(a.out1, out_at(), a.g_type, z);
        }
    }

    int it0 = 0, stretch = 0;
    for (int o = o_lo; o < o_hi; o += kStretch, ++stretch) {
        const int nt = min(kStretch, o_hi - o);
        if (warp == 0) {                                     // the tiles of ordinals o .. o + nt - 1
            int before = 0;
            const int words = (g.QT + 31) >> 5;
            for (int w0 = 0; w0 < words && before < o + nt; w0 += 32) {
                uint32_t w = w0 + lane < words ? bits[w0 + lane] : 0;
                int pre = __popc(w);
                const int mine = pre;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, pre, d);
                    if (lane >= d) pre += x;
                }
                const int all = __shfl_sync(0xffffffffu, pre, 31);
                int ord = before + pre - mine;
                while (w) {
                    const int b = __ffs(w) - 1;
                    w &= w - 1;
                    if (ord >= o && ord < o + nt) s_list[ord - o] = (w0 + lane) * 32 + b;
                    ++ord;
                }
                before += all;
            }
        }
        __syncthreads();

        if (warp == kCompute / 32) {
            // ---------------- TMA ----------------------------------------
            if (lane == 0) {
                const uint32_t box = static_cast<uint32_t>(box_rows) * D * 2;
                int q_out = 0, o_out = 0;                    // loads issued in this stretch
                for (int i = 0; i < nt; ++i) {
                    const int it = it0 + i, st = it & (kStages - 1), ph = (it / kStages) & 1;
                    const int qt = s_list[i];
                    const QTile t = q_tile(g, group, hk, qt);
                    if (it >= kStages && !wait(B_QEMPTY + st, ph ^ 1)) break;
                    tc::mbar_expect_tx(bar(B_QLAND + st), box + kInfoBytes);
                    for (int b = 0; b < D / 64; ++b)
                        tc::tma_load_5d(sbase + L::kOffQ + st * L::kTileBytes + b * kHalf, &tq, 64 * b, t.g0, hk,
                                        static_cast<int>(t.t0), group, bar(B_QLAND + st));
                    tc::bulk_load(sbase + L::kOffInfo + st * kInfoBytes, a.info + (tile0 + qt) * (kInfoRows * kTile), kInfoBytes,
                                  bar(B_QLAND + st));
                    ++q_out;
                    if (it >= kStages && !wait(B_OEMPTY + st, ph ^ 1)) break;
                    tc::mbar_expect_tx(bar(B_OLAND + st), box);
                    for (int b = 0; b < D / 64; ++b)
                        tc::tma_load_5d(sbase + L::kOffO + st * L::kTileBytes + b * kHalf, &to, 64 * b, t.g0, hk,
                                        static_cast<int>(t.t0), group, bar(B_OLAND + st));
                    ++o_out;
                }
                s_loads[0] = it0 + q_out;
                s_loads[1] = it0 + o_out;
            }
        } else if (warp == kCompute / 32 + 1 || warp == kCompute / 32 + 2) {
            // ---------------- products: dV(j), S(j+1), and dK(j), dP(j+1) ----
            {
                const uint32_t one = tc::elect_one();        // the lane that issues; all of the warp waits
                const bool second = warp == kCompute / 32 + 2;
                constexpr uint32_t kIdescS = tc::idesc_f16(kTile, kTile, false);
                constexpr uint32_t kIdescV = tc::idesc_f16(kTile, D, true);
                // S = K Q^T or dP = V dO^T (both operands K-major); dV = P^T dO or dK = dS^T Q (B MN-major)
                const uint64_t da = tc::smem_desc(sbase + (second ? L::kOffV : L::kOffK), 16, 1024);
                const uint64_t db = tc::smem_desc(sbase + (second ? L::kOffO : L::kOffQ), 16, 1024);
                const uint64_t dn = tc::smem_desc(sbase + (second ? L::kOffQ : L::kOffO), kHalf, 1024);
                const uint32_t col = tmem + (second ? kColP : kColS), acc = tmem + (second ? kColK : kColV);
                const int b_in = second ? B_OFULL : B_QFULL, b_in2 = second ? B_QFULL : B_OFULL;
                const int b_out = second ? B_DP : B_S, b_ready = second ? B_DS : B_P;
                const int b_mine = second ? B_TURN : B_TURN + 1, b_other = second ? B_TURN + 1 : B_TURN;
                auto scores = [&](int it, bool pass) {
                    const int st = it & (kStages - 1);
                    if (!__all_sync(0xffffffffu, wait(b_in + st, (it / kStages) & 1))) return false;
                    tc::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                        if (pass && one && kk == D / 16 - 2) tc::mbar_arrive(bar(b_other));   // ahead of the end of its wait
                        tc::mma_f16_ss_if(one, col, tc::desc_add(da, off), tc::desc_add(db, st * L::kTileBytes + off), kIdescS, kk > 0);
                    }
                    tc::mma_commit_if(one, bar(b_out));
                    if (second) tc::mma_commit_if(one, bar(B_OEMPTY + st));
                    return true;
                };
                bool ok = __all_sync(0xffffffffu, wait(B_KV, 0)) && scores(it0, second);   // (the first dV goes first)
                for (int i = 0; ok && i < nt; ++i) {
                    const int it = it0 + i, st = it & (kStages - 1);
                    // what is there early first: the compute warps' arrival is then the last wait before the products
                    ok = wait(b_mine, it & 1) && wait(b_in2 + st, (it / kStages) & 1) && wait(b_ready, it & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        tc::mma_f16_ts_if(one, acc, col + (kk & 1) * 8 + (kk >> 1) * kCols, tc::desc_add(dn, st * L::kTileBytes + kk * 2048),
                                       kIdescV, (i > 0 || kk > 0) ? 1u : 0u);
                    if constexpr (TWO) {
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            tc::mma_f16_ts_if(one, acc, col + kLow + (kk & 1) * 8 + (kk >> 1) * kCols, tc::desc_add(dn, st * L::kTileBytes + kk * 2048),
                                           kIdescV, 1u);
                    }
                    tc::mma_commit_if(one, bar((second ? B_QEMPTY : B_OEMPTY) + st));
                    if (i + 1 < nt) ok = scores(it + 1, true);
                    else if (!second && one) tc::mbar_arrive(bar(b_other));
                }
                tc::mma_commit_if(one, bar(second ? B_ACC + 1 : B_ACC));
            }
        } else if (warp == kCompute / 32 + 3) {
            // ---------------- each tile as it has landed --------------------
            for (int i = 0; i < nt; ++i) {
                const int it = it0 + i, st = it & (kStages - 1), ph = (it / kStages) & 1;
                bool ok = wait(B_QLAND + st, ph);
                if (!__all_sync(0xffffffffu, ok)) break;
                float *info = reinterpret_cast<float *>(sm + L::kOffInfo + st * kInfoBytes);
                float4 l4 = reinterpret_cast<float4 *>(info)[lane];
                float4 d4 = reinterpret_cast<float4 *>(info + kTile)[lane];
                const int4 c4 = reinterpret_cast<int4 *>(info + 2 * kTile)[lane];
                const int4 m4 = reinterpret_cast<int4 *>(info + 3 * kTile)[lane];
                l4.x = -(l4.x + static_cast<float>(cmax - c4.x));
                l4.y = -(l4.y + static_cast<float>(cmax - c4.y));
                l4.z = -(l4.z + static_cast<float>(cmax - c4.z));
                l4.w = -(l4.w + static_cast<float>(cmax - c4.w));
                d4.x *= -sigma;
                d4.y *= -sigma;
                d4.z *= -sigma;
                d4.w *= -sigma;
                reinterpret_cast<float4 *>(info)[lane] = l4;
                reinterpret_cast<float4 *>(info + kTile)[lane] = d4;
                auto cuts = [&](int m) { return m > 0 && m < j0 + kTile; };
                const bool need = __any_sync(0xffffffffu, cuts(m4.x) || cuts(m4.y) || cuts(m4.z) || cuts(m4.w));
                if (lane == 0) s_need[st] = need;
                const uint32_t nib = (m4.x < 0) | (m4.y < 0) << 1 | (m4.z < 0) << 2 | (m4.w < 0) << 3;
                const bool dirty = __any_sync(0xffffffffu, nib != 0);
                auto clear = [&](int off) {
                    for (int s = 0; s < 32; ++s) {
                        uint32_t w = __shfl_sync(0xffffffffu, nib, s);
                        while (w) {
                            const int r = 4 * s + __ffs(w) - 1;
                            w &= w - 1;
                            if (lane < D / 8)
                                *reinterpret_cast<uint4 *>(sm + off + st * L::kTileBytes + (lane >> 3) * kHalf + r * 128 + (lane & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                        }
                    }
                    tc::fence_proxy_async_smem();
                };
                if (dirty) clear(L::kOffQ);
                tc::mbar_arrive(bar(B_QFULL + st));
                ok = wait(B_OLAND + st, ph);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (dirty) clear(L::kOffO);
                tc::mbar_arrive(bar(B_OFULL + st));
            }
        } else {
            // ---------------- P and dS --------------------------------------
            // A thread holds, of each eight columns (rows of the tile) of its part, two columns of four keys: L and D
            // then come in 8 loads of two values, of which a warp's threads read four different ones.  (A key a
            // thread, each of its columns' values read by the whole warp, took 1370 clocks of shared memory's time
            // for a tile, beside the products' 2050.)
            const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            const uint32_t ts = lane_base + kColS + part * kCols, tp = lane_base + kColP + part * kCols;
            const float2 c1 = make_float2(a.scale * 1.4426950408889634f, a.scale * 1.4426950408889634f);
            const float2 sg = make_float2(sigma, sigma);
            const int key4 = (warp & 3) * 32 + (lane >> 2);  // its first key in the tile; the others 8, 16, 24 on
            constexpr int G8 = kCols / 8;                    // groups of eight columns
            for (int i = 0; i < nt; ++i) {
                const int it = it0 + i, st = it & (kStages - 1);
                const float *info = reinterpret_cast<const float *>(sm + L::kOffInfo + st * kInfoBytes) + part * kCols + 2 * (lane & 3);
                bool ok = wait(B_QFULL + st, (it / kStages) & 1);
                ok = ok && wait(B_S, it & 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc::tc_fence_after();
                float p[2 * 4 * G8];                         // [16 lanes][group][key, key + 8][two columns]
                {
                    uint32_t r[2][4 * G8];
                    tc::tmem_ld16x32(ts, r[0]);
                    tc::tmem_ld16x32(ts + (16u << 16), r[1]);
                    const bool need = s_need[st] != 0;
                    tc::tmem_wait_ld16(r[0]);
                    tc::tmem_wait_ld16(r[1]);
#pragma unroll
                    for (int g8 = 0; g8 < G8; ++g8) {
                        const float2 l2 = *reinterpret_cast<const float2 *>(info + 8 * g8);   // -L
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint32_t *x = &r[u >> 1][4 * g8 + 2 * (u & 1)];
                            const float2 e = __ffma2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), c1, l2);
                            float *pp = &p[(u >> 1) * 4 * G8 + 4 * g8 + 2 * (u & 1)];
                            pp[0] = fast_exp2(e.x);
                            pp[1] = fast_exp2(e.y);
                        }
                    }
                    if (need) {
#pragma unroll
                        for (int g8 = 0; g8 < G8; ++g8) {
                            const int2 m = *reinterpret_cast<const int2 *>(info + 3 * kTile + 8 * g8);
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                float *pp = &p[(u >> 1) * 4 * G8 + 4 * g8 + 2 * (u & 1)];
                                if (j0 + key4 + 8 * u >= m.x) pp[0] = 0.f;
                                if (j0 + key4 + 8 * u >= m.y) pp[1] = 0.f;
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t ph[2 * G8];
#pragma unroll
                        for (int c = 0; c < 2 * G8; ++c) ph[c] = pack_half2(p[4 * G8 * u + 2 * c], p[4 * G8 * u + 2 * c + 1]);
                        tc::tmem_st16x16(ts + (static_cast<uint32_t>(16 * u) << 16), ph);
                        if constexpr (TWO) {
#pragma unroll
                            for (int c = 0; c < 2 * G8; ++c) ph[c] = low_part(ph[c], p[4 * G8 * u + 2 * c], p[4 * G8 * u + 2 * c + 1]);
                            tc::tmem_st16x16(ts + kLow + (static_cast<uint32_t>(16 * u) << 16), ph);
                        }
                    }
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                tc::mbar_arrive(bar(B_P));
                ok = wait(B_DP, it & 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc::tc_fence_after();
                uint32_t r[2][4 * G8];
                tc::tmem_ld16x32(tp, r[0]);
                tc::tmem_ld16x32(tp + (16u << 16), r[1]);
                float2 d2[G8];                               // -D
#pragma unroll
                for (int g8 = 0; g8 < G8; ++g8) d2[g8] = *reinterpret_cast<const float2 *>(info + kTile + 8 * g8);
                tc::tmem_wait_ld16(r[0]);
                tc::tmem_wait_ld16(r[1]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t dh[2 * G8], dl[2 * G8];
#pragma unroll
                    for (int c = 0; c < 2 * G8; ++c) {       // group c / 2, key + 8 (c % 2)
                        float2 x = __ffma2_rn(make_float2(__uint_as_float(r[u][2 * c]), __uint_as_float(r[u][2 * c + 1])), sg, d2[c >> 1]);
                        x = __fmul2_rn(x, make_float2(p[4 * G8 * u + 2 * c], p[4 * G8 * u + 2 * c + 1]));
                        dh[c] = pack_half2(x.x, x.y);
                        if (TWO) dl[c] = low_part(dh[c], x.x, x.y);
                    }
                    tc::tmem_st16x16(tp + (static_cast<uint32_t>(16 * u) << 16), dh);
                    if constexpr (TWO) tc::tmem_st16x16(tp + kLow + (static_cast<uint32_t>(16 * u) << 16), dl);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                tc::mbar_arrive(bar(B_DS));
            }
            // ---------------- sums of this stretch ------------------------------
            bool ok = !*reinterpret_cast<volatile int *>(&s_abort);
            ok = ok && wait(B_ACC, stretch & 1);
            ok = ok && wait(B_ACC + 1, stretch & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tc::tc_fence_after();
                const bool last = o + kStretch >= o_hi;
#pragma unroll
                for (int which = 0; which < 2; ++which) {    // dk, dv
                    const Pow2 f(which ? 1.f : a.scale, which ? cmax - kPShift : cmax - sig_e - kPShift);
                    float v[NC];
                    load_cols<NC>(lane_base + (which ? kColV : kColK) + part * NC, v);
#pragma unroll
                    for (int c = 0; c < NC; ++c) v[c] = there ? f(v[c]) : 0.f;
                    if (key < g.n) {
                        if (stretch > 0) add_row<NC>(slot_of(which), v);
                        if (last && a.pieces == 1) store_row<NC>(which ? a.out1 : a.out0, out_at(), a.g_type, v);
                        else store_row<NC>(slot_of(which), 0, SKV_F32, v);
                    }
                }
                tc::tc_fence_before();
            }
        }
        __syncwarp();
        if (__syncthreads_or(s_abort)) {                     // (all of the CTA or none) nothing runs on when it leaves
            if (tid == kCompute) {
                tc::mbar_wait(bar(B_KV), 0, nullptr, kDrainNs);
                for (int i = max(0, s_loads[0] - kStages); i < s_loads[0]; ++i)
                    tc::mbar_wait(bar(B_QLAND + (i & (kStages - 1))), (i / kStages) & 1, nullptr, kDrainNs);
                for (int i = max(0, s_loads[1] - kStages); i < s_loads[1]; ++i)
                    tc::mbar_wait(bar(B_OLAND + (i & (kStages - 1))), (i / kStages) & 1, nullptr, kDrainNs);
            }
            if (tid == kCompute + 32 || tid == kCompute + 64) tc::mbar_wait(bar(B_ACC + (warp - kCompute / 32 - 1)), stretch & 1, nullptr, kDrainNs);
            break;
        }
        it0 += nt;
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after();
        tc::tmem_dealloc<512>(tmem);
    }
}

}  // namespace kv
}  // namespace bwd
}  // namespace skv
