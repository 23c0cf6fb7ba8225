// bwd_q.cuh -- dq: a CTA owns a query tile (TMEM lanes) and walks over the key tiles that it
// sees.
//
//   S = Q K^T   dP = dO V^T   [128 rows x 128 keys]
//   dS = 2^(S c - L) (dP sigma - D)   over dP in tensor memory
//   dQ += dS K                        (A from tensor memory)
// K serves S as the K-major and dQ as the MN-major B operand: one TMA load for both.
// Tensor memory: S, two dP buffers, dQ.  S(j+1) goes out as soon as S(j) has been loaded, dP(j+1) once
// dQ(j-1) has read the dS that stood in its buffer: both are there before the compute warps
// have done tile j.  (Two S buffers with dS over them and one dP: S(j+1) then waits for dQ(j-1) behind
// dP(j); it took 1140 us for 16384 x 16384, 8 heads on 2, where this order now takes 1000: 1649 TFLOP/s
// of the three products, 83 % of the measured fp16 rate.)
//
// What rounding dS to fp16 takes from a row's terms, eps_k, would come out as sum_k eps_k K_k.  Keys of a
// head have much in common (a mean that all scores share and the softmax ignores), so the sum of
// a row's eps is kept in fp32 and times the mean of the CTA's first keys given back: any
// vector would do, and what all keys share drops out of the error.  (Keys of N(0, 1) plus half as much in
// common: dq's error 3.2e-4 -> 2.9e-4 of its norm, 2.1e-4 of which is its own rounding.  It costs 4 % of dq's time.)
//
// Warps: 0-15 compute (four threads a row, 32 keys of the tile each; a row's L, D, sigma
// and limit are registers), 16 TMA, 17 issues S and dP, 18 issues dQ, 19 looks each K tile
// over: absent keys of lists, and rows behind the last key that any row sees, which
// hold anything, are cleared.
//
// Every wait is bounded; a CTA that gives up waits for its loads and products as bwd_kv.cuh says.
#pragma once

#include "bwd.cuh"

namespace skv {
namespace bwd {
namespace q {

constexpr int kK = 3, kV = 2;                               // K and V tiles in shared memory
constexpr int kHalf = kTile * 128;

template <int D>
struct Lay {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kOffQ = 0;
    static constexpr int kOffO = kTileBytes;
    static constexpr int kOffK = 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kK * kTileBytes;
    static constexpr int kOffBar = kOffV + kV * kTileBytes;
    static constexpr int kBytes = kOffBar + 256 + 1024;
};
static_assert(Lay<128>::kBytes <= 227 * 1024 - 128, "shared memory per CTA");

enum { B_QO, B_KLAND, B_KFULL = B_KLAND + kK, B_KEMPTY = B_KFULL + kK, B_VFULL = B_KEMPTY + kK,
       B_VEMPTY = B_VFULL + kV, B_DP = B_VEMPTY + kV, B_DS = B_DP + 2, B_DQ = B_DS + 2, B_S = B_DQ + 2, B_SFREE,
       B_ACC, B_END, B_COUNT = B_END + 2 };
static_assert(B_COUNT * 8 <= 256, "barrier area");

constexpr int kColS = 0, kColP = 128, kColQ = 384;

// TWO: ds in two fp16 parts (bwd.cuh); nothing is given back then.
template <int D, bool TWO>
__device__ __forceinline__ void run(const CUtensorMap &tq, const CUtensorMap &to, const CUtensorMap &tk, const CUtensorMap &tv,
                                    const MainArgs &a, int unit, int piece, uint8_t *smem_raw)
{
    using L = Lay<D>;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_addr(sm);
    auto bar = [&](int i) { return sbase + L::kOffBar + 8u * static_cast<uint32_t>(i); };
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_ew, s_last, s_loads[2];
    __shared__ float s_mean[D];                              // mean of the first keys
    __shared__ float s_sum[2][kTile];                        // its parts; what rounding took from dS, by halves
    __shared__ uint32_t s_here[kK][4];                       // keys of a tile that are there

    const Geo &g = a.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the last tokens first: under causal positions they see the most keys
    const int heads = g.Hk * g.groups * g.GG;
    const int ti = g.TT - 1 - unit / heads, rest = unit % heads;
    const int gi = rest % g.GG, gh = rest / g.GG;
    const int group = gh / g.Hk, hk = gh - group * g.Hk;
    const int qt = gi * g.TT + ti;
    const int64_t tile = static_cast<int64_t>(gh) * g.QT + qt;
    const QTile t = q_tile(g, group, hk, qt);
    const int box_rows = g.Gb * g.Tb;
    const int lim_tile = a.sum[tile].lim_max;

    if (tid == 0) {
        s_abort = 0;
        s_ew = -100;
        s_last = -1;
    }
    if (warp == 0) {
        tc::tmem_alloc<512>(smem_addr(&s_tmem));
        tc::tmem_relinquish();
    }
    if (tid == kCompute) {
        tc::mbar_init(bar(B_QO), 1);
        for (int i = 0; i < kK; ++i) {
            tc::mbar_init(bar(B_KLAND + i), 1);
            tc::mbar_init(bar(B_KFULL + i), 32);
            tc::mbar_init(bar(B_KEMPTY + i), 1);
        }
        for (int i = 0; i < kV; ++i) {
            tc::mbar_init(bar(B_VFULL + i), 1);
            tc::mbar_init(bar(B_VEMPTY + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(B_DP + i), 1);
            tc::mbar_init(bar(B_DS + i), kCompute);
            tc::mbar_init(bar(B_DQ + i), 1);
        }
        tc::mbar_init(bar(B_S), 1);
        tc::mbar_init(bar(B_SFREE), kCompute);
        tc::mbar_init(bar(B_ACC), 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(bar(B_END + i), 1);   // used by a CTA that gives up
        tc::fence_barrier_init();
        // the rows, while the keys' exponents are looked through
        tc::mbar_expect_tx(bar(B_QO), 2u * box_rows * D * 2);
        for (int b = 0; b < D / 64; ++b) {
            tc::tma_load_5d(sbase + L::kOffQ + b * kHalf, &tq, 64 * b, t.g0, hk, static_cast<int>(t.t0), group, bar(B_QO));
            tc::tma_load_5d(sbase + L::kOffO + b * kHalf, &to, 64 * b, t.g0, hk, static_cast<int>(t.t0), group, bar(B_QO));
        }
        tc::prefetch_tmap(&tk);
        tc::prefetch_tmap(&tv);
    }
    __syncthreads();
    // ---- the largest |v| of the keys that the tile sees, and the last key that is there ----
    {
        const int4 *ew = reinterpret_cast<const int4 *>(a.ew + static_cast<int64_t>(gh) * g.KT * kTile);
        int top = -100, last = -1;
        for (int i = tid; i < (lim_tile + 15) / 16; i += kThreads) {
            const int4 x = __ldg(ew + i);
            const int w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int b = 0; b < 16; ++b) {
                const int e = static_cast<int8_t>(w[b >> 2] >> (8 * (b & 3)));
                if (e != kAbsent && 16 * i + b < lim_tile) {
                    top = max(top, e);
                    last = 16 * i + b;
                }
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        last = __reduce_max_sync(0xffffffffu, last);
        if (lane == 0) {
            atomicMax(&s_ew, top);
            atomicMax(&s_last, last);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int n_all = (s_last + kTile) / kTile;              // key tiles up to the last key
    const int j_lo = static_cast<int>(static_cast<int64_t>(n_all) * piece / a.pieces);
    const int j_hi = static_cast<int>(static_cast<int64_t>(n_all) * (piece + 1) / a.pieces);

    auto wait = [&](int b, uint32_t parity) -> bool {
        if (tc::mbar_try_wait(bar(b), parity)) return true;
        if (*reinterpret_cast<volatile int *>(&s_abort)) return false;
        if (bounded_wait(bar(b), parity, a.status)) return true;
        s_abort = 1;
        atomicOr(a.status, 1);
        return false;
    };

    // ---- a compute thread's row ----
    constexpr int NC = D / kParts;
    const int m = (warp & 3) * 32 + lane, part = warp >> 2;
    float row_L = INFINITY, row_D = 0.f, sigma = 1.f;
    int lim = 0, out_e = 0;
    if (warp < kCompute / 32) {
        const float *info = a.info + tile * (kInfoRows * kTile) + m;
        row_L = info[0];
        lim = max(0, __float_as_int(info[3 * kTile]));
        const int c = __float_as_int(info[2 * kTile]), ex = __float_as_int(info[4 * kTile]);
        const int e = max(-100, min(100, max((ex >> 16) + s_ew, static_cast<int>(static_cast<int16_t>(ex & 0xffff))) + 1));
        sigma = pow2(-e);
        row_D = info[kTile] * sigma;
        out_e = e + c - kPShift;
    }
    // (where this thread's result goes; worked out where it is stored)
    auto slot_of = [&](int64_t row) {
        return a.slot + piece * (static_cast<int64_t>(g.groups) * g.T * g.H * D) + row * D + part * NC;
    };

    if (j_lo >= j_hi && tid == kCompute) tc::mbar_wait(bar(B_QO), 0, nullptr, kDrainNs);   // the loads land before the CTA leaves
    if (j_lo >= j_hi && warp < kCompute / 32) {                          // no keys
        const int64_t row = q_row(g, t, m);
        float z[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) z[i] = 0.f;
        if (row >= 0) {
            if (a.pieces > 1) store_row<NC>(slot_of(row), 0, SKV_F32, z);
            else store_row<NC>(a.out0, row * D + part * NC, a.g_type, z);
        }
    }

    int it0 = 0, stretch = 0;
    for (int j = j_lo; j < j_hi; j += kStretch, ++stretch) {
        const int nt = min(kStretch, j_hi - j);
        if (warp == kCompute / 32) {
            // ---------------- TMA ----------------------------------------
            if (lane == 0) {
                int k_out = 0, v_out = 0;
                for (int i = 0; i < nt; ++i) {
                    const int it = it0 + i, ks = it % kK, vs = it % kV;
                    const int y = (j + i) * kTile;
                    if (it >= kK && !wait(B_KEMPTY + ks, (it / kK - 1) & 1)) break;
                    tc::mbar_expect_tx(bar(B_KLAND + ks), L::kTileBytes);
                    for (int b = 0; b < D / 64; ++b)
                        tc::tma_load_3d(sbase + L::kOffK + ks * L::kTileBytes + b * kHalf, &tk, hk * D + 64 * b, y, group, bar(B_KLAND + ks));
                    ++k_out;
                    if (it >= kV && !wait(B_VEMPTY + vs, (it / kV - 1) & 1)) break;
                    tc::mbar_expect_tx(bar(B_VFULL + vs), L::kTileBytes);
                    for (int b = 0; b < D / 64; ++b)
                        tc::tma_load_3d(sbase + L::kOffV + vs * L::kTileBytes + b * kHalf, &tv, hk * D + 64 * b, y, group, bar(B_VFULL + vs));
                    ++v_out;
                }
                s_loads[0] = it0 + k_out;
                s_loads[1] = it0 + v_out;
            }
        } else if (warp == kCompute / 32 + 1) {
            // ---------------- S and dP ------------------------------------
            {
                const uint32_t one = tc::elect_one();        // the lane that issues; all of the warp waits
                constexpr uint32_t kIdescS = tc::idesc_f16(kTile, kTile, false);
                const uint64_t dq0 = tc::smem_desc(sbase + L::kOffQ, 16, 1024);
                const uint64_t do0 = tc::smem_desc(sbase + L::kOffO, 16, 1024);
                const uint64_t dk0 = tc::smem_desc(sbase + L::kOffK, 16, 1024);
                const uint64_t dv0 = tc::smem_desc(sbase + L::kOffV, 16, 1024);
                bool ok = __all_sync(0xffffffffu, wait(B_QO, 0));
                for (int i = 0; ok && i < nt; ++i) {
                    const int it = it0 + i, ks = it % kK, vs = it % kV, sb = it & 1;
                    ok = wait(B_KFULL + ks, (it / kK) & 1);
                    ok = ok && (it < 1 || wait(B_SFREE, (it - 1) & 1));
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                        tc::mma_f16_ss_if(one, tmem + kColS, tc::desc_add(dq0, off), tc::desc_add(dk0, ks * L::kTileBytes + off), kIdescS, kk > 0);
                    }
                    tc::mma_commit_if(one, bar(B_S));
                    // (the buffer's last dS has been read)
                    ok = wait(B_VFULL + vs, (it / kV) & 1) && (it < 2 || wait(B_DQ + sb, ((it >> 1) - 1) & 1));
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                        tc::mma_f16_ss_if(one, tmem + kColP + sb * kTile, tc::desc_add(do0, off), tc::desc_add(dv0, vs * L::kTileBytes + off), kIdescS, kk > 0);
                    }
                    tc::mma_commit_if(one, bar(B_DP + sb));
                    tc::mma_commit_if(one, bar(B_VEMPTY + vs));
                }
            }
        } else if (warp == kCompute / 32 + 2) {
            // ---------------- dQ --------------------------------------------
            {
                const uint32_t one = tc::elect_one();        // the lane that issues; all of the warp waits
                constexpr uint32_t kIdescQ = tc::idesc_f16(kTile, D, true);
                const uint64_t dk0 = tc::smem_desc(sbase + L::kOffK, kHalf, 1024);
                for (int i = 0; i < nt; ++i) {
                    const int it = it0 + i, ks = it % kK, sb = it & 1;
                    const bool ok = wait(B_DS + sb, (it >> 1) & 1) && wait(B_KFULL + ks, (it / kK) & 1);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        tc::mma_f16_ts_if(one, tmem + kColQ, tmem + kColP + sb * kTile + (kk & 1) * 8 + (kk >> 1) * kCols,
                                       tc::desc_add(dk0, ks * L::kTileBytes + kk * 2048), kIdescQ, (i > 0 || kk > 0) ? 1u : 0u);
                    if constexpr (TWO) {
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            tc::mma_f16_ts_if(one, tmem + kColQ, tmem + kColP + sb * kTile + kLow + (kk & 1) * 8 + (kk >> 1) * kCols,
                                           tc::desc_add(dk0, ks * L::kTileBytes + kk * 2048), kIdescQ, 1u);
                    }
                    tc::mma_commit_if(one, bar(B_KEMPTY + ks));
                    tc::mma_commit_if(one, bar(B_DQ + sb));
                    if (i + 1 == nt) tc::mma_commit_if(one, bar(B_ACC));
                }
            }
        } else if (warp == kCompute / 32 + 3) {
            // ---------------- each K tile as it has landed -------------------
            const int8_t *ew = a.ew + static_cast<int64_t>(gh) * g.KT * kTile;
            for (int i = 0; i < nt; ++i) {
                const int it = it0 + i, st = it % kK;
                const int jt = (j + i) * kTile;
                const uint32_t e4 = *reinterpret_cast<const uint32_t *>(ew + jt + 4 * lane);
                uint32_t w = 0;                              // this lane's four keys
#pragma unroll
                for (int b = 0; b < 4; ++b) w |= (((e4 >> (8 * b)) & 255u) != 128u ? 1u : 0u) << b;
                w <<= 4 * (lane & 7);
                w |= __shfl_xor_sync(0xffffffffu, w, 1);
                w |= __shfl_xor_sync(0xffffffffu, w, 2);
                w |= __shfl_xor_sync(0xffffffffu, w, 4);
                bool ok = wait(B_KLAND + st, (it / kK) & 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                if ((lane & 7) == 0) s_here[st][lane >> 3] = w;
                if (jt + kTile > lim_tile) {                 // rows that no token of the tile sees
                    for (int x = lane; x < (jt + kTile - lim_tile) * (D / 8); x += 32) {
                        const int r = lim_tile - jt + x / (D / 8), ch = x % (D / 8);
                        *reinterpret_cast<uint4 *>(sm + L::kOffK + st * L::kTileBytes + (ch >> 3) * kHalf + r * 128 + (ch & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_proxy_async_smem();
                }
                tc::mbar_arrive(bar(B_KFULL + st));
            }
        } else {
            // ---------------- dS --------------------------------------------
            const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            const float c1 = a.scale * 1.4426950408889634f;
            auto compute_sync = [&]() { asm volatile("bar.sync 5, %0;\n" ::"n"(kCompute) : "memory"); };
            if (!TWO && stretch == 0) {
                // the mean of the first tile's keys: the first 256 threads add up two channels of 32 or 16 rows,
                // the upper half of them leaves its sums, the lower one adds its own
                constexpr int PAIRS = D / 2, ROWS = kTile / (256 / PAIRS);
                float *sum = &s_sum[0][0] + (tid & 127) * 2;
                float2 m2 = make_float2(0.f, 0.f);
                const bool ok = wait(B_KFULL, 0);
                if (__all_sync(0xffffffffu, ok) && tid < 256) {
                    const int pr = tid % PAIRS, r0 = tid / PAIRS * ROWS;
                    const uint8_t *col = sm + L::kOffK + (pr >> 5) * kHalf + (pr & 3) * 4;
                    for (int r = r0; r < r0 + ROWS; ++r) {
                        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(col + r * 128 + ((((pr & 31) >> 2) ^ (r & 7)) << 4)));
                        m2.x += x.x;
                        m2.y += x.y;
                    }
                }
                if (tid >= 128 && tid < 256) {
                    sum[0] = m2.x;
                    sum[1] = m2.y;
                }
                compute_sync();
                if (tid < 128) {
                    sum[0] += m2.x;
                    sum[1] += m2.y;
                }
                compute_sync();
                if (tid < D) {
                    float m1 = 0.f;
                    for (int k = tid; k < 256; k += D) m1 += (&s_sum[0][0])[k];
                    s_mean[tid] = m1 * (1.f / kTile);
                }
                compute_sync();
            }
            float2 eps2 = make_float2(0.f, 0.f);
            for (int i = 0; i < nt; ++i) {
                const int it = it0 + i, st = it % kK, sb = it & 1;
                const uint32_t cs = lane_base + kColS + part * kCols, cp = lane_base + kColP + sb * kTile + part * kCols;
                bool ok = wait(B_KFULL + st, (it / kK) & 1);
                const uint32_t here = s_here[st][part];
                const int left = lim - (j + i) * kTile - part * kCols;   // columns of this part that the row sees
                ok = ok && wait(B_S, it & 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc::tc_fence_after();
                float p[kCols];
                uint32_t r[kCols];
                tc::tmem_ld32(cs, r);
                tc::tmem_wait_ld(r);
                tc::tc_fence_before();
                tc::mbar_arrive(bar(B_SFREE));
#pragma unroll
                for (int c = 0; c < kCols; c += 2) {
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), make_float2(c1, c1),
                                                make_float2(-row_L, -row_L));
                    p[c] = fast_exp2(x.x);
                    p[c + 1] = fast_exp2(x.y);
                }
                ok = wait(B_DP + sb, (it >> 1) & 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc::tc_fence_after();
                tc::tmem_ld32(cp, r);
                tc::tmem_wait_ld(r);
#pragma unroll
                for (int c = 0; c < kCols; c += 2) {
                    float2 x = __ffma2_rn(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), make_float2(sigma, sigma),
                                          make_float2(-row_D, -row_D));
                    x = __fmul2_rn(x, make_float2(p[c], p[c + 1]));
                    p[c] = x.x;
                    p[c + 1] = x.y;
                }
                if (__any_sync(0xffffffffu, left < kCols || here != 0xffffffffu)) {
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        if (c >= left || !((here >> c) & 1u)) p[c] = 0.f;
                }
                uint32_t dh[kCols / 2];
#pragma unroll
                for (int c = 0; c < kCols / 2; ++c) dh[c] = pack_half2(p[2 * c], p[2 * c + 1]);
                tc::tmem_st16u(cp, dh);
                if constexpr (TWO) {
                    uint32_t dl[kCols / 2];
#pragma unroll
                    for (int c = 0; c < kCols / 2; ++c) dl[c] = low_part(dh[c], p[2 * c], p[2 * c + 1]);
                    tc::tmem_st16u(cp + kLow, dl);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                tc::mbar_arrive(bar(B_DS + sb));
                // (while the products run)
                if constexpr (!TWO) {
#pragma unroll
                    for (int c = 0; c < kCols / 2; ++c) {
                        const __half2 h2 = *reinterpret_cast<const __half2 *>(&dh[c]);
                        eps2 = __fadd2_rn(eps2, make_float2(sub_h(__low2half(h2), p[2 * c]), sub_h(__high2half(h2), p[2 * c + 1])));
                    }
                }
            }
            // ---------------- the sum of this stretch ----------------------------
            float eps = eps2.x + eps2.y;
            if constexpr (!TWO) {
                if (part >= 2) s_sum[part - 2][m] = eps;
                compute_sync();
                if (part < 2) s_sum[part][m] += eps;
                compute_sync();
                eps = -(s_sum[0][m] + s_sum[1][m]);
            }
            bool ok = !*reinterpret_cast<volatile int *>(&s_abort);
            ok = ok && wait(B_ACC, stretch & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tc::tc_fence_after();
                const Pow2 f(a.scale, out_e);
                float v[NC];
                load_cols<NC>(lane_base + kColQ + part * NC, v);
#pragma unroll
                for (int c = 0; c < NC; ++c) v[c] = lim > 0 ? f(TWO ? v[c] : fmaf(eps, s_mean[part * NC + c], v[c])) : 0.f;
                const int64_t row = q_row(g, t, m);
                if (row >= 0) {
                    if (stretch > 0) add_row<NC>(slot_of(row), v);
                    if (j + kStretch >= j_hi && a.pieces == 1) store_row<NC>(a.out0, row * D + part * NC, a.g_type, v);
                    else store_row<NC>(slot_of(row), 0, SKV_F32, v);
                }
                tc::tc_fence_before();
            }
        }
        __syncwarp();
        const bool gave_up = __syncthreads_or(s_abort);      // all of the CTA or none
        tc::tc_fence_after();
        if (gave_up) {                                       // nothing runs on when it leaves
            if (tid == kCompute) {
                tc::mbar_wait(bar(B_QO), 0, nullptr, kDrainNs);
                for (int i = max(0, s_loads[0] - kK); i < s_loads[0]; ++i) tc::mbar_wait(bar(B_KLAND + i % kK), (i / kK) & 1, nullptr, kDrainNs);
                for (int i = max(0, s_loads[1] - kV); i < s_loads[1]; ++i) tc::mbar_wait(bar(B_VFULL + i % kV), (i / kV) & 1, nullptr, kDrainNs);
            }
            if (warp == kCompute / 32 + 1 || warp == kCompute / 32 + 2) {
                // (the thread that issued, the same one as there; its commit covers all its products)
                tc::mma_commit_if(tc::elect_one(), bar(B_END + warp - kCompute / 32 - 1));
                tc::mbar_wait(bar(B_END + warp - kCompute / 32 - 1), 0, nullptr, kDrainNs);
            }
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

}  // namespace q
}  // namespace bwd
}  // namespace skv
