// q8_decode.cu -- attention of a few query rows per KV head over 8-bit pages.
//
// The mathematics.  Over a page the score of key j is (scale * d_k) * (q . c_j)
// and its value d_v * c_vj, so the codes go into the products as they are
// (int8 is exact in fp16) and the page's scales multiply fp32 numbers.  With m
// the running reference of a query row and r the largest |d_v| so far,
//   p_j = 2^(s_j - m + 10),  l = sum p_j,  O = sum (p_j * d_v / r) c_vj,
// and o = r O / l.  The weights p_j d_v / r stay below 2^15, and each enters the
// product as two fp16 numbers (itself rounded, and what the rounding left), which
// keeps it to 2^-22 of its value down to 2^-24: results are good to fp32.
//
// Work split.  All pages of all (sequence, KV head, row group) units form one
// line, of which every CTA takes an equal piece; a piece that covers several
// units works through them, and a unit that several pieces share is put
// together by the last CTA to finish with it, in piece order (so results do not
// depend on timing).  Lengths are read on the device: a call costs its keys, not
// its lists' capacity, and ragged batches stay balanced.
//
// A CTA's four warps take its pages in turn, each on its own: K and V bytes go
// from global memory into registers as mma fragments without shared memory.  A
// thread (g, t) of the fragment layout reads 16-byte pieces: of key rows g and
// g + 8 the channels 16t .. (the order of the channels inside the product is
// free, the queries follow it), and of value rows 2t, 2t+1, 2t+8, 2t+9 the
// channels 16g .. (pairs of rows are interleaved by byte permutes).  Keys are
// the M side of S = K Q^T and channels that of O^T = V^T P^T, so that the eight
// query columns of a product carry a KV head's query heads.  32 keys at a time: V
// is requested before S is computed, the next 32 keys' K after it.
//
// Bound: the pages' bytes at long lengths (see the table in the design notes);
// launch, plan and merge at short ones.
#include "q8.cuh"

namespace skv {
namespace q8 {

constexpr float kShift = 10.f;      // weights are kept times 2^10 ...
constexpr float kGrow = 4.f;        // ... and their reference moves when a score passes it by 2^4
constexpr int kThreads = kDecodeWarps * 32;

// Where a piece of the line of pages lies.
struct Place {
    int list;                       // sequence, or sequence x token with a selection
    int64_t np;                     // its pages
    int64_t base;                   // the line's position of its first page
};

__device__ __forceinline__ int64_t pages_of(const AttnArgs &a, int list)
{
    if (a.sel) return a.n_sel;
    return (list_len(a.L, list) + kPage - 1) / kPage;
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

template <int D, int NC, bool HILO, bool F16>
__global__ void __launch_bounds__(kThreads, NC == 2 ? 2 : kDecodeCtas) decode_kernel(const AttnArgs a)
{
    constexpr int KS = D / 16;                      // k-steps of S
    constexpr int CH = D / 64;                      // 16-byte chunks of a key row per thread
    constexpr int MT = D / 16;                      // m-tiles of O^T
    constexpr int VW = D / 32;                      // words of a value row per thread
    constexpr int LDO = D + 4;
    __shared__ float s_o[kDecodeWarps][8][LDO];
    __shared__ float s_ml[kDecodeWarps][8][2];
    __shared__ uint2 s_q[NC * KS * 32];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int n_lists = a.sel ? a.L.S * a.nq : a.L.S;
    const int64_t mult = static_cast<int64_t>(a.L.Hk) * a.row_groups;   // units per list

    // ---- the plan: total pages, this CTA's piece, the list that it starts in --
    int64_t total;
    if (a.sel) {
        total = static_cast<int64_t>(n_lists) * a.n_sel;
    } else {
        total = 0;
        for (int i = lane; i < n_lists; i += 32) {
            const int64_t n = pages_of(a, i);
            total += n;
            if (n * kPage < max(0, a.L.kv_len[i]) && blockIdx.x == 0) atomicOr(a.L.status, kStatusList);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    total *= mult;
    int64_t chunk = (total + gridDim.x - 1) / gridDim.x;
    chunk = max(int64_t(kDecodeWarps), (chunk + kDecodeWarps - 1) / kDecodeWarps * kDecodeWarps);
    int64_t pos = blockIdx.x * chunk;
    const int64_t pos_end = min(total, pos + chunk);
    const int64_t pos0 = pos;

    // lists without a page: their rows are written here
    if (!a.sel) {
        for (int i = blockIdx.x; i < n_lists; i += gridDim.x) {
            if (pages_of(a, i) != 0) continue;
            const int64_t r0 = static_cast<int64_t>(i) * a.nq * a.H, nr = static_cast<int64_t>(a.nq) * a.H;
            for (int64_t e = tid; e < nr * D; e += kThreads) {
                if (F16) static_cast<__half *>(a.o)[r0 * D + e] = __float2half(0.f);
                else static_cast<float *>(a.o)[r0 * D + e] = 0.f;
            }
            for (int64_t e = tid; e < nr; e += kThreads) a.lse[r0 + e] = -INFINITY;
        }
    }
    if (pos >= pos_end) return;

    Place at = {0, 0, 0};
    if (a.sel) {
        at.np = a.n_sel;
        at.list = static_cast<int>(pos / (at.np * mult));
        at.base = at.list * (at.np * mult);
    } else {
        int64_t before = 0;
        for (int c0 = 0; c0 < n_lists; c0 += 32) {
            const int64_t n = c0 + lane < n_lists ? pages_of(a, c0 + lane) : 0;
            int64_t inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, (before + inc) * mult > pos);
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

    while (pos < pos_end) {
        // ---- the next unit: its pages [pg0, pg1) are this CTA's ---------------
        while (pos >= at.base + at.np * mult) {     // the next list with pages
            at.base += at.np * mult;
            ++at.list;
            at.np = pages_of(a, at.list);
        }
        const int64_t u_in = (pos - at.base) / at.np;
        const int64_t unit0 = at.base + u_in * at.np;              // the line's position of the unit's first page
        const int pg0 = static_cast<int>(pos - unit0);
        const int pg1 = static_cast<int>(min(at.np, pos_end - unit0));
        const int kh = static_cast<int>(u_in / a.row_groups);
        const int rg = static_cast<int>(u_in - static_cast<int64_t>(kh) * a.row_groups);
        const int seq = a.sel ? at.list / a.nq : at.list;
        const int64_t tok0 = a.sel ? at.list : static_cast<int64_t>(at.list) * a.nq;   // token of row 0
        const int row0 = rg * 8 * NC;
        const int len = static_cast<int>(list_len(a.L, seq));
        const int32_t *ids = a.L.ids + (static_cast<int64_t>(seq) * a.L.Hk + kh) * a.L.cap;
        const int32_t *sel = a.sel ? a.sel + (static_cast<int64_t>(at.list) * a.L.Hk + kh) * a.n_sel : nullptr;
        auto out_row = [&](int row) { return (tok0 + row / a.G) * a.H + kh * a.G + row % a.G; };

        // query fragments into shared memory: lane (g, t) of k-step (c, w) holds
        // channels 64c + 16t + 4w .. + 3 of column g
        for (int x = tid; x < NC * KS * 32; x += kThreads) {
            const int row = row0 + x / (KS * 32) * 8 + ((x & 31) >> 2);
            const int ks = x / 32 % KS;
            uint2 v = make_uint2(0, 0);
            if (row < a.rows)
                v = __ldg(reinterpret_cast<const uint2 *>(a.q + out_row(row) * D + 64 * (ks >> 2) + 16 * (x & 3) + 4 * (ks & 3)));
            s_q[x] = v;
        }
        int lim[NC][2];                             // keys that columns 2t, 2t+1 see
        int lim_min = len, lim_max = a.q_pos ? 0 : len;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = row0 + j * 8 + 2 * t + e;
                lim[j][e] = len;
                if (a.q_pos && r < a.rows) {
                    const int qp = a.q_pos[tok0 + r / a.G];
                    lim[j][e] = qp < 0 ? 0 : (qp < len ? qp + 1 : len);
                    lim_min = min(lim_min, lim[j][e]);
                    lim_max = max(lim_max, lim[j][e]);
                }
            }
        }
        if (a.q_pos) {
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));
                lim_max = max(lim_max, __shfl_xor_sync(0xffffffffu, lim_max, o));
            }
        }

        __syncthreads();                            // s_q is written
        float m_ref[NC][2], l_sum[NC][2], acc[NC][MT][4];
        float r_ref = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            m_ref[j][0] = m_ref[j][1] = -INFINITY;
            l_sum[j][0] = l_sum[j][1] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][i][e] = 0.f;
        }

        // ---- pages, 32 at a time: lane i holds what is known of the i-th -------
        struct Meta {
            int id, blk;
            float ks, vs;
        };
        auto load_meta = [&](int first) {
            Meta x = {-1, 0, 0.f, 0.f};
            const int p = first + kDecodeWarps * lane;
            if (p < pg1) {
                const int64_t blk = sel ? __ldg(sel + p) : p;
                if (blk >= 0 && blk * kPage < lim_max) x.id = checked_page(a.L, __ldg(ids + blk));
                x.blk = static_cast<int>(blk);
                if (x.id >= 0) {
                    x.ks = __ldg(a.k_scale + x.id) * a.scale_log2;
                    x.vs = __ldg(a.v_scale + x.id);
                } else if (a.page_lse) {
                    for (int c = 0; c < 8 * NC; ++c) {
                        const int row = row0 + c;
                        if (row >= a.rows) break;
                        const int64_t rr = a.sel ? (at.list % a.nq) * a.G + row : row;
                        a.page_lse[((static_cast<int64_t>(seq) * a.L.Hk + kh) * a.nq * a.G + rr) * a.page_ld + p] = -INFINITY;
                    }
                }
            }
            return x;
        };
        uint4 kr[2][2][CH];
        auto load_k = [&](int id, int h) {
            const int8_t *base = a.k + static_cast<int64_t>(id) * (kPage * D) + (32 * h + g) * D + 16 * t;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int rr = 0; rr < 2; ++rr)
#pragma unroll
                    for (int c = 0; c < CH; ++c) kr[i][rr][c] = ld_stream16(base + (16 * i + 8 * rr) * D + 64 * c);
        };
        int first = pg0 + warp;
        Meta cur = load_meta(first);
        while (first < pg1) {
            const int next_first = first + 32 * kDecodeWarps;
            unsigned todo = __ballot_sync(0xffffffffu, cur.id >= 0);
            const Meta nxt = next_first < pg1 ? load_meta(next_first) : Meta{-1, 0, 0.f, 0.f};
            if (todo) load_k(__shfl_sync(0xffffffffu, cur.id, __ffs(todo) - 1), 0);
            while (todo) {
                const int src = __ffs(todo) - 1;
                todo &= todo - 1;
                const int id = __shfl_sync(0xffffffffu, cur.id, src);
                // (blk * 64 < lim_max <= 2^31 - 1)
                const int key0 = __shfl_sync(0xffffffffu, cur.blk, src) * kPage;
                const float ks = __shfl_sync(0xffffffffu, cur.ks, src);
                const float vs = __shfl_sync(0xffffffffu, cur.vs, src);
                const int id_next = todo ? __shfl_sync(0xffffffffu, cur.id, __ffs(todo) - 1) : -1;
                const bool masked = lim_min - key0 < kPage;
                if (fabsf(vs) > 2.f * r_ref) {
                    const float b = r_ref / fabsf(vs);
                    r_ref = fabsf(vs);
#pragma unroll
                    for (int j = 0; j < NC; ++j)
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[j][i][e] *= b;
                }
                const float f = r_ref > 0.f ? vs / r_ref : 0.f;
                float l_page[NC][2];
#pragma unroll
                for (int j = 0; j < NC; ++j) l_page[j][0] = l_page[j][1] = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // V of these 32 keys: rows 16i + 2t + {0, 1, 8, 9}
                    uint32_t vr[2][4][VW];
                    {
                        const int8_t *base =
                            a.v + static_cast<int64_t>(id) * (kPage * D) + (32 * h + 2 * t) * D + (D / 8) * g;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int rr = 0; rr < 4; ++rr) {
                                const int8_t *p = base + (16 * i + (rr & 1) + 8 * (rr >> 1)) * D;
                                if constexpr (VW == 4) {
                                    const uint4 x = ld_stream16(p);
                                    vr[i][rr][0] = x.x;
                                    vr[i][rr][1] = x.y;
                                    vr[i][rr][2] = x.z;
                                    vr[i][rr][3] = x.w;
                                } else {
                                    const uint2 x = ld_stream8(p);
                                    vr[i][rr][0] = x.x;
                                    vr[i][rr][1] = x.y;
                                }
                            }
                    }
                    // S = K Q^T
                    float s[NC][2][4];
#pragma unroll
                    for (int j = 0; j < NC; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[j][i][e] = 0.f;
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            uint2 qf[NC];
#pragma unroll
                            for (int j = 0; j < NC; ++j) qf[j] = s_q[(j * KS + c * 4 + w) * 32 + lane];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t x = word(kr[i][0][c], w) ^ 0x80808080u;
                                const uint32_t y = word(kr[i][1][c], w) ^ 0x80808080u;
                                const uint32_t a0 = codes_lo(x), a1 = codes_lo(y), a2 = codes_hi(x), a3 = codes_hi(y);
#pragma unroll
                                for (int j = 0; j < NC; ++j) mma_16816(s[j][i], a0, a1, a2, a3, qf[j].x, qf[j].y);
                            }
                        }
                    // the next 32 keys' K
                    if (h == 0) load_k(id, 1);
                    else if (id_next >= 0) load_k(id_next, 0);

                    uint32_t bh[NC][2][2], bl[NC][2][2];
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                s[j][i][e] *= ks;
                                if (masked && 32 * h + 16 * i + 8 * (e >> 1) + g >= lim[j][e & 1] - key0)
                                    s[j][i][e] = -INFINITY;
                            }
                        float top[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            top[e] = fmaxf(fmaxf(s[j][0][e], s[j][0][e + 2]), fmaxf(s[j][1][e], s[j][1][e + 2]));
                        // m_ref + kGrow is -inf at first, and then any score moves it
                        if (__any_sync(0xffffffffu, top[0] > m_ref[j][0] + kGrow || top[1] > m_ref[j][1] + kGrow)) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x = top[e];
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                                if (x > m_ref[j][e] + kGrow) {
                                    const float b = fast_exp2(m_ref[j][e] - x);
                                    m_ref[j][e] = x;
                                    l_sum[j][e] *= b;
                                    l_page[j][e] *= b;
#pragma unroll
                                    for (int i = 0; i < MT; ++i) {
                                        acc[j][i][e] *= b;
                                        acc[j][i][e + 2] *= b;
                                    }
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                float w[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float off = m_ref[j][e] == -INFINITY ? 0.f : kShift - m_ref[j][e];
                                    const float p = fast_exp2(s[j][i][half * 2 + e] + off);
                                    l_page[j][e] += p;
                                    w[e] = p * f;
                                }
                                const uint32_t hw = pack_half2(w[0], w[1]);
                                bh[j][i][half] = movmatrix_trans(hw);
                                if (HILO) {
                                    const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hw));
                                    bl[j][i][half] = movmatrix_trans(pack_half2(w[0] - back.x, w[1] - back.y));
                                }
                            }
                    }
                    // O^T += V^T P^T
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int w = 0; w < VW; ++w) {
                            uint32_t x[4];
#pragma unroll
                            for (int rr = 0; rr < 4; ++rr) x[rr] = vr[i][rr][w] ^ 0x80808080u;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                // channels (D/8) g + 4w + 2e (m = g) and + 1 (m = g + 8)
                                const uint32_t p01 = __byte_perm(x[0], x[1], e ? 0x7362 : 0x5140);
                                const uint32_t p89 = __byte_perm(x[2], x[3], e ? 0x7362 : 0x5140);
                                const uint32_t a0 = codes_lo(p01), a1 = codes_hi(p01);
                                const uint32_t a2 = codes_lo(p89), a3 = codes_hi(p89);
#pragma unroll
                                for (int j = 0; j < NC; ++j) {
                                    mma_16816(acc[j][2 * w + e], a0, a1, a2, a3, bh[j][i][0], bh[j][i][1]);
                                    if (HILO) mma_16816(acc[j][2 * w + e], a0, a1, a2, a3, bl[j][i][0], bl[j][i][1]);
                                }
                            }
                        }
                }
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    l_sum[j][0] += l_page[j][0];
                    l_sum[j][1] += l_page[j][1];
                }
                if (a.page_lse) {
                    const int p = first + kDecodeWarps * src;
#pragma unroll
                    for (int j = 0; j < NC; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = l_page[j][e];
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                            const int row = row0 + j * 8 + 2 * t + e;
                            if (g == 0 && row < a.rows) {
                                const int64_t rr = a.sel ? (at.list % a.nq) * a.G + row : row;
                                a.page_lse[((static_cast<int64_t>(seq) * a.L.Hk + kh) * a.nq * a.G + rr) * a.page_ld + p] =
                                    x > 0.f ? m_ref[j][e] - kShift + log2f(x) : -INFINITY;
                            }
                        }
                }
            }
            cur = nxt;
            first = next_first;
        }

        // ---- the warps' results together, eight columns at a time ---------------
        const bool whole = pg0 == 0 && pg1 == at.np;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (pos == pos0 ? 0 : 1);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            __syncthreads();                        // the buffers of the last round are read
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l_sum[j][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (g == 0) {
                    s_ml[warp][2 * t + e][0] = m_ref[j][e];
                    s_ml[warp][2 * t + e][1] = x;
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)        // channels (D/8) g + 2i, + 1
                    *reinterpret_cast<float2 *>(&s_o[warp][2 * t + e][(D / 8) * g + 2 * i]) =
                        make_float2(acc[j][i][e] * r_ref, acc[j][i][e + 2] * r_ref);
            }
            __syncthreads();
#pragma unroll
            for (int it = 0; it < 8 * D / kThreads; ++it) {
                const int c = (it * kThreads + tid) / D, d = (it * kThreads + tid) % D;
                const int row = row0 + j * 8 + c;
                if (row >= a.rows) continue;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < kDecodeWarps; ++w) M = fmaxf(M, s_ml[w][c][0]);
                float Lw = 0.f, O = 0.f;
                if (M != -INFINITY) {
#pragma unroll
                    for (int w = 0; w < kDecodeWarps; ++w) {
                        const float b = fast_exp2(s_ml[w][c][0] - M);
                        Lw = fmaf(b, s_ml[w][c][1], Lw);
                        O = fmaf(b, s_o[w][c][d], O);
                    }
                }
                if (whole) {
                    const int64_t r = out_row(row);
                    const float v = Lw > 0.f ? O / Lw : 0.f;
                    if (F16) static_cast<__half *>(a.o)[r * D + d] = __float2half_rn(v);
                    else static_cast<float *>(a.o)[r * D + d] = v;
                    if (d == 0) a.lse[r] = Lw > 0.f ? (M - kShift + log2f(Lw)) * 0.6931471805599453f : -INFINITY;
                } else {
                    a.part_o[(slot * (8 * NC) + j * 8 + c) * D + d] = O;
                    if (d == 0) {
                        a.part_ml[(slot * (8 * NC) + j * 8 + c) * 2] = M;
                        a.part_ml[(slot * (8 * NC) + j * 8 + c) * 2 + 1] = Lw;
                    }
                }
            }
        }
        if (!whole) {
            // ---- the last CTA of the unit puts the pieces together, in order -----
            const int64_t u = at.list * mult + u_in;
            const int64_t c_lo = unit0 / chunk, c_hi = (unit0 + at.np - 1) / chunk;
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(a.counters + u, 1) == static_cast<int>(c_hi - c_lo);
            __syncthreads();
            if (s_last) {
                __threadfence();
                auto slot_of = [&](int64_t c) { return 2 * c + (c == c_lo && unit0 > c * chunk ? 1 : 0); };
                for (int e = tid; e < 8 * NC * (D / 4); e += kThreads) {
                    const int c = e / (D / 4), d4 = e % (D / 4);
                    const int row = row0 + c;
                    if (row >= a.rows) continue;
                    float M = -INFINITY;
                    for (int64_t x = c_lo; x <= c_hi; ++x)
                        M = fmaxf(M, __ldcg(a.part_ml + (slot_of(x) * (8 * NC) + c) * 2));
                    float Ls = 0.f;
                    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (M != -INFINITY) {
#pragma unroll 8
                        for (int64_t x = c_lo; x <= c_hi; ++x) {
                            const int64_t sl = slot_of(x) * (8 * NC) + c;
                            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.part_ml) + sl);
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.part_o + sl * D) + d4);
                            const float b = fast_exp2(ml.x - M);
                            Ls = fmaf(b, ml.y, Ls);
                            O.x = fmaf(b, v.x, O.x);
                            O.y = fmaf(b, v.y, O.y);
                            O.z = fmaf(b, v.z, O.z);
                            O.w = fmaf(b, v.w, O.w);
                        }
                    }
                    const float inv = Ls > 0.f ? 1.f / Ls : 0.f;
                    O.x *= inv;
                    O.y *= inv;
                    O.z *= inv;
                    O.w *= inv;
                    const int64_t r = out_row(row);
                    if (F16)
                        *reinterpret_cast<uint2 *>(static_cast<__half *>(a.o) + r * D + d4 * 4) =
                            make_uint2(pack_half2(O.x, O.y), pack_half2(O.z, O.w));
                    else
                        *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + r * D + d4 * 4) = O;
                    if (d4 == 0)
                        a.lse[r] = Ls > 0.f ? (M - kShift + log2f(Ls)) * 0.6931471805599453f : -INFINITY;
                }
                if (tid == 0) a.counters[u] = 0;
            }
        }
        pos = unit0 + pg1;
    }
}

// Attention weight of each page from its log sums: mass += sum over rows of
// 2^(page - row).  Rows are added in their order.
__global__ void __launch_bounds__(128) mass_kernel(const AttnArgs a, float *mass)
{
    const int kh = blockIdx.y, s = blockIdx.z;
    const int64_t unit = static_cast<int64_t>(s) * a.L.Hk + kh;
    const int rows = a.nq * a.G;
    const int64_t len = list_len(a.L, s);
    const float *pl = a.page_lse + unit * rows * a.page_ld;
    float *out = mass + unit * a.L.cap;
    auto lse2 = [&](int r) {
        return a.lse[(static_cast<int64_t>(s) * a.nq + r / a.G) * a.H + kh * a.G + r % a.G] * 1.4426950408889634f;
    };
    if (!a.sel) {
        const int64_t p = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
        if (p * kPage >= len) return;
        float sum = 0.f;
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
            const float z = lse2(r);
            const float x = __ldcg(pl + r * a.page_ld + p);
            sum += z == -INFINITY ? 0.f : fast_exp2(x - z);
        }
        out[p] += sum;
        return;
    }
    // with a selection: token by token (a token's pages are different ones, or
    // the same page with the same weight: the order of their additions is free)
    for (int t = 0; t < a.nq; ++t) {
        const int32_t *sel = a.sel + ((static_cast<int64_t>(s) * a.nq + t) * a.L.Hk + kh) * a.n_sel;
        for (int i = threadIdx.x; i < a.n_sel; i += 128) {
            const int64_t blk = sel[i];
            if (blk < 0 || blk * kPage >= len) continue;
            float sum = 0.f;
            for (int g = 0; g < a.G; ++g) {
                const float z = lse2(t * a.G + g);
                const float x = __ldcg(pl + (t * a.G + g) * a.page_ld + i);
                sum += z == -INFINITY ? 0.f : fast_exp2(x - z);
            }
            if (sum > 0.f) atomicAdd(out + blk, sum);
        }
        __syncthreads();
    }
}

int launch_mass(skv_handle *h, const AttnArgs &a, float *mass, cudaStream_t st)
{
    const unsigned bx = a.sel ? 1u : static_cast<unsigned>((a.L.cap + 127) / 128);
    mass_kernel<<<dim3(bx, a.L.Hk, a.L.S), 128, 0, st>>>(a, mass);
    return cuda_fail(h, cudaGetLastError(), "page weight launch");
}

template <int D>
static void launch_decode_d(const AttnArgs &a, bool f16, int grid, int nc, cudaStream_t st)
{
    // One column group always takes both parts of the weights (its products are
    // a small part of a page's time); more of them only when o is fp32.
    if (nc == 1) {
        if (f16) decode_kernel<D, 1, true, true><<<grid, kThreads, 0, st>>>(a);
        else decode_kernel<D, 1, true, false><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (f16) decode_kernel<D, 2, false, true><<<grid, kThreads, 0, st>>>(a);
        else decode_kernel<D, 2, true, false><<<grid, kThreads, 0, st>>>(a);
    }
}

int launch_decode(skv_handle *h, const AttnArgs &a, int D, bool f16, int grid, int nc, cudaStream_t st)
{
    if (h->prof_before) cudaEventRecord(h->prof_before, st);
    if (D == 128) launch_decode_d<128>(a, f16, grid, nc, st);
    else launch_decode_d<64>(a, f16, grid, nc, st);
    const cudaError_t e = cudaGetLastError();
    if (h->prof_after) cudaEventRecord(h->prof_after, st);
    return cuda_fail(h, e, "8-bit decode launch");
}

}  // namespace q8
}  // namespace skv
