// bwd_prep.cu -- before the gradient kernels: statistics of the query rows, the sizes of
// the values, gathered rows of lists; after them: sums of a split result's pieces.
//
// Memory-bound: o and d_o are read once for delta = d_o.o - d_lse, v once for the
// exponents of its rows.  16384 tokens, 8 heads on 2 (109 MB): 26 us, 4.2 TB/s; four lists of 2048 rows and
// as many tokens, 32 heads on 8 (268 MB with the gathered rows): 49 us, 5.5 TB/s.  A row a warp, its
// loads one after the other, took 68 and 122.
#include "bwd.cuh"

namespace skv {
namespace bwd {

constexpr int kPrepThreads = 256;

// A query tile.  First the sums of its rows, D/8 lanes a row, eight values a lane, all
// loads of a thread's rows before their sums; then a thread for each row.
template <int D, bool F32DO>
__device__ void prep_rows(const PrepArgs &a, int64_t tile)
{
    constexpr int LPR = D / 8, RPP = kPrepThreads / LPR, IT = kTile / RPP;   // rows of a pass, passes: 8 or 4
    constexpr int U = 4;                                                    // passes in flight
    const Geo &g = a.g;
    const int tid = threadIdx.x, l = tid % LPR;
    const int qt = static_cast<int>(tile % g.QT);
    const int gh = static_cast<int>(tile / g.QT);
    const QTile t = q_tile(g, gh / g.Hk, gh % g.Hk, qt);
    __shared__ float s_dot[kTile], s_n2[kTile];
    __shared__ int s_c[kTile];
#pragma unroll
    for (int i0 = 0; i0 < IT; i0 += U) {
        uint4 xr[U][F32DO ? 2 : 1];
        float4 y[U][2];
        int64_t row[U];
        bool live[U];
        float dl[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            row[u] = q_row(g, t, (i0 + u) * RPP + tid / LPR);
            const int64_t rr = row[u] < 0 ? 0 : row[u];
            const int64_t at = rr * D + 8 * l;
            if constexpr (F32DO) {
                const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(a.d_o) + at);
                xr[u][0] = __ldg(p);
                xr[u][1] = __ldg(p + 1);
                dl[u] = a.d_lse ? a.d_lse[rr] : 0.f;
            } else {
                xr[u][0] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __half *>(a.d_o) + at));
            }
            const float4 *o = reinterpret_cast<const float4 *>(a.o + at);
            y[u][0] = __ldg(o);
            y[u][1] = __ldg(o + 1);
            if (F32DO) live[u] = row[u] >= 0 && a.lse[rr] != -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = (i0 + u) * RPP + tid / LPR;
            float x[8];
            int c = 0;
            if constexpr (F32DO) {
                const uint32_t w[8] = {xr[u][0].x, xr[u][0].y, xr[u][0].z, xr[u][0].w, xr[u][1].x, xr[u][1].y, xr[u][1].z, xr[u][1].w};
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = live[u] ? __uint_as_float(w[i]) : 0.f;
                    m = fmaxf(m, fabsf(x[i]));
                }
#pragma unroll
                for (int o = LPR / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                // the row's largest value at 2^13 .. 2^14; a d_lse far beyond it keeps delta' in range
                c = max(exp_of(m) - 14, exp_of(fabsf(dl[u])) - 40);
                c = max(-120, min(115, c));
                const float f = pow2(-c / 2), f2 = pow2(-c - (-c / 2));
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2 hh = __floats2half2_rn(x[2 * i] * f * f2, x[2 * i + 1] * f * f2);
                    h[i] = *reinterpret_cast<const uint32_t *>(&hh);
                    const float2 v = __half22float2(hh);
                    x[2 * i] = v.x;
                    x[2 * i + 1] = v.y;
                }
                if (row[u] >= 0)
                    *reinterpret_cast<uint4 *>(a.doh + row[u] * D + 8 * l) = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
                const uint32_t w[4] = {xr[u][0].x, xr[u][0].y, xr[u][0].z, xr[u][0].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                    x[2 * i] = v.x;
                    x[2 * i + 1] = v.y;
                }
            }
            const float yy[8] = {y[u][0].x, y[u][0].y, y[u][0].z, y[u][0].w, y[u][1].x, y[u][1].y, y[u][1].z, y[u][1].w};
            float dot = 0.f, n2 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dot = fmaf(x[i], yy[i], dot);
                n2 = fmaf(x[i], x[i], n2);
            }
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) {
                dot += __shfl_xor_sync(0xffffffffu, dot, o);
                n2 += __shfl_xor_sync(0xffffffffu, n2, o);
            }
            if (l == 0) {
                s_dot[r] = dot;
                s_n2[r] = n2;
                if (F32DO) s_c[r] = c;
            }
        }
    }
    // this thread's row
    int lim_max = 0, mN = kNoExp, mD = kNoExp, mC = -1000;
    int64_t row = -1, lim = 0;
    float lse = 0.f, dl = 0.f;
    if (tid < kTile) {
        row = q_row(g, t, tid);
        const int64_t rr = row < 0 ? 0 : row;
        lse = a.lse[rr];
        dl = a.d_lse ? a.d_lse[rr] : 0.f;
        lim = g.n;
        if (a.q_pos) {
            const int64_t tok = row < 0 ? 0 : t.group * g.T + t.t0 + tid / g.Gb;
            lim = min(g.n, max(static_cast<int64_t>(0), static_cast<int64_t>(a.q_pos[tok]) - a.pos0 + 1));
        }
    }
    __syncthreads();
    if (tid < kTile) {
        float *info = a.info + tile * (kInfoRows * kTile) + tid;
        const int c = F32DO ? s_c[tid] : 0;
        const float delta = s_dot[tid] - dl * pow2(-c / 2) * pow2(-c - (-c / 2));
        const int eN = max(kNoExp, min(60, exp_of_norm2(s_n2[tid]))), eD = exp_of(fabsf(delta));
        // rows that see nothing get p' = 0 through L, and lim -1 where their q and d_o exist
        const bool sees = row >= 0 && lse != -INFINITY && lim > 0;
        info[0] = sees ? lse * 1.4426950408889634f - static_cast<float>(kPShift) : INFINITY;
        info[kTile] = sees ? delta : 0.f;
        info[2 * kTile] = __int_as_float(sees ? c : 0);
        info[3 * kTile] = __int_as_float(sees ? static_cast<int>(lim) : row >= 0 ? -1 : 0);
        info[4 * kTile] = __int_as_float(sees ? (eN << 16) | (eD & 0xffff) : (kNoExp << 16) | (kNoExp & 0xffff));
        if (sees) {
            lim_max = static_cast<int>(lim);
            if (eN > kNoExp) mN = eN + c;
            if (eD > kNoExp) mD = eD + c;
            if (eN > kNoExp || eD > kNoExp) mC = c;
        }
    }
    __shared__ int s_red[4][4];
    if (tid < kTile) {
        lim_max = __reduce_max_sync(0xffffffffu, lim_max);
        mN = __reduce_max_sync(0xffffffffu, mN);
        mD = __reduce_max_sync(0xffffffffu, mD);
        mC = __reduce_max_sync(0xffffffffu, mC);
        if ((tid & 31) == 0) {
            s_red[tid >> 5][0] = lim_max;
            s_red[tid >> 5][1] = mN;
            s_red[tid >> 5][2] = mD;
            s_red[tid >> 5][3] = mC;
        }
    }
    __syncthreads();
    if (tid < 4)
        reinterpret_cast<int *>(a.sum + tile)[tid] =
            max(max(s_red[0][tid], s_red[1][tid]), max(s_red[2][tid], s_red[3][tid]));
}

// A key tile: D/8 lanes a key, eight values a lane.
template <int D>
__device__ void prep_keys(const PrepArgs &a, int64_t tile)
{
    constexpr int LPK = D / 8, KPP = kPrepThreads / LPK;
    const Geo &g = a.g;
    const int kt = static_cast<int>(tile % g.KT);
    const int64_t gh = tile / g.KT;
    const int group = static_cast<int>(gh / g.Hk), hk = static_cast<int>(gh % g.Hk);
    const int l = threadIdx.x % LPK;
    constexpr int U = kTile / KPP;                          // keys of a thread: 8 or 4
    uint4 v[U], k[U];
    bool in[U], there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t key = static_cast<int64_t>(kt) * kTile + u * KPP + threadIdx.x / LPK;
        in[u] = key < g.n;
        int64_t row = key;
        if (in[u] && a.rows) {
            const int64_t list = a.rows_per_head ? static_cast<int64_t>(group) * g.Hk + hk : group;
            row = a.rows[list * a.rows_ld + key];
        }
        there[u] = in[u] && row >= 0;
        v[u] = k[u] = make_uint4(0, 0, 0, 0);
        if (there[u]) {
            const int64_t off = (static_cast<int64_t>(hk) * D + 8 * l) * 2;
            v[u] = *reinterpret_cast<const uint4 *>(a.v + row * a.v_row_bytes + off);
            if (a.rows) k[u] = *reinterpret_cast<const uint4 *>(a.k + row * a.k_row_bytes + off);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t key = static_cast<int64_t>(kt) * kTile + u * KPP + threadIdx.x / LPK;
        if (a.rows && in[u]) {
            const int64_t at = ((group * g.n + key) * g.Hk + hk) * D + 8 * l;
            *reinterpret_cast<uint4 *>(a.vg + at) = v[u];
            *reinterpret_cast<uint4 *>(a.kg + at) = k[u];
        }
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        float n2 = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            n2 = fmaf(f.x, f.x, n2);
            n2 = fmaf(f.y, f.y, n2);
        }
#pragma unroll
        for (int o = LPK / 2; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
        if (l == 0) {
            const int e = max(-100, min(20, exp_of_norm2(n2)));     // fp16 rows stay below 2^20
            a.ew[(gh * g.KT + kt) * kTile + u * KPP + threadIdx.x / LPK] = static_cast<int8_t>(there[u] ? e : kAbsent);
        }
    }
}

template <int D, bool F32DO>
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(const PrepArgs a, int64_t row_tiles)
{
    if (blockIdx.x < row_tiles) prep_rows<D, F32DO>(a, blockIdx.x);
    else prep_keys<D>(a, blockIdx.x - row_tiles);
}

int launch_prep(skv_handle *h, const PrepArgs &a, int do_type, cudaStream_t st)
{
    const int64_t row_tiles = static_cast<int64_t>(a.g.groups) * a.g.Hk * a.g.QT;
    const int64_t key_tiles = static_cast<int64_t>(a.g.groups) * a.g.Hk * a.g.KT;
    if (row_tiles + key_tiles > INT32_MAX) return fail(h, SKV_EUNSUPPORTED, "too many tiles for one launch");
    const unsigned grid = static_cast<unsigned>(row_tiles + key_tiles);
    if (a.g.D == 64) {
        if (do_type == SKV_F32) prep_kernel<64, true><<<grid, kPrepThreads, 0, st>>>(a, row_tiles);
        else prep_kernel<64, false><<<grid, kPrepThreads, 0, st>>>(a, row_tiles);
    } else {
        if (do_type == SKV_F32) prep_kernel<128, true><<<grid, kPrepThreads, 0, st>>>(a, row_tiles);
        else prep_kernel<128, false><<<grid, kPrepThreads, 0, st>>>(a, row_tiles);
    }
    return cuda_fail(h, cudaGetLastError(), "gradient preparation launch");
}

// out[i] = sum over pieces of slot[piece][out][i], in their order.
__global__ void __launch_bounds__(256) join_kernel(const float4 *slot, int pieces, int64_t n4, int g_type, void *out0, void *out1)
{
    const int64_t all = n4 * gridDim.y;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n4; i += gridDim.x * 256ll) {
        const float4 *p = slot + blockIdx.y * n4 + i;
        float4 s = p[0];
#pragma unroll 4
        for (int k = 1; k < pieces; ++k) {
            const float4 x = p[k * all];
            s.x += x.x;
            s.y += x.y;
            s.z += x.z;
            s.w += x.w;
        }
        void *out = blockIdx.y ? out1 : out0;
        if (g_type == SKV_F16) reinterpret_cast<uint2 *>(out)[i] = make_uint2(pack_half2(s.x, s.y), pack_half2(s.z, s.w));
        else reinterpret_cast<float4 *>(out)[i] = s;
    }
}

int launch_join(skv_handle *h, const float *slot, int pieces, int64_t n, int outs, int g_type, void *out0, void *out1,
                cudaStream_t st)
{
    const int64_t n4 = n / 4, blocks = (n4 + 255) / 256, most = 16 * static_cast<int64_t>(h->sm_count);
    const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most), static_cast<unsigned>(outs));
    join_kernel<<<grid, 256, 0, st>>>(reinterpret_cast<const float4 *>(slot), pieces, n4, g_type, out0, out1);
    return cuda_fail(h, cudaGetLastError(), "gradient join launch");
}

}  // namespace bwd
}  // namespace skv
