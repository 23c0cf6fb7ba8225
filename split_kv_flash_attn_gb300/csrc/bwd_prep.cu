// bwd_prep.cu -- before the gradient kernels: statistics of the query rows, the sizes of
// the values, gathered rows of lists; after them: sums of a split result's pieces.
//
// Memory-bound: o and d_o are read once for delta = d_o.o - d_lse, v once for the
// exponents of its rows.
#include "bwd.cuh"

namespace skv {
namespace bwd {

constexpr int kPrepThreads = 256;

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// A query tile: a warp takes a row at a time, D/32 values a lane, four rows in flight.
template <int D, bool F32DO>
__device__ void prep_rows(const PrepArgs &a, int64_t tile)
{
    constexpr int V = D / 32, U = 4;
    const Geo &g = a.g;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int qt = static_cast<int>(tile % g.QT);
    const int64_t gh = tile / g.QT;
    const QTile t = q_tile(g, static_cast<int>(gh / g.Hk), static_cast<int>(gh % g.Hk), qt);
    float *info = a.info + tile * (kInfoRows * kTile);
    int lim_max = 0, mN = kNoExp, mD = kNoExp, mC = -1000;
    for (int r0 = warp * (kTile / 8); r0 < (warp + 1) * (kTile / 8); r0 += U) {
        int64_t row[U];
        float x[U][V], y[U][V], lse[U], dl[U];
        int32_t pos[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            row[u] = q_row(g, t, r0 + u);
            const int64_t rr = row[u] < 0 ? 0 : row[u];
            const int64_t at = rr * D + lane * V;
            if constexpr (F32DO) {
                if constexpr (V == 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.d_o) + at);
                    x[u][0] = f.x; x[u][1] = f.y; x[u][2] = f.z; x[u][3] = f.w;
                } else {
                    const float2 f = *reinterpret_cast<const float2 *>(static_cast<const float *>(a.d_o) + at);
                    x[u][0] = f.x; x[u][1] = f.y;
                }
            } else {
                const __half *p = static_cast<const __half *>(a.d_o) + at;
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(p + i));
                    x[u][i] = f.x;
                    x[u][i + 1] = f.y;
                }
            }
            if constexpr (V == 4) {
                const float4 f = *reinterpret_cast<const float4 *>(a.o + at);
                y[u][0] = f.x; y[u][1] = f.y; y[u][2] = f.z; y[u][3] = f.w;
            } else {
                const float2 f = *reinterpret_cast<const float2 *>(a.o + at);
                y[u][0] = f.x; y[u][1] = f.y;
            }
            lse[u] = a.lse[rr];
            dl[u] = a.d_lse ? a.d_lse[rr] : 0.f;
            pos[u] = a.q_pos ? a.q_pos[rr / g.H] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u;
            int64_t lim = g.n;
            if (a.q_pos) lim = min(g.n, max(static_cast<int64_t>(0), static_cast<int64_t>(pos[u]) - a.pos0 + 1));
            const bool dead = row[u] >= 0 && lse[u] == -INFINITY;
            const bool live = row[u] >= 0 && !dead;
            int c = 0;
            if constexpr (F32DO) {
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(x[u][i]));
                m = warp_max(m);
                // the row's largest value at 2^13 .. 2^14; a d_lse far beyond it keeps delta' in range
                c = max(exp_of(m) - 14, exp_of(fabsf(dl[u])) - 40);
                c = max(-120, min(115, c));
                const float f = pow2(-c / 2), f2 = pow2(-c - (-c / 2));
#pragma unroll
                for (int i = 0; i < V; ++i) x[u][i] = __half2float(__float2half_rn(x[u][i] * f * f2));
                if (!live) {
#pragma unroll
                    for (int i = 0; i < V; ++i) x[u][i] = 0.f;
                }
                if (row[u] >= 0) {
                    __half *p = a.doh + row[u] * D + lane * V;
#pragma unroll
                    for (int i = 0; i < V; i += 2)
                        *reinterpret_cast<__half2 *>(p + i) = __floats2half2_rn(x[u][i], x[u][i + 1]);
                }
                dl[u] = dl[u] * f * f2;
            }
            float dot = 0.f, n2 = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dot = fmaf(x[u][i], y[u][i], dot);
                n2 = fmaf(x[u][i], x[u][i], n2);
            }
            dot = warp_sum(dot);
            n2 = warp_sum(n2);
            const float delta = dot - dl[u];
            const int eN = max(kNoExp, min(60, exp_of_norm2(n2))), eD = exp_of(fabsf(delta));
            if (lane == 0) {
                // rows that see nothing get p' = 0 through L, and lim -1 where their q and d_o exist
                const bool sees = live && lim > 0;
                info[r] = sees ? lse[u] * 1.4426950408889634f - static_cast<float>(kPShift) : INFINITY;
                info[kTile + r] = sees ? delta : 0.f;
                info[2 * kTile + r] = __int_as_float(sees ? c : 0);
                info[3 * kTile + r] = __int_as_float(sees ? static_cast<int>(lim) : row[u] >= 0 ? -1 : 0);
                info[4 * kTile + r] = __int_as_float(sees ? (eN << 16) | (eD & 0xffff) : (kNoExp << 16) | (kNoExp & 0xffff));
            }
            if (live && lim > 0) {
                lim_max = max(lim_max, static_cast<int>(lim));
                if (eN > kNoExp) mN = max(mN, eN + c);
                if (eD > kNoExp) mD = max(mD, eD + c);
                if (eN > kNoExp || eD > kNoExp) mC = max(mC, c);
            }
        }
    }
    __shared__ int s_red[8][4];
    if (lane == 0) {
        s_red[warp][0] = lim_max;
        s_red[warp][1] = mN;
        s_red[warp][2] = mD;
        s_red[warp][3] = mC;
    }
    __syncthreads();
    if (threadIdx.x < 4) {
        int x = s_red[0][threadIdx.x];
        for (int w = 1; w < 8; ++w) x = max(x, s_red[w][threadIdx.x]);
        reinterpret_cast<int *>(a.sum + tile)[threadIdx.x] = x;
    }
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
