// q8_append.cu -- writing tokens into 8-bit pages.
//
// One CTA for each (page touched, K or V, KV head, sequence).  It holds the
// page's new values in registers (at most 64 rows of D: 8 values of up to 4
// rows a thread), takes their largest magnitude, d' = max(d, fp32(amax/127)),
// and writes the codes nearest x/d' and, for K, the channels' smallest and
// largest codes.  Only when d' > d and the page holds earlier tokens are those
// read and recoded, through a table of the 255 codes (one fp64 division each:
// c*d has 31 significant bits, so c*d/d' cannot be rounded onto a half-integer
// that it is not); rounding is monotone, so the old extremes recode like codes.
//
// A code is rint(t), t = x (1/d') with an approximate reciprocal, when t is further
// than 2^-13 from every half-integer: t is off by less than 2^-21.4 * 128 = 2^-14.4
// and |x/d'| never exceeds 127 + 2^-16, so nothing is left to clamp.  Nearer ones (one
// value in 4000), infinities and NaN are decided by the exact quotient, eight at a
// time; with that division for every value a 4096-token prompt took 31 us.
//
// Bound: a token's append is two dependent reads (length, page id) and one
// write deep, the prompt's by its bytes (x read once, codes written once).
#include "q8.cuh"

namespace skv {
namespace q8 {

constexpr int kAppendThreads = 256;

struct AppendArgs {
    Lists L;
    int8_t *codes[2];              // K, V
    float *scale[2];
    int8_t *k_min, *k_max;
    const void *x[2];              // [S][n_max][Hk][D]
    const int32_t *n_new;
    int n_max;
};

// Eight values as they come, and as fp32 numbers.
template <typename X>
struct Eight {
    uint4 raw[sizeof(X) / 2];

    __device__ __forceinline__ void load(const X *p)
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(X) / 2); ++i) raw[i] = ld_stream16(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(X) / 2); ++i) raw[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
        if constexpr (sizeof(X) == 4) {
            const uint32_t z[4] = {raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(w[i]);
                v[4 + i] = __uint_as_float(z[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
};

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d)
{
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

template <int D, typename X>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(const AppendArgs a)
{
    constexpr int TPR = D / 8;                       // threads a row
    constexpr int RPP = kAppendThreads / TPR;        // rows a pass
    constexpr int PASSES = kPage / RPP;
    __shared__ float s_max[kAppendThreads / 32];
    __shared__ int8_t s_lut[256];
    __shared__ uint32_t s_lo[kAppendThreads / 32][TPR][2], s_hi[kAppendThreads / 32][TPR][2];
    start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int which = blockIdx.x & 1;
    const int kh = blockIdx.y, s = blockIdx.z;
    const int64_t len = max(0, __ldg(a.L.kv_len + s));
    const int n = min(a.n_max, a.n_new ? max(0, __ldg(a.n_new + s)) : a.n_max);
    if (n == 0) return;
    const int64_t blk = len / kPage + (blockIdx.x >> 1);
    const int64_t p0 = blk * kPage;                  // token of the page's row 0
    if (p0 >= len + n) return;
    const int r_lo = static_cast<int>(max(int64_t(0), len - p0));            // first row written
    const int r_hi = static_cast<int>(min(int64_t(kPage), len + n - p0));
    const int c8 = (tid % TPR) * 8, r0 = tid / TPR;
    const X *x = static_cast<const X *>(a.x[which]);
    // the values and the page's id are on their way together
    Eight<X> in[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = r0 + i * RPP;
        if (r >= r_lo && r < r_hi)
            in[i].load(x + ((static_cast<int64_t>(s) * a.n_max + (p0 + r - len)) * a.L.Hk + kh) * D + c8);
        else
            in[i].clear();
    }
    const int64_t entry = (static_cast<int64_t>(s) * a.L.Hk + kh) * a.L.cap + blk;
    const int64_t id = blk < a.L.cap ? __ldg(a.L.ids + entry) : -1;
    if (id < 0 || id >= a.L.n_pages) {
        if (tid == 0) atomicOr(a.L.status, kStatusAppend);
        return;
    }
    const float d0 = r_lo > 0 ? a.scale[which][id] : 0.f;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        float v[8];
        in[i].values(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float m = fabsf(v[e]);
            amax = fmaxf(amax, m <= 3.402823466e38f ? m : 0.f);             // finite values only
        }
    }
    // (magnitudes: their order is that of their bits)
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if (lane == 0) s_max[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
    const float d1 = fmaxf(d0, __fdiv_rn(amax, 127.f));
    const bool recode = r_lo > 0 && d1 != d0;
    int8_t *page = a.codes[which] + id * (kPage * D);
    const float up = d1 < 0x1p-100f ? 0x1p40f : 1.f;                        // see nearest_code
    float rd;                                                               // 1 / (d' up), off by 2^-22 at most
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rd) : "f"(d1 * up));
    uint32_t lo[2] = {0x7f7f7f7fu, 0x7f7f7f7fu}, hi[2] = {0x81818181u, 0x81818181u};
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = r0 + i * RPP;
        if (r < r_lo || r >= r_hi) continue;
        float v[8];
        in[i].values(v);
        int q[8];
        bool sure = d1 > 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float t = v[e] * up * rd;
            const float r = rintf(t);
            sure = sure && fabsf(t - r) < 0.5f - 0x1p-13f;               // (false for what is not finite)
            q[e] = static_cast<int>(r);
        }
        if (!sure) {
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = d1 > 0.f ? nearest_code(v[e] * up, d1 * up) : 0;
        }
        const uint32_t w0 = pack4(q[0], q[1], q[2], q[3]), w1 = pack4(q[4], q[5], q[6], q[7]);
        *reinterpret_cast<uint2 *>(page + r * D + c8) = make_uint2(w0, w1);
        lo[0] = __vmins4(lo[0], w0);
        lo[1] = __vmins4(lo[1], w1);
        hi[0] = __vmaxs4(hi[0], w0);
        hi[1] = __vmaxs4(hi[1], w1);
    }
    if (recode) {
        const int c = static_cast<int8_t>(tid);
        double t = d1 > 0.f ? rint(static_cast<double>(c) * static_cast<double>(d0) / static_cast<double>(d1)) : 0.0;
        s_lut[tid] = static_cast<int8_t>(fmin(fmax(t, -127.0), 127.0));
        __syncthreads();
        for (int i = tid; i < r_lo * TPR; i += kAppendThreads) {
            uint2 w = *reinterpret_cast<const uint2 *>(page + i * 8);
            uint8_t *b = reinterpret_cast<uint8_t *>(&w);
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = static_cast<uint8_t>(s_lut[b[e]]);
            *reinterpret_cast<uint2 *>(page + i * 8) = w;
        }
    }
    if (tid == 0) a.scale[which][id] = d1;
    if (which != 0) return;
    // the channels' extremes: over a thread's rows, the warp's, then the CTA's
#pragma unroll
    for (int o = TPR; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            lo[e] = __vmins4(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
            hi[e] = __vmaxs4(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
        }
    if (lane < TPR) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            s_lo[warp][lane][e] = lo[e];
            s_hi[warp][lane][e] = hi[e];
        }
    }
    __syncthreads();
    if (tid < TPR * 2) {
        const int c = tid >> 1, e = tid & 1;
        uint32_t l = s_lo[0][c][e], m = s_hi[0][c][e];
#pragma unroll
        for (int w = 1; w < kAppendThreads / 32; ++w) {
            l = __vmins4(l, s_lo[w][c][e]);
            m = __vmaxs4(m, s_hi[w][c][e]);
        }
        uint32_t *pl = reinterpret_cast<uint32_t *>(a.k_min + id * D) + tid;
        uint32_t *pm = reinterpret_cast<uint32_t *>(a.k_max + id * D) + tid;
        if (r_lo > 0) {
            uint32_t ol = *pl, om = *pm;
            if (recode) {
                uint8_t *bl = reinterpret_cast<uint8_t *>(&ol), *bm = reinterpret_cast<uint8_t *>(&om);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    bl[i] = static_cast<uint8_t>(s_lut[bl[i]]);
                    bm[i] = static_cast<uint8_t>(s_lut[bm[i]]);
                }
            }
            l = __vmins4(l, ol);
            m = __vmaxs4(m, om);
        }
        *pl = l;
        *pm = m;
    }
}

int launch_append(skv_handle *h, const skv_q8_pool &pool, const Lists &L, int n_max, int x_type, const void *k_new,
                  const void *v_new, const int32_t *n_new, cudaStream_t st)
{
    AppendArgs a;
    a.L = L;
    a.codes[0] = pool.k;
    a.codes[1] = pool.v;
    a.scale[0] = pool.k_scale;
    a.scale[1] = pool.v_scale;
    a.k_min = pool.k_min;
    a.k_max = pool.k_max;
    a.x[0] = k_new;
    a.x[1] = v_new;
    a.n_new = n_new;
    a.n_max = n_max;
    // a run of n tokens touches at most ceil((n + 63) / 64) pages
    const int64_t blocks = (static_cast<int64_t>(n_max) + 2 * kPage - 2) / kPage;
    const dim3 grid(static_cast<unsigned>(2 * blocks), L.Hk, L.S);
    cudaError_t e;
    if (x_type == SKV_F32)
        e = pool.D == 128 ? launch(append_kernel<128, float>, grid, kAppendThreads, 0, st, a)
                          : launch(append_kernel<64, float>, grid, kAppendThreads, 0, st, a);
    else
        e = pool.D == 128 ? launch(append_kernel<128, __half>, grid, kAppendThreads, 0, st, a)
                          : launch(append_kernel<64, __half>, grid, kAppendThreads, 0, st, a);
    return cuda_fail(h, e, "8-bit append launch");
}

}  // namespace q8
}  // namespace skv
