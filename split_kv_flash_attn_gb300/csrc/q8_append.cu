// q8_append.cu -- writing tokens into 8-bit pages.
//
// One CTA for each (page touched, K or V, KV head, sequence).  It holds the
// page's new values in registers (at most 64 rows of D: 8 values of 4 or 8 rows
// a thread), takes their largest magnitude, d' = max(|d|, fp32(amax/127)),
// and writes the codes nearest x/d' and, for K, the channels' smallest and
// largest codes.  Only when d' is not d and the page holds earlier tokens are those
// read and recoded, through a table of the 255 codes (one fp64 division each:
// c*d has 31 significant bits, so c*d/d' cannot be rounded onto a half-integer
// that it is not); rounding is monotone, so the old extremes recode like codes
// (d negative: the smallest becomes the largest).
//
// A code is rint(t), t = x (1/d') with an approximate reciprocal, when t is further
// than 2^-13 from every half-integer: t is off by less than 2^-21.4 * 128 = 2^-14.4
// and |x/d'| never exceeds 127 + 2^-16, so nothing is left to clamp.  Nearer ones (one
// value in 4000) are decided by the sign of x - h d' at the half-integer h; tiny d',
// infinities and NaN go by the exact quotient, which for every value took 31 us
// with a 4096-token prompt.
//
// Bound: a token's append is two dependent reads (length, page id) and one write deep
// (4.0 us for 32 sequences); a prompt's is bound by its instructions, close to 20
// of a warp for 32 values (two prompts of 4096 tokens, eight heads of D = 128: 14.7 us from
// fp16, 3.5 TB/s, and 16.9 from fp32, 5.0 TB/s; x read once, codes written once).
// 1024 threads a SM: three quarters and half of that took 18.7 and 23 us from fp32.
#include <algorithm>

#include "q8.cuh"

namespace skv {
namespace q8 {

// Threads of a CTA.  The same bytes as four prompts of 4096 tokens with D = 64 took 21.5
// us (fp16) and 22.8 (fp32) with 256 threads, 14.7 and 15.9 with 128; with D = 128 fp16
// rows 15.5 with 256 and 14.7 with 128, fp32 rows 16.9 and 27.5 (64 registers of rows).
__host__ __device__ constexpr int append_threads(int D, bool f16) { return f16 ? 128 : 2 * D; }

struct AppendArgs {
    Lists L;
    int8_t *codes[2];              // K, V
    float *scale[2];
    int8_t *k_min, *k_max;
    const void *x[2];              // [S][n_max][Hk][D]
    const int32_t *n_new;
    int n_max;
    int64_t page0;                 // of the pages that a list's tokens touch, the launch's first
};

__device__ __forceinline__ float max_nan(float a, float b)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

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
    // the largest magnitude, or NaN
    __device__ __forceinline__ float top() const
    {
        if constexpr (sizeof(X) == 4) {
            float v[8];
            values(v);
            return max_nan(max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3]))),
                           max_nan(max_nan(fabsf(v[4]), fabsf(v[5])), max_nan(fabsf(v[6]), fabsf(v[7]))));
        } else {
            const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
            __half2 m = __habs2(*reinterpret_cast<const __half2 *>(&w[0]));
#pragma unroll
            for (int i = 1; i < 4; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __half2 *>(&w[i])));
            const float2 f = __half22float2(m);
            return max_nan(f.x, f.y);
        }
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

// Four codes through the table.
__device__ __forceinline__ uint32_t recode4(const int8_t *lut, uint32_t w)
{
    return pack4(lut[w & 255u], lut[(w >> 8) & 255u], lut[(w >> 16) & 255u], lut[w >> 24]);
}

template <int D, typename X>
__global__ void __launch_bounds__(append_threads(D, sizeof(X) == 2), 1024 / append_threads(D, sizeof(X) == 2)) append_kernel(const AppendArgs a)
{
    constexpr int kThreads = append_threads(D, sizeof(X) == 2);
    constexpr int TPR = D / 8;                       // threads a row
    constexpr int RPP = kThreads / TPR;        // rows a pass
    constexpr int PASSES = kPage / RPP;
    __shared__ float s_max[kThreads / 32];
    __shared__ int8_t s_lut[256];
    __shared__ uint32_t s_lo[kThreads / 32][TPR][2], s_hi[kThreads / 32][TPR][2];
    start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // (heads side by side: their rows of a token are neighbours in memory)
    const int which = blockIdx.y & 1;
    const int kh = blockIdx.x, s = blockIdx.z;
    const int64_t len = max(0, __ldg(a.L.kv_len + s));
    const int n = min(a.n_max, a.n_new ? max(0, __ldg(a.n_new + s)) : a.n_max);
    if (n == 0) return;
    const int64_t blk = len / kPage + a.page0 + (blockIdx.y >> 1);
    const int64_t p0 = blk * kPage;                  // token of the page's row 0
    if (p0 >= len + n) return;
    const int r_lo = static_cast<int>(max(int64_t(0), len - p0));            // first row written
    const int r_hi = static_cast<int>(min(int64_t(kPage), len + n - p0));
    const int c8 = (tid % TPR) * 8, r0 = tid / TPR;
    // (not by index: that would copy the arguments to local memory)
    const X *x = static_cast<const X *>(which ? a.x[1] : a.x[0]);
    int8_t *const codes = which ? a.codes[1] : a.codes[0];
    float *const scale = which ? a.scale[1] : a.scale[0];
    auto at_of = [&](int r) { return ((static_cast<int64_t>(s) * a.n_max + (p0 + r - len)) * a.L.Hk + kh) * D + c8; };
    // the values and the page's id are on their way together
    Eight<X> in[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = r0 + i * RPP;
        if (r >= r_lo && r < r_hi)
            in[i].load(x + at_of(r));
        else
            in[i].clear();
    }
    const int64_t entry = (static_cast<int64_t>(s) * a.L.Hk + kh) * a.L.cap + blk;
    const int64_t id = blk < a.L.cap ? __ldg(a.L.ids + entry) : -1;
    if (id < 0 || id >= a.L.n_pages) {
        if (tid == 0) atomicOr(a.L.status, kStatusAppend);
        return;
    }
    const float d0 = r_lo > 0 ? scale[id] : 0.f;
    // the largest magnitude; NaN where there is one
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) amax = max_nan(amax, in[i].top());
    const bool odd = !(amax <= 3.402823466e38f);                            // a NaN or an infinity among the values
    if (odd) {                                                              // finite values only
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            float v[8];
            in[i].values(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]) <= 3.402823466e38f ? fabsf(v[e]) : 0.f);
        }
    }
    // (magnitudes: their order is that of their bits)
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if (lane == 0) s_max[warp] = amax;
    const bool any_odd = __syncthreads_or(odd);
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
    const float d1 = fmaxf(fabsf(d0), over_127(amax));                      // (a negative scale leaves with its codes turned)
    const bool recode = r_lo > 0 && d1 != d0;
    const bool plain = !any_odd && d1 >= 0x1p-100f;                         // every value finite, d' not tiny
    int8_t *page = codes + id * (kPage * D);
    const float up = d1 < 0x1p-100f ? 0x1p40f : 1.f;                        // see nearest_code
    float rd;                                                               // 1 / d', off by 2^-22 at most
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rd) : "f"(d1));
    float lo[8], hi[8];                                                     // of the thread's channels
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        lo[e] = 127.f;
        hi[e] = -127.f;
    }
    if (plain) {
        // v / d' + 1.5 2^23 rounds to an integer, whose low byte is the sum's
        constexpr float kMagic = 12582912.f;
        float c[2][8];                                                      // of two rows; NaN: none
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int r = r0 + i * RPP;
            float(&ci)[8] = c[i & 1];
            if (r >= r_lo && r < r_hi) {
                float v[8], side[8];
                uint32_t q[8];
                in[i].values(v);
                float off = 0.f;
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float m0, m1;
                    fma2(m0, m1, v[e], v[e + 1], rd, kMagic);
                    q[e] = __float_as_uint(m0);
                    q[e + 1] = __float_as_uint(m1);
                    add2(m0, m1, -kMagic, -kMagic);
                    ci[e] = m0;
                    ci[e + 1] = m1;
                    side[e] = -m0;
                    side[e + 1] = -m1;
                    fma2_to(side[e], side[e + 1], v[e], v[e + 1], rd);
                    off = max3(off, fabsf(side[e]), fabsf(side[e + 1]));
                }
                if (!(off < 0.5f - 0x1p-13f)) {
                    // next to a half-integer h, the sign of x - h d' decides (one rounding,
                    // so the sign is exact; d' is not tiny)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float rem = __fmaf_rn(-(ci[e] + copysignf(0.5f, side[e])), d1, v[e]) * copysignf(1.f, side[e]);
                        if (rem > 0.f || (rem == 0.f && fabsf(side[e]) > 0.25f && (q[e] & 1u))) {
                            ci[e] += copysignf(1.f, side[e]);
                            q[e] = __float_as_uint(ci[e] + kMagic);
                        }
                    }
                }
                *reinterpret_cast<uint2 *>(page + r * D + c8) = make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) ci[e] = __uint_as_float(0x7fffffffu);
            }
            if ((i & 1) && which == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    lo[e] = min3(lo[e], c[0][e], c[1][e]);
                    hi[e] = max3(hi[e], c[0][e], c[1][e]);
                }
            }
        }
        static_assert(PASSES % 2 == 0, "rows in pairs");
    } else {
        // the values once more, one by one
        for (int r = r0; r < r_hi; r += RPP) {
            if (r < r_lo) continue;
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                const float v = static_cast<float>(x[at_of(r) + e]);
                const int q = d1 > 0.f ? nearest_code(v * up, d1 * up) : 0;
                page[r * D + c8 + e] = static_cast<int8_t>(q);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    lo[k] = e == k ? fminf(lo[k], static_cast<float>(q)) : lo[k];
                    hi[k] = e == k ? fmaxf(hi[k], static_cast<float>(q)) : hi[k];
                }
            }
        }
    }
    if (recode) {
        for (int i = tid; i < 256; i += kThreads) {
            const int c = static_cast<int8_t>(i);
            const double t = d1 > 0.f ? rint(static_cast<double>(c) * static_cast<double>(d0) / static_cast<double>(d1)) : 0.0;
            s_lut[i] = static_cast<int8_t>(fmin(fmax(t, -127.0), 127.0));
        }
        __syncthreads();
        for (int i = tid; i < r_lo * TPR; i += kThreads) {
            const uint2 w = *reinterpret_cast<const uint2 *>(page + i * 8);
            *reinterpret_cast<uint2 *>(page + i * 8) = make_uint2(recode4(s_lut, w.x), recode4(s_lut, w.y));
        }
    }
    if (tid == 0) scale[id] = d1;
    if (which != 0) return;
    // the channels' extremes: over a thread's rows, the warp's, then the CTA's
    uint32_t lo4[2], hi4[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        lo4[e] = pack4(static_cast<int>(lo[4 * e]), static_cast<int>(lo[4 * e + 1]), static_cast<int>(lo[4 * e + 2]), static_cast<int>(lo[4 * e + 3]));
        hi4[e] = pack4(static_cast<int>(hi[4 * e]), static_cast<int>(hi[4 * e + 1]), static_cast<int>(hi[4 * e + 2]), static_cast<int>(hi[4 * e + 3]));
    }
#pragma unroll
    for (int o = TPR; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            lo4[e] = __vmins4(lo4[e], __shfl_xor_sync(0xffffffffu, lo4[e], o));
            hi4[e] = __vmaxs4(hi4[e], __shfl_xor_sync(0xffffffffu, hi4[e], o));
        }
    if (lane < TPR) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            s_lo[warp][lane][e] = lo4[e];
            s_hi[warp][lane][e] = hi4[e];
        }
    }
    __syncthreads();
    if (tid < TPR * 2) {
        const int c = tid >> 1, e = tid & 1;
        uint32_t l = s_lo[0][c][e], m = s_hi[0][c][e];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) {
            l = __vmins4(l, s_lo[w][c][e]);
            m = __vmaxs4(m, s_hi[w][c][e]);
        }
        uint32_t *pl = reinterpret_cast<uint32_t *>(a.k_min + id * D) + tid;
        uint32_t *pm = reinterpret_cast<uint32_t *>(a.k_max + id * D) + tid;
        if (r_lo > 0) {
            uint32_t ol = *pl, om = *pm;
            if (recode) {
                const uint32_t rl = recode4(s_lut, ol), rm = recode4(s_lut, om);
                ol = __vmins4(rl, rm);              // (a negative d exchanges the two)
                om = __vmaxs4(rl, rm);
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
    constexpr int64_t most = 65535 / 2;              // (a grid's y)
    for (a.page0 = 0; a.page0 < blocks; a.page0 += most) {
        const dim3 grid(L.Hk, static_cast<unsigned>(2 * std::min(most, blocks - a.page0)), L.S);
        cudaError_t e;
        const int threads = append_threads(pool.D, x_type == SKV_F16);
        if (x_type == SKV_F32)
            e = pool.D == 128 ? launch(append_kernel<128, float>, grid, threads, 0, st, a)
                              : launch(append_kernel<64, float>, grid, threads, 0, st, a);
        else
            e = pool.D == 128 ? launch(append_kernel<128, __half>, grid, threads, 0, st, a)
                              : launch(append_kernel<64, __half>, grid, threads, 0, st, a);
        if (e != cudaSuccess) return cuda_fail(h, e, "8-bit append launch");
    }
    return SKV_OK;
}

}  // namespace q8
}  // namespace skv
