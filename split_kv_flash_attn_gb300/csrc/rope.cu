// rope.cu -- norm and rotation of query and key rows, the same with the keys and
// values written into cache rows, and the gradients.
//
// A row is one head of one token, D values; D/8 neighbouring lanes hold it, eight
// consecutive values each (one 16-byte load of fp16), so a row's sums are
// three or four shuffles and the partner of value i in split halves, i + R/2, is eight
// values of another lane of the row (R/2 is a multiple of 8 there).
//
// Angles.  theta = pos * freq in whole turns is pos * (freq / 2 pi), of which only the
// fraction counts.  freq = m 2^e with a 24-bit m, so its turns per position are the
// product of m and the 64 leading bits of 1 / 2 pi, shifted: an integer in units of
// 2^-64 turns, off by less than freq / 2 units.  The product with pos wraps modulo
// one turn by itself, in integers, and stays exact to 2^-33 turns for
// every 32-bit position.  Its quadrant is taken off and sincospif gives the rest.
// A CTA takes a run of rows, token after token, and computes the angles of its
// tokens once (an fp64 product and cosine for each pair would cost more than the
// rows: this GPU's fp64 rate is a hundredth of its fp32 rate).
#include "internal.h"
#include "kv_encode.cuh"

namespace skv {
namespace rope {

constexpr int kThreads = 256;
// Rows of a thread, all loaded before any is computed.
constexpr int kIter = 4;

struct Side {                 // queries, or keys
    const void *x;            // rows [n][heads][D], `stride` elements a token
    int64_t stride;
    const float *w;           // norm weight or null
    void *out;                // results (forward) or gradients of x (backward)
    int64_t out_stride;
    const void *g;            // backward: gradients of the results, contiguous
};

struct Dst {                  // cache region pair
    int type;
    int64_t row_bytes;
    uint8_t *d0, *d1;
    int64_t n0, n1;
    int vec16;                // 16-byte stores are aligned (fp16 rows)
};

struct Args {
    Side q, k;
    const void *v;
    int64_t v_stride;
    int64_t n;
    int H, Hk, Hv;            // heads of q, k and (append) v
    int n_axes, half, inter;
    const int32_t *pos, *axis;
    const float *freq;
    float factor, eps;
    int o_type;               // results (forward), gradients of results (backward)
    const int32_t *positions;
    Dst kd, vd;
    int *status;
    int64_t chunks;
    float *dw;                // backward: partial weight gradients [grid][2][D]
};

// floor(2^64 / 2 pi)
constexpr uint64_t kTurns = 0x28be60db9391054aull;

// freq / 2 pi modulo one turn, in units of 2^-64 turns.
__device__ __forceinline__ uint64_t turns_of(float freq)
{
    const uint32_t bits = __float_as_uint(freq);
    const int e = (bits >> 23) & 255;
    const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int sh = 150 - max(e, 1);                    // freq = m 2^-sh
    const uint64_t lo = m * kTurns, hi = __umul64hi(m, kTurns);
    uint64_t t;
    if (sh <= 0) t = sh > -64 ? lo << -sh : 0;
    else if (sh < 64) t = (lo >> sh) | (hi << (64 - sh));
    else t = sh < 128 ? hi >> (sh - 64) : 0;
    return (bits >> 31) ? 0 - t : t;
}

// factor * (cos, sin) of pos * freq.
__device__ __forceinline__ float2 cos_sin(int32_t pos, float freq, float factor)
{
    const uint64_t phase = turns_of(freq) * static_cast<uint64_t>(static_cast<int64_t>(pos)) + 0x80000000ull;
    const int32_t ph = static_cast<int32_t>(phase >> 32);                     // 2^-32 turns
    const int32_t quad = static_cast<int32_t>(static_cast<uint32_t>(ph) + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(ph) - (static_cast<uint32_t>(quad) << 30));
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    s *= factor;
    c *= factor;
    if (quad & 1) {
        const float x = c;
        c = -s;
        s = x;
    }
    if (quad & 2) {
        c = -c;
        s = -s;
    }
    return make_float2(c, s);
}

// Eight values of a type as loaded, and as fp32.
template <int XT>
struct Raw {
    uint4 a[XT == SKV_F32 ? 2 : 1];
};
template <int XT>
__device__ __forceinline__ Raw<XT> load8(const void *p, int64_t at)
{
    Raw<XT> r;
    if constexpr (XT == SKV_F32) {
        const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + at);
        r.a[0] = __ldg(s);
        r.a[1] = __ldg(s + 1);
    } else {
        r.a[0] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at));
    }
    return r;
}
template <int XT>
__device__ __forceinline__ Raw<XT> zero8()
{
    Raw<XT> r;
    r.a[0] = make_uint4(0, 0, 0, 0);
    if constexpr (XT == SKV_F32) r.a[1] = r.a[0];
    return r;
}
template <int XT>
__device__ __forceinline__ void to_f32(const Raw<XT> &r, float (&v)[8])
{
    const uint32_t w[4] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w};
    if constexpr (XT == SKV_F32) {
        const uint32_t u[4] = {r.a[1].x, r.a[1].y, r.a[1].z, r.a[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(w[i]);
            v[4 + i] = __uint_as_float(u[i]);
        }
    } else if constexpr (XT == SKV_F16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store_as(int type, void *p, int64_t at, const float (&v)[8])
{
    if (type == SKV_F32) {
        float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if (type == SKV_F16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) =
            make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
}

// The run of rows [first, first + rows) that a CTA takes, its tokens' angles in `tab`
// [token][half], for tokens from `t0` on.
struct Chunk {
    int64_t t0;
    int head0, heads, rows;
};
template <int D>
constexpr int kRows = kThreads / (D / 8) * kIter;

template <int D>
__device__ __forceinline__ Chunk chunk_of(const Args &a, int64_t c)
{
    Chunk k;
    k.heads = a.H + a.Hk + a.Hv;
    const int64_t first = c * kRows<D>;
    k.t0 = first / k.heads;
    k.head0 = static_cast<int>(first - k.t0 * k.heads);
    const int64_t left = a.n * k.heads - first;
    k.rows = left < kRows<D> ? static_cast<int>(left) : kRows<D>;
    return k;
}
__device__ __forceinline__ void angles(const Args &a, const Chunk &k, float2 *tab)
{
    const int tokens = (k.head0 + k.rows - 1) / k.heads + 1;
    for (int i = threadIdx.x; i < tokens * a.half; i += kThreads) {
        const int t = i / a.half, p = i - t * a.half;
        int ax = a.axis ? __ldg(a.axis + p) : 0;
        if (static_cast<unsigned>(ax) >= static_cast<unsigned>(a.n_axes)) ax = 0;
        tab[i] = cos_sin(__ldg(a.pos + ax * a.n + k.t0 + t), __ldg(a.freq + p), a.factor);
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float s)
{
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Turn a row's values (lane l of its LPR lanes) by its token's angles; back: by
// their negatives.  All lanes of the warp take part.
template <int LPR, bool BACK>
__device__ __forceinline__ void turn(const Args &a, const float2 *tab, int l, float (&v)[8])
{
    if (a.inter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = 4 * l + i;
            if (p < a.half) {
                const float2 cs = tab[p];
                const float sn = BACK ? -cs.y : cs.y;
                const float x = v[2 * i], y = v[2 * i + 1];
                v[2 * i] = x * cs.x - y * sn;
                v[2 * i + 1] = x * sn + y * cs.x;
            }
        }
    } else {
        const int hl = a.half >> 3;                        // lanes of a half
        const int lane = threadIdx.x & 31;
        const bool lower = l < hl, in = l < 2 * hl;
        const int src = lower ? lane + hl : in ? lane - hl : lane;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, v[i], src);
        if (in) {
            const float4 *cs = reinterpret_cast<const float4 *>(tab + 8 * (lower ? l : l - hl));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 c = cs[i];                    // (cos, sin) of two pairs
                const bool neg = BACK ? !lower : lower;    // lower: a cos - b sin, upper: b cos + a sin
                v[2 * i] = v[2 * i] * c.x + (neg ? -c.y : c.y) * o[2 * i];
                v[2 * i + 1] = v[2 * i + 1] * c.z + (neg ? -c.w : c.w) * o[2 * i + 1];
            }
        }
    }
}

__device__ __forceinline__ void load_weight(const float *w, int l, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __ldg(w + 8 * l + i);
}

// One row's part into its cache row; p: its position, or negative.
__device__ __forceinline__ void put_cache(const Dst &d, int D, int64_t p, int head, int l, const float (&v)[8], int *status)
{
    const bool quant = d.type != SKV_F16;
    __half d16;
    uint32_t w0 = 0, w1 = 0;
    if (quant) {                                           // the whole warp takes part
        if (d.type == SKV_Q8_0) encode8<SKV_Q8_0>(v, d16, w0, w1);
        else encode8<SKV_Q4_0>(v, d16, w0, w1);
    }
    if (p < 0) return;
    if (p >= d.n0 + d.n1) {
        if (l == 0 && head == 0) atomicOr(status, 2);
        return;
    }
    uint8_t *row = p < d.n0 ? d.d0 + p * d.row_bytes : d.d1 + (p - d.n0) * d.row_bytes;
    if (quant) {
        const int blk = d.type == SKV_Q8_0 ? 34 : 18;
        uint8_t *b = row + (static_cast<int64_t>(head) * (D / 32) + (l >> 2)) * blk;
        if (d.type == SKV_Q8_0) store8<SKV_Q8_0>(b, l, d16, w0, w1);
        else store8<SKV_Q4_0>(b, l, d16, w0, w1);
        return;
    }
    uint8_t *o = row + (static_cast<int64_t>(head) * D + 8 * l) * 2;
    const uint32_t h[4] = {pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7])};
    if (d.vec16) {
        *reinterpret_cast<uint4 *>(o) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t *>(o)[i] = h[i];   // rows are 4-byte aligned
    }
}

template <int XT, int D, bool CACHE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Args a)
{
    constexpr int LPR = D / 8, RPI = kThreads / LPR;
    extern __shared__ float4 smem4[];
    float2 *tab = reinterpret_cast<float2 *>(smem4);
    const Chunk ck = chunk_of<D>(a, blockIdx.x);
    const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
    Raw<XT> raw[kIter];
    int tok[kIter], head[kIter];                           // token after t0 and head, or head -1
    int32_t at[kIter], p0[kIter];
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        const int r = it * RPI + g;
        raw[it] = zero8<XT>();
        tok[it] = 0;
        head[it] = -1;
        at[it] = -1;
        p0[it] = -1;
        if (r < ck.rows) {
            const int x = ck.head0 + r;
            tok[it] = x / ck.heads;
            const int hd = x - tok[it] * ck.heads;
            head[it] = hd;
            const int64_t t = ck.t0 + tok[it];
            if (hd < a.H) raw[it] = load8<XT>(a.q.x, t * a.q.stride + hd * D + 8 * l);
            else if (hd < a.H + a.Hk) raw[it] = load8<XT>(a.k.x, t * a.k.stride + (hd - a.H) * D + 8 * l);
            else raw[it] = load8<XT>(a.v, t * a.v_stride + (hd - a.H - a.Hk) * D + 8 * l);
            p0[it] = __ldg(a.pos + t);
            if (CACHE && hd >= a.H) at[it] = __ldg(a.positions + t);
        }
    }
    angles(a, ck, tab);
    __syncthreads();
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
        float v[8];
        const int hd = head[it];
        const bool isq = hd < a.H, isk = !isq && hd < a.H + a.Hk;
        to_f32<XT>(p0[it] < 0 ? zero8<XT>() : raw[it], v); // a padding token's rows are zeros
        if (a.q.w || a.k.w) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
            ss = row_sum<LPR>(ss);
            const float *w = hd < 0 ? nullptr : isq ? a.q.w : isk ? a.k.w : nullptr;
            if (w) {
                const float rs = rsqrtf(ss * (1.f / D) + a.eps);
                float wv[8];
                load_weight(w, l, wv);
                // padding stays zero whatever eps is
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = p0[it] < 0 ? 0.f : v[i] * rs * wv[i];
            }
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i];
        turn<LPR, false>(a, tab + tok[it] * a.half, l, y);
        if (!isq && !isk) {                                // values do not turn
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = v[i];
        }
        if (p0[it] < 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = 0.f;
        }
        const int64_t t = ck.t0 + tok[it];
        if (hd >= 0 && isq) store_as(CACHE ? SKV_F16 : a.o_type, a.q.out, (t * a.H + hd) * D + 8 * l, y);
        if constexpr (CACHE) {
            const int64_t p = p0[it] < 0 ? -1 : at[it];
            if (__any_sync(0xffffffffu, isk)) put_cache(a.kd, D, isk ? p : -1, hd - a.H, l, y, a.status);
            const bool isv = hd >= a.H + a.Hk;
            if (__any_sync(0xffffffffu, isv)) put_cache(a.vd, D, isv ? p : -1, hd - a.H - a.Hk, l, y, a.status);
        } else {
            if (isk) store_as(a.o_type, a.k.out, (t * a.Hk + hd - a.H) * D + 8 * l, y);
        }
    }
}

// Gradients.  With a norm, each thread also sums its eight columns of the weights'
// gradients over its rows; a CTA takes chunks in turn (a fixed deal), adds up its
// threads' sums at the end and leaves them in its own slot of dw.
template <int GT, int XT, int D, bool NORM>
__global__ void __launch_bounds__(kThreads) rope_back_kernel(const Args a)
{
    constexpr int LPR = D / 8, RPI = kThreads / LPR;
    extern __shared__ float4 smem4[];
    float2 *tab = reinterpret_cast<float2 *>(smem4);
    const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
    float sq[8], sk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sq[i] = sk[i] = 0.f;
    for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        const Chunk ck = chunk_of<D>(a, c);
        Raw<XT> raw[NORM ? kIter : 1];
        Raw<GT> grad[kIter];
        int tok[kIter], head[kIter];
        int32_t p0[kIter];
#pragma unroll
        for (int it = 0; it < kIter; ++it) {
            const int r = it * RPI + g;
            if (NORM) raw[it] = zero8<XT>();
            grad[it] = zero8<GT>();
            tok[it] = 0;
            head[it] = -1;
            p0[it] = -1;
            if (r < ck.rows) {
                const int x = ck.head0 + r;
                tok[it] = x / ck.heads;
                const int hd = x - tok[it] * ck.heads;
                head[it] = hd;
                const int64_t t = ck.t0 + tok[it];
                const Side &s = hd < a.H ? a.q : a.k;
                const int hh = hd < a.H ? hd : hd - a.H, hs = hd < a.H ? a.H : a.Hk;
                grad[it] = load8<GT>(s.g, (t * hs + hh) * D + 8 * l);
                if (NORM && s.w) raw[it] = load8<XT>(s.x, t * s.stride + hh * D + 8 * l);
                p0[it] = __ldg(a.pos + t);
            }
        }
        angles(a, ck, tab);
        __syncthreads();
#pragma unroll
        for (int it = 0; it < kIter; ++it) {
            const int hd = head[it];
            const bool isq = hd < a.H, pad = p0[it] < 0;
            float y[8];
            to_f32<GT>(pad ? zero8<GT>() : grad[it], y);
            turn<LPR, true>(a, tab + tok[it] * a.half, l, y);
            if (NORM) {
                const float *w = hd < 0 ? nullptr : isq ? a.q.w : a.k.w;
                float x[8];
                to_f32<XT>(pad ? zero8<XT>() : raw[it], x);
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
                ss = row_sum<LPR>(ss);
                const float rs = rsqrtf(ss * (1.f / D) + a.eps);
                float u[8], m = 0.f;
                float wv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) wv[i] = 1.f;
                if (w) load_weight(w, l, wv);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] *= rs;
                    u[i] = y[i] * wv[i];
                    m = fmaf(u[i], x[i], m);
                }
                m = row_sum<LPR>(m) * (1.f / D);
                if (w && !pad) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float s = y[i] * x[i];
                        if (isq) sq[i] += s;
                        else sk[i] += s;
                        y[i] = rs * (u[i] - x[i] * m);
                    }
                }
            }
            if (pad) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = 0.f;
            }
            if (hd >= 0) {
                const Side &s = isq ? a.q : a.k;
                const int64_t t = ck.t0 + tok[it];
                store_as(XT, s.out, t * s.out_stride + (isq ? hd : hd - a.H) * D + 8 * l, y);
            }
        }
        __syncthreads();                                   // the table is used again
    }
    if constexpr (NORM) {
        float *red = reinterpret_cast<float *>(smem4);     // [warp][2][D]
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) {
                sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], o);
                sk[i] += __shfl_xor_sync(0xffffffffu, sk[i], o);
            }
            if (lane < LPR) {
                red[(warp * 2) * D + 8 * l + i] = sq[i];
                red[(warp * 2 + 1) * D + 8 * l + i] = sk[i];
            }
        }
        __syncthreads();
        if (threadIdx.x < 2 * D) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) s += red[w * 2 * D + threadIdx.x];
            a.dw[static_cast<int64_t>(blockIdx.x) * 2 * D + threadIdx.x] = s;
        }
    }
}

// The partial sums of the weights' gradients, in the order of their CTAs: 32 columns
// a CTA, 32 threads a column.
__global__ void __launch_bounds__(1024) rope_weight_kernel(const float *dw, int parts, int D, float *dqw, float *dkw)
{
    __shared__ float red[32][33];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    float s = 0.f;
    for (int p = g; p < parts; p += 32) s += dw[static_cast<int64_t>(p) * 2 * D + col];
    red[g][c] = s;
    __syncthreads();
    s = red[c][g];                                         // column g's sum of group c
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (c == 0) {
        const int out = blockIdx.x * 32 + g;
        float *d = out < D ? dqw : dkw;
        if (d) d[out < D ? out : out - D] = s;
    }
}

static int elem_size(int type) { return type == SKV_F32 ? 4 : 2; }
static bool row_type(int t) { return t == SKV_F32 || t == SKV_F16 || t == SKV_BF16; }
static bool misaligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

static int check(skv_handle *h, const skv_rope_spec *s, int64_t n, int32_t H, int32_t Hk, int32_t x_type, const int32_t *pos)
{
    if (!s) return fail(h, SKV_EINVAL, "spec is NULL");
    if (s->D != 64 && s->D != 128) return fail(h, SKV_EUNSUPPORTED, "head dim %d (supported: 64, 128)", s->D);
    if (s->rot_dims < 0 || s->rot_dims > s->D || s->rot_dims % 2)
        return fail(h, SKV_EINVAL, "rot_dims %d: even and at most D is wanted", s->rot_dims);
    if (!s->interleaved && s->rot_dims % 16)
        return fail(h, SKV_EUNSUPPORTED, "rot_dims %d: a multiple of 16 is wanted for split halves", s->rot_dims);
    if (s->n_axes < 1 || s->n_axes > 8) return fail(h, SKV_EINVAL, "n_axes %d: 1 to 8", s->n_axes);
    if (s->rot_dims && !s->freq) return fail(h, SKV_EINVAL, "freq is NULL");
    if (n < 0 || n > INT32_MAX || H < 0 || Hk < 0 || H > 65535 || Hk > 65535)
        return fail(h, SKV_EINVAL, "bad sizes n=%lld H=%d Hk=%d", (long long)n, H, Hk);
    if (!row_type(x_type)) return fail(h, SKV_EINVAL, "unknown row type %d", x_type);
    if (n > 0 && !pos) return fail(h, SKV_EINVAL, "pos is NULL");
    if (misaligned(pos, 4) || misaligned(s->freq, 4) || misaligned(s->axis, 4))
        return fail(h, SKV_EUNSUPPORTED, "pos, freq and axis must be 4-byte aligned");
    return SKV_OK;
}
static int check_rows(skv_handle *h, const char *name, const void *p, int64_t stride, int heads, int D, int type, int64_t n)
{
    if (!heads || !n) return SKV_OK;
    if (!p) return fail(h, SKV_EINVAL, "%s is NULL", name);
    if (n > 1 && (stride < static_cast<int64_t>(heads) * D || stride > (int64_t(1) << 40)))
        return fail(h, SKV_EINVAL, "%s: stride %lld holds no %d heads of %d", name, (long long)stride, heads, D);
    if (misaligned(p, 16) || (n > 1 && stride * elem_size(type) % 16))
        return fail(h, SKV_EUNSUPPORTED, "%s: base and stride must be multiples of 16 bytes", name);
    return SKV_OK;
}
static int check_dst(skv_handle *h, const char *name, const skv_cache_dst *c, int Hk, int D, Dst *d)
{
    if (!c) return fail(h, SKV_EINVAL, "%s is NULL", name);
    const int64_t seg = segment_bytes(c->type, D);
    if (seg < 0) return fail(h, SKV_EINVAL, "%s: unknown element type %d", name, c->type);
    if (c->n_rows0 < 0 || c->n_rows1 < 0 || c->row_bytes < Hk * seg)
        return fail(h, SKV_EINVAL, "%s: bad sizes (rows %lld + %lld of %lld bytes)", name, (long long)c->n_rows0,
                    (long long)c->n_rows1, (long long)c->row_bytes);
    if ((c->n_rows0 > 0 && !c->dst0) || (c->n_rows1 > 0 && !c->dst1)) return fail(h, SKV_EINVAL, "%s: NULL region", name);
    int rc = device_address(h, c->n_rows0 > 0 ? c->dst0 : nullptr, &d->d0);
    if (!rc) rc = device_address(h, c->n_rows1 > 0 ? c->dst1 : nullptr, &d->d1);
    if (rc) return rc;
    const int al = c->type == SKV_F16 ? 4 : 2;
    if (c->row_bytes % al || misaligned(d->d0, al) || misaligned(d->d1, al))
        return fail(h, SKV_EUNSUPPORTED, "%s: base and row stride must be %d-byte aligned", name, al);
    d->type = c->type;
    d->row_bytes = c->row_bytes;
    d->n0 = c->n_rows0;
    d->n1 = c->n_rows1;
    d->vec16 = c->row_bytes % 16 == 0 && !misaligned(d->d0, 16) && !misaligned(d->d1, 16);
    return SKV_OK;
}

static Args base_args(skv_handle *h, const skv_rope_spec *s, int64_t n, int H, int Hk, int Hv, const int32_t *pos)
{
    Args a{};
    a.n = n;
    a.H = H;
    a.Hk = Hk;
    a.Hv = Hv;
    a.n_axes = s->n_axes;
    a.half = s->rot_dims / 2;
    a.inter = s->interleaved ? 1 : 0;
    a.pos = pos;
    a.axis = s->n_axes > 1 ? s->axis : nullptr;
    a.freq = s->freq;
    a.factor = s->factor;
    a.eps = s->eps;
    a.status = h->status;
    const int64_t rows = n * (H + Hk + Hv), per = kThreads / (s->D / 8) * kIter;
    a.chunks = (rows + per - 1) / per;
    return a;
}
// Shared memory of a chunk's angles: at most its rows' tokens.
static int table_bytes(const Args &a, int D)
{
    const int rows = kThreads / (D / 8) * kIter, heads = a.H + a.Hk + a.Hv;
    const int tokens = heads == 1 ? rows : (rows - 2) / heads + 2;
    return tokens * a.half * static_cast<int>(sizeof(float2));
}

template <bool CACHE>
static int launch(skv_handle *h, const Args &a, int x_type, int D, cudaStream_t st)
{
    if (a.chunks > INT32_MAX) return fail(h, SKV_EUNSUPPORTED, "too many rows for one launch");
    const int smem = table_bytes(a, D);
    const dim3 grid(static_cast<unsigned>(a.chunks));
#define SKV_ROPE(T)                                                        \
    do {                                                                   \
        if (D == 64) rope_kernel<T, 64, CACHE><<<grid, kThreads, smem, st>>>(a); \
        else rope_kernel<T, 128, CACHE><<<grid, kThreads, smem, st>>>(a);  \
    } while (0)
    if (x_type == SKV_F32) SKV_ROPE(SKV_F32);
    else if (x_type == SKV_F16) SKV_ROPE(SKV_F16);
    else SKV_ROPE(SKV_BF16);
#undef SKV_ROPE
    return cuda_fail(h, cudaGetLastError(), "rope launch");
}

}  // namespace rope
}  // namespace skv

using namespace skv;

extern "C" int skv_rope(skv_handle *h, const skv_rope_spec *spec, int64_t n, int32_t H, int32_t Hk, int32_t x_type,
                        const void *q, int64_t q_stride, const void *k, int64_t k_stride, const float *q_weight,
                        const float *k_weight, const int32_t *pos, int32_t o_type, void *q_out, void *k_out, void *stream)
{
    if (!h) return SKV_EINVAL;
    h->err[0] = 0;
    int rc = rope::check(h, spec, n, H, Hk, x_type, pos);
    if (rc) return rc;
    if (!rope::row_type(o_type)) return fail(h, SKV_EINVAL, "unknown row type %d", o_type);
    const int D = spec->D;
    rc = rope::check_rows(h, "q", q, q_stride, H, D, x_type, n);
    if (!rc) rc = rope::check_rows(h, "k", k, k_stride, Hk, D, x_type, n);
    if (!rc) rc = rope::check_rows(h, "q_out", q_out, static_cast<int64_t>(H) * D, H, D, o_type, n);
    if (!rc) rc = rope::check_rows(h, "k_out", k_out, static_cast<int64_t>(Hk) * D, Hk, D, o_type, n);
    if (rc) return rc;
    if (rope::misaligned(q_weight, 4) || rope::misaligned(k_weight, 4))
        return fail(h, SKV_EUNSUPPORTED, "weights must be 4-byte aligned");
    if (n == 0 || H + Hk == 0) return SKV_OK;
    OnDevice on(h->device);
    rope::Args a = rope::base_args(h, spec, n, H, Hk, 0, pos);
    a.q = rope::Side{q, q_stride, q_weight, q_out, 0, nullptr};
    a.k = rope::Side{k, k_stride, k_weight, k_out, 0, nullptr};
    a.o_type = o_type;
    return rope::launch<false>(h, a, x_type, D, static_cast<cudaStream_t>(stream));
}

extern "C" int skv_rope_append(skv_handle *h, const skv_rope_spec *spec, int64_t n, int32_t H, int32_t Hk, int32_t x_type,
                               const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                               int64_t v_stride, const float *q_weight, const float *k_weight, const int32_t *pos,
                               const int32_t *positions, void *q_out, const skv_cache_dst *k_dst,
                               const skv_cache_dst *v_dst, void *stream)
{
    if (!h) return SKV_EINVAL;
    h->err[0] = 0;
    int rc = rope::check(h, spec, n, H, Hk, x_type, pos);
    if (rc) return rc;
    if (Hk < 1) return fail(h, SKV_EINVAL, "Hk %d: rows to append are wanted", Hk);
    const int D = spec->D;
    rc = rope::check_rows(h, "q", q, q_stride, H, D, x_type, n);
    if (!rc) rc = rope::check_rows(h, "k", k, k_stride, Hk, D, x_type, n);
    if (!rc) rc = rope::check_rows(h, "v", v, v_stride, Hk, D, x_type, n);
    if (!rc) rc = rope::check_rows(h, "q_out", q_out, static_cast<int64_t>(H) * D, H, D, SKV_F16, n);
    if (rc) return rc;
    if (n > 0 && !positions) return fail(h, SKV_EINVAL, "positions is NULL");
    if (rope::misaligned(positions, 4) || rope::misaligned(q_weight, 4) || rope::misaligned(k_weight, 4))
        return fail(h, SKV_EUNSUPPORTED, "positions and weights must be 4-byte aligned");
    OnDevice on(h->device);
    rope::Args a = rope::base_args(h, spec, n, H, Hk, Hk, pos);
    rc = rope::check_dst(h, "k_dst", k_dst, Hk, D, &a.kd);
    if (!rc) rc = rope::check_dst(h, "v_dst", v_dst, Hk, D, &a.vd);
    if (rc || n == 0) return rc;
    a.q = rope::Side{q, q_stride, q_weight, q_out, 0, nullptr};
    a.k = rope::Side{k, k_stride, k_weight, nullptr, 0, nullptr};
    a.v = v;
    a.v_stride = v_stride;
    a.positions = positions;
    return rope::launch<true>(h, a, x_type, D, static_cast<cudaStream_t>(stream));
}

extern "C" int skv_rope_backward(skv_handle *h, const skv_rope_spec *spec, int64_t n, int32_t H, int32_t Hk, int32_t x_type,
                                 const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                 const float *q_weight, const float *k_weight, const int32_t *pos, int32_t g_type,
                                 const void *dq_out, const void *dk_out, void *dq, int64_t dq_stride, void *dk,
                                 int64_t dk_stride, float *dq_weight, float *dk_weight, void *stream)
{
    if (!h) return SKV_EINVAL;
    h->err[0] = 0;
    int rc = rope::check(h, spec, n, H, Hk, x_type, pos);
    if (rc) return rc;
    if (!rope::row_type(g_type)) return fail(h, SKV_EINVAL, "unknown row type %d", g_type);
    const int D = spec->D;
    const bool norm = q_weight || k_weight;
    if (q_weight) rc = rope::check_rows(h, "q", q, q_stride, H, D, x_type, n);
    if (!rc && k_weight) rc = rope::check_rows(h, "k", k, k_stride, Hk, D, x_type, n);
    if (!rc) rc = rope::check_rows(h, "dq_out", dq_out, static_cast<int64_t>(H) * D, H, D, g_type, n);
    if (!rc) rc = rope::check_rows(h, "dk_out", dk_out, static_cast<int64_t>(Hk) * D, Hk, D, g_type, n);
    if (!rc) rc = rope::check_rows(h, "dq", dq, dq_stride, H, D, x_type, n);
    if (!rc) rc = rope::check_rows(h, "dk", dk, dk_stride, Hk, D, x_type, n);
    if (rc) return rc;
    if (!q_weight != !dq_weight || !k_weight != !dk_weight)
        return fail(h, SKV_EINVAL, "a weight and its gradient go together");
    if (rope::misaligned(q_weight, 4) || rope::misaligned(k_weight, 4) || rope::misaligned(dq_weight, 4) ||
        rope::misaligned(dk_weight, 4))
        return fail(h, SKV_EUNSUPPORTED, "weights must be 4-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    OnDevice on(h->device);
    rope::Args a = rope::base_args(h, spec, n, H, Hk, 0, pos);
    a.q = rope::Side{q, q_stride, q_weight, dq, dq_stride, dq_out};
    a.k = rope::Side{k, k_stride, k_weight, dk, dk_stride, dk_out};
    if (!norm && a.chunks == 0) return SKV_OK;
    if (a.chunks > INT32_MAX) return fail(h, SKV_EUNSUPPORTED, "too many rows for one launch");
    // with weights: as many CTAs as are resident at once, each with a slot of sums
    const int64_t most = norm ? 4 * static_cast<int64_t>(h->sm_count) : INT32_MAX;
    const unsigned grid = static_cast<unsigned>(a.chunks < most ? a.chunks : most);
    if (norm && grid) {
        if ((rc = ensure_workspace(h, static_cast<size_t>(grid) * 2 * D * sizeof(float), st))) return rc;
        a.dw = static_cast<float *>(h->workspace);
    }
    int smem = rope::table_bytes(a, D);
    if (norm && smem < rope::kThreads / 32 * 2 * D * 4) smem = rope::kThreads / 32 * 2 * D * 4;
    if (grid) {
#define SKV_BACK(G, X, N)                                                                           \
    do {                                                                                            \
        if (D == 64) rope::rope_back_kernel<G, X, 64, N><<<grid, rope::kThreads, smem, st>>>(a);    \
        else rope::rope_back_kernel<G, X, 128, N><<<grid, rope::kThreads, smem, st>>>(a);           \
    } while (0)
#define SKV_BACK_N(G, X)              \
    do {                              \
        if (norm) SKV_BACK(G, X, true); \
        else SKV_BACK(G, X, false);   \
    } while (0)
#define SKV_BACK_X(G)                                             \
    do {                                                          \
        if (x_type == SKV_F32) SKV_BACK_N(G, SKV_F32);            \
        else if (x_type == SKV_F16) SKV_BACK_N(G, SKV_F16);       \
        else SKV_BACK_N(G, SKV_BF16);                             \
    } while (0)
        if (g_type == SKV_F32) SKV_BACK_X(SKV_F32);
        else if (g_type == SKV_F16) SKV_BACK_X(SKV_F16);
        else SKV_BACK_X(SKV_BF16);
#undef SKV_BACK_X
#undef SKV_BACK_N
#undef SKV_BACK
        rc = cuda_fail(h, cudaGetLastError(), "rope gradient launch");
        if (rc) return rc;
    }
    if (norm) {
        rope::rope_weight_kernel<<<2 * D / 32, 1024, 0, st>>>(a.dw, static_cast<int>(grid), D, dq_weight, dk_weight);
        rc = cuda_fail(h, cudaGetLastError(), "rope weight launch");
    }
    return rc;
}
