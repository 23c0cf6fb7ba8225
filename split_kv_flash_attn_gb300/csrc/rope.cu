// rope.cu -- norm and rotation of query and key rows, the same with the keys and
// values written into cache rows, and the gradients.
//
// A row is one head of one token, D values; D/8 neighbouring lanes hold it, a lane two groups of
// four consecutive values chosen so that both values of a pair are its own: in split halves
// groups l and R/8 + l.  So a row costs no exchange but the sum of its squares, and since a
// normed row is 1/rms times the row times weights, the weights go into the angles' factors.
//
// The rows of all tokens stand in one line: a token's query rows, key rows and value rows, cut into
// batches of 2 KB.  Each warp takes an equal run of batches and keeps a token's angles in registers for
// all rows of one kind.  It asks for a batch while it computes the one before (across tokens
// too); the gradients, which read twice as much for a row, keep three batches in flight
// into the warp's own shared memory.
//
// Angles.  theta = pos * freq in whole turns is pos * (freq / 2 pi), of which only the
// fraction counts.  freq = m 2^e with a 24-bit m, so its turns per position are the
// product of m and the 64 leading bits of 1 / 2 pi, shifted: an integer in units of
// 2^-64 turns, off by less than freq / 2 units.  The product with pos wraps modulo
// one turn by itself, in integers, and stays exact to 2^-33 turns for
// every 32-bit position.  Its quadrant is taken off and sincospif gives the rest.
// (An fp64 product and cosine for each pair would cost more than the rows: this
// GPU's fp64 rate is a hundredth of its fp32 rate.)  A lane computes two pairs of the token's
// and shuffles bring it those of its values.
//
// Bound by latency and instructions rather than by memory: sixteen warps an SM, a batch's chain of
// sums and a root in each.  8192 tokens of 32 + 8 heads of 128, fp16, normed (168 MB): 30.0 us, 5.6 TB/s;
// a pass of a batch's rows after the other 32, all four passes side by side (spilled) 31.6; then also batches
// of half the size 36, three CTAs an SM (80 registers, spilled) 36, the ring of the
// gradients 35, a row's values consecutive in a lane and partners by shuffles 75.  Its gradients
// (252 MB): 49 us and 3 for the weights' sums; passes side by side 48, batches in registers 60, a token a warp 83.
#include "internal.h"
#include "kv_encode.cuh"

namespace skv {
namespace rope {

constexpr int kThreads = 256;
// Shared memory of a warp for the gradients' batches in flight.
constexpr int kRing = 8192;
// CTAs resident on an SM (registers).
constexpr int kCtas = 2;

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
    int vec8;                 // 8-byte stores are aligned (fp16 rows)
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
    int bq, bk, bv;           // batches of a token's queries, keys and values
    int64_t batches;          // of all tokens
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

// factor * (cos, sin) of pos positions, `turns` each.
__device__ __forceinline__ float2 cos_sin(int32_t pos, uint64_t turns, float factor)
{
    const uint64_t phase = turns * static_cast<uint64_t>(static_cast<int64_t>(pos)) + 0x80000000ull;
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

constexpr int elem(int type) { return type == SKV_F32 ? 4 : 2; }
// A lane's two groups of four values as loaded, and as fp32.
template <int XT>
struct Raw {
    uint32_t w[2 * elem(XT)];
};
template <int XT>
__device__ __forceinline__ Raw<XT> zero_rows()
{
    Raw<XT> r;
#pragma unroll
    for (int i = 0; i < 2 * elem(XT); ++i) r.w[i] = 0;
    return r;
}
template <int XT>
__device__ __forceinline__ Raw<XT> load_rows(const void *x, int64_t at, int a, int b)
{
    Raw<XT> r;
    if constexpr (XT == SKV_F32) {
        const float *p = static_cast<const float *>(x) + at;
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p + a)), v = __ldg(reinterpret_cast<const uint4 *>(p + b));
        r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
        r.w[4] = v.x; r.w[5] = v.y; r.w[6] = v.z; r.w[7] = v.w;
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(x) + at;
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p + a)), v = __ldg(reinterpret_cast<const uint2 *>(p + b));
        r.w[0] = u.x; r.w[1] = u.y; r.w[2] = v.x; r.w[3] = v.y;
    }
    return r;
}
template <int XT>
__device__ __forceinline__ void to_f32(const Raw<XT> &r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 2 * elem(XT); ++i) {
        if constexpr (XT == SKV_F32) {
            v[i] = __uint_as_float(r.w[i]);
        } else if constexpr (XT == SKV_F16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        } else {
            v[2 * i] = __uint_as_float(r.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
        }
    }
}
// Copy a row of D values to shared memory, 16 bytes at a time, neighbouring lanes side by side (zeros
// unless `in`).
template <int XT, int LPR>
__device__ __forceinline__ void copy_row(uint32_t dst, const void *x, int64_t at, int l, bool in)
{
    const uint8_t *src = static_cast<const uint8_t *>(x) + at * elem(XT);
#pragma unroll
    for (int k = 0; k < elem(XT) / 2; ++k) cp_async16(dst + (k * LPR + l) * 16, src + (k * LPR + l) * 16, in ? 16 : 0);
}
// A lane's two groups of a row in shared memory.
template <int XT>
__device__ __forceinline__ void read_row(const uint8_t *row, int a, int b, float (&v)[8])
{
    Raw<XT> r;
    if constexpr (XT == SKV_F32) {
        const uint4 x = *reinterpret_cast<const uint4 *>(row + 4 * a), y = *reinterpret_cast<const uint4 *>(row + 4 * b);
        r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
        r.w[4] = y.x; r.w[5] = y.y; r.w[6] = y.z; r.w[7] = y.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(row + 2 * a), y = *reinterpret_cast<const uint2 *>(row + 2 * b);
        r.w[0] = x.x; r.w[1] = x.y; r.w[2] = y.x; r.w[3] = y.y;
    }
    to_f32<XT>(r, v);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// A lane's two groups as rows of a type.
__device__ __forceinline__ void store_as(int type, void *out, int64_t at, int a, int b, const float (&v)[8])
{
    if (type == SKV_F32) {
        float *p = static_cast<float *>(out) + at;
        *reinterpret_cast<float4 *>(p + a) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + b) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint16_t *p = static_cast<uint16_t *>(out) + at;
        uint2 x, y;
        if (type == SKV_F16) {
            x = make_uint2(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]));
            y = make_uint2(pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
        } else {
            x = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            y = make_uint2(pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        }
        *reinterpret_cast<uint2 *>(p + a) = x;
        *reinterpret_cast<uint2 *>(p + b) = y;
    }
}

// Two fp32 operations in one instruction; the values stand in pairs of registers.
__device__ __forceinline__ void mul2(float &d0, float &d1, float a0, float a1, float b0, float b1)
{
    const float2 d = __fmul2_rn(make_float2(a0, a1), make_float2(b0, b1));
    d0 = d.x;
    d1 = d.y;
}
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b0, float b1, float c0, float c1)
{
    const float2 d = __ffma2_rn(make_float2(a0, a1), make_float2(b0, b1), make_float2(c0, c1));
    d0 = d.x;
    d1 = d.y;
}
template <typename F>
__device__ __forceinline__ void pairs(F f)
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) f(i);
}

// The groups of lane l: their first values.
struct Groups {
    int a, b;
};
template <int LPR, bool INTER>
__device__ __forceinline__ Groups groups_of(int half, int l)
{
    if (INTER) return Groups{8 * l, 8 * l + 4};
    const int hl = half >> 2;                              // lanes of a half; the others hold what passes
    return l < hl ? Groups{4 * l, half + 4 * l} : Groups{8 * l, 8 * l + 4};
}

// What a lane needs of its token's angles: its values turn as
//   y = c v + s partner(v),
// partner: the other value of its pair; `in`: pairs that turn (of four, the first ones; the others
// have c = 1 or the weight).  back: the angles' negatives.
struct Turn {
    float c[8], s[8];
    int in;
};
struct Pairs {
    float2 p[2];                                           // (cos, sin) of pairs 2 lane, 2 lane + 1
};
// The lane's pairs: turns a position, and the axis of their positions.
struct Lane {
    uint64_t turns[2];
    int axis[2];                                           // -1: no such pair
};
__device__ __forceinline__ Lane lane_of(const Args &a)
{
    Lane r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int p = 2 * (threadIdx.x & 31) + i;
        r.turns[i] = 0;
        r.axis[i] = -1;
        if (p < a.half) {
            int ax = a.axis ? __ldg(a.axis + p) : 0;
            if (static_cast<unsigned>(ax) >= static_cast<unsigned>(a.n_axes)) ax = 0;
            r.axis[i] = ax;
            r.turns[i] = turns_of(__ldg(a.freq + p));
        }
    }
    return r;
}
// A token's positions for the lane's pairs, its first axis' one, and its cache row.
struct Token {
    int32_t pos[2], first, at;
};
__device__ __forceinline__ Token token_of(const Args &a, const Lane &ln, int t)
{
    Token r;
#pragma unroll
    for (int i = 0; i < 2; ++i) r.pos[i] = ln.axis[i] >= 0 ? __ldg(a.pos + ln.axis[i] * a.n + t) : 0;
    r.first = __ldg(a.pos + t);
    r.at = a.positions ? __ldg(a.positions + t) : -1;
    return r;
}
__device__ __forceinline__ Pairs pairs_of(const Args &a, const Lane &ln, const Token &tk)
{
    Pairs r;
#pragma unroll
    for (int i = 0; i < 2; ++i) r.p[i] = cos_sin(tk.pos[i], ln.turns[i], a.factor);
    return r;
}
// A place in the line of batches.
struct Place {
    int t, b;
    __device__ __forceinline__ void step(int per)
    {
        if (++b == per) {
            b = 0;
            ++t;
        }
    }
};

// (All lanes of the warp take part.)
template <bool BACK, bool INTER>
__device__ __forceinline__ Turn turn_of(const Args &a, const Pairs &pr, int l)
{
    Turn r;
    r.in = min(4, max(0, a.half - 4 * l));
#pragma unroll
    for (int i = 0; i < 4; ++i) {                          // pair 4l + i
        float c = __shfl_sync(0xffffffffu, pr.p[i & 1].x, 2 * l + (i >> 1));
        float s = __shfl_sync(0xffffffffu, pr.p[i & 1].y, 2 * l + (i >> 1));
        if (i >= r.in) c = 1.f;
        if (BACK) s = -s;
        r.c[INTER ? 2 * i : i] = r.c[INTER ? 2 * i + 1 : 4 + i] = c;
        r.s[INTER ? 2 * i : i] = -s;
        r.s[INTER ? 2 * i + 1 : 4 + i] = s;
    }
    return r;
}
template <bool INTER>
__device__ __forceinline__ constexpr int partner(int i) { return INTER ? i ^ 1 : i ^ 4; }

// c v + s partner(v)
template <bool INTER>
__device__ __forceinline__ void turn(const Turn &t, const float (&v)[8], float (&y)[8])
{
    pairs([&](int i) { mul2(y[i], y[i + 1], v[i], v[i + 1], t.c[i], t.c[i + 1]); });
    if (t.in == 4) {
        pairs([&](int i) { fma2(y[i], y[i + 1], v[partner<INTER>(i)], v[partner<INTER>(i + 1)], t.s[i], t.s[i + 1], y[i], y[i + 1]); });
    } else if (INTER) {                                    // (split halves turn whole lanes)
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < t.in) fma2(y[2 * i], y[2 * i + 1], v[2 * i + 1], v[2 * i], t.s[2 * i], t.s[2 * i + 1], y[2 * i], y[2 * i + 1]);
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float s)
{
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

__device__ __forceinline__ void load_weight(const float *w, const Groups &gr, float (&v)[8])
{
    const float4 x = __ldg(reinterpret_cast<const float4 *>(w + gr.a)), y = __ldg(reinterpret_cast<const float4 *>(w + gr.b));
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
}
// The weight enters the angles' factors: the value's own with c, its partner's with s.
template <bool INTER>
__device__ __forceinline__ void weigh(Turn &t, const float *w, const Groups &gr)
{
    float wv[8];
    load_weight(w, gr, wv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t.c[i] *= wv[i];
        t.s[i] *= wv[partner<INTER>(i)];
    }
}

// A lane's groups into the cache row at position p (negative: none).  Blocks of quantised rows want
// eight consecutive values of a lane: `stage` (the warp's, 32 x 8 floats) puts them in
// order where the groups are not.  All lanes of the warp take part.
template <int LPR, bool ORDERED>
__device__ __forceinline__ void put_cache(const Dst &d, int64_t p, int head, int l, const Groups &gr, float (&v)[8], float *stage,
                                          int *status)
{
    constexpr int D = LPR * 8;
    __half d16;
    uint32_t w0 = 0, w1 = 0;
    if (d.type != SKV_F16) {
        if (!ORDERED) {
            float *row = stage + ((threadIdx.x & 31) / LPR) * D;
            __syncwarp();
            *reinterpret_cast<float4 *>(row + gr.a) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(row + gr.b) = make_float4(v[4], v[5], v[6], v[7]);
            __syncwarp();
            const float4 x = reinterpret_cast<const float4 *>(row)[2 * l], y = reinterpret_cast<const float4 *>(row)[2 * l + 1];
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
            v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
        }
        if (d.type == SKV_Q8_0) encode8<SKV_Q8_0>(v, d16, w0, w1);
        else encode8<SKV_Q4_0>(v, d16, w0, w1);
    }
    if (p < 0) return;
    if (p >= d.n0 + d.n1) {
        if (l == 0 && head == 0) atomicOr(status, 2);
        return;
    }
    uint8_t *row = p < d.n0 ? d.d0 + p * d.row_bytes : d.d1 + (p - d.n0) * d.row_bytes;
    if (d.type != SKV_F16) {
        const int blk = d.type == SKV_Q8_0 ? 34 : 18;
        uint8_t *b = row + (static_cast<int64_t>(head) * (D / 32) + (l >> 2)) * blk;
        if (d.type == SKV_Q8_0) store8<SKV_Q8_0>(b, l, d16, w0, w1);
        else store8<SKV_Q4_0>(b, l, d16, w0, w1);
        return;
    }
    uint8_t *o = row + static_cast<int64_t>(head) * D * 2;
    const uint2 x = make_uint2(pack_half2(v[0], v[1]), pack_half2(v[2], v[3])), y = make_uint2(pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
    if (d.vec8) {
        *reinterpret_cast<uint2 *>(o + 2 * gr.a) = x;
        *reinterpret_cast<uint2 *>(o + 2 * gr.b) = y;
    } else {                                               // rows are 4-byte aligned
        uint32_t *q = reinterpret_cast<uint32_t *>(o + 2 * gr.a), *r = reinterpret_cast<uint32_t *>(o + 2 * gr.b);
        q[0] = x.x;
        q[1] = x.y;
        r[0] = y.x;
        r[1] = y.y;
    }
}

// Rows of a thread in a batch, by the bytes of an element that it loads.
constexpr int iter_of(int bytes) { return bytes <= 2 ? 4 : bytes <= 4 ? 2 : 1; }

template <int XT, int D, bool CACHE, bool INTER>
__global__ void __launch_bounds__(kThreads, kCtas) rope_kernel(const Args a)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR;             // lanes of a row, rows of a warp at a time
    constexpr int IT = iter_of(elem(XT)), RB = RPW * IT;   // rows of a batch
    __shared__ __align__(16) float s_stage[CACHE && !INTER ? kThreads / 32 : 1][CACHE && !INTER ? 256 : 1];
    const int lane = threadIdx.x & 31, l = lane % LPR, g = lane / LPR;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    const int64_t w0 = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t lo = a.batches / warps * w0 + min(w0, a.batches % warps);
    int left = static_cast<int>(a.batches / warps) + (w0 < a.batches % warps);
    if (!left) return;                                     // (whole warps)
    const int per = a.bq + a.bk + a.bv;
    const Groups turned = groups_of<LPR, INTER>(a.half, l), plain{8 * l, 8 * l + 4};
    Place next{static_cast<int>(lo / per), static_cast<int>(lo % per)};
    Raw<XT> asked[IT];
    auto ask = [&]() {
        const int seg = next.b < a.bq ? 0 : !CACHE || next.b < a.bq + a.bk ? 1 : 2;
        const int h0 = (seg == 0 ? next.b : seg == 1 ? next.b - a.bq : next.b - a.bq - a.bk) * RB + g, heads = seg == 0 ? a.H : a.Hk;
        const void *x = seg == 0 ? a.q.x : seg == 1 ? a.k.x : a.v;
        const int64_t x0 = static_cast<int64_t>(next.t) * (seg == 0 ? a.q.stride : seg == 1 ? a.k.stride : a.v_stride);
        const Groups gr = CACHE && seg == 2 ? plain : turned;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            asked[it] = zero_rows<XT>();
            if (h0 + it * RPW < heads) asked[it] = load_rows<XT>(x, x0 + (h0 + it * RPW) * D, gr.a, gr.b);
        }
    };
    ask();
    const Lane ln = lane_of(a);
    Token coming = token_of(a, ln, next.t);
    Pairs pr;
    Turn tr;
    bool pad = false;
    int at = -1, seg_last = -1;
    int t_last = -1;
#pragma unroll 1
    for (; left; --left) {
        const Place p = next;
        Raw<XT> raw[IT];
#pragma unroll
        for (int it = 0; it < IT; ++it) raw[it] = asked[it];
        next.step(per);
        if (left > 1) ask();
        const int seg = p.b < a.bq ? 0 : !CACHE || p.b < a.bq + a.bk ? 1 : 2;
        const float *w = seg == 0 ? a.q.w : seg == 1 ? a.k.w : nullptr;
        if (p.t != t_last) {
            pad = coming.first < 0;                        // a padding token's results are zeros
            at = pad ? -1 : coming.at;
            pr = pairs_of(a, ln, coming);
            if (p.t + 1 < a.n) coming = token_of(a, ln, p.t + 1);
        }
        if (p.t != t_last || seg != seg_last) {
            if (!CACHE || seg < 2) {
                tr = turn_of<false, INTER>(a, pr, l);
                if (w) weigh<INTER>(tr, w, turned);
            }
            t_last = p.t;
            seg_last = seg;
        }
        const int h0 = (seg == 0 ? p.b : seg == 1 ? p.b - a.bq : p.b - a.bq - a.bk) * RB, heads = seg == 0 ? a.H : a.Hk;
        const int64_t o0 = static_cast<int64_t>(p.t) * heads * D;
        // Step by step for U rows, so that their chains run side by side (rows that are none are zeros).
        constexpr int U = IT < 2 ? IT : 2;
#pragma unroll
        for (int u0 = 0; u0 < IT; u0 += U) {
            float y[U][8];
            if (!CACHE || seg < 2) {
                float ss[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float v[8], s0, s1;
                    to_f32<XT>(raw[u0 + u], v);
                    turn<INTER>(tr, v, y[u]);
                    mul2(s0, s1, v[0], v[1], v[0], v[1]);
#pragma unroll
                    for (int i = 2; i < 8; i += 2) fma2(s0, s1, v[i], v[i + 1], v[i], v[i + 1], s0, s1);
                    ss[u] = s0 + s1;
                }
                if (w) {
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1) {
#pragma unroll
                        for (int u = 0; u < U; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], o);
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float rs = rsqrtf(ss[u] * (1.f / D) + a.eps);
                        pairs([&](int i) { mul2(y[u][i], y[u][i + 1], y[u][i], y[u][i + 1], rs, rs); });
                    }
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) to_f32<XT>(raw[u0 + u], y[u]);
            }
            if (pad) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[u][i] = 0.f;
                }
            }
            auto store = [&](auto put) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int hd = h0 + (u0 + u) * RPW + g;
                    put(hd, hd < heads, y[u]);
                }
            };
            if (CACHE && seg == 2) {
                store([&](int hd, bool in, float (&v)[8]) { put_cache<LPR, true>(a.vd, in ? at : -1, hd, l, plain, v, nullptr, a.status); });
            } else if (CACHE && seg == 1) {
                store([&](int hd, bool in, float (&v)[8]) {
                    put_cache<LPR, INTER>(a.kd, in ? at : -1, hd, l, turned, v, s_stage[INTER ? 0 : threadIdx.x >> 5], a.status);
                });
            } else {
                void *out = seg == 0 ? a.q.out : a.k.out;
                const int type = CACHE ? SKV_F16 : a.o_type;
                if (type == SKV_F32) store([&](int hd, bool in, float (&v)[8]) { if (in) store_as(SKV_F32, out, o0 + hd * D, turned.a, turned.b, v); });
                else if (type == SKV_F16) store([&](int hd, bool in, float (&v)[8]) { if (in) store_as(SKV_F16, out, o0 + hd * D, turned.a, turned.b, v); });
                else store([&](int hd, bool in, float (&v)[8]) { if (in) store_as(SKV_BF16, out, o0 + hd * D, turned.a, turned.b, v); });
            }
        }
    }
}

// Gradients.  With a norm, each thread also sums its eight columns of the weights'
// gradients over its rows; a CTA adds up its threads' sums at the end and leaves them in its own
// slot of dw.
template <int GT, int XT, int D, bool NORM, bool INTER>
__global__ void __launch_bounds__(kThreads, kCtas) rope_back_kernel(const Args a)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    constexpr int IT = iter_of(elem(GT) + (NORM ? elem(XT) : 0)), RB = RPW * IT;
    constexpr int ROWG = D * elem(GT), ROWX = NORM ? D * elem(XT) : 0;
    constexpr int BATCH = RB * (ROWG + ROWX), DEPTH = kRing / BATCH;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *ring = smem + (threadIdx.x >> 5) * kRing;
    const uint32_t ring_s = smem_addr(ring);
    const int lane = threadIdx.x & 31, l = lane % LPR, g = lane / LPR;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    const int64_t w0 = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t lo = a.batches / warps * w0 + min(w0, a.batches % warps);
    int left = static_cast<int>(a.batches / warps) + (w0 < a.batches % warps);
    const Groups gr = groups_of<LPR, INTER>(a.half, l);
    float sum[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[0][i] = sum[1][i] = 0.f;
    if (left) {
        const int per = a.bq + a.bk;
        Place next{static_cast<int>(lo / per), static_cast<int>(lo % per)};
        Place p = next;
        int asks = left, slot = 0, filled = 0;
        auto ask = [&]() {
            if (asks > 0) {
                --asks;
                const bool isq = next.b < a.bq;
                const Side &s = isq ? a.q : a.k;
                const int h0 = (isq ? next.b : next.b - a.bq) * RB + g, heads = isq ? a.H : a.Hk;
                const int64_t g0 = static_cast<int64_t>(next.t) * heads * D, x0 = next.t * s.stride;
                const uint32_t dst = ring_s + filled * BATCH;
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const bool in = h0 + it * RPW < heads;
                    const int hd = in ? h0 + it * RPW : 0;
                    copy_row<GT, LPR>(dst + (it * RPW + g) * ROWG, s.g, g0 + hd * D, l, in);
                    if (NORM && s.w) copy_row<XT, LPR>(dst + RB * ROWG + (it * RPW + g) * ROWX, s.x, x0 + hd * D, l, in);
                }
                next.step(per);
                filled = filled + 1 == DEPTH ? 0 : filled + 1;
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < DEPTH - 1; ++i) ask();
        const Lane ln = lane_of(a);
        Token coming = token_of(a, ln, p.t);
        Pairs pr;
        Turn tr;
        float wv[8];
        bool pad = false;
        int t_last = -1;
        int seg_last = -1;
#pragma unroll 1
        for (; left; --left) {
            __syncwarp();
            ask();
            const bool isq = p.b < a.bq;
            const Side &s = isq ? a.q : a.k;
            const bool norm = NORM && s.w;
            if (p.t != t_last) {
                pad = coming.first < 0;
                pr = pairs_of(a, ln, coming);
                if (p.t + 1 < a.n) coming = token_of(a, ln, p.t + 1);
            }
            if (p.t != t_last || isq != seg_last) {
                tr = turn_of<true, INTER>(a, pr, l);
                if (norm) load_weight(s.w, gr, wv);
                t_last = p.t;
                seg_last = isq;
            }
            cp_async_wait<DEPTH - 1>();
            __syncwarp();
            const int h0 = (isq ? p.b : p.b - a.bq) * RB, heads = isq ? a.H : a.Hk;
            const int64_t o0 = p.t * s.out_stride;
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                if (h0 + it * RPW >= heads) break;
                const int hd = h0 + it * RPW + g;
                float y[8], v[8];
                read_row<GT>(ring + slot * BATCH + (it * RPW + g) * ROWG, gr.a, gr.b, y);
                turn<INTER>(tr, y, v);
                if (norm) {
                    float x[8], u[8], s0, s1, m0, m1;
                    read_row<XT>(ring + slot * BATCH + RB * ROWG + (it * RPW + g) * ROWX, gr.a, gr.b, x);
                    pairs([&](int i) { mul2(u[i], u[i + 1], v[i], v[i + 1], wv[i], wv[i + 1]); });
                    mul2(s0, s1, x[0], x[1], x[0], x[1]);
                    mul2(m0, m1, u[0], u[1], x[0], x[1]);
#pragma unroll
                    for (int i = 2; i < 8; i += 2) {
                        fma2(s0, s1, x[i], x[i + 1], x[i], x[i + 1], s0, s1);
                        fma2(m0, m1, u[i], u[i + 1], x[i], x[i + 1], m0, m1);
                    }
                    float ss = s0 + s1, ux = m0 + m1;
#pragma unroll
                    for (int d = LPR / 2; d; d >>= 1) {
                        ss += __shfl_xor_sync(0xffffffffu, ss, d);
                        ux += __shfl_xor_sync(0xffffffffu, ux, d);
                    }
                    const float rs = rsqrtf(ss * (1.f / D) + a.eps);
                    pairs([&](int i) { mul2(x[i], x[i + 1], x[i], x[i + 1], rs, rs); });
                    if (!pad && hd < heads) {              // (rows that are none are zeros, but eps may be 0)
                        if (isq) pairs([&](int i) { fma2(sum[0][i], sum[0][i + 1], v[i], v[i + 1], x[i], x[i + 1], sum[0][i], sum[0][i + 1]); });
                        else pairs([&](int i) { fma2(sum[1][i], sum[1][i + 1], v[i], v[i + 1], x[i], x[i + 1], sum[1][i], sum[1][i + 1]); });
                    }
                    // u - (x rs) mean(u x rs)
                    const float k = -(ux * rs) * (1.f / D);
                    pairs([&](int i) { fma2(u[i], u[i + 1], x[i], x[i + 1], k, k, u[i], u[i + 1]); });
                    pairs([&](int i) { mul2(v[i], v[i + 1], u[i], u[i + 1], rs, rs); });
                }
                if (pad) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = 0.f;
                }
                if (hd < heads) store_as(XT, s.out, o0 + hd * D, gr.a, gr.b, v);
            }
            slot = slot + 1 == DEPTH ? 0 : slot + 1;
            p.step(per);
        }
    }
    if constexpr (NORM) {
        __syncthreads();                                   // the rings are free
        float(*red)[2][D] = reinterpret_cast<float(*)[2][D]>(smem);
        const int warp = threadIdx.x >> 5;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) {
                sum[0][i] += __shfl_xor_sync(0xffffffffu, sum[0][i], o);
                sum[1][i] += __shfl_xor_sync(0xffffffffu, sum[1][i], o);
            }
            if (lane < LPR) {
                const int at = i < 4 ? gr.a + i : gr.b + i - 4;
                red[warp][0][at] = sum[0][i];
                red[warp][1][at] = sum[1][i];
            }
        }
        __syncthreads();
        if (threadIdx.x < 2 * D) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) s += red[w][threadIdx.x / D][threadIdx.x % D];
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

static bool row_type(int t) { return t == SKV_F32 || t == SKV_F16 || t == SKV_BF16; }
static bool misaligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

static int check(skv_handle *h, const skv_rope_spec *s, int64_t n, int32_t H, int32_t Hk, int32_t x_type, const int32_t *pos)
{
    if (!s) return fail(h, SKV_EINVAL, "spec is NULL");
    if (s->D != 64 && s->D != 128) return fail(h, SKV_EUNSUPPORTED, "head dim %d (supported: 64, 128)", s->D);
    if (s->rot_dims < 0 || s->rot_dims > s->D || s->rot_dims % 2)
        return fail(h, SKV_EINVAL, "rot_dims %d: even and at most D is wanted", s->rot_dims);
    if (!s->interleaved && s->rot_dims % 8)
        return fail(h, SKV_EUNSUPPORTED, "rot_dims %d: a multiple of 8 is wanted for split halves", s->rot_dims);
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
    if (misaligned(p, 16) || (n > 1 && stride * elem(type) % 16))
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
    d->vec8 = c->row_bytes % 8 == 0 && !misaligned(d->d0, 8) && !misaligned(d->d1, 8);
    return SKV_OK;
}

static Args base_args(skv_handle *h, const skv_rope_spec *s, int64_t n, int H, int Hk, int Hv, const int32_t *pos, int bytes)
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
    // rows of a batch, as the kernels have them
    const int rb = 256 / s->D * iter_of(bytes);
    a.bq = (H + rb - 1) / rb;
    a.bk = (Hk + rb - 1) / rb;
    a.bv = (Hv + rb - 1) / rb;
    a.batches = n * (a.bq + a.bk + a.bv);                  // below 2^47; a warp's share below 2^31 (2^36 / resident warps: memory ends before)
    return a;
}
// CTAs for the line of batches: as many as are resident, or a warp for each batch.
static unsigned grid_of(skv_handle *h, const Args &a, int ctas)
{
    const int64_t most = static_cast<int64_t>(ctas) * h->sm_count, need = (a.batches + kThreads / 32 - 1) / (kThreads / 32);
    return static_cast<unsigned>(need < most ? need : most);
}

template <int XT, int D, bool CACHE, bool INTER>
static cudaError_t launch_t(const Args &a, unsigned grid, cudaStream_t st)
{
    rope_kernel<XT, D, CACHE, INTER><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <int XT, bool CACHE>
static cudaError_t launch_x(const Args &a, int D, unsigned grid, cudaStream_t st)
{
    if (D == 64) return a.inter ? launch_t<XT, 64, CACHE, true>(a, grid, st) : launch_t<XT, 64, CACHE, false>(a, grid, st);
    return a.inter ? launch_t<XT, 128, CACHE, true>(a, grid, st) : launch_t<XT, 128, CACHE, false>(a, grid, st);
}
template <bool CACHE>
static int launch(skv_handle *h, const Args &a, int x_type, int D, cudaStream_t st)
{
    const unsigned grid = grid_of(h, a, kCtas);
    cudaError_t e;
    if (x_type == SKV_F32) e = launch_x<SKV_F32, CACHE>(a, D, grid, st);
    else if (x_type == SKV_F16) e = launch_x<SKV_F16, CACHE>(a, D, grid, st);
    else e = launch_x<SKV_BF16, CACHE>(a, D, grid, st);
    return cuda_fail(h, e, "rope launch");
}

template <int GT, int XT, int D, bool NORM, bool INTER>
static cudaError_t launch_back_t(const Args &a, unsigned grid, cudaStream_t st)
{
    static KernelAttrCache attr;
    constexpr int smem = kThreads / 32 * kRing;
    const cudaError_t e = kernel_smem_optin(attr, reinterpret_cast<const void *>(rope_back_kernel<GT, XT, D, NORM, INTER>), smem, kThreads, nullptr);
    if (e == cudaSuccess) rope_back_kernel<GT, XT, D, NORM, INTER><<<grid, kThreads, smem, st>>>(a);
    return e;
}
template <int GT, int XT, int D>
static cudaError_t launch_back_d(const Args &a, bool norm, unsigned grid, cudaStream_t st)
{
    if (norm) return a.inter ? launch_back_t<GT, XT, D, true, true>(a, grid, st) : launch_back_t<GT, XT, D, true, false>(a, grid, st);
    return a.inter ? launch_back_t<GT, XT, D, false, true>(a, grid, st) : launch_back_t<GT, XT, D, false, false>(a, grid, st);
}
template <int GT>
static cudaError_t launch_back_g(const Args &a, int x_type, int D, bool norm, unsigned grid, cudaStream_t st)
{
    if (x_type == SKV_F32) return D == 64 ? launch_back_d<GT, SKV_F32, 64>(a, norm, grid, st) : launch_back_d<GT, SKV_F32, 128>(a, norm, grid, st);
    if (x_type == SKV_F16) return D == 64 ? launch_back_d<GT, SKV_F16, 64>(a, norm, grid, st) : launch_back_d<GT, SKV_F16, 128>(a, norm, grid, st);
    return D == 64 ? launch_back_d<GT, SKV_BF16, 64>(a, norm, grid, st) : launch_back_d<GT, SKV_BF16, 128>(a, norm, grid, st);
}
static int launch_back(skv_handle *h, const Args &a, int g_type, int x_type, int D, bool norm, unsigned grid, cudaStream_t st)
{
    cudaError_t e;
    if (g_type == SKV_F32) e = launch_back_g<SKV_F32>(a, x_type, D, norm, grid, st);
    else if (g_type == SKV_F16) e = launch_back_g<SKV_F16>(a, x_type, D, norm, grid, st);
    else e = launch_back_g<SKV_BF16>(a, x_type, D, norm, grid, st);
    if (e == cudaSuccess) e = cudaGetLastError();
    return cuda_fail(h, e, "rope gradient launch");
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
    if (rope::misaligned(q_weight, 16) || rope::misaligned(k_weight, 16))
        return fail(h, SKV_EUNSUPPORTED, "weights must be 16-byte aligned");
    if (n == 0 || H + Hk == 0) return SKV_OK;
    OnDevice on(h->device);
    rope::Args a = rope::base_args(h, spec, n, H, Hk, 0, pos, rope::elem(x_type));
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
    if (rope::misaligned(positions, 4) || rope::misaligned(q_weight, 16) || rope::misaligned(k_weight, 16))
        return fail(h, SKV_EUNSUPPORTED, "positions must be 4-byte and weights 16-byte aligned");
    OnDevice on(h->device);
    rope::Args a = rope::base_args(h, spec, n, H, Hk, Hk, pos, rope::elem(x_type));
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
    if (rope::misaligned(q_weight, 16) || rope::misaligned(k_weight, 16) || rope::misaligned(dq_weight, 4) ||
        rope::misaligned(dk_weight, 4))
        return fail(h, SKV_EUNSUPPORTED, "weights must be 16-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    OnDevice on(h->device);
    rope::Args a = rope::base_args(h, spec, n, H, Hk, 0, pos, rope::elem(g_type) + (norm ? rope::elem(x_type) : 0));
    a.q = rope::Side{q, q_stride, q_weight, dq, dq_stride, dq_out};
    a.k = rope::Side{k, k_stride, k_weight, dk, dk_stride, dk_out};
    const unsigned grid = rope::grid_of(h, a, rope::kCtas);
    if (norm && grid) {
        if ((rc = ensure_workspace(h, static_cast<size_t>(grid) * 2 * D * sizeof(float), st))) return rc;
        a.dw = static_cast<float *>(h->workspace);
    }
    if (grid && (rc = rope::launch_back(h, a, g_type, x_type, D, norm, grid, st))) return rc;
    if (norm) {
        rope::rope_weight_kernel<<<2 * D / 32, 1024, 0, st>>>(a.dw, static_cast<int>(grid), D, dq_weight, dk_weight);
        rc = cuda_fail(h, cudaGetLastError(), "rope weight launch");
    }
    return rc;
}
