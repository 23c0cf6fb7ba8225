// bwd.cuh -- gradients of attention: what the kernels of the call share.
//
// With p = exp(scale q.k - lse), delta = d_o.o - d_lse and ds = p (d_o.v - delta),
//   dv = sum_q p d_o,  dk = scale sum_q ds q,  dq = scale sum_k ds k.
//
// Two launches: prepare (row statistics; gathered rows of lists), and one of CTAs for
// dk and dv (each owns 128 keys of a KV head and walks over the query tiles that see one of
// them) and of CTAs for dq (each owns a query tile and walks over its keys).  S and d_o.v are
// computed in both: 7 products instead of 5, but no sum of dq crosses CTAs.
// Adding it up in memory instead would move 4 bytes for every key tile, query row and
// channel: 64 KB for each 128 x 128 tile.  A tile of dk and dv takes 1.64 us for its four products; at that
// rate five take about 2 us, and 152 SMs then add up 4.9 TB/s, half of that if two CTAs shared a
// tile of dq.  Not built or timed: whether it would be faster than 7 products is open.  Its sums
// would change from run to run unless CTAs took turns on a tile.
//
// A query tile is Tb tokens x Gb heads of a KV head's group, Tb * Gb <= 128 rows
// (row = token * Gb + head), chosen for the fewest tiles.
//
// Powers of two.  The products take fp16 operands, and p and ds reach far below
// fp16's range over long rows.  So
//   p'  = 2^15 p                       (normal down to p = 2^-29, subnormal to 2^-39),
//   ds' = p' (d_o.v - delta) 2^-e      with 2^e at least the largest |d_o.v - delta|,
// by |d_o.v| <= |d_o| |v| and the exponents of the rows' 2-norms: the query row's own e
// for dq, the largest of the rows that a key tile meets for dk.  An fp32 d_o is
// rounded to fp16 after a division by 2^c of its row (d_o' = d_o 2^-c); c then goes
// into p' for dv: p' = 2^(15 + c - cmax) p.
//
// Two parts.  Small calls hold p' and ds' as high + low, each fp16: high stands in the first half of the columns that the
// fp32 numbers had in tensor memory, low in the other half, and its product follows high's.
#pragma once

#include "internal.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace skv {
namespace bwd {

constexpr int kTile = 128;               // rows of a query tile, keys of a key tile
// Threads of the gradient kernels: sixteen compute warps and four others (96 registers).  A thread's
// chain of tensor-memory loads, exponentials and stores is mostly latency: four warps for each
// quarter of an SM where two left it idle.
constexpr int kThreads = 640, kCompute = 512;
constexpr int kParts = kCompute / 128;   // compute threads that share a lane of tensor memory: columns of a tile in as many parts
constexpr int kCols = kTile / kParts;    // columns of a thread
constexpr int kLow = kCols / 2;          // where the low parts stand among a part's columns of tensor memory
enum { kOnePart, kTwoOfDq, kTwoParts };  // how p and ds enter their products
constexpr int kPShift = 15;              // p' = 2^15 p
// Tiles after which an accumulator is added to fp32 memory.  The tensor core cuts its
// sums off instead of rounding them, and loses about 2^-24 of a sum's size for
// each of its steps of 16: 6e-5 over the 1024 steps of 128 tiles, where all
// addends have one sign.
constexpr int kStretch = 128;
constexpr int kInfoRows = 5;             // L, delta', c, lim; exponents
constexpr int kInfoBytes = 4 * kTile * 4;   // the four that the dk/dv kernel's stages hold
constexpr int kMaxQTiles = 32768;        // query tiles of a KV head (a bitmap in shared memory)
constexpr int kNoExp = -200;             // exponent of zero
constexpr int kAbsent = -128;            // a key that is not there (padding of a list)

struct Geo {
    int groups;                          // sequences of row lists, or 1: all share the keys
    int64_t T;                           // tokens of a group
    int Hk, G, H, D;
    int Gb, Tb, TT, GG, QT;              // query tiles: heads x tokens; tiles along tokens and heads, of a KV head
    int64_t n;                           // keys
    int KT;                              // key tiles
};

// What a query tile's rows have in common; exponents are of true values (2^c put back).
struct __align__(16) TileSum {
    int lim_max;                         // keys that the row that sees most sees
    int eN, eD, c;                       // largest exponents of |d_o|, |delta|, and c
};

struct PrepArgs {
    Geo g;
    const void *d_o;                     // fp16 or fp32 [S][nq][H][D]
    const float *o, *lse, *d_lse;
    const int32_t *q_pos;
    int64_t pos0;                        // position of local key 0
    __half *doh;                         // fp32 d_o: its fp16 form
    float *info;                         // [tile][kInfoRows][128]
    TileSum *sum;                        // [tile]
    // keys
    const uint8_t *k, *v;                // row of local key 0, or of row 0 (lists)
    int64_t k_row_bytes, v_row_bytes;
    const int32_t *rows;                 // lists, entry of local key 0
    int64_t rows_ld;
    int rows_per_head;
    __half *kg, *vg;                     // lists: gathered rows [group][n][Hk][D]
    int8_t *ew;                          // [group][Hk][KT * 128] exponents of |v|
};

struct MainArgs {
    Geo g;
    float scale;
    float *info;
    const TileSum *sum;
    const int8_t *ew;
    int pieces;
    float *slot;                         // fp32 sums [piece][...] or null
    int g_type;
    void *out0, *out1;                   // dk, dv or dq
    int *status;
};

// Limit of the waits for what is in flight when a CTA gives up.
constexpr uint64_t kDrainNs = 100000000ull;

// Wait for a phase of an mbarrier: gives up after two seconds, or when another wait of
// the kernel has (bit 0 of the status word; other bits say other things).
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, const int *status)
{
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if ((i & 255u) == 0) {
            if (*reinterpret_cast<const volatile int *>(status) & 1) return false;
            const uint64_t t = tc::globaltimer_ns();
            if (i == 0) t0 = t;
            else if (t - t0 > 2000000000ull) return false;
        }
    }
}

// Smallest e with x <= 2^e for x = sqrt(n2) and for x >= 0.
__device__ __forceinline__ int exp_of_norm2(float n2)
{
    if (!(n2 > 0.f)) return kNoExp;
    const int x = static_cast<int>(__float_as_uint(n2) >> 23) - 127;      // n2 < 2^(x + 1); inf: 128
    return (x + 2) >> 1;
}
__device__ __forceinline__ int exp_of(float x)
{
    if (!(x > 0.f)) return kNoExp;
    return static_cast<int>(__float_as_uint(x) >> 23) - 126;
}
__device__ __forceinline__ float pow2(int e)                                // |e| <= 126
{
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// x * f * 2^e without leaving the range on the way.
struct Pow2 {
    float a, b;
    __device__ __forceinline__ Pow2(float f, int e)
    {
        e = max(-250, min(250, e));
        a = f * pow2(e / 2);
        b = pow2(e - e / 2);
    }
    __device__ __forceinline__ float operator()(float x) const { return x * a * b; }
};

// Query tile `tile` of all -> its group, KV head and place.
struct QTile {
    int group, hk, g0;
    int64_t t0;
};
__device__ __forceinline__ QTile q_tile(const Geo &g, int group, int hk, int qt)
{
    QTile t;
    t.group = group;
    t.hk = hk;
    const int gi = qt / g.TT;
    t.g0 = gi * g.Gb;
    t.t0 = static_cast<int64_t>(qt - gi * g.TT) * g.Tb;
    return t;
}
// Row r of a tile -> [S*nq*H] row, or -1.
__device__ __forceinline__ int64_t q_row(const Geo &g, const QTile &t, int r)
{
    const int tt = r / g.Gb, gg = t.g0 + r - tt * g.Gb;
    const int64_t tok = t.t0 + tt;
    if (tt >= g.Tb || gg >= g.G || tok >= g.T) return -1;
    return (t.group * g.T + tok) * g.H + static_cast<int64_t>(t.hk) * g.G + gg;
}

// What two numbers in fp16 leave of them, in fp16.
__device__ __forceinline__ uint32_t low_part(uint32_t high, float a, float b)
{
    const __half2 h2 = *reinterpret_cast<const __half2 *>(&high);
    return pack_half2(-sub_h(__low2half(h2), a), -sub_h(__high2half(h2), b));
}

// Part of a row of results: NC values at `at`, as g_type.
template <int NC>
__device__ __forceinline__ void store_row(void *base, int64_t at, int g_type, const float (&v)[NC])
{
    if (g_type == SKV_F16) {
        __half *p = static_cast<__half *>(base) + at;
#pragma unroll
        for (int i = 0; i < NC; i += 8)
            *reinterpret_cast<uint4 *>(p + i) = make_uint4(pack_half2(v[i], v[i + 1]), pack_half2(v[i + 2], v[i + 3]),
                                                           pack_half2(v[i + 4], v[i + 5]), pack_half2(v[i + 6], v[i + 7]));
    } else {
        float *p = static_cast<float *>(base) + at;
#pragma unroll
        for (int i = 0; i < NC; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}
// Add what this thread left there before.
template <int NC>
__device__ __forceinline__ void add_row(const float *p, float (&v)[NC])
{
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p + i);
        v[i] += x.x;
        v[i + 1] += x.y;
        v[i + 2] += x.z;
        v[i + 3] += x.w;
    }
}

// NC (32 or 16) columns of this thread's lane.
template <int NC>
__device__ __forceinline__ void load_cols(uint32_t taddr, float (&v)[NC])
{
    static_assert(NC == 32 || NC == 16, "columns of a thread");
    uint32_t r[NC];
    if constexpr (NC == 32) {
        tc::tmem_ld32(taddr, r);
        tc::tmem_wait_ld(r);
    } else {
        tc::tmem_ld16(taddr, r);
        tc::tmem_wait_ld16(r);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) v[i] = __uint_as_float(r[i]);
}

int launch_prep(skv_handle *h, const PrepArgs &a, int do_type, cudaStream_t st);
int launch_join(skv_handle *h, const float *slot, int pieces, int64_t n, int outs, int g_type, void *out0, void *out1,
                cudaStream_t st);
// One launch of both: kv_args.out0 or q_args.out0 NULL leaves a part out.
int launch_main(skv_handle *h, const CUtensorMap &mq, const CUtensorMap &mo, const CUtensorMap &mk, const CUtensorMap &mv,
                const MainArgs &kv_args, const MainArgs &q_args, bool q_first, int parts, cudaStream_t st);

}  // namespace bwd
}  // namespace skv
