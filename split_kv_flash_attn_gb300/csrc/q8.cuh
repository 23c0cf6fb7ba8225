// q8.cuh -- what the kernels over 8-bit pages share: argument blocks, the
// look-up of a page through a list, and the exact conversion of int8 codes to
// fp16.
#pragma once

#include "internal.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace skv {
namespace q8 {

constexpr int kPage = SKV_Q8_PAGE;
constexpr int kStatusAppend = 2;   // a token had no page to go to
constexpr int kStatusList = 4;     // a page id outside the pool, or a length beyond its list

// The lists of a call.
struct Lists {
    const int32_t *ids;            // [S][Hk][cap]
    const int32_t *kv_len;         // [S]
    int64_t cap;
    int64_t n_pages;               // pages of the pool
    int S, Hk;
    int *status;
};

struct AttnArgs {
    Lists L;
    const int8_t *k, *v;           // pages [n_pages][64][D]
    const float *k_scale, *v_scale;
    const __half *q;               // [S][nq][H][D]
    const int32_t *q_pos;          // [S][nq] or null
    const int32_t *sel;            // [S][nq][Hk][n_sel] or null
    int n_sel;
    int nq, H, G;                  // nq: tokens of this launch
    int nq_ld, tok0;               // tokens a sequence in q, q_pos, sel, o and lse; the first of this launch
    int rows;                      // query rows of one unit: nq * G, or G with sel
    int row_groups;                // units per (list, KV head)
    float scale_log2;              // scale * log2(e)
    void *o;                       // [S][nq][H][D]
    float *lse;                    // [S][nq][H]
    // scratch
    float *part_o;                 // [2 * grid][columns][D] partials
    float *part_ml;                // [2 * grid][columns][2] reference (log2) and sum (prefill: one log sum)
    int *counters;                 // arrivals, zero between launches
    float *page_lse;               // mass: [S][Hk][nq * G][page_ld] log2 sums of half pages, or null
    int64_t page_ld;               // 2 cap, or 2 n_sel with sel

    // Index of token t of sequence s in q, q_pos, o and lse.
    __host__ __device__ int64_t token(int s, int t) const { return static_cast<int64_t>(s) * nq_ld + tok0 + t; }
};

// Programmatic dependent launch.  Every kernel over 8-bit pages is launched while
// the one before it on the stream ends; it reads and writes nothing of memory
// before start(), which waits for the whole of that kernel (and so, as each one
// waits, for all before it).  About 1 us a launch.  None lets its successor come
// any earlier: CTAs that wait on an SM keep those that work from spreading (62
// against 73 us for a selection with its attention).
__device__ __forceinline__ void start() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// Tokens of sequence s that its list can hold.
__device__ __forceinline__ int64_t list_len(const Lists &L, int s)
{
    const int64_t n = max(0, __ldg(L.kv_len + s));
    return min(n, L.cap * kPage);
}

// A page id that may be read, or -1.
__device__ __forceinline__ int checked_page(const Lists &L, int id)
{
    if (id >= L.n_pages) {
        atomicOr(L.status, kStatusList);
        return -1;
    }
    return id;
}

// Four int8 codes c to fp16, exactly: with the sign bit flipped a byte is u = c
// + 128, and 0x6400 | u is the fp16 number 1024 + u; less 1152 it is c.  `w`
// holds the codes with their sign bits flipped.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w)   // bytes 0, 1
{
    const uint32_t h = __byte_perm(w, 0x64646464u, 0x4140);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&h), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w)   // bytes 2, 3
{
    const uint32_t h = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&h), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// 16 bytes of a page, read once.
__device__ __forceinline__ uint4 ld_stream16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void *p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// The integer nearest x / d (ties to even), clamped to [-127, 127]; d > 0.  The
// fp32 quotient t is rounded correctly and half-integers are fp32 values, so t
// and x / d lie on the same side of every half-integer unless t is one: then
// the sign of x - t d (one rounding, so its sign is exact) decides.  x and d
// come scaled up together when d is tiny, which keeps that residual normal.
__device__ __forceinline__ int nearest_code(float x, float d)
{
    const float t = __fdiv_rn(x, d);
    float r = rintf(t);
    const float fl = floorf(t);
    if (t - fl == 0.5f) {
        const float rem = __fmaf_rn(-t, d, x);
        if (rem > 0.f) r = fl + 1.f;
        else if (rem < 0.f) r = fl;
    }
    if (!(r == r)) return 0;                        // NaN
    return static_cast<int>(fminf(fmaxf(r, -127.f), 127.f));
}

// Pages as a tensor [n_pages][64][D] of bytes, `rows` rows of a page a box, its
// 16-byte pieces swizzled (128 bytes a row for D = 128, 64 for D = 64).
int page_map(skv_handle *h, CUtensorMap *map, const int8_t *pages, int64_t n_pages, int D, int rows);
// Fewest pages of a CTA's piece in the decode kernel: with fewer, putting the
// pieces together costs more than it gains.
constexpr int kPieceMin = 4;
int launch_decode(skv_handle *h, const AttnArgs &a, int64_t n_pages, int D, bool out_f16, int grid, int nc,
                  cudaStream_t st);
// fp32(top / 127).  In 64 bits the product with 1/127 is within 2^-52 of the quotient,
// and no quotient of an fp32 number by 127 comes nearer than 2^-32 to a number on
// which fp32 rounding turns (127 m has a bit more than m, so none lies on one).
__device__ __forceinline__ float over_127(float top) { return __double2float_rn(static_cast<double>(top) * (1.0 / 127.0)); }

int launch_prefill(skv_handle *h, const AttnArgs &a, int D, bool out_f16, uint32_t *plan, int n_pairs, float *mass,
                   int grid, cudaStream_t st);
int launch_mass(skv_handle *h, const AttnArgs &a, float *mass, cudaStream_t st);
int launch_append(skv_handle *h, const skv_q8_pool &pool, const Lists &L, int n_max, int x_type, const void *k_new,
                  const void *v_new, const int32_t *n_new, cudaStream_t st);
struct SelectArgs {
    Lists L;
    const int8_t *k_min, *k_max;   // [n_pages][D]
    const float *k_scale;
    const __half *q;
    const int32_t *q_pos;
    int nq, H, G;                  // nq: tokens of this launch
    int nq_ld, tok0;               // as in AttnArgs
    int n_sel, n_first, n_last;
    uint32_t *keys;                // scratch [S][nq][Hk][cap]
    int *counters;                 // arrivals, zero between launches
    int32_t *sel;

    __host__ __device__ int64_t token(int s, int t) const { return static_cast<int64_t>(s) * nq_ld + tok0 + t; }
};
int launch_select(skv_handle *h, const SelectArgs &a, int D, cudaStream_t st);
int launch_evict(skv_handle *h, const Lists &L, const float *mass, int n_keep, int n_first, int n_last,
                 int32_t *ids_out, float *mass_out, int32_t *kv_len_out, int32_t *freed_out, cudaStream_t st);

}  // namespace q8
}  // namespace skv
