// kv_encode.cuh -- the stored form of eight consecutive values of a cache row
// (the rule and its proof stand at the top of append.cu); used by the kernels
// that write rows.
#pragma once

#include "ptx.cuh"

namespace skv {

// fp16(fl(amax / qmax)) without a division unless the product could round
// to another fp16 value (see the header).
__device__ __forceinline__ __half block_scale(float amax, float qmax, float inv_qmax)
{
    const float s0 = __fmul_rn(amax, inv_qmax);
    const __half h = __float2half_rn(s0);
    const __half lo = __float2half_rn(__fmul_rn(s0, 1.f - 0x1p-20f));
    const __half hi = __float2half_rn(__fmul_rn(s0, 1.f + 0x1p-20f));
    if (__half_as_ushort(lo) == __half_as_ushort(h) && __half_as_ushort(hi) == __half_as_ushort(h)) return h;
    return __float2half_rn(__fdiv_rn(amax, qmax));
}

// 1/d to within 2^-22 (relative), one instruction; d is a normal fp32 value.
__device__ __forceinline__ float rcp_approx(float d)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}

// Bytes 0 of four words, in order, as one word.
__device__ __forceinline__ uint32_t low_bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Codes of eight values of a 32-value block held by four neighbouring lanes (lane
// l & 3 has values 8 (l & 3) ..): the block's scale, and the lane's code bytes in
// w0, w1 (q4_0: valid in the block's lanes 0 and 1, their bytes 8 (l & 3) ..).  All
// lanes of the warp take part.
template <int T>
__device__ __forceinline__ void encode8(const float (&v)[8], __half &d16, uint32_t &w0, uint32_t &w1)
{
    constexpr float QMAX = T == SKV_Q8_0 ? 127.f : 7.f;
    constexpr float INV_QMAX = 1.f / QMAX;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    d16 = block_scale(amax, QMAX, INV_QMAX);
    const float d = __half2float(d16);
    const float rd = d > 0.f ? rcp_approx(d) : 0.f;           // d = 0: every code 0
    int q[8];
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t0 = __fmul_rn(v[i], rd);
        const float r0 = rintf(t0);
        off = fmaxf(off, fabsf(t0 - r0));
        q[i] = static_cast<int>(r0);
    }
    if (off >= 0.5f - 0x1p-13f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __float2int_rn(__fdiv_rn(v[i], d));
    }
    if (d < 0x1p-14f) {
        constexpr int QLO = T == SKV_Q8_0 ? -127 : -8, QHI = T == SKV_Q8_0 ? 127 : 7;   // codes -127..127, 0..15
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = max(QLO, min(QHI, q[i]));
    }
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = static_cast<uint32_t>(T == SKV_Q8_0 ? q[i] : q[i] + 8);
    w0 = low_bytes4(c[0], c[1], c[2], c[3]);
    w1 = low_bytes4(c[4], c[5], c[6], c[7]);
    if (T == SKV_Q4_0) {
        // byte j holds value j (low nibble) and value j + 16 (high nibble):
        // the lane two further on holds values j0 + 16 ..
        const uint32_t h0 = __shfl_down_sync(0xffffffffu, w0, 2), h1 = __shfl_down_sync(0xffffffffu, w1, 2);
        w0 |= h0 << 4;
        w1 |= h1 << 4;
    }
}

// Store a lane's part of a block (lane l & 3 of its four); the block is 2-byte aligned.
template <int T>
__device__ __forceinline__ void store8(uint8_t *blk, int l, __half d16, uint32_t w0, uint32_t w1)
{
    const int j0 = (l & 3) * 8;
    if (T == SKV_Q8_0 || j0 < 16) {
        uint16_t *dst = reinterpret_cast<uint16_t *>(blk + 2 + j0);
        dst[0] = static_cast<uint16_t>(w0);
        dst[1] = static_cast<uint16_t>(w0 >> 16);
        dst[2] = static_cast<uint16_t>(w1);
        dst[3] = static_cast<uint16_t>(w1 >> 16);
    }
    if (j0 == 0) *reinterpret_cast<__half *>(blk) = d16;
}

}  // namespace skv
