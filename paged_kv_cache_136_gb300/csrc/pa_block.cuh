// pa_block.cuh -- what the block-scaled 8-bit cache, the key bounds and the
// block-sparse decode share: power-of-two scales, e4m3 conversions and the
// small matrix instructions of the kernels that hold their tiles in registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace block {

// Scales are 2^e with e in [-kExpRange, kExpRange].  A power of two multiplies
// exactly, so codes can move to a larger scale without a second rounding
// (except into e4m3's subnormals) and a sum of integer codes times scales has
// one value whatever its order.  The range leaves every product of two scales
// and a code sum (below 2^21) an exact fp32 number once 2^-16 is taken out.
constexpr int kExpRange = 60;

__device__ __forceinline__ float two_to(int e) // -126 <= e <= 127
{
    return __int_as_float((e + 127) << 23);
}

// Smallest 2^e with amax <= top * 2^e, e held to the range; amax >= 0 finite.
// TOP is 448 (e4m3) or 127 (int8): 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6, so
// the exponents are compared and then the mantissas.
template <int TOP> __device__ __forceinline__ float pow2_scale(float amax)
{
    static_assert(TOP == 448 || TOP == 127, "448 or 127");
    constexpr int top_exp = TOP == 448 ? 8 : 6;
    constexpr uint32_t top_mant = TOP == 448 ? 0x600000u : 0x7E0000u;
    const uint32_t b = __float_as_uint(amax);
    int e = (int)(b >> 23) - 127 - top_exp + ((b & 0x7FFFFFu) > top_mant ? 1 : 0);
    e = max(-kExpRange, min(kExpRange, e)); // zero and subnormals: the smallest
    return two_to(e);
}

// 1 / s of a power of two s = 2^e with |e| <= 126.
__device__ __forceinline__ float pow2_inverse(float s)
{
    return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// Two floats to two e4m3 codes (a in the low byte), nearest even, magnitudes
// above 448 (infinities too) to 448, NaN to NaN.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Two e4m3 codes (low 16 bits) to two halves, exactly.
__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint32_t codes)
{
    uint32_t r;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo; }"
        : "=r"(r)
        : "r"(codes));
    return r;
}

// The same of the high 16 bits.
__device__ __forceinline__ uint32_t half2_of_e4m3x2_hi(uint32_t codes)
{
    uint32_t r;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi; }"
        : "=r"(r)
        : "r"(codes));
    return r;
}

template <typename T> __device__ __forceinline__ float2 float2_of(uint32_t v);
template <> __device__ __forceinline__ float2 float2_of<__half>(uint32_t v)
{
    return __half22float2(*reinterpret_cast<__half2 *>(&v));
}
template <> __device__ __forceinline__ float2 float2_of<__nv_bfloat16>(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

// Two floats to a pair of T, nearest even, a in the low half.
template <typename T> __device__ __forceinline__ uint32_t pair_of(float a, float b);
template <> __device__ __forceinline__ uint32_t pair_of<__half>(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t pair_of<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// c += a * b on one warp: a 16 x 16, b 16 x 8, c 16 x 8 in fp32.  Lane 4g + t
// holds a of rows g and g + 8, columns 2t, 2t+1 and 2t+8, 2t+9; b of column g,
// rows 2t, 2t+1 and 2t+8, 2t+9; c of rows g and g + 8, columns 2t, 2t+1.
template <typename T>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1,
                                                  uint32_t a2, uint32_t a3, uint32_t b0,
                                                  uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1,
                                                         uint32_t a2, uint32_t a3, uint32_t b0,
                                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit values, one row pair a lane.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// kv heads that a CTA of up to eight warps takes side by side: the most, up to
// 8, that divide them, so that what lies together is read together.
inline int heads_together(int num_kv_heads)
{
    int h = 8;
    while (num_kv_heads % h)
        --h;
    return h;
}

// 16- and 8-byte loads that do not stay in L1.
__device__ __forceinline__ uint4 load16(const void *p)
{
    uint4 v;
    asm("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint2 load8(const void *p)
{
    uint2 v;
    asm("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "l"(p));
    return v;
}

// The tokens of request r that a call adds, checked: positions
// [len - fresh, len), rows [row, row + fresh) of the packed new tokens.
struct Request {
    int len, fresh, row;
};

// False for a request without new tokens, and for one whose metadata is out
// of range, which is flagged.
__device__ __forceinline__ bool read_request(Request &q, int r, const int32_t *seq_lens,
                                             const int32_t *query_start_loc, int num_tokens,
                                             int max_query_len, int len_cap, bool report,
                                             unsigned int *err)
{
    const int a = query_start_loc[r], b = query_start_loc[r + 1];
    q.len = seq_lens[r];
    q.row = a;
    q.fresh = b - a;
    if (a < 0 || b < a || b > num_tokens || q.fresh > max_query_len || q.len < q.fresh ||
        q.len > len_cap) {
        if (report)
            atomicOr(err, PA_DEVERR_SEQ_LEN_);
        return false;
    }
    return q.fresh > 0;
}

} // namespace block
} // namespace pa
