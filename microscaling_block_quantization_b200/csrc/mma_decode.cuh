// Pieces shared by the decode-time kernels (few activation rows against
// block-scaled codes): 4-bit code words to f16 pairs, block scales to
// binary32, the m16n8 matrix instructions and 16-byte asynchronous copies.
//
// Every element grid here is exact in f16, so the matrix instruction forms
// exact products q x of a code value and an f16 activation piece and sums
// them in binary32; the block scale multiplies that sum.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

#include "mx_device.cuh"

namespace mxk {

// element kinds of a packed 4-bit word
enum { GE_E2M1 = 0, GE_E3M0 = 1, GE_INT4 = 2, GE_UINT4 = 3 };

__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hadd2_u(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight codes of a word -> four f16x2 of their grid values, codes (2i, 2i+1)
// in h[i].  E2M1: the conversion instruction.  INT4 (integers under an f16
// exponent, Kim, Henry, Fahim and Hassan Awadalla, "Who Says Elephants Can't Run",
// 2022): a byte's nibbles spread
// to the two halves (multiply by 2^12 + 1, mask) under the exponent of 1024,
// where an f16 ulp is 1, then 1024 (+ 8 for two's complement, whose sign bit
// is flipped first) taken off: exact.  E3M0: the 3-bit magnitude is an f16
// exponent field (0 -> 0), times 2^12.
template <int ELEM>
__device__ __forceinline__ void codes8_halves(uint32_t w, uint32_t h[4])
{
    if (ELEM == GE_E2M1) {
        e2m1x8_halves(w, h);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = __byte_perm(w, 0u, 0x4440u + i);
        if (ELEM == GE_E3M0) {
            const uint32_t mag = (b * 0x00400400u) & 0x1c001c00u;   // b << 10 | b << 22
            const uint32_t sgn = (b * 0x01001000u) & 0x80008000u;   // b << 12 | b << 24
            h[i] = hmul2_u(mag | sgn, 0x6c006c00u);                 // 2^12
        } else if (ELEM == GE_INT4) {
            h[i] = hadd2_u(((b * 0x1001u) & 0x000f000fu) ^ 0x64086408u, 0xe408e408u);
        } else {
            h[i] = hadd2_u(((b * 0x1001u) & 0x000f000fu) ^ 0x64006400u, 0xe400e400u);
        }
    }
}

// Eight INT4 codes of a word -> four f16x2 with codes (i, i + 4) in h[i]: the
// nibbles of a half word where they stand, under the exponent of 1024 (an f16
// ulp is 1: 1024 + n, or 1024 + 16 n four bits up), then the constant off:
// half the integer operations of neighbouring pairs.
template <int ELEM>
__device__ __forceinline__ void int4_halves_spread(uint32_t w, uint32_t h[4])
{
    constexpr uint32_t F = ELEM == GE_INT4 ? 0x8u : 0x0u;   // two's complement: flip the sign bit, take 8 off
    const uint32_t lo = 0x64006400u | F | (F << 16), hi = 0x64006400u | (F << 4) | (F << 20);
    const uint32_t off = ELEM == GE_INT4 ? 0xe408e408u : 0xe400e400u;       // -(1024 + 8), -1024
    const uint32_t off16 = ELEM == GE_INT4 ? 0xd480d480u : 0xd400d400u;     // -(64 + 8), -64
    const uint32_t v = w >> 8;
    h[0] = hadd2_u((w & 0x000f000fu) ^ lo, off);
    h[2] = hadd2_u((v & 0x000f000fu) ^ lo, off);
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[1]) : "r"((w & 0x00f000f0u) ^ hi), "r"(0x2c002c00u), "r"(off16));   // / 16
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[3]) : "r"((v & 0x00f000f0u) ^ hi), "r"(0x2c002c00u), "r"(off16));
}

// A block-scale code -> binary32.  Unsigned minifloats with 3 mantissa bits:
// the byte shifted into an exponent and mantissa, rescaled by an exact power
// of two.
__device__ __forceinline__ float scale1(int fmt, uint32_t b)
{
    if (fmt == S_E8M0) return b == 0xffu ? bits2f(0x7fc00000u) : b ? bits2f(b << 23) : bits2f(0x00400000u);
    const float up = fmt == S_UE4M3 ? 0x1p120f : 0x1p112f;
    const uint32_t nan_code = fmt == S_UE4M3 ? 0x7fu : 0xffu;
    return b >= nan_code ? bits2f(0x7fc00000u) : __fmul_rn(bits2f(b << 20), up);
}

// Four codes of a word.
__device__ __forceinline__ void scales4(int fmt, uint32_t w, float s[4])
{
    if (fmt == S_E8M0) {
        // 2^(code - 127), 0xFF -> NaN, code 0 -> 2^-127: exact in bf16
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\t"
            "cvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
        s[0] = bits2f(lo << 16);
        s[1] = bits2f(lo & 0xffff0000u);
        s[2] = bits2f(hi << 16);
        s[3] = bits2f(hi & 0xffff0000u);
        return;
    }
    if (fmt == S_UE4M3) {
        // the E4M3 conversion (0x7F is its NaN); bytes from 0x80 on, which no
        // finite scale has, are NaN too
        const uint32_t top = w & 0x80808080u;
        if (top) w |= (top >> 7) * 0x7fu;
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        s[0] = a.x; s[1] = a.y; s[2] = b.x; s[3] = b.y;
        return;
    }
    // UE5M3: the byte shifted into a binary32 exponent and mantissa
    // (subnormal codes become binary32 subnormals), rescaled exactly
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = scale1(fmt, (w >> (8 * i)) & 0xffu);
}

// Four codes of a word, each times a power of two m[i] (a bf16): the E8M0
// codes' bf16 values enter a mixed-precision multiply-add (exact), which
// widens and scales at once on the FMA pipe.
__device__ __forceinline__ float bf16_mul_f32(uint32_t pair, int high, float m)
{
    float r;
    const uint32_t mb = __float_as_uint(m) >> 16;
    if (high)
        asm("{\n\t.reg .b16 a, b, c;\n\tmov.b32 {a, b}, %1;\n\tcvt.u16.u32 c, %2;\n\tfma.rn.f32.bf16 %0, b, c, 0f80000000;\n\t}"
            : "=f"(r) : "r"(pair), "r"(mb));
    else
        asm("{\n\t.reg .b16 a, b, c;\n\tmov.b32 {a, b}, %1;\n\tcvt.u16.u32 c, %2;\n\tfma.rn.f32.bf16 %0, a, c, 0f80000000;\n\t}"
            : "=f"(r) : "r"(pair), "r"(mb));
    return r;
}
__device__ __forceinline__ void scales4_times(int fmt, uint32_t w, const float m[4], float s[4])
{
    if (fmt == S_E8M0) {
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\t"
            "cvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
        s[0] = bf16_mul_f32(lo, 0, m[0]);
        s[1] = bf16_mul_f32(lo, 1, m[1]);
        s[2] = bf16_mul_f32(hi, 0, m[2]);
        s[3] = bf16_mul_f32(hi, 1, m[3]);
        return;
    }
    scales4(fmt, w, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = __fmul_rn(s[i], m[i]);
}

// D (16 x 8, binary32) += A (16 x 16, f16) B (16 x 8, f16); lane = 4 g + t
// holds A rows g, g + 8 at k = 2t, 2t + 1 (a0, a1) and 2t + 8, 2t + 9 (a2,
// a3), B column g at the same k, D rows g, g + 8 at columns 2t, 2t + 1.
__device__ __forceinline__ void mma_16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same from zero
__device__ __forceinline__ void mma_16816_zero(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// 8 values of k, from zero
__device__ __forceinline__ void mma_1688_zero(float d[4], uint32_t a0, uint32_t a1, uint32_t b0)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a0), "r"(a1), "r"(b0), "f"(0.0f));
}

// D (16 x 8, binary32) += A (16 x 8, TF32) B (8 x 8, TF32): A rows g, g + 8 at
// k = t (a0, a1) and t + 4 (a2, a3), B column g at the same k.
__device__ __forceinline__ void mma_1688_tf32(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// binary32 rounded to TF32 (11 significant bits), and one half of an f16 pair as TF32 (exact)
__device__ __forceinline__ uint32_t tf32_of(float x)
{
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t tf32_of_half(uint32_t pair, int high)
{
    const __half2 h = *reinterpret_cast<const __half2 *>(&pair);
    return __float_as_uint(high ? __high2float(h) : __low2float(h));
}

// asynchronous global -> shared copies; bytes beyond src_bytes are zero
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int src_bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int src_bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a)
{
    uint16_t r;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}

// exponent of the power of two that brings amax into [2^14, 2^15) (f16
// without overflow after rounding): 14 - floor(log2 amax).  An infinite or
// NaN amax gives 2^-114: the finite values beside it no longer matter to the
// sums it enters.  Below 2^-100 the scale stays at 2^114.
__device__ __forceinline__ int f16_scale_exponent(float amax)
{
    const int e = (int)(__float_as_uint(amax) >> 23) - 127;
    return 14 - max(e, -100);
}

}  // namespace mxk
