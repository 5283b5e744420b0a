// Attention of one query token per sequence over a paged block-scaled cache
// (mx_attn_decode).
//
//   o_h = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q_h . k_t - m_h),  t over the visible tokens;
//   k_t, v_t = q s_b (s_T) of the cache's codes.
//
// Bound: the visible rows' codes and scales read once for all query heads of
// a key head.  Per key element a group of G heads takes 2 G multiply-adds, so
// the products run on the matrix instruction, and the work per byte is the
// codes' conversion to f16.
//
// A warp takes a (sequence, key head, eight query heads, stretch of tokens)
// and walks it 16 tokens at a time, rows fetched through the page table by
// asynchronous copies into a private ring; warps do not wait for one another.
// Consecutive warps take consecutive key heads, whose rows are contiguous.
//
// * Scores: 16 tokens x 8 heads, codes as the 16-row operand, queries as f16
//   pieces scaled by a power of two per head (bf16: one piece exact down to
//   2^-31 of the head's largest; binary32: two, to 2^-23); each block's sum times
//   its scale in binary32.
// * One pass with a running maximum m (reference for the exponentials) and
//   sum l per head in binary32.  m moves only when a score exceeds it by 4
//   (in powers of two), so most tiles rescale nothing.
// * p v: tokens are the reduction dimension, but a decoded code pair holds
//   neighbours along the head.  The reduction index is (token, parity), the
//   eight columns (head, parity), and the weight of column (h, r) at (t, e) is
//   p_t(h) where e = r, else 0: code pairs enter the instruction as decoded,
//   nothing is transposed, and each m16 tile is one 32-block of the head, so
//   that the block's scale multiplies the weight: w = p s_b, in binary32 (E8M0
//   scales and bf16 results, VM = 2: in f16, by a power of two).
// * E4M3 scales with E2M1 codes (NVFP4; VM = 1) need no such folding: the
//   product of code and scale is an f16 exactly, so the codes are scaled as
//   they are decoded, on the FMA pipe, and w is p alone.
// * A tile's scale bytes are decoded once, a share a lane, and read back by all
//   as words (157 -> 138 us below, NVFP4 67 -> 58 us).
// * w as f16: scaled by 2^7 and, per 32-block, by a reference exponent of the
//   block scales that also moves rarely, so w stays in [0, 2^15] and is dropped
//   below 2^-25, which is p s_b below 2^-32 of the reference.  One f16 rounding
//   (2^-12 of the weight) for bf16 results; for binary32 a second piece holds
//   the rounding's remainder (2^-23).
// * A stretch in which a block's scale (but code 0) has been below 2^-6 of the
//   reference, or has moved it up, could lose its largest products that way: a
//   token of weight 1 and a value 2^-26 of another's.  From that tile on the
//   products p v are formed with w as TF32, the same 11 bits (binary32: two
//   pieces) with binary32's exponents, four m16n8k8 instructions for two, and
//   nothing is dropped, in a loop of its own: as a branch of the one loop it cost
//   every call 5% (64 x 8192 134 -> 140 us, this way 136; with every stretch wide
//   316 us).  So w is dropped only below 2^-24 of the largest weight times the
//   block's smallest scale (2^-26 but at the top of UE5M3).  VM = 1, whose weights
//   are p alone, drops p below 2^-35 of the largest.
// * Partial results (each stretch's own attention, m, l) of a sequence's
//   stretches meet in a fixed order: where a CTA's warps hold them all, in
//   shared memory at the end of the kernel, else in a second launch.
//
// Measured (32 query heads, 8 key heads of 128): 64 sequences of up to 8192
// tokens in MXFP4 134 us (3.2 TB/s), one of 131072 in NVFP4 56 us: the integer
// and conversion pipe is 57% and the issue slots 64% taken (378 instructions for
// 16 tokens of a key head), with four warps a scheduler to hide what each waits
// for.  One sequence of 1000 tokens 8.9 us: two launches, and 0.6 us for each
// 16 tokens of a warp.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mma_decode.cuh"
#include "mx_internal.h"

namespace mxk {

// element kinds: the 4-bit ones of GE_*, then one code per byte
enum { AE_E2M3 = 4, AE_E3M2 = 5 };

constexpr int kAtWarps = 4;   // of a CTA whose warps are not joined
// warps of an SM, and the most of a CTA: 128 or 168 registers a thread
template <int D, int BS, int NTH, int HP> __host__ __device__ constexpr int at_warps() { return HP || NTH == 2 || D == 256 || BS == 16 ? 12 : 16; }

template <int EL, int D, int BS> struct AtGeom {
    static constexpr int BITS = EL >= AE_E2M3 ? 8 : 4;
    static constexpr int NB = D / 32;                  // 32-blocks of a head
    static constexpr int ROW = D * BITS / 8;           // bytes of a head's codes
    static constexpr int NPC = ROW / 16;               // 16-byte pieces
    // bytes kept of a token's scales: all of them (blocks of 16), a word at least
    static constexpr int SW = BS == 16 ? D / 16 : (D / 32 < 4 ? 4 : D / 32);
    // scales that may be fewer bytes than a word: found in the aligned word
    // around them (BS 64 stands for blocks of 64 and 128)
    static constexpr bool NARROW = BS == 64 || (BS == 32 && D == 64);
    static constexpr int K_AT = 0, V_AT = 16 * ROW, KS_AT = 32 * ROW, VS_AT = KS_AT + 16 * SW, META_AT = VS_AT + 16 * SW;
    // a stage is a multiple of a row, so that a row's pieces are reached by an
    // exclusive or of its address
    static constexpr int STAGE = (META_AT + 16 + ROW - 1) / ROW * ROW;
    static constexpr int STAGES = STAGE * 4 * kAtWarps <= 48 * 1024 ? 4 : 3;
    // a tile's decoded scales: words of key scales, then of value scales
    static constexpr int SCALES_AT = STAGES * STAGE, WARP = SCALES_AT + (NARROW ? 0 : 128 * SW);
    // piece swizzle by row: the eight rows a K read touches at once, and the
    // four of a V read, fall on different banks.  Rows 8 apart have the same,
    // and of row t + 4 i (t < 4) it is swz(t) ^ swz4(i).
    static __host__ __device__ constexpr int swz(int row)
    {
        return BITS == 8 && NPC == 4 ? (row & 2) | ((row >> 2) & 1) : BITS == 8 ? ((row & 3) << 1) | ((row >> 2) & 1)
               : NPC == 2 ? (row >> 2) & 1 : NPC == 4 ? (row >> 1) & 3 : row & 7;
    }
    static __host__ __device__ constexpr int swz4(int i) { return swz(4 * (i & 1)); }
};

__device__ __forceinline__ void cp_async_n(uint32_t dst, const void *src, int n, int src_bytes)
{
    if (n == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
    else if (n == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// shared loads at an immediate offset
template <int OFF> __device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2+%3];" : "=r"(r.x), "=r"(r.y) : "r"(a), "n"(OFF));
    return r;
}
template <int OFF> __device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1+%2];" : "=r"(r) : "r"(a), "n"(OFF));
    return r;
}
template <int OFF> __device__ __forceinline__ uint32_t lds16(uint32_t a)
{
    uint16_t r;
    asm volatile("ld.shared.b16 %0, [%1+%2];" : "=h"(r) : "r"(a), "n"(OFF));
    return r;
}

__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y)
{
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 2^x, good to 2 ulp; results below 2^-126 are zero
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// x as f16 in both halves
__device__ __forceinline__ uint32_t half2_of(float x)
{
    const __half2 h = __floats2half2_rn(x, x);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// two code pairs (16 bits of 4-bit codes, 32 of FP6) -> two f16x2
template <int EL> __device__ __forceinline__ void pairs2(uint32_t c, uint32_t &lo, uint32_t &hi)
{
    if (EL == GE_E2M1) {
        // (c is no value loaded in 8 or 16 bits: of such a one, nvcc 12.9's
        // conversion of another byte than the first came out wrong)
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %2;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(c));
    } else if (EL == AE_E2M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e2m3x2 %0, a;\n\tcvt.rn.f16x2.e2m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(c));
    } else if (EL == AE_E3M2) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e3m2x2 %0, a;\n\tcvt.rn.f16x2.e3m2x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(c));
    } else {
        uint32_t h[4];
        codes8_halves<EL>(c, h);
        lo = h[0];
        hi = h[1];
    }
}

// Eight codes of lane t in 32-block b of a key row -> four f16x2.  at: the
// lane's place in row g, swizzle and lane part of the piece included; OFF: to
// the row.
template <int EL, int D, int BS, int OFF>
__device__ __forceinline__ void at_key_codes(uint32_t at, int b, int t, uint32_t h[4])
{
    using G = AtGeom<EL, D, BS>;
    if constexpr (G::BITS == 4) {
        const uint32_t p = at ^ (b << 4);
        uint32_t w;
        if (BS == 16) w = __byte_perm(lds32<OFF>(p), lds32<OFF + 8>(p), (t & 1) ? 0x7632u : 0x5410u);
        else w = lds32<OFF>(p);
        codes8_halves<EL>(w, h);
    } else {
        uint2 w;
        if (BS == 16) w = make_uint2(lds32<OFF>(at ^ (b << 5)), lds32<OFF>(at ^ (b << 5) ^ 16));   // four codes of each half
        else w = lds64<OFF>(at ^ (b << 5));
        pairs2<EL>(w.x, h[0], h[1]);
        pairs2<EL>(w.y, h[2], h[3]);
    }
}
template <int EL, int D, int BS> __device__ __forceinline__ uint32_t at_key_lane(int g, int t)
{
    using G = AtGeom<EL, D, BS>;
    const uint32_t row = g * G::ROW + (G::swz(g) << 4);
    if (G::BITS == 4) return row + (BS == 16 ? 4 * (t >> 1) : 4 * t);
    return BS == 16 ? row + 4 * t : (row ^ ((t >> 1) << 4)) + 8 * (t & 1);
}

// Code pairs 2g, 2g + 1 (blocks of 16: g and g + 8) of 32-block b of value rows
// t + 4 I and t + 4 I + 4 -> the operand's rows g and g + 8.  at: the lane's place
// in row t; sel: which bytes of its words the lane takes (at_value_sel).
template <int EL, int D, int BS, int I>
__device__ __forceinline__ void at_value_codes(uint32_t at, int b, uint32_t sel, uint32_t lo[2], uint32_t hi[2])
{
    using G = AtGeom<EL, D, BS>;
    constexpr int OFF = 4 * I * G::ROW, OFF2 = OFF + 4 * G::ROW;
    if constexpr (G::BITS == 4) {
        const uint32_t p = at ^ ((b ^ G::swz4(I)) << 4), p2 = at ^ ((b ^ G::swz4(I + 1)) << 4);
        if constexpr (BS == 16) {
            // byte g of each half, out of the word around it
            const uint32_t w = __byte_perm(lds32<OFF>(p), lds32<OFF + 8>(p), sel), w2 = __byte_perm(lds32<OFF2>(p2), lds32<OFF2 + 8>(p2), sel);
            pairs2<EL>(w, lo[0], hi[0]);
            pairs2<EL>(w2, lo[1], hi[1]);
        } else {
            // two bytes of each row's word
            const uint32_t w = __byte_perm(lds32<OFF>(p), lds32<OFF2>(p2), sel);
            uint32_t h[4];
            codes8_halves<EL>(w, h);
            lo[0] = h[0];
            hi[0] = h[1];
            lo[1] = h[2];
            hi[1] = h[3];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t p = at ^ (((2 * b) ^ G::swz4(I + k)) << 4);
            const uint32_t w = BS == 16 ? __byte_perm(lds16<OFF>(p + k * 4 * G::ROW), lds16<OFF>((p ^ 16) + k * 4 * G::ROW), 0x5410u)
                                        : lds32<OFF>(p + k * 4 * G::ROW);
            pairs2<EL>(w, lo[k], hi[k]);
        }
    }
}
template <int BS> __device__ __forceinline__ uint32_t at_value_sel(int g)
{
    return BS == 16 ? (uint32_t)((g & 3) | ((g & 3) + 4) << 4) : (g & 1) ? 0x7632u : 0x5410u;
}
template <int EL, int D, int BS> __device__ __forceinline__ uint32_t at_value_lane(int g, int t)
{
    using G = AtGeom<EL, D, BS>;
    const uint32_t row = G::V_AT + t * G::ROW + (G::swz(t) << 4);
    if (G::BITS == 4) return row + (BS == 16 ? (g & 4) : 2 * (g & 6));
    return BS == 16 ? row + 2 * g : (row ^ ((g >> 2) << 4)) + 4 * (g & 3);
}

// A token's scales -> binary32, one per 32-block (two with blocks of 16).
template <int EL, int D, int BS>
__device__ __forceinline__ void at_scales(const AttnParams &p, uint32_t area, int tok, uint32_t shifts, const uint32_t sel[2],
                                          const float *m, float *s)
{
    // (m: a power of two per 32-block)
    using G = AtGeom<EL, D, BS>;
    const uint32_t a = area + tok * G::SW;
    if (BS == 16) {
#pragma unroll
        for (int i = 0; i < G::SW / 4; ++i) {
            const float f[4] = {m[2 * i], m[2 * i], m[2 * i + 1], m[2 * i + 1]};
            scales4_times(p.sfmt, lds32(a + 4 * i), f, s + 4 * i);
        }
        return;
    }
    float f4[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f4[i] = i < G::NB ? m[i < G::NB ? i : 0] : 1.0f;
    uint32_t w0 = lds32(a), w1 = 0u;
    if (G::SW > 4) w1 = lds32(a + 4);
    if (G::NARROW) w0 >>= shifts;
    float f[4];
    scales4_times(p.sfmt, BS == 64 ? __byte_perm(w0, w1, sel[0]) : w0, f4, f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < G::NB) s[i] = f[i];
    if (G::NB > 4) {
        scales4_times(p.sfmt, BS == 64 ? __byte_perm(w0, w1, sel[1]) : w1, f4 + 4, f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 + i < G::NB) s[4 + i] = f[i];
    }
}

// Eight consecutive query values.
__device__ __forceinline__ void at_load8(const AttnParams &p, int64_t at, bool on, float v[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (!on) return;
    if (p.q_fp32) {
        const float *x = static_cast<const float *>(p.q) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[i];
    } else {
        const uint16_t *x = static_cast<const uint16_t *>(p.q) + at;
        if (p.q_vec) {
            const uint4 a = *reinterpret_cast<const uint4 *>(x);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bits2f(w[i] << 16);
                v[2 * i + 1] = bits2f(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = bits2f((uint32_t)x[i] << 16);
        }
    }
}

// The scale of 32-block j (blocks of 16: its half u) of a tile's value token, by
// itself.  shift: bits to the token's first scale in its word.
template <int EL, int D, int BS>
__device__ __forceinline__ float at_value_scale(const AttnParams &p, uint32_t st, int tok, uint32_t shift, int j, int u)
{
    using G = AtGeom<EL, D, BS>;
    const uint32_t at = BS == 16 ? 2 * j + u : G::NARROW ? (shift >> 3) + ((32 * j) >> p.log2B) : j;
    uint32_t b;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b) : "r"(st + G::VS_AT + tok * G::SW + at));
    return scale1(p.sfmt, b);
}

// visible tokens of a sequence, and the token of visible index i
__device__ __forceinline__ void at_visible(const AttnParams &p, int b, int &n, int &vis, int &sinks)
{
    n = max(p.lengths[b], 0);
    n = (int)min((int64_t)n, (int64_t)p.max_pages * p.page_size);
    sinks = 0;
    vis = n;
    if (p.window > 0) {
        const int first = max(n - p.window, 0);      // the window's first token
        sinks = min(p.sinks, first);
        vis = n - first + sinks;
    }
}

// The weight of a stretch's result (m, l) at the common maximum: one without a
// visible token has m = -inf, l = 0; one whose scores are NaN makes the result NaN.
__device__ __forceinline__ float at_weight(float2 ml, float m)
{
    return ml.y == 0.0f ? 0.0f : ml.y != ml.y ? ml.y : ml.y * exp2f(ml.x - m);
}
// Over the sum of the weights: nothing where there are none.
__device__ __forceinline__ float at_over(float l) { return l > 0.0f || l != l ? __fdiv_rn(1.0f, l) : 0.0f; }
// Four elements of a head; l: the sum of weights at the maximum m.
__device__ __forceinline__ void at_store4(const AttnParams &p, int seq, int head, int d, float m, float l, const float o[4])
{
    const bool any = l > 0.0f || l != l;
    const int64_t at = (int64_t)seq * p.ldo + (int64_t)head * p.head_dim + d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float y = any ? o[i] : 0.0f;
        if (p.o_fp32) static_cast<float *>(p.out)[at + i] = y;
        else static_cast<__nv_bfloat16 *>(p.out)[at + i] = __float2bfloat16_rn(y);
    }
    if (d == 0 && p.lse) p.lse[(int64_t)seq * p.q_heads + head] = any ? (m + log2f(l)) * 0.693147180559945309417f : -INFINITY;
}

// Four E4M3 scale bytes -> their f16 pairs (s, s).
__device__ __forceinline__ void e4m3_pairs(uint32_t w, uint32_t s[4])
{
    const uint32_t top = w & 0x80808080u;   // (no finite scale has the sign bit: NaN)
    if (top) w |= (top >> 7) * 0x7fu;
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    s[0] = __byte_perm(lo, lo, 0x1010u);
    s[1] = __byte_perm(lo, lo, 0x3232u);
    s[2] = __byte_perm(hi, hi, 0x1010u);
    s[3] = __byte_perm(hi, hi, 0x3232u);
}
// f16 pairs (s, s) of the scales of value blocks (E4M3): SUB of 32-block j
template <int EL, int D, int BS>
__device__ __forceinline__ void at_scales_half(uint32_t area, int tok, uint32_t shifts, uint32_t *s)
{
    using G = AtGeom<EL, D, BS>;
    const uint32_t a = area + tok * G::SW;
#pragma unroll
    for (int i = 0; i < G::SW / 4; ++i) {
        uint32_t w = lds32(a + 4 * i);
        if (G::NARROW) w >>= shifts;
        uint32_t x[4];
        e4m3_pairs(w, x);
        constexpr int N = G::NB * (BS == 16 ? 2 : 1);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (4 * i + k < N) s[4 * i + k] = x[k];
    }
}

// The lane's share of a tile's scale bytes (SW / 2 of them, at `from`), each
// decoded once, into words for all lanes: binary32 times m (null: 1), f16 pairs
// of that (HALF), f16 pairs of E4M3 bytes (E4M3).
enum { AS_F32 = 0, AS_HALF = 1, AS_E4M3 = 2 };
template <int SW, int TO>
__device__ __forceinline__ void at_spread_scales(int fmt, uint32_t from, uint32_t to, int lane, const float *m)
{
    from += lane * (SW / 2);
    to += lane * (SW * 2);
#pragma unroll
    for (int i = 0; i < (SW + 7) / 8; ++i) {
        const uint32_t w = SW == 4 ? lds16(from) : lds32(from + 4 * i);
        uint32_t o[4];
        if (TO == AS_E4M3) {
            e4m3_pairs(w, o);
        } else {
            float f[4];
            if (m) {
                const float m4[4] = {m[4 * i], m[4 * i + 1], m[SW == 4 ? 0 : 4 * i + 2], m[SW == 4 ? 0 : 4 * i + 3]};
                scales4_times(fmt, w, m4, f);
            } else {
                scales4(fmt, w, f);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = TO == AS_HALF ? half2_of(f[k]) : __float_as_uint(f[k]);
        }
        if (SW == 4) sts64(to, o[0], o[1]);
        else sts128(to + 16 * i, o[0], o[1], o[2], o[3]);
    }
}
// A token's words.
template <int SW> __device__ __forceinline__ void at_token_words(uint32_t area, int tok, uint32_t *w)
{
#pragma unroll
    for (int i = 0; i < SW / 4; ++i) {
        const uint4 x = lds128(area + tok * (SW * 4) + 16 * i);
        w[4 * i] = x.x;
        w[4 * i + 1] = x.y;
        w[4 * i + 2] = x.z;
        w[4 * i + 3] = x.w;
    }
}

// NTH: groups of four heads (1 or 2); HP: binary32 precision (two pieces of
// queries and weights); VM: 1, value codes scaled as f16 (E2M1 with E4M3 scales);
// 2, weights scaled as f16 (E8M0 scales: powers of two, so that only the weight is rounded)
template <int EL, int D, int BS, int NTH, int HP, int VM>
__global__ void __launch_bounds__(32 * at_warps<D, BS, NTH, HP>(), 1) k_attn(const __grid_constant__ AttnParams p)
{
    using G = AtGeom<EL, D, BS>;
    constexpr int NB = G::NB, SUB = BS == 16 ? 2 : 1, PC = HP ? 2 : 1;
    constexpr int PB = VM == 1 ? 10 : 7;           // the weights' f16 exponent
    extern __shared__ __align__(256) uint8_t smem_at[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    pdl_trigger();
    pdl_wait();

    // the warp's task: key head fastest, then head group, split, sequence; the
    // warps of a joined CTA are the splits
    const int warps = blockDim.x >> 5;
    int64_t task = p.joined ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * warps + warp;
    if (task >= p.tasks) return;
    const int kh = (int)(task % p.kv_heads);
    task /= p.kv_heads;
    const int hg = (int)(task % p.head_groups);
    task /= p.head_groups;
    const int split = p.joined ? warp : (int)(task % p.splits);
    const int seq = (int)(p.joined ? task : task / p.splits);
    const int h0 = kh * p.group + hg * (4 * NTH);           // first query head
    const int hn = min(4 * NTH, p.group - hg * (4 * NTH));  // heads of this task
    int n, vis, sinks;
    at_visible(p, seq, n, vis, sinks);
    const int tiles = (vis + 15) >> 4, per = (tiles + p.splits - 1) / p.splits;
    const int tile0 = split * per, tile1 = min(tile0 + per, tiles);
    // (the join's launch reads no more than the splits in use)
    if (tile0 >= tile1 && p.splits > 1 && !p.joined) return;

    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem_at) + warp * G::WARP;
    const int skip = n - vis;                 // tokens between the sinks and the window
    const int32_t *table = p.table + (int64_t)seq * p.ld_table;
    const int nsc = D >> p.log2B;             // scales of a head
    const uint32_t code_row = (uint32_t)p.kv_heads * G::ROW, sc_row = (uint32_t)(p.kv_heads * nsc);   // (under 2^20)
    const uint8_t *kc = p.k_codes + kh * G::ROW, *vc = p.v_codes + kh * G::ROW;
    // lanes 0..15 copy key scales of their token, 16..31 value scales
    const uint8_t *sc = (lane < 16 ? p.k_scales : p.v_scales) + (G::NARROW ? 0 : kh * nsc);

    // Rows are looked up for two tiles at a time, a token a lane: the page
    // number of a lane's token is loaded two tiles before its row is used.
    const auto page_of = [&](int tile, int &off) {
        const int i = tile * 16 + lane;
        if (i >= vis || (lane >= 16 && tile + 1 >= tile1)) return -1;
        const int tok = i < sinks ? i : i + skip;
        const int pg = p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_size;
        off = tok - pg * p.page_size;
        return (int)table[pg];
    };
    int next_off = 0, next_page = tile0 < tile1 ? page_of(tile0, next_off) : -1, it = tile0;
    uint32_t rows = 0u, there = 0u;           // of the two tiles: the lane's row, the tokens that are there
    uint32_t st_w = ring;
    constexpr int RPI = 32 / G::NPC;          // rows of one round of copies (NPC <= 32)
    const uint32_t pr = lane / G::NPC, pc = lane % G::NPC;
    kc += pc * 16;
    vc += pc * 16;
    const auto issue = [&]() {
        if (it < tile1) {
            const int second = (it - tile0) & 1;
            if (!second) {
                const bool ok = (uint32_t)next_page < (uint32_t)p.pages;
                rows = ok ? (uint32_t)(next_page * p.page_size + next_off) : 0u;
                there = __ballot_sync(0xffffffffu, ok);
                if (it + 2 < tile1) next_page = page_of(it + 2, next_off);
            }
            const uint32_t mask = second ? there >> 16 : there & 0xffffu;
            ++it;
#pragma unroll
            for (int i = 0; i < 16 / RPI; ++i) {
                const int r = i * RPI + pr;
                const uint64_t at = (uint64_t)__shfl_sync(0xffffffffu, rows, r + 16 * second) * code_row;
                const int nb = (mask >> r) & 1 ? 16 : 0;
                const uint32_t dst = st_w + r * G::ROW + ((pc ^ G::swz(r)) << 4);
                cp_async16(dst + G::K_AT, kc + at, nb);
                cp_async16(dst + G::V_AT, vc + at, nb);
            }
            const uint32_t row = __shfl_sync(0xffffffffu, rows, (lane & 15) + 16 * second);
            const bool ok = (mask >> (lane & 15)) & 1;
            const uint32_t dst = st_w + (lane < 16 ? G::KS_AT : G::VS_AT) + (lane & 15) * G::SW;
            if (!G::NARROW) {
                // (BS 32: a byte per 32-block, BS 16: two)
                cp_async_n(dst, sc + (uint64_t)row * sc_row, G::SW, ok ? G::SW : 0);
                if (lane == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(st_w + G::META_AT), "r"(mask) : "memory");
            } else {
                const uint64_t at = (uint64_t)row * sc_row + kh * nsc;
                int shift = 0;
                if (nsc >= 4) {
                    cp_async_n(dst, sc + at, nsc, ok ? nsc : 0);
                } else {
                    // one or two bytes: the aligned word around them
                    shift = (int)(at & 3);
                    const uint64_t w = at & ~(uint64_t)3;
                    cp_async_n(dst, sc + w, 4, ok ? (int)min((int64_t)4, p.scale_bytes - (int64_t)w) : 0);
                }
                const uint32_t b0 = __ballot_sync(0xffffffffu, shift & 1), b1 = __ballot_sync(0xffffffffu, shift & 2);
                if (lane == 0)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(st_w + G::META_AT), "r"(mask), "r"(b0 & 0xffffu),
                                 "r"(b1 & 0xffffu), "r"(0u) : "memory");
            }
        }
        st_w = st_w + G::STAGE == ring + G::STAGES * G::STAGE ? ring : st_w + G::STAGE;
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < G::STAGES - 1; ++i) issue();

    // queries: lane (g, t) holds head h0 + g at the k places of its code words
    uint32_t qf[PC][NB][4];
    float qe;                                 // 2^-e of head h0 + g
    {
        float v[NB][8];
        uint32_t m = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int64_t at = (int64_t)seq * p.ldq + (int64_t)(h0 + g) * D + 32 * b;
            if (BS == 16) {
                // codes 4t.. of the first half, 4t.. of the second
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t e = at + 16 * (i >> 2) + 4 * t + (i & 3);
                    v[b][i] = g >= hn ? 0.0f : p.q_fp32 ? static_cast<const float *>(p.q)[e]
                                                        : bits2f((uint32_t)static_cast<const uint16_t *>(p.q)[e] << 16);
                }
            } else {
                at_load8(p, at + 8 * t, g < hn, v[b]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[b][i]) & 0x7fffffffu);
        }
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = f16_scale_exponent(bits2f(m));
        const float f = exp2i(e);
        qe = exp2i(-e);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = __fmul_rn(v[b][2 * i], f), y = __fmul_rn(v[b][2 * i + 1], f);
                const __half2 h = __floats2half2_rn(x, y);
                qf[0][b][i] = *reinterpret_cast<const uint32_t *>(&h);
                if (HP) {
                    const float2 back = __half22float2(h);
                    float rx = __fmul_rn(__fsub_rn(x, back.x), 2048.0f), ry = __fmul_rn(__fsub_rn(y, back.y), 2048.0f);
                    rx = rx == rx ? rx : 0.0f;
                    ry = ry == ry ? ry : 0.0f;
                    const __half2 h2 = __floats2half2_rn(rx, ry);
                    qf[PC - 1][b][i] = *reinterpret_cast<const uint32_t *>(&h2);
                }
            }
    }
    // score factor of heads 2t and 2t + 1: softmax scale, log2 e, tensor scale
    const float base = p.scale * 1.44269504088896340736f;
    const float kts = p.k_ts ? *p.k_ts : 1.0f;
    const float fac0 = __fmul_rn(__fmul_rn(base, kts), __shfl_sync(0xffffffffu, qe, 8 * t));
    const float fac1 = __fmul_rn(__fmul_rn(base, kts), __shfl_sync(0xffffffffu, qe, 8 * t + 4));
    // scale bytes of the 32-blocks within the token's words
    uint32_t sel[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) sel[i >> 2] |= (uint32_t)((32 * i) >> p.log2B) << (4 * (i & 3));

    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;   // heads 2t, 2t + 1
    float cb[NB];                             // 2^-E of the value blocks' reference exponents
    float acc[NTH][NB][4];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        cb[j] = VM == 1 ? 1.0f : 0.0f;        // (none yet)
#pragma unroll
        for (int q = 0; q < NTH; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[q][j][i] = 0.0f;
    }

    const uint32_t k_lane = at_key_lane<EL, D, BS>(g, t), v_lane = at_value_lane<EL, D, BS>(g, t), v_sel = at_value_sel<BS>(g);
    uint32_t lim[(G::SW + 7) / 8] = {};       // upper limits of the lane's share of value scale bytes
    const uint32_t span = p.sfmt == S_E8M0 ? 9u : 72u;   // codes from 2^-6 to 2^3 (an exponent is 8 codes of a minifloat)
    bool wide = false;                        // value scales too far apart for f16 weights
    float cl[(G::SW + 7) / 8 * 4] = {};       // and their blocks' 2^-E
    const uint32_t words = ring + G::SCALES_AT;
    uint32_t st = ring;
    uint4 meta;                               // tokens that are there, and
    // where a token's scales begin in their word
    const auto shift_of = [&](int tk) { return G::NARROW ? (((meta.y >> tk) & 1) | (((meta.z >> tk) & 1) << 1)) * 8 : 0u; };
    // A tile's scores, weights and products, and on to the next.
    const auto tile_sums = [&](auto wide_tag) {
        constexpr bool WIDE = decltype(wide_tag)::value;
        // the tile's scales, each decoded by one lane
        if constexpr (!G::NARROW) {
            at_spread_scales<G::SW, AS_F32>(p.sfmt, st + G::KS_AT, words, lane, nullptr);
            at_spread_scales<G::SW, VM == 0 ? AS_F32 : VM == 1 ? AS_E4M3 : AS_HALF>(p.sfmt, st + G::VS_AT, words + 64 * G::SW, lane, cl);
            __syncwarp();
        }

        // scores of tokens g, g + 8 (heads 2t, 2t + 1)
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        {
            float kl[NB * SUB], kg[NB * SUB];
            if constexpr (!G::NARROW) {
                uint32_t wl[NB * SUB], wg[NB * SUB];
                at_token_words<G::SW>(words, g, wl);
                at_token_words<G::SW>(words, g + 8, wg);
#pragma unroll
                for (int j = 0; j < NB * SUB; ++j) {
                    kl[j] = bits2f(wl[j]);
                    kg[j] = bits2f(wg[j]);
                }
            } else {
                float one[NB];
#pragma unroll
                for (int j = 0; j < NB; ++j) one[j] = 1.0f;
                at_scales<EL, D, BS>(p, st + G::KS_AT, g, shift_of(g), sel, one, kl);
                at_scales<EL, D, BS>(p, st + G::KS_AT, g + 8, shift_of(g + 8), sel, one, kg);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t lo[4], hi[4];
                at_key_codes<EL, D, BS, 0>(st + k_lane, b, t, lo);
                at_key_codes<EL, D, BS, 8 * G::ROW>(st + k_lane, b, t, hi);
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    float d[4], e[4];
                    if (SUB == 2) {
                        mma_16816_zero(d, lo[2 * u], hi[2 * u], lo[2 * u + 1], hi[2 * u + 1], qf[0][b][2 * u], qf[0][b][2 * u + 1]);
                        if (HP) mma_16816_zero(e, lo[2 * u], hi[2 * u], lo[2 * u + 1], hi[2 * u + 1], qf[PC - 1][b][2 * u], qf[PC - 1][b][2 * u + 1]);
                    } else {
                        mma_16816_zero(d, lo[0], hi[0], lo[1], hi[1], qf[0][b][0], qf[0][b][1]);
                        mma_16816(d, lo[2], hi[2], lo[3], hi[3], qf[0][b][2], qf[0][b][3]);
                        if (HP) {
                            mma_16816_zero(e, lo[0], hi[0], lo[1], hi[1], qf[PC - 1][b][0], qf[PC - 1][b][1]);
                            mma_16816(e, lo[2], hi[2], lo[3], hi[3], qf[PC - 1][b][2], qf[PC - 1][b][3]);
                        }
                    }
                    if (HP) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) d[i] = fmaf(e[i], 0x1p-11f, d[i]);
                    }
                    s[0] = fmaf(kl[b * SUB + u], d[0], s[0]);
                    s[1] = fmaf(kl[b * SUB + u], d[1], s[1]);
                    s[2] = fmaf(kg[b * SUB + u], d[2], s[2]);
                    s[3] = fmaf(kg[b * SUB + u], d[3], s[3]);
                }
            }
        }
        s[0] = __fmul_rn(s[0], fac0);
        s[1] = __fmul_rn(s[1], fac1);
        s[2] = __fmul_rn(s[2], fac0);
        s[3] = __fmul_rn(s[3], fac1);
        if (meta.x != 0xffffu) {
            if (!((meta.x >> g) & 1)) s[0] = s[1] = -INFINITY;
            if (!((meta.x >> (g + 8)) & 1)) s[2] = s[3] = -INFINITY;
        }

        // move the reference when a score passes it by 2^4
        if (__any_sync(0xffffffffu, fmaxf(s[0], s[2]) > m0 + 4.0f || fmaxf(s[1], s[3]) > m1 + 4.0f)) {
            float a = fmaxf(m0, fmaxf(s[0], s[2])), c = fmaxf(m1, fmaxf(s[1], s[3]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
                c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, d));
            }
            const float r0 = m0 == a ? 1.0f : ex2(m0 - a), r1 = m1 == c ? 1.0f : ex2(m1 - c);
            m0 = a;
            m1 = c;
            l0 *= r0;
            l1 *= r1;
            // the sums of head t (+ 4): its factor is with lane t >> 1 (+ 2)
#pragma unroll
            for (int q = 0; q < NTH; ++q) {
                const float x = __shfl_sync(0xffffffffu, r0, (t >> 1) + 2 * q), y = __shfl_sync(0xffffffffu, r1, (t >> 1) + 2 * q);
                const float r = (t & 1) ? y : x;
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[q][j][i] *= r;
            }
        }
        // weights and their sums times 2^PB
        const float b0 = m0 == -INFINITY ? 0.0f : m0 - PB, b1 = m1 == -INFINITY ? 0.0f : m1 - PB;
        s[0] = ex2(s[0] - b0);
        s[1] = ex2(s[1] - b1);
        s[2] = ex2(s[2] - b0);
        s[3] = ex2(s[3] - b1);
        l0 += s[0] + s[2];
        l1 += s[1] + s[3];

        if constexpr (WIDE) {
            // Token t + 4 i of parity e is k = t (+ 4) of the instruction for that
            // parity: the columns of the other parity have weight zero.
#pragma unroll
            for (int q = 0; q < NTH; ++q) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int from = (t + 4 * (i & 1)) * 4 + (g >> 2) + 2 * q;
                    const float x0 = __shfl_sync(0xffffffffu, s[i & 2], from), x1 = __shfl_sync(0xffffffffu, s[(i & 2) + 1], from);
                    w[i] = (g >> 1) & 1 ? x1 : x0;
                }
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    uint32_t lo[4], hi[4];
                    at_value_codes<EL, D, BS, 0>(st + v_lane, j, v_sel, lo, hi);
                    at_value_codes<EL, D, BS, 2>(st + v_lane, j, v_sel, lo + 2, hi + 2);
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            float x[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int tk = t + 4 * (i + k);
                                x[k] = __fmul_rn(w[i + k], __fmul_rn(at_value_scale<EL, D, BS>(p, st, tk, shift_of(tk), j, u), cb[j]));
                            }
#pragma unroll
                            for (int piece = 0; piece < PC; ++piece) {
                                uint32_t b[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    b[k] = tf32_of(x[k]);
                                    x[k] = __fsub_rn(x[k], bits2f(b[k]));
                                }
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const uint32_t b0 = (g & 1) == e ? b[0] : 0u, b1 = (g & 1) == e ? b[1] : 0u;
                                    // (blocks of 16: the rows of the half's own pairs)
                                    const bool l = SUB == 1 || u == 0, h = SUB == 1 || u == 1;
                                    mma_1688_tf32(acc[q][j], l ? tf32_of_half(lo[i], e) : 0u, h ? tf32_of_half(hi[i], e) : 0u,
                                                  l ? tf32_of_half(lo[i + 1], e) : 0u, h ? tf32_of_half(hi[i + 1], e) : 0u, b0, b1);
                                }
                            }
                        }
                    }
                }
            }
            st = st + G::STAGE == ring + G::STAGES * G::STAGE ? ring : st + G::STAGE;
            return;
        }

        float vs[4][NB * SUB];                // (VM 0) value scales of tokens t, t + 4, t + 8, t + 12 over the references
        uint32_t vh[4][NB * SUB];             // (else) as f16 pairs: the scales, or over the references
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (!G::NARROW) {
                uint32_t w[NB * SUB];
                at_token_words<G::SW>(words + 64 * G::SW, t + 4 * i, w);
#pragma unroll
                for (int j = 0; j < NB * SUB; ++j) {
                    if (VM) vh[i][j] = w[j];
                    else vs[i][j] = bits2f(w[j]);
                }
            } else if constexpr (VM) {
                at_scales_half<EL, D, BS>(st + G::VS_AT, t + 4 * i, shift_of(t + 4 * i), vh[i]);
            } else {
                at_scales<EL, D, BS>(p, st + G::VS_AT, t + 4 * i, shift_of(t + 4 * i), sel, cb, vs[i]);
            }
        }
        // weights of the lane's tokens and column: head g >> 1 (+ 4 q), parity g & 1
        float pw[NTH][4];                     // (VM 0, or two pieces)
        uint32_t wv[NTH][PC][4];              // (VM 1, 2) as f16 pieces, (w, 0) or (0, w)
        const bool odd = (g >> 1) & 1;
        const uint32_t par = (g & 1) ? 0x3c000000u : 0x00003c00u;
        if constexpr (VM && !HP) {
            const __half2 h0 = __floats2half2_rn(s[0], s[1]), h1 = __floats2half2_rn(s[2], s[3]);
            const uint32_t k0 = *reinterpret_cast<const uint32_t *>(&h0), k1 = *reinterpret_cast<const uint32_t *>(&h1);
            const uint32_t pick = (g & 1) ? (odd ? 0x3244u : 0x1044u) : odd ? 0x4432u : 0x4410u;
#pragma unroll
            for (int q = 0; q < NTH; ++q)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int from = (t + 4 * i) * 4 + (g >> 2) + 2 * q;
                    wv[q][0][i] = __byte_perm(__shfl_sync(0xffffffffu, k0, from), 0u, pick);
                    wv[q][0][2 + i] = __byte_perm(__shfl_sync(0xffffffffu, k1, from), 0u, pick);
                }
        } else {
#pragma unroll
            for (int q = 0; q < NTH; ++q) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int from = (t + 4 * i) * 4 + (g >> 2) + 2 * q;
                    const float x0 = __shfl_sync(0xffffffffu, s[0], from), x1 = __shfl_sync(0xffffffffu, s[1], from);
                    const float y0 = __shfl_sync(0xffffffffu, s[2], from), y1 = __shfl_sync(0xffffffffu, s[3], from);
                    pw[q][i] = odd ? x1 : x0;
                    pw[q][2 + i] = odd ? y1 : y0;
                }
                if constexpr (VM) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t h = half2_of(pw[q][i]);
                        const float back = __low2float(*reinterpret_cast<const __half2 *>(&h));
                        wv[q][0][i] = hmul2_u(h, par);
                        wv[q][PC - 1][i] = hmul2_u(half2_of(__fmul_rn(__fsub_rn(pw[q][i], back), 2048.0f)), par);
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            uint32_t lo[4], hi[4];
            at_value_codes<EL, D, BS, 0>(st + v_lane, j, v_sel, lo, hi);
            at_value_codes<EL, D, BS, 2>(st + v_lane, j, v_sel, lo + 2, hi + 2);
            if constexpr (VM == 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo[i] = hmul2_u(lo[i], vh[i][j * SUB]);
                    hi[i] = hmul2_u(hi[i], vh[i][j * SUB + SUB - 1]);
                }
#pragma unroll
                for (int q = 0; q < NTH; ++q) {
                    mma_16816(acc[q][j], lo[0], hi[0], lo[1], hi[1], wv[q][0][0], wv[q][0][1]);
                    mma_16816(acc[q][j], lo[2], hi[2], lo[3], hi[3], wv[q][0][2], wv[q][0][3]);
                    if (HP) {
                        float e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma_16816(e, lo[0], hi[0], lo[1], hi[1], wv[q][PC - 1][0], wv[q][PC - 1][1]);
                        mma_16816(e, lo[2], hi[2], lo[3], hi[3], wv[q][PC - 1][2], wv[q][PC - 1][3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[q][j][i] = fmaf(e[i], 0x1p-11f, acc[q][j][i]);
                    }
                }
                continue;
            }
#pragma unroll
            for (int q = 0; q < NTH; ++q)
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    uint32_t w[PC][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (VM == 2) {
                            // (a power of two times an f16: exact but below 2^-14)
                            w[0][i] = hmul2_u(wv[q][0][i], vh[i][j * SUB + u]);
                            continue;
                        }
                        const float x = __fmul_rn(pw[q][i], vs[i][j * SUB + u]);
                        const uint32_t h = half2_of(x);
                        w[0][i] = hmul2_u(h, par);   // (on the FMA pipe: the integer pipe is the busy one)
                        if (HP) {
                            const float back = __low2float(*reinterpret_cast<const __half2 *>(&h));
                            w[PC - 1][i] = hmul2_u(half2_of(__fmul_rn(__fsub_rn(x, back), 2048.0f)), par);
                        }
                    }
                    // blocks of 16: rows below 8 are the first half's pairs,
                    // the others the second's, each against its own weights
                    const uint32_t z = 0u;
#define AT_PV(d, wt)                                                                                                          \
    if (SUB == 1) {                                                                                                           \
        mma_16816(d, lo[0], hi[0], lo[1], hi[1], wt[0], wt[1]);                                                               \
        mma_16816(d, lo[2], hi[2], lo[3], hi[3], wt[2], wt[3]);                                                               \
    } else if (u == 0) {                                                                                                      \
        mma_16816(d, lo[0], z, lo[1], z, wt[0], wt[1]);                                                                       \
        mma_16816(d, lo[2], z, lo[3], z, wt[2], wt[3]);                                                                       \
    } else {                                                                                                                  \
        mma_16816(d, z, hi[0], z, hi[1], wt[0], wt[1]);                                                                       \
        mma_16816(d, z, hi[2], z, hi[3], wt[2], wt[3]);                                                                       \
    }
                    AT_PV(acc[q][j], w[0])
                    if (HP) {
                        float e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        AT_PV(e, w[PC - 1])
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[q][j][i] = fmaf(e[i], 0x1p-11f, acc[q][j][i]);
                    }
#undef AT_PV
                }
        }
        st = st + G::STAGE == ring + G::STAGES * G::STAGE ? ring : st + G::STAGE;
    };
    // Is a value scale of the tile past 2^3 times its block's reference, or below
    // 2^-6 of it?  Code 0 is not: a block of zeros, or a token that is not there
    // (2^-127 beside larger scales counts as zero).  Each lane looks at its share of
    // the tile's scales; their codes order like their values.
    const auto outside = [&]() {
        bool past = false;
        if (G::NARROW) {
            // (a token a lane, its even or odd 32-blocks)
#pragma unroll
            for (int j = 0; j < NB; j += 2) {
                const float y = at_value_scale<EL, D, BS>(p, st, lane & 15, shift_of(lane & 15), j + (lane >> 4), 0);
                const float x = __fmul_rn(y, lane < 16 ? cb[j] : cb[j + 1]);
                past |= x > 8.0f || (x < 0x1p-6f && y > 0x1p-127f);
            }
        } else {
            const uint32_t a = st + G::VS_AT + lane * (G::SW / 2);
#pragma unroll
            for (int i = 0; i < (G::SW + 7) / 8; ++i) {
                const uint32_t w = G::SW == 4 ? lds16(a) : lds32(a + 4 * i);
#pragma unroll
                for (int k = 0; k < (G::SW == 4 ? 2 : 4); ++k) {
                    const uint32_t c = (w >> (8 * k)) & 0xffu;
                    past |= ((lim[i] >> (8 * k)) & 0xffu) - c > span && c;
                }
            }
        }
        return past;
    };
    // New references where the tile's value scales ask for them; and are they too far
    // apart for f16 weights from here on?
    const auto references = [&]() {
        float x[NB], one[NB];
        bool far = false;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            x[j] = 0.0f;
            one[j] = 1.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[NB * SUB];
            at_scales<EL, D, BS>(p, st + G::VS_AT, t + 4 * i, shift_of(t + 4 * i), sel, one, y);
#pragma unroll
            for (int j = 0; j < NB * SUB; ++j) x[j / SUB] = fmaxf(x[j / SUB], y[j]);
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            x[j] = fmaxf(x[j], __shfl_xor_sync(0xffffffffu, x[j], 1));
            x[j] = fmaxf(x[j], __shfl_xor_sync(0xffffffffu, x[j], 2));
            // 2^-floor(log2 x), itself and 2^E normal numbers
            const int e = min(max((int)(__float_as_uint(x[j]) >> 23) - 127, -126), 126);
            const float c = exp2i(-e);
            if (cb[j] == 0.0f || 8.0f * c <= cb[j]) {
                far |= cb[j] != 0.0f;
                const float r = cb[j] == 0.0f ? 1.0f : __fmul_rn(c, exp2i(127 - (int)(__float_as_uint(cb[j]) >> 23)));
#pragma unroll
                for (int q = 0; q < NTH; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[q][j][i] *= r;
                cb[j] = c;
            }
        }
        if (!G::NARROW) {
            // the limits of the lane's bytes: the code of 2^(E + 3)
#pragma unroll
            for (int i = 0; i < (G::SW + 7) / 8; ++i) {
                lim[i] = 0u;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = (lane * (G::SW / 2) + 4 * i + k) & (G::SW - 1);   // the byte's scale
                    int e = 0;
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        if (at / SUB == j) e = 127 - (int)(__float_as_uint(cb[j]) >> 23);
                    const int code = p.sfmt == S_E8M0 ? e + 130 : (e + 3 + (p.sfmt == S_UE4M3 ? 7 : 15)) * 8;
                    lim[i] |= (uint32_t)min(max(code, 0), 255) << (8 * k);
                    cl[4 * i + k] = exp2i(-e);
                }
            }
        }
        wide |= __any_sync(0xffffffffu, far || outside());
    };
    const auto arrive = [&]() {
        cp_async_wait<G::STAGES - 2>();
        __syncwarp();                         // the tile is in, and the last one is read
        issue();
        if (G::NARROW) meta = lds128(st + G::META_AT);
        else meta = make_uint4(lds32(st + G::META_AT), 0u, 0u, 0u);
    };
    int tile = tile0;
    for (; tile < tile1; ++tile) {
        arrive();
        if constexpr (VM != 1) {
            if (__any_sync(0xffffffffu, outside() || tile == tile0)) {
                references();
                if (wide) break;
            }
        }
        tile_sums(std::false_type());
    }
    if constexpr (VM != 1) {
        // the rest of a stretch, whose tile is in
        while (tile < tile1) {
            tile_sums(std::true_type());
            if (++tile == tile1) break;
            arrive();
            references();
        }
    }
    cp_async_wait<0>();

    // the sums over the lanes that share heads
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    const float vts = p.v_ts ? *p.v_ts : 1.0f;
    // a joined CTA's results, in the warps' own rings: 4 NTH heads, then (m, l) of each
    float *mine = reinterpret_cast<float *>(smem_at + warp * G::WARP);
    static_assert(4 * NTH * (D + 2) * 4 <= G::SCALES_AT, "a warp's results fit its ring");
    __syncwarp();                             // the ring is read
#pragma unroll
    for (int q = 0; q < NTH; ++q) {
        const int src = (t >> 1) + 2 * q, head = t + 4 * q;
        const float ma = __shfl_sync(0xffffffffu, m0, src), mb = __shfl_sync(0xffffffffu, m1, src);
        const float la = __shfl_sync(0xffffffffu, l0, src), lb = __shfl_sync(0xffffffffu, l1, src);
        const float m = (t & 1) ? mb : ma, l = (t & 1) ? lb : la;
        if (head >= hn) continue;
        const int64_t out = (int64_t)seq * p.q_heads + h0 + head;
        const bool whole = p.splits == 1;
        // over the sum (a stretch's too, whose sum of large values might pass
        // binary32); of no tokens: zeros
        const float div = at_over(l);
        if (g == 0) {
            if (p.joined) *reinterpret_cast<float2 *>(mine + 4 * NTH * D + 2 * head) = make_float2(m - PB, l);
            else if (!whole) p.part_ml[out * p.splits + split] = make_float2(m - PB, l);
            else if (p.lse) p.lse[out] = l > 0.0f || l != l ? (m - PB + log2f(l)) * 0.693147180559945309417f : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            // 2^E of the block, the tensor scale
            const float f = cb[j] == 0.0f ? 0.0f : __fmul_rn(exp2i(127 - (int)(__float_as_uint(cb[j]) >> 23)), vts);
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = div == 0.0f ? 0.0f : __fmul_rn(__fmul_rn(acc[q][j][i], div), f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int d = 32 * j + (BS == 16 ? 2 * g + 16 * i : 4 * g + 2 * i);
                if (p.joined) {
                    *reinterpret_cast<float2 *>(mine + head * D + d) = make_float2(o[2 * i], o[2 * i + 1]);
                } else if (!whole) {
                    *reinterpret_cast<float2 *>(p.part_o + (out * p.splits + split) * D + d) = make_float2(o[2 * i], o[2 * i + 1]);
                } else {
                    const int64_t at = (int64_t)seq * p.ldo + (int64_t)(h0 + head) * D + d;
                    if (p.o_fp32) {
                        static_cast<float *>(p.out)[at] = o[2 * i];
                        static_cast<float *>(p.out)[at + 1] = o[2 * i + 1];
                    } else {
                        static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(o[2 * i]);
                        static_cast<__nv_bfloat16 *>(p.out)[at + 1] = __float2bfloat16_rn(o[2 * i + 1]);
                    }
                }
            }
        }
    }
    if (!p.joined) return;

    // The join of a CTA's warps, at the common maximum: a lane takes four
    // elements of a head, or of more than four splits every fourth (four lanes,
    // whose sums are added).
    __syncthreads();
    const int items = hn * (D / 4), share = p.splits > 4 ? 2 : 0, step = 1 << share, sub = lane & (step - 1);
    for (int i0 = split * (32 >> share); i0 < items; i0 += p.splits * (32 >> share)) {
        const int item = i0 + (lane >> share), head = min(item / (D / 4), hn - 1), d = 4 * (item & (D / 4 - 1));
        float m = -INFINITY;
#pragma unroll 4
        for (int s = sub; s < p.splits; s += step) {
            const float *r = reinterpret_cast<const float *>(smem_at + s * G::WARP);
            m = fmaxf(m, r[4 * NTH * D + 2 * head]);
        }
        for (int x = 1; x < step; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int s = sub; s < p.splits; s += step) {
            const float *r = reinterpret_cast<const float *>(smem_at + s * G::WARP);
            l += at_weight(*reinterpret_cast<const float2 *>(r + 4 * NTH * D + 2 * head), m);
        }
        __syncwarp();
        for (int x = 1; x < step; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        const float inv = at_over(l);         // (weights of 1 at most: no sum passes binary32)
#pragma unroll 4
        for (int s = sub; s < p.splits; s += step) {
            const float *r = reinterpret_cast<const float *>(smem_at + s * G::WARP);
            const float w = __fmul_rn(at_weight(*reinterpret_cast<const float2 *>(r + 4 * NTH * D + 2 * head), m), inv);
            const float4 v = *reinterpret_cast<const float4 *>(r + head * D + d);
            o[0] = fmaf(w, v.x, o[0]);
            o[1] = fmaf(w, v.y, o[1]);
            o[2] = fmaf(w, v.z, o[2]);
            o[3] = fmaf(w, v.w, o[3]);
        }
        __syncwarp();
        for (int x = 1; x < step; x <<= 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], x);
        }
        if (sub == 0 && item < items) at_store4(p, seq, h0 + head, d, m, l, o);
    }
}

typedef void (*AtKernel)(const AttnParams);
struct AtPick { AtKernel k; int ring; };   // ring: bytes of a warp

template <int EL, int D, int BS, int VM> AtPick at_pick_nth(int nth, int hp)
{
    const int ring = AtGeom<EL, D, BS>::WARP;
    if constexpr (VM != 2) {
        if (hp) return {nth == 1 ? k_attn<EL, D, BS, 1, 1, VM> : k_attn<EL, D, BS, 2, 1, VM>, ring};
    }
    return {nth == 1 ? k_attn<EL, D, BS, 1, 0, VM> : k_attn<EL, D, BS, 2, 0, VM>, ring};
}
// bs: 16, 32, or 64 for blocks of 64 and 128
template <int EL, int D> AtPick at_pick_bs(int bs, int nth, int hp, int sfmt)
{
    if constexpr (EL == GE_E2M1)
        if (sfmt == S_UE4M3 && bs < 64) return bs == 16 ? at_pick_nth<EL, D, 16, 1>(nth, hp) : at_pick_nth<EL, D, 32, 1>(nth, hp);
    if (sfmt == S_E8M0 && !hp && bs == 16) return at_pick_nth<EL, D, 16, 2>(nth, hp);
    if constexpr (D >= 128)
        if (sfmt == S_E8M0 && !hp && bs == 32) return at_pick_nth<EL, D, 32, 2>(nth, hp);
    return bs == 16 ? at_pick_nth<EL, D, 16, 0>(nth, hp) : bs == 32 ? at_pick_nth<EL, D, 32, 0>(nth, hp) : at_pick_nth<EL, D, 64, 0>(nth, hp);
}

// the kernels of one element kind and head length, in translation units of their own
#define AT_DECLARE(EL, D) AtPick at_kernel_##EL##_##D(int bs, int nth, int hp, int sfmt);
#define AT_DECLARE3(EL) AT_DECLARE(EL, 64) AT_DECLARE(EL, 128) AT_DECLARE(EL, 256)
AT_DECLARE3(GE_E2M1)
AT_DECLARE3(GE_E3M0)
AT_DECLARE3(GE_INT4)
AT_DECLARE3(AE_E2M3)
AT_DECLARE3(AE_E3M2)
#undef AT_DECLARE3
#undef AT_DECLARE
#define AT_DEFINE(EL, D) \
    AtPick at_kernel_##EL##_##D(int bs, int nth, int hp, int sfmt) { return at_pick_bs<EL, D>(bs, nth, hp, sfmt); }

}  // namespace mxk
