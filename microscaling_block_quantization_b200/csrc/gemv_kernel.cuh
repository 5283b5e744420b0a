// y = x (W^Q)^T for few rows x: matrix-vector products on 4-bit block-scaled
// weights (mx_gemv).
//
//   y[m][n] = s_T sum_b s_b(n) S_M(n) sum_{k in b} q(n, k) x[m][k]  (+ o_b sum_{k in b} x[m][k])
//
// Bound: the codes and scales are read once (K / 2 + K / B bytes a row), so a
// call costs (their bytes) / (HBM bandwidth) while m is small.  Arithmetic
// per byte is 2 codes x m multiply-adds, which the CUDA cores could not feed
// past m = 2; the matrix instruction m16n8k16 takes 16 weight rows by 8
// activation columns for one price, and the cost that remains is turning
// codes into f16 (64 conversions of a code pair per clock and SM, 128 codes;
// HBM delivers about 44 codes per clock and SM).
//
// * x as f16 pieces.  Products of codes and f16 values are exact in the
//   matrix instruction and summed in binary32.  Each 128-column chunk of a
//   token is scaled by a power of two to [2^14, 2^15): a bf16 value down to
//   2^-31 of its chunk's largest is one f16 exactly; a binary32 value is two,
//   the second scaled by 2^11: of the at most 12 bits that the first leaves it
//   holds 11, so a quarter of values lose their last bit, 2^-23 at most (a third
//   piece would be half as many matrix instructions again).  Smaller values are
//   rounded at 2^-39 (bf16) or 2^-50 of the chunk's largest.
// * Work is split into units of 16 rows x 256 columns (128 where K is no
//   multiple of 256).  A cluster of C CTAs splits K (each CTA keeps its slice of x in shared memory), its CTAs' 16
//   warps split rows and, KS ways, the slice.  Each warp streams its units
//   through a private ring of asynchronous 16-byte copies (no registers, no
//   CTA barrier), and the partial sums of a row tile meet once, through
//   distributed shared memory, in a fixed order: results do not depend on
//   timing, and no workspace is needed.
// * A warp's unit in shared memory: 16 rows of 16-byte pieces, XOR-swizzled by
//   row, so that lane (g, t) reads word t of a block's 16 bytes for rows g and
//   g + 8 without bank conflicts: the four lanes of a row share a block, hence
//   its scale, in each matrix instruction.
//
// Measured: MXFP4 65536 x 8192, one token 58.5 us (4.9 TB/s, 74% of a copy's
// rate), 16 tokens 107 us; NVFP4, one token 87 us; INT4 80 us.  Of few weights
// (4096 x 4096, 5.6 us) 4.3 us are the launch, the staging of x and the join.
#pragma once
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mma_decode.cuh"
#include "mx_internal.h"

namespace cg = cooperative_groups;

namespace mxk {

constexpr int kGvWarps = 16;
constexpr int kGvThreads = kGvWarps * 32;
constexpr int kGvPart = 8 * 20;   // floats of a tile's partial sums of 8 columns

// How a unit's scales are laid out, and how wide the unit is:
//   GM_BLOCK  blocks of 8, 16 or 32 and K a multiple of 256: 256 columns, whose
//             256 / B scales of a row are whole words (row-major or chunked);
//   GM_GROUP  blocks of 128 or 256, K a multiple of 256: 256 columns, two
//             scales (and offsets) of a row, or one;
//   GM_ANY    everything else, 128 columns: windows of aligned words around
//             the scales, a ragged last chunk, macro scales, offsets of small
//             blocks.
// The wide units' 128-byte rows halve the addresses, waits and scale reads of
// a chunk (65536 x 8192, one token: 128-column units 64 us).
enum { GM_BLOCK = 0, GM_GROUP = 1, GM_ANY = 2 };

// 128-column chunks of a unit, ring stages
__host__ __device__ constexpr int gv_chunks(int mode) { return mode == GM_ANY ? 1 : 2; }
__host__ __device__ constexpr int gv_stages(int mode) { return mode == GM_ANY ? 4 : 3; }

// scale words of a row in a stage.  GM_ANY: enough for the aligned words that
// cover 128 / B scales anywhere (BC 32: up to 4 in 2 words; 16: 8 at an even
// byte in 3; 8: 16 in 4)
template <int MODE, int BC> __host__ __device__ constexpr int gv_scale_words()
{
    return MODE == GM_BLOCK ? 64 / BC : MODE == GM_GROUP ? 1 : BC == 32 ? 2 : 4;
}
// one ring stage of a warp: codes, scales, offsets (GM_GROUP a word a row,
// GM_ANY four), macro bytes; a multiple of the code row for GM_BLOCK, GM_GROUP
template <int MODE> __host__ __device__ constexpr int gv_sc_at() { return 1024 * gv_chunks(MODE); }
template <int MODE, int BC> __host__ __device__ constexpr int gv_off_at() { return gv_sc_at<MODE>() + 64 * gv_scale_words<MODE, BC>(); }
template <int MODE, int BC> __host__ __device__ constexpr int gv_mac_at()
{
    return gv_off_at<MODE, BC>() + (MODE == GM_GROUP ? 64 : MODE == GM_ANY && BC == 32 ? 256 : 0);
}
template <int MODE, int BC> __host__ __device__ constexpr int gv_stage_bytes()
{
    return gv_mac_at<MODE, BC>() + (MODE == GM_ANY ? 64 : 0);
}

struct GvGeom {
    int xs_at, ex_at, xsum_at, part_at;  // shared-memory places
    int xc;            // x held at a time, in units of columns
    int tiles_wave;    // row tiles whose partial sums are held
    int tile_floats;   // stride of a row tile's partial sums: 16 mod 32, so that a join's reads spread over the banks
    int C, KS;
};

// Where a lane's copies of a row tile come from (32-bit: a call has fewer than
// 2^32 weights).
struct GvSource {
    uint32_t code[2];   // bytes: rows g and g + 8, 16-byte piece t of unit 0
    uint32_t sc[4];     // scales of the rows this lane copies words of
    uint32_t off[2];
    uint32_t mac;
};

template <int MODE, int BC>
__device__ __forceinline__ void gv_source(const GvParams &p, GvSource &src, uint32_t tile, int lane)
{
    constexpr int W = gv_scale_words<MODE, BC>();
    const uint32_t row0 = tile * 16, last = (uint32_t)p.N - 1, S = (uint32_t)p.S;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i < 2) {
            const uint32_t row = min(row0 + (lane >> 2) + 8 * i, last);
            src.code[i] = row * (uint32_t)(p.K >> 1) + (lane & 3) * 16;
            if (MODE == GM_ANY) src.off[i] = min(row0 + (lane + 32 * i) / 4, last) * S;
        }
        if (32 * i < 16 * W) {
            const int w = (lane + 32 * i) % W;
            const uint32_t r = min(row0 + ((lane + 32 * i) / W & 15), last);
            const uint32_t base = p.sf_chunk ? (uint32_t)sf_chunk_index(r, 0, 0) + (r >> 7) * (S >> 2) * 512u : r * S;
            src.sc[i] = base + (MODE == GM_BLOCK ? w * (p.sf_chunk ? 512u : 4u) : 0u);
        }
    }
    if (MODE == GM_GROUP) src.off[0] = min(row0 + (lane & 15), last) * S;
    if (MODE == GM_ANY) src.mac = min(row0 + (lane & 15), last) * (uint32_t)(p.K >> 7);
}

// Copy a unit (the source's tile, unit u of its columns) into a stage.
template <int MODE, int BC>
__device__ __forceinline__ void gv_issue(const GvParams &p, uint32_t stage, const GvSource &src, uint32_t u, int lane)
{
    constexpr int W = gv_scale_words<MODE, BC>();
    const int g = lane >> 2, t = lane & 3;
    if (MODE != GM_ANY) {
        // rows of eight pieces, piece b of row r at place b ^ (r & 7)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t *from = p.codes + (src.code[i] + u * 128u);
            const uint32_t to = stage + (g + 8 * i) * 128 + ((t ^ g) << 4);
            cp_async16(to, from, 16);
            cp_async16(to ^ 64u, from + 64, 16);
        }
    } else {
        const uint32_t left = (uint32_t)p.K - u * 128u;   // columns from this chunk on
        const bool in = t * 32u < left;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            cp_async16(stage + (g + 8 * i) * 64 + ((t ^ ((g >> 1) & 3)) << 4), p.codes + (in ? src.code[i] + u * 64u : 0u),
                       in ? 16 : 0);
    }
    const uint32_t sc = stage + gv_sc_at<MODE>();
    if (MODE == GM_BLOCK) {
        const uint32_t step = p.sf_chunk ? 512u * W : 4u * W;
#pragma unroll
        for (int i = 0; i < W / 2; ++i) cp_async4(sc + (lane + 32 * i) * 4, p.scales + (src.sc[i] + u * step), 4);
        return;
    }
    const uint32_t j0 = (u * (128u * gv_chunks(MODE))) >> p.log2B, n_scales = (uint32_t)p.n_scales;
    // the aligned words covering the unit's scales of every row
#pragma unroll
    for (int i = 0; i < (W + 1) / 2; ++i) {
        const int w = (lane + 32 * i) % W;
        const uint32_t at = p.sf_chunk ? src.sc[i] + ((j0 >> 2) + w) * 512u : ((src.sc[i] + j0) & ~3u) + 4 * w;
        const int nb = at + 4 <= n_scales ? 4 : at < n_scales ? (int)(n_scales - at) : 0;
        if (W >= 2 || lane < 16) cp_async4(sc + (lane + 32 * i) * 4, p.scales + (nb ? at : 0u), nb);
    }
    if (p.off && (MODE == GM_GROUP || BC == 32)) {
        // bf16 offsets, row-major whatever the scales' layout: the aligned
        // words covering the unit's (four at most with blocks of 32)
        constexpr int OW = MODE == GM_GROUP ? 1 : 4;
#pragma unroll
        for (int i = 0; i < (OW + 1) / 2; ++i) {
            const uint32_t at = ((2 * (src.off[i] + j0)) & ~3u) + 4 * (lane & (OW - 1)), n = 2 * n_scales;
            const int nb = at + 4 <= n ? 4 : at < n ? (int)(n - at) : 0;
            if (OW > 1 || lane < 16)
                cp_async4(stage + gv_off_at<MODE, BC>() + (lane + 32 * i) * 4,
                          reinterpret_cast<const uint8_t *>(p.off) + (nb ? at : 0u), nb);
        }
    }
    if (MODE == GM_ANY && p.macro && lane < 16) {
        const uint32_t at = (src.mac + u) & ~3u, n = (uint32_t)p.N * (uint32_t)(p.K >> 7);
        cp_async4(stage + gv_mac_at<MODE, BC>() + lane * 4, p.macro + at, at + 4 <= n ? 4 : (int)(n - at));
    }
}

// Scales of one row's blocks in a 128-column unit, macro scale included.  at:
// the row's first scale (row S); mat: its first macro scale.
template <int BC>
__device__ __forceinline__ void gv_scales(const GvParams &p, uint32_t stage, uint32_t at, uint32_t mat, int r,
                                          uint32_t chunk, float *s)
{
    const uint32_t sc = stage + 1024 + r * gv_scale_words<GM_ANY, BC>() * 4;
    const uint32_t j0 = (chunk * 128u) >> p.log2B;
    const int sh = (int)((p.sf_chunk ? j0 : at + j0) & 3u) * 8;
    if (BC == 32) {
        uint32_t w = __funnelshift_r(lds32(sc), lds32(sc + 4), sh);
        if (p.log2B == 6) w = __byte_perm(w, 0u, 0x1100u);
        else if (p.log2B > 6) w = __byte_perm(w, 0u, 0x0000u);
        scales4(p.sfmt, w, s);
    } else if (BC == 16) {
        const uint32_t a = lds32(sc), b = lds32(sc + 4), c = lds32(sc + 8);
        scales4(p.sfmt, __funnelshift_r(a, b, sh), s);
        scales4(p.sfmt, __funnelshift_r(b, c, sh), s + 4);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) scales4(p.sfmt, lds32(sc + 4 * i), s + 4 * i);
    }
    // blocks behind the last column: their codes are zeros, but the bytes
    // read for their scales are the next row's
    const uint32_t left = (uint32_t)p.K - chunk * 128u;
    if (left < 128u) {
#pragma unroll
        for (int i = 0; i < 128 / BC; ++i)
            if (i * BC >= left) s[i] = 0.0f;
    }
    if (p.macro) {
        const uint32_t w = lds32(stage + gv_mac_at<GM_ANY, BC>() + r * 4);
        const float m = e4m3_value((w >> (8 * ((mat + chunk) & 3u))) & 0xffu);
#pragma unroll
        for (int i = 0; i < 128 / BC; ++i) s[i] = __fmul_rn(s[i], m);
    }
}

// Eight consecutive x values, as loaded.
template <bool FP32> struct GvRaw;
template <> struct GvRaw<false> { uint32_t w[4]; };
template <> struct GvRaw<true> { float v[8]; };

__device__ __forceinline__ void gv_load8(const GvParams &p, int64_t at, bool on, GvRaw<false> &r)
{
    const uint16_t *x = static_cast<const uint16_t *>(p.x) + at;
    uint4 a = make_uint4(0u, 0u, 0u, 0u);
    if (on && p.x_vec) a = *reinterpret_cast<const uint4 *>(x);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    if (on && !p.x_vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = x[2 * i] | ((uint32_t)x[2 * i + 1] << 16);
    }
}
__device__ __forceinline__ void gv_load8(const GvParams &p, int64_t at, bool on, GvRaw<true> &r)
{
    const float *x = static_cast<const float *>(p.x) + at;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
    if (on && p.x_vec) {
        a = *reinterpret_cast<const float4 *>(x);
        b = *reinterpret_cast<const float4 *>(x + 4);
    }
    r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
    r.v[4] = b.x; r.v[5] = b.y; r.v[6] = b.z; r.v[7] = b.w;
    if (on && !p.x_vec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = x[i];
    }
}
// the bits of the largest magnitude (NaN above infinity)
__device__ __forceinline__ uint32_t gv_amax(const GvRaw<false> &r)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, r.w[i] & 0x7fff7fffu);
    return max(m & 0xffff0000u, m << 16);
}
__device__ __forceinline__ uint32_t gv_amax(const GvRaw<true> &r)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(r.v[i]) & 0x7fffffffu);
    return m;
}
__device__ __forceinline__ float2 gv_pair(const GvRaw<false> &r, int i)
{
    return make_float2(bits2f(r.w[i] << 16), bits2f(r.w[i] & 0xffff0000u));
}
__device__ __forceinline__ float2 gv_pair(const GvRaw<true> &r, int i) { return make_float2(r.v[2 * i], r.v[2 * i + 1]); }

// x chunks [c0, c0 + n) of the token group as f16 pieces in the order the
// matrix instruction's lanes read them: 16 lanes per (chunk, token), 8
// consecutive values each.
template <int BC, int NT, bool FP32, bool SPREAD, bool GROUP>
__device__ void gv_stage_x(const GvParams &p, const GvGeom &gm, uint8_t *smem, int64_t tok0, int toks, int c0, int n)
{
    const int l = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
    float *ex = reinterpret_cast<float *>(smem + gm.ex_at);
    float *xsum = reinterpret_cast<float *>(smem + gm.xsum_at);
    const int items = n * toks, q = l & 3;
    constexpr int P = FP32 ? 2 : 1, kStep = kGvThreads / 16;
    constexpr int kBatch = FP32 ? 2 : 4;   // items whose loads are in flight together
    for (int it0 = (int)(threadIdx.x >> 4); it0 - half < items; it0 += kBatch * kStep) {
        GvRaw<FP32> v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int it = it0 + j * kStep, tok = it / n;
            const int64_t k = (int64_t)(c0 + it - tok * n) * 128 + 8 * l;
            gv_load8(p, (tok0 + tok) * p.ldx + k, it < items && k < p.K, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int it = it0 + j * kStep;
            if (it - half >= items) break;   // (both halves of the warp)
            const int tok = it / n, c = it - tok * n;
            uint32_t m = gv_amax(v[j]);
#pragma unroll
            for (int d = 8; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
            float sum = 0.0f;
            if (p.off) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = gv_pair(v[j], i);
                    sum = __fadd_rn(sum, __fadd_rn(u.x, u.y));
                }
                sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 1));
                sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 2));
                if (GROUP) {
                    sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 4));
                    sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 8));
                }
            }
            if (it >= items) continue;
            const int e = f16_scale_exponent(bits2f(m));
            const float f = exp2i(e);
            uint32_t h[P][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 u = gv_pair(v[j], i);
                const float a = __fmul_rn(u.x, f), b = __fmul_rn(u.y, f);
                const __half2 hh = __floats2half2_rn(a, b);
                h[0][i] = *reinterpret_cast<const uint32_t *>(&hh);
                if (FP32) {
                    // what the first piece leaves (12 bits at most); an infinite or NaN
                    // value is all in the first piece
                    const float2 back = __half22float2(hh);
                    float ra = __fmul_rn(__fsub_rn(a, back.x), 2048.0f), rb = __fmul_rn(__fsub_rn(b, back.y), 2048.0f);
                    ra = ra == ra ? ra : 0.0f;
                    rb = rb == rb ? rb : 0.0f;
                    const __half2 h2 = __floats2half2_rn(ra, rb);
                    h[P - 1][i] = *reinterpret_cast<const uint32_t *>(&h2);
                }
            }
#pragma unroll
            for (int pc = 0; pc < P; ++pc) {
                const int col = tok * P + pc;
                uint8_t *dst = smem + gm.xs_at + (((c * 4 + (l >> 2)) * NT + (col >> 3)) << 9) + (col & 7) * 64;
                if (SPREAD) {
                    // pairs (i, i + 4), as int4_halves_spread leaves them
                    *reinterpret_cast<uint4 *>(dst + q * 16) =
                        make_uint4(__byte_perm(h[pc][0], h[pc][2], 0x5410u), __byte_perm(h[pc][0], h[pc][2], 0x7632u),
                                   __byte_perm(h[pc][1], h[pc][3], 0x5410u), __byte_perm(h[pc][1], h[pc][3], 0x7632u));
                } else if (BC == 32) {
                    *reinterpret_cast<uint4 *>(dst + q * 16) = make_uint4(h[pc][0], h[pc][1], h[pc][2], h[pc][3]);
                } else if (BC == 16) {
                    const int t = 2 * (q & 1), o = (q >> 1) * 8;
                    *reinterpret_cast<uint2 *>(dst + t * 16 + o) = make_uint2(h[pc][0], h[pc][1]);
                    *reinterpret_cast<uint2 *>(dst + t * 16 + 16 + o) = make_uint2(h[pc][2], h[pc][3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t *>(dst + i * 16 + q * 4) = h[pc][i];
                }
                if (l == 0) ex[c * 8 * NT + col] = exp2i(-e - 11 * pc);
                if (p.off && GROUP) {
                    if (l == 0) xsum[c * 8 * NT + col] = pc ? 0.0f : sum;
                } else if (p.off && q == 0) {
                    xsum[(c * 4 + (l >> 2)) * 8 * NT + col] = pc ? 0.0f : sum;
                }
            }
        }
    }
}

// INT4 words whose eight codes share a block are decoded in pairs (i, i + 4)
template <int ELEM, int BC> __host__ __device__ constexpr bool gv_spread() { return BC == 32 && (ELEM == GE_INT4 || ELEM == GE_UINT4); }

// A lane's codes of 32-block b of a row (its 16-byte piece at `at`, the lane's
// word of it included) -> four f16x2.  OFF: bytes to the row.
template <int ELEM, int BC, int OFF>
__device__ __forceinline__ void gv_codes(uint32_t at, int t, uint32_t h[4])
{
    uint32_t w;
    if (BC == 32) {
        w = lds32(at + OFF);
    } else if (BC == 16) {
        // 16-bit pieces t and t + 4: four codes of each 16-block
        w = __byte_perm(lds32(at + OFF), lds32(at + OFF + 8), (t & 1) ? 0x7632u : 0x5410u);
    } else {
        // byte t of each 8-block
        const uint4 x = lds128(at + OFF);
        const uint32_t sel = (uint32_t)t | ((uint32_t)(t + 4) << 4);
        w = __byte_perm(__byte_perm(x.x, x.y, sel), __byte_perm(x.z, x.w, sel), 0x5410u);
    }
    if constexpr (gv_spread<ELEM, BC>()) int4_halves_spread<ELEM>(w, h);
    else codes8_halves<ELEM>(w, h);
}

// One unit of a warp: acc += (16 rows x the unit's columns of codes in the
// stage) x (its chunks of the staged x).
template <int ELEM, int MODE, int BC, int NT>
__device__ __forceinline__ void gv_unit(const GvParams &p, uint32_t st, uint32_t xs, const float *ex, const float *xsum,
                                        uint32_t a_lo, uint32_t a_hi, uint32_t m_lo, uint32_t m_hi, uint32_t unit,
                                        int lane, float acc[NT][4])
{
    const int g = lane >> 2, t = lane & 3;
    constexpr int UC = gv_chunks(MODE), NS = MODE == GM_GROUP ? 1 : 128 / BC, ROW = 64 * UC;
    // the lane's word of piece 0 of row g, swizzle included; piece b of a row
    // by exclusive or
    const uint32_t place = MODE == GM_ANY ? 0u : st + g * ROW + (g << 4) + (BC == 32 ? 4 * t : BC == 16 ? 4 * (t >> 1) : 0);
    uint32_t gs_lo = 0u, gs_hi = 0u;
    if (MODE == GM_GROUP) {
        // the unit's scales of a row: one or two bytes of the word
        const uint32_t j0 = (unit * 256u) >> p.log2B;
        gs_lo = lds32(st + gv_sc_at<MODE>() + g * 4) >> (8 * ((p.sf_chunk ? j0 : a_lo + j0) & 3u));
        gs_hi = lds32(st + gv_sc_at<MODE>() + (g + 8) * 4) >> (8 * ((p.sf_chunk ? j0 : a_hi + j0) & 3u));
    }
#pragma unroll
    for (int c = 0; c < UC; ++c) {
        float s_lo[NS], s_hi[NS];
        if (MODE == GM_BLOCK) {
            constexpr int W = 32 / BC;   // words of a chunk
#pragma unroll
            for (int i = 0; i < W; ++i) {
                scales4(p.sfmt, lds32(st + gv_sc_at<MODE>() + (g * UC * W + c * W + i) * 4), s_lo + 4 * i);
                scales4(p.sfmt, lds32(st + gv_sc_at<MODE>() + ((g + 8) * UC * W + c * W + i) * 4), s_hi + 4 * i);
            }
        } else if (MODE == GM_GROUP) {
            const int sh = c && p.log2B == 7 ? 8 : 0;
            s_lo[0] = scale1(p.sfmt, (gs_lo >> sh) & 0xffu);
            s_hi[0] = scale1(p.sfmt, (gs_hi >> sh) & 0xffu);
        } else {
            gv_scales<BC>(p, st, a_lo, m_lo, g, unit, s_lo);
            gv_scales<BC>(p, st, a_hi, m_hi, g + 8, unit, s_hi);
        }
        float ca[NT][4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            // (a 128-column stage is no multiple of its rows: the piece's place
            // by itself)
            const uint32_t at = MODE == GM_ANY ? st + g * ROW + ((b ^ ((g >> 1) & 3)) << 4) + (BC == 32 ? 4 * t : BC == 16 ? 4 * (t >> 1) : 0)
                                               : place ^ ((4 * c + b) << 4);
            uint32_t hl[4], hh[4];
            gv_codes<ELEM, BC, 0>(at, t, hl);
            gv_codes<ELEM, BC, 8 * ROW>(at, t, hh);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 xb = lds128(xs + (((4 * c + b) * NT + n) << 9) + lane * 16);
                if (MODE == GM_GROUP) {
                    // one scale for the whole chunk: one sum
                    if (b == 0) mma_16816_zero(ca[n], hl[0], hh[0], hl[1], hh[1], xb.x, xb.y);
                    else mma_16816(ca[n], hl[0], hh[0], hl[1], hh[1], xb.x, xb.y);
                    mma_16816(ca[n], hl[2], hh[2], hl[3], hh[3], xb.z, xb.w);
                    continue;
                }
                const uint32_t xw[4] = {xb.x, xb.y, xb.z, xb.w};
                constexpr int PER = 32 / BC == 0 ? 1 : 32 / BC;   // scales of a 32-block
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    float d[4];
                    if (BC == 32) {
                        mma_16816_zero(d, hl[0], hh[0], hl[1], hh[1], xw[0], xw[1]);
                        mma_16816(d, hl[2], hh[2], hl[3], hh[3], xw[2], xw[3]);
                    } else if (BC == 16) {
                        mma_16816_zero(d, hl[2 * i & 3], hh[2 * i & 3], hl[(2 * i + 1) & 3], hh[(2 * i + 1) & 3], xw[2 * i & 3],
                                       xw[(2 * i + 1) & 3]);
                    } else {
                        mma_1688_zero(d, hl[i], hh[i], xw[i]);
                    }
                    const float sl = s_lo[(b * PER + i) % NS], sh = s_hi[(b * PER + i) % NS];
                    if (b == 0 && i == 0) {
                        ca[n][0] = __fmul_rn(sl, d[0]);
                        ca[n][1] = __fmul_rn(sl, d[1]);
                        ca[n][2] = __fmul_rn(sh, d[2]);
                        ca[n][3] = __fmul_rn(sh, d[3]);
                    } else {
                        ca[n][0] = fmaf(sl, d[0], ca[n][0]);
                        ca[n][1] = fmaf(sl, d[1], ca[n][1]);
                        ca[n][2] = fmaf(sh, d[2], ca[n][2]);
                        ca[n][3] = fmaf(sh, d[3], ca[n][3]);
                    }
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float2 e = *reinterpret_cast<const float2 *>(ex + (c * NT + n) * 8 + 2 * t);
            float2 f = e;
            if (MODE == GM_GROUP) {
                // the scale with the power of two: exact while in range
                f = make_float2(__fmul_rn(e.x, s_hi[0]), __fmul_rn(e.y, s_hi[0]));
                e = make_float2(__fmul_rn(e.x, s_lo[0]), __fmul_rn(e.y, s_lo[0]));
            }
            acc[n][0] = fmaf(e.x, ca[n][0], acc[n][0]);
            acc[n][1] = fmaf(e.y, ca[n][1], acc[n][1]);
            acc[n][2] = fmaf(f.x, ca[n][2], acc[n][2]);
            acc[n][3] = fmaf(f.y, ca[n][3], acc[n][3]);
        }
    }
    if (!p.off || MODE == GM_BLOCK || (MODE == GM_ANY && BC != 32)) return;
    // block offsets times the sums of x over the blocks (GM_GROUP: over the
    // chunks; a block of 256 has one offset for both)
    const uint32_t ob = st + gv_off_at<MODE, BC>(), row = MODE == GM_GROUP ? 4u : 16u;
    const uint32_t j0 = (unit * (128u * UC)) >> p.log2B;
    const uint32_t ol = ob + g * row + 2 * ((a_lo + j0) & 1u), oh = ob + (g + 8) * row + 2 * ((a_hi + j0) & 1u);
#pragma unroll
    for (int b = 0; b < (MODE == GM_GROUP ? UC : 4); ++b) {
        if (MODE == GM_ANY && unit * 128u + b * 32u >= (uint32_t)p.K) break;
        const uint32_t j = ((MODE == GM_GROUP ? b * 128u : b * 32u) >> p.log2B) * 2u;
        const float fl = bits2f(lds16(ol + j) << 16), fh = bits2f(lds16(oh + j) << 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 v = *reinterpret_cast<const float2 *>(xsum + (b * NT + n) * 8 + 2 * t);
            acc[n][0] = fmaf(fl, v.x, acc[n][0]);
            acc[n][1] = fmaf(fl, v.y, acc[n][1]);
            acc[n][2] = fmaf(fh, v.x, acc[n][2]);
            acc[n][3] = fmaf(fh, v.y, acc[n][3]);
        }
    }
}

template <int ELEM, int MODE, int BC, int NT>
__global__ void __launch_bounds__(kGvThreads, 1) k_gemv(const __grid_constant__ GvParams p,
                                                        const __grid_constant__ GvGeom gm)
{
    extern __shared__ __align__(128) uint8_t smem[];
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int SB = gv_stage_bytes<MODE, BC>(), UC = gv_chunks(MODE), STAGES = gv_stages(MODE);
    constexpr bool SPREAD = gv_spread<ELEM, BC>();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int rank = (int)(blockIdx.x % gm.C);
    const uint32_t cl = blockIdx.x / gm.C, ncl = gridDim.x / gm.C;
    const int64_t tok0 = (int64_t)blockIdx.y * p.group;
    const int toks = (int)min((int64_t)p.group, p.M - tok0);
    const int P = p.x_fp32 ? 2 : 1;
    const uint32_t tiles = (uint32_t)((p.N + 15) >> 4);
    const int mine = cl < tiles ? (int)((tiles - cl + ncl - 1) / ncl) : 0;   // tiles cl, cl + ncl, ...
    const int c_lo = (int)((int64_t)p.units * rank / gm.C), c_hi = (int)((int64_t)p.units * (rank + 1) / gm.C);
    const int ks = warp % gm.KS, tg = warp / gm.KS, TG = kGvWarps / gm.KS;
    const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t ring = sbase + warp * STAGES * SB, ring_end = ring + STAGES * SB;
    float *part = reinterpret_cast<float *>(smem + gm.part_at);
    const float *ex = reinterpret_cast<const float *>(smem + gm.ex_at);
    const float *xsum = reinterpret_cast<const float *>(smem + gm.xsum_at);
    const bool resident = c_hi - c_lo <= gm.xc;

    pdl_trigger();
    pdl_wait();

    for (int w0 = 0; w0 < mine; w0 += gm.tiles_wave) {
        const int wt = min(gm.tiles_wave, mine - w0);
        // (a CTA whose share of K is empty makes one pass that stores zeros)
        for (int s0 = c_lo; s0 == c_lo || s0 < c_hi; s0 += gm.xc) {
            const int sn = min(gm.xc, c_hi - s0);
            const int a = s0 + sn * ks / gm.KS, nc = s0 + sn * (ks + 1) / gm.KS - a;
            const int nt_mine = tg < wt ? (wt - tg + TG - 1) / TG : 0;
            int left = nt_mine * nc;            // units still to copy
            int it = tg, ic = 0;                // the next one
            uint32_t st_w = ring;
            GvSource src;
            auto issue = [&]() {
                if (left > 0) {
                    if (ic == 0) gv_source<MODE, BC>(p, src, cl + (uint32_t)(w0 + it) * ncl, lane);
                    gv_issue<MODE, BC>(p, st_w, src, a + ic, lane);
                    if (++ic == nc) { ic = 0; it += TG; }
                    --left;
                }
                st_w = st_w + SB == ring_end ? ring : st_w + SB;
                cp_async_commit();
            };
#pragma unroll
            for (int i = 0; i < STAGES - 1; ++i) issue();
            if (!resident || w0 == 0) {
                if (s0 != c_lo || w0 != 0) __syncthreads();   // the last slice of x is no longer read
                if (p.x_fp32) gv_stage_x<BC, NT, true, SPREAD, MODE == GM_GROUP>(p, gm, smem, tok0, toks, s0 * UC, sn * UC);
                else gv_stage_x<BC, NT, false, SPREAD, MODE == GM_GROUP>(p, gm, smem, tok0, toks, s0 * UC, sn * UC);
                __syncthreads();
            }
            uint32_t st = ring;
            for (int lt = tg; lt < wt; lt += TG) {   // tiles within the wave
                const uint32_t tile = cl + (uint32_t)(w0 + lt) * ncl;
                const uint32_t r_lo = min(tile * 16 + g, (uint32_t)p.N - 1), r_hi = min(tile * 16 + g + 8, (uint32_t)p.N - 1);
                const uint32_t a_lo = r_lo * (uint32_t)p.S, a_hi = r_hi * (uint32_t)p.S;
                const uint32_t m_lo = r_lo * (uint32_t)(p.K >> 7), m_hi = r_hi * (uint32_t)(p.K >> 7);
                float acc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
                int cx = a - s0;
                for (int c = 0; c < nc; ++c, ++cx) {
                    cp_async_wait<STAGES - 2>();
                    __syncwarp();   // every lane's copies of this unit are in, and the last unit is read
                    issue();
                    gv_unit<ELEM, MODE, BC, NT>(p, st, sbase + gm.xs_at + cx * UC * (NT << 11), ex + cx * UC * NT * 8,
                                                xsum + cx * UC * NT * (MODE == GM_GROUP ? 8 : 32), a_lo, a_hi, m_lo, m_hi, a + c, lane, acc);
                    st = st + SB == ring_end ? ring : st + SB;
                }
                // this warp's partial sums of the tile: 16 rows of each
                // column, columns 20 floats apart (no bank conflicts)
                float *pt = part + lt * gm.tile_floats + ks * kGvPart * NT;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float *q = pt + (n * 8 + 2 * t + (i & 1)) * 20 + g + (i >> 1) * 8;
                        *q = s0 != c_lo ? *q + acc[n][i] : acc[n][i];
                    }
                }
            }
            cp_async_wait<0>();
            __syncwarp();
        }
        // join: a thread adds four rows of one token over the cluster's CTAs
        // and their K splits, in order; each CTA joins its share
        if (gm.C > 1) cluster.sync();
        else __syncthreads();
        const float sT = p.ts ? *p.ts : 1.0f;
        const int items = wt * 4 * toks;
        for (int e = rank * kGvThreads + (int)threadIdx.x; e < items; e += gm.C * kGvThreads) {
            const int tok = e / (wt * 4), r = e - tok * wt * 4;
            const int at = (r >> 2) * gm.tile_floats + tok * P * 20 + (r & 3) * 4;
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int c = 0; c < gm.C; ++c) {
                const float *q = (gm.C > 1 ? cluster.map_shared_rank(part, c) : part) + at;
#pragma unroll 4
                for (int i = 0; i < gm.KS; ++i, q += kGvPart * NT) {
                    float4 v = *reinterpret_cast<const float4 *>(q);
                    if (P == 2) {
                        const float4 u = *reinterpret_cast<const float4 *>(q + 20);
                        v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                    }
                    sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
                }
            }
            const uint32_t row = (cl + (uint32_t)(w0 + (r >> 2)) * ncl) * 16 + (r & 3) * 4;
            const float o[4] = {sum.x, sum.y, sum.z, sum.w};
            const int64_t y = (tok0 + tok) * p.ldy + row;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (row + i >= (uint32_t)p.N) break;
                const float v = p.ts ? __fmul_rn(o[i], sT) : o[i];
                if (p.y_fp32) static_cast<float *>(p.y)[y + i] = v;
                else static_cast<__nv_bfloat16 *>(p.y)[y + i] = __float2bfloat16_rn(v);
            }
        }
        if (gm.C > 1) cluster.sync();                            // no CTA leaves or overwrites sums still read
        else if (w0 + wt < mine) __syncthreads();
    }
}

typedef void (*GvKernel)(const GvParams, const GvGeom);

template <int ELEM, int MODE, int BC> GvKernel gv_pick_nt(int nt)
{
    return nt == 1 ? k_gemv<ELEM, MODE, BC, 1> : k_gemv<ELEM, MODE, BC, 2>;
}
template <int ELEM> GvKernel gv_pick_mode(int mode, int bc, int nt)
{
    if (mode == GM_GROUP) return gv_pick_nt<ELEM, GM_GROUP, 32>(nt);
    if (mode == GM_BLOCK)
        return bc == 32 ? gv_pick_nt<ELEM, GM_BLOCK, 32>(nt) : bc == 16 ? gv_pick_nt<ELEM, GM_BLOCK, 16>(nt)
                                                                        : gv_pick_nt<ELEM, GM_BLOCK, 8>(nt);
    return bc == 32 ? gv_pick_nt<ELEM, GM_ANY, 32>(nt) : bc == 16 ? gv_pick_nt<ELEM, GM_ANY, 16>(nt)
                                                                  : gv_pick_nt<ELEM, GM_ANY, 8>(nt);
}

// the kernels of one element kind, in translation units of their own
GvKernel gv_kernel_e2m1(int mode, int bc, int nt);
GvKernel gv_kernel_e3m0(int mode, int bc, int nt);
GvKernel gv_kernel_int4(int mode, int bc, int nt);
GvKernel gv_kernel_uint4(int mode, int bc, int nt);

}  // namespace mxk
