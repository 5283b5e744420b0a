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
//   2^-31 of its chunk's largest is one f16 exactly; a binary32 value is the
//   sum of two (11 + 12 bits) exactly, the second scaled by 2^11.  Smaller
//   values are rounded at 2^-39 (bf16) or 2^-50 of the chunk's largest.
// * Work is split into units of 16 rows x 128 columns.  A cluster of C CTAs
//   splits K (each CTA keeps its slice of x in shared memory), its CTAs' 16
//   warps split rows and, KS ways, the slice.  Each warp streams its units
//   through a private ring of asynchronous 16-byte copies (no registers, no
//   CTA barrier), and the partial sums of a row tile meet once, through
//   distributed shared memory, in a fixed order: results do not depend on
//   timing, and no workspace is needed.
// * A warp's unit in shared memory: 16 rows x 64 bytes, 16-byte pieces
//   XOR-swizzled by row pair, so that lane (g, t) reads word t of a block's
//   16 bytes for rows g and g + 8 without bank conflicts: the four lanes of
//   a row share a block, hence its scale, in each matrix instruction.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "mma_decode.cuh"
#include "mx_internal.h"

namespace cg = cooperative_groups;

namespace mxk {

constexpr int kGvWarps = 16;
constexpr int kGvThreads = kGvWarps * 32;
constexpr int kGvStages = 4;

// scale words of a row in a unit: enough for the aligned words that cover
// its 128 / B scales (BC 32: up to 4 scales anywhere in 2 words; 16: 8 scales
// at an even byte in 3; 8: 16 scales in 4)
template <int BC> constexpr int kGvScaleWords = BC == 32 ? 2 : 4;

struct GvGeom {
    int stage_bytes;   // one ring stage of a warp
    int off_at, mac_at;  // offsets and macro bytes in a stage (0: absent)
    int xs_at, ex_at, xsum_at, part_at;  // shared-memory places
    int xc;            // chunks of x held at a time
    int tiles_wave;    // row tiles whose partial sums are held
    int C, KS;
};

__device__ __forceinline__ float gv_load(const GvParams &p, int64_t i)
{
    return p.x_fp32 ? static_cast<const float *>(p.x)[i]
                    : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.x)[i]);
}


// Copy unit (tile, chunk) into a stage.
template <int BC>
__device__ __forceinline__ void gv_issue(const GvParams &p, const GvGeom &gm, uint32_t stage, int64_t tile, int chunk,
                                         int lane)
{
    const int g = lane >> 2, t = lane & 3;
    const int bytes = (int64_t)chunk * 128 + t * 32 < p.K ? 16 : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = g + 8 * i;
        const int64_t row = min(tile * 16 + r, p.N - 1);
        const uint8_t *src = p.codes + row * (p.K >> 1) + (bytes ? (int64_t)chunk * 64 + t * 16 : 0);
        cp_async16(stage + r * 64 + ((t ^ ((r >> 1) & 3)) << 4), src, bytes);
    }
    // scales: aligned words covering the chunk's scales of every row
    constexpr int W = kGvScaleWords<BC>;
    const uint32_t sc = stage + 1024;
#pragma unroll
    for (int i = lane; i < 16 * W; i += 32) {
        const int r = i / W, w = i % W;
        const int64_t row = min(tile * 16 + r, p.N - 1);
        const int64_t j0 = ((int64_t)chunk * 128) >> p.log2B;
        int64_t at;
        if (p.sf_chunk) at = sf_chunk_index(row, (j0 & ~(int64_t)3) + 4 * w, p.S);
        else at = ((row * p.S + j0) & ~(int64_t)3) + 4 * w;
        const bool in = p.sf_chunk ? (j0 & ~(int64_t)3) + 4 * w < p.S : at < p.n_scales;
        const int nb = in ? (int)min((int64_t)4, p.n_scales - at) : 0;
        cp_async4(sc + (r * W + w) * 4, p.scales + (in ? at : 0), nb);
    }
    if (BC == 32 && p.off) {
        // bf16 offsets, row-major whatever the scales' layout: the aligned
        // words covering the unit's, at most four
        const uint8_t *ob = reinterpret_cast<const uint8_t *>(p.off);
#pragma unroll
        for (int i = lane; i < 64; i += 32) {
            const int r = i >> 2, w = i & 3;
            const int64_t row = min(tile * 16 + r, p.N - 1);
            const int64_t j0 = ((int64_t)chunk * 128) >> p.log2B;
            const int64_t at = ((2 * (row * p.S + j0)) & ~(int64_t)3) + 4 * w;
            const bool in = at < 2 * p.n_scales;
            const int nb = in ? (int)min((int64_t)4, 2 * p.n_scales - at) : 0;
            cp_async4(stage + gm.off_at + (r * 4 + w) * 4, ob + (in ? at : 0), nb);
        }
    }
    if (p.macro && lane < 16) {
        const int64_t row = min(tile * 16 + lane, p.N - 1);
        const int64_t at = (row * (p.K >> 7) + chunk) & ~(int64_t)3, n = p.N * (p.K >> 7);
        cp_async4(stage + gm.mac_at + lane * 4, p.macro + at, (int)min((int64_t)4, n - at));
    }
}

// Scales of one row's blocks in a unit, macro scale included.
template <int BC>
__device__ __forceinline__ void gv_scales(const GvParams &p, const GvGeom &gm, uint32_t stage, int64_t row, int r,
                                          int chunk, float *s)
{
    constexpr int W = kGvScaleWords<BC>;
    const uint32_t sc = stage + 1024 + r * W * 4;
    const int64_t j0 = ((int64_t)chunk * 128) >> p.log2B;
    const int sh = (int)((p.sf_chunk ? j0 : row * p.S + j0) & 3) * 8;
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
    const int64_t left = p.K - (int64_t)chunk * 128;
    if (left < 128) {
#pragma unroll
        for (int i = 0; i < 128 / BC; ++i)
            if (i * BC >= left) s[i] = 0.0f;
    }
    if (p.macro) {
        const uint32_t w = lds32(stage + gm.mac_at + r * 4);
        const float m = e4m3_value((w >> (8 * (int)((row * (p.K >> 7) + chunk) & 3))) & 0xffu);
#pragma unroll
        for (int i = 0; i < 128 / BC; ++i) s[i] = __fmul_rn(s[i], m);
    }
}

// x chunks [c0, c0 + n) of the token group as f16 pieces in the order the
// matrix instruction's lanes read them: 16 lanes per (chunk, token), 8
// consecutive values each.
template <int BC, int NT>
__device__ void gv_stage_x(const GvParams &p, const GvGeom &gm, uint8_t *smem, int64_t tok0, int toks, int c0, int n)
{
    const int l = threadIdx.x & 15;
    float *ex = reinterpret_cast<float *>(smem + gm.ex_at);
    float *xsum = reinterpret_cast<float *>(smem + gm.xsum_at);
    const int items = n * toks;
    for (int it0 = 0; it0 < items; it0 += kGvThreads / 16) {
        const int it = it0 + (int)(threadIdx.x >> 4);
        const bool on = it < items;
        const int c = on ? it / toks : 0, tok = on ? it - c * toks : 0;
        const int64_t k = (int64_t)(c0 + c) * 128 + 8 * l;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (on && k < p.K) {
            const int64_t at = (tok0 + tok) * p.ldx + k;
            if (p.x_vec) {
                if (p.x_fp32) {
                    const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + at);
                    const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + at + 4);
                    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
                } else {
                    const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.x) + at);
                    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[2 * i] = bits2f(w[i] << 16);
                        v[2 * i + 1] = bits2f(w[i] & 0xffff0000u);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = gv_load(p, at + i);
            }
        }
        uint32_t m = 0;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
            sum = __fadd_rn(sum, v[i]);
        }
#pragma unroll
        for (int d = 8; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (p.off) {
            sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 1));
            sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 2));
        }
        if (!on) continue;
        const int e = f16_scale_exponent(bits2f(m));
        const float f = exp2i(e);
        uint32_t h1[4], h2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = __fmul_rn(v[2 * i], f), b = __fmul_rn(v[2 * i + 1], f);
            const __half ha = __float2half_rn(a), hb = __float2half_rn(b);
            h1[i] = (uint32_t)__half_as_ushort(ha) | ((uint32_t)__half_as_ushort(hb) << 16);
            // what the first piece leaves of a binary32 value, exact; an
            // infinite or NaN value is all in the first piece
            float ra = __fmul_rn(__fsub_rn(a, __half2float(ha)), 2048.0f);
            float rb = __fmul_rn(__fsub_rn(b, __half2float(hb)), 2048.0f);
            ra = ra == ra ? ra : 0.0f;
            rb = rb == rb ? rb : 0.0f;
            h2[i] = (uint32_t)__half_as_ushort(__float2half_rn(ra)) |
                    ((uint32_t)__half_as_ushort(__float2half_rn(rb)) << 16);
        }
        const int P = p.x_fp32 ? 2 : 1;
        const int q = l & 3;
        for (int pc = 0; pc < P; ++pc) {
            const int col = tok * P + pc;
            const uint32_t *h = pc ? h2 : h1;
            uint8_t *dst = smem + gm.xs_at + (((c * 4 + (l >> 2)) * NT + (col >> 3)) << 9) + (col & 7) * 64;
            if (BC == 32) {
                *reinterpret_cast<uint4 *>(dst + q * 16) = make_uint4(h[0], h[1], h[2], h[3]);
            } else if (BC == 16) {
                const int t = 2 * (q & 1), o = (q >> 1) * 8;
                *reinterpret_cast<uint2 *>(dst + t * 16 + o) = make_uint2(h[0], h[1]);
                *reinterpret_cast<uint2 *>(dst + t * 16 + 16 + o) = make_uint2(h[2], h[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t *>(dst + i * 16 + q * 4) = h[i];
            }
            if (l == 0) ex[c * 8 * NT + col] = exp2i(-e - 11 * pc);
            if (p.off && q == 0) xsum[(c * 4 + (l >> 2)) * 8 * NT + col] = pc ? 0.0f : sum;
        }
    }
}

template <int ELEM, int BC, int NT>
__global__ void __launch_bounds__(kGvThreads, 1) k_gemv(const GvParams p, const GvGeom gm)
{
    extern __shared__ __align__(128) uint8_t smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int rank = (int)(blockIdx.x % gm.C);
    const int64_t cl = blockIdx.x / gm.C, ncl = gridDim.x / gm.C;
    const int64_t tok0 = (int64_t)blockIdx.y * p.group;
    const int toks = (int)min((int64_t)p.group, p.M - tok0);
    const int P = p.x_fp32 ? 2 : 1;
    const int64_t tiles = (p.N + 15) >> 4;
    const int64_t mine = cl < tiles ? (tiles - cl + ncl - 1) / ncl : 0;   // tiles cl, cl + ncl, ...
    const int c_lo = (int)((int64_t)p.chunks * rank / gm.C), c_hi = (int)((int64_t)p.chunks * (rank + 1) / gm.C);
    const int ks = warp % gm.KS, tg = warp / gm.KS, TG = kGvWarps / gm.KS;
    const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t ring = sbase + warp * kGvStages * gm.stage_bytes;
    float *part = reinterpret_cast<float *>(smem + gm.part_at);
    const float *ex = reinterpret_cast<const float *>(smem + gm.ex_at);
    const float *xsum = reinterpret_cast<const float *>(smem + gm.xsum_at);
    const bool resident = c_hi - c_lo <= gm.xc;

    pdl_trigger();
    pdl_wait();

    for (int64_t w0 = 0; w0 < mine; w0 += gm.tiles_wave) {
        const int wt = (int)min((int64_t)gm.tiles_wave, mine - w0);
        // (a CTA whose share of K is empty makes one pass that stores zeros)
        for (int s0 = c_lo; s0 == c_lo || s0 < c_hi; s0 += gm.xc) {
            const int sn = min(gm.xc, c_hi - s0);
            const int a = s0 + sn * ks / gm.KS, nc = s0 + sn * (ks + 1) / gm.KS - a;
            const int nt_mine = tg < wt ? (wt - tg + TG - 1) / TG : 0;
            const int units = nt_mine * nc;
            int it = tg, ic = 0, iu = 0;   // next unit to copy
            auto issue = [&]() {
                if (iu < units) {
                    gv_issue<BC>(p, gm, ring + (iu % kGvStages) * gm.stage_bytes, cl + (w0 + it) * ncl, a + ic, lane);
                    if (++ic == nc) { ic = 0; it += TG; }
                }
                ++iu;
                cp_async_commit();
            };
#pragma unroll
            for (int i = 0; i < kGvStages - 1; ++i) issue();
            if (!resident || w0 == 0) {
                if (s0 != c_lo || w0 != 0) __syncthreads();   // the last slice of x is no longer read
                gv_stage_x<BC, NT>(p, gm, smem, tok0, toks, s0, sn);
                __syncthreads();
            }
            int u = 0;
            for (int jt = 0; jt < nt_mine; ++jt) {
                const int lt = tg + jt * TG;   // tile within the wave
                const int64_t tile = cl + (w0 + lt) * ncl;
                float acc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
                for (int c = 0; c < nc; ++c, ++u) {
                    cp_async_wait<kGvStages - 2>();
                    __syncwarp();   // every lane's copies of unit u are in, and unit u - 1 is read
                    issue();
                    const uint32_t st = ring + (u % kGvStages) * gm.stage_bytes;
                    const int chunk = a + c, cx = chunk - s0;
                    float s_lo[128 / BC], s_hi[128 / BC];
                    const int64_t r_lo = min(tile * 16 + g, p.N - 1), r_hi = min(tile * 16 + g + 8, p.N - 1);
                    gv_scales<BC>(p, gm, st, r_lo, g, chunk, s_lo);
                    gv_scales<BC>(p, gm, st, r_hi, g + 8, chunk, s_hi);
                    float ca[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) ca[n][i] = 0.0f;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint32_t pl = st + g * 64 + ((b ^ ((g >> 1) & 3)) << 4);
                        const uint32_t ph = pl + 512;
                        uint32_t wl, wh;
                        if (BC == 32) {
                            wl = lds32(pl + 4 * t);
                            wh = lds32(ph + 4 * t);
                        } else if (BC == 16) {
                            // 16-bit pieces t and t + 4: four codes of each 16-block
                            const uint32_t sel = (t & 1) ? 0x7632u : 0x5410u;
                            wl = __byte_perm(lds32(pl + 4 * (t >> 1)), lds32(pl + 8 + 4 * (t >> 1)), sel);
                            wh = __byte_perm(lds32(ph + 4 * (t >> 1)), lds32(ph + 8 + 4 * (t >> 1)), sel);
                        } else {
                            // byte t of each 8-block
                            const uint4 x0 = lds128(pl), x1 = lds128(ph);
                            const uint32_t sel = (uint32_t)t | ((uint32_t)(t + 4) << 4);
                            wl = __byte_perm(__byte_perm(x0.x, x0.y, sel), __byte_perm(x0.z, x0.w, sel), 0x5410u);
                            wh = __byte_perm(__byte_perm(x1.x, x1.y, sel), __byte_perm(x1.z, x1.w, sel), 0x5410u);
                        }
                        uint32_t hl[4], hh[4];
                        codes8_halves<ELEM>(wl, hl);
                        codes8_halves<ELEM>(wh, hh);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4 xb = lds128(sbase + gm.xs_at + (((cx * 4 + b) * NT + n) << 9) + lane * 16);
                            if (BC == 32) {
                                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                mma_16816(d, hl[0], hh[0], hl[1], hh[1], xb.x, xb.y);
                                mma_16816(d, hl[2], hh[2], hl[3], hh[3], xb.z, xb.w);
                                ca[n][0] = fmaf(s_lo[b], d[0], ca[n][0]);
                                ca[n][1] = fmaf(s_lo[b], d[1], ca[n][1]);
                                ca[n][2] = fmaf(s_hi[b], d[2], ca[n][2]);
                                ca[n][3] = fmaf(s_hi[b], d[3], ca[n][3]);
                            } else if (BC == 16) {
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                    mma_16816(d, hl[2 * i], hh[2 * i], hl[2 * i + 1], hh[2 * i + 1],
                                              i ? xb.z : xb.x, i ? xb.w : xb.y);
                                    ca[n][0] = fmaf(s_lo[2 * b + i], d[0], ca[n][0]);
                                    ca[n][1] = fmaf(s_lo[2 * b + i], d[1], ca[n][1]);
                                    ca[n][2] = fmaf(s_hi[2 * b + i], d[2], ca[n][2]);
                                    ca[n][3] = fmaf(s_hi[2 * b + i], d[3], ca[n][3]);
                                }
                            } else {
                                const uint32_t xw[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                    mma_1688(d, hl[i], hh[i], xw[i]);
                                    ca[n][0] = fmaf(s_lo[4 * b + i], d[0], ca[n][0]);
                                    ca[n][1] = fmaf(s_lo[4 * b + i], d[1], ca[n][1]);
                                    ca[n][2] = fmaf(s_hi[4 * b + i], d[2], ca[n][2]);
                                    ca[n][3] = fmaf(s_hi[4 * b + i], d[3], ca[n][3]);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float2 e = *reinterpret_cast<const float2 *>(ex + (cx * NT + n) * 8 + 2 * t);
                        acc[n][0] = fmaf(e.x, ca[n][0], acc[n][0]);
                        acc[n][1] = fmaf(e.y, ca[n][1], acc[n][1]);
                        acc[n][2] = fmaf(e.x, ca[n][2], acc[n][2]);
                        acc[n][3] = fmaf(e.y, ca[n][3], acc[n][3]);
                    }
                    if (BC == 32 && p.off) {
                        const int64_t j0 = ((int64_t)chunk * 128) >> p.log2B;
                        const int ol = (int)((r_lo * p.S + j0) & 1);
                        const int oh = (int)((r_hi * p.S + j0) & 1);
                        const uint8_t *ob = smem + (st - sbase) + gm.off_at;
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            if ((int64_t)chunk * 128 + b * 32 >= p.K) break;
                            const int j = (b * 32) >> p.log2B;
                            const float fl = bits2f((uint32_t)*reinterpret_cast<const uint16_t *>(ob + g * 16 + 2 * (ol + j)) << 16);
                            const float fh = bits2f((uint32_t)*reinterpret_cast<const uint16_t *>(ob + g * 16 + 128 + 2 * (oh + j)) << 16);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const float2 xs = *reinterpret_cast<const float2 *>(xsum + ((cx * 4 + b) * NT + n) * 8 + 2 * t);
                                acc[n][0] = fmaf(fl, xs.x, acc[n][0]);
                                acc[n][1] = fmaf(fl, xs.y, acc[n][1]);
                                acc[n][2] = fmaf(fh, xs.x, acc[n][2]);
                                acc[n][3] = fmaf(fh, xs.y, acc[n][3]);
                            }
                        }
                    }
                }
                // this warp's partial sums of the tile: [row][virtual token]
                float *pt = part + (size_t)(lt * gm.KS + ks) * 16 * 8 * NT;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float2 *lo = reinterpret_cast<float2 *>(pt + (g * NT + n) * 8 + 2 * t);
                    float2 *hi = reinterpret_cast<float2 *>(pt + ((g + 8) * NT + n) * 8 + 2 * t);
                    float2 a0 = make_float2(acc[n][0], acc[n][1]), a1 = make_float2(acc[n][2], acc[n][3]);
                    if (s0 != c_lo) {
                        a0.x += lo->x; a0.y += lo->y;
                        a1.x += hi->x; a1.y += hi->y;
                    }
                    *lo = a0;
                    *hi = a1;
                }
            }
            cp_async_wait<0>();
            __syncwarp();
        }
        // join: each CTA of the cluster adds its share of the outputs over
        // the cluster's CTAs and their K splits, in order
        cluster.sync();
        const int outs = wt * 16 * toks;
        const float sT = p.ts ? *p.ts : 1.0f;
        for (int e = rank * kGvThreads + (int)threadIdx.x; e < outs; e += gm.C * kGvThreads) {
            const int tok = e / (wt * 16), r = e - tok * wt * 16;
            const int64_t row = (cl + (w0 + (r >> 4)) * ncl) * 16 + (r & 15);
            if (row >= p.N) continue;
            float sum = 0.0f;
            for (int c = 0; c < gm.C; ++c) {
                const float *rp = cluster.map_shared_rank(part, c);
                for (int k = 0; k < gm.KS; ++k) {
                    const float *q = rp + ((size_t)((r >> 4) * gm.KS + k) * 16 + (r & 15)) * 8 * NT + tok * P;
                    sum += P == 2 ? q[0] + q[1] : q[0];
                }
            }
            if (p.ts) sum = __fmul_rn(sum, sT);
            const int64_t at = (tok0 + tok) * p.ldy + row;
            if (p.y_fp32) static_cast<float *>(p.y)[at] = sum;
            else static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(sum);
        }
        cluster.sync();
    }
}

namespace {

typedef void (*GvKernel)(const GvParams, const GvGeom);

template <int ELEM, int BC> GvKernel gv_pick(int nt) { return nt == 1 ? k_gemv<ELEM, BC, 1> : k_gemv<ELEM, BC, 2>; }
template <int ELEM> GvKernel gv_pick(int bc, int nt)
{
    return bc == 32 ? gv_pick<ELEM, 32>(nt) : bc == 16 ? gv_pick<ELEM, 16>(nt) : gv_pick<ELEM, 8>(nt);
}
GvKernel gv_pick(int elem, int bc, int nt)
{
    switch (elem) {
    case GE_E2M1: return gv_pick<GE_E2M1>(bc, nt);
    case GE_E3M0: return gv_pick<GE_E3M0>(bc, nt);
    case GE_INT4: return gv_pick<GE_INT4>(bc, nt);
    default: return gv_pick<GE_UINT4>(bc, nt);
    }
}

constexpr int kGvSmem = 227 * 1024;

// Clusters of C one-CTA-per-SM CTAs that the current device holds at once
// (a GPC with a number of SMs that C does not divide leaves some out).
int resident_clusters(int C)
{
    static std::mutex mu;
    static int known[64][4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    const int i = C == 1 ? 0 : C == 2 ? 1 : C == 4 ? 2 : 3;
    std::lock_guard<std::mutex> lock(mu);
    int *slot = dev < 64 ? &known[dev][i] : nullptr;
    if (slot && *slot) return *slot;
    GvKernel k = gv_pick(GE_E2M1, 32, 1);
    int n = 0;
    if (!raise_smem_limit(reinterpret_cast<const void *>(k), kGvSmem)) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(C);
        cfg.blockDim = dim3(kGvThreads);
        cfg.dynamicSmemBytes = kGvSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = C;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) n = 0;
    }
    if (n < 1) n = device_sm_count() / C > 0 ? device_sm_count() / C : 1;
    if (slot) *slot = n;
    return n;
}

}  // namespace

int launch_gemv(GvParams p, cudaStream_t st)
{
    const int bc = p.log2B >= 5 ? 32 : p.log2B == 4 ? 16 : 8;
    const int P = p.x_fp32 ? 2 : 1;
    const int nt = p.M * P > 8 ? 2 : 1;
    p.group = 8 * nt / P;
    p.chunks = (int)((p.K + 127) / 128);
    const int64_t tiles = (p.N + 15) / 16;

    GvGeom gm = {};
    gm.stage_bytes = 1024 + 16 * 4 * (bc == 32 ? 2 : 4);
    if (p.off) { gm.off_at = gm.stage_bytes; gm.stage_bytes += 256; }
    if (p.macro) { gm.mac_at = gm.stage_bytes; gm.stage_bytes += 64; }
    const int ring = kGvWarps * kGvStages * gm.stage_bytes;
    const int per_chunk = 2048 * nt + 32 * nt + (p.off ? 128 * nt : 0);

    // the split of K over a cluster (C) and over a CTA's warps (KS): least
    // units on the busiest warp, a larger cluster where x would not stay
    GvKernel k = gv_pick(p.elem, bc, nt);
    if (raise_smem_limit(reinterpret_cast<const void *>(k), kGvSmem)) return 1;
    int64_t best = -1;
    for (int C = 1; C <= 8; C *= 2) {
        const int cpc = (p.chunks + C - 1) / C;
        const int64_t lim = resident_clusters(C);
        const int64_t ncl = tiles < lim ? tiles : lim;
        const int64_t per = (tiles + ncl - 1) / ncl;
        for (int KS = 1; KS <= kGvWarps; KS *= 2) {
            const int64_t tg = kGvWarps / KS;
            const int64_t units = ((per + tg - 1) / tg) * ((cpc + KS - 1) / KS);
            const bool fits = (int64_t)cpc * per_chunk <= 64 * 1024;
            const int64_t cost = units * 8 + (fits ? 0 : units * 8 + 64) + C + KS / 4;
            if (best < 0 || cost < best) {
                best = cost;
                gm.C = C;
                gm.KS = KS;
                gm.xc = cpc;
            }
        }
    }
    const int xc_max = 64 * 1024 / per_chunk;
    if (gm.xc > xc_max) gm.xc = xc_max;
    if (gm.xc < 1) gm.xc = 1;
    int at = ring;
    gm.xs_at = at; at += gm.xc * 2048 * nt;
    gm.ex_at = at; at += gm.xc * 32 * nt;
    gm.xsum_at = at; at += p.off ? gm.xc * 128 * nt : 0;
    gm.part_at = at;
    const int64_t ncl_max = resident_clusters(gm.C);
    const int64_t ncl = tiles < ncl_max ? tiles : ncl_max;
    const int64_t per = (tiles + ncl - 1) / ncl;
    const int tile_bytes = gm.KS * 512 * nt;
    const int64_t room = (kGvSmem - at) / tile_bytes;
    gm.tiles_wave = (int)(per < room ? per : room);
    const int smem = at + gm.tiles_wave * tile_bytes;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ncl * gm.C), (unsigned)((p.M + p.group - 1) / p.group));
    cfg.blockDim = dim3(kGvThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = gm.C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, p, gm) == cudaSuccess ? 0 : 1;
}

}  // namespace mxk
