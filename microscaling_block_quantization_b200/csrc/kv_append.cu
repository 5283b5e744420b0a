// Queries, keys and values of new tokens into attention's operands
// (mx_kv_append): per-head RMS norm and position rotation of queries and keys
// in one pass, keys and values quantized into rows of a paged cache.
//
//   h = x rsqrt(sum x^2 / D + eps) g,   (a, b) -> (a cos f - b sin f, b cos f + a sin f),
//   f = position inv_freq_i,  rounded once to the input's type; then the row's
//   blocks as mx_quantize writes them, bit for bit.
//
// Bound: every input read and every output written once (HBM bandwidth) for
// many tokens, latency for a few.  A warp takes a token, or a share of its
// heads when tokens are few, and goes over query, key and value heads in
// turn.  Eight consecutive elements a lane (16-byte bf16 loads): D / 8 lanes
// hold a head, a rotation partner D' / 2 elements away is the same register of
// another lane (D' / 2 a multiple of 8) or, in neighbouring pairs, in the lane
// itself; a block is block / 8 lanes, so norm, partner and block maximum are
// shuffles.  A token's angles serve all its heads and stay in registers, as do
// the gains.  Each lane copies its own pieces of the coming heads into a ring
// in shared memory (seven 512-byte loads of a warp in flight).  Angles:
// position times inv_freq / 2 pi in binary64, reduced to a fraction of a turn
// there (2^-53 of the turns), then one sincospi, shared by the warp.
//
// Measured: 8192 tokens of 32 query and 8 key heads of 128 into NVFP4, 72 us
// (2.7 TB/s): the issue slots, 253 instructions a head of norm, rotation and
// nearest scales, are 66% taken.  8 tokens 4 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mma_decode.cuh"
#include "mx_internal.h"

namespace mxk {

constexpr int kKvThreads = 256;
constexpr int kKvWarps = kKvThreads / 32;
constexpr int kKvRing = 4096;   // bytes of a warp's ring

// elements of the quantized rows: conversion instructions, or the general rounding
enum { KE_E2M1 = 0, KE_E2M3 = 1, KE_E3M2 = 2, KE_ANY = 3 };
// block scales: powers of two in E8M0, nearest unsigned minifloat, powers of two in one
enum { KS_E8M0 = 0, KS_NEAR = 1, KS_POW2 = 2 };

// Eight values of a row as loaded, and in binary32.
template <bool FP32> struct KvRaw { uint32_t w[FP32 ? 8 : 4]; };

template <bool FP32> __device__ __forceinline__ void kv_load8(const void *src, KvRaw<FP32> &r)
{
    if (FP32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[FP32 ? i : 0] = static_cast<const uint32_t *>(src)[i];
    } else {
        const uint16_t *x = static_cast<const uint16_t *>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = x[2 * i] | ((uint32_t)x[2 * i + 1] << 16);
    }
}
template <bool FP32> __device__ __forceinline__ void kv_values(const KvRaw<FP32> &r, float v[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = FP32 ? bits2f(r.w[FP32 ? 2 * i : 0]) : bits2f(r.w[i] << 16);
        v[2 * i + 1] = FP32 ? bits2f(r.w[FP32 ? 2 * i + 1 : 0]) : bits2f(r.w[i] & 0xffff0000u);
    }
}

// Store eight values rounded to the type, and leave the rounded values in v.
template <bool FP32> __device__ __forceinline__ void kv_round_store8(void *base, int64_t at, bool vec, bool store, float v[8])
{
    if (FP32) {
        if (!store) return;
        float *y = static_cast<float *>(base) + at;
        if (vec) {
            *reinterpret_cast<float4 *>(y) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(y + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = v[i];
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
            v[2 * i] = bits2f(w[i] << 16);
            v[2 * i + 1] = bits2f(w[i] & 0xffff0000u);
        }
        if (!store) return;
        uint16_t *y = static_cast<uint16_t *>(base) + at;
        if (vec) {
            *reinterpret_cast<uint4 *>(y) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// Quantize the lane's eight values of a row (blocks of `block` / 8 lanes) and
// store codes and scale; every lane of the warp takes part in the shuffles.
template <int EK, int SK>
__device__ __forceinline__ void kv_quantize8(const KvAppendParams &p, const NearScale &ns, const float v[8], bool store,
                                             uint8_t *codes, uint8_t *scales, int64_t at)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    for (int d = 1; d < p.lanes_per_block; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (!store) return;
    const int nonfinite = m >= 0x7f800000u;
    const float alpha = bits2f(m);
    BlockScale bs;
    if (SK == KS_E8M0) bs = e8m0_block_scale(alpha, nonfinite, p.ed.emax, p.thr_m);
    else if (SK == KS_NEAR) bs = near_block_scale(p.sd, ns, alpha, nonfinite);
    else bs = block_scale(p.ed, p.sd, alpha, nonfinite, 1.0f);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = __fmul_rn(v[i], bs.inv);
    if (EK == KE_E2M1) {
        *reinterpret_cast<uint32_t *>(codes + (at >> 1)) = bs.zero ? 0u : cvt_e2m1x8(s);
    } else if (EK == KE_E2M3 || EK == KE_E3M2) {
        uint32_t w[2] = {0u, 0u};
        if (!bs.zero) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint16_t r;
                if (EK == KE_E2M3) asm("cvt.rn.satfinite.e2m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(s[2 * i + 1]), "f"(s[2 * i]));
                else asm("cvt.rn.satfinite.e3m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(s[2 * i + 1]), "f"(s[2 * i]));
                w[i >> 1] |= (uint32_t)r << (16 * (i & 1));
            }
        }
        *reinterpret_cast<uint2 *>(codes + at) = make_uint2(w[0], w[1]);
    } else {
        uint32_t w[2] = {0u, 0u};
        if (!bs.zero) {
            const int bits = p.ed.code_bits == 4 ? 4 : 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float q;
                const uint32_t c = encode_elem(p.ed, p.round_mode, s[i], 0u, q);
                if (bits == 4) w[0] |= c << (4 * i);
                else w[i >> 2] |= c << (8 * (i & 3));
            }
        }
        if (p.ed.code_bits == 4) *reinterpret_cast<uint32_t *>(codes + (at >> 1)) = w[0];
        else *reinterpret_cast<uint2 *>(codes + at) = make_uint2(w[0], w[1]);
    }
    if (((threadIdx.x & 31) & (p.lanes_per_block - 1)) == 0) scales[at >> p.log2B] = (uint8_t)bs.code;
}

template <int D, bool FP32, int EK, int SK>
__global__ void __launch_bounds__(kKvThreads, 3) k_kv_append(const __grid_constant__ KvAppendParams p)
{
    constexpr int L = D / 8, RPW = 32 / L;            // lanes of a head, heads of a warp
    __shared__ float2 cs_all[kKvWarps][D / 2];        // cos, sin of a warp's token
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (L - 1), sub = lane / L;
    const int half = p.rot >> 1;
    float2 *cs = cs_all[warp];
    pdl_trigger();
    pdl_wait();

    // nearest scales: the scale and its reciprocal for every code, of keys and of values
    __shared__ float2 tab[SK == KS_NEAR ? 512 : 1];
    NearScale ns_k, ns_v;
    if (SK == KS_NEAR) {
        const auto make = [&](NearScale &ns, const float *ts, float2 *t) {
            const float sT = ts ? *ts : 1.0f;
            for (int c = threadIdx.x; c < 256; c += kKvThreads) {
                const float d = __fmul_rn(ue_value(p.sd, (uint32_t)c), sT);
                t[c] = c < p.sd.ue_nan_code ? make_float2(d, __fdiv_rn(1.0f, d)) : make_float2(bits2f(0x7fc00000u), 0.0f);
            }
            ns.maxv = p.ed.maxv;
            ns.r_max = __fdiv_rn(1.0f, p.ed.maxv);
            ns.sT = sT;
            ns.r_T = (sT >= 0x1p-125f && sT <= 0x1p125f) ? __fdiv_rn(1.0f, sT) : 0.0f;
            const float ms = __fmul_rn(p.ed.maxv, sT);
            ns.c = (ms >= 0x1p-125f && ms <= 0x1p125f) ? __fdiv_rn(1.0f, ms) : 0.0f;
            ns.tab = t;
        };
        make(ns_k, p.k_ts, tab);
        make(ns_v, p.v_ts, tab + (SK == KS_NEAR ? 256 : 0));
        __syncthreads();
    }

    const bool turns = 8 * l < p.rot;                 // the lane's elements are rotated
    const int dl = p.rot >> 4;                        // lanes to the partner (pairs rot / 2 apart)
    const bool lo = l < dl;
    const int from = (lane & ~(L - 1)) | ((lo ? l + dl : l - dl) & (L - 1));

    // a token's heads in units of RPW: queries, keys, values
    const int nq = (p.q_heads + RPW - 1) / RPW, nk = (p.kv_heads + RPW - 1) / RPW, units = nq + 2 * nk;
    const int64_t tasks = p.tokens * p.parts, stride = (int64_t)gridDim.x * kKvWarps;
    const int64_t first = (int64_t)blockIdx.x * kKvWarps + warp;

    // where a lane's eight values of a unit are
    constexpr int ES = FP32 ? 4 : 2;
    const auto source = [&](int64_t tok, int u) {
        const char *src;
        int64_t ld;
        int h0;
        if (u < nq) src = static_cast<const char *>(p.q), ld = p.ldq, h0 = u;
        else if (u < nq + nk) src = static_cast<const char *>(p.k), ld = p.ldk, h0 = u - nq;
        else src = static_cast<const char *>(p.v), ld = p.ldv, h0 = u - nq - nk;
        return src + (tok * ld + (h0 * RPW + sub) * D + 8 * l) * ES;
    };
    // (the last unit of a kind may have fewer heads than the warp has room for)
    const auto present = [&](int u) {
        const int h = (u < nq ? u : u < nq + nk ? u - nq : u - nq - nk) * RPW + sub;
        return h < (u < nq ? p.q_heads : p.kv_heads);
    };
    // the lane's ring: pieces of the units to come, this task's and the next
    constexpr int PIECE = FP32 ? 32 : 16, STAGES = kKvRing / (32 * PIECE);
    extern __shared__ __align__(16) uint8_t ring_all[];
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_all) + warp * kKvRing + lane * 16;
    const uint32_t ring_end = ring + STAGES * 32 * PIECE;
    const auto span = [&](int64_t task, int64_t &tok, int &u0, int &u1) {
        if (p.parts == 1) {
            tok = task;
            u0 = 0;
            u1 = units;
        } else {
            tok = task / p.parts;
            const int part = (int)(task - tok * p.parts);
            u0 = units * part / p.parts;
            u1 = units * (part + 1) / p.parts;
        }
    };
    int64_t ahead = first, atok = 0;
    int au = 0, aend = 0;
    const char *asrc = nullptr;
    uint32_t st_w = ring, st_r = ring;
    const auto issue = [&]() {
        if (ahead < tasks) {
            const bool in = present(au);
            const char *src = in ? asrc : static_cast<const char *>(p.k);
            cp_async16(st_w, src, in ? 16 : 0);
            if (FP32) cp_async16(st_w + 512, in ? src + 16 : src, in ? 16 : 0);
            ++au;
            asrc += RPW * D * ES;
            if (au == aend) {
                ahead += stride;
                if (ahead < tasks) {
                    span(ahead, atok, au, aend);
                    asrc = source(atok, au);
                }
            } else if (au == nq || au == nq + nk) {
                asrc = source(atok, au);
            }
        }
        cp_async_commit();
        st_w = st_w + 32 * PIECE == ring_end ? ring : st_w + 32 * PIECE;
    };
    if (p.in_vec && first < tasks) {
        span(first, atok, au, aend);
        asrc = source(atok, au);
        for (int i = 0; i < STAGES - 1; ++i) issue();
    }

    for (int64_t task = first; task < tasks; task += stride) {
        int64_t tok;
        int u0, u1;
        span(task, tok, u0, u1);
        const int64_t slot = p.slots[tok];
        const bool stored = slot >= 0 && slot < p.cache_rows;
        float2 c[8];
        if (half && u0 < nq + nk) {
            const double pos = (double)p.positions[tok];
            __syncwarp();                             // the last token's angles are read
            for (int i = lane; i < half; i += 32) {
                const double t = pos * ((double)p.inv_freq[i] * 0.15915494309189533577);
                float sn, cn;
                sincospif(2.0f * (float)(t - rint(t)), &sn, &cn);
                cs[i] = make_float2(cn, sn);
            }
            __syncwarp();
            if (turns) {
                // (a cos - b sin, b cos + a sin): the sine of the first of a
                // pair with its sign
                const int at = p.interleaved ? 4 * l : 8 * (lo ? l : l - dl);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    c[j] = cs[at + (p.interleaved ? j >> 1 : j)];
                    if (p.interleaved ? (j & 1) == 0 : lo) c[j].y = -c[j].y;
                }
            }
        }
        const auto take = [&](int u, float v[8]) {
            KvRaw<FP32> raw;
            if (p.in_vec) {
                cp_async_wait<STAGES - 2>();
                const uint4 x = lds128(st_r);
                raw.w[0] = x.x; raw.w[1] = x.y; raw.w[2] = x.z; raw.w[3] = x.w;
                if (FP32) {
                    const uint4 y = lds128(st_r + 512);
                    raw.w[FP32 ? 4 : 0] = y.x; raw.w[FP32 ? 5 : 0] = y.y; raw.w[FP32 ? 6 : 0] = y.z; raw.w[FP32 ? 7 : 0] = y.w;
                }
                st_r = st_r + 32 * PIECE == ring_end ? ring : st_r + 32 * PIECE;
                issue();
            } else {
                kv_load8<FP32>(present(u) ? source(tok, u) : static_cast<const char *>(p.k), raw);
            }
            kv_values<FP32>(raw, v);
        };
        // norm and rotation of queries or keys
        const auto turn = [&](const float *gain, const float g[8], float v[8]) {
            if (gain) {
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
                for (int d = L / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
                const float f = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.0f / D), p.eps));
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(__fmul_rn(v[j], f), g[j]);
            }
            if (half) {
                float o[8];
                if (p.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = v[j ^ 1];
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(0xffffffffu, v[j], from);
                }
                if (turns) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j], c[j].x, __fmul_rn(o[j], c[j].y));
                }
            }
        };
        const auto gains = [&](const float *gain, float g[8]) {
            if (!gain) return;
            const float4 a = *reinterpret_cast<const float4 *>(gain + 8 * l), b = *reinterpret_cast<const float4 *>(gain + 8 * l + 4);
            g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
            g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
        };
        const int64_t row = stored ? slot * p.cols : 0;
        int u = u0;
        if (u < nq) {
            float g[8];
            gains(p.q_gain, g);
            const int64_t out = tok * p.ldqo + 8 * l;
            for (const int e = min(u1, nq); u < e; ++u) {
                float v[8];
                take(u, v);
                turn(p.q_gain, g, v);
                const int head = u * RPW + sub;
                kv_round_store8<FP32>(p.q_out, out + head * D, p.out_vec, head < p.q_heads, v);
            }
        }
        if (u < u1 && u < nq + nk) {
            float g[8];
            gains(p.k_gain, g);
            const int64_t out = tok * p.ldko + 8 * l;
            for (const int e = min(u1, nq + nk); u < e; ++u) {
                float v[8];
                take(u, v);
                turn(p.k_gain, g, v);
                const int head = (u - nq) * RPW + sub;
                const bool on = head < p.kv_heads;
                kv_round_store8<FP32>(p.k_out, out + head * D, p.out_vec, on && p.k_out, v);
                kv_quantize8<EK, SK>(p, ns_k, v, on && stored, p.k_codes, p.k_scales, row + head * D + 8 * l);
            }
        }
        for (; u < u1; ++u) {
            float v[8];
            take(u, v);
            const int head = (u - nq - nk) * RPW + sub;
            kv_quantize8<EK, SK>(p, ns_v, v, head < p.kv_heads && stored, p.v_codes, p.v_scales, row + head * D + 8 * l);
        }
    }
}

namespace {

typedef void (*KvKernel)(const KvAppendParams);

template <int D, bool FP32, int EK> KvKernel kv_pick_sk(int sk)
{
    return sk == KS_E8M0 ? k_kv_append<D, FP32, EK, KS_E8M0> : sk == KS_NEAR ? k_kv_append<D, FP32, EK, KS_NEAR>
                                                                             : k_kv_append<D, FP32, EK, KS_POW2>;
}
template <int D, bool FP32> KvKernel kv_pick_ek(int ek, int sk)
{
    switch (ek) {
    case KE_E2M1: return kv_pick_sk<D, FP32, KE_E2M1>(sk);
    case KE_E2M3: return kv_pick_sk<D, FP32, KE_E2M3>(sk);
    case KE_E3M2: return kv_pick_sk<D, FP32, KE_E3M2>(sk);
    default: return kv_pick_sk<D, FP32, KE_ANY>(sk);
    }
}
template <int D> KvKernel kv_pick_type(bool fp32, int ek, int sk)
{
    return fp32 ? kv_pick_ek<D, true>(ek, sk) : kv_pick_ek<D, false>(ek, sk);
}

}  // namespace

int launch_kv_append(KvAppendParams p, int head_dim, int in_fp32, cudaStream_t st)
{
    const int ek = p.round_mode != RD_RTNE ? KE_ANY : p.ed.elem == E2M1 ? KE_E2M1 : p.ed.elem == E2M3 ? KE_E2M3
                 : p.ed.elem == E3M2 ? KE_E3M2 : KE_ANY;
    const int sk = p.sd.fmt == S_E8M0 ? KS_E8M0 : p.sd.rule == R_NEAREST ? KS_NEAR : KS_POW2;
    KvKernel k = head_dim == 64 ? kv_pick_type<64>(in_fp32, ek, sk) : head_dim == 128 ? kv_pick_type<128>(in_fp32, ek, sk)
                                                                    : kv_pick_type<256>(in_fp32, ek, sk);
    // few tokens: a token's heads over as many warps as the device holds, one
    // unit each at the least; many: a warp a token
    const int rpw = 256 / head_dim;
    const int64_t units = (p.q_heads + rpw - 1) / rpw + 2 * ((p.kv_heads + rpw - 1) / rpw);
    const int64_t warps = (int64_t)device_sm_count() * 3 * kKvWarps;
    int64_t parts = warps / p.tokens;
    parts = parts < 1 ? 1 : parts > units ? units : parts;
    p.parts = (int)parts;
    const int64_t ctas = (p.tokens * parts + kKvWarps - 1) / kKvWarps, most = 16 * (int64_t)device_sm_count();
    return launch_pdl(k, (unsigned)(ctas < most ? ctas : most), kKvThreads, kKvWarps * kKvRing, st, p) == cudaSuccess ? 0 : 1;
}

}  // namespace mxk
