// Queries, keys and values of new tokens into attention's operands
// (mx_kv_append): per-head RMS norm and position rotation of queries and keys
// in one pass, keys and values quantized into rows of a paged cache.
//
//   h = x rsqrt(sum x^2 / D + eps) g,   (a, b) -> (a cos f - b sin f, b cos f + a sin f),
//   f = position inv_freq_i,  rounded once to the input's type; then the row's
//   blocks as mx_quantize writes them, bit for bit.
//
// Bound: every input read and every output written once (HBM bandwidth) for
// many tokens, latency for a few.  Eight consecutive elements a lane (16-byte
// bf16 loads): D / 8 lanes hold a head, a rotation partner D' / 2 elements
// away is the same register of another lane (D' / 2 a multiple of 8) or, in
// neighbouring pairs, in the lane itself; a block is block / 8 lanes, so norm,
// partner and block maximum are shuffles and nothing goes through shared
// memory but the angles.  A token's angles serve all its heads: position
// times inv_freq / 2 pi in binary64, reduced to a fraction of a turn there
// (exact to 2^-53 turns per turn at any position), then one sincospi each,
// computed once per token and CTA.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_internal.h"

namespace mxk {

constexpr int kKvThreads = 256;
constexpr int kKvWarps = kKvThreads / 32;

// elements of the quantized rows: conversion instructions, or the general rounding
enum { KE_E2M1 = 0, KE_E2M3 = 1, KE_E3M2 = 2, KE_ANY = 3 };
// block scales: powers of two in E8M0, nearest unsigned minifloat, powers of two in one
enum { KS_E8M0 = 0, KS_NEAR = 1, KS_POW2 = 2 };

template <bool FP32> __device__ __forceinline__ void kv_load8(const void *base, int64_t at, bool vec, float v[8])
{
    if (FP32) {
        const float *x = static_cast<const float *>(base) + at;
        if (vec) {
            const float4 a = *reinterpret_cast<const float4 *>(x), b = *reinterpret_cast<const float4 *>(x + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = x[i];
        }
    } else {
        const uint16_t *x = static_cast<const uint16_t *>(base) + at;
        uint32_t w[4];
        if (vec) {
            const uint4 a = *reinterpret_cast<const uint4 *>(x);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = x[2 * i] | ((uint32_t)x[2 * i + 1] << 16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bits2f(w[i] << 16);
            v[2 * i + 1] = bits2f(w[i] & 0xffff0000u);
        }
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
                                             uint8_t *codes, uint8_t *scales, int64_t row, int col)
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
    const int64_t at = row * p.cols + col;
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
__global__ void __launch_bounds__(kKvThreads) k_kv_append(const __grid_constant__ KvAppendParams p)
{
    constexpr int L = D / 8, RPW = 32 / L;      // lanes of a head, heads of a warp
    extern __shared__ float2 cs[];              // cos, sin: [tokens of a group][rot / 2]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (L - 1), sub = lane / L;
    const int half = p.rot >> 1;
    pdl_trigger();
    pdl_wait();

    // nearest scales: the scale and its reciprocal for every code, of keys and of values
    __shared__ float2 tab[SK == KS_NEAR ? 512 : 1];
    NearScale ns[2];   // (indexed by constants only)
    if (SK == KS_NEAR) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float *ts = i ? p.v_ts : p.k_ts;
            const float sT = ts ? *ts : 1.0f;
            for (int c = threadIdx.x; c < 256; c += kKvThreads) {
                const float d = __fmul_rn(ue_value(p.sd, (uint32_t)c), sT);
                tab[256 * i + c] = c < p.sd.ue_nan_code ? make_float2(d, __fdiv_rn(1.0f, d)) : make_float2(bits2f(0x7fc00000u), 0.0f);
            }
            ns[i].maxv = p.ed.maxv;
            ns[i].r_max = __fdiv_rn(1.0f, p.ed.maxv);
            ns[i].sT = sT;
            ns[i].r_T = (sT >= 0x1p-125f && sT <= 0x1p125f) ? __fdiv_rn(1.0f, sT) : 0.0f;
            const float ms = __fmul_rn(p.ed.maxv, sT);
            ns[i].c = (ms >= 0x1p-125f && ms <= 0x1p125f) ? __fdiv_rn(1.0f, ms) : 0.0f;
            ns[i].tab = tab + 256 * i;
        }
    }

    const int rows = p.q_heads + 2 * p.kv_heads;   // heads of a token: queries, keys, values
    const int per_y = (rows + gridDim.y - 1) / gridDim.y;
    const int r0 = blockIdx.y * per_y, rn = min(per_y, rows - r0);
    for (int64_t t0 = (int64_t)blockIdx.x * p.group; t0 < p.tokens; t0 += (int64_t)gridDim.x * p.group) {
        const int tn = (int)min((int64_t)p.group, p.tokens - t0);
        __syncthreads();   // the last group's angles are no longer read
        for (int i = threadIdx.x; i < tn * half; i += kKvThreads) {
            const int tk = i / half;
            const double turns = (double)p.positions[t0 + tk] * ((double)p.inv_freq[i - tk * half] * 0.15915494309189533577);
            float sn, cn;
            sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cn);
            cs[i] = make_float2(cn, sn);
        }
        __syncthreads();
        const int items = tn * rn;
        for (int i0 = warp * RPW; i0 < items; i0 += kKvWarps * RPW) {
            const int i = min(i0 + sub, items - 1);
            const bool on = i0 + sub < items;
            const int tk = i / rn, r = r0 + i - tk * rn;
            const int64_t tok = t0 + tk;
            const int kind = r < p.q_heads ? 0 : r < p.q_heads + p.kv_heads ? 1 : 2;
            const int head = r - (kind == 0 ? 0 : kind == 1 ? p.q_heads : p.q_heads + p.kv_heads);
            const void *src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
            const int64_t ld = kind == 0 ? p.ldq : kind == 1 ? p.ldk : p.ldv;
            float v[8];
            kv_load8<FP32>(src, tok * ld + head * D + 8 * l, p.in_vec, v);
            const float *gain = kind == 0 ? p.q_gain : kind == 1 ? p.k_gain : nullptr;
            if (p.q_gain || p.k_gain) {
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
                for (int d = L / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
                if (gain) {
                    const float f = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.0f / D), p.eps));
                    const float4 a = *reinterpret_cast<const float4 *>(gain + 8 * l), b = *reinterpret_cast<const float4 *>(gain + 8 * l + 4);
                    const float g[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(__fmul_rn(v[j], f), g[j]);
                }
            }
            if (p.rot) {
                if (p.interleaved) {
                    if (kind < 2 && 8 * l < p.rot) {
                        const float2 *c = cs + tk * half + 4 * l;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float a = v[2 * j], b = v[2 * j + 1];
                            v[2 * j] = fmaf(a, c[j].x, -__fmul_rn(b, c[j].y));
                            v[2 * j + 1] = fmaf(b, c[j].x, __fmul_rn(a, c[j].y));
                        }
                    }
                } else {
                    // element i of the first half pairs with i + rot / 2: the
                    // same register rot / 16 lanes on
                    const int dl = p.rot >> 4;
                    const bool lo = l < dl;
                    const int from = (lane & ~(L - 1)) | ((lo ? l + dl : l - dl) & (L - 1));
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(0xffffffffu, v[j], from);
                    if (kind < 2 && 8 * l < p.rot) {
                        const float2 *c = cs + tk * half + 8 * (lo ? l : l - dl);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float t = __fmul_rn(o[j], c[j].y);
                            v[j] = fmaf(v[j], c[j].x, lo ? -t : t);
                        }
                    }
                }
            }
            if (kind == 0) kv_round_store8<FP32>(p.q_out, tok * p.ldqo + head * D + 8 * l, p.out_vec, on, v);
            else kv_round_store8<FP32>(p.k_out, tok * p.ldko + head * D + 8 * l, p.out_vec, on && kind == 1 && p.k_out, v);
            const int64_t slot = p.slots[tok];
            const bool store = on && kind != 0 && slot >= 0 && slot < p.cache_rows;
            if (__any_sync(0xffffffffu, store))
            {
                NearScale n = ns[0];
                if (SK == KS_NEAR && kind == 2) n = ns[1];
                kv_quantize8<EK, SK>(p, n, v, store, kind == 1 ? p.k_codes : p.v_codes,
                                     kind == 1 ? p.k_scales : p.v_scales, slot, head * D + 8 * l);
            }
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
    // few tokens: one a CTA, its heads over several CTAs (a warp's worth of
    // work each); many: groups of four, whose angles one barrier covers
    const int rows = p.q_heads + 2 * p.kv_heads, pass = kKvWarps * (256 / head_dim);
    const int64_t slots = 4 * (int64_t)device_sm_count();
    p.group = p.tokens > 4 * slots ? 4 : 1;
    const int64_t groups = (p.tokens + p.group - 1) / p.group;
    int64_t y = (rows + pass - 1) / pass;
    if (groups * y > slots) y = slots / groups > 1 ? slots / groups : 1;
    const int64_t x = groups < slots ? groups : slots;
    const size_t smem = (size_t)p.group * (p.rot / 2) * sizeof(float2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)x, (unsigned)y);
    cfg.blockDim = dim3(kKvThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, p) == cudaSuccess ? 0 : 1;
}

}  // namespace mxk
