// mx_attn_decode's launches: the kernel of the cache's format, the split of
// the sequences, and the join of the partial results.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_kernel.cuh"

namespace mxk {

namespace {

constexpr int kJoinCols = 64;   // elements of a head a join CTA takes

// One CTA per (sequence, query head, 64 elements of the head): the stretches'
// results weighted by their sums at the common maximum, added in a fixed order.  Groups of 16
// threads hold the 64 elements and take every (threads / 16)-th split; the
// groups' sums meet in shared memory.  Every warp finds the common maximum and
// sum of weights by itself, so that one barrier is all.
__global__ void __launch_bounds__(512) k_attn_join(const __grid_constant__ AttnParams p)
{
    __shared__ float4 red[512];
    const int lane = threadIdx.x & 31, groups = blockDim.x / 16, d4 = threadIdx.x & 15, grp = threadIdx.x / 16;
    const int D = p.head_dim, chunks = D / kJoinCols;
    const int64_t out = blockIdx.x / chunks;            // sequence * q_heads + head
    const int d = (blockIdx.x % chunks) * kJoinCols + 4 * d4;
    const int seq = (int)(out / p.q_heads), head = (int)(out % p.q_heads);
    pdl_trigger();
    pdl_wait();
    int n, vis, sinks;
    at_visible(p, seq, n, vis, sinks);
    const int tiles = (vis + 15) >> 4, per = (tiles + p.splits - 1) / p.splits;
    const int used = per ? (tiles + per - 1) / per : 0;
    const float2 *ml = p.part_ml + out * p.splits;
    float m = -INFINITY;
    for (int s = lane; s < used; s += 32) m = fmaxf(m, ml[s].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    // a stretch without a visible token has m = -inf, l = 0; one whose scores
    // are NaN makes the result NaN
    const auto weight = [m](float2 x) { return x.y == 0.0f ? 0.0f : x.y != x.y ? x.y : x.y * exp2f(x.x - m); };
    float l = 0.0f;
    for (int s = lane; s < used; s += 32) l += weight(ml[s]);
#pragma unroll
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float *part = p.part_o + out * p.splits * D + d;
#pragma unroll 4
    for (int s = grp; s < used; s += groups) {
        const float w = weight(ml[s]);
        const float4 v = *reinterpret_cast<const float4 *>(part + (int64_t)s * D);
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
    }
    red[threadIdx.x] = o;
    __syncthreads();
    if (grp) return;
    for (int i = 1; i < groups; ++i) {
        const float4 v = red[i * 16 + d4];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
    }
    const bool any = l > 0.0f || l != l;
    const float inv = any ? __fdiv_rn(1.0f, l) : 0.0f;
    const float v[4] = {o.x, o.y, o.z, o.w};
    const int64_t at = (int64_t)seq * p.ldo + (int64_t)head * D + d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float y = any ? __fmul_rn(v[i], inv) : 0.0f;
        if (p.o_fp32) static_cast<float *>(p.out)[at + i] = y;
        else static_cast<__nv_bfloat16 *>(p.out)[at + i] = __float2bfloat16_rn(y);
    }
    if (d == 0 && p.lse) p.lse[out] = any ? (m + log2f(l)) * 0.693147180559945309417f : -INFINITY;
}

AtPick at_pick(int el, int d, int bs, int nth, int hp, int vm)
{
#define AT_CASE(EL) \
    case EL: return d == 64 ? at_kernel_##EL##_64(bs, nth, hp, vm) : d == 128 ? at_kernel_##EL##_128(bs, nth, hp, vm) : at_kernel_##EL##_256(bs, nth, hp, vm);
    switch (el) {
        AT_CASE(GE_E2M1)
        AT_CASE(GE_E3M0)
        AT_CASE(GE_INT4)
        AT_CASE(AE_E2M3)
    default: return d == 64 ? at_kernel_AE_E3M2_64(bs, nth, hp, vm) : d == 128 ? at_kernel_AE_E3M2_128(bs, nth, hp, vm) : at_kernel_AE_E3M2_256(bs, nth, hp, vm);
    }
#undef AT_CASE
}

}  // namespace

// Splits of every sequence for a call of these sizes.  One sequence is split
// into as many stretches as run at once (`warps` of the kernel an SM); several,
// whose lengths differ, into twice as many, so that a warp that is done makes
// room for another (64 of up to 8192: 154 us, four times as many 161).
// Stretches of 64 tokens at least.
int attn_splits(int64_t seqs, int kv_heads, int q_heads, int64_t most_tokens, int warps)
{
    const int group = q_heads / kv_heads;
    const int hg = group <= 4 ? 1 : (group + 7) / 8;
    const int64_t rows = seqs * kv_heads * hg;
    if (rows <= 0) return 1;
    const int64_t want = (int64_t)device_sm_count() * warps * (seqs == 1 ? 1 : 2);
    int64_t s = want / rows;
    const int64_t cap = (most_tokens + 63) / 64;
    s = s < cap ? s : cap;
    return s < 1 ? 1 : s > kAttnMaxSplits ? kAttnMaxSplits : (int)s;
}

// Warps of the call's kernel that an SM holds, by its registers.
int attn_warps(int head_dim, int block, int q_heads, int kv_heads, int hp)
{
    return hp || q_heads / kv_heads > 4 || head_dim == 256 || block == 16 ? 12 : 16;
}

int launch_attn(AttnParams p, int el, int hp, cudaStream_t st)
{
    p.group = p.q_heads / p.kv_heads;
    const int nth = p.group <= 4 ? 1 : 2;
    p.head_groups = (p.group + 4 * nth - 1) / (4 * nth);
    p.tasks = p.seqs * p.splits * p.head_groups * p.kv_heads;
    const AtPick k = at_pick(el, p.head_dim, p.log2B == 4 ? 16 : p.log2B == 5 ? 32 : 64, nth, hp, p.sfmt == S_UE4M3);
    if (k.smem > 48 * 1024 && raise_smem_limit(reinterpret_cast<const void *>(k.k), k.smem)) return 1;
    const int64_t ctas = (p.tasks + kAtWarps - 1) / kAtWarps;
    if (launch_pdl(k.k, (unsigned)ctas, kAtThreads, k.smem, st, p) != cudaSuccess) return 1;
    if (p.splits == 1) return 0;
    int groups = 4;
    while (groups < 32 && groups < p.splits) groups *= 2;
    return launch_pdl(k_attn_join, (unsigned)(p.seqs * p.q_heads * (p.head_dim / kJoinCols)), groups * 16, 0, st, p) == cudaSuccess ? 0 : 1;
}

}  // namespace mxk
