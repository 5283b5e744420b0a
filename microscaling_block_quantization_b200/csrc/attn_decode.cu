// mx_attn_decode's launches: the kernel of the cache's format, the split of
// the sequences, and the join of the partial results.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_kernel.cuh"

namespace mxk {

namespace {

constexpr int kAttnSmem = 227 * 1024;
constexpr int kJoinCols = 64;   // elements of a head a join CTA takes

// One CTA per (sequence, query head, 64 elements of the head): the stretches'
// results weighted by their sums at the common maximum, added in a fixed order.
// Groups of 16 threads hold the 64 elements and take every (threads / 16)-th
// split; the groups' sums meet in shared memory.  Every warp finds the common
// maximum and sum of weights by itself, so that one barrier is all.
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
    float l = 0.0f;
    for (int s = lane; s < used; s += 32) l += at_weight(ml[s], m);
#pragma unroll
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    const float inv = at_over(l);             // (weights of 1 at most: no sum passes binary32)
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float *part = p.part_o + out * p.splits * D + d;
#pragma unroll 4
    for (int s = grp; s < used; s += groups) {
        const float w = __fmul_rn(at_weight(ml[s], m), inv);
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
    const float v[4] = {o.x, o.y, o.z, o.w};
    at_store4(p, seq, head, d, m, l, v);
}

AtPick at_pick(int el, int d, int bs, int nth, int hp, int sfmt)
{
#define AT_CASE(EL) \
    case EL: return d == 64 ? at_kernel_##EL##_64(bs, nth, hp, sfmt) : d == 128 ? at_kernel_##EL##_128(bs, nth, hp, sfmt) : at_kernel_##EL##_256(bs, nth, hp, sfmt);
    switch (el) {
        AT_CASE(GE_E2M1)
        AT_CASE(GE_E3M0)
        AT_CASE(GE_INT4)
        AT_CASE(AE_E2M3)
    default: return d == 64 ? at_kernel_AE_E3M2_64(bs, nth, hp, sfmt) : d == 128 ? at_kernel_AE_E3M2_128(bs, nth, hp, sfmt) : at_kernel_AE_E3M2_256(bs, nth, hp, sfmt);
    }
#undef AT_CASE
}

}  // namespace

// How a call of these sizes is split (times on a B200, both sides measured with one
// kernel, 157 us for the first of these sizes, and not again; 32 query and 8 key heads of 128, MXFP4 unless said).  As many stretches of 32 tokens at least as run at
// once (`warps_sm` warps of the kernel an SM); where several long sequences give
// stretches of 256 tokens and more, twice as many, so that a warp that is done
// makes room for another: 64 sequences of up to 8192 tokens 176 -> 156 us, but
// 256 of up to 300 33 -> 39 us.
// A second launch costs 2.5 us empty, and 3 to 5 with the join in it.  Where there are
// CTAs for half the SMs and more, a CTA's warps are a sequence's stretches and
// join them: 16 x 1000 15.3 -> 12.4 us, NVFP4 64 x 1000 42 -> 37 us, 128 x 2048 92 -> 85
// us.  With fewer CTAs, warps that share few SMs lose more than the launch costs
// (8 x 8192 31 against 44 us, clusters of CTAs included), but for up to 4 stretches
// of 64 tokens (1 x 200 8.5 -> 7.5 us); stretches past 512 tokens are better off as
// tasks of their own (64 x 8192 156 against 162 us).
AttnPlan attn_plan(int64_t seqs, int kv_heads, int q_heads, int64_t most_tokens, int warps_sm)
{
    const int group = q_heads / kv_heads;
    const int hg = group <= 4 ? 1 : (group + 7) / 8;
    const int64_t rows = seqs * kv_heads * hg, sms = device_sm_count();
    AttnPlan plan = {1, 0, kAtWarps};
    if (rows <= 0) return plan;
    if (2 * rows < sms && most_tokens <= 256) {
        plan.splits = most_tokens <= 64 ? 1 : (int)((most_tokens + 63) / 64);
        plan.joined = plan.splits > 1;
        if (plan.joined) plan.warps = plan.splits;
        return plan;
    }
    const int64_t once = sms * warps_sm / rows, twice = 2 * sms * warps_sm / rows, most = (most_tokens + 31) / 32;
    int64_t s = once < most ? once : most;
    if (seqs > 1 && twice > 1 && most_tokens >= 256 * twice) s = twice;
    if (s < 2) return plan;
    int w = (int)(s < warps_sm ? s : warps_sm);
    if (2 * rows >= sms && most_tokens <= 512 * w) {
        // more CTAs than SMs: so many warps each that an SM's warps divide by them
        while (rows > sms && warps_sm % w) --w;
        plan.splits = plan.warps = w;
        plan.joined = w > 1;
        if (!plan.joined) plan.warps = kAtWarps;
        return plan;
    }
    plan.splits = s > kAttnMaxSplits ? kAttnMaxSplits : (int)s;
    return plan;
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
    const AtPick k = at_pick(el, p.head_dim, p.log2B == 4 ? 16 : p.log2B == 5 ? 32 : 64, nth, hp, p.sfmt);
    // (the rings of 8-bit codes of long heads leave room for fewer warps)
    while (p.warps * k.ring > kAttnSmem) p.warps = p.splits = p.warps - 1;
    const int smem = p.warps * k.ring;
    p.tasks = p.seqs * (p.joined ? 1 : p.splits) * p.head_groups * p.kv_heads;
    if (smem > 48 * 1024 && raise_smem_limit(reinterpret_cast<const void *>(k.k), kAttnSmem)) return 1;
    const int64_t ctas = p.joined ? p.tasks : (p.tasks + p.warps - 1) / p.warps;
    if (launch_pdl(k.k, (unsigned)ctas, p.warps * 32, smem, st, p) != cudaSuccess) return 1;
    if (p.splits == 1 || p.joined) return 0;
    int groups = 4;
    while (groups < 32 && groups < p.splits) groups *= 2;
    return launch_pdl(k_attn_join, (unsigned)(p.seqs * p.q_heads * (p.head_dim / kJoinCols)), groups * 16, 0, st, p) == cudaSuccess ? 0 : 1;
}

}  // namespace mxk
