// mx_gemv's launch: the kernel of the element kind and block size, and the
// split of the work over clusters, CTAs and warps.
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "gemv_kernel.cuh"

namespace mxk {

namespace {

GvKernel gv_pick(int elem, int mode, int bc, int nt)
{
    switch (elem) {
    case GE_E2M1: return gv_kernel_e2m1(mode, bc, nt);
    case GE_E3M0: return gv_kernel_e3m0(mode, bc, nt);
    case GE_INT4: return gv_kernel_int4(mode, bc, nt);
    default: return gv_kernel_uint4(mode, bc, nt);
    }
}

template <int MODE> int gv_stage_size(int bc)
{
    return bc == 32 ? gv_stage_bytes<MODE, 32>() : bc == 16 ? gv_stage_bytes<MODE, 16>() : gv_stage_bytes<MODE, 8>();
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
    GvKernel k = gv_pick(GE_E2M1, GM_BLOCK, 32, 1);
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
    const int64_t tiles = (p.N + 15) / 16;

    const bool wide = p.K % 256 == 0 && !p.macro;
    const int mode = wide && p.log2B >= 7 ? GM_GROUP : wide && p.log2B <= 5 && !p.off ? GM_BLOCK : GM_ANY;
    const int uc = gv_chunks(mode);
    p.units = (int)((p.K + 128 * uc - 1) / (128 * uc));
    GvGeom gm = {};
    const int stage = mode == GM_GROUP ? gv_stage_bytes<GM_GROUP, 32>()
                    : mode == GM_BLOCK ? gv_stage_size<GM_BLOCK>(bc) : gv_stage_size<GM_ANY>(bc);
    const int ring = kGvWarps * gv_stages(mode) * stage;
    const int x_room = kGvSmem - ring - 32 * 1024;   // x beside the ring and the partial sums
    const int per_unit = uc * (2048 * nt + 32 * nt + (p.off ? 128 * nt : 0));

    // The split of K over a cluster (C) and over a CTA's warps (KS), by an
    // estimate in nanoseconds from sweeps on a B200: a warp's 128-column chunk
    // takes 480 (NT = 2: 800) beside 15 others; a (chunk, token) of x 12 to
    // stage; the join reads C KS sums an output, from other CTAs at 150 against
    // 60 each round, and a wave of partial sums more costs 1500.  4096 x 4096,
    // one token: C, KS = 1, 8 5.6 us, 4, 4 6.9, 1, 1 9.5; 4096 x 14336 INT4, 4
    // tokens: 4, 2 17.5, 1, 8 25.4, 1, 1 56.7; 65536 x 8192, 16 tokens: 4, 1
    // 107, 1, 1 131, 1, 8 285.
    GvKernel k = gv_pick(p.elem, mode, bc, nt);
    if (raise_smem_limit(reinterpret_cast<const void *>(k), kGvSmem)) return 1;
    const int toks = (int)(p.M < p.group ? p.M : p.group);
    int64_t best = -1;
    for (int C = 1; C <= 8; C *= 2) {
        const int cpc = (p.units + C - 1) / C;
        const int64_t lim = resident_clusters(C);
        const int64_t ncl = tiles < lim ? tiles : lim;
        const int64_t per = (tiles + ncl - 1) / ncl;
        const bool fits = (int64_t)cpc * per_unit <= x_room;
        for (int KS = 1; KS <= kGvWarps; KS *= 2) {
            const int64_t tg = kGvWarps / KS;
            const int64_t units = ((per + tg - 1) / tg) * ((cpc + KS - 1) / KS);
            const int64_t x_bytes = (fits ? cpc : x_room / per_unit) * (int64_t)per_unit;
            const int64_t held = (kGvSmem - ring - x_bytes) / ((KS * kGvPart * nt + 16) * 4);
            const int64_t waves = held < 1 ? 1000 : (per + held - 1) / held;
            const int64_t rounds = (per * 4 * toks + C * kGvThreads - 1) / (C * kGvThreads);
            const int64_t cost = units * uc * (nt == 1 ? 480 : 800) + (fits ? 1 : waves) * cpc * uc * toks * 12 +
                                 rounds * C * KS * (C > 1 ? 150 : 60) + (C > 1 ? 500 : 0) + (waves - 1) * 1500;
            if (best < 0 || cost < best) {
                best = cost;
                gm.C = C;
                gm.KS = KS;
                gm.xc = cpc;
            }
        }
    }
    const int xc_max = x_room / per_unit;
    if (gm.xc > xc_max) gm.xc = xc_max;
    if (gm.xc < 1) gm.xc = 1;
    int at = ring;
    gm.xs_at = at; at += gm.xc * uc * 2048 * nt;
    gm.ex_at = at; at += gm.xc * uc * 32 * nt;
    gm.xsum_at = at; at += p.off ? gm.xc * uc * 128 * nt : 0;
    gm.part_at = at;
    const int64_t ncl_max = resident_clusters(gm.C);
    const int64_t ncl = tiles < ncl_max ? tiles : ncl_max;
    const int64_t per = (tiles + ncl - 1) / ncl;
    gm.tile_floats = gm.KS * kGvPart * nt + 16;
    const int tile_bytes = gm.tile_floats * 4;
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
