// linear_product.cuh -- the second kernel of a compressed linear layer: the decoded fp16 weight times
// every token on the 5th-generation tensor cores, with bias, activation, gating and residual in the
// epilogue (linear_common.cuh states the operator and its scales).
//
// Two CTAs of a cluster share one tile of 256 weight rows x up to 256 tokens (tcgen05.mma,
// cta_group::2): the weight rows are the M side, 128 per CTA, so that bias and row scale are one value
// per thread and the number of tokens, which varies, is the N side in steps of 32.  Each CTA loads its
// 128 weight rows and its half of the tokens (TMA, 128-byte swizzle, 64 columns of K per stage); fp32
// accumulators sit in both CTAs' TMEM, two sets of 256 columns, so that one tile's epilogue runs under
// the next tile's products.  Warp 0 loads, warp 1 of the leading CTA issues the products, warps 2 to 9
// run the epilogue.
//
// A persistent grid walks the tiles of all groups.  Tiles that do not fill a last round of pairs are
// split along K over the idle pairs; partial sums go through the workspace and the pair that arrives
// last adds them in the order of the splits, so results do not depend on timing.
#pragma once
#include <cuda.h>
#include "linear_common.cuh"

namespace llvq {

constexpr int kLpThreads = 320;
constexpr int kLpEpilogueWarps = 8;
constexpr int kLpStages = 6;
constexpr int kLpK = 64;                                   // columns of K per stage: one 128-byte swizzle row
constexpr int kLpABytes = 128 * kLpK * 2;                  // 128 weight rows
constexpr int kLpBBytes = kLinTokens / 2 * kLpK * 2;       // up to 128 tokens
constexpr int kLpStageBytes = kLpABytes + kLpBBytes;
constexpr int kLpBand = 8;                                 // row tiles of a band (L2 reuse of the tokens)
constexpr int kLpMinSplit = 4;                             // least K stages of a split

struct LpShared {
    unsigned long long full[kLpStages], empty[kLpStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort, nact, last;
    int tiles, whole, split, units;
    int id[kLinExperts], lo[kLinExperts], hi[kLinExperts], first[kLinExperts + 1];
};
__host__ __device__ constexpr size_t lp_smem(bool grouped) {
    return 1024 + (size_t)kLpStages * kLpStageBytes + (grouped ? sizeof(LpShared) : sizeof(LpShared) - 4 * 4 * (kLinExperts - 4));
}

struct LpMaps {
    CUtensorMap w;                                         // box 128 rows x 64 columns
    CUtensorMap x[4];                                      // boxes of 128, 64, 32, 16 tokens x 64 columns
};
struct LpArgs {
    LinArgs lin;
    const void *bias, *residual;
    long long ld_res;
    void *Y;
    long long ldy;
    int act;
    float *partial;                                        // [pairs][2][tokens of a tile][128]
    uint32_t wait_tries;
};

__device__ __forceinline__ uint32_t lp_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// the address of the leading CTA's copy of a shared-memory word
__device__ __forceinline__ uint32_t lp_leader(uint32_t addr) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ void lp_init_barrier(uint32_t bar, uint32_t arrivals) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(arrivals) : "memory");
}
// bounded wait; false when it gave up
__device__ __forceinline__ bool lp_wait(uint32_t bar, uint32_t parity, uint32_t tries) {
    for (uint32_t i = 0; i < tries; i++)
        if (mbar_try_wait_parity(bar, parity)) return true;
    return false;
}
// barrier of the epilogue warps; true when every thread says so
__device__ __forceinline__ bool lp_epilogue_all(bool mine) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)mine), "r"(kLpEpilogueWarps * 32)
        : "memory");
    return all != 0u;
}
__device__ __forceinline__ void lp_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void lp_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// K-major operand, 128-byte swizzle: rows 128 B apart, groups of 8 rows 1024 B apart
__device__ __forceinline__ uint64_t lp_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// D f32, A and B f16, both K-major, M = 256 over the pair
__device__ __forceinline__ uint32_t lp_idesc(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kLinRows >> 4) << 24);
}
__device__ __forceinline__ void lp_commit(uint32_t bar) {             // to this barrier of both CTAs
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(bar), "h"((unsigned short)3) : "memory");
}
__device__ __forceinline__ void lp_tmem_load(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}

// One unit of a pair's work: a tile, or one K split of it.
struct LpUnit {
    int expert, group;                        // weight's place in the stack, in the decoded weight
    int row0;                                 // first weight row of the tile (within the matrix, workspace order)
    int t0, t1, n;                            // tokens [t0, t1), columns of the accumulator
    int k0, k1;                               // K stages
    int split, slot, tile;                    // splits of the tile (1: whole), partial slot of this one, counter
};
template <bool GROUPED>
__device__ __forceinline__ LpUnit lp_unit(const LpArgs &a, const LpShared &H, int u, int nk) {
    LpUnit x;
    int tile = u, part = 0;
    x.split = 1;
    x.slot = x.tile = 0;
    if (u >= H.whole) {
        const int i = u - H.whole;
        x.split = H.split;
        x.tile = i / H.split;
        part = i - x.tile * H.split;
        x.slot = i;
        tile = H.whole + x.tile;
    }
    int g = 0, lo = 0, hi = (int)a.lin.tokens, local = tile;
    x.expert = 0;
    if (GROUPED) {
        int b = 0, e = H.nact;                // last group whose first tile is not beyond this one
        while (e - b > 1) {
            const int m = (b + e) >> 1;
            if (H.first[m] <= tile) b = m; else e = m;
        }
        g = b;
        lo = H.lo[g];
        hi = H.hi[g];
        local = tile - H.first[g];
        x.expert = H.id[g];
    }
    x.group = g;
    const int rt = (a.lin.rows + kLinRows - 1) / kLinRows;
    const int tt = (hi - lo + kLinTokens - 1) / kLinTokens;
    const int n = ((hi - lo + tt - 1) / tt + 31) & ~31;
    const int band = local / (kLpBand * tt), in_band = local - band * kLpBand * tt;
    const int width = min(kLpBand, rt - band * kLpBand);
    const int ti = in_band / width;
    x.row0 = (band * kLpBand + in_band - ti * width) * kLinRows;
    x.t0 = lo + ti * n;
    x.t1 = min(x.t0 + n, hi);
    x.n = (x.t1 - x.t0 + 31) & ~31;
    x.k0 = (int)((long long)nk * part / x.split);
    x.k1 = (int)((long long)nk * (part + 1) / x.split);
    return x;
}

// The outputs of N columns (tokens t ..) of this thread's weight row, from its accumulators.
template <bool GATED, class T, int N>
__device__ __forceinline__ void lp_outputs(const LpArgs &a, float (&z)[N], float row_scale, float bias, int t, int t1,
                                           int row, bool row_in, int lane) {
    const T *res = static_cast<const T *>(a.residual);
    T *Y = static_cast<T *>(a.Y);
    if (a.lin.stage == 2) {
#pragma unroll
        for (int c = 0; c < N; c++) {
            const float ts = t + c < t1 ? __ldg(a.lin.token_scale + t + c) : 0.f;
            z[c] = fmaf(z[c] * row_scale, ts, bias);
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; c++) z[c] = fmaf(z[c], row_scale, bias);
    }
    if constexpr (GATED) {
        // lanes 2 i and 2 i + 1 hold gate and up of output i: the even lane finishes the even tokens
        const bool up = lane & 1;
        float g[N / 2], m[N / 2];
#pragma unroll
        for (int c = 0; c < N / 2; c++) {
            const float mine = up ? z[2 * c + 1] : z[2 * c];
            const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? z[2 * c] : z[2 * c + 1], 1);
            g[c] = up ? got : mine;
            m[c] = up ? mine : got;
        }
        lin_activate(g, a.act);
        const long long o = row >> 1;
        const int tt = t + (int)up;
        float r[N / 2];
#pragma unroll
        for (int c = 0; c < N / 2; c++)
            r[c] = res && row_in && tt + 2 * c < t1 ? lin_load(res + (long long)(tt + 2 * c) * a.ld_res + o) : 0.f;
#pragma unroll
        for (int c = 0; c < N / 2; c++)
            if (row_in && tt + 2 * c < t1)
                Y[(long long)(tt + 2 * c) * a.ldy + o] = lin_round<T>(res ? fmaf(g[c], m[c], r[c]) : g[c] * m[c]);
    } else {
        lin_activate(z, a.act);
        if (res) {
            float r[N];
#pragma unroll
            for (int c = 0; c < N; c++) r[c] = row_in && t + c < t1 ? lin_load(res + (long long)(t + c) * a.ld_res + row) : 0.f;
#pragma unroll
            for (int c = 0; c < N; c++) z[c] += r[c];
        }
#pragma unroll
        for (int c = 0; c < N; c++)
            if (row_in && t + c < t1) Y[(long long)(t + c) * a.ldy + row] = lin_round<T>(z[c]);
    }
}

template <bool GROUPED, bool GATED, class T>
__global__ void __launch_bounds__(kLpThreads, 1) __cluster_dims__(2, 1, 1)
    k_linear_product(const __grid_constant__ LpMaps maps, const __grid_constant__ LpArgs a) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    LpShared &H = *reinterpret_cast<LpShared *>(smem_raw + (base - smem_u32(smem_raw)) + kLpStages * kLpStageBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = lp_rank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const uint32_t tries = a.wait_tries;
    const int nk = (a.lin.cols + kLpK - 1) / kLpK;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        for (int s = 0; s < kLpStages; s++) {
            lp_init_barrier(smem_u32(&H.full[s]), 1);
            lp_init_barrier(smem_u32(&H.empty[s]), 1);
        }
        for (int b = 0; b < 2; b++) {
            lp_init_barrier(smem_u32(&H.acc_full[b]), 1);
            lp_init_barrier(smem_u32(&H.acc_empty[b]), 2 * kLpEpilogueWarps);
        }
        lp_init_barrier(smem_u32(&H.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        H.abort = 0;
        H.nact = 1;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&H.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    // the decoded weight, the scales, the counters and the restated tokens are the first kernel's
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int rt = (a.lin.rows + kLinRows - 1) / kLinRows;
    if (warp == 0) {
        int tiles = 0;
        if (GROUPED) {
            const int n = max(lin_groups<true>(a.lin, H.id, H.lo, H.hi), 0);
            __syncwarp();
            for (int g0 = 0; g0 < n; g0 += 32) {              // tiles before each group
                const int g = g0 + lane;
                const int mine = g < n ? rt * ((H.hi[g] - H.lo[g] + kLinTokens - 1) / kLinTokens) : 0;
                int sum = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                    if (lane >= o) sum += v;
                }
                if (g < n) H.first[g] = tiles + sum - mine;
                tiles += __shfl_sync(0xFFFFFFFFu, sum, 31);
            }
            if (lane == 0) H.nact = n;
        } else {
            tiles = rt * (int)((a.lin.tokens + kLinTokens - 1) / kLinTokens);
        }
        if (lane == 0) {
            const int rest = tiles % pairs;
            H.tiles = tiles;
            H.whole = tiles - rest;
            H.split = rest ? max(1, min(pairs / rest, nk / kLpMinSplit)) : 1;
            H.units = H.whole + rest * H.split;
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    lp_cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = H.tmem;
    const int units = H.units;
    volatile int *abort_flag = &H.abort;

    if (warp == 0) {
        if (lane == 0) {
            // ---- loads of this CTA: its 128 weight rows and its half of the tokens, for the leader's barrier
            uint32_t it = 0;
            bool ok = true;
            for (int u = pair; u < units && ok; u += pairs) {
                const LpUnit x = lp_unit<GROUPED>(a, H, u, nk);
                const int half = x.n >> 1;
                const int wrow = x.group * a.lin.rows + x.row0 + 128 * (int)rank;
                const int trow = x.t0 + half * (int)rank;
                for (int k = x.k0; k < x.k1; k++, it++) {
                    const int s = it % kLpStages;
                    ok = lp_wait(smem_u32(&H.empty[s]), ((it / kLpStages) & 1u) ^ 1u, tries) && !*abort_flag;
                    if (!ok) break;
                    const uint32_t bar = lp_leader(smem_u32(&H.full[s]));
                    if (leader)
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                                     ::"r"(smem_u32(&H.full[s])), "r"((uint32_t)(2 * (kLpABytes + half * kLpK * 2))) : "memory");
                    const uint32_t st = base + s * kLpStageBytes;
                    lp_load(st, &maps.w, k * kLpK, wrow, bar);
                    uint32_t at = 0;
#pragma unroll
                    for (int b = 0; b < 4; b++) {
                        const int box = 128 >> b;
                        if (half & box) {
                            lp_load(st + kLpABytes + at * kLpK * 2, &maps.x[b], k * kLpK, trow + (int)at, bar);
                            at += box;
                        }
                    }
                }
            }
            // the last products' releases of the stages must have arrived before this CTA may leave
            for (uint32_t back = min(it, (uint32_t)kLpStages); ok && back > 0; back--) {
                const uint32_t i = it - back;
                ok = lp_wait(smem_u32(&H.empty[i % kLpStages]), (i / kLpStages) & 1u, tries);
            }
            if (!ok) *abort_flag = 1;
            // copies still under way after a wait gave up: the leader waits for the last of each stage
            if (leader && !ok)
                for (uint32_t back = 1; back <= (uint32_t)kLpStages && back <= it; back++) {
                    const uint32_t i = it - back;
                    lp_wait(smem_u32(&H.full[i % kLpStages]), (i / kLpStages) & 1u, kBulkWaitTries);
                }
        }
    } else if (warp == 1) {
        if (leader && lane == 0) {
            // ---- products: one thread issues for both CTAs
            uint32_t it = 0, tile = 0;
            bool ok = true;
            for (int u = pair; u < units && ok; u += pairs, tile++) {
                const LpUnit x = lp_unit<GROUPED>(a, H, u, nk);
                const uint32_t b = tile & 1u;
                ok = lp_wait(smem_u32(&H.acc_empty[b]), ((tile >> 1) & 1u) ^ 1u, tries);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t idesc = lp_idesc(x.n), d = tmem + b * kLinTokens;
                for (int k = x.k0; k < x.k1; k++, it++) {
                    const int s = it % kLpStages;
                    ok = lp_wait(smem_u32(&H.full[s]), (it / kLpStages) & 1u, tries) && !*abort_flag;
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint64_t ad = lp_desc(base + s * kLpStageBytes), bd = lp_desc(base + s * kLpStageBytes + kLpABytes);
#pragma unroll
                    for (int q = 0; q < kLpK / 16; q++)       // 16 columns are 32 bytes along the swizzled row
                        asm volatile(
                            "{\n\t.reg .pred p;\n\t"
                            "setp.ne.b32 p, %4, 0;\n\t"
                            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                            ::"r"(d), "l"(ad + 2 * q), "l"(bd + 2 * q), "r"(idesc), "r"((uint32_t)(k > x.k0 || q > 0)));
                    lp_commit(smem_u32(&H.empty[s]));
                }
                if (ok) lp_commit(smem_u32(&H.acc_full[b]));
            }
            if (!ok) {
                // products under way read shared memory and write TMEM: wait for them before leaving
                *abort_flag = 1;
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                             ::"r"(smem_u32(&H.drain)) : "memory");
                if (!lp_wait(smem_u32(&H.drain), 0, kBulkWaitTries)) *abort_flag = 2;
            }
        }
    } else {
        // ---- epilogue: warp quarter (TMEM lanes) and which of the 32-column chunks
        const int quarter = warp & 3, odd = (warp - 2) >> 2;
        const int lrow = quarter * 32 + lane;                  // row within the CTA's 128
        const uint32_t tlane = tmem + ((uint32_t)(quarter * 32) << 16);
        uint32_t tile = 0;
        bool ok = true;
        for (int u = pair; u < units; u += pairs, tile++) {
            const LpUnit x = lp_unit<GROUPED>(a, H, u, nk);
            const uint32_t b = tile & 1u;
            const int row = x.row0 + 128 * (int)rank + lrow;   // in workspace order
            const bool row_in = row < a.lin.rows;
            float rs = 0.f, bias = 0.f;
            if (row_in) {
                rs = __ldg(a.lin.row_scale + (long long)x.group * a.lin.rows + row);
                if (a.bias)
                    bias = lin_load(static_cast<const T *>(a.bias) + (long long)x.expert * a.lin.rows +
                                    (GATED ? (row >> 1) + (row & 1) * a.lin.half : row));
            }
            // all epilogue warps go on, or none (they meet at a barrier again when a tile is split)
            ok = lp_wait(smem_u32(&H.acc_full[b]), (tile >> 1) & 1u, tries) && !*abort_flag;
            ok = lp_epilogue_all(ok);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            float *slot = x.split > 1 ? a.partial + ((long long)x.slot * 2 + rank) * kLinTokens * 128 : nullptr;
            for (int c0 = odd * 32; c0 < x.n; c0 += 64) {
                uint32_t v[32];
                lp_tmem_load(tlane + b * kLinTokens + c0, v);
                if (slot) {
#pragma unroll
                    for (int c = 0; c < 32; c++) __stcg(slot + (c0 + c) * 128 + lrow, __uint_as_float(v[c]));
                } else {
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        float z[16];
#pragma unroll
                        for (int c = 0; c < 16; c++) z[c] = __uint_as_float(v[16 * h + c]);
                        if (x.t0 + c0 + 16 * h < x.t1)
                            lp_outputs<GATED, T>(a, z, rs, bias, x.t0 + c0 + 16 * h, x.t1, row, row_in, lane);
                    }
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                             ::"r"(lp_leader(smem_u32(&H.acc_empty[b]))) : "memory");
            if (x.split > 1) {
                // this CTA's half of the tile: whoever arrives last adds the splits, in their order
                __threadfence();
                lp_epilogue_all(true);
                if (tid == 64) H.last = atomicAdd(a.lin.counters + x.tile * 2 + rank, 1u) == (unsigned)(x.split - 1);
                lp_epilogue_all(true);
                if (H.last) {
                    __threadfence();
                    const float *first = a.partial + ((long long)x.tile * x.split * 2 + rank) * kLinTokens * 128;
                    for (int c0 = odd * 16; c0 < x.n && x.t0 + c0 < x.t1; c0 += 32) {
                        float z[16];
#pragma unroll
                        for (int c = 0; c < 16; c++) z[c] = 0.f;
                        for (int p = 0; p < x.split; p++) {
                            const float *src = first + (long long)p * 2 * kLinTokens * 128 + c0 * 128 + lrow;
#pragma unroll
                            for (int c = 0; c < 16; c++) z[c] += __ldcg(src + c * 128);
                        }
                        lp_outputs<GATED, T>(a, z, rs, bias, x.t0 + c0, x.t1, row, row_in, lane);
                    }
                }
            }
        }
        if (!ok && lane == 0) *abort_flag = 1;
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && H.abort) atomicOr(a.lin.flags, LLVQ_FLAG_WAIT_TIMEOUT);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    lp_cluster_sync();                                         // the peer's barriers and tiles are no longer used
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    // products that would not end keep their columns rather than have them freed underneath
    if (warp == 1 && H.abort != 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

}  // namespace llvq
