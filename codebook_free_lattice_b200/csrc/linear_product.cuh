// linear_product.cuh -- the second kernel of a compressed linear layer: the decoded fp16 weight times
// every token on the 5th-generation tensor cores, with bias, activation, gating and residual in the
// epilogue (linear_common.cuh states the operator and its scales).
//
// Two CTAs of a cluster share one tile of 256 weight rows x up to 256 tokens (tcgen05.mma,
// cta_group::2): the weight rows are the M side, 128 per CTA, so that bias and row scale are one value
// per thread and the number of tokens, which varies, is the N side in steps of 32.  Each CTA loads its
// 128 weight rows and its half of the tokens (TMA, 128-byte swizzle, 64 columns of K per stage); fp32
// accumulators sit in both CTAs' TMEM, two sets of 256 columns, so that one tile's epilogue runs under
// the next tile's products.  Warp 0 loads, warp 1 of the leading CTA issues the products, warps 2 to 17
// run the epilogue.
//
// A persistent grid walks the tiles of all groups.  Tiles that do not fill a last round of pairs are
// split along K over the idle pairs; partial sums go through the workspace, and whichever pair brings the
// last part of a chunk of 16 columns adds its parts in the order of the splits, so results do not
// depend on timing and the adding spreads over the pairs.
#pragma once
#include <cuda.h>
#include "linear_common.cuh"

namespace llvq {

constexpr int kLpEpilogueWarps = 16;                       // four per quarter of the TMEM lanes
constexpr int kLpEach = kLpEpilogueWarps / 4;              // a warp takes every fourth chunk of 16 columns
constexpr int kLpThreads = 32 * (2 + kLpEpilogueWarps);
constexpr int kLpStages = 6;
constexpr int kLpK = 64;                                   // columns of K per stage: one 128-byte swizzle row
constexpr int kLpABytes = 128 * kLpK * 2;                  // 128 weight rows
constexpr int kLpBBytes = kLinTokens / 2 * kLpK * 2;       // up to 128 tokens
constexpr int kLpStageBytes = kLpABytes + kLpBBytes;
constexpr int kLpBand = 8;                                 // row tiles of a band (L2 reuse of the tokens)
constexpr int kLpMinSplit = 4;                             // least K stages of a split
constexpr int kLpCounters = 2 * 4 * 16;                    // per split tile: CTA, warp quarter, chunk of 16 columns

struct LpShared {
    unsigned long long full[kLpStages], empty[kLpStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort, nact;
    uint32_t issued, bytes[kLpStages];                     // stages that this CTA has loaded, and of how many bytes
    int whole, split, units, cap;
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
    float *partial;                                        // [pairs][2][tokens of a tile / 4][128][4]
    uint32_t wait_tries;
};

// One lane of a converged warp.  The loading and the issuing warp run their loops whole and with values
// that are uniform over the warp, and elect a lane for the instructions themselves: under a plain
// `lane == 0` the operands, which these instructions take from uniform registers, cost several times as much to
// bring there (0.43 us per stage of 64 columns instead of what the products take).
__device__ __forceinline__ bool lp_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int lp_uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
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
// A wait gave up: both CTAs are to stop.
__device__ __forceinline__ uint32_t lp_peer(uint32_t addr) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(lp_rank() ^ 1u));
    return r;
}
__device__ __forceinline__ void lp_abort(LpShared &H) {
    *(volatile int *)&H.abort = 1;
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(lp_peer(smem_u32(&H.abort))), "r"(1) : "memory");
}
__device__ __forceinline__ uint32_t lp_of_peer(const uint32_t &word) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(lp_peer(smem_u32(&word))) : "memory");
    return v;
}
// bounded wait; false when it gave up
__device__ __forceinline__ bool lp_wait(uint32_t bar, uint32_t parity, uint32_t tries) {
    for (uint32_t i = 0; i < tries; i++)
        if (mbar_try_wait_parity(bar, parity)) return true;
    return false;
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
__device__ __forceinline__ void lp_tmem_load(uint32_t addr, float (&z)[16]) {
    uint32_t v[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
#pragma unroll
    for (int c = 0; c < 16; c++) z[c] = __uint_as_float(v[c]);
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
__device__ __noinline__ LpUnit lp_unit(const LpArgs &a, const LpShared &H, int u, int nk) {
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
    const int tt = (hi - lo + H.cap - 1) / H.cap;
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

// The time of a call's tiles of at most `cap` tokens, in ns, and how many ways its last tiles are split.
// Measured on 74 pairs: a stage of 64 columns takes 0.33 us with 256 tokens and no less than 0.27 us; the
// epilogue 0.6 us and 0.3 us per 32 tokens, under the next tile's products but for the last; parts of a split
// tile 3 us and 0.4 us per 32 tokens more.  Whole tiles go in rounds of all pairs, the rest is split along K while pairs would idle.
__host__ __device__ __forceinline__ int lp_cost(int tiles, int cap, int pairs, int nk, int &split) {
    const int stage = max(270, 330 * cap / kLinTokens), ends = 600 + 10 * cap;
    const int rest = tiles % pairs;
    long long ns = (long long)(tiles / pairs) * max(nk * stage, ends) + ends;
    split = 1;
    if (rest) {
        const int ways = max(1, min(pairs / rest, nk / kLpMinSplit));
        const int whole = nk * stage, parts = (nk + ways - 1) / ways * stage + 3000 + 12 * cap;
        split = parts < whole ? ways : 1;
        ns += min(whole, parts);
    }
    return (int)min(ns, 0x7FFFFFFFll);
}
// The tile size of a call, by one warp: tokens[g] of n groups (in shared memory; or `all` tokens of one).  More
// and smaller tiles fill idle pairs and shorten the last epilogue, larger ones feed the tensor cores better.
template <bool GROUPED>
__device__ __forceinline__ void lp_schedule(LpShared &H, int n, int all, int rt, int pairs, int nk) {
    const int lane = threadIdx.x & 31, cap = 32 * ((lane & 7) + 1);         // lane i: tiles of 32 (i + 1) tokens
    int tiles = 0;
    if (GROUPED) {
        for (int g = lane >> 3; g < n; g += 4) tiles += (H.hi[g] - H.lo[g] + cap - 1) / cap;
        tiles += __shfl_xor_sync(0xFFFFFFFFu, tiles, 8);
        tiles += __shfl_xor_sync(0xFFFFFFFFu, tiles, 16);
    } else {
        tiles = (all + cap - 1) / cap;
    }
    tiles *= rt;
    int split;
    const int ns = lp_cost(tiles, cap, pairs, nk, split);
    const unsigned best = __ballot_sync(0xFFFFFFFFu, ns == __reduce_min_sync(0xFFFFFFFFu, ns)) & 0xFFu;
    if (lane == 31 - __clz(best)) {                           // larger tiles where times are equal
        H.cap = cap;
        H.split = split;
        H.whole = tiles - tiles % pairs;
        H.units = H.whole + tiles % pairs * split;
    }
    __syncwarp();
}

// What a chunk of 16 columns (tokens t .. t1 - 1 of them) needs from memory besides its accumulators: the
// residual of this thread's row, and the tokens' scales, one per lane.  Loaded a chunk ahead.
template <bool GATED, class T>
struct LpEnds {
    static constexpr int N = GATED ? 8 : 16;
    T res[N];
    float scale;
};
// tokens of a chunk that this thread writes, from its first one: n of them (0 for a row beyond the weight),
// for a gated weight every other token (lanes 2 i and 2 i + 1 share the outputs of row pair i)
template <bool GATED>
__device__ __forceinline__ int lp_count(int t, int t1, bool row_in, int lane) {
    const int n = row_in ? t1 - t : 0;
    return GATED ? (n + 1 - (lane & 1)) >> 1 : n;
}
template <bool GATED, class T>
__device__ __forceinline__ void lp_load_ends(const LpArgs &a, LpEnds<GATED, T> &e, int t, int t1, int row, bool row_in, int lane) {
    if (a.residual) {
        const int n = lp_count<GATED>(t, t1, row_in, lane);
        const T *res = static_cast<const T *>(a.residual) + (long long)(t + (GATED ? lane & 1 : 0)) * a.ld_res + (GATED ? row >> 1 : row);
        const long long step = (GATED ? 2 : 1) * a.ld_res;
#pragma unroll
        for (int c = 0; c < LpEnds<GATED, T>::N; c++) {
            e.res[c] = c < n ? *res : T(0.f);
            res += step;
        }
    }
    if (a.lin.stage == 2) e.scale = lane < min(16, t1 - t) ? __ldcg(a.lin.token_scale + t + lane) : 0.f;
}

// The outputs of a chunk of this thread's weight row, from its accumulators.  Addresses step from token to
// token and a count tells which are written: with a comparison and a product per column the code is three
// times as slow.
template <bool GATED, class T>
__device__ __forceinline__ void lp_outputs(const LpArgs &a, float (&z)[16], const LpEnds<GATED, T> &e, float row_scale, float bias,
                                           int t, int t1, int row, bool row_in, int lane) {
    constexpr int N = LpEnds<GATED, T>::N;
    if (a.lin.stage == 2) {
#pragma unroll
        for (int c = 0; c < 16; c++) z[c] = fmaf(z[c] * row_scale, __shfl_sync(0xFFFFFFFFu, e.scale, c), bias);
    } else {
#pragma unroll
        for (int c = 0; c < 16; c++) z[c] = fmaf(z[c], row_scale, bias);
    }
    float y[N];
    if constexpr (GATED) {
        // lanes 2 i and 2 i + 1 hold gate and up of output i: the even lane finishes the even tokens
        const bool up = lane & 1;
        float m[N];
#pragma unroll
        for (int c = 0; c < N; c++) {
            const float mine = up ? z[2 * c + 1] : z[2 * c];
            const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? z[2 * c] : z[2 * c + 1], 1);
            y[c] = up ? got : mine;
            m[c] = up ? mine : got;
        }
        lin_activate(y, a.act);
#pragma unroll
        for (int c = 0; c < N; c++) y[c] *= m[c];
    } else {
#pragma unroll
        for (int c = 0; c < N; c++) y[c] = z[c];
        lin_activate(y, a.act);
    }
    if (a.residual) {
#pragma unroll
        for (int c = 0; c < N; c++) y[c] += lin_float(e.res[c]);
    }
    const int n = lp_count<GATED>(t, t1, row_in, lane);
    T *out = static_cast<T *>(a.Y) + (long long)(t + (GATED ? lane & 1 : 0)) * a.ldy + (GATED ? row >> 1 : row);
    const long long step = (GATED ? 2 : 1) * a.ldy;
#pragma unroll
    for (int c = 0; c < N; c++) {
        if (c < n) *out = lin_round<T>(y[c]);
        out += step;
    }
}

template <bool GROUPED, bool GATED, class T>
__global__ void __launch_bounds__(kLpThreads, 1) __cluster_dims__(2, 1, 1)
    k_linear_product(const __grid_constant__ LpMaps maps, const __grid_constant__ LpArgs a) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    LpShared &H = *reinterpret_cast<LpShared *>(smem_raw + (base - smem_u32(smem_raw)) + kLpStages * kLpStageBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const uint32_t rank = lp_rank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const uint32_t tries = a.wait_tries;
    const int nk = (a.lin.terms + kLpK - 1) / kLpK;

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
    const int rt = (a.lin.rows + kLinRows - 1) / kLinRows;
    if (warp == 0) {
        if (lane < 5) asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &maps.w : &maps.x[lane - 1]) : "memory");
        if (!GROUPED) lp_schedule<false>(H, 1, (int)a.lin.tokens, rt, pairs, nk);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    lp_cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    // the decoded weight, the scales, the counters and the restated tokens are the first kernel's
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (GROUPED) {
        if (warp == 0) {
            const int n = max(lin_groups<true>(a.lin, kLinExperts, H.id, H.lo, H.hi), 0);
            __syncwarp();
            lp_schedule<true>(H, n, 0, rt, pairs, nk);
            const int cap = H.cap;
            int tiles = 0;
            for (int g0 = 0; g0 < n; g0 += 32) {              // tiles before each group
                const int g = g0 + lane;
                const int mine = g < n ? rt * ((H.hi[g] - H.lo[g] + cap - 1) / cap) : 0;
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
        }
        __syncthreads();
    }
    const uint32_t tmem = H.tmem;
    const int units = H.units;
    volatile int *abort_flag = &H.abort;

    if (warp == 0) {
        // ---- loads of this CTA: its 128 weight rows and its half of the tokens, for the leader's barrier
        const uint32_t full0 = lp_uniform((int)lp_leader(smem_u32(&H.full[0]))), empty0 = smem_u32(&H.empty[0]);
        uint32_t s = 0, phase = 1, issued = 0;
        bool ok = true;
        for (int u = pair; u < units && ok; u += pairs) {
            const LpUnit x = lp_unit<GROUPED>(a, H, u, nk);
            const int half = lp_uniform(x.n >> 1), k1 = lp_uniform(x.k1);
            const int wrow = lp_uniform(x.group * a.lin.rows + x.row0 + 128 * (int)rank);
            const int trow = lp_uniform(x.t0 + half * (int)rank);
            const uint32_t bytes = (uint32_t)(kLpABytes + half * kLpK * 2);          // of each CTA
            for (int k = lp_uniform(x.k0); k < k1; k++) {
                ok = lp_wait(empty0 + 8 * s, phase, tries);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                const uint32_t st = base + s * kLpStageBytes, bar = full0 + 8 * s;
                if (lp_elect()) {
                    if (leader)
                        asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(2u * bytes) : "memory");
                    H.bytes[s] = bytes;
                    lp_load(st, &maps.w, k * kLpK, wrow, bar);
                    if (half == 128) {
                        lp_load(st + kLpABytes, &maps.x[0], k * kLpK, trow, bar);
                    } else {
                        int at = 0;
#pragma unroll
                        for (int b = 1; b < 4; b++) {
                            if (half & (128 >> b)) {
                                lp_load(st + kLpABytes + at * kLpK * 2, &maps.x[b], k * kLpK, trow + at, bar);
                                at += 128 >> b;
                            }
                        }
                    }
                }
                __syncwarp();
                issued++;
                if (++s == kLpStages) { s = 0; phase ^= 1u; }
            }
        }
        // the last products' releases of the stages must have arrived before this CTA may leave
        for (uint32_t back = min(issued, (uint32_t)kLpStages); ok && back > 0; back--) {
            const uint32_t i = issued - back;
            ok = lp_wait(empty0 + 8 * (i % kLpStages), (i / kLpStages) & 1u, tries);
        }
        if (lane == 0) {
            H.issued = issued;
            if (!ok) lp_abort(H);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            // ---- products: one thread issues for both CTAs
            const uint32_t full0 = smem_u32(&H.full[0]), empty0 = smem_u32(&H.empty[0]);
            const uint32_t tmem0 = lp_uniform((int)tmem);
            uint32_t s = 0, phase = 0, tile = 0;
            bool ok = true;
            for (int u = pair; u < units && ok; u += pairs, tile++) {
                const LpUnit x = lp_unit<GROUPED>(a, H, u, nk);
                const uint32_t b = tile & 1u;
                ok = lp_wait(smem_u32(&H.acc_empty[b]), ((tile >> 1) & 1u) ^ 1u, tries);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t idesc = lp_idesc(lp_uniform(x.n)), d = tmem0 + b * kLinTokens;
                const int k0 = lp_uniform(x.k0), k1 = lp_uniform(x.k1);
                for (int k = k0; k < k1; k++) {
                    ok = lp_wait(full0 + 8 * s, phase, tries);
                    if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint64_t ad = lp_desc(base + s * kLpStageBytes), bd = lp_desc(base + s * kLpStageBytes + kLpABytes);
                    if (lp_elect()) {
#pragma unroll
                        for (int q = 0; q < kLpK / 16; q++)       // 16 columns are 32 bytes along the swizzled row
                            asm volatile(
                                "{\n\t.reg .pred p;\n\t"
                                "setp.ne.b32 p, %4, 0;\n\t"
                                "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                                ::"r"(d), "l"(ad + 2 * q), "l"(bd + 2 * q), "r"(idesc), "r"((uint32_t)(k > k0 || q > 0)));
                        lp_commit(empty0 + 8 * s);
                    }
                    __syncwarp();
                    if (++s == kLpStages) { s = 0; phase ^= 1u; }
                }
                if (ok && lp_elect()) lp_commit(smem_u32(&H.acc_full[b]));
                __syncwarp();
            }
            if (!ok) {
                // products under way read shared memory and write TMEM: wait for them before leaving
                if (lane == 0) lp_abort(H);
                __syncwarp();
                if (lp_elect())
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                                 ::"r"(smem_u32(&H.drain)) : "memory");
                __syncwarp();
                lp_wait(smem_u32(&H.drain), 0, kBulkWaitTries);
            }
        }
    } else {
        // ---- epilogue: warp quarter (TMEM lanes) and which of the chunks
        const int quarter = warp & 3, part = (warp - 2) >> 2;
        const int lrow = quarter * 32 + lane;                  // row within the CTA's 128
        const uint32_t tlane = tmem + ((uint32_t)(quarter * 32) << 16);
        uint32_t tile = 0;
        bool ok = true;
        // a tile, and the scale and bias of this thread's row in it
        auto load_row = [&](const LpUnit &x, float &rs, float &bias) {
            const int row = x.row0 + 128 * (int)rank + lrow;   // in workspace order
            rs = bias = 0.f;
            if (row < a.lin.rows) {
                rs = __ldcg(a.lin.row_scale + (long long)x.group * a.lin.rows + row);
                if (a.bias)
                    bias = lin_load(static_cast<const T *>(a.bias) + (long long)x.expert * a.lin.rows +
                                    (GATED ? (row >> 1) + (row & 1) * a.lin.half : row));
            }
        };
        LpUnit next{};
        float next_rs = 0.f, next_bias = 0.f;
        if (pair < units) {
            next = lp_unit<GROUPED>(a, H, pair, nk);
            load_row(next, next_rs, next_bias);
        }
        for (int u = pair; u < units; u += pairs, tile++) {
            const LpUnit x = next;
            const float rs = next_rs, bias = next_bias;
            const uint32_t b = tile & 1u;
            const int row = x.row0 + 128 * (int)rank + lrow;
            const bool row_in = row < a.lin.rows;
            ok = lp_wait(smem_u32(&H.acc_full[b]), (tile >> 1) & 1u, tries) && !*abort_flag;
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (u + pairs < units) {                           // the next tile's row, on its way during this one
                next = lp_unit<GROUPED>(a, H, u + pairs, nk);
                load_row(next, next_rs, next_bias);
            }
            // this warp's chunks of 16 columns: part, part + kLpEach, ...
            const int chunks = (x.t1 - x.t0 + 15) >> 4;
            const uint32_t acc = tlane + b * kLinTokens;
            uint32_t mine = 0xFFFFFFFFu;                       // chunks to finish here
            const float4 *parts = nullptr;
            if (x.split > 1) {
                // partial sums to the workspace, four columns of a row together; whichever split of a
                // chunk arrives last finishes it
                float4 *own = reinterpret_cast<float4 *>(a.partial) + ((long long)x.slot * 2 + rank) * (kLinTokens * 32) + lrow;
                for (int c = part; c < chunks; c += kLpEach) {
                    float z[16];
                    lp_tmem_load(acc + 16 * c, z);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        __stcg(own + (4 * c + i) * 128, make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]));
                }
                __threadfence();
                __syncwarp();
                unsigned before = 0;
                const int c = kLpEach * lane + part;
                if (lane < 16 / kLpEach && c < chunks) before = atomicAdd(a.lin.counters + ((x.tile * 2 + rank) * 4 + quarter) * 16 + c, 1u);
                mine = __ballot_sync(0xFFFFFFFFu, lane < 16 / kLpEach && c < chunks && before == (unsigned)(x.split - 1));
                __threadfence();
                parts = reinterpret_cast<const float4 *>(a.partial) +
                        ((long long)x.tile * x.split * 2 + rank) * (kLinTokens * 32) + lrow;
            }
            mine &= (1u << ((chunks - part + kLpEach - 1) / kLpEach)) - 1u;
            LpEnds<GATED, T> ends;
            if (mine) lp_load_ends<GATED, T>(a, ends, x.t0 + 16 * (kLpEach * (__ffs(mine) - 1) + part), x.t1, row, row_in, lane);
            while (mine) {
                const int c = kLpEach * (__ffs(mine) - 1) + part;
                mine &= mine - 1u;
                float z[16];
                if (x.split > 1) {
#pragma unroll
                    for (int i = 0; i < 16; i++) z[i] = 0.f;
#pragma unroll 4
                    for (int p = 0; p < x.split; p++) {        // in the order of the splits
                        const float4 *src = parts + (long long)p * 2 * (kLinTokens * 32) + 4 * c * 128;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const float4 q = __ldcg(src + i * 128);
                            z[4 * i] += q.x;
                            z[4 * i + 1] += q.y;
                            z[4 * i + 2] += q.z;
                            z[4 * i + 3] += q.w;
                        }
                    }
                } else {
                    lp_tmem_load(acc + 16 * c, z);
                }
                const LpEnds<GATED, T> now = ends;
                if (mine) lp_load_ends<GATED, T>(a, ends, x.t0 + 16 * (kLpEach * (__ffs(mine) - 1) + part), x.t1, row, row_in, lane);
                lp_outputs<GATED, T>(a, z, now, rs, bias, x.t0 + 16 * c, x.t1, row, row_in, lane);
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];"
                             ::"r"(lp_leader(smem_u32(&H.acc_empty[b]))) : "memory");
        }
        if (!ok && lane == 0) lp_abort(H);
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && H.abort) atomicOr(a.lin.flags, LLVQ_FLAG_WAIT_TIMEOUT);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    lp_cluster_sync();                                         // the peer's barriers and tiles are no longer used
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (*abort_flag) {
        // Copies may still be under way to either CTA, which may not leave before them.  They are counted by the
        // leader's barriers; where one CTA has loaded a stage and the other has not, the barrier is told so.  (Neither
        // is ever more than a ring of stages ahead: a slot is free once the products have used both CTAs' tiles.)
        if (leader && warp == 0) {
            const uint32_t mine = H.issued, theirs = lp_of_peer(H.issued), last = max(mine, theirs);
            if (lane == 0) {
                for (uint32_t i = mine; i < theirs; i++)
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                                 ::"r"(smem_u32(&H.full[i % kLpStages])), "r"(lp_of_peer(H.bytes[i % kLpStages])) : "memory");
                for (uint32_t i = theirs; i < mine; i++)
                    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;"
                                 ::"r"(smem_u32(&H.full[i % kLpStages])), "r"(H.bytes[i % kLpStages]) : "memory");
            }
            __syncwarp();
            for (uint32_t i = last - min(last, (uint32_t)kLpStages); i < last; i++)
                lp_wait(smem_u32(&H.full[i % kLpStages]), (i / kLpStages) & 1u, kBulkWaitTries);
        }
        lp_cluster_sync();
    }
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

}  // namespace llvq
