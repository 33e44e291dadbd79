// linear_dequant.cuh -- the first kernel of a compressed linear layer: every block of the experts
// that have tokens is decoded once, and written as 24 scaled fp16 weights (linear_common.cuh; a gated fp16
// layer's in two parts) or, for a few tokens, multiplied with them at once (k_linear_finish then adds each row's dot
// products in order).
//
// "Leech Lattice Vector Quantization for Efficient LLM Compression", papernotes.org notes,
// 方法详解 / 关键设计 2: index -> shell, class, codeword, signs, arrangement -> integer vector.
//
// Integer work bounds it: about 700 thread instructions per 48-bit block, against 8 bytes read and 48 written (or 96,
// in three stores of 32 bytes: 18944 x 8192 in 211 us against 188 for 48 bytes in three of 16; six of 16 took 344).
// Each CTA takes an equal run of blocks (not of rows: a run may begin and end inside a row, so few long rows still
// spread over all SMs).  48-bit blocks use the warp-private rings of the fused GEMV
// (kernels_gemv48.cuh): a warp classifies 32 consecutive blocks, sorts them by coset into two rings and
// decodes a ring once it holds 32, so that all lanes run the same decode.
#pragma once
#include "codec72.cuh"
#include "codec96.cuh"
#include "linear_common.cuh"

namespace llvq {

constexpr int kDqThreads = 1024;
constexpr int kDqWarps = kDqThreads / 32;
constexpr int kDqRing = 64;                   // records per ring (a warp drains a ring at 32)
constexpr int kDqRare = 64;                   // records of rare classes kept to the end
constexpr int kDqAhead = 64;                  // slices between the words read and the words prefetched
using DqRec = uint4;                          // like BinRec: x, y, z the digits, w = local row | block << 16

struct DqShared {
    int slice_next, stage_next, nact, nrare;
    unsigned long long bar;
    unsigned long long pad2;
    int left[2][32], head[2][32];             // what the rings hold at the end, and where
    uint4 rare[kDqRare];                      // blocks of the rare classes, decoded at the end
    int id[kLinExperts];                      // the active experts (weights), or DqDots in this place (dots)
};
// Few tokens: the activations as fp16, one row of nb * 24 values per token (zero beyond the columns), follow, or are
// in the workspace where they do not fit (kDqDotsFar: restated by k_linear_stage, read through L1).
struct DqDots {
    int id[kLinDots], lo[kLinDots], hi[kLinDots];
    uint32_t top[kLinDots];
    float scale[kLinDots];
};
enum DqOut { kDqWeights = 0, kDqDots = 1, kDqDotsFar = 2, kDqTwoParts = 3 };
__host__ __device__ constexpr bool dq_weights(int out) { return out == kDqWeights || out == kDqTwoParts; }
constexpr size_t kDqHead = 32 + 4 * 32 * sizeof(int) + kDqRare * sizeof(uint4);              // DqShared without its list
__host__ __device__ constexpr size_t dq_tail(int out, bool grouped, long long tokens, int nb) {
    return kDqHead + (out == kDqDots ? sizeof(DqDots) + (size_t)tokens * nb * 48
                      : out == kDqDotsFar ? sizeof(DqDots) : grouped ? sizeof(int) * kLinExperts : 0);
}
__host__ __device__ constexpr size_t dq48_fixed() { return sizeof(SmemGv48) + sizeof(DqRec) * (kDqWarps * 2 * kDqRing); }
template <class D>
__host__ __device__ constexpr size_t dq_fixed() { return (sizeof(typename D::Smem) + 15) / 16 * 16; }

// The run of blocks of one CTA, counted through the active experts' rows in order.
struct DqRun {
    int total;                                // blocks
    int first;                                // block of its first row where it begins
    int row0, nrows;                          // active rows it touches
};
__device__ __forceinline__ DqRun dq_run(const LinArgs &a, int nact) {
    DqRun r{0, 0, 0, 0};
    const long long all = (long long)nact * a.rows * a.nb;
    // whole warps of blocks, so that only the last CTA has a partial slice
    const long long per = ((all + gridDim.x - 1) / gridDim.x + 31) / 32 * 32;
    const long long b0 = min(all, per * blockIdx.x), b1 = min(all, b0 + per);
    if (b1 <= b0) return r;
    r.total = (int)(b1 - b0);
    r.row0 = (int)(b0 / a.nb);
    r.first = (int)(b0 - (long long)r.row0 * a.nb);
    r.nrows = (int)((b1 - 1) / a.nb) - r.row0 + 1;
    return r;
}

// Where an active row lives: its row of the stacked weight and its row of the workspace.
template <bool GROUPED>
__device__ __forceinline__ void dq_row(const LinArgs &a, const int *id, int active, long long &src, long long &dst) {
    if (GROUPED) {
        const int e = (int)div_by((uint32_t)active, (uint32_t)a.rows, a.rows_recip);
        const int r = active - e * a.rows;
        src = (long long)id[e] * a.rows + r;
        dst = (long long)e * a.rows + lin_place(r, a.half);
    } else {
        src = active;
        dst = lin_place(active, a.half);
    }
}

// What fp16(scale) leaves of a block's scale; nothing of an infinite one (the difference would be a NaN).
__device__ __forceinline__ __half dq_rest(float scale, __half hi) {
    return __float2half_rn(fabsf(scale) <= 65504.f ? scale - __half2float(hi) : 0.f);
}

// 24 integers (12 exact fp16 pairs) times the block's scale, each rounded once to fp16.  Direct gains
// times a power of two are fp16 values, one product.  A table gain over |v| is not: its rounding
// error goes in as a second factor, w = v s_hi + (v s_lo), so that the sum is rounded once.
template <int GAIN>
__device__ __forceinline__ void dq_store(const uint32_t wh[12], float scale, __half *out) {
    const __half hi = __float2half_rn(scale);
    const __half2 hi2 = __halves2half2(hi, hi);
    const __half lo = dq_rest(scale, hi);
    const __half2 lo2 = __halves2half2(lo, lo);
    uint32_t o[12];
#pragma unroll
    for (int q = 0; q < 12; q++) {
        const __half2 v = *reinterpret_cast<const __half2 *>(&wh[q]);
        const __half2 w = GAIN == 0 ? __hmul2(v, hi2) : __hfma2(v, hi2, __hmul2(v, lo2));
        o[q] = *reinterpret_cast<const uint32_t *>(&w);
    }
    uint4 *p = reinterpret_cast<uint4 *>(out);
    p[0] = make_uint4(o[0], o[1], o[2], o[3]);
    p[1] = make_uint4(o[4], o[5], o[6], o[7]);
    p[2] = make_uint4(o[8], o[9], o[10], o[11]);
}
// 32 bytes at once (32-byte aligned)
__device__ __forceinline__ void dq_store32(__half *out, const uint32_t *o) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(out), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]) : "memory");
}
// The same weights in two parts, fp16(w) and fp16(w - fp16(w)): v s_hi - fp16(w) is a multiple of s_hi's last place and
// at most a few of fp16(w)'s, so it is exact, and v s_lo joins it with one rounding.  An infinite gain has no rest.
// values: coordinates of the block that are columns of the layer.
template <int GAIN>
__device__ __forceinline__ void dq_store_two(const uint32_t wh[12], float scale, int values, __half *out) {
    const __half hi = __float2half_rn(scale);
    const __half2 hi2 = __halves2half2(hi, hi);
    const __half lo = dq_rest(scale, hi);
    const __half2 lo2 = __halves2half2(lo, lo);
    const bool finite = fabsf(scale) <= 65504.f;
    uint32_t o[24];
#pragma unroll
    for (int q = 0; q < 12; q++) {
        const __half2 v = *reinterpret_cast<const __half2 *>(&wh[q]);
        const __half2 w = GAIN == 0 ? __hmul2(v, hi2) : __hfma2(v, hi2, __hmul2(v, lo2));
        __half2 rest = __hfma2(v, hi2, __hneg2(w));
        if (GAIN != 0) rest = __hfma2(v, lo2, rest);
        o[q] = *reinterpret_cast<const uint32_t *>(&w);
        o[12 + q] = finite ? *reinterpret_cast<const uint32_t *>(&rest) : 0u;
    }
#pragma unroll
    for (int i = 0; i < 3; i++) dq_store32(out + 16 * i, o + 8 * i);
    // coordinates beyond the columns meet zeros, which an infinity would make a NaN
    if (!finite)
        for (int i = values; i < 24; i++) out[i] = __float2half_rn(0.f);
}
template <int PARTS>
__device__ __forceinline__ void dq_store_zero(__half *out) {
    uint4 *p = reinterpret_cast<uint4 *>(out);
#pragma unroll
    for (int i = 0; i < 3 * PARTS; i++) p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// A block's dot products with the tokens of its expert: 24 exact products each, fp32 sums.
template <int OUT>
__device__ __forceinline__ void dq_dots(const LinArgs &a, const DqDots &D, const uint32_t wh[12], float scale, int t0, int t1,
                                        long long row, int j) {
    const uint4 *x = reinterpret_cast<const uint4 *>(&D + 1) + 3 * j;
    for (int t = t0; t < t1; t++) {
        const uint4 *xt = OUT == kDqDots ? x + 3 * t * a.nb : reinterpret_cast<const uint4 *>(a.Xs + t * a.ldxs) + 3 * j;
        float d0 = 0.f, d1 = 0.f;
#pragma unroll
        for (int c = 0; c < 3; c++) {
            const uint4 q = OUT == kDqDots ? xt[c] : __ldca(xt + c);
            d0 = fma2_f16_f32(wh[4 * c + 0], q.x, d0);
            d1 = fma2_f16_f32(wh[4 * c + 1], q.y, d1);
            d0 = fma2_f16_f32(wh[4 * c + 2], q.z, d0);
            d1 = fma2_f16_f32(wh[4 * c + 3], q.w, d1);
        }
        a.dots[((long long)t * a.held + row) * a.nb + j] = scale * (d0 + d1) * D.scale[t];
    }
}

// What becomes of a decoded block (12 exact fp16 pairs; its gain, over |v| for table gains).
template <int OUT, int GAIN, bool GROUPED>
__device__ __forceinline__ void dq_block(const LinArgs &a, const DqShared &H, const uint32_t wh[12], float scale, int active,
                                         long long dst, int j) {
    if constexpr (dq_weights(OUT)) {
        const float s = scale * pow2_inverse(a.row_scale[dst]);
        if constexpr (OUT == kDqWeights) dq_store<GAIN>(wh, s, a.W + dst * a.ldw + j * 24);
        else dq_store_two<GAIN>(wh, s, a.cols - j * 24, a.W + dst * a.ldw + j * 48);
    } else {
        const DqDots &D = *reinterpret_cast<const DqDots *>(H.id);
        const int e = GROUPED ? (int)div_by((uint32_t)active, (uint32_t)a.rows, a.rows_recip) : 0;
        dq_dots<OUT>(a, D, wh, scale, GROUPED ? D.lo[e] : 0, GROUPED ? D.hi[e] : (int)a.tokens, dst, j);
    }
}
// ... and of a block whose index is not coded
template <int OUT, bool GROUPED>
__device__ __forceinline__ void dq_no_block(const LinArgs &a, const DqShared &H, int active, long long dst, int j) {
    if constexpr (dq_weights(OUT)) {
        constexpr int parts = OUT == kDqWeights ? 1 : 2;
        dq_store_zero<parts>(a.W + dst * a.ldw + j * 24 * parts);
    } else {
        const uint32_t none[12] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        dq_block<OUT, 0, GROUPED>(a, H, none, 0.f, active, dst, j);
    }
}

// The activations of a call of few tokens, in this CTA's shared memory, by all its threads; bf16 values
// with a power of two per token (as in lin_stage_token).  A barrier must follow.
__device__ __forceinline__ void dq_stage_dots(const LinArgs &a, DqDots &D) {
    uint4 *x = reinterpret_cast<uint4 *>(&D + 1);
    const int n8 = 3 * a.nb;                  // 16-byte units of a token
    const int total = (int)a.tokens * n8;
    auto load = [&](int i, int &t) {
        t = i / n8;
        const uint16_t *src = static_cast<const uint16_t *>(a.X) + t * a.ldx;
        return lin_load8(src, 8 * (i - t * n8), a.cols, lin_wide(src));
    };
    if (!a.bf16) {
        for (int i = threadIdx.x; i < total; i += blockDim.x) {
            int t;
            x[i] = load(i, t);
        }
        if (threadIdx.x < kLinDots) D.scale[threadIdx.x] = 1.f;
        return;
    }
    if (threadIdx.x < kLinDots) D.top[threadIdx.x] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < total; i += blockDim.x) {
        int t;
        const uint32_t top = lin_top8(load(i, t));
        if (top > D.top[t]) atomicMax(&D.top[t], top);
    }
    __syncthreads();
    if (threadIdx.x < a.tokens) D.scale[threadIdx.x] = lin_token_scale(D.top[threadIdx.x]);
    for (int i = threadIdx.x; i < total; i += blockDim.x) {
        int t;
        const uint4 q = load(i, t);
        x[i] = lin_restate8(q, pow2_inverse(lin_token_scale(D.top[t])));
    }
}

// What a CTA does before its blocks: the group list and its run; then the counters of the product and its rows'
// scales, or the activations of a call of few tokens (a barrier must follow).
template <int OUT, bool GROUPED>
__device__ __forceinline__ DqRun dq_groups(const LinArgs &a, DqShared &H) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int nact = 1;
    if (GROUPED) {
        if (warp == 0) {
            DqDots &D = *reinterpret_cast<DqDots *>(H.id);
            const int n = !dq_weights(OUT) ? lin_groups<true>(a, kLinDots, D.id, D.lo, D.hi)
                                         : lin_groups<false>(a, kLinExperts, H.id, nullptr, nullptr);
            if (lane == 0) H.nact = max(n, 0);
            if (n < 0 && lane == 0 && blockIdx.x == 0) atomicOr(a.flags, LLVQ_FLAG_OFFSETS);
        }
        __syncthreads();
        nact = H.nact;
    }
    return dq_run(a, nact);
}
template <int OUT, bool GROUPED>
__device__ __forceinline__ void dq_begin(const LinArgs &a, DqShared &H, const DqRun &run) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if constexpr (OUT == kDqDots) {
        dq_stage_dots(a, *reinterpret_cast<DqDots *>(H.id));
        return;
    }
    if constexpr (OUT == kDqDotsFar) {
        if (threadIdx.x < a.tokens) reinterpret_cast<DqDots *>(H.id)->scale[threadIdx.x] = a.bf16 ? __ldcg(a.token_scale + threadIdx.x) : 1.f;
        return;
    }
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.ncounters; i += gridDim.x * blockDim.x) a.counters[i] = 0u;
    for (int i = warp; i < run.nrows; i += warps) {
        long long src, dst;
        dq_row<GROUPED>(a, H.id, run.row0 + i, src, dst);
        const float s = lin_row_scale(a, warp_max(lin_row_top(a, src)));
        if (lane == 0) a.row_scale[dst] = s;       // a row shared with the next CTA gets the same value twice
    }
}

// The tokens a CTA restates: every gridDim.x-th of the tokens in use, one warp per token.
template <bool GROUPED>
__device__ __forceinline__ void dq_stage(const LinArgs &a, DqShared &H) {
    if (a.stage == 0) return;
    const int lane = threadIdx.x & 31;
    long long lo = 0, hi = a.tokens;
    if (GROUPED) {
        if (H.nact == 0) return;
        lo = __ldca(a.offsets);
        hi = __ldca(a.offsets + a.experts);
    }
    while (true) {
        int i = 0;
        if (lane == 0) i = atomicAdd(&H.stage_next, 1);
        i = __shfl_sync(0xFFFFFFFFu, i, 0);
        const long long t = lo + blockIdx.x + (long long)i * gridDim.x;
        if (t >= hi) break;
        lin_stage_token(static_cast<const uint16_t *>(a.X) + t * a.ldx, reinterpret_cast<uint4 *>(a.Xs + t * a.ldxs), a.cols,
                        a.parts == 2 ? a.nb : 0, a.stage == 2 ? a.token_scale + t : nullptr);
    }
}

struct Dq48Args {
    const SmemGv48 *image;
    unsigned long long npoints;
    const uint32_t *tabC;
    const unsigned long long *words;
    uint32_t wait_tries;
};

// Decode a record of the given kind (0 odd fast path, 1 even table path, 2 rare) and pass the block on.
template <int KIND, int OUT, int GAIN, bool GROUPED>
__device__ __forceinline__ void dq48_consume(const LinArgs &a, const SmemGv48 &S, const DqShared &H, const DqRec e, int row0) {
    const int cls = (int)(e.y & 0x1FFu);
    const uint32_t r = (e.y >> 9) & 0xFFFu;
    const uint32_t info = S.c_info[cls];
    const int j = (int)(e.w >> 16), active = row0 + (int)(e.w & 0xFFFFu);
    long long src, dst;
    dq_row<GROUPED>(a, H.id, active, src, dst);
    const float scale = GAIN == 0 ? __half2float(__ldg(a.gains + src * a.nb + j))
                                  : __half2float(__ldg(a.gains + src * 256 + (e.z >> 24))) * S.invnorm[info_m(info)];
    const unsigned long long p = (unsigned long long)((e.y >> 21) & 1u) << 32 | e.x;
    uint32_t wh[12];
    if constexpr (KIND == 0) {
        arrange_odd48_f16(S, cls, p, r, wh);
    } else if constexpr (KIND == 1) {
        arrange_even48_f16(S, cls, info, e.y >> 21, r, e.z & 0xFFFFFFu, e.x, wh);
    } else {
        const uint32_t word = (info & kInfoOdd) ? odd_codeword48(S, r)
                                                : S.gweight[min((S.c_info2[cls] & 0xFFFu) + r, 4095u)];
        uint32_t v[6];
        arrange48_word(S, cls, info, word, p, e.z & 0xFFFFFFu, true, v);
#pragma unroll
        for (int q = 0; q < 6; q++) i8x4_to_h2x2(v[q], wh[2 * q], wh[2 * q + 1]);
    }
    dq_block<OUT, GAIN, GROUPED>(a, H, wh, scale, active, dst, j);
}

template <int OUT, int GAIN, bool GROUPED>
__global__ void __launch_bounds__(kDqThreads, 1) k_dequant48(LinArgs a, Dq48Args d) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SmemGv48 &S = *reinterpret_cast<SmemGv48 *>(smem_raw);
    DqRec *rings = reinterpret_cast<DqRec *>(smem_raw + sizeof(SmemGv48));
    DqShared &H = *reinterpret_cast<DqShared *>(rings + kDqWarps * 2 * kDqRing);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned lanes_below = (1u << lane) - 1u;
    DqRec *ring_odd = rings + warp * 2 * kDqRing;
    DqRec *ring_even = ring_odd + kDqRing;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        H.slice_next = kDqWarps;              // slices 0..31 go to warps 0..31 directly
        H.stage_next = 0;
        H.nrare = 0;
    }
    {
        void *const dst[1] = {&S};
        const void *const src[1] = {d.image};
        const uint32_t bytes[1] = {(uint32_t)sizeof(SmemGv48)};
        bulk_load_issue(dst, src, bytes, &H.bar);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const DqRun run = dq_groups<OUT, GROUPED>(a, H);
    const int nb = a.nb, total = run.total, nslices = (total + 31) / 32;
    const bool dense = a.word_pitch == (long long)nb && !GROUPED;
    const unsigned long long *wfirst = d.words + (long long)run.row0 * nb + run.first;     // dense only
    auto word_at = [&](int t) -> const unsigned long long * {
        if (dense) return wfirst + t;
        const uint32_t b = (uint32_t)(run.first + t), rl = div_by(b, (uint32_t)nb, a.nb_recip);
        long long src, dst;
        dq_row<GROUPED>(a, H.id, run.row0 + (int)rl, src, dst);
        return d.words + src * a.word_pitch + (b - rl * (uint32_t)nb);
    };
    // Words come to L2 well before they are read: every 16th word's line of the slices ahead.  (Loading a slice's
    // words a slice ahead instead means taking slices ahead, and then some warps end with two slices to go
    // while others have none: 10 to 15% of the time on 5k to 25k blocks per SM.)
    auto prefetch = [&](int t) {
        if (t < total) asm volatile("prefetch.global.L2 [%0];" ::"l"(word_at(t)));
    };
    if (tid < 2 * (kDqWarps + kDqAhead)) prefetch(16 * tid);

    dq_begin<OUT, GROUPED>(a, H, run);
    if (!bulk_load_wait(&H.bar, d.wait_tries)) {
        if (tid == 0) atomicOr(a.flags, LLVQ_FLAG_WAIT_TIMEOUT);
        return;
    }
    // odd warps restate tokens (memory latency) while the even ones decode (instruction issue)
    if (dq_weights(OUT) && (warp & 1)) dq_stage<GROUPED>(a, H);

    bool bad = false;
    int oh = 0, ot = 0, eh = 0, et = 0;       // ring heads and tails (warp-uniform)
    auto append = [&](const DqRec &rec, int k) {       // k: 0 odd, 1 even, else none
        const unsigned mo = __ballot_sync(0xFFFFFFFFu, k == 0);
        const unsigned me = __ballot_sync(0xFFFFFFFFu, k == 1);
        if (k == 0) ring_odd[(ot + __popc(mo & lanes_below)) & (kDqRing - 1)] = rec;
        if (k == 1) ring_even[(et + __popc(me & lanes_below)) & (kDqRing - 1)] = rec;
        ot += __popc(mo);
        et += __popc(me);
        __syncwarp();
        if (ot - oh >= 32) {
            dq48_consume<0, OUT, GAIN, GROUPED>(a, S, H, ring_odd[(oh + lane) & (kDqRing - 1)], run.row0);
            oh += 32;
        }
        if (et - eh >= 32) {
            dq48_consume<1, OUT, GAIN, GROUPED>(a, S, H, ring_even[(eh + lane) & (kDqRing - 1)], run.row0);
            eh += 32;
        }
        __syncwarp();
    };
    int sl = warp;
    while (sl < nslices) {
        const int t = sl * 32 + lane;
        const bool valid = t < total;
        const unsigned long long w = valid ? __ldg(word_at(t)) : 0ull;
        if (lane < 2) prefetch((sl + kDqAhead) * 32 + 16 * lane);
        const Cls48 cl = classify48(w, S, d.npoints);
        const bool enq = valid && cl.ok;
        const bool odd = cl.info & kInfoOdd;
        int kind = odd ? (info_val4(cl.info) == 0u ? 0 : 2) : ((cl.info & kInfoTable) ? 1 : 2);
        if (!enq) kind = 3;
        const uint32_t b = (uint32_t)(run.first + (valid ? t : 0)), rl = div_by(b, (uint32_t)nb, a.nb_recip);
        DqRec rec;
        rec.x = (uint32_t)cl.p;
        rec.y = (uint32_t)cl.cls | cl.r << 9 | (uint32_t)(cl.p >> 32) << 21;
        rec.z = cl.s | (uint32_t)((w >> 48) & 0xFFu) << 24;
        rec.w = rl | (b - rl * (uint32_t)nb) << 16;
        if (kind == 1) {
            uint32_t pS;
            const uint32_t pC = even48_pC(S, cl.cls, (uint32_t)cl.p, pS);
            rec.x = __ldg(d.tabC + (S.c_offs[cl.cls] & 0x7FFFFu) + pC);
            rec.y = (uint32_t)cl.cls | cl.r << 9 | pS << 21;
        }
        // Odd classes of five magnitude groups and even ones off the tables, 0.12% of the points: a warp that
        // decoded one where it is met would spend 1500 instructions on one lane, 7% of the kernel's
        // time, so they wait for the end (as long as there is room)
        if (kind == 2) {
            const int at = atomicAdd(&H.nrare, 1);
            if (at < kDqRare) H.rare[at] = rec;
            else dq48_consume<2, OUT, GAIN, GROUPED>(a, S, H, rec, run.row0);
        }
        if (valid && !cl.ok) {                // an index beyond the coded points: nothing
            bad = true;
            long long src, dst;
            dq_row<GROUPED>(a, H.id, run.row0 + (int)rl, src, dst);
            dq_no_block<OUT, GROUPED>(a, H, run.row0 + (int)rl, dst, (int)(b - rl * (uint32_t)nb));
        }
        append(rec, kind);
        if (lane == 0) sl = atomicAdd(&H.slice_next, 1);
        sl = __shfl_sync(0xFFFFFFFFu, sl, 0);
    }
    // What is left in the rings (fewer than 32 records each) is pooled over the CTA, again in whole warps, rather
    // than decoded by half-empty ones: 41.7 us against 44.4 for a call of 4.7k blocks per SM.  Record i of the
    // pool is found by the rings' cumulative counts.
    H.left[0][warp] = ot - oh;
    H.left[1][warp] = et - eh;
    H.head[0][warp] = oh & (kDqRing - 1);
    H.head[1][warp] = eh & (kDqRing - 1);
    __syncthreads();
    for (int kind = 0; kind < 2; kind++) {
        int upto = H.left[kind][lane];                       // ring `lane`'s count, then the counts up to it
        const int mine = upto;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
        }
        const int all = __shfl_sync(0xFFFFFFFFu, upto, 31);
        // warps take the even records from the other end, so that a warp rarely gets a batch of both
        for (int i0 = 32 * (kind == 0 ? warp : kDqWarps - 1 - warp); i0 < all; i0 += 32 * kDqWarps) {
            const int i = min(i0 + lane, all - 1);
            int ring = 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)                 // the first ring whose count up to it is beyond i
                if (__shfl_sync(0xFFFFFFFFu, upto, ring + o - 1) <= i) ring += o;
            const int at = i - __shfl_sync(0xFFFFFFFFu, upto - mine, ring) + H.head[kind][ring];
            const DqRec rec = rings[(2 * ring + kind) * kDqRing + (at & (kDqRing - 1))];
            if (i0 + lane < all) {
                if (kind == 0) dq48_consume<0, OUT, GAIN, GROUPED>(a, S, H, rec, run.row0);
                else dq48_consume<1, OUT, GAIN, GROUPED>(a, S, H, rec, run.row0);
            }
        }
    }
    // the rare blocks, by warps that are the last to get a batch of the pool
    if (warp >= kDqWarps / 2 && warp < kDqWarps / 2 + kDqRare / 32) {
        const int i = 32 * (warp - kDqWarps / 2) + lane;
        if (i < min(H.nrare, kDqRare)) dq48_consume<2, OUT, GAIN, GROUPED>(a, S, H, H.rare[i], run.row0);
    }
    if (dq_weights(OUT)) dq_stage<GROUPED>(a, H);
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(a.flags, LLVQ_FLAG_INDEX_RANGE);
}

// 72- and 96-bit blocks: one block per thread at a time, the generic decoders.
template <class D, int OUT, bool GROUPED>
__global__ void __launch_bounds__(512, D::kCtasPerSm) k_dequant(LinArgs a, typename D::Args d,
                                                               const typename D::Word *__restrict__ words) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    typename D::Smem &S = *reinterpret_cast<typename D::Smem *>(smem_raw);
    DqShared &H = *reinterpret_cast<DqShared *>(smem_raw + (sizeof(typename D::Smem) + 15) / 16 * 16);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) H.stage_next = 0;
    load_smem_image(&S, d.image, sizeof(typename D::Smem));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const DqRun run = dq_groups<OUT, GROUPED>(a, H);
    dq_begin<OUT, GROUPED>(a, H, run);
    __syncthreads();
    if (dq_weights(OUT)) dq_stage<GROUPED>(a, H);
    bool bad = false;
    for (int t = threadIdx.x; t < run.total; t += blockDim.x) {
        const uint32_t b = (uint32_t)(run.first + t), rl = div_by(b, (uint32_t)a.nb, a.nb_recip);
        const int j = (int)(b - rl * (uint32_t)a.nb);
        long long src, dst;
        dq_row<GROUPED>(a, H.id, run.row0 + (int)rl, src, dst);
        const typename D::Word w = D::load(words + src * a.word_pitch + j);
        uint32_t v[6], wh[12];
        int m;
        const bool ok = D::decode(w, S, d, v, m);
        bad |= !ok;
#pragma unroll
        for (int q = 0; q < 6; q++) i8x4_to_h2x2(ok ? v[q] : 0u, wh[2 * q], wh[2 * q + 1]);
        const int active = run.row0 + (int)rl;
        if (!ok) dq_no_block<OUT, GROUPED>(a, H, active, dst, j);
        else if (a.gain_mode == 0) dq_block<OUT, 0, GROUPED>(a, H, wh, __half2float(__ldg(a.gains + src * a.nb + j)), active, dst, j);
        else dq_block<OUT, 1, GROUPED>(a, H, wh, __half2float(__ldg(a.gains + src * 256 + D::gain_code(w))) * D::invnorm(S, m), active, dst, j);
    }
    if (__any_sync(0xFFFFFFFFu, bad) && (threadIdx.x & 31) == 0) atomicOr(a.flags, LLVQ_FLAG_INDEX_RANGE);
}

// The second kernel of a call of few tokens: a warp, or 2^k lanes of one for short rows, per output adds the dot
// products of its row (or gate and up rows), lane by lane and then across the lanes, always in the same order, and
// applies the epilogue.  Bound by its latency: 2.8 MB are read for a 4096 x 4104 layer and one token.
struct DqEnds {
    const void *bias, *residual;
    long long ld_res;
    void *Y;
    long long ldy;
    int act;
};
constexpr int kDqFinishWarps = 8;
// lanes of an output
__host__ __device__ constexpr int finish_width(int nb) { return nb > 32 ? 32 : nb > 4 ? 8 : 1; }
template <bool GROUPED, bool GATED, class T, int WIDTH>
__global__ void __launch_bounds__(32 * kDqFinishWarps) k_linear_finish(LinArgs a, DqEnds q) {
    __shared__ int id[kLinDots], lo[kLinDots], hi[kLinDots], count;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (GROUPED) {
        if (warp == 0) {
            const int n = lin_groups<true>(a, kLinDots, id, lo, hi);
            if (lane == 0) count = n;
        }
        __syncthreads();
        if (count < 1) return;
    }
    const int outs = GATED ? a.half : a.rows;
    const int t = blockIdx.y;
    int e = 0, expert = 0;
    if (GROUPED) {
        while (e < count && hi[e] <= t) e++;
        if (e == count || t < lo[e]) return;
        expert = id[e];
    }
    constexpr int each = 32 / WIDTH;                                       // outputs of a warp
    const int sub = lane & (WIDTH - 1);
    for (int o0 = (blockIdx.x * kDqFinishWarps + warp) * each; o0 < outs; o0 += gridDim.x * kDqFinishWarps * each) {
        const int o = min(o0 + lane / WIDTH, outs - 1);
        const float *row = a.dots + ((long long)t * a.held + (long long)e * a.rows + (GATED ? 2 * o : o)) * a.nb;
        // bias and residual are on their way while the row is added
        float zb = 0.f, ub = 0.f, res = 0.f;
        const bool writes = sub == 0 && o0 + lane / WIDTH < outs;
        if (writes) {
            if (q.bias) {
                const T *b = static_cast<const T *>(q.bias) + (long long)expert * a.rows + o;
                zb = lin_load(b);
                if (GATED) ub = lin_load(b + a.half);
            }
            if (q.residual) res = lin_load(static_cast<const T *>(q.residual) + t * q.ld_res + o);
        }
        float z = 0.f, up = 0.f;
        for (int j0 = sub; j0 < a.nb; j0 += 4 * WIDTH) {
            float v[4], u[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int j = j0 + WIDTH * i;
                v[i] = j < a.nb ? __ldcg(row + j) : 0.f;
                if (GATED) u[i] = j < a.nb ? __ldcg(row + a.nb + j) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                z += v[i];
                if (GATED) up += u[i];
            }
        }
#pragma unroll
        for (int s = WIDTH / 2; s > 0; s >>= 1) {
            z += __shfl_xor_sync(0xFFFFFFFFu, z, s);
            if (GATED) up += __shfl_xor_sync(0xFFFFFFFFu, up, s);
        }
        if (writes) {
            z += zb;
            up += ub;
            float y = q.act == kActNone ? z : lin_activate1(z, q.act);
            if (GATED) y *= up;
            if (q.residual) y += res;
            static_cast<T *>(q.Y)[t * q.ldy + o] = lin_round<T>(y);
        }
    }
}

}  // namespace llvq
