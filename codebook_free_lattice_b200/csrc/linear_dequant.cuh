// linear_dequant.cuh -- the first kernel of a compressed linear layer: every block of the experts
// that have tokens is decoded once and written as 24 scaled fp16 weights (linear_common.cuh).
//
// "Leech Lattice Vector Quantization for Efficient LLM Compression", papernotes.org notes,
// 方法详解 / 关键设计 2: index -> shell, class, codeword, signs, arrangement -> integer vector.
//
// Integer work bounds it: about 700 thread instructions per 48-bit block, against 8 bytes read and 48
// written.  Each CTA takes an equal run of blocks (not of rows: a run may begin and end inside a row, so
// few long rows still spread over all SMs).  48-bit blocks use the warp-private rings of the fused GEMV
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
using DqRec = uint4;                          // like BinRec: x, y, z the digits, w = local row | block << 16

struct DqShared {
    int slice_next, stage_next, nact, pad;
    unsigned long long bar;
    unsigned long long pad2;
    int id[kLinExperts];
};
__host__ __device__ constexpr size_t dq48_smem(bool grouped) {
    return sizeof(SmemGv48) + sizeof(DqRec) * (kDqWarps * 2 * kDqRing) + (grouped ? sizeof(DqShared) : 32);
}
template <class D>
__host__ __device__ constexpr size_t dq_smem(bool grouped) {
    return (sizeof(typename D::Smem) + 15) / 16 * 16 + (grouped ? sizeof(DqShared) : 32);
}

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

// 24 integers (12 exact fp16 pairs) times the block's scale, each rounded once to fp16.  Direct gains
// times a power of two are fp16 values, one product.  A table gain over |v| is not: its rounding
// error goes in as a second factor, w = v s_hi + (v s_lo), so that the sum is rounded once.
template <int GAIN>
__device__ __forceinline__ void dq_store(const uint32_t wh[12], float scale, __half *out) {
    const __half hi = __float2half_rn(scale);
    const __half2 hi2 = __halves2half2(hi, hi);
    const __half lo = __float2half_rn(scale - __half2float(hi));
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
__device__ __forceinline__ void dq_store_zero(__half *out) {
    uint4 *p = reinterpret_cast<uint4 *>(out);
    p[0] = p[1] = p[2] = make_uint4(0u, 0u, 0u, 0u);
}

// What a CTA does before its blocks: the group list, the counters of the product, its rows' scales.
// Ends with the scales written (a barrier must follow before they are read).
template <bool GROUPED>
__device__ __forceinline__ DqRun dq_begin(const LinArgs &a, DqShared &H) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int nact = 1;
    if (GROUPED) {
        if (warp == 0) {
            const int n = lin_groups<false>(a, H.id, nullptr, nullptr);
            if (lane == 0) H.nact = max(n, 0);
            if (n < 0 && lane == 0 && blockIdx.x == 0) atomicOr(a.flags, LLVQ_FLAG_OFFSETS);
        }
        __syncthreads();
        nact = H.nact;
    }
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.ncounters; i += gridDim.x * blockDim.x) a.counters[i] = 0u;
    const DqRun run = dq_run(a, nact);
    for (int i = warp; i < run.nrows; i += warps) {
        long long src, dst;
        dq_row<GROUPED>(a, H.id, run.row0 + i, src, dst);
        const float s = lin_row_scale(a, src);
        if (lane == 0) a.row_scale[dst] = s;       // a row shared with the next CTA gets the same value twice
    }
    return run;
}

// The tokens a CTA restates: every gridDim.x-th of the tokens in use, one warp per token.
template <bool GROUPED>
__device__ __forceinline__ void dq_stage(const LinArgs &a, DqShared &H) {
    if (a.stage == 0) return;
    const int lane = threadIdx.x & 31;
    long long lo = 0, hi = a.tokens;
    if (GROUPED) {
        if (H.nact == 0) return;
        lo = __ldg(a.offsets);
        hi = __ldg(a.offsets + a.experts);
    }
    while (true) {
        int i = 0;
        if (lane == 0) i = atomicAdd(&H.stage_next, 1);
        i = __shfl_sync(0xFFFFFFFFu, i, 0);
        const long long t = lo + blockIdx.x + (long long)i * gridDim.x;
        if (t >= hi) break;
        lin_stage_token(static_cast<const uint16_t *>(a.X) + t * a.ldx, reinterpret_cast<uint4 *>(a.Xs + t * a.ldxs), a.cols,
                        a.stage == 2 ? a.token_scale + t : nullptr);
    }
}

struct Dq48Args {
    const SmemGv48 *image;
    unsigned long long npoints;
    const uint32_t *tabC;
    const unsigned long long *words;
    uint32_t wait_tries;
};

// Decode a record of the given kind (0 odd fast path, 1 even table path, 2 rare) and write it.
template <int KIND, int GAIN, bool GROUPED>
__device__ __forceinline__ void dq48_consume(const LinArgs &a, const SmemGv48 &S, const int *id, const DqRec e, int row0) {
    const int cls = (int)(e.y & 0x1FFu);
    const uint32_t r = (e.y >> 9) & 0xFFFu;
    const uint32_t info = S.c_info[cls];
    const int j = (int)(e.w >> 16);
    long long src, dst;
    dq_row<GROUPED>(a, id, row0 + (int)(e.w & 0xFFFFu), src, dst);
    const float f = pow2_inverse(a.row_scale[dst]);
    const float scale = f * (GAIN == 0 ? __half2float(__ldg(a.gains + src * a.nb + j))
                                       : __half2float(__ldg(a.gains + src * 256 + (e.z >> 24))) * S.invnorm[info_m(info)]);
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
    dq_store<GAIN>(wh, scale, a.W + dst * a.ldw + j * 24);
}

template <int GAIN, bool GROUPED>
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
    }
    {
        void *const dst[1] = {&S};
        const void *const src[1] = {d.image};
        const uint32_t bytes[1] = {(uint32_t)sizeof(SmemGv48)};
        bulk_load_issue(dst, src, bytes, &H.bar);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const DqRun run = dq_begin<GROUPED>(a, H);
    if (!bulk_load_wait(&H.bar, d.wait_tries)) {
        if (tid == 0) atomicOr(a.flags, LLVQ_FLAG_WAIT_TIMEOUT);
        return;
    }
    // odd warps restate tokens (memory latency) while the even ones decode (instruction issue)
    if (warp & 1) dq_stage<GROUPED>(a, H);

    const int nb = a.nb, total = run.total, nslices = (total + 31) / 32;
    const bool dense = a.word_pitch == (long long)nb && !GROUPED;
    const unsigned long long *wfirst = d.words + (long long)run.row0 * nb + run.first;     // dense only
    auto word_at = [&](int t) -> unsigned long long {
        if (t >= total) return 0ull;
        if (dense) return __ldg(wfirst + t);
        const uint32_t b = (uint32_t)(run.first + t), rl = div_by(b, (uint32_t)nb, a.nb_recip);
        long long src, dst;
        dq_row<GROUPED>(a, H.id, run.row0 + (int)rl, src, dst);
        return __ldg(d.words + src * a.word_pitch + (b - rl * (uint32_t)nb));
    };

    bool bad = false;
    int oh = 0, ot = 0, eh = 0, et = 0;       // ring heads and tails (warp-uniform)
    DqRec prec;                               // the previous slice's record, written one slice late
    int pk = 3;                               // 0 odd, 1 even, 3 none
    prec.x = prec.y = prec.z = prec.w = 0u;
    auto append = [&](const DqRec &rec, int k) {
        const unsigned mo = __ballot_sync(0xFFFFFFFFu, k == 0);
        const unsigned me = __ballot_sync(0xFFFFFFFFu, k == 1);
        if (k == 0) ring_odd[(ot + __popc(mo & lanes_below)) & (kDqRing - 1)] = rec;
        if (k == 1) ring_even[(et + __popc(me & lanes_below)) & (kDqRing - 1)] = rec;
        ot += __popc(mo);
        et += __popc(me);
        __syncwarp();
        if (ot - oh >= 32) {
            dq48_consume<0, GAIN, GROUPED>(a, S, H.id, ring_odd[(oh + lane) & (kDqRing - 1)], run.row0);
            oh += 32;
        }
        if (et - eh >= 32) {
            dq48_consume<1, GAIN, GROUPED>(a, S, H.id, ring_even[(eh + lane) & (kDqRing - 1)], run.row0);
            eh += 32;
        }
        __syncwarp();
    };
    int sl = warp;
    unsigned long long w = sl < nslices ? word_at(sl * 32 + lane) : 0ull;
    while (sl < nslices) {
        int sn = 0;
        if (lane == 0) sn = atomicAdd(&H.slice_next, 1);
        sn = __shfl_sync(0xFFFFFFFFu, sn, 0);
        const unsigned long long wn = sn < nslices ? word_at(sn * 32 + lane) : 0ull;
        const int t = sl * 32 + lane;
        const bool valid = t < total;
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
        if (kind == 2) dq48_consume<2, GAIN, GROUPED>(a, S, H.id, rec, run.row0);
        if (valid && !cl.ok) {                // an index beyond the coded points: a zero block
            bad = true;
            long long src, dst;
            dq_row<GROUPED>(a, H.id, run.row0 + (int)rl, src, dst);
            dq_store_zero(a.W + dst * a.ldw + (b - rl * (uint32_t)nb) * 24);
        }
        append(prec, pk);
        prec = rec;
        pk = kind;
        w = wn;
        sl = sn;
    }
    append(prec, pk);
    if (lane < ot - oh) dq48_consume<0, GAIN, GROUPED>(a, S, H.id, ring_odd[(oh + lane) & (kDqRing - 1)], run.row0);
    if (lane < et - eh) dq48_consume<1, GAIN, GROUPED>(a, S, H.id, ring_even[(eh + lane) & (kDqRing - 1)], run.row0);
    dq_stage<GROUPED>(a, H);
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(a.flags, LLVQ_FLAG_INDEX_RANGE);
}

// 72- and 96-bit blocks: one block per thread at a time, the generic decoders.
template <class D, bool GROUPED>
__global__ void __launch_bounds__(512, D::kCtasPerSm) k_dequant(LinArgs a, typename D::Args d,
                                                               const typename D::Word *__restrict__ words) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    typename D::Smem &S = *reinterpret_cast<typename D::Smem *>(smem_raw);
    DqShared &H = *reinterpret_cast<DqShared *>(smem_raw + (sizeof(typename D::Smem) + 15) / 16 * 16);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) H.stage_next = 0;
    load_smem_image(&S, d.image, sizeof(typename D::Smem));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const DqRun run = dq_begin<GROUPED>(a, H);
    __syncthreads();
    dq_stage<GROUPED>(a, H);
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
        const float f = pow2_inverse(a.row_scale[dst]);
        __half *out = a.W + dst * a.ldw + j * 24;
        if (!ok) dq_store_zero(out);
        else if (a.gain_mode == 0) dq_store<0>(wh, f * __half2float(__ldg(a.gains + src * a.nb + j)), out);
        else dq_store<1>(wh, f * (__half2float(__ldg(a.gains + src * 256 + D::gain_code(w))) * D::invnorm(S, m)), out);
    }
    if (__any_sync(0xFFFFFFFFu, bad) && (threadIdx.x & 31) == 0) atomicOr(a.flags, LLVQ_FLAG_INDEX_RANGE);
}

}  // namespace llvq
