// linear_common.cuh -- what the kernels of the compressed linear layers share: the arguments of a
// call, the groups of tokens, the row and token scales, and the epilogue's activations.
//
// A linear layer over a compressed weight (papernotes.org notes, 方法详解 / 关键设计 4 gives the
// product; bias, activation, residual, gating and experts are what a language model puts around it):
//
//   z[t][r] = sum_k w[r][k] x[t][k] + b[r]        y[t][o] = act(z[t][o]) [* z[t][F + o]] + res[t][o]
//
// runs as two kernels: the blocks are decoded once into an fp16 weight in the caller's workspace
// (linear_dequant.cuh), and a tile product on the tensor cores multiplies it with every token and
// applies the epilogue (linear_product.cuh).  A few tokens are multiplied with each block as it is
// decoded, and the second kernel adds the rows up.
//
// Scales.  A weight is stored as fp16(w 2^s) with one power of two per row, chosen so that the
// row's largest gain lies just below the end of the fp16 range: no row, however small or large its gains, is
// lost to fp16's subnormals or overflows, and w keeps 11 significant bits.  bf16 activations are
// restated as fp16(x 2^u) with one power of two per token: 8 significant bits fit in 11, so the
// restatement is exact down to 2^-28 of the token's largest value and off by at most 2^-39 of it
// below that, less than the fp32 accumulation of the product rounds.  Both powers leave again in
// the epilogue, exactly.  A bf16 weight would have lost 3 bits that fp16 keeps.
//
// Against the definition in 64 bits, one fp16 value per weight leaves a bf16 output 1.01 times as far off as its
// own rounding does, and a plain fp16 output 1.3 to 1.45 times (the weight's rounding is as large as the output's, and
// independent of it).  A gated fp16 output multiplies two such sums and would be 1.75 times as far off (3.6e-4
// against 2.1e-4), so its weights have two fp16 values, the second the rest of the first: 22 bits, 1.00 times,
// for twice the products and twice the decoded weight.  A block's 24 values and their 24 rests follow one another,
// and so do a token's 24 values and the same again: to the product this is one sum over twice the columns.
#pragma once
#include <cuda_bf16.h>
#include "codec48.cuh"

namespace llvq {

// Loads.  A layer's kernels start before the ones ahead of them on the stream have ended (griddepcontrol), so what
// those write is written while the reader is alive: the workspace, but also x, the residual and the offsets,
// which may be another layer's outputs.  They are read by coherent loads after griddepcontrol.wait (__ldca, __ldcg,
// plain ones), never by __ldg, whose loads promise nothing for such data.  The weight's words and gains and the
// codec's tables are not written while a layer may run, and take __ldg.

constexpr int kLinExperts = 2048;             // most experts of one call (their groups sit in shared memory)
constexpr int kLinRows = 256;                 // weight rows of a tile (one pair of CTAs)
constexpr int kLinTokens = 256;               // most tokens of a tile
constexpr int kLinDots = 16;                  // most tokens of a call without a decoded weight

struct LinArgs {
    // the layer: `experts` stacked matrices of `rows` rows; half = rows / 2 when gated, else 0
    int rows, half, cols, nb, experts;
    int gain_mode;
    const __half *gains;
    long long word_pitch;
    // tokens: offsets (experts + 1 entries) or null for one matrix and every token
    const int *offsets;
    long long tokens;
    // the decoded weight [active expert][row] (gated: row pairs gate, up interleaved), rows of ldw values,
    // and 1 / (its power of two) per row
    __half *W;
    long long ldw;
    int parts;                                // fp16 values of a weight: 1, or 2 (and of an activation: the same twice)
    int terms;                                // products of an output: cols, or 48 per block with two parts
    float *row_scale;
    uint32_t rows_recip, nb_recip;            // ceil(2^32 / rows), ceil(2^32 / nb) (0 for 1)
    // the split tiles' arrival counters
    unsigned *counters;
    int ncounters;
    // activations restated in the workspace: stage 0 none, 1 fp16 copied, 2 bf16 to fp16 with scales
    int stage;
    const void *X;
    long long ldx;
    __half *Xs;
    long long ldxs;
    float *token_scale;
    // few tokens: the blocks' dot products [token][row of the decoded weight][nb] instead of the weight
    float *dots;
    long long held;                           // rows of the decoded weight
    int bf16;
    unsigned *flags;
};

// n / d for n < 2^32 by a multiply-high with recip = ceil(2^32 / d): the product overshoots by less
// than n / 2^32 < 1, so one correction makes it exact.
__device__ __forceinline__ uint32_t div_by(uint32_t n, uint32_t d, uint32_t recip) {
    if (recip == 0u) return n;                                  // d = 1
    uint32_t q = __umulhi(n, recip);
    if ((unsigned long long)q * d > n) q--;
    return q;
}

// row of the decoded weight that holds row r of a matrix
__device__ __forceinline__ int lin_place(int r, int half) {
    return half == 0 ? r : r < half ? 2 * r : 2 * (r - half) + 1;
}

// The experts that have tokens, in order, by one warp: id[i], and with EDGES their token ranges
// lo[i], hi[i]; at most `room` of them are written (offsets in order never leave more than room).  Offsets
// that fall, start below zero or end beyond the tokens leave no expert (the flag is raised by the
// caller); returns the count, or -1 for such offsets.
template <bool EDGES>
__device__ __forceinline__ int lin_groups(const LinArgs &a, int room, int *id, int *lo, int *hi) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    bool bad = false;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
        const int e = e0 + lane;
        int s = 0, t = 0;
        if (e < a.experts) {
            s = __ldca(a.offsets + e);
            t = __ldca(a.offsets + e + 1);
            bad |= t < s || s < 0 || (long long)t > a.tokens;
        }
        const unsigned m = __ballot_sync(0xFFFFFFFFu, t > s);
        if (t > s) {
            const int i = n + __popc(m & ((1u << lane) - 1u));
            if (i < room) {
                id[i] = e;
                if (EDGES) {
                    lo[i] = s;
                    hi[i] = t;
                }
            }
        }
        n += __popc(m);
    }
    return __any_sync(0xFFFFFFFFu, bad) ? -1 : n;
}

// largest finite magnitude, as its fp32 bits (ordered like the values)
__device__ __forceinline__ uint32_t finite_bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) {
    return __reduce_max_sync(0xFFFFFFFFu, v);
}
// 2^k for -126 <= k <= 127, and its inverse from its bits
__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float(0x7F000000u - __float_as_uint(p)); }

// The largest finite gain of one row, by one warp: each lane's share of it, as fp32 bits.
__device__ __forceinline__ uint32_t lin_row_top(const LinArgs &a, long long row) {
    const int lane = threadIdx.x & 31;
    uint32_t top = 0;
    if (a.gain_mode == 0) {
        const __half *g = a.gains + row * a.nb;
        for (int j = lane; j < a.nb; j += 32) top = max(top, finite_bits(__half2float(__ldg(g + j))));
    } else {
        const __half *g = a.gains + row * 256;
        if (((unsigned long long)a.gains & 15ull) == 0ull) {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(g) + lane);
            const uint32_t h[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                top = max(top, max(finite_bits(f.x), finite_bits(f.y)));
            }
        } else {
            for (int j = lane; j < 256; j += 32) top = max(top, finite_bits(__half2float(__ldg(g + j))));
        }
    }
    return top;
}
// The scale of a row whose largest gain has these bits: 2^-s with s such that the row's largest weight lies in
// the top binades of fp16.  Table gains bound the weights themselves (a direction's coordinates are
// at most 1), direct gains leave out |v_i| < 64.
__device__ __forceinline__ float lin_row_scale(const LinArgs &a, uint32_t top) {
    if (top == 0u) return 1.f;
    const int ex = (int)(top >> 23) - 127;                      // fp16 values: -24 .. 15
    return pow2(ex - (a.gain_mode == 0 ? 9 : 14));
}

// Eight consecutive 16-bit values from element i (a multiple of 8) of a row of n; elements at and beyond n read
// as zero.  Rows that do not start on 16 bytes (not wide) are read in pairs or value by value.
__device__ __forceinline__ bool lin_wide(const uint16_t *row) { return ((unsigned long long)row & 15ull) == 0ull; }
__device__ __forceinline__ uint4 lin_load8(const uint16_t *row, int i, int n, bool wide) {
    if (wide && i + 8 <= n) return __ldca(reinterpret_cast<const uint4 *>(row + i));
    if (((unsigned long long)row & 3ull) == 0ull && i + 8 <= n) {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(row + i);
        return make_uint4(__ldca(p), __ldca(p + 1), __ldca(p + 2), __ldca(p + 3));
    }
    uint32_t h[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; k++)
        if (i + k < n) h[k >> 1] |= (uint32_t)__ldca(row + i + k) << (16 * (k & 1));
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// The scale of a bf16 token whose largest finite magnitude has these bits: 2^-u, leaving that value in fp16's
// top binade (subnormals: exponent -126 stands for all of them; 2^126 is the most its inverse can be).
__device__ __forceinline__ float lin_token_scale(uint32_t top) {
    return pow2(top == 0u ? 0 : max(max((int)(top >> 23) - 127, -126) - 14, -126));
}
// eight bf16 values scaled to fp16, and their largest finite magnitude
__device__ __forceinline__ uint4 lin_restate8(uint4 q, float f) {
    const uint32_t h[4] = {q.x, q.y, q.z, q.w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const __half2 v = __floats2half2_rn(__uint_as_float(h[k] << 16) * f, __uint_as_float(h[k] & 0xFFFF0000u) * f);
        o[k] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint32_t lin_top8(uint4 q) {
    const uint32_t h[4] = {q.x, q.y, q.z, q.w};
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; k++)
        top = max(top, max(finite_bits(__uint_as_float(h[k] << 16)), finite_bits(__uint_as_float(h[k] & 0xFFFF0000u))));
    return top;
}

// Unit i of 8 values where a block's 3 units are there twice.  An infinity or a NaN is there once: it belongs to the
// weight, and times the weight's rest (zero, or of the other sign) would make a NaN of an infinity.
__device__ __forceinline__ uint32_t lin_finite2(uint32_t h) {
    return h & __hle2_mask(__habs2(*reinterpret_cast<const __half2 *>(&h)), __float2half2_rn(65504.f));
}
__device__ __forceinline__ void lin_twice(uint4 *dst, int i, uint4 q) {
    uint4 *p = dst + i + i / 3 * 3;
    p[0] = q;
    p[3] = make_uint4(lin_finite2(q.x), lin_finite2(q.y), lin_finite2(q.z), lin_finite2(q.w));
}

// One token restated for the product, by one warp: fp16 copied to an aligned row (no scale), bf16 scaled by a
// power of two and rounded to fp16 (see above).  The row is read twice; the second time it is in L1.
// nb > 0: the nb blocks' values twice, for a weight of two parts.
__device__ __noinline__ void lin_stage_token(const uint16_t *src, uint4 *dst, int cols, int nb, float *scale) {
    const int lane = threadIdx.x & 31;
    const int n8 = (cols + 7) / 8;
    const bool wide = lin_wide(src);
    if (nb) {
#pragma unroll 4
        for (int i = lane; i < 3 * nb; i += 32) lin_twice(dst, i, lin_load8(src, 8 * i, cols, wide));
        return;
    }
    if (!scale) {
#pragma unroll 4
        for (int i = lane; i < n8; i += 32) dst[i] = lin_load8(src, 8 * i, cols, wide);
        return;
    }
    uint32_t top = 0;
#pragma unroll 4
    for (int i = lane; i < n8; i += 32) top = max(top, lin_top8(lin_load8(src, 8 * i, cols, wide)));
    top = warp_max(top);
    const float inv = lin_token_scale(top), f = pow2_inverse(inv);
    if (lane == 0) *scale = inv;
#pragma unroll 4
    for (int i = lane; i < n8; i += 32) dst[i] = lin_restate8(lin_load8(src, 8 * i, cols, wide), f);
}

// Many tokens restated by a kernel of their own, one CTA per token, the row held in registers between the scale
// and the conversion (the part of a row beyond 64 values per thread is read again): the bytes of x once in and
// once out.  units: 16-byte units of a row to write, zero beyond the columns.
constexpr int kLinStageMost = 1024;           // threads: a row's 16-byte units over 4, in whole warps
template <bool BF16>
__global__ void __launch_bounds__(kLinStageMost) k_linear_stage(LinArgs a, int units) {
    constexpr int kHeld = 8;
    __shared__ uint32_t tops[2][kLinStageMost / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, threads = blockDim.x;
    long long lo = 0, hi = a.tokens;
    if (a.offsets) {                          // rows that no group has are not read; bad offsets are the decode's to tell
        lo = max(0, __ldca(a.offsets));
        hi = min(a.tokens, (long long)__ldca(a.offsets + a.experts));
    }
    const int n8 = units;
    int turn = 0;
    for (long long t = lo + blockIdx.x; t < hi; t += gridDim.x, turn ^= 1) {
        const uint16_t *src = static_cast<const uint16_t *>(a.X) + t * a.ldx;
        uint4 *dst = reinterpret_cast<uint4 *>(a.Xs + t * a.ldxs);
        const bool wide = ((unsigned long long)src & 15ull) == 0ull;
        uint4 held[kHeld];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kHeld; i++) {
            const int k = tid + threads * i;
            if (k < n8) held[i] = lin_load8(src, 8 * k, a.cols, wide);
        }
        float f = 1.f;
        if (BF16) {
#pragma unroll
            for (int i = 0; i < kHeld; i++)
                if (tid + threads * i < n8) top = max(top, lin_top8(held[i]));
            for (int k = tid + threads * kHeld; k < n8; k += threads) top = max(top, lin_top8(lin_load8(src, 8 * k, a.cols, wide)));
            top = warp_max(top);
            if ((tid & 31) == 0) tops[turn][tid >> 5] = top;
            __syncthreads();
            top = warp_max((tid & 31) < threads >> 5 ? tops[turn][tid & 31] : 0u);
            const float inv = lin_token_scale(top);
            if (tid == 0) a.token_scale[t] = inv;
            f = pow2_inverse(inv);
        }
#pragma unroll
        for (int i = 0; i < kHeld; i++) {
            const int k = tid + threads * i;
            if (k < n8) {
                if (!BF16 && a.parts == 2) lin_twice(dst, k, held[i]);
                else dst[k] = BF16 ? lin_restate8(held[i], f) : held[i];
            }
        }
        for (int k = tid + threads * kHeld; k < n8; k += threads) {
            const uint4 q = lin_load8(src, 8 * k, a.cols, wide);
            if (!BF16 && a.parts == 2) lin_twice(dst, k, q);
            else dst[k] = BF16 ? lin_restate8(q, f) : q;
        }
    }
}

// Activations, four values at a time and out of line: the code of one activation is fetched once, and
// a kernel that needs none of it does not step over it.  Each keeps the relative accuracy of its negative tail,
// which a gate can bring back: z P(z) with P(z) = erfc(-z / sqrt 2) / 2 for gelu, and z e^u / (1 + e^u) below
// zero for the others, so that the denominator lies between 1 and 2.  erfc(x) e^x^2 is t q(t) with t = 1 / (1 + 3/8 x) and
// q of degree 6, the polynomial whose largest relative error on 0 <= x <= 9.5 (beyond, P leaves fp32's range) is
// least, 6.3e-7, found as a linear program over 4000 Chebyshev points; 1.0e-6 as evaluated in fp32.  (With erfcf
// 333 tokens over 1001 x 999 take 19.4 us instead of 18.6.)  The quick division is good to a few fp32 steps, the quick
// exponential to 1.2 |u| more: 2^-16 where e^u is about to leave fp32's range, a thirty-second of fp16's half step.
enum LinAct { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };
__device__ __forceinline__ float lin_activate1(float z, int act) {
    if (act == kActRelu) return z < 0.f ? 0.f : z;                              // NaN stays
    if (act == kActGelu) {
        const float x = fabsf(z) * 0.70710678118654752f;
        const float t = __fdividef(1.f, fmaf(0.375f, x, 1.f));
        float q = fmaf(-0.135078266f, t, 0.387873024f);
        q = fmaf(q, t, -0.129502341f);
        q = fmaf(q, t, 0.282991320f);
        q = fmaf(q, t, 0.166691899f);
        q = fmaf(q, t, 0.215683907f);
        q = fmaf(q, t, 0.211339846f);
        const float tail = 0.5f * q * t * __expf(-x * x);                       // P(-|z|)
        return z * (z < 0.f ? tail : 1.f - tail);
    }
    const float u = act == kActSilu ? z : 1.5957691216057308f * (z + 0.044715f * z * z * z);     // 2 sqrt(2 / pi)
    const float e = __expf(-fabsf(u));
    return __fdividef(u < 0.f ? z * e : z, 1.f + e);
}
__device__ __noinline__ float4 lin_activate4(float4 z, int act) {
    return make_float4(lin_activate1(z.x, act), lin_activate1(z.y, act), lin_activate1(z.z, act), lin_activate1(z.w, act));
}
template <int N>
__device__ __forceinline__ void lin_activate(float (&z)[N], int act) {
    if (act == kActNone) return;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 y = lin_activate4(make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]), act);
        z[i] = y.x;
        z[i + 1] = y.y;
        z[i + 2] = y.z;
        z[i + 3] = y.w;
    }
}

template <class T> __device__ __forceinline__ float lin_load(const T *p);
template <> __device__ __forceinline__ float lin_load<__half>(const __half *p) { return __half2float(*p); }
template <> __device__ __forceinline__ float lin_load<__nv_bfloat16>(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
template <class T> __device__ __forceinline__ float lin_float(T v) { return lin_load(&v); }
template <class T> __device__ __forceinline__ T lin_round(float v);
template <> __device__ __forceinline__ __half lin_round<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 lin_round<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

}  // namespace llvq
