// linear.cu -- host side of the compressed linear layers (llvq_linear, llvq_linear_grouped): argument
// checks, the workspace's layout, tensor maps and the two launches of a call.  Kernels:
// linear_dequant.cuh, linear_product.cuh.
#include <algorithm>
#include <cuda.h>

#include "codec.h"
#include "linear_dequant.cuh"
#include "linear_product.cuh"

using namespace llvq;

namespace {

constexpr int kMaxColumnBlocks = 0xFFFF;                   // column field of a record
// Activations of this many values, or in rows this long, that are restated at all are restated by a kernel of their
// own, others beside the decode, where a warp takes a token: 8192 tokens over 2048 x 5504 168 us against 203, 4096
// over 4096 x 4096 133 against 137, 512 over 1024 x 1024 26 against 19 (one more launch).
constexpr long long kStageValues = 1 << 21;
constexpr int kStageCols = 4096;
// A wait of the product covers a whole tile (milliseconds for the longest rows), not one round of few products:
// 16 times the polls
constexpr uint32_t kWaitRounds = 16;
constexpr long long kMaxRunRows = 0xFFFF;                  // row field of a record

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
uint32_t reciprocal(uint32_t d) { return d > 1 ? (uint32_t)(((1ull << 32) + d - 1) / d) : 0u; }

// Makes the codec's device current for a scope.
struct DeviceScope {
    int before = -1;
    bool ok = false, moved = false;
    explicit DeviceScope(int device) {
        if (cudaGetDevice(&before) != cudaSuccess) return;
        ok = before == device || (moved = true, cudaSetDevice(device) == cudaSuccess);
    }
    ~DeviceScope() {
        if (moved) cudaSetDevice(before);
    }
};

// The layer of one call and the places of its workspace.
struct Plan {
    int experts = 1, rows = 0, outs = 0;                   // matrices, their rows, outputs per token
    int stage = 0;                                         // LinArgs::stage
    long long held = 0;                                    // rows of the decoded weight
    long long w_pitch = 0, xs_pitch = 0;
    bool dots = false;                                     // few tokens: no decoded weight
    bool far = false;                                      // ... with the activations in the workspace
    int parts = 1, terms = 0;                              // LinArgs::parts, terms
    size_t w = 0, row_scale = 0, counters = 0, partial = 0, xs = 0, token_scale = 0, bytes = 0;
};

llvq_status refuse(const char *why, llvq_status st = LLVQ_ERR_ARG) {
    g_last_error = why;
    return st;
}

constexpr size_t kSmemLimit = 232448;                      // opt-in shared memory per block on sm_100

size_t dequant_smem(int bits, int out, bool grouped, long long tokens, int nb) {
    return (bits == 48 ? dq48_fixed() : bits == 72 ? dq_fixed<Dec72>() : dq_fixed<Dec96>()) + dq_tail(out, grouped, tokens, nb);
}
int dequant_ctas(int bits) { return bits == 48 ? 1 : bits == 72 ? Dec72::kCtasPerSm : Dec96::kCtasPerSm; }

// Whether a call multiplies its tokens block by block as they are decoded (no decoded weight, no tile product).
// Every further token of an expert costs such a call 3.6 ps per block, the other form about 10 us and 48
// written bytes per block once.  Measured on one matrix, with and without a decoded weight: 4096 x 4096, 1 / 2 / 3
// tokens 27.8 / 30.5 / 33.5 us against 37.4; 22016 x 4096, 1 / 3 tokens 103 / 130 us against 145.  Over experts
// what counts is how many tokens one gets, two on average: 8 tokens over 4 experts of 2816 x 2048 40.6 us against
// 41.9, 16 over 8 of 1408 x 1024 27.0 against 27.6.  Larger budgets decode more slowly, in both forms, and turn at
// the same place: 4096 x 4096, 1 / 3 / 4 fp16 tokens at 72 bits 72.2 / 76.8 / 78.6 us against 79.5 (bf16: 4 tokens 80.9
// against 79.7), at 96 bits 141.6 / 146.8 / 149.3 against 152.5; 16 over 8 experts 64.0 against 67.3 and 121 against 132.
// Decoded weights of two parts (gated fp16) cost twice as much, and their layers turn later: 4096 x 4096, 4 / 5 tokens
// 35.7 / 38.2 us against 43.5; 22016 x 2048, 4 / 6 / 8 tokens 78 / 93 / 109 against 107; 2048 x 2048, 6 / 8 tokens
// 20.1 / 21.6 against 25; at 72 bits 22016 x 4096, 6 / 8 tokens 410 / 445 against 419; 9 over 3 experts of 5632 x 2048
// 64 against 94, 16 over 8 of 1408 x 1024 29.4 against 39.9.
//
// Activations that do not fit in shared memory beside the decoder's tables are restated in the workspace and read
// through L1, dearer per token: two tokens of one matrix (4096 x 11008: 70.7 us against 74.5; one of 8192 x 28672
// 287 against 341), four over as many experts (1408 x 7168: 51 against 59), else one for every fourth expert (16 over
// 64 of 1408 x 7168 196 against 221, over 16 162 against 121).
enum Few { kManyTokens, kFewNear, kFewFar };
Few few_tokens(int bits, bool grouped, bool two_parts, int64_t tokens, int experts, int nb) {
    const int near = std::max(two_parts ? 6 : 3, experts > 1 ? std::min((two_parts ? 3 : 2) * experts, kLinDots) : 1);
    if (tokens > near) return kManyTokens;
    if (dequant_smem(bits, kDqDots, grouped, tokens, nb) <= kSmemLimit / dequant_ctas(bits) - 1024) return kFewNear;
    return tokens <= std::max({2, std::min(experts, 4), experts / 4}) ? kFewFar : kManyTokens;
}

// Checks a call (everything but the workspace) and lays out its workspace.
llvq_status make_plan(const llvq_codec *c, const llvq_weight *w, const llvq_linear_call *q, bool grouped, Plan &p) {
    g_last_error.clear();
    if (!c || !q) return refuse("null codec or call");
    const llvq_status st = check_weight(c, w);
    if (st != LLVQ_OK) return refuse("weight: null or misaligned pointer, size, pitch or budget mismatch");
    if (w->cols < 1) return refuse("a linear layer has at least one column");
    if (q->tokens < 0 || q->tokens > 1ll << 30) return refuse("tokens out of range");
    if (q->dtype != LLVQ_DTYPE_FP16 && q->dtype != LLVQ_DTYPE_BF16) return refuse("dtype is neither fp16 nor bf16");
    if (q->activation < LLVQ_ACT_NONE || q->activation > LLVQ_ACT_SILU) return refuse("unknown activation");
    if (q->gated != 0 && q->gated != 1) return refuse("gated is 0 or 1");
    if (grouped) {
        if (q->experts < 1) return refuse("experts out of range");
        if (q->experts > kLinExperts) return refuse("more than 2048 experts", LLVQ_ERR_UNSUPPORTED);
        if (w->rows % q->experts) return refuse("the weight's rows are not a multiple of the experts");
        p.experts = q->experts;
    } else if (q->experts != 0 && q->experts != 1) {
        return refuse("experts without groups");
    }
    p.rows = w->rows / p.experts;
    if (q->gated && p.rows % 2) return refuse("a gated layer has an even number of weight rows");
    p.outs = q->gated ? p.rows / 2 : p.rows;
    if (q->x_stride < w->cols && q->tokens > 1) return refuse("x_stride below the columns");
    if (q->y_stride < p.outs && q->tokens > 1) return refuse("y_stride below the outputs");
    if (q->residual && q->residual_stride < p.outs && q->residual_stride != 0 && q->tokens > 1)
        return refuse("residual_stride below the outputs and not zero");
    if (!aligned(q->x, 2) || !aligned(q->y, 2) || !aligned(q->bias, 2) || !aligned(q->residual, 2) || !aligned(q->offsets, 4))
        return refuse("misaligned pointer");
    if (w->blocks_per_row > kMaxColumnBlocks) return refuse("more than 65535 blocks per row", LLVQ_ERR_UNSUPPORTED);
    // only experts that have a token are decoded, and there are at most as many as tokens
    p.held = (long long)p.rows * std::min<long long>(p.experts, std::max<long long>(q->tokens, 1));
    if ((p.held + c->num_sms - 1) / c->num_sms + 2 > kMaxRunRows) return refuse("too many rows", LLVQ_ERR_UNSUPPORTED);
    // whole 128-byte lines per row: a box row that straddles two lines costs the tensor copies twice
    p.w_pitch = ((long long)w->blocks_per_row * 24 + 63) / 64 * 64;
    p.xs_pitch = ((long long)w->cols + 63) / 64 * 64;
    p.terms = w->cols;
    size_t at = 0;
    auto place = [&](size_t bytes) {
        const size_t here = at;
        at += round256(bytes);
        return here;
    };
    const bool two_parts = q->gated && q->dtype == LLVQ_DTYPE_FP16;
    const Few few = few_tokens(c->index_bits, grouped, two_parts, q->tokens, p.experts, w->blocks_per_row);
    if (few != kManyTokens) {
        p.dots = true;
        p.w = place((size_t)q->tokens * p.held * w->blocks_per_row * sizeof(float));
        p.far = few == kFewFar;
        if (p.far) {
            p.xs_pitch = (long long)w->blocks_per_row * 24;
            p.xs = place((size_t)q->tokens * p.xs_pitch * sizeof(__half));
            p.token_scale = place((size_t)q->tokens * sizeof(float));
        }
        p.bytes = at;
        return LLVQ_OK;
    }
    // more than two tokens from here on
    p.stage = q->dtype == LLVQ_DTYPE_BF16 ? 2 : aligned(q->x, 16) && q->x_stride % 8 == 0 ? 0 : 1;
    if (two_parts) {
        p.parts = 2;
        p.stage = 1;
        p.terms = w->blocks_per_row * 48;
        p.w_pitch = p.xs_pitch = ((long long)p.terms + 63) / 64 * 64;
    }
    p.w = place((size_t)p.held * p.w_pitch * sizeof(__half));
    p.row_scale = place((size_t)p.held * sizeof(float));
    p.counters = place((size_t)c->pairs * kLpCounters * sizeof(unsigned));
    p.partial = place((size_t)c->pairs * 2 * kLinTokens * 128 * sizeof(float));
    if (p.stage) p.xs = place((size_t)q->tokens * p.xs_pitch * sizeof(__half));
    if (p.stage == 2) p.token_scale = place((size_t)q->tokens * sizeof(float));
    p.bytes = at;
    return LLVQ_OK;
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult got;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got) != cudaSuccess ||
            got != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

// fp16 matrix [rows][cols] of the given pitch as a map of boxes of box_rows rows x 64 columns, in the
// product's swizzled layout; reads beyond rows or cols give zero.
bool make_map(CUtensorMap &m, const void *base, long long rows, long long cols, long long pitch, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
    const cuuint32_t box[2] = {(cuuint32_t)kLpK, (cuuint32_t)box_rows}, unit[2] = {1, 1};
    return encode_tiled()(&m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(base), dims, strides, box, unit,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch whose prologue may overlap the end of the kernel before it on the stream.
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

cudaError_t launch_stage(const llvq_codec *c, const LinArgs &a, bool bf16, int units, cudaStream_t st) {
    const dim3 grid((unsigned)std::min<long long>(a.tokens, (long long)c->num_sms * 32));
    const int threads = std::min(kLinStageMost, (units + 127) / 128 * 32);
    return launch(bf16 ? k_linear_stage<true> : k_linear_stage<false>, grid, threads, 0, st, a, units);
}

template <int OUT, bool GROUPED>
cudaError_t launch_dequant(const llvq_codec *c, const llvq_weight *w, const LinArgs &a, cudaStream_t st) {
    const size_t smem = dequant_smem(c->index_bits, OUT, GROUPED, a.tokens, a.nb);
    const int grid = c->num_sms * dequant_ctas(c->index_bits);
    if (c->index_bits == 48) {
        Dq48Args d{};
        d.image = (const SmemGv48 *)c->d_gv48;
        d.npoints = (unsigned long long)c->npoints;
        d.tabC = c->d_tabC48;
        d.words = (const unsigned long long *)w->words;
        d.wait_tries = g_first_wait_tries.load();
        auto kernel = w->gain_mode == LLVQ_GAIN_FP16_DIRECT ? k_dequant48<OUT, 0, GROUPED> : k_dequant48<OUT, 1, GROUPED>;
        return launch(kernel, dim3((unsigned)grid), kDqThreads, smem, st, a, d);
    }
    const unsigned long long lo = (unsigned long long)c->npoints, hi = (unsigned long long)(c->npoints >> 64);
    if (c->index_bits == 72) {
        const Dec72::Args d{(const Smem72 *)c->d_image, c->d_recs72, c->d_guide72, lo, hi};
        return launch(k_dequant<Dec72, OUT, GROUPED>, dim3((unsigned)grid), 512, smem, st, a, d, (const Dec72::Word *)w->words);
    }
    const Dec96::Args d{(const Smem96 *)c->d_image, c->d_recs96, c->d_guide96, lo, (uint32_t)hi};
    return launch(k_dequant<Dec96, OUT, GROUPED>, dim3((unsigned)grid), 512, smem, st, a, d, (const Dec96::Word *)w->words);
}

template <bool GROUPED, bool GATED, class T>
cudaError_t launch_finish(const LinArgs &a, const DqEnds &e, cudaStream_t st) {
    const int outs = GATED ? a.half : a.rows;
    const int each = kDqFinishWarps * 32 / finish_width(a.nb);             // outputs of a block
    const int blocks = std::min((outs + each - 1) / each, 4096);
    auto kernel = finish_width(a.nb) == 32  ? k_linear_finish<GROUPED, GATED, T, 32>
                  : finish_width(a.nb) == 8 ? k_linear_finish<GROUPED, GATED, T, 8>
                                            : k_linear_finish<GROUPED, GATED, T, 1>;
    return launch(kernel, dim3((unsigned)blocks, (unsigned)a.tokens), 32 * kDqFinishWarps, 0, st, a, e);
}
template <bool GROUPED>
cudaError_t finish_dispatch(const LinArgs &a, const DqEnds &e, bool gated, bool bf16, cudaStream_t st) {
    if (gated) return bf16 ? launch_finish<GROUPED, true, __nv_bfloat16>(a, e, st) : launch_finish<GROUPED, true, __half>(a, e, st);
    return bf16 ? launch_finish<GROUPED, false, __nv_bfloat16>(a, e, st) : launch_finish<GROUPED, false, __half>(a, e, st);
}

template <bool GROUPED, bool GATED, class T>
cudaError_t launch_product(const llvq_codec *c, const LpMaps &m, const LpArgs &a, cudaStream_t st) {
    return launch(k_linear_product<GROUPED, GATED, T>, dim3((unsigned)(2 * c->pairs)), kLpThreads, lp_smem(GROUPED), st, m, a);
}
template <bool GROUPED>
cudaError_t product_dispatch(const llvq_codec *c, const LpMaps &m, const LpArgs &a, bool gated, bool bf16, cudaStream_t st) {
    if (gated) return bf16 ? launch_product<GROUPED, true, __nv_bfloat16>(c, m, a, st) : launch_product<GROUPED, true, __half>(c, m, a, st);
    return bf16 ? launch_product<GROUPED, false, __nv_bfloat16>(c, m, a, st) : launch_product<GROUPED, false, __half>(c, m, a, st);
}

llvq_status run_linear(const llvq_codec *c, const llvq_weight *w, const llvq_linear_call *q, bool grouped, void *workspace,
                       size_t workspace_bytes, void *stream) {
    Plan p;
    const llvq_status st = make_plan(c, w, q, grouped, p);
    if (st != LLVQ_OK) return st;
    if (q->tokens == 0 || p.rows == 0) return LLVQ_OK;
    if (!q->x || !q->y) return refuse("null x or y");
    if (q->x == q->y) return refuse("y is x: other outputs still need what would be overwritten");
    if (q->residual == q->y && q->tokens > 1 && q->residual_stride != q->y_stride)
        return refuse("the residual is y with another stride: rows are overwritten that others still add");
    if (grouped != (q->offsets != nullptr)) return refuse(grouped ? "null offsets" : "offsets without groups");
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < p.bytes) return refuse("workspace null, misaligned or too small");
    DeviceScope scope(c->device);
    if (!scope.ok) return LLVQ_ERR_CUDA;
    unsigned char *ws = (unsigned char *)workspace;
    LpArgs a{};
    LinArgs &l = a.lin;
    l.rows = p.rows;
    l.half = q->gated ? p.rows / 2 : 0;
    l.cols = w->cols;
    l.nb = w->blocks_per_row;
    l.experts = p.experts;
    l.gain_mode = w->gain_mode;
    l.gains = (const __half *)w->gains;
    l.word_pitch = w->row_pitch_words;
    l.offsets = grouped ? q->offsets : nullptr;
    l.tokens = q->tokens;
    l.W = (__half *)(ws + p.w);
    l.ldw = p.w_pitch;
    l.parts = p.parts;
    l.terms = p.terms;
    l.row_scale = (float *)(ws + p.row_scale);
    l.rows_recip = reciprocal((uint32_t)p.rows);
    l.nb_recip = reciprocal((uint32_t)l.nb);
    l.counters = (unsigned *)(ws + p.counters);
    l.ncounters = c->pairs * kLpCounters;
    l.stage = p.stage;
    l.X = q->x;
    l.ldx = q->x_stride;
    l.Xs = (__half *)(ws + p.xs);
    l.ldxs = p.xs_pitch;
    l.token_scale = (float *)(ws + p.token_scale);
    l.dots = (float *)(ws + p.w);
    l.held = p.held;
    l.bf16 = q->dtype == LLVQ_DTYPE_BF16;
    l.flags = c->d_flags;
    cudaStream_t s = (cudaStream_t)stream;
    const bool bf16 = l.bf16;
    if (p.dots) {
        const DqEnds ends{q->bias, q->residual, q->residual_stride, q->y, q->y_stride, q->activation};
        cudaError_t e = p.far ? launch_stage(c, l, bf16, 3 * l.nb, s) : cudaSuccess;
        if (e == cudaSuccess)
            e = p.far ? (grouped ? launch_dequant<kDqDotsFar, true>(c, w, l, s) : launch_dequant<kDqDotsFar, false>(c, w, l, s))
                      : (grouped ? launch_dequant<kDqDots, true>(c, w, l, s) : launch_dequant<kDqDots, false>(c, w, l, s));
        if (e == cudaSuccess) e = grouped ? finish_dispatch<true>(l, ends, q->gated, bf16, s) : finish_dispatch<false>(l, ends, q->gated, bf16, s);
        return e == cudaSuccess ? LLVQ_OK : refuse(cudaGetErrorString(e), LLVQ_ERR_CUDA);
    }
    if (!encode_tiled()) return refuse("the driver has no cuTensorMapEncodeTiled", LLVQ_ERR_CUDA);
    a.bias = q->bias;
    a.residual = q->residual;
    a.ld_res = q->residual_stride;
    a.Y = q->y;
    a.ldy = q->y_stride;
    a.act = q->activation;
    a.partial = (float *)(ws + p.partial);
    a.wait_tries = std::min(g_mma_wait_tries.load(), 1u << 27) * kWaitRounds;
    LpMaps m;
    bool ok = make_map(m.w, l.W, p.held, l.terms, l.ldw, 128);
    const void *x = p.stage ? (const void *)l.Xs : q->x;
    for (int b = 0; b < 4; b++) ok = ok && make_map(m.x[b], x, q->tokens, l.terms, p.stage ? p.xs_pitch : q->x_stride, 128 >> b);
    if (!ok) return refuse("sizes or strides beyond a tensor map", LLVQ_ERR_UNSUPPORTED);
    cudaError_t e = cudaSuccess;
    LinArgs first = l;
    if (l.stage && (l.cols > kStageCols || q->tokens * l.cols >= kStageValues)) {
        e = launch_stage(c, l, bf16, p.parts == 2 ? 3 * l.nb : (l.cols + 7) / 8, s);
        first.stage = 0;
    }
    if (e == cudaSuccess)
        e = p.parts == 1 ? (grouped ? launch_dequant<kDqWeights, true>(c, w, first, s) : launch_dequant<kDqWeights, false>(c, w, first, s))
                         : (grouped ? launch_dequant<kDqTwoParts, true>(c, w, first, s) : launch_dequant<kDqTwoParts, false>(c, w, first, s));
    if (e == cudaSuccess)
        e = grouped ? product_dispatch<true>(c, m, a, q->gated, bf16, s) : product_dispatch<false>(c, m, a, q->gated, bf16, s);
    if (e == cudaSuccess) return LLVQ_OK;
    return refuse(cudaGetErrorString(e), LLVQ_ERR_CUDA);
}

// The largest dynamic shared memory of every kernel of the layers; the first error.
template <bool GROUPED>
cudaError_t allow_all() {
    cudaError_t e = cudaSuccess;
    auto allow = [&](auto kernel, size_t smem) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    };
    allow(k_dequant48<kDqWeights, 0, GROUPED>, kSmemLimit);
    allow(k_dequant48<kDqWeights, 1, GROUPED>, kSmemLimit);
    allow(k_dequant48<kDqTwoParts, 0, GROUPED>, kSmemLimit);
    allow(k_dequant48<kDqTwoParts, 1, GROUPED>, kSmemLimit);
    allow(k_dequant48<kDqDots, 0, GROUPED>, kSmemLimit);
    allow(k_dequant48<kDqDots, 1, GROUPED>, kSmemLimit);
    allow(k_dequant48<kDqDotsFar, 0, GROUPED>, kSmemLimit);
    allow(k_dequant48<kDqDotsFar, 1, GROUPED>, kSmemLimit);
    allow(k_dequant<Dec72, kDqWeights, GROUPED>, kSmemLimit);
    allow(k_dequant<Dec72, kDqTwoParts, GROUPED>, kSmemLimit);
    allow(k_dequant<Dec72, kDqDots, GROUPED>, kSmemLimit);
    allow(k_dequant<Dec72, kDqDotsFar, GROUPED>, kSmemLimit);
    allow(k_dequant<Dec96, kDqWeights, GROUPED>, kSmemLimit);
    allow(k_dequant<Dec96, kDqTwoParts, GROUPED>, kSmemLimit);
    allow(k_dequant<Dec96, kDqDots, GROUPED>, kSmemLimit);
    allow(k_dequant<Dec96, kDqDotsFar, GROUPED>, kSmemLimit);
    allow(k_linear_product<GROUPED, false, __half>, lp_smem(GROUPED));
    allow(k_linear_product<GROUPED, true, __half>, lp_smem(GROUPED));
    allow(k_linear_product<GROUPED, false, __nv_bfloat16>, lp_smem(GROUPED));
    allow(k_linear_product<GROUPED, true, __nv_bfloat16>, lp_smem(GROUPED));
    return e;
}

}  // namespace

cudaError_t llvq::set_linear_attrs(llvq_codec *c) {
    static_assert(dq48_fixed() + dq_tail(kDqWeights, true, 0, 0) <= kSmemLimit && lp_smem(true) <= kSmemLimit, "shared memory of an SM");
    cudaError_t e = allow_all<false>();
    if (e == cudaSuccess) e = allow_all<true>();
    if (e != cudaSuccess) return e;
    // pairs of CTAs that are resident at once, one CTA per SM
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(c->num_sms / 2 * 2));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = lp_smem(true);
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, k_linear_product<true, false, __half>, &cfg);
    if (e != cudaSuccess) return e;
    c->pairs = std::max(1, std::min(n, c->num_sms / 2));
    encode_tiled();                                        // looked up here, not inside a stream capture
    return cudaSuccess;
}

extern "C" {

size_t llvq_linear_workspace(const llvq_codec *c, const llvq_weight *w, const llvq_linear_call *q) {
    Plan p;
    return make_plan(c, w, q, q && q->experts > 0, p) == LLVQ_OK ? p.bytes : 0;
}

llvq_status llvq_linear(const llvq_codec *c, const llvq_weight *w, const llvq_linear_call *q, void *workspace,
                        size_t workspace_bytes, void *stream) {
    return run_linear(c, w, q, false, workspace, workspace_bytes, stream);
}

llvq_status llvq_linear_grouped(const llvq_codec *c, const llvq_weight *w, const llvq_linear_call *q, void *workspace,
                                size_t workspace_bytes, void *stream) {
    return run_linear(c, w, q, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
