// mx_fp8.cuh -- what the translation units of the FP8 block-scaled operators
// share: argument blocks, launchers, and the device helpers of their kernels.
//
// Numbers: e4m3 values with one fp32 scale for each 128 columns of an
// activation row and for each 128 x 128 block of a weight matrix.
#pragma once

#include "mx_common.cuh"
#include "mx_internal.h"
#include "mx_moe.h"

namespace mx {
namespace fp8 {

constexpr int kBlk = 128;        // columns (and weight rows) that share a scale
constexpr float kMaxE4M3 = 448.0f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: a block of zeros keeps a usable scale
constexpr int kFewTokens = 64;   // largest T of the layer's few-token form (all tokens as one operand tile)

__host__ __device__ constexpr int blocks(int n) { return (n + kBlk - 1) / kBlk; }
__host__ __device__ constexpr int64_t up16(int64_t n) { return (n + 15) & ~int64_t(15); }

// What a launch computes: kProduct in mx_fp8_gemm.cu and mx_fp8_rows.cu, kGateUp in
// the second, the others in the first.
enum Mode {
    kProduct = 0,  // out = rows x W^T, rows grouped by matrix (or one matrix)
    kGateUp = 1,   // h = Q(act(rows Wg^T) * (rows Wu^T)), rows grouped by matrix
    kFewGateUp = 2,  // the same for every active expert and the shared one, all tokens in each
    kFewDown = 3     // out = residual + lambda * (sum over the active experts' and the shared expert's blocks)
};

// Types of a product's results; kOutF16: scaled rows, with a factor for each 64 columns.
enum OutKind { kOutF32 = 0, kOutBf16 = 1, kOutF16 = 2 };

struct GemmArgs {
    CUtensorMap wa, wb;  // weights: (gate, up) or one matrix stack
    CUtensorMap sa, sb;  // few tokens: the shared expert's
    CUtensorMap xm;      // e4m3 operand rows (tokens)
    int rows;            // operand rows (an upper bound when `offsets` is given)
    int K, N, E;         // inner columns, weight rows per matrix, matrices
    const int32_t *offsets;  // [E + 1] first row of each matrix's group, nullable: one group of all rows
    const float *sx;         // operand scales: row r, block b at r * sx_r + b * sx_b
    int64_t sx_r, sx_b;
    const float *swa, *swb;  // weight scales [E][blocks(N)][blocks(K)]
    const float *ssa, *ssb;  // few tokens: the shared expert's
    void *out;               // kProduct, kFewDown
    int64_t ldo;
    int out_kind;        // kOutF32 or kOutBf16
    int out_vec;         // 16 bytes of neighbouring outputs may be stored at once
    uint8_t *h;          // kFewGateUp: e4m3 hidden tiles
    float *hs;           // their factors
    int act;             // mx_activation
    // few tokens
    const int32_t *idx;  // [T][topk]
    const float *wts;    // [T][topk]
    int T, topk, IB, SB; // hidden blocks of a routed and of the shared expert
    const void *residual;
    float lam;
    unsigned *err;
    int stages, cl;      // ring depth, cluster size (split of the inner dimension)
    unsigned cl_inv;     // kFewDown, cl > 1: 2^32 / cl rounded up
    int pdl;             // lets the next launch start before this one has ended
};

cudaError_t launch_gemm(Mode mode, int nt, const GemmArgs &a, int grid, cudaStream_t s);

// The same for many rows (mx_fp8_rows.cu): one or two products, or gate/up
// products, in one launch.
struct RowsProblem {
    CUtensorMap wa, wb, xm;
    int rows, K, N, E;       // rows 0: no second problem
    const int32_t *offsets;  // first problem only; nullable: one group of all rows
    const float *sx;
    int64_t sx_r, sx_b;
    const float *swa, *swb;
    void *out;               // kProduct
    int64_t ldo;
    int out_kind, out_vec;
    float *out_scale;        // kOutF16: a row's factor for each 64 columns
    int64_t out_scale_ld;
    uint8_t *h;              // kGateUp
    int64_t ldh;
    float *hs;
    int64_t hs_ld;
};
struct RowsArgs {
    RowsProblem p[2];
    int act;
    unsigned *err;
};
constexpr int kRowsBox = 32;  // token rows of one copy (32, 64 and 128 measured alike)

// Tiles of 128 tokens x bn (128, 256; kGateUp: 256) weight rows.
cudaError_t launch_rows(Mode mode, int bn, const RowsArgs &a, int grid, cudaStream_t s);

// Dynamic shared memory of a launch_gemm with `stages` stages.
size_t gemm_smem(Mode mode, int nt, int stages);

// One to eight rows (mx_fp8_gemv.cu).
constexpr int kGemvRows = 8;
struct GemvArgs {
    int T, K, N;  // rows, inner columns, weight rows (the layer: K = d_model)
    // product
    const uint8_t *q;
    int64_t ldq;
    const float *sx;
    int64_t sx_r, sx_b;
    const uint8_t *w;
    int64_t ldw;
    const float *sw;
    int64_t ldo;
    int out_bf16;
    void *out;
    // layer (T 1): x [K], routed gate / up / down stacks, the shared expert's (S 0: none)
    const void *x;
    int bf16, act, topk, E, I, S;
    const int32_t *idx;
    const float *wts;
    const uint8_t *w_gate, *w_up, *w_down, *sw_gate, *sw_up, *sw_down;
    int64_t ld_gate, ld_up, ld_down, ld_sgate, ld_sup, ld_sdown;
    const float *s_gate, *s_up, *s_down, *ss_gate, *ss_up, *ss_down;
    uint8_t *h8;         // hidden [block][128] e4m3 and its factors [block]
    float *hf;
    const void *residual;
    float lam;
};
cudaError_t launch_gemv(const GemvArgs &a, cudaStream_t s);
cudaError_t launch_gemv_moe(const GemvArgs &a, cudaStream_t s);
constexpr int kGemvMoeCols = 32768;  // largest d_model of launch_gemv_moe
int gemv_moe_blocks(int K);          // hidden blocks that its first launch works on at one time (0: none)

struct QuantArgs {
    const void *x;       // [rows][cols]
    int64_t rows, ldx;
    int cols, bf16, pow2;
    int vec;             // (set by the launch) rows start at multiples of 16 bytes
    uint8_t *q;          // [rows][cols], row pitch ldq
    int64_t ldq;
    float *scales;       // row r, block b at r * s_r + b * s_b
    int64_t s_r, s_b;
    // copies of each row at the positions of its slots (nullable)
    const int32_t *pos;  // [rows][topk], -1: none
    int topk;
    uint8_t *qr;         // row pitch ldq
    float *sr;           // position p, block b at p + b * sr_b
    int64_t sr_b;
    int pdl;             // let the next launch start early
};
cudaError_t launch_quantize(const QuantArgs &a, int sms, cudaStream_t s);

// Slots grouped by expert: offsets [E + 1] and pos [n] (-1 for an index outside
// [0, E)).  counts and cursor: [E] scratch.  The order inside a group is not
// fixed; no result depends on it.
cudaError_t launch_group(const int32_t *idx, int n, int E, int32_t *counts, int32_t *cursor, int32_t *offsets,
                         int32_t *pos, cudaStream_t s);

struct CombineArgs {
    const void *Y;       // [slots][D] fp32, or FP16 with a factor for each 64 columns
    const float *Yf;     // [slots][ceil(D / 64)], nullable: fp32
    const void *Ys;      // [T][D], nullable
    const float *Ysf;
    const int32_t *pos;  // [T][topk]
    const float *wts;
    const void *residual;
    void *out;
    int T, D, topk, bf16;
    float lam;
};
cudaError_t launch_combine(const CombineArgs &a, cudaStream_t s);

// ------------------------------------------------------------ device helpers

// Two floats to e4m3 (round to nearest even, saturating, NaN kept): lo in bits 0-7.
__device__ __forceinline__ uint32_t e4m3_x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The scale of a block whose largest magnitude is amax (a NaN stays one), by CUDA's
// division.  Not inlined: the compiler would otherwise run it beside the fast form
// below for every block and choose afterwards.
static __device__ __noinline__ float scale_any(float amax, int pow2)
{
    float s = __fdiv_rn(amax, kMaxE4M3);
    s = s < kMinScale ? kMinScale : s;
    if (pow2 && s < INFINITY)
        s = __uint_as_float((__float_as_uint(s) + 0x7FFFFFu) & 0xFF800000u);
    return s;
}

static __device__ __noinline__ float divide_any(float x, float s) { return __fdiv_rn(x, s); }

// Magnitudes whose quotients the fast forms round correctly: 2^-80 to 2^100.
__device__ __forceinline__ bool plain_range(float amax) { return amax >= 8.271806e-25f && amax <= 1.2676506e30f; }

// Correctly rounded x / s for many x and one s.  Markstein's theorem (IBM J. Res.
// Dev. 34, 1990): with r the correctly rounded 1 / s and q = fl(x r), fl(q + fl(x -
// q s) r) is the correctly rounded quotient as long as nothing leaves the normal
// range (a quotient below 2^-11 quantises to 0 either way).  Three instructions a
// value, or a pair of them, instead of a dozen; equal to CUDA's division on 8e9
// random and bf16 pairs, and for the scale on every amax.
__device__ __forceinline__ float divide_fast(float x, float s, float r)
{
    const float q = x * r;
    return fmaf(fmaf(-q, s, x), r, q);
}

__device__ __forceinline__ float scale_of(float amax, int pow2)
{
    if (!plain_range(amax))
        return scale_any(amax, pow2);
    const float s = divide_fast(amax, kMaxE4M3, 1.0f / kMaxE4M3);
    return pow2 ? __uint_as_float((__float_as_uint(s) + 0x7FFFFFu) & 0xFF800000u) : s;
}

// The same for a pair, in e4m3 (two bytes), from pairs of s and -r.  By way of -(x / s), whose
// sign is flipped at the end: the sum that leaves the quotient of a negative zero would make it
// a positive one, this one keeps it.
__device__ __forceinline__ uint32_t e4m3_quotients(uint64_t x, uint64_t s, uint64_t nr)
{
    uint64_t q = mul_f32x2(x, nr);
    fma_f32x2(x, q, s);
    fma_f32x2(q, x, nr);
    float lo, hi;
    unpair_f32(q, lo, hi);
    return e4m3_x2(lo, hi) ^ 0x8080u;
}

// Quotients of a hidden block, x / s for its scale s: outside the plain range both are taken
// times a power of two that brings them there, which leaves the quotient as it is (but for what
// quantises to 0 either way; an infinite or NaN scale makes it NaN).
struct Quotient {
    float s, r, m;

    __device__ __forceinline__ Quotient(float amax, float scale)
    {
        m = plain_range(amax) ? 1.0f : amax < 1.0f ? 1.2676506e30f : 9.094947e-13f;  // 2^100, 2^-40
        s = scale * m;
        r = __frcp_rn(s);
    }

    // Two values that have been taken times m, as two e4m3 bytes.
    __device__ __forceinline__ uint32_t e4m3_of(float lo, float hi) const
    {
        return e4m3_quotients(pair_f32(lo, hi), pair_f32(s, s), pair_f32(-r, -r));
    }
};

// Quantise pairs of values of a block whose largest magnitude has the bits `amax`:
// e[j] = two e4m3 bytes.  Returns the scale.
template <int N>
__device__ __forceinline__ float quantize_pairs(const uint64_t (&p)[N], uint32_t amax, int pow2, uint32_t (&e)[N])
{
    const float top = __uint_as_float(amax), s = scale_of(top, pow2);
    if (plain_range(top)) {
        const float r = __frcp_rn(s);
        const uint64_t s2 = pair_f32(s, s), nr2 = pair_f32(-r, -r);
#pragma unroll
        for (int j = 0; j < N; ++j)
            e[j] = e4m3_quotients(p[j], s2, nr2);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float lo, hi;
            unpair_f32(p[j], lo, hi);
            if (top != 0.0f)  // (not a block of zeros, as padding has them)
                lo = divide_any(lo, s), hi = divide_any(hi, s);
            e[j] = e4m3_x2(lo, hi);
        }
    }
    return s;
}

__device__ __forceinline__ float load_act(const void *p, int64_t i, int bf16)
{
    return bf16 ? bf2f(__ldg(reinterpret_cast<const uint16_t *>(p) + i)) : __ldg(reinterpret_cast<const float *>(p) + i);
}

}  // namespace fp8
}  // namespace mx
