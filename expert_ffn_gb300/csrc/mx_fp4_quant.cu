// mx_fp4_quant.cu -- quantisation of activations to e2m1 with block scales.
//
//   e8m0  s = the smallest power of two with 6 s >= max |x|;         q = e2m1(x / s)
//   e4m3  s = e4m3(fl(max |x| * fl(1 / fl(6 t))));  q = e2m1(fl(x * fl(1 / fl(s t))))
//
// Every step is a correctly rounded fp32 operation (a power of two's product is exact), so
// the stored codes are the same on every machine.  6 = 1.5 * 4: the power of two is the
// maximum's exponent less 2, one more where its mantissa is above 1.5, and takes no division.
//
// A thread has sixteen neighbouring columns, so a block of 16 is its own and a block of 32 takes
// one exchange with its neighbour; the scale and its reciprocal are worked out once for sixteen values.
// The pieces of the matrix are dealt out in order, so a ragged width leaves no warp idle; a
// thread's next piece is a constant number of rows and columns on.  HBM bounds large matrices: 32768 x 4096 bf16 take
// 58 us (0.89 of the copy rate), 4096 x 4096 9.5.  Of widths that are no multiple of 256 a row's last stage goes value by value
// through shared memory: 32768 x 704 19.2 us (8.8 by its bytes; x 768 13.0), 4096 x 2112 6.5 (3.3; x 2048 4.5).
#include "mx_fp4.cuh"
#include "mx_host.h"

#include <algorithm>

namespace mx {
namespace fp4 {

namespace {

constexpr int kThreads = 256, kPiece = 16;

// Pieces of a thread under way: 64 bytes.
template <bool BF16>
constexpr int kAhead = BF16 ? 2 : 1;

// Sixteen values as they were loaded.
template <bool BF16>
struct Raw {
    uint4 r[BF16 ? 2 : 4];
};

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const QuantArgs &a, int64_t at)
{
    Raw<BF16> v;
    const uint4 *p = BF16 ? reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + at)
                          : reinterpret_cast<const uint4 *>(static_cast<const float *>(a.x) + at);
#pragma unroll
    for (int i = 0; i < (BF16 ? 2 : 4); ++i)
        v.r[i] = p[i];
    return v;
}

// Of a ragged or misaligned stage of 256 columns, by its sixteen lanes: value by value, neighbouring
// lanes neighbouring columns, zeros behind the last of n, and exchanged through shared memory.
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_slow(const QuantArgs &a, int64_t at, int n, uint32_t *mine)
{
    const int l = threadIdx.x & 15;
    const unsigned half = 0xFFFFu << (threadIdx.x & 16);
    uint32_t w[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
        const int c = i * 16 + l;
        w[i] = 0;
        if (c < n)
            w[i] = BF16 ? static_cast<const uint16_t *>(a.x)[at + c] : static_cast<const uint32_t *>(a.x)[at + c];
    }
    __syncwarp(half);
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
        mine[i * 17 + l] = w[i];
    __syncwarp(half);
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
        w[i] = mine[l * 17 + i];
    Raw<BF16> v;
#pragma unroll
    for (int i = 0; i < (BF16 ? 2 : 4); ++i) {
        const uint32_t *b = w + (BF16 ? 8 : 4) * i;
        v.r[i] = BF16 ? make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[BF16 ? 4 : 0] | b[BF16 ? 5 : 0] << 16,
                                   b[BF16 ? 6 : 0] | b[BF16 ? 7 : 0] << 16)
                      : make_uint4(b[0], b[1], b[2], b[3]);
    }
    return v;
}

// Bits of the largest magnitude (two bf16 values to an operation).
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t largest(const Raw<true> &v)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        m = max_u16x2(m, max_u16x2(max_u16x2(v.r[i].x & 0x7FFF7FFFu, v.r[i].y & 0x7FFF7FFFu),
                                   max_u16x2(v.r[i].z & 0x7FFF7FFFu, v.r[i].w & 0x7FFF7FFFu)));
    return max(m & 0xFFFF0000u, m << 16);
}

__device__ __forceinline__ uint32_t largest(const Raw<false> &v)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max(max(max(m, v.r[i].x & 0x7FFFFFFFu), max(v.r[i].y & 0x7FFFFFFFu, v.r[i].z & 0x7FFFFFFFu)),
                v.r[i].w & 0x7FFFFFFFu);
    return m;
}

// Values 2 j and 2 j + 1.
__device__ __forceinline__ uint64_t pair_of(const Raw<true> &v, int j)
{
    const uint4 r = v.r[j >> 2];
    const uint32_t w = (j & 3) == 0 ? r.x : (j & 3) == 1 ? r.y : (j & 3) == 2 ? r.z : r.w;
    return pair_f32(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint64_t pair_of(const Raw<false> &v, int j)
{
    const uint4 r = v.r[j >> 1];
    return (j & 1) ? pair_f32(__uint_as_float(r.z), __uint_as_float(r.w)) : pair_f32(__uint_as_float(r.x), __uint_as_float(r.y));
}

// Eight e2m1 codes, the first in the lowest nibble (round to nearest even, at most 6).
__device__ __forceinline__ uint32_t e2m1_x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// An e4m3 code of a value >= 0 (at most 448), and what it stands for.
__device__ __forceinline__ uint32_t to_e4m3(float v)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xFFu;
}

__device__ __forceinline__ float from_e4m3(uint32_t c)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

// WHOLE: every stage of 256 columns is complete and may be moved in vectors.  (A kernel of its own: with the slow path in
// it half as many warps fit, 4096 x 4096 10.4 us instead of 9.5.)
template <bool BF16, int BLOCK, bool WHOLE>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantArgs a)
{
    pdl_trigger();  // (a product may set itself up meanwhile; it waits for this launch's end before it reads)
    pdl_wait();
    constexpr int PER = kStageCols / BLOCK, AHEAD = kAhead<BF16>;  // blocks of a stage
    __shared__ uint32_t swap[WHOLE ? 1 : kThreads / 16][16 * 17];
    // pieces of a row, whole stages: a block of 32 has neighbouring lanes of one warp, and the scales behind
    // the last block are written too, as zeros
    const int ppr = stages_of(a.cols) * (kStageCols / kPiece);
    const int64_t stride = (int64_t)gridDim.x * kThreads, first = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int dr = (int)(stride / ppr), dp = (int)(stride - (int64_t)dr * ppr);
    int64_t row = first / ppr;
    int p = (int)(first - row * ppr);
    float t = 1.0f, inv6t = 0.0f;
    if (BLOCK == 16) {
        if (a.tensor_scale)
            t = *a.tensor_scale;
        inv6t = __frcp_rn(__fmul_rn(6.0f, t));
    }
    // (a lane behind the last row still takes part in the warp's shuffles)
    while (__any_sync(0xFFFFFFFFu, row < a.rows)) {
        Raw<BF16> raw[AHEAD];
        int64_t rows[AHEAD];
        int ps[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            rows[i] = row;
            ps[i] = p;
            const int c0 = kPiece * (p & ~15);  // the stage's first column: the same row and stage for sixteen lanes
            raw[i] = Raw<BF16>{};
            if (row < a.rows) {
                if (WHOLE || (a.vx && c0 + kStageCols <= a.cols))
                    raw[i] = load_raw<BF16>(a, row * a.ldx + kPiece * p);
                else
                    raw[i] = load_slow<BF16>(a, row * a.ldx + c0, a.cols - c0, swap[WHOLE ? 0 : threadIdx.x >> 4]);
            }
            row += dr;
            p += dp;
            if (p >= ppr)
                p -= ppr, ++row;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            uint32_t m = largest(raw[i]);
            if (BLOCK == 32)
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            uint32_t code;
            float inv;
            if (BLOCK == 32) {
                const int e = max((int)(m >> 23) - 2 + ((m & 0x7FFFFFu) > 0x400000u), 0);
                code = (uint32_t)e;
                inv = __uint_as_float((uint32_t)(254 - e) << 23);
            } else {
                code = to_e4m3(__uint_as_float(m) * inv6t);
                const float s = from_e4m3(code) * t;
                inv = s >= 1.17549435e-38f ? __frcp_rn(s) : 0.0f;
            }
            uint32_t q[2];
            const uint64_t inv2 = pair_f32(inv, inv);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    unpair_f32(mul_f32x2(pair_of(raw[i], 4 * h + j), inv2), v[2 * j], v[2 * j + 1]);
                q[h] = e2m1_x8(v);
            }
            if (m >= 0x7F800000u) {  // a NaN or an infinity
                code = BLOCK == 32 ? 255u : 127u;
                q[0] = q[1] = 0;
            }
            if (rows[i] < a.rows) {
                const int n = a.cols - kPiece * ps[i];
                uint8_t *to = a.q + rows[i] * a.ldq + kPiece / 2 * ps[i];
                if (WHOLE || (a.vq && n >= kPiece - 1)) {
                    *reinterpret_cast<uint2 *>(to) = make_uint2(q[0], q[1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (2 * j < n)
                            to[j] = (uint8_t)(q[j >> 2] >> (8 * (j & 3)));
                }
                if (BLOCK == 16 || !(ps[i] & 1)) {
                    const int b = BLOCK == 16 ? ps[i] : ps[i] >> 1;
                    a.scales[((int64_t)(b / PER) * a.rows + rows[i]) * PER + b % PER] = n > 0 ? (uint8_t)code : 0;
                }
            }
        }
    }
}

template <bool BF16, int BLOCK>
cudaError_t launch_t(const QuantArgs &a, int sms, cudaStream_t s)
{
    const int64_t pieces = (int64_t)a.rows * stages_of(a.cols) * (kStageCols / kPiece);
    const int64_t most = 8 * (int64_t)sms, one = (pieces + kThreads - 1) / kThreads;
    const int grid = (int)std::min(most, one);
    if (a.vx && a.vq && a.cols % kStageCols == 0)
        return launch_dependent(quantize_kernel<BF16, BLOCK, true>, grid, kThreads, 0, s, a);
    return launch_dependent(quantize_kernel<BF16, BLOCK, false>, grid, kThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_quantize(int block, const QuantArgs &a, int sms, cudaStream_t s)
{
    if (block == 16)
        return a.bf16 ? launch_t<true, 16>(a, sms, s) : launch_t<false, 16>(a, sms, s);
    return a.bf16 ? launch_t<true, 32>(a, sms, s) : launch_t<false, 32>(a, sms, s);
}

}  // namespace fp4
}  // namespace mx
