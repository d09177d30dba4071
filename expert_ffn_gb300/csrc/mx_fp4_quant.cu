// mx_fp4_quant.cu -- quantisation of activations to e2m1 with block scales.
//
//   e8m0  s = the smallest power of two with 6 s >= max |x|;         q = e2m1(x / s)
//   e4m3  s = e4m3(fl(max |x| * fl(1 / fl(6 t))));  q = e2m1(fl(x * fl(1 / fl(s t))))
//
// Every step is a correctly rounded fp32 operation (a power of two's product is exact), so
// the stored codes are the same on every machine.  6 = 1.5 * 4: the power of two is the
// maximum's exponent less 2, one more where its mantissa is above 1.5, and takes no division.
//
// A thread has eight neighbouring columns, a block two or four neighbouring lanes: loads
// of 16 (fp32: 32) bytes and stores of 4 are whole lines for a warp.  The pieces of the
// matrix are dealt out in order, so a ragged width leaves no warp idle; a thread's next
// piece is a constant number of rows and columns on.  HBM bounds large matrices.
#include "mx_fp4.cuh"

#include <algorithm>

namespace mx {
namespace fp4 {

namespace {

constexpr int kThreads = 256, kAhead = 4;

template <bool BF16>
struct Raw {
    uint4 r[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const QuantArgs &a, int64_t at, int n)
{
    Raw<BF16> v{};
    if (a.vx && n >= 8) {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i)
            v.r[i] = *(BF16 ? reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + at)
                            : reinterpret_cast<const uint4 *>(static_cast<const float *>(a.x) + at + 4 * i));
        return v;
    }
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        w[j] = 0;
        if (j < n)
            w[j] = BF16 ? static_cast<const uint16_t *>(a.x)[at + j] : static_cast<const uint32_t *>(a.x)[at + j];
    }
    if (BF16) {
        v.r[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    } else {
        v.r[0] = make_uint4(w[0], w[1], w[2], w[3]);
        v.r[BF16 ? 0 : 1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return v;
}

template <bool BF16>
__device__ __forceinline__ void unpack(const Raw<BF16> &r, float (&v)[8])
{
    const uint32_t w[4] = {r.r[0].x, r.r[0].y, r.r[0].z, r.r[0].w};
    if (BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const uint4 b = r.r[BF16 ? 0 : 1];
        v[0] = __uint_as_float(w[0]), v[1] = __uint_as_float(w[1]), v[2] = __uint_as_float(w[2]), v[3] = __uint_as_float(w[3]);
        v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
    }
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

template <bool BF16, int BLOCK>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantArgs a)
{
    pdl_trigger();  // (a product may set itself up meanwhile; it waits for this launch's end before it reads)
    pdl_wait();
    constexpr int LANES = BLOCK / 8, PER = kStageCols / BLOCK;  // lanes of a block; blocks of a stage
    // pieces of a row, whole stages: a block has neighbouring lanes of one warp, and the scales behind the
    // last block are written too, as zeros
    const int ppr = stages_of(a.cols) * (kStageCols / 8);
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
        Raw<BF16> raw[kAhead];
        int64_t rows[kAhead];
        int ps[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            rows[i] = row;
            ps[i] = p;
            raw[i] = row < a.rows ? load_raw<BF16>(a, row * a.ldx + 8 * p, a.cols - 8 * p) : Raw<BF16>{};
            row += dr;
            p += dp;
            if (p >= ppr)
                p -= ppr, ++row;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            float v[8];
            unpack(raw[i], v);
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1)
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
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
            const bool bad = m >= 0x7F800000u;  // a NaN or an infinity
            if (bad)
                code = BLOCK == 32 ? 255u : 127u;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = bad ? 0.0f : v[j] * inv;
            const uint32_t q = e2m1_x8(v);
            if (rows[i] < a.rows) {
                const int n = a.cols - 8 * ps[i];
                uint8_t *to = a.q + rows[i] * a.ldq + 4 * ps[i];
                if (a.vq && n >= 7) {
                    *reinterpret_cast<uint32_t *>(to) = q;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (2 * j < n)
                            to[j] = (uint8_t)(q >> (8 * j));
                }
                if (ps[i] % LANES == 0) {
                    const int b = ps[i] / LANES;
                    a.scales[((int64_t)(b / PER) * a.rows + rows[i]) * PER + b % PER] = n > 0 ? (uint8_t)code : 0;
                }
            }
        }
    }
}

template <bool BF16, int BLOCK>
cudaError_t launch_t(const QuantArgs &a, int sms, cudaStream_t s)
{
    const int64_t pieces = (int64_t)a.rows * stages_of(a.cols) * (kStageCols / 8);
    const int64_t most = 6 * (int64_t)sms, one = (pieces + kThreads - 1) / kThreads;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)std::min(most, one));
    c.blockDim = dim3(kThreads);
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, quantize_kernel<BF16, BLOCK>, a);
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
