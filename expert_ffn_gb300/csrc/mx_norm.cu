// mx_norm.cu -- RMS norm with the residual's addition and an e4m3 output.
//
//   h = x + residual;  r = 1 / sqrt(mean(h^2) + eps);  y = (h r) w;  (q, s) = quantise(y)
//
// One CTA per row, one pass over memory: a thread keeps V pieces of eight
// neighbouring columns of h in registers from the load to the stores, so that sixteen
// lanes hold one block of 128 columns, which they quantise as mx_fp8_quant.cu does.
//
// Exactness.  e4m3 numbers lie 2^-3 apart, so a statistic that is off by an ulp moves a
// few values of a large matrix to their neighbours.  The sum of squares is
// therefore kept as two floats (Knuth's two-sum; a bf16 square is exact in fp32, an fp32
// square's error comes from an fma), and the root is rounded once: Newton's correction of
// rsqrtf, with the residual of r0^2 A = D computed exactly.  That is about ten
// instructions a value, which a kernel bound by memory has to spare.
//
// What bounds it: HBM.  4096 x 4096 bf16 with residual, sum, out and q move 151 MB, 22.4 us at
// the copy rate.
#include "mx_fp8.cuh"
#include "mx_host.h"

#include <algorithm>
#include <cmath>

namespace mx {
namespace norm {

namespace {

using fp8::kBlk;

constexpr int kMaxCols = 32768;

struct Args {
    const void *x, *residual, *weight;
    void *sum, *out;
    uint8_t *q;
    float *scales;
    int64_t ldx, ldr, lds, ldo, ldq, s_r, s_b;
    int rows, cols;
    int w_bf16, out_bf16, pow2;
    int vx, vr, vw, vs, vo, vq;  // pieces of these may be moved as vectors
    float eps, offset;
};

struct Two {
    float hi, lo;
};

// a + b = s + error, exactly.  (__fmul_rn below keeps the compiler from making an fma of a
// product and the sum that it enters.)
__device__ __forceinline__ float two_sum(float a, float b, float &err)
{
    const float s = a + b, bb = s - a;
    err = (a - (s - bb)) + (b - bb);
    return s;
}

__device__ __forceinline__ void add_square(Two &t, float h, bool exact)
{
    const float p = __fmul_rn(h, h);
    float e;
    t.hi = two_sum(t.hi, p, e);
    t.lo += exact ? e : e + fmaf(h, h, -p);
}

__device__ __forceinline__ Two add_two(Two a, Two b)
{
    float e;
    const float s = two_sum(a.hi, b.hi, e);
    return Two{s, a.lo + b.lo + e};
}

template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t at, int n, bool vec, float (&v)[8])
{
    if (vec && n >= 8) {
        if (BF16) {
            const uint4 r = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
            const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
            const float4 a = f[0], b = f[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = 0.0f;
            if (j < n)
                v[j] = BF16 ? bf2f(static_cast<const uint16_t *>(p)[at + j]) : static_cast<const float *>(p)[at + j];
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t at, int n, bool vec, const float (&v)[8])
{
    if (vec && n >= 8) {
        if (BF16) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = f2bf(v[2 * i]) | (uint32_t)f2bf(v[2 * i + 1]) << 16;
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
            f[0] = make_float4(v[0], v[1], v[2], v[3]);
            f[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) {
                if (BF16)
                    static_cast<uint16_t *>(p)[at + j] = f2bf(v[j]);
                else
                    static_cast<float *>(p)[at + j] = v[j];
            }
    }
}

// Sum over the CTA's threads: every thread gets the same two floats.
__device__ __forceinline__ Two block_sum(Two t, Two *part, int warps)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        t = add_two(t, Two{__shfl_xor_sync(0xFFFFFFFFu, t.hi, o), __shfl_xor_sync(0xFFFFFFFFu, t.lo, o)});
    if (lane == 0)
        part[threadIdx.x >> 5] = t;
    __syncthreads();
    t = lane < warps ? part[lane] : Two{0.0f, 0.0f};
    for (int o = 16; o; o >>= 1)
        if (o < warps)
            t = add_two(t, Two{__shfl_xor_sync(0xFFFFFFFFu, t.hi, o), __shfl_xor_sync(0xFFFFFFFFu, t.lo, o)});
    t.hi = __shfl_sync(0xFFFFFFFFu, t.hi, 0);
    t.lo = __shfl_sync(0xFFFFFFFFu, t.lo, 0);
    return t;
}

// sqrt(D / (S + D eps)), rounded once.
__device__ __forceinline__ float root(Two S, float D, float eps)
{
    const float pe = __fmul_rn(D, eps), ee = fmaf(D, eps, -pe);
    float t;
    const float b = two_sum(S.hi, pe, t), bl = S.lo + t + ee;
    const float a = b + bl, al = bl - (a - b);
    if (!(a > 0.0f && a < INFINITY))
        return a == 0.0f ? INFINITY : S.hi != S.hi ? NAN : 0.0f;
    const float r0 = rsqrtf(__fdividef(a, D));
    const float th = __fmul_rn(r0, r0), tl = fmaf(r0, r0, -th), u = __fmul_rn(th, a), ul = fmaf(th, a, -u);
    const float rho = ((D - u) - ul) - fmaf(tl, a, th * al);
    const float d = __fdividef(rho, D);  // r0^2 A / D = 1 - d
    return fmaf(r0, d * fmaf(0.375f, d, 0.5f), r0);
}

template <bool BF16, int V>
__global__ void norm_kernel(const Args a)
{
    __shared__ Two part[2][32];
    const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5;
    const int64_t row = blockIdx.x;
    const float D = (float)a.cols;
    float h[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (i * threads + tid) * 8, n = a.cols - c;
        load8<BF16>(a.x, row * a.ldx + c, n, a.vx, h[i]);
    }
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * threads + tid) * 8, n = a.cols - c;
            float r[8];
            load8<BF16>(a.residual, row * a.ldr + c, n, a.vr, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] += r[j];
                if (BF16)
                    h[i][j] = bf2f(f2bf(h[i][j]));
            }
        }
    }
    if (a.sum) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * threads + tid) * 8, n = a.cols - c;
            store8<BF16>(a.sum, row * a.lds + c, n, a.vs, h[i]);
        }
    }
    if (!a.out && !a.q)
        return;
    Two S{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            add_square(S, h[i][j], BF16);
    S = block_sum(S, part[0], warps);
    float r;
    if (S.hi < 1.2676506e30f && S.hi + D * a.eps > 8.6736174e-19f) {
        r = root(S, D, a.eps);
    } else {
        // squares beyond fp32's range (2^100, 2^-60): once more with h times a power of two
        const float f = S.hi < 1.0f ? 1.1529215e18f : 8.4703295e-22f;  // 2^60, 2^-70
        S = Two{0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                add_square(S, h[i][j] * f, false);
        S = block_sum(S, part[1], warps);
        r = root(S, D, a.eps * f * f) * f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (i * threads + tid) * 8, n = a.cols - c;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = j < n ? h[i][j] * r : 0.0f;
        if (a.weight) {
            float w[8];
            if (a.w_bf16)
                load8<true>(a.weight, c, n, a.vw, w);
            else
                load8<false>(a.weight, c, n, a.vw, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n)
                    y[j] *= a.offset + w[j];
        }
        if (a.out) {
            if (a.out_bf16)
                store8<true>(a.out, row * a.ldo + c, n, a.vo, y);
            else
                store8<false>(a.out, row * a.ldo + c, n, a.vo, y);
        }
        if (a.q) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m = max(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
#pragma unroll
            for (int o = 8; o; o >>= 1)
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            uint64_t p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p[j] = pair_f32(y[2 * j], y[2 * j + 1]);
            uint32_t e[4];
            const float s = fp8::quantize_pairs(p, m, a.pow2, e);
            if (n > 0) {
                uint8_t *q = a.q + row * a.ldq + c;
                const uint2 w = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
                if (a.vq && n >= 8) {
                    *reinterpret_cast<uint2 *>(q) = w;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < n)
                            q[j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
                }
                if ((tid & 15) == 0)
                    a.scales[row * a.s_r + (int64_t)(c / kBlk) * a.s_b] = s;
            }
        }
    }
}

template <bool BF16, int V>
cudaError_t launch_v(const Args &a, int threads, cudaStream_t s)
{
    norm_kernel<BF16, V><<<a.rows, threads, 0, s>>>(a);
    return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch(const Args &a, cudaStream_t s)
{
    const int pieces = (a.cols + 7) / 8;
    const int V = pieces <= 512 ? 1 : pieces <= 1024 ? 2 : pieces <= 2048 ? 4 : 8;
    const int threads = ((pieces + V - 1) / V + 31) / 32 * 32;
    switch (V) {
    case 1: return launch_v<BF16, 1>(a, threads, s);
    case 2: return launch_v<BF16, 2>(a, threads, s);
    case 4: return launch_v<BF16, 4>(a, threads, s);
    default: return launch_v<BF16, 8>(a, threads, s);
    }
}

mx_status check_operand(const void *p, int64_t ld, int cols, int dtype, const char *name)
{
    if (ld < cols)
        return fail(MX_ERR_INVALID_ARG, "%s: row pitch %lld is below the %d columns", name, (long long)ld, cols);
    if (ld > ((int64_t)1 << 36))
        return fail(MX_ERR_UNSUPPORTED, "%s: row pitch %lld is too large", name, (long long)ld);
    if (!aligned(p, dtype_bytes(dtype)))
        return fail(MX_ERR_ALIGNMENT, "%s is misaligned", name);
    return MX_OK;
}

}  // namespace
}  // namespace norm
}  // namespace mx

using namespace mx;

extern "C" mx_status mx_fp8_rmsnorm(const mx_rmsnorm *n, void *stream)
{
    mx_status st;
    if (!n)
        return fail(MX_ERR_INVALID_ARG, "args is NULL");
    if ((st = check_dtype(n->dtype, "dtype")) != MX_OK ||
        (n->weight && (st = check_dtype(n->weight_dtype, "weight_dtype")) != MX_OK) ||
        (n->out && (st = check_dtype(n->out_dtype, "out_dtype")) != MX_OK))
        return st;
    if (n->rows < 0)
        return fail(MX_ERR_INVALID_ARG, "%d rows", n->rows);
    if (n->cols < 1 || n->cols > norm::kMaxCols)
        return fail(MX_ERR_UNSUPPORTED, "%d columns must be within [1, %d]", n->cols, norm::kMaxCols);
    if (n->pow2 != 0 && n->pow2 != 1)
        return fail(MX_ERR_INVALID_ARG, "pow2 %d is not 0 or 1", n->pow2);
    if (!(n->eps >= 0.0f) || !std::isfinite(n->eps) || !std::isfinite(n->weight_offset))
        return fail(MX_ERR_INVALID_ARG, "eps must be finite and at least 0, weight_offset finite");
    if (!n->sum && !n->out && !n->q)
        return fail(MX_ERR_INVALID_ARG, "one of sum, out and q must be given");
    if (n->q && (n->q->rows != n->rows || n->q->cols != n->cols))
        return fail(MX_ERR_INVALID_ARG, "q is [%d, %d], x is [%d, %d]", n->q->rows, n->q->cols, n->rows, n->cols);
    if (n->rows == 0)
        return MX_OK;
    if (!n->x)
        return fail(MX_ERR_INVALID_ARG, "x is NULL");
    if ((st = norm::check_operand(n->x, n->ldx, n->cols, n->dtype, "x")) != MX_OK ||
        (n->residual && (st = norm::check_operand(n->residual, n->ldr, n->cols, n->dtype, "residual")) != MX_OK) ||
        (n->sum && (st = norm::check_operand(n->sum, n->lds, n->cols, n->dtype, "sum")) != MX_OK) ||
        (n->out && (st = norm::check_operand(n->out, n->ldo, n->cols, n->out_dtype, "out")) != MX_OK))
        return st;
    if (n->weight && !aligned(n->weight, dtype_bytes(n->weight_dtype)))
        return fail(MX_ERR_ALIGNMENT, "weight is misaligned");
    const int es = (int)dtype_bytes(n->dtype), bf16 = n->dtype == MX_BF16;
    norm::Args a{};
    if (n->q) {
        const mx_fp8_rows &q = *n->q;
        if (!q.q || !q.scales)
            return fail(MX_ERR_INVALID_ARG, "q has a NULL pointer");
        if (q.ld < q.cols || q.scale_row < 0 || q.scale_block < 0)
            return fail(MX_ERR_INVALID_ARG, "q: row pitch %lld is below its %d columns, or a scale stride is negative",
                        (long long)q.ld, q.cols);
        if (q.ld > ((int64_t)1 << 36))
            return fail(MX_ERR_UNSUPPORTED, "q: row pitch %lld is too large", (long long)q.ld);
        if (!aligned(q.scales, 4))
            return fail(MX_ERR_ALIGNMENT, "q: scales must be 4-byte aligned");
        a.q = static_cast<uint8_t *>(q.q);
        a.scales = q.scales;
        a.ldq = q.ld;
        a.s_r = q.scale_row;
        a.s_b = q.scale_block;
        a.vq = aligned(q.q, 8) && q.ld % 8 == 0;
    }
    a.x = n->x;
    a.residual = n->residual;
    a.weight = n->weight;
    a.sum = n->sum;
    a.out = n->out;
    a.ldx = n->ldx;
    a.ldr = n->ldr;
    a.lds = n->lds;
    a.ldo = n->ldo;
    a.rows = n->rows;
    a.cols = n->cols;
    a.w_bf16 = n->weight_dtype == MX_BF16;
    a.out_bf16 = n->out_dtype == MX_BF16;
    a.pow2 = n->pow2;
    a.vx = aligned(n->x, 16) && n->ldx * es % 16 == 0;
    a.vr = aligned(n->residual, 16) && n->ldr * es % 16 == 0;
    a.vs = aligned(n->sum, 16) && n->lds * es % 16 == 0;
    a.vo = vec16(n->out, n->ldo, a.out_bf16);
    a.vw = aligned(n->weight, 16);
    a.eps = n->eps;
    a.offset = n->weight_offset;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = bf16 ? norm::launch<true>(a, s) : norm::launch<false>(a, s);
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "RMS norm");
}
