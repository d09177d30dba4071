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
// rsqrtf, with the residual of r0^2 A = D computed exactly.
//
// What bounds it: HBM, where instructions allow it.  4096 x 4096 bf16 with residual, sum, out and
// q move 151 MB, 22.4 us at the copy rate; a warp's 256 columns took 568 instructions in a
// first form and 40 us.  So values go two to an instruction (f32x2), a warp's sums are added
// as integers (redux, at the scale of the largest: 50 bits) instead of by five exchanges of two floats,
// and one warp joins them and takes the root: 387 instructions and 30.7 us, 61 % of the issue slots and 0.73 of the copy
// rate: neither is full, warps wait at a row's two barriers most.  Of more than 4096 columns a thread has two pieces and more,
// an SM one CTA, and little covers its barriers: 4096 x 4104 60.8 us (22.7 by its bytes), x 7168 68.5 (39.6), x 16384
// 142 (90.4).
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

__device__ __forceinline__ Two add_two(Two a, Two b)
{
    float e;
    const float s = two_sum(a.hi, b.hi, e);
    return Two{s, a.lo + b.lo + e};
}

__device__ __forceinline__ uint64_t sub_f32x2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The squares of a pair of values onto a pair of sums.
template <bool EXACT>  // squares that fp32 holds
__device__ __forceinline__ void add_squares(uint64_t &hi, uint64_t &lo, uint64_t h)
{
    const uint64_t p = mul_f32x2(h, h);
    const uint64_t s = add_f32x2(hi, p), bb = sub_f32x2(s, hi);
    uint64_t e = add_f32x2(sub_f32x2(hi, sub_f32x2(s, bb)), sub_f32x2(p, bb));
    if (!EXACT) {
        uint64_t r = mul_f32x2(p, pair_f32(-1.0f, -1.0f));
        fma_f32x2(r, h, h);  // h^2 - p
        e = add_f32x2(e, r);
    }
    hi = s;
    lo = add_f32x2(lo, e);
}

__device__ __forceinline__ uint32_t bf16_x2(uint64_t v)
{
    float lo, hi;
    unpair_f32(v, lo, hi);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint64_t of_bf16_x2(uint32_t w)
{
    return pair_f32(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Eight neighbouring values as they were loaded, zeros behind the last of n.
template <bool BF16>
struct Raw {
    uint4 r[BF16 ? 1 : 2];
};

template <bool BF16, bool FAST>
__device__ __forceinline__ Raw<BF16> load8(const char *p, uint32_t at, int n, bool vec)
{
    Raw<BF16> v{};
    if (FAST && n <= 0)
        return v;
    if (FAST || (vec && n >= 8)) {
        const uint4 *q = reinterpret_cast<const uint4 *>(p + at * (BF16 ? 2 : 4));
        v.r[0] = q[0];
        if (!BF16)
            v.r[BF16 ? 0 : 1] = q[1];
    } else {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = 0;
            if (j < n)
                w[j] = BF16 ? reinterpret_cast<const uint16_t *>(p)[at + j] : reinterpret_cast<const uint32_t *>(p)[at + j];
        }
        if (BF16) {
            v.r[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        } else {
            v.r[0] = make_uint4(w[0], w[1], w[2], w[3]);
            v.r[BF16 ? 0 : 1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
    return v;
}

// The same as pairs.
template <bool BF16>
__device__ __forceinline__ void pairs(const Raw<BF16> &x, uint64_t (&v)[4])
{
    const uint4 a = x.r[0], b = x.r[BF16 ? 0 : 1];
    if (BF16) {
        v[0] = of_bf16_x2(a.x), v[1] = of_bf16_x2(a.y), v[2] = of_bf16_x2(a.z), v[3] = of_bf16_x2(a.w);
    } else {
        v[0] = pair_f32(__uint_as_float(a.x), __uint_as_float(a.y)), v[1] = pair_f32(__uint_as_float(a.z), __uint_as_float(a.w));
        v[2] = pair_f32(__uint_as_float(b.x), __uint_as_float(b.y)), v[3] = pair_f32(__uint_as_float(b.z), __uint_as_float(b.w));
    }
}

template <bool BF16, bool FAST>
__device__ __forceinline__ void store8(char *p, uint32_t at, int n, bool vec, const uint64_t (&v)[4])
{
    if (FAST && n <= 0)
        return;
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        unpair_f32(v[j], f[2 * j], f[2 * j + 1]);
    if (FAST || (vec && n >= 8)) {
        if (BF16) {
            *reinterpret_cast<uint4 *>(p + at * 2) = make_uint4(bf16_x2(v[0]), bf16_x2(v[1]), bf16_x2(v[2]), bf16_x2(v[3]));
        } else {
            float4 *to = reinterpret_cast<float4 *>(p + at * 4);
            to[0] = make_float4(f[0], f[1], f[2], f[3]);
            to[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) {
                if (BF16)
                    reinterpret_cast<uint16_t *>(p)[at + j] = f2bf(f[j]);
                else
                    reinterpret_cast<float *>(p)[at + j] = f[j];
            }
    }
}

// A warp's sum of hi + lo (hi >= 0, lo within half an ulp of it) as integers: hi below 2^25 at the scale
// of the warp's largest, the rest in units 2^-25 of that.  Every lane gets it.
struct Part {
    int hi, lo;
    uint32_t top;  // bits of the largest hi
};
__device__ __forceinline__ int part_scale(uint32_t top) { return 151 - max((int)(top >> 23), 27); }
__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(127 + k) << 23); }

__device__ __forceinline__ Part warp_part(float hi, float lo)
{
    Part p;
    p.top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(hi));  // (a NaN's bits are above infinity's)
    const float f = pow2(part_scale(p.top)), h = hi * f;
    const int hi_i = __float2int_rn(h);
    const int lo_i = __float2int_rn(((h - (float)hi_i) + __fmul_rn(lo, f)) * 33554432.0f);
    p.hi = __reduce_add_sync(0xFFFFFFFFu, hi_i);
    p.lo = __reduce_add_sync(0xFFFFFFFFu, lo_i);
    return p;
}

__device__ __forceinline__ Two of_part(Part p)
{
    if (p.top >= 0x7F800000u)
        return Two{__uint_as_float(p.top), 0.0f};
    const float g = pow2(-part_scale(p.top));
    const float hi = (float)(p.hi & ~127), lo = (float)(p.hi & 127) + (float)p.lo * 2.9802322e-8f;
    return Two{hi * g, lo * g};
}

// f sqrt(D / (S + D eps)), rounded once; f: a power of two, and S and eps those of f h.
__device__ __forceinline__ float root(Two S, float D, float eps, float f)
{
    const float pe = __fmul_rn(D, eps), ee = fmaf(D, eps, -pe);
    float t;
    const float b = two_sum(S.hi, pe, t), bl = S.lo + t + ee;
    const float a = b + bl, al = bl - (a - b);
    if (!(a > 0.0f && a < INFINITY))
        return a == 0.0f ? INFINITY : S.hi != S.hi ? NAN : 0.0f;
    float r0 = rsqrtf(__fdividef(a, D));
    if (f < 1.0f)  // (of 20 bits, so that f r0 is exact where it is subnormal)
        r0 = __uint_as_float(__float_as_uint(r0) & ~15u);
    const float th = __fmul_rn(r0, r0), tl = fmaf(r0, r0, -th), u = __fmul_rn(th, a), ul = fmaf(th, a, -u);
    const float rho = ((D - u) - ul) - fmaf(tl, a, th * al);
    const float d = __fdividef(rho, D);  // r0^2 A / D = 1 - d
    const float c = d * fmaf(0.375f, d, 0.5f);
    return f < 1.0f ? fmaf(r0 * f, c, r0 * f) : fmaf(r0, c, r0) * f;
}

// The largest of m, |a| and |b|; a NaN stays one.
__device__ __forceinline__ float max_abs(float m, float a, float b)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

// A CTA takes every gridDim.x-th row; the next one's loads are under way while one is worked on (`AHEAD`).
// FAST: every tensor may be moved in whole pieces, and the columns end with one.
template <bool BF16, int V, bool FAST>
__global__ void __launch_bounds__(512, V == 1 ? (BF16 ? 3 : 2) : 1) norm_kernel(const Args a)
{
    constexpr bool AHEAD = V <= 2;
    __shared__ Part part[32];
    __shared__ float shared_r, shared_f;
    const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5, lane = tid & 31;
    const float D = (float)a.cols;
    // first column of piece i, and how many of the eight there are
    auto column = [&](int i) { return (i * threads + tid) * 8; };
    auto count = [&](int i) { return FAST ? (column(i) < a.cols ? 8 : 0) : a.cols - column(i); };
    constexpr int ES = BF16 ? 2 : 4;
    // (rows by addresses that the whole CTA shares, a thread's columns by 32-bit offsets)
    auto row_of = [](const void *p, int64_t at) { return const_cast<char *>(static_cast<const char *>(p)) + at; };
    Raw<BF16> x[V], res[V];
    auto fetch = [&](int64_t row) {
        const char *px = row_of(a.x, row * a.ldx * ES), *pr = row_of(a.residual, row * a.ldr * ES);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = load8<BF16, FAST>(px, column(i), count(i), a.vx);
            if (a.residual)
                res[i] = load8<BF16, FAST>(pr, column(i), count(i), a.vr);
        }
    };
    // (the launch behind may set itself up; it waits for this one's end)
    pdl_trigger();
    pdl_wait();
    if (AHEAD)
        fetch(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (!AHEAD)
            fetch(row);
        uint64_t h[V][4];
        char *psum = row_of(a.sum, row * a.lds * ES);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            pairs<BF16>(x[i], h[i]);
            if (a.residual) {
                uint64_t r[4];
                pairs<BF16>(res[i], r);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[i][j] = add_f32x2(h[i][j], r[j]);
                if (BF16) {
                    Raw<true> w;
                    w.r[0] = make_uint4(bf16_x2(h[i][0]), bf16_x2(h[i][1]), bf16_x2(h[i][2]), bf16_x2(h[i][3]));
                    pairs<true>(w, h[i]);
                    if (FAST && a.sum && count(i) > 0)
                        *reinterpret_cast<uint4 *>(psum + column(i) * 2) = w.r[0];
                }
            }
            if (a.sum && !(BF16 && FAST && a.residual))
                store8<BF16, FAST>(psum, column(i), count(i), a.vs, h[i]);
        }
        if (AHEAD && row + gridDim.x < a.rows)
            fetch(row + gridDim.x);
        if (!a.out && !a.q)
            continue;

        float r, f = 1.0f;
        // (a second time, with h times a power of two, where squares leave fp32's range)
        for (int pass = 0;; ++pass) {
            uint64_t hi2 = 0, lo2 = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (pass == 0)
                        add_squares<BF16>(hi2, lo2, h[i][j]);
                    else
                        add_squares<false>(hi2, lo2, mul_f32x2(h[i][j], pair_f32(f, f)));
                }
            float h0, h1, l0, l1, e;
            unpair_f32(hi2, h0, h1);
            unpair_f32(lo2, l0, l1);
            const float s = two_sum(h0, h1, e), l = l0 + l1 + e, hi = s + l, lo = l - (hi - s);
            const Part p = warp_part(s < INFINITY ? hi : s, lo);
            if (lane == 0)
                part[tid >> 5] = p;
            __syncthreads();
            if (tid < 32) {
                Two S = lane < warps ? of_part(part[lane]) : Two{0.0f, 0.0f};
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    S = add_two(S, Two{__shfl_xor_sync(0xFFFFFFFFu, S.hi, o), __shfl_xor_sync(0xFFFFFFFFu, S.lo, o)});
                // h times 2^-80: its largest square, from 2^85 on, comes to 2^-75 to 2^96.  Times 2^60 where S + D eps is at
                // most 2^-60; times 2^110, which takes the least h to 2^-39, where that is below 2^-100.
                float g = 0.0f;  // (done)
                if (pass == 0 && !(S.hi < 0x1p100f && S.hi + D * a.eps > 0x1p-60f))
                    g = !(S.hi < 1.0f) ? 0x1p-80f : S.hi + D * a.eps > 0x1p-100f ? 0x1p60f : 0x1p110f;
                if (lane == 0) {
                    shared_r = root(S, D, a.eps * f * f, f);
                    shared_f = g;
                }
            }
            __syncthreads();
            r = shared_r;
            if (shared_f == 0.0f)
                break;
            f = shared_f;
        }

        const uint64_t r2 = pair_f32(r, r), off2 = pair_f32(a.offset, a.offset);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = column(i), n = count(i);
            uint64_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = mul_f32x2(h[i][j], r2);
            if (a.weight) {
                uint64_t w[4];
                if (a.w_bf16)
                    pairs<true>(load8<true, FAST>(static_cast<const char *>(a.weight), c, n, a.vw), w);
                else
                    pairs<false>(load8<false, FAST>(static_cast<const char *>(a.weight), c, n, a.vw), w);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    y[j] = mul_f32x2(y[j], add_f32x2(off2, w[j]));
            }
            if (n < 8) {  // (behind the last column: zeros, whatever r is)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lo, hi;
                    unpair_f32(y[j], lo, hi);
                    y[j] = FAST ? 0 : pair_f32(2 * j < n ? lo : 0.0f, 2 * j + 1 < n ? hi : 0.0f);
                }
            }
            if (a.out) {
                char *po = row_of(a.out, row * a.ldo * (a.out_bf16 ? 2 : 4));
                if (a.out_bf16)
                    store8<true, FAST>(po, c, n, a.vo, y);
                else
                    store8<false, FAST>(po, c, n, a.vo, y);
            }
            if (a.q) {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lo, hi;
                    unpair_f32(y[j], lo, hi);
                    top = max_abs(top, lo, hi);
                }
                uint32_t m = __float_as_uint(top);
#pragma unroll
                for (int o = 8; o; o >>= 1)
                    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                uint32_t e[4];
                const float s = fp8::quantize_pairs(y, m, a.pow2, e);
                if (n > 0) {
                    char *q = row_of(a.q, row * a.ldq);
                    const uint2 w = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
                    if (FAST || (a.vq && n >= 8)) {
                        *reinterpret_cast<uint2 *>(q + (uint32_t)c) = w;
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < n)
                                reinterpret_cast<uint8_t *>(q)[c + j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
                    }
                    if ((tid & 15) == 0)
                        (a.scales + row * a.s_r)[(int64_t)(c / kBlk) * a.s_b] = s;
                }
            }
        }
    }
}

template <bool BF16, int V>
cudaError_t launch_v(const Args &a, int threads, cudaStream_t s)
{
    const bool fast = a.vx && a.cols % 8 == 0 && (!a.residual || a.vr) && (!a.sum || a.vs) && (!a.out || a.vo) &&
                      (!a.q || a.vq) && (!a.weight || a.vw);
    const int per_sm = V == 1 ? (BF16 ? 1536 : 1024) / threads : 1;
    const int grid = std::min(a.rows, num_sms() * std::max(1, per_sm));
    return fast ? launch_dependent(norm_kernel<BF16, V, true>, grid, threads, 0, s, a)
                : launch_dependent(norm_kernel<BF16, V, false>, grid, threads, 0, s, a);
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
    if (!(n->eps >= 0.0f && n->eps <= 1e30f) || !std::isfinite(n->weight_offset))
        return fail(MX_ERR_INVALID_ARG, "eps must be in [0, 1e30], weight_offset finite");
    const mx_fp8_rows &q = n->q;
    if (q.q && (q.rows != n->rows || q.cols != n->cols))
        return fail(MX_ERR_INVALID_ARG, "q is [%d, %d], x is [%d, %d]", q.rows, q.cols, n->rows, n->cols);
    if (n->rows == 0)
        return MX_OK;
    if (!n->sum && !n->out && !q.q)
        return fail(MX_ERR_INVALID_ARG, "one of sum, out and q must be given");
    if (!n->x)
        return fail(MX_ERR_INVALID_ARG, "x is NULL");
    if ((st = norm::check_operand(n->x, n->ldx, n->cols, n->dtype, "x")) != MX_OK ||
        (n->residual && (st = norm::check_operand(n->residual, n->ldr, n->cols, n->dtype, "residual")) != MX_OK) ||
        (n->sum && (st = norm::check_operand(n->sum, n->lds, n->cols, n->dtype, "sum")) != MX_OK) ||
        (n->out && (st = norm::check_operand(n->out, n->ldo, n->cols, n->out_dtype, "out")) != MX_OK))
        return st;
    if (n->weight && !aligned(n->weight, dtype_bytes(n->weight_dtype)))
        return fail(MX_ERR_ALIGNMENT, "weight is misaligned");
    // in place: a thread reads its columns of a row before it writes them, so the rows have to be the same
    if (n->sum && ((n->sum == n->x && n->lds != n->ldx) || (n->sum == n->residual && n->lds != n->ldr)))
        return fail(MX_ERR_INVALID_ARG, "sum in place of x or residual needs the same row pitch");
    if (n->out && ((n->out == n->x && (n->ldo != n->ldx || n->out_dtype != n->dtype)) ||
                   (n->out == n->residual && (n->ldo != n->ldr || n->out_dtype != n->dtype))))
        return fail(MX_ERR_INVALID_ARG, "out in place of x or residual needs the same type and row pitch");
    if ((n->sum && n->sum == n->out) || (q.q && (q.q == n->sum || q.q == n->out || q.q == n->x || q.q == n->residual)))
        return fail(MX_ERR_INVALID_ARG, "sum, out and q must be different buffers, q none of the inputs");
    const int es = (int)dtype_bytes(n->dtype), bf16 = n->dtype == MX_BF16;
    norm::Args a{};
    if (q.q) {
        if (!q.scales)
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
