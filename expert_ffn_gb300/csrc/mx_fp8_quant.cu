// mx_fp8_quant.cu -- the elementwise parts of the FP8 operators: quantisation of
// activations in blocks of 128 columns, the grouping of slots by expert, and the
// weighted sum of the experts' rows.
#include "mx_fp8.cuh"

#include <cuda_fp16.h>

namespace mx {
namespace fp8 {

namespace {

// Quantisation.  For a block of 128 columns of a row: a = max |x|, s =
// max(a / 448, 2^-126) (rounded up to a power of two on request), q = e4m3(x / s),
// both divisions correctly rounded, so the stored values are the same on every
// machine.  The maximum is taken over the bit patterns of |x|, which order as
// integers and keep a NaN or an infinity: such a block gets a NaN or infinite
// scale and dequantises to NaN instead of to plausible numbers.
//
// Half a warp per (row, block): 16 lanes of 8 columns.  A CTA of 16 half-warps
// walks down one block column, 16 neighbouring rows at a time, so the scales of a
// block column, which the products read along the rows, leave in whole sectors, and
// its addresses advance by constants; neighbouring CTAs have neighbouring block
// columns.  The bound is HBM (3 bytes a bf16 value), but only if a row of 128 takes
// few instructions: quotients go two to an instruction, the maximum of bf16 values
// is taken on pairs, the next three loads are under way, and CUDA's division, which
// made this 250 instructions instead of 90, is left to blocks of extreme magnitude.
// 4096 x 4096 bf16 values take 13 us, 3.9 TB/s (HBM 7.5); with CUDA's division 20.  A lane of
// eight values pays for four shuffles, the scale and a reciprocal.
constexpr int kThreads = 256, kHalves = kThreads / 16, kAhead = 3;

// Eight values as they were loaded.
template <bool BF16>
struct Raw {
    uint4 r[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const void *x, int64_t at)
{
    Raw<BF16> v;
    if (BF16) {
        v.r[0] = ldg_u4(reinterpret_cast<const uint16_t *>(x) + at);
    } else {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i)
            v.r[i] = ldg_u4(reinterpret_cast<const float *>(x) + at + 4 * i);
    }
    return v;
}

// Of a ragged or misaligned block: column by column, zeros behind the last.
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_slow(const void *x, int64_t at, int n)
{
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        w[j] = 0;
        if (j < n)
            w[j] = BF16 ? __ldg(reinterpret_cast<const uint16_t *>(x) + at + j)
                        : __ldg(reinterpret_cast<const uint32_t *>(x) + at + j);
    }
    Raw<BF16> v;
    if (BF16) {
        v.r[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    } else {
        v.r[0] = make_uint4(w[0], w[1], w[2], w[3]);
        v.r[BF16 ? 0 : 1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return v;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Bits of the largest magnitude among the 16 lanes' values.
__device__ __forceinline__ uint32_t largest(const Raw<true> &v)
{
    const uint4 r = v.r[0];
    uint32_t m = max_u16x2(max_u16x2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu), max_u16x2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = 8; o; o >>= 1)
        m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return max(m & 0xFFFF0000u, m << 16);
}

__device__ __forceinline__ uint32_t largest(const Raw<false> &v)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        m = max(max(max(m, v.r[i].x & 0x7FFFFFFFu), max(v.r[i].y & 0x7FFFFFFFu, v.r[i].z & 0x7FFFFFFFu)),
                v.r[i].w & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 8; o; o >>= 1)
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return m;
}

// Values 2 j and 2 j + 1.
__device__ __forceinline__ uint64_t pair_of(const Raw<true> &v, int j)
{
    const uint32_t w = j == 0 ? v.r[0].x : j == 1 ? v.r[0].y : j == 2 ? v.r[0].z : v.r[0].w;
    return pair_f32(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint64_t pair_of(const Raw<false> &v, int j)
{
    const uint4 r = v.r[j >> 1];
    return (j & 1) ? pair_f32(__uint_as_float(r.z), __uint_as_float(r.w)) : pair_f32(__uint_as_float(r.x), __uint_as_float(r.y));
}

__device__ __forceinline__ void store8(uint8_t *q, int n, bool vec, uint2 w)
{
    if (vec) {
        *reinterpret_cast<uint2 *>(q) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n)
                q[j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
    }
}

template <bool BF16, bool FULL>
__device__ __forceinline__ void quantize_column(const QuantArgs &a, int b, int64_t row, int64_t dr)
{
    const int l = threadIdx.x & 15, c = b * kBlk + 8 * l, n = a.cols - c;
    const int64_t dx = dr * a.ldx, dq = dr * a.ldq, ds = dr * a.s_r;
    int64_t xp = row * a.ldx + c, prow = row;
    uint8_t *qp = a.q + row * a.ldq + c;
    float *sp = a.scales + row * a.s_r + b * a.s_b;
    // (a half-warp whose row is behind the last still takes part in the warp's shuffles)
    auto fetch = [&]() {
        Raw<BF16> v{};
        if (prow < a.rows)
            v = FULL ? load_raw<BF16>(a.x, xp) : load_slow<BF16>(a.x, xp, n);
        xp += dx;
        prow += dr;
        return v;
    };
    Raw<BF16> v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        v[i] = fetch();
    for (int64_t first = row - (threadIdx.x >> 4); first < a.rows;) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (first >= a.rows)
                break;
            const Raw<BF16> x = v[i];
            v[i] = fetch();
            uint64_t p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p[j] = pair_of(x, j);
            uint32_t e[4];
            const float s = quantize_pairs(p, largest(x), a.pow2, e);
            const uint2 q = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
            if (row < a.rows) {
                if (a.q) {
                    store8(qp, n, FULL, q);
                    if (l == 0)
                        *sp = s;
                }
                if (a.pos)
                    for (int k = 0; k < a.topk; ++k) {
                        const int to = __ldg(a.pos + row * a.topk + k);
                        if (to < 0)
                            continue;
                        store8(a.qr + (int64_t)to * a.ldq + c, n, FULL, q);
                        if (l == 0)
                            a.sr[to + b * a.sr_b] = s;
                    }
            }
            qp += dq;
            sp += ds;
            row += dr;
            first += dr;
        }
    }
}

// gridDim.x: a multiple of the block columns.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, BF16 ? 4 : 3) quantize_kernel(const QuantArgs a)
{
    if (a.pdl)
        pdl_trigger();
    const unsigned nb = blocks(a.cols), part = blockIdx.x / nb;
    const int b = blockIdx.x - part * nb;
    const int64_t row = (int64_t)part * kHalves + (threadIdx.x >> 4), dr = (int64_t)(gridDim.x / nb) * kHalves;
    if (a.vec && (b + 1) * kBlk <= a.cols)
        quantize_column<BF16, true>(a, b, row, dr);
    else
        quantize_column<BF16, false>(a, b, row, dr);
}

// ------------------------------------------------------------------ grouping

constexpr int kGrp = 1024;     // slots per block
constexpr int kGrpOne = 4096;  // slots that one block groups by itself

// Up to kGrpOne slots: counted, scanned and ranked in shared memory by one block, one
// launch of about 3 us; more take a memset and two launches, 7 us together.
__global__ void __launch_bounds__(1024) group_one(const int32_t *__restrict__ idx, int n, int E, int32_t *offsets,
                                                  int32_t *pos)
{
    __shared__ int h[kMaxExperts], wsum[kMaxExperts / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < kMaxExperts)
        h[tid] = 0;
    __syncthreads();
    int e[kGrpOne / 1024], r[kGrpOne / 1024];
#pragma unroll
    for (int i = 0; i < kGrpOne / 1024; ++i) {
        const int s = i * 1024 + tid;
        e[i] = s < n ? __ldg(idx + s) : -1;
    }
#pragma unroll
    for (int i = 0; i < kGrpOne / 1024; ++i)
        r[i] = e[i] >= 0 && e[i] < E ? atomicAdd(&h[e[i]], 1) : -1;
    __syncthreads();
    const int c = tid < kMaxExperts ? h[tid] : 0;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o)
            incl += y;
    }
    if (tid < kMaxExperts && lane == 31)
        wsum[warp] = incl;
    __syncthreads();
    if (tid < kMaxExperts) {
        for (int w = 0; w < warp; ++w)
            incl += wsum[w];
        h[tid] = incl - c;
        if (tid < E)
            offsets[tid] = incl - c;
        if (tid == E - 1)
            offsets[E] = incl;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGrpOne / 1024; ++i) {
        const int s = i * 1024 + tid;
        if (s < n)
            pos[s] = r[i] < 0 ? -1 : h[e[i]] + r[i];
    }
}

__global__ void __launch_bounds__(256) group_count(const int32_t *__restrict__ idx, int n, int E, int32_t *counts)
{
    __shared__ int h[kMaxExperts];
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        h[e] = 0;
    __syncthreads();
    const int hi = min(n, (int)(blockIdx.x + 1) * kGrp);
    for (int s = blockIdx.x * kGrp + threadIdx.x; s < hi; s += blockDim.x) {
        const int e = __ldg(idx + s);
        if (e >= 0 && e < E)
            atomicAdd(&h[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        if (h[e])
            atomicAdd(&counts[e], h[e]);
}

// Every block scans the counts itself, ranks its slots within it in shared
// memory and reserves a range of each expert's group.
__global__ void __launch_bounds__(512) group_scatter(const int32_t *__restrict__ idx, int n, int E,
                                                     const int32_t *__restrict__ counts, int32_t *cursor,
                                                     int32_t *offsets, int32_t *pos)
{
    __shared__ int h[kMaxExperts], base[kMaxExperts], wsum[16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = tid < E ? __ldg(counts + tid) : 0;
    h[tid] = 0;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o)
            incl += y;
    }
    if (lane == 31)
        wsum[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w)
        before += wsum[w];
    const int off = before + incl - c;
    if (blockIdx.x == 0 && tid < E) {
        offsets[tid] = off;
        if (tid == E - 1)
            offsets[E] = off + c;
    }
    int e[kGrp / 512], r[kGrp / 512];
#pragma unroll
    for (int i = 0; i < kGrp / 512; ++i) {
        const int s = blockIdx.x * kGrp + i * 512 + tid;
        e[i] = s < n ? __ldg(idx + s) : -1;
        if (e[i] < 0 || e[i] >= E)
            e[i] = -1;
        r[i] = e[i] >= 0 ? atomicAdd(&h[e[i]], 1) : 0;
    }
    __syncthreads();
    if (tid < E)
        base[tid] = off + (h[tid] ? atomicAdd(&cursor[tid], h[tid]) : 0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGrp / 512; ++i) {
        const int s = blockIdx.x * kGrp + i * 512 + tid;
        if (s < n)
            pos[s] = e[i] >= 0 ? base[e[i]] + r[i] : -1;
    }
}

// ------------------------------------------------------------------- combine

// out[t] = residual + lambda * (Ys[t] + sum_k w_k Y[pos[t,k]]), k ascending, in fp32.
// A thread has 16 bytes of each row.  The positions of eight slots are read at once, then
// their rows and factors, a slot without an expert reading the first row and leaving it
// out: behind a test for each slot its load waited for the one before (4096 tokens, top-8,
// d_model 4096: 105 us, now 75; the bytes take HBM 50).
template <bool HALF>
__global__ void __launch_bounds__(256, 3) combine_kernel(const CombineArgs a)
{
    constexpr int C = HALF ? 8 : 4, kStep = 8;
    const int d = (blockIdx.x * 256 + threadIdx.x) * C;
    if (d >= a.D)
        return;
    const int n = min(C, a.D - d), nb = (a.D + 63) / 64, blk = d / 64;
    const bool vec = a.D % C == 0;
    float acc[C];
    auto load = [&](const void *y, int64_t row) -> uint4 {
        if (vec)
            return ld_stream_u4(static_cast<const char *>(y) + (row * a.D + d) * (HALF ? 2 : 4));
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < C; ++j)
            h[j] = j >= n ? 0
                 : HALF ? __ldg(static_cast<const uint16_t *>(y) + row * a.D + d + j)
                        : __ldg(static_cast<const uint32_t *>(y) + row * a.D + d + j);
        return HALF ? make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4 % C] | h[5 % C] << 16, h[6 % C] | h[7 % C] << 16)
                    : make_uint4(h[0], h[1], h[2], h[3]);
    };
    auto add = [&](const uint4 &r, float w) {
        const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const float v = HALF ? __half2float(__ushort_as_half((unsigned short)(x[j / 2 % 4] >> (16 * (j & 1)))))
                                 : __uint_as_float(x[j % 4]);
            acc[j] = fmaf(w, v, acc[j]);
        }
    };
#pragma unroll
    for (int j = 0; j < C; ++j)
        acc[j] = 0.0f;
    const int64_t t = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (t >= a.T)
        return;
    const int32_t *pos = a.pos + t * a.topk;
    const float *wts = a.wts + t * a.topk;
    uint4 shared = make_uint4(0, 0, 0, 0);
    float fs = 0.0f;
    if (a.Ys) {
        shared = load(a.Ys, t);
        fs = HALF ? __ldg(a.Ysf + t * nb + blk) : 1.0f;
    }
    for (int k0 = 0; k0 < a.topk; k0 += kStep) {
        int p[kStep];
        uint4 y[kStep];
        float w[kStep], f[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            const int k = min(k0 + i, a.topk - 1);
            p[i] = __ldg(pos + k);
            w[i] = __ldg(wts + k);
        }
#pragma unroll
        for (int i = 0; i < kStep; ++i)
            if (k0 + i < a.topk) {  // (the same for the whole grid)
                const int64_t row = max(p[i], 0);
                y[i] = load(a.Y, row);
                f[i] = HALF ? __ldg(a.Yf + row * nb + blk) : 1.0f;
            }
#pragma unroll
        for (int i = 0; i < kStep; ++i)
            if (k0 + i < a.topk && p[i] >= 0)
                add(y[i], w[i] * f[i]);
    }
    if (a.Ys)
        add(shared, fs);
    const int64_t at = t * a.D + d;
#pragma unroll
    for (int j = 0; j < C; ++j)
        acc[j] = j < n ? fmaf(a.lam, acc[j], a.residual ? load_act(a.residual, at + j, a.bf16) : 0.0f) : 0.0f;
    if (vec && HALF) {
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = f2bf(acc[2 * j % C]) | (uint32_t)f2bf(acc[(2 * j + 1) % C]) << 16;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at) = make_uint4(x[0], x[1], x[2], x[3]);
    } else if (vec) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    } else {
#pragma unroll
        for (int j = 0; j < C; ++j)
            if (j < n) {
                if (a.bf16)
                    static_cast<uint16_t *>(a.out)[at + j] = f2bf(acc[j]);
                else
                    static_cast<float *>(a.out)[at + j] = acc[j];
            }
    }
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs &a, int sms, cudaStream_t s)
{
    if (a.rows == 0)
        return cudaSuccess;
    const size_t es = a.bf16 ? 2 : 4;
    QuantArgs v = a;
    v.vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.ldx * es) % 16 == 0 &&
            reinterpret_cast<uintptr_t>(a.q) % 8 == 0 && a.ldq % 8 == 0;
    // four CTAs to an SM, in whole rows of block columns
    const int64_t groups = (a.rows + kHalves - 1) / kHalves, nb = blocks(a.cols), want = 4 * sms / nb;
    const unsigned grid = (unsigned)((want < 1 ? 1 : want < groups ? want : groups) * nb);
    if (a.bf16)
        quantize_kernel<true><<<grid, kThreads, 0, s>>>(v);
    else
        quantize_kernel<false><<<grid, kThreads, 0, s>>>(v);
    return cudaGetLastError();
}

cudaError_t launch_group(const int32_t *idx, int n, int E, int32_t *counts, int32_t *cursor, int32_t *offsets,
                         int32_t *pos, cudaStream_t s)
{
    cudaError_t e;
    if (n <= kGrpOne) {
        group_one<<<1, 1024, 0, s>>>(idx, n, E, offsets, pos);
        return cudaGetLastError();
    }
    // counts and cursor are neighbours
    if ((e = cudaMemsetAsync(counts, 0, (size_t)(cursor + E - counts) * 4, s)) != cudaSuccess)
        return e;
    const int nb = (n + kGrp - 1) / kGrp;
    group_count<<<nb, 256, 0, s>>>(idx, n, E, counts);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    group_scatter<<<nb, 512, 0, s>>>(idx, n, E, counts, cursor, offsets, pos);
    return cudaGetLastError();
}

cudaError_t launch_combine(const CombineArgs &a, cudaStream_t s)
{
    const int per = 256 * (a.Yf ? 8 : 4), ny = a.T < 32768 ? a.T : 32768;
    const dim3 grid((a.D + per - 1) / per, ny, (a.T + ny - 1) / ny);
    if (a.Yf)
        combine_kernel<true><<<grid, 256, 0, s>>>(a);
    else
        combine_kernel<false><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace fp8
}  // namespace mx
