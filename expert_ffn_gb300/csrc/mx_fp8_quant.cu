// mx_fp8_quant.cu -- the elementwise parts of the FP8 operators: quantisation of
// activations in blocks of 128 columns, the grouping of slots by expert, and the
// weighted sum of the experts' rows.
#include "mx_fp8.cuh"

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
// Half a warp per (row, block): 16 lanes of 8 columns.  A CTA covers kRows rows
// of one block column, so the scales of a block column, which the products read
// along the rows, leave in whole sectors.
constexpr int kRows = 32, kThreads = 256;

template <bool VEC>
__device__ __forceinline__ void load8(const QuantArgs &a, int64_t row, int c0, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = 0.0f;
    if (row >= a.rows)
        return;
    const int64_t at = row * a.ldx + c0;
    if (VEC && c0 + 8 <= a.cols) {
        if (a.bf16) {
            const uint4 r = ldg_u4(reinterpret_cast<const uint16_t *>(a.x) + at);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        } else {
            const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(a.x) + at);
            const float4 r0 = __ldg(p), r1 = __ldg(p + 1);
            v[0] = r0.x, v[1] = r0.y, v[2] = r0.z, v[3] = r0.w;
            v[4] = r1.x, v[5] = r1.y, v[6] = r1.z, v[7] = r1.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c0 + j < a.cols)
                v[j] = load_act(a.x, at + j, a.bf16);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint8_t *q, int64_t at, int c0, int cols, uint2 w)
{
    if (VEC && c0 + 8 <= cols) {
        *reinterpret_cast<uint2 *>(q + at) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c0 + j < cols)
                q[at + j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
    }
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantArgs a)
{
    if (a.pdl)
        pdl_trigger();
    const int tid = threadIdx.x, hw = tid >> 4, l = tid & 15;
    const int b = blockIdx.y;
    const int64_t row0 = (int64_t)blockIdx.x * kRows + hw;
    const int c0 = b * kBlk + 8 * l;
    constexpr int kPer = kRows / (kThreads / 16);
    float v[kPer][8];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        load8<VEC>(a, row0 + i * (kThreads / 16), c0, v[i]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t row = row0 + i * (kThreads / 16);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 8; o; o >>= 1)
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (row >= a.rows)
            continue;
        const float s = scale_of(__uint_as_float(m), a.pow2);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = e4m3_x2(__fdiv_rn(v[i][2 * j], s), __fdiv_rn(v[i][2 * j + 1], s));
        const uint2 q = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        if (a.q) {
            store8<VEC>(a.q, row * a.ldq + c0, c0, a.cols, q);
            if (l == 0)
                a.scales[row * a.s_r + b * a.s_b] = s;
        }
        if (a.pos)
            for (int k = 0; k < a.topk; ++k) {
                const int p = __ldg(a.pos + row * a.topk + k);
                if (p < 0)
                    continue;
                store8<VEC>(a.qr, (int64_t)p * a.ldq + c0, c0, a.cols, q);
                if (l == 0)
                    a.sr[p + b * a.sr_b] = s;
            }
    }
}

// ------------------------------------------------------------------ grouping

constexpr int kGrp = 1024;  // slots per block

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

// out[t] = residual + lambda * (Ys[t] + sum_k w_k Y[pos[t,k]]), k ascending.
// One thread per four columns.
__global__ void __launch_bounds__(256) combine_kernel(const CombineArgs a)
{
    const int t = blockIdx.y;
    const int d = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (d >= a.D)
        return;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int n = min(4, a.D - d);
    const bool vec = (a.D & 3) == 0;
    auto add = [&](const float *row, float w) {
        if (vec) {
            const float4 y = __ldg(reinterpret_cast<const float4 *>(row + d));
            acc[0] = fmaf(w, y.x, acc[0]), acc[1] = fmaf(w, y.y, acc[1]);
            acc[2] = fmaf(w, y.z, acc[2]), acc[3] = fmaf(w, y.w, acc[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n)
                    acc[j] = fmaf(w, __ldg(row + d + j), acc[j]);
        }
    };
    for (int k = 0; k < a.topk; ++k) {
        const int p = __ldg(a.pos + (int64_t)t * a.topk + k);
        if (p >= 0)
            add(a.Y + (int64_t)p * a.D, __ldg(a.wts + (int64_t)t * a.topk + k));
    }
    if (a.Ys)
        add(a.Ys + (int64_t)t * a.D, 1.0f);
    const int64_t at = (int64_t)t * a.D + d;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j >= n)
            break;
        const float v = fmaf(a.lam, acc[j], a.residual ? load_act(a.residual, at + j, a.bf16) : 0.0f);
        if (a.bf16)
            reinterpret_cast<uint16_t *>(a.out)[at + j] = f2bf(v);
        else
            reinterpret_cast<float *>(a.out)[at + j] = v;
    }
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs &a, cudaStream_t s)
{
    if (a.rows == 0)
        return cudaSuccess;
    const size_t es = a.bf16 ? 2 : 4;
    const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.ldx * es) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.q) % 8 == 0 && a.ldq % 8 == 0;
    const dim3 grid((unsigned)((a.rows + kRows - 1) / kRows), blocks(a.cols));
    if (vec)
        quantize_kernel<true><<<grid, kThreads, 0, s>>>(a);
    else
        quantize_kernel<false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_group(const int32_t *idx, int n, int E, int32_t *counts, int32_t *cursor, int32_t *offsets,
                         int32_t *pos, cudaStream_t s)
{
    cudaError_t e;
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
    // (tokens on the y axis: at most 65535 per launch)
    for (int t0 = 0; t0 < a.T; t0 += 65535) {
        CombineArgs b = a;
        const size_t es = a.bf16 ? 2 : 4;
        b.T = a.T - t0 < 65535 ? a.T - t0 : 65535;
        b.pos += (int64_t)t0 * a.topk;
        b.wts += (int64_t)t0 * a.topk;
        if (b.Ys)
            b.Ys += (int64_t)t0 * a.D;
        if (b.residual)
            b.residual = (const char *)b.residual + (int64_t)t0 * a.D * es;
        b.out = (char *)b.out + (int64_t)t0 * a.D * es;
        combine_kernel<<<dim3((a.D + 1023) / 1024, b.T), 256, 0, s>>>(b);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace fp8
}  // namespace mx
