// mx_fp4_gemv.cu -- one row times a microscaled e2m1 matrix.
//
// Twice an e2m1 number is an integer (0, 1, 2, 3, 4, 6, 8, 12, and their negatives), so a block's sum
// of products is an exact integer sum, dp4a on bytes:
//   4 sum q q' = P - 2 N,  P = dp4a(|2q|, 2q'),  N the same over the negative q alone
// A byte permutation looks four magnitudes up by their codes, and another, in its mode that repeats a
// byte's sign by the selector's top bit, which is the code's sign, makes the mask of the negative ones.
// 13 instructions for eight weights, a few more for a block's scales.
//
// A warp has one weight row, a lane 32 neighbouring columns of each 1024; a CTA has sixteen rows, four lines of the
// packed scales (rows i, 32 + i, 64 + i, 96 + i), so that these are read whole.  The row of activations is
// turned into signed bytes in shared memory once per CTA, behind the first requests for weights.
//
// What bounds it: the launch and two trips to memory.
#include "mx_fp4.cuh"
#include "mx_host.h"

namespace mx {
namespace fp4 {

namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kChunk = 1024;  // columns of a warp's step
constexpr int kAhead = 4;     // steps under way

constexpr uint32_t kMagLo = 0x03020100u, kMagHi = 0x0C080604u;  // |2q| by code

__device__ __forceinline__ uint32_t magnitudes(uint32_t codes) { return __byte_perm(kMagLo, kMagHi, codes & 0x7777u); }
// 0xFF for a negative code, else 0x80 (which no magnitude has)
__device__ __forceinline__ uint32_t negative(uint32_t codes)
{
    uint32_t r;  // (__byte_perm would mask the selector's sign bits away)
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(r) : "r"(0x80808080u), "r"(codes));
    return r;
}

// Four signed bytes 2q of four codes.
__device__ __forceinline__ uint32_t signed_bytes(uint32_t codes)
{
    const uint32_t m = (negative(codes) & 0x01010101u) * 255u;
    return __vsub4(magnitudes(codes) ^ m, m);
}

template <int BLOCK>
__device__ __forceinline__ float scale_value(uint32_t byte)
{
    if (BLOCK == 32)
        return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

// acc + n f g for a block's sum n of products.  Two e8m0 scales may leave fp32's range together where the block's term does
// not (n = 0, or the one far below 1), so the smaller meets n first, exactly; two e4m3 scales do not.
template <int BLOCK>
__device__ __forceinline__ float add_block(float acc, int n, float f, float g)
{
    if (BLOCK == 16)
        return fmaf((float)n, f * g, acc);
    float lo;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(lo) : "f"(f), "f"(g));
    return fmaf((float)n * lo, fmaxf(f, g), acc);
}

// Read once: kept out of L1.  (Not by the read-only path: the launch may have begun before its predecessor's end.)
__device__ __forceinline__ uint4 load_once(const void *p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

template <int BLOCK>
__global__ void __launch_bounds__(kThreads) gemv_kernel(const GemvArgs a)
{
    constexpr int NA = atoms_of(BLOCK), NB = 32 / BLOCK, PER = kStageCols / BLOCK;  // blocks of a lane's piece, of a stage
    extern __shared__ __align__(16) uint8_t xs[];  // 2q of the row [padded], then a quarter of its scales
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int chunks = (a.K + kChunk - 1) / kChunk, padded = chunks * kChunk;
    float *fs = reinterpret_cast<float *>(xs + padded);
    const int f = blockIdx.x >> 3, line = (blockIdx.x & 7) * 4 + (warp >> 2), group = warp & 3;
    const int row = f * 128 + group * 32 + line;
    const bool live = row < a.N;
    const int KB = stages_of(a.K);
    const uint8_t *w = a.w + (int64_t)(live ? row : 0) * a.ldw;
    const uint8_t *sw = a.sw + (int64_t)f * KB * NA * 512 + line * 16 + group * 4;
    pdl_wait();

    uint4 v[kAhead];
    uint32_t s[kAhead];
    auto fetch = [&](int c, uint4 &q, uint32_t &scales) {
        const int col = c * kChunk + 32 * lane;
        q = make_uint4(0, 0, 0, 0);
        scales = 0;
        if (live && col < a.K) {
            q = load_once(w + col / 2);
            const int b = col / BLOCK;
            const uint8_t *p = sw + (int64_t)(b / 4) * 512 + b % 4;
            scales = NB == 2 ? *reinterpret_cast<const uint16_t *>(p) : *p;
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        fetch(i, v[i], s[i]);

    const Factors t = factors_of(a.tx ? *a.tx : 1.0f, a.tw ? *a.tw : 1.0f);

    for (int i = tid; i < padded / 8; i += kThreads) {
        uint32_t q = 0;
        if (8 * i < a.K) {
            q = reinterpret_cast<const uint32_t *>(a.q)[i];
            if (8 * i + 8 > a.K)  // (what lies behind the last column is not a part of the row)
                q &= 0xFFFFFFFFu >> (4 * (8 * i + 8 - a.K));
        }
        reinterpret_cast<uint2 *>(xs)[i] = make_uint2(signed_bytes(q), signed_bytes(q >> 16));
    }
    for (int b = tid; b < padded / BLOCK; b += kThreads)
        fs[b] = b * BLOCK < a.K ? 0.25f * scale_value<BLOCK>(a.sx[(int64_t)(b / PER) * PER + b % PER]) : 0.0f;
    __syncthreads();

    float acc = 0.0f;
    for (int c0 = 0; c0 < chunks; c0 += kAhead)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int c = c0 + i, col = c * kChunk + 32 * lane;
            if (c >= chunks)
                break;
            const uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            const uint32_t sc = s[i];
            fetch(c + kAhead, v[i], s[i]);
            const uint4 x0 = *reinterpret_cast<const uint4 *>(xs + col), x1 = *reinterpret_cast<const uint4 *>(xs + col + 16);
            const uint32_t x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            int p[NB] = {}, n[NB] = {};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t codes = (j & 1) ? q[j >> 1] >> 16 : q[j >> 1];
                const uint32_t m = magnitudes(codes);
                const int b = j * NB / 8;
                p[b] = __dp4a((int)m, (int)x[j], p[b]);
                n[b] = __dp4a((int)(m & negative(codes)), (int)x[j], n[b]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (col + b * BLOCK < a.K)  // (a scale behind the last block is not read)
                    acc = add_block<BLOCK>(acc, p[b] - 2 * n[b], scale_value<BLOCK>(sc >> (8 * b) & 255u), fs[col / BLOCK + b]);
        }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
    if (lane == 0 && live) {
        const float y = acc * t.a * t.b;
        if (a.out_bf16)
            static_cast<uint16_t *>(a.out)[row] = f2bf(y);
        else
            static_cast<float *>(a.out)[row] = y;
    }
}

template <int BLOCK>
cudaError_t launch_t(const GemvArgs &a, cudaStream_t s)
{
    const int padded = (a.K + kChunk - 1) / kChunk * kChunk;
    return launch_dependent(gemv_kernel<BLOCK>, (a.N + 127) / 128 * 8, kThreads, padded + padded / BLOCK * 4, s, a);
}

}  // namespace

cudaError_t launch_gemv(int block, const GemvArgs &a, cudaStream_t s)
{
    return block == 16 ? launch_t<16>(a, s) : launch_t<32>(a, s);
}

}  // namespace fp4
}  // namespace mx
