// mx_fp8_tc.cuh -- tensor-core, TMEM, TMA and barrier helpers of the FP8 products.
#pragma once

#include "mx_fp8.cuh"

namespace mx {
namespace fp8 {

__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// e4m3 A and B (K-major), fp32 D, M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_e4m3(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | (8u << 24); }

// D = A B^T over a block of 128 columns: four MMAs of K = 32, the first of which
// overwrites D.  By one elected lane of a converged warp.  In one statement, with the
// election inside: as four statements behind a branch on it they took 200 cycles an
// MMA to issue, whatever N; so they take the 128 that N = 256 needs.
__device__ __forceinline__ void umma_block(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
                 "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
                 "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
                 "elect.sync _|q, 0xffffffff;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, !p;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, p;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, p;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc)
                 : "memory");
}

// One lane of the converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Arrive on both barriers when the MMAs issued so far are done (one elected lane).
__device__ __forceinline__ void umma_commit2(uint64_t *x, uint64_t *y)
{
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(smem_u32(x)),
                 "r"(smem_u32(y))
                 : "memory");
}

// The warp's index, known to the compiler to be the same in all its lanes.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0); }

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define MX_R16(r, o)                                                                                                \
    "=r"(r[o + 0]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), \
        "=r"(r[o + 7]), "=r"(r[o + 8]), "=r"(r[o + 9]), "=r"(r[o + 10]), "=r"(r[o + 11]), "=r"(r[o + 12]),          \
        "=r"(r[o + 13]), "=r"(r[o + 14]), "=r"(r[o + 15])

// Request 16 columns of this warp's 32 TMEM lanes; r holds them after tmem_wait.
__device__ __forceinline__ void tmem_ld16(uint32_t ta, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
                 "[%16];"
                 : MX_R16(r, 0)
                 : "r"(ta)
                 : "memory");
}

// Wait for the requested columns.
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// A column's value as it is behind the wait.
__device__ __forceinline__ float tmem_value(uint32_t r)
{
    float v;
    asm volatile("mov.b32 %0, %1;" : "=f"(v) : "r"(r));
    return v;
}

// d += (lo, hi) * f, a pair of columns.  Volatile, so that it stays behind the wait for
// lo and hi; with the registers as operands of the wait instead, the compiler moved
// each of them once or twice (1.5 moves an FMA).
__device__ __forceinline__ void fma_after(uint64_t &d, uint32_t lo, uint32_t hi, uint64_t f)
{
    asm volatile("{\n\t.reg .b64 p;\n\tmov.b64 p, {%1, %2};\n\tfma.rn.f32x2 %0, p, %3, %0;\n\t}"
                 : "+l"(d)
                 : "r"(lo), "r"(hi), "l"(f));
}

__device__ __forceinline__ void tma_2d(void *dst, const CUtensorMap *map, int c0, int c1, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
                 "%3}], [%4];" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(c0), "r"(c1), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void tma_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
                 "%3, %4}], [%5];" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Bounded wait: false once this CTA has given up.
__device__ __forceinline__ bool bwait(uint64_t *bar, uint32_t parity, unsigned *err, volatile int *abort)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort)
            return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, kErrTimeout);
            *abort = 1;
            return false;
        }
    }
    return true;
}

// The same by a whole warp: every lane gets one answer.
__device__ __forceinline__ bool wwait(uint64_t *bar, uint32_t parity, unsigned *err, volatile int *abort)
{
    return __all_sync(0xFFFFFFFFu, bwait(bar, parity, err, abort));
}

// Barrier over `count` threads that tells each whether all of them passed true.
__device__ __forceinline__ bool named_and(int id, int count, bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.and.pred q, %1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"(count), "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ float act_of(float g, int act)
{
    return act == MX_SILU ? __fdividef(g, 1.0f + __expf(-g)) : gelu_fast(g);
}

// Row groups of the matrices as token tiles of `nt` rows (one warp): tile offsets
// tt[E + 1], first rows lo[E], lengths len[E].  A group outside the rows is cut
// to them.
__device__ __forceinline__ void group_table(const int32_t *offsets, int E, int rows, int nt, int lane, int *tt, int *lo,
                                            int *len)
{
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int b = 0, c = 0;
        if (e < E) {
            b = offsets ? min(max(__ldg(offsets + e), 0), rows) : 0;
            const int d = offsets ? min(max(__ldg(offsets + e + 1), 0), rows) : rows;
            c = max(d - b, 0);
        }
        const int t = (c + nt - 1) / nt;
        int incl = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o)
                incl += y;
        }
        if (e < E) {
            tt[e] = run + incl - t;
            lo[e] = b;
            len[e] = c;
        }
        run += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0)
        tt[E] = run;
}

}  // namespace fp8
}  // namespace mx
