// mx_fp8_gemm.cu -- products of e4m3 rows with block-scaled e4m3 matrices on the
// 5th-generation tensor cores (tcgen05, accumulators in TMEM).
//
//   y[m, o] = sum_b (sx[m, b] * sw[o / 128, b]) * sum_{k in block b} qx[m, k] qw[o, k]
//
// The tensor core sums one block of 128 columns; the block's scales are applied
// in fp32 by CUDA cores, which keep the running sums in registers.  The weights
// take the M side of the MMA (128 rows = one block of weight scales, so the
// weight scale is one number per MMA tile and block) and the tokens its N side
// (16 to 256): a single token then costs the smallest N, a group of tokens is
// padded to 16 rather than to 128, and weights stream from HBM straight into
// the MMA's operand layout without passing through a thread.
//
// A CTA walks units (128 weight rows x one token tile, or what Mode says).  Warps:
//   0 .. EW-1  sums: tcgen05.ld of a block's products (lane quadrant = warp % 4;
//              with EW = 8 two warpgroups take alternate chunks of 16 tokens),
//              packed two-lane FMA by the block's factors, and the epilogue
//   EW         TMA producer: weight tiles 128 x 128 bytes and token tiles
//              (SWIZZLE_128B) into a ring of stages
//   EW + 1     MMA: one lane issues four tcgen05.mma (K = 32) per matrix and block
//              into a ring of TMEM buffers
//   EW + 2     factors: sx * sw of a block for each token into a ring in shared
//              memory, so that the summing warps read them as broadcast vectors
// Few units: a cluster of `cl` CTAs splits the inner dimension; each CTA reduces
// every cl-th token column over the others' partial sums, which they store into
// its shared memory, in rank order, so the result does not depend on timing.
//
// Every wait is bounded: a wait that gives up sets the caller's error word and
// ends the CTA's work.
#include "mx_fp8.cuh"

namespace mx {
namespace fp8 {

namespace {

constexpr uint32_t kTile = 128 * 128;  // bytes of one weight tile
constexpr int kFacRing = 8;            // blocks of factors in flight

constexpr int epi_warps(int nt) { return nt > 64 ? 8 : 4; }
constexpr int n_mats(int mode) { return mode == kGateUp || mode == kFewGateUp ? 2 : 1; }
// TMEM buffers: at most 256 columns up to 64 tokens (two CTAs of an SM share 512).
constexpr int n_acc(int mode, int nt)
{
    const int cols = n_mats(mode) * nt, lim = nt > 64 ? 512 : 256;
    return lim / cols > 4 ? 4 : lim / cols;
}
constexpr uint32_t tmem_cols(int mode, int nt)
{
    uint32_t c = 32;
    while (c < (uint32_t)(n_acc(mode, nt) * n_mats(mode) * nt))
        c *= 2;
    return c;
}
constexpr uint32_t stage_bytes(int mode, int nt) { return n_mats(mode) * kTile + nt * 128; }

// Dynamic shared memory after the ring (byte offsets from its end).
struct Tail {
    int fac, am, red, tab, bars, total;
};
__host__ __device__ constexpr Tail tail_of(int mode, int nt, int cl, int ncol_own)
{
    Tail t{};
    int o = 0;
    t.fac = o;
    o += kFacRing * n_mats(mode) * nt * 4;
    t.am = o;  // per-warp column maxima (two units) and reciprocal scales
    if (n_mats(mode) == 2)
        o += 3 * 4 * nt * 4;
    t.red = o;  // partial sums of the other CTAs of the cluster
    if (cl > 1)
        o += cl * ncol_own * n_mats(mode) * 128 * 4;
    t.tab = o;  // expert tables
    o += (3 * kMaxExperts + 16) * 4;
    t.bars = o;
    o += 640;
    t.total = o;
    return t;
}

__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// e4m3 A and B (K-major), fp32 D, M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_e4m3(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | (8u << 24); }

__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}

__device__ __forceinline__ void umma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define MX_R16(r, o)                                                                                                \
    "=r"(r[o + 0]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), \
        "=r"(r[o + 7]), "=r"(r[o + 8]), "=r"(r[o + 9]), "=r"(r[o + 10]), "=r"(r[o + 11]), "=r"(r[o + 12]),          \
        "=r"(r[o + 13]), "=r"(r[o + 14]), "=r"(r[o + 15])

// 16 columns of this warp's 32 TMEM lanes; the wait is part of the statement, so
// nothing that reads r can be scheduled before it.
__device__ __forceinline__ void tmem_ld16(uint32_t ta, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
                 "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
                 : MX_R16(r, 0)
                 : "r"(ta)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
                 "[%32];\n\t"
                 "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
                 "%30,%31}, [%33];\n\ttcgen05.wait::ld.sync.aligned;"
                 : MX_R16(r, 0), MX_R16(r, 16)
                 : "r"(ta), "r"(tb)
                 : "memory");
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

__device__ __forceinline__ void st_cluster(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

// Bounded wait: false once this CTA has given up.
template <bool CLUSTER = false>
__device__ __forceinline__ bool bwait(uint64_t *bar, uint32_t parity, unsigned *err, volatile int *abort)
{
    auto done = [&] { return CLUSTER ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (done())
        return true;
    const unsigned long long t0 = global_ns();
    while (!done()) {
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
template <bool CLUSTER = false>
__device__ __forceinline__ bool wwait(uint64_t *bar, uint32_t parity, unsigned *err, volatile int *abort)
{
    return __all_sync(0xFFFFFFFFu, bwait<CLUSTER>(bar, parity, err, abort));
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

// A unit of work.
struct Unit {
    int e;           // matrix; -1: the shared expert (few tokens)
    int f;           // tile of 128 weight rows
    int tok0, n;     // first operand row, rows
    int item;        // kFewGateUp: hidden block among all experts'
};

// What the roles need to find units: tables in shared memory.
struct Walk {
    int n_units, first, step;  // this cluster's units
    int kb0, kb1;              // blocks of the inner dimension (items for kFewDown)
    int FT, n_act;
    const int *tt, *lo, *len;  // by tokens: token-tile offsets [E + 1], group starts and lengths [E]
    const int *act;            // few tokens: active experts
};

template <int MODE, int NT>
__device__ __forceinline__ Unit unit_of(const GemmArgs &a, const Walk &w, int u)
{
    Unit U{};
    if (MODE == kProduct || MODE == kGateUp) {
        const int tile = u / w.FT;
        U.f = u - tile * w.FT;
        int lo = 0, hi = a.E;
        while (lo + 1 < hi) {
            const int mid = (lo + hi) >> 1;
            if (w.tt[mid] <= tile)
                lo = mid;
            else
                hi = mid;
        }
        U.e = lo;
        const int tt = tile - w.tt[lo];
        U.tok0 = w.lo[lo] + NT * tt;
        U.n = min(NT, w.len[lo] - NT * tt);
    } else if (MODE == kFewGateUp) {
        U.n = a.T;
        U.item = u;
        if (u < w.n_act * a.IB) {
            const int i = u / a.IB;
            U.e = w.act[i];
            U.f = u - i * a.IB;
        } else {
            U.e = -1;
            U.f = u - w.n_act * a.IB;
        }
    } else {
        U.n = a.T;
        U.f = u;
    }
    return U;
}

// Weight tile of block kb of a unit: matrix (-1: shared), row tile, block column.
template <int MODE>
__device__ __forceinline__ void tile_of(const GemmArgs &a, const Walk &w, const Unit &U, int kb, int &e, int &c)
{
    if (MODE == kFewDown) {
        if (kb < w.n_act * a.IB) {
            const int i = kb / a.IB;
            e = w.act[i];
            c = kb - i * a.IB;
        } else {
            e = -1;
            c = kb - w.n_act * a.IB;
        }
    } else {
        e = U.e;
        c = kb;
    }
}

template <int MODE, int NT>
__global__ void __launch_bounds__((epi_warps(NT) + 3) * 32, NT <= 32 ? 2 : 1) gemm_kernel(const __grid_constant__ GemmArgs a)
{
    constexpr int NMAT = n_mats(MODE), EW = epi_warps(NT), NWG = EW / 4, NB = n_acc(MODE, NT);
    constexpr int NCH = NT / 16 / NWG, NCOL = NCH * 16;  // chunks and columns of a summing thread
    constexpr uint32_t kStage = stage_bytes(MODE, NT), kCols = NMAT * NT, kTmem = tmem_cols(MODE, NT);
    constexpr bool FEW = MODE == kFewGateUp || MODE == kFewDown;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // (the same offset in every CTA of the cluster: remote addresses rely on it)
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const int NS = a.stages, cl = a.cl;
    uint8_t *tail = ring + NS * kStage;
    const Tail T = tail_of(MODE, NT, cl, a.ncol_own);
    float *fac = reinterpret_cast<float *>(tail + T.fac);
    float *am = reinterpret_cast<float *>(tail + T.am);
    float *red = reinterpret_cast<float *>(tail + T.red);
    int *tab = reinterpret_cast<int *>(tail + T.tab);
    uint64_t *full = reinterpret_cast<uint64_t *>(tail + T.bars), *empty = full + 16;
    uint64_t *tfull = empty + 16, *tempty = tfull + 4, *ffull = tempty + 4, *fempty = ffull + kFacRing;
    uint64_t *rfull = fempty + kFacRing;  // one per lane quadrant: partial sums have come in (4), then may be
                                          // overwritten (4)
    uint32_t *tslot = reinterpret_cast<uint32_t *>(rfull + 8);
    volatile int *abort = reinterpret_cast<volatile int *>(tslot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cl > 1 ? cluster_rank() : 0;
    constexpr int kThreads = (EW + 3) * 32;

    if (a.pdl)
        pdl_trigger();
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(tfull + i, 1);
            mbar_init(tempty + i, EW);
        }
        for (int i = 0; i < kFacRing; ++i) {
            mbar_init(ffull + i, 1);
            mbar_init(fempty + i, EW);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(rfull + i, cl > 1 ? cl - 1 : 1);
            mbar_init(rfull + 4 + i, cl > 1 ? cl - 1 : 1);
        }
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == EW + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }

    // Tables of the units.
    Walk w{};
    const int KB = blocks(a.K);
    w.FT = blocks(a.N);
    if (FEW) {
        // active experts: a bit each, then their list in ascending order
        uint32_t *mask = reinterpret_cast<uint32_t *>(tab + kMaxExperts);
        int *act = tab;
        if (tid < kMaxExperts / 32)
            mask[tid] = 0;
        __syncthreads();
        for (int s = tid; s < a.T * a.topk; s += kThreads) {
            const int e = __ldg(a.idx + s);
            if (e >= 0 && e < a.E)
                atomicOr(mask + (e >> 5), 1u << (e & 31));
        }
        __syncthreads();
        int n = 0;
        for (int i = 0; i < kMaxExperts / 32; ++i)
            n += __popc(mask[i]);
        for (int e = tid; e < a.E; e += kThreads)
            if (mask[e >> 5] >> (e & 31) & 1) {
                int at = __popc(mask[e >> 5] & ((1u << (e & 31)) - 1));
                for (int i = 0; i < e >> 5; ++i)
                    at += __popc(mask[i]);
                act[at] = e;
            }
        w.n_act = n;
        w.act = act;
        w.n_units = MODE == kFewGateUp ? n * a.IB + a.SB : w.FT;
    } else {
        int *tt = tab, *lo = tab + kMaxExperts + 1, *len = lo + kMaxExperts;
        if (warp == 0) {
            int run = 0;
            for (int e0 = 0; e0 < a.E; e0 += 32) {
                const int e = e0 + lane;
                int b = 0, c = 0;
                if (e < a.E) {
                    // a group outside the rows is cut to them
                    b = a.offsets ? min(max(__ldg(a.offsets + e), 0), a.rows) : 0;
                    const int d = a.offsets ? min(max(__ldg(a.offsets + e + 1), 0), a.rows) : a.rows;
                    c = max(d - b, 0);
                }
                const int t = (c + NT - 1) / NT;
                int incl = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                    if (lane >= o)
                        incl += y;
                }
                if (e < a.E) {
                    tt[e] = run + incl - t;
                    lo[e] = b;
                    len[e] = c;
                }
                run += __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
            if (lane == 0)
                tt[a.E] = run;
        }
        w.tt = tt;
        w.lo = lo;
        w.len = len;
    }
    fence_before();
    if (cl > 1)
        cluster_sync();
    else
        __syncthreads();
    fence_after();
    if (!FEW)
        w.n_units = w.tt[a.E] * w.FT;
    w.first = blockIdx.x / cl;
    w.step = gridDim.x / cl;
    {
        const int n = MODE == kFewDown ? w.n_act * a.IB + a.SB : KB;
        w.kb0 = (int)((int64_t)n * rank / cl);
        w.kb1 = (int)((int64_t)n * (rank + 1) / cl);
    }
    const uint32_t tmem = *tslot;

    if (warp == EW) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            auto weights = [&](const Unit &U, int kb, int s) {
                uint8_t *st = ring + s * kStage;
                int e, c;
                tile_of<MODE>(a, w, U, kb, e, c);
                const bool sh = FEW && e < 0;
                tma_3d(st, sh ? &a.sa : &a.wa, c * kBlk, U.f * kBlk, sh ? 0 : e, full + s);
                if (NMAT == 2)
                    tma_3d(st + kTile, sh ? &a.sb : &a.wb, c * kBlk, U.f * kBlk, sh ? 0 : e, full + s);
            };
            auto tokens = [&](const Unit &U, int kb, int s) {
                uint8_t *st = ring + s * kStage + NMAT * kTile;
                if (MODE == kFewDown)
                    tma_2d(st, &a.xm, 0, kb * NT, full + s);
                else
                    for (int r = 0; r < U.n; r += a.xbox)
                        tma_2d(st + r * 128, &a.xm, kb * kBlk, U.tok0 + r, full + s);
            };
            auto bytes = [&](const Unit &U) -> uint32_t {
                return NMAT * kTile + (MODE == kFewDown ? NT : (U.n + a.xbox - 1) / a.xbox * a.xbox) * 128;
            };
            int early = 0;  // stages whose weights were requested before the launch's inputs were complete
            if (FEW) {
                for (int u = w.first; u < w.n_units && early < NS; u += w.step) {
                    const Unit U = unit_of<MODE, NT>(a, w, u);
                    for (int kb = w.kb0; kb < w.kb1 && early < NS; ++kb, ++early) {
                        mbar_arrive_expect_tx(full + early, bytes(U));
                        weights(U, kb, early);
                    }
                }
                pdl_wait();
            }
            int it = 0, s = 0;
            uint32_t ph = 1;
            for (int u = w.first; u < w.n_units; u += w.step) {
                const Unit U = unit_of<MODE, NT>(a, w, u);
                for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    if (it >= early) {
                        if (!bwait(empty + s, ph, a.err, abort))
                            goto produced;
                        mbar_arrive_expect_tx(full + s, bytes(U));
                        weights(U, kb, s);
                    }
                    tokens(U, kb, s);
                    if (++s == NS)
                        s = 0, ph ^= 1;
                }
            }
        }
    produced:;
    } else if (warp == EW + 1) {
        // --------------------------------------------------------------- MMA
        if (lane == 0) {
            int s = 0, b = 0;
            uint32_t ph = 0, tph = 1;
            for (int u = w.first; u < w.n_units; u += w.step) {
                const Unit U = unit_of<MODE, NT>(a, w, u);
                const uint32_t idesc = idesc_e4m3((U.n + 15) & ~15);
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!bwait(tempty + b, tph, a.err, abort) || !bwait(full + s, ph, a.err, abort))
                        goto issued;
                    fence_after();
                    const uint32_t st = smem_u32(ring + s * kStage);
                    const uint64_t xd = sw128_desc(st + NMAT * kTile);
#pragma unroll
                    for (int m = 0; m < NMAT; ++m) {
                        const uint64_t wd = sw128_desc(st + m * kTile);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_f8(tmem + b * kCols + m * NT, wd + 2 * k, xd + 2 * k, idesc, k > 0);
                    }
                    umma_commit(empty + s);
                    umma_commit(tfull + b);
                    if (++s == NS)
                        s = 0, ph ^= 1;
                    if (++b == NB)
                        b = 0, tph ^= 1;
                }
            }
        }
    issued:;
    } else if (warp == EW + 2) {
        // ----------------------------------------------------------- factors
        if (FEW)
            pdl_wait();
        constexpr int NL = (NT + 31) / 32, BATCH = NT > 64 ? 2 : 4;
        int q = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int u = w.first; u < w.n_units && ok; u += w.step) {
            const Unit U = unit_of<MODE, NT>(a, w, u);
            for (int kb0 = w.kb0; kb0 < w.kb1 && ok; kb0 += BATCH) {
                float x[BATCH][NL], s0[BATCH], s1[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int kb = kb0 + i;
                    s0[i] = s1[i] = 0.0f;
#pragma unroll
                    for (int j = 0; j < NL; ++j)
                        x[i][j] = 0.0f;
                    if (kb < w.kb1) {
                        int e, c;
                        tile_of<MODE>(a, w, U, kb, e, c);
                        if (FEW && e < 0) {
                            const int64_t at = (int64_t)U.f * (MODE == kFewDown ? a.SB : KB) + c;
                            s0[i] = __ldg(a.ssa + at);
                            if (NMAT == 2)
                                s1[i] = __ldg(a.ssb + at);
                        } else {
                            const int64_t at = ((int64_t)e * w.FT + U.f) * (MODE == kFewDown ? a.IB : KB) + c;
                            s0[i] = __ldg(a.swa + at);
                            if (NMAT == 2)
                                s1[i] = __ldg(a.swb + at);
                        }
#pragma unroll
                        for (int j = 0; j < NL; ++j) {
                            const int n = lane + 32 * j;
                            if (n < U.n)  // (written by the launch before: not through the read-only path)
                                x[i][j] = MODE == kFewDown ? a.hs[(int64_t)kb * NT + n]
                                                           : a.sx[(U.tok0 + n) * a.sx_r + kb * a.sx_b];
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    if (kb0 + i >= w.kb1 || !ok)
                        break;
                    ok = wwait(fempty + q, ph, a.err, abort);
                    float *o = fac + q * NMAT * NT;
#pragma unroll
                    for (int j = 0; j < NL; ++j) {
                        const int n = lane + 32 * j;
                        if (n < NT) {
                            o[n] = x[i][j] * s0[i];
                            if (NMAT == 2)
                                o[NT + n] = x[i][j] * s1[i];
                        }
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(ffull + q);
                    if (++q == kFacRing)
                        q = 0, ph ^= 1;
                }
            }
        }
    } else {
        // -------------------------------------------------------------- sums
        const int wg = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t ta = tmem + ((uint32_t)quad << 21);
        int b = 0, q = 0, parity = 0;
        uint32_t tph = 0, fph = 0, rph = 0;
        bool ok = true;
        for (int u = w.first; u < w.n_units && ok; u += w.step, parity ^= 1) {
            const Unit U = unit_of<MODE, NT>(a, w, u);
            uint64_t acc[NMAT][NCOL / 2];
#pragma unroll
            for (int m = 0; m < NMAT; ++m)
#pragma unroll
                for (int i = 0; i < NCOL / 2; ++i)
                    acc[m][i] = 0;
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                if (!wwait(ffull + q, fph, a.err, abort) || !wwait(tfull + b, tph, a.err, abort)) {
                    ok = false;
                    break;
                }
                fence_after();
                const float *f = fac + q * NMAT * NT;
                const uint32_t tb = ta + b * kCols;
#pragma unroll
                for (int m = 0; m < NMAT; ++m) {
                    auto fma16 = [&](int ch, const uint32_t *r) {
                        const float4 *fv = reinterpret_cast<const float4 *>(f + m * NT + (ch * NWG + wg) * 16);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 v = fv[i];
                            fma_f32x2(acc[m][ch * 8 + 2 * i],
                                      pair_f32(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])),
                                      pair_f32(v.x, v.y));
                            fma_f32x2(acc[m][ch * 8 + 2 * i + 1],
                                      pair_f32(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])),
                                      pair_f32(v.z, v.w));
                        }
                    };
                    if (NCH >= 2) {
#pragma unroll
                        for (int ch = 0; ch + 1 < NCH; ch += 2) {
                            if ((ch * NWG + wg) * 16 >= U.n)
                                break;
                            uint32_t r[32];
                            tmem_ld16x2(tb + m * NT + (ch * NWG + wg) * 16, tb + m * NT + ((ch + 1) * NWG + wg) * 16, r);
                            fma16(ch, r);
                            fma16(ch + 1, r + 16);
                        }
                    } else {
                        uint32_t r[16];
                        tmem_ld16(tb + m * NT + wg * 16, r);
                        fma16(0, r);
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(tempty + b);
                    mbar_arrive(fempty + q);
                }
                if (++b == NB)
                    b = 0, tph ^= 1;
                if (++q == kFacRing)
                    q = 0, fph ^= 1;
            }
            float v[NMAT][NCOL];
#pragma unroll
            for (int m = 0; m < NMAT; ++m)
#pragma unroll
                for (int i = 0; i < NCOL / 2; ++i)
                    unpair_f32(acc[m][i], v[m][2 * i], v[m][2 * i + 1]);
            // token column of this thread's i-th sum
            auto col = [&](int i) { return ((i >> 4) * NWG + wg) * 16 + (i & 15); };

            if (NWG == 1 && cl > 1) {
                // The cluster's partial sums: column n belongs to CTA n % cl.
                const int sh = 31 - __clz(cl), own = a.ncol_own;
                if (u != w.first)
                    ok = ok && wwait<true>(rfull + 4 + quad, rph ^ 1, a.err, abort);
#pragma unroll
                for (int i = 0; i < NCOL; ++i)
                    if (i < U.n && (i & (cl - 1)) != (int)rank) {
#pragma unroll
                        for (int m = 0; m < NMAT; ++m)
                            st_cluster(mapa(smem_u32(red + ((rank * own + (i >> sh)) * NMAT + m) * 128 + row),
                                            i & (cl - 1)),
                                       v[m][i]);
                    }
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                __syncwarp();
                if (lane < cl && lane != (int)rank)
                    arrive_cluster(mapa(smem_u32(rfull + quad), lane));
                ok = ok && wwait<true>(rfull + quad, rph, a.err, abort);
#pragma unroll
                for (int i = 0; i < NCOL; ++i)
                    if (i < U.n && (i & (cl - 1)) == (int)rank) {
#pragma unroll
                        for (int m = 0; m < NMAT; ++m) {
                            float sum = 0.0f;
                            for (int r = 0; r < cl; ++r)
                                sum += r == (int)rank ? v[m][i] : red[((r * own + (i >> sh)) * NMAT + m) * 128 + row];
                            v[m][i] = sum;
                        }
                    }
                __syncwarp();
                if (lane < cl && lane != (int)rank)
                    arrive_cluster(mapa(smem_u32(rfull + 4 + quad), lane));
                rph ^= 1;
            }
            // (n % 1 == 0: without a cluster every column is this CTA's)
            auto mine = [&](int n) { return n < U.n && (n & (cl - 1)) == (int)rank; };

            if constexpr (NMAT == 2) {
                // h = act(g) u, then e4m3 by the largest |h| of the tile's 128 hidden columns
                float *am4 = am + (parity * NWG + wg) * 4 * NCOL, *rcp = am + 2 * 4 * NT + warp * NCOL;
                uint32_t keep = 0;
#pragma unroll
                for (int i = 0; i < NCOL; ++i) {
                    const float h = act_of(v[0][i], a.act) * v[1][i];
                    v[0][i] = h;
                    uint32_t m = 0;
                    if (mine(col(i)))  // (the whole warp agrees)
                        m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h) & 0x7FFFFFFFu);
                    if ((i & 31) == lane)
                        keep = m;
                    if ((i & 31) == 31 || i == NCOL - 1) {
                        const int at = (i & ~31) + lane;
                        if (at < NCOL)
                            am4[quad * NCOL + at] = __uint_as_float(keep);
                    }
                }
                // (the four warps of a warpgroup give up together: none is left at the barrier)
                __syncwarp();
                ok = named_and(1 + wg, 128, ok);
                if (!ok)
                    break;
#pragma unroll
                for (int j = 0; j < (NCOL + 31) / 32; ++j) {
                    const int i = lane + 32 * j;
                    if (i < NCOL) {
                        const int n = col(i);
                        uint32_t m = 0;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            m = max(m, __float_as_uint(am4[r * NCOL + i]));
                        const float s = scale_of(__uint_as_float(m), 0);
                        // (h by a reciprocal: it is a rounded sum, on no border between two e4m3 numbers)
                        float inv = __frcp_rn(s), sc = s;
                        if (MODE == kFewGateUp && U.e >= 0 && n < a.T) {
                            // the routing weight joins the scale; a token that did not choose the expert adds nothing
                            float wt = 0.0f;
                            bool routed = false;
                            for (int k = 0; k < a.topk; ++k)
                                if (__ldg(a.idx + n * a.topk + k) == U.e) {
                                    wt += __ldg(a.wts + n * a.topk + k);
                                    routed = true;
                                }
                            sc = routed ? s * wt : 0.0f;
                            inv = routed ? inv : 0.0f;
                        }
                        rcp[i] = inv;
                        if (quad == 0 && mine(n))
                            a.hs[MODE == kFewGateUp ? (int64_t)U.item * NT + n : (int64_t)U.f * a.hs_ld + U.tok0 + n] = sc;
                    }
                }
                __syncwarp();
                uint8_t *h = a.h + (MODE == kFewGateUp ? (int64_t)U.item * NT * 128
                                                       : (int64_t)U.tok0 * a.ldh + U.f * kBlk) + row;
                const int64_t ld = MODE == kFewGateUp ? 128 : a.ldh;
#pragma unroll
                for (int i = 0; i < NCOL; i += 2) {
                    const float r0 = rcp[i], r1 = rcp[i + 1];
                    const uint32_t e = e4m3_x2(r0 != 0.0f ? v[0][i] * r0 : 0.0f, r1 != 0.0f ? v[0][i + 1] * r1 : 0.0f);
                    if (mine(col(i)))
                        h[col(i) * ld] = (uint8_t)e;
                    if (mine(col(i + 1)))
                        h[col(i + 1) * ld] = (uint8_t)(e >> 8);
                }
            } else {
                if (!ok)
                    break;
                const int o = U.f * kBlk + row;
                if (o < a.N) {
#pragma unroll
                    for (int i = 0; i < NCOL; ++i) {
                        const int n = col(i);
                        if (!mine(n))
                            continue;
                        const int64_t at = (int64_t)(U.tok0 + n) * a.ldo + o;
                        float y = v[0][i];
                        if (MODE == kFewDown)
                            y = fmaf(a.lam, y, a.residual ? load_act(a.residual, at, a.out_bf16) : 0.0f);
                        if (a.out_bf16)
                            reinterpret_cast<uint16_t *>(a.out)[at] = f2bf(y);
                        else
                            reinterpret_cast<float *>(a.out)[at] = y;
                    }
                }
            }
        }
    }

    fence_before();
    if (*abort) {
        // let this CTA's copies and MMAs in flight land before its memory goes to another
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 200000ull)
            __nanosleep(1000);
    }
    __syncthreads();
    if (cl > 1)
        cluster_sync();
    fence_after();
    __syncwarp();
    if (warp == EW + 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
}

template <int MODE, int NT>
cudaError_t launch_t(const GemmArgs &a, int grid, cudaStream_t s)
{
    const size_t smem = gemm_smem((Mode)MODE, NT, a.stages, a.cl, a.ncol_own);
    cudaError_t e = smem_optin((const void *)gemm_kernel<MODE, NT>, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3((epi_warps(NT) + 3) * 32);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[2];
    unsigned n = 0;
    if (a.cl > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim = {(unsigned)a.cl, 1, 1};
        ++n;
    }
    if (MODE == kFewGateUp || MODE == kFewDown) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    c.attrs = at;
    c.numAttrs = n;
    return cudaLaunchKernelEx(&c, gemm_kernel<MODE, NT>, a);
}

}  // namespace

size_t gemm_smem(Mode mode, int nt, int stages, int cl, int ncol_own)
{
    return 1024 + (size_t)stages * stage_bytes(mode, nt) + tail_of(mode, nt, cl, ncol_own).total;
}

cudaError_t launch_gemm(Mode mode, int nt, const GemmArgs &a, int grid, cudaStream_t s)
{
#define MX_CASE(M, N)            \
    if (mode == M && nt == N)    \
        return launch_t<M, N>(a, grid, s)
    MX_CASE(kProduct, 16);
    MX_CASE(kProduct, 32);
    MX_CASE(kProduct, 64);
    MX_CASE(kProduct, 128);
    MX_CASE(kProduct, 256);
    MX_CASE(kGateUp, 16);
    MX_CASE(kGateUp, 32);
    MX_CASE(kGateUp, 64);
    MX_CASE(kGateUp, 128);
    MX_CASE(kFewGateUp, 16);
    MX_CASE(kFewGateUp, 32);
    MX_CASE(kFewGateUp, 64);
    MX_CASE(kFewDown, 16);
    MX_CASE(kFewDown, 32);
    MX_CASE(kFewDown, 64);
#undef MX_CASE
    return cudaErrorInvalidValue;
}

}  // namespace fp8
}  // namespace mx
