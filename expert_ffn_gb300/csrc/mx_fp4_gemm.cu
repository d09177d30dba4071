// mx_fp4_gemm.cu -- products of microscaled e2m1 rows and matrices on the 5th-generation
// tensor cores (tcgen05.mma kind::mxf4nvf4, block scales and accumulators in TMEM).
//
//   y[r, o] = tx tw sum_b sx[r, b] sw[o, b] sum_{c in b} qx[r, c] qw[o, c]
//
// The tensor core takes the block scales itself (scale_vec::4X for blocks of 16 e4m3,
// 2X for blocks of 32 e8m0) and keeps a tile's whole sum in TMEM, so nothing is left to the
// CUDA cores but the tensors' factors.  The weights take the M side (128 rows), the tokens
// the N side (any multiple of 16 up to the tile's width), so one kernel serves one row and
// thousands: a short group costs what its rows need.
//
// A stage of the ring is 256 columns: 128 bytes of each row (SWIZZLE_128B) and their
// scales, 16 or 8 bytes a row.  The tensor core wants the scales of 128 rows and four blocks as 32
// lines of 16 bytes, line i with those of the rows i, 32 + i, 64 + i, 96 + i.  The weights' are laid out
// so once (mx_fp4_pack_scales) and come by one bulk copy.  A token tile may begin at any row, so a
// lane loads the 16 bytes of four rows 32 apart (neighbouring lanes neighbouring rows: the
// quantiser keeps a stage's scales of all rows together) and stores four lines, a transposition
// that costs no instruction.  (Both gathered from rows in memory by 4-byte asynchronous copies
// bounded the kernel: 4096^3 82 us, without them 52.)
//
// Warps:
//   0-7  results: TMEM (lane quadrant = warp % 4, every other 16 tokens) to global memory, bf16 ones by
//        way of shared memory in pieces of 16 bytes
//   8    TMA producer: weight and token tiles
//   9    MMA: per stage the copies of its scales to TMEM (tcgen05.cp, in order with the
//        MMAs) and four MMAs (K = 64)
//   10-11  the tokens' scales, every other stage each
// Two TMEM accumulators: a tile's results leave while the next one is summed.  Few units of many stages: a
// cluster of `cl` CTAs splits the inner dimension of one unit, and its partial sums are added
// through distributed shared memory in rank order.
//
// What bounds it: 4096 x 4096 x 4096 takes 30 us, of which another 4096 columns of K add 18 (7.6
// PFLOP/s: the slope of this form, K = 64 by one CTA; the chip's FP4 rate is higher); the rest is launch, the first fill, the
// last tile's results, and results that reach memory.  32768 rows of 256 matrices 1024 x 4096 are bound by HBM, 119 us
// (0.85 of the copy rate); 64 x 4096 x 4096 by its chain on 32 SMs, 6.6 us (blocks of 32: 6.3): launch, fill,
// the MMAs of sixteen stages.  So are a few rows of grouped matrices, which no cluster splits: 8 rows of 8 matrices 704 x 2816 6.6 us.
//
// Every wait is bounded: a wait that gives up sets the caller's error word and ends the
// CTA's work.
#include "mx_fp4.cuh"
#include "mx_fp8_tc.cuh"

#include <type_traits>

namespace mx {
namespace fp4 {

namespace {

using fp8::bwait;
using fp8::cluster_rank;
using fp8::cluster_sync;
using fp8::elect_one;
using fp8::fence_after;
using fp8::fence_before;
using fp8::group_table;
using fp8::ld_cluster;
using fp8::mapa;
using fp8::sw128_desc;
using fp8::tma_2d;
using fp8::tma_3d;
using fp8::tmem_ld16;
using fp8::tmem_value;
using fp8::tmem_wait;
using fp8::warp_index;
using fp8::wwait;

constexpr uint32_t kTile = 128 * 128;  // bytes of one weight tile
constexpr int kOutWarps = 8, kScaleWarps = 2, kThreads = (kOutWarps + 2 + kScaleWarps) * 32;
constexpr int kAcc = 2;                // TMEM accumulators
constexpr int kMaxStages = 12;

constexpr int halves(int nt) { return (nt + 127) / 128; }
constexpr uint32_t scale_bytes(int block, int nt) { return atoms_of(block) * 512 * (1 + halves(nt)); }
constexpr uint32_t stage_bytes(int block, int nt) { return kTile + nt * 128 + scale_bytes(block, nt); }
constexpr int acc_cols(int nt) { return nt; }
constexpr uint32_t tmem_cols(int block, int nt)
{
    const uint32_t need = kAcc * acc_cols(nt) + atoms_of(block) * 4 * (1 + halves(nt));
    uint32_t c = 32;
    while (c < need)
        c *= 2;
    return c;
}

// Dynamic shared memory after the ring.
struct Tail {
    int out, tab, bars, total;
};
__host__ __device__ constexpr Tail tail_of()
{
    Tail t{};
    int o = 0;
    t.out = o;  // a warp's results on their way out: 16 tokens x 32 bf16
    o += kOutWarps * 1024;
    t.tab = o;
    o += (3 * kMaxExperts + 16) * 4;
    t.bars = o;
    o += 512;
    t.total = o;
    return t;
}

// e2m1 A and B (K-major), fp32 D, M = 128, N = n; scale type e8m0 (bit 23) or e4m3.
__device__ __forceinline__ uint32_t idesc_e2m1(int n, int block)
{
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (block == 32 ? 1u << 23 : 0u) | (8u << 24);
}

// 32 lines of 16 bytes without a swizzle (8 lines to a core matrix, 128 bytes apart).
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// N scale pieces to TMEM, four columns each.  One elected lane of a converged warp.
template <int N>
__device__ __forceinline__ void scales_to_tmem(uint32_t to, uint64_t desc)
{
    static_assert(N == 2 || N == 4 || N == 8, "pieces");
#define MX_CP "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [t], d;\n\tadd.u32 t, t, 4;\n\tadd.s64 d, d, 32;\n\t"
#define MX_CP_HEAD "{\n\t.reg .pred q;\n\t.reg .b32 t;\n\t.reg .b64 d;\n\tmov.b32 t, %0;\n\tmov.b64 d, %1;\n\telect.sync _|q, 0xffffffff;\n\t"
    if constexpr (N == 2)
        asm volatile(MX_CP_HEAD MX_CP MX_CP "}" ::"r"(to), "l"(desc) : "memory");
    else if constexpr (N == 4)
        asm volatile(MX_CP_HEAD MX_CP MX_CP MX_CP MX_CP "}" ::"r"(to), "l"(desc) : "memory");
    else
        asm volatile(MX_CP_HEAD MX_CP MX_CP MX_CP MX_CP MX_CP MX_CP MX_CP MX_CP "}" ::"r"(to), "l"(desc) : "memory");
#undef MX_CP
#undef MX_CP_HEAD
}

// Four MMAs of K = 64, the first of which overwrites D unless `more`.  xs: TMEM columns of a
// token piece.  (In one statement with the election inside: behind a branch on it the compiler
// issues each in a loop over lanes.)
template <int BLOCK>
__device__ __forceinline__ void umma_stage(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                           uint32_t xs, bool more)
{
    const uint32_t i2 = idesc | (BLOCK == 32 ? (2u << 29) | (2u << 4) : 0u);  // (second half of a piece)
    // scale addresses of the four: a piece for each (blocks of 16) or for two (blocks of 32)
    const uint32_t s1 = BLOCK == 32 ? 0 : 1, s2 = BLOCK == 32 ? 1 : 2, s3 = BLOCK == 32 ? 1 : 3;
#define MX_MMA(vec)                                                                                                    \
    asm volatile(                                                                                                      \
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"                                               \
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"                                           \
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"                                           \
        "elect.sync _|q, 0xffffffff;\n\tsetp.ne.u32 p, %13, 0;\n\t"                                                    \
        "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::" vec " [%0], %1, %2, %3, [%5], [%9], p;\n\t"  \
        "setp.ne.u32 p, %3, 0;\n\t"                                                                                    \
        "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::" vec " [%0], a1, b1, %4, [%6], [%10], p;\n\t" \
        "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::" vec " [%0], a2, b2, %3, [%7], [%11], p;\n\t" \
        "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::" vec " [%0], a3, b3, %4, [%8], [%12], p;\n\t" \
        "}" ::"r"(d),                                                                                                  \
        "l"(a), "l"(b), "r"(idesc), "r"(i2), "r"(sfa), "r"(sfa + 4 * s1), "r"(sfa + 4 * s2), "r"(sfa + 4 * s3),        \
        "r"(sfb), "r"(sfb + xs * s1), "r"(sfb + xs * s2), "r"(sfb + xs * s3), "r"((uint32_t)more)                      \
        : "memory")
    if constexpr (BLOCK == 32)
        MX_MMA("2X");
    else
        MX_MMA("4X");
#undef MX_MMA
}

__device__ __forceinline__ void umma_commit(uint64_t *x)
{
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(x))
                 : "memory");
}

// Request 16 lanes of 16 columns as the accumulator fragments of an m16n8 product: r[4 k ..] of columns 8 k on, lane l has
// row l / 4, columns 2 (l % 4) and the next, then the same of row l / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t ta, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(ta)
                 : "memory");
}

// Four 8 x 8 matrices of such fragments, each transposed: lane 8 m + i has the address of matrix m's column i.
__device__ __forceinline__ void store_transposed(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Two results times their factors as bf16.
__device__ __forceinline__ uint32_t scaled_bf16(uint32_t lo, uint32_t hi, float f, float g)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(tmem_value(hi) * f * g), "f"(tmem_value(lo) * f * g));
    return r;
}

__device__ __forceinline__ float ld_cluster1(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

struct Unit {
    int e, f;      // matrix, tile of 128 weight rows
    int tok0, n;   // first token row, rows
};

struct Walk {
    int n_units, first, step;
    int kb0, kb1;  // this rank's stages of the inner dimension
    int FT;
    const int *tt, *lo, *len;
};

template <int NT>
__device__ __forceinline__ Unit unit_of(const GemmArgs &a, const Walk &w, int u)
{
    Unit U;
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
    const int t = tile - w.tt[lo];
    U.tok0 = w.lo[lo] + NT * t;
    U.n = min(NT, w.len[lo] - NT * t);
    return U;
}

template <int NT, int BLOCK>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs a)
{
    constexpr int NA = atoms_of(BLOCK), NH = halves(NT);  // scale pieces of 128 rows, of a stage; token halves
    constexpr uint32_t kStage = stage_bytes(BLOCK, NT), kTmem = tmem_cols(BLOCK, NT);
    constexpr int BOX = box_rows(NT);
    constexpr Tail T = tail_of();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // (the same offset in every CTA of the cluster: remote addresses rely on it)
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const int NS = a.stages, cl = a.cl;
    uint8_t *tail = ring + NS * kStage;
    int *tab = reinterpret_cast<int *>(tail + T.tab);
    uint64_t *full = reinterpret_cast<uint64_t *>(tail + T.bars), *empty = full + kMaxStages;
    uint64_t *tfull = empty + kMaxStages, *tempty = tfull + kAcc;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(tempty + kAcc);
    volatile int *abort = reinterpret_cast<volatile int *>(tslot + 1);
    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const uint32_t rank = cl > 1 ? cluster_rank() : 0;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, 2);  // copies, tokens' scales
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < kAcc; ++i) {
            mbar_init(tfull + i, 1);
            mbar_init(tempty + i, kOutWarps);
        }
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == kOutWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == kOutWarps && lane < 2)  // (the descriptors are the launch's own)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &a.xm : &a.wm) : "memory");
    pdl_wait();  // (nothing before this reads what an earlier launch may still write)
    Walk w{};
    {
        int *tt = tab, *lo = tab + kMaxExperts + 1, *len = lo + kMaxExperts;
        if (warp == 0)
            group_table(a.offsets, a.E, a.rows, NT, lane, tt, lo, len);
        w.tt = tt;
        w.lo = lo;
        w.len = len;
    }
    fence_before();
    __syncthreads();  // (the CTAs of a cluster meet when each has its partial sums)
    fence_after();
    const int KB = stages_of(a.K);
    w.FT = (a.N + 127) / 128;
    w.n_units = w.tt[a.E] * w.FT;
    w.first = blockIdx.x / cl;
    w.step = gridDim.x / cl;
    w.kb0 = KB * rank / cl;
    w.kb1 = KB * (rank + 1) / cl;
    const uint32_t tmem = *tslot, tsw = tmem + kAcc * acc_cols(NT), tsx = tsw + 4 * NA;

    if (warp == kOutWarps) {
        // ------------------------------------------------------ TMA producer
        int s = 0;
        uint32_t ph = 1;
        for (int u = w.first; u < w.n_units; u += w.step) {
            const Unit U = unit_of<NT>(a, w, u);
            const int boxes = (U.n + BOX - 1) / BOX;
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                if (!wwait(empty + s, ph, a.err, abort))
                    goto produced;
                uint8_t *st = ring + s * kStage;
                if (elect_one()) {
                    mbar_arrive_expect_tx(full + s, kTile + boxes * BOX * 128 + NA * 512);
                    tma_3d(st, &a.wm, kb * 128, U.f * 128, U.e, full + s);
                    bulk_g2s(st + kTile + NT * 128, a.sw + (((int64_t)U.e * w.FT + U.f) * KB + kb) * (NA * 512), NA * 512,
                             full + s);
                    for (int b = 0; b < boxes; ++b)
                        tma_2d(st + kTile + b * BOX * 128, &a.xm, kb * 128, U.tok0 + b * BOX, full + s);
                }
                __syncwarp();
                if (++s == NS)
                    s = 0, ph ^= 1;
            }
        }
    produced:;
    } else if (warp == kOutWarps + 1) {
        // --------------------------------------------------------------- MMA
        int s = 0, b = 0;
        uint32_t ph = 0, tph = 1;
        for (int u = w.first; u < w.n_units; u += w.step) {
            const Unit U = unit_of<NT>(a, w, u);
            const uint32_t idesc = idesc_e2m1((U.n + 15) & ~15, BLOCK);
            if (!wwait(tempty + b, tph, a.err, abort))
                goto issued;
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                if (!wwait(full + s, ph, a.err, abort))
                    goto issued;
                fence_after();
                const uint32_t st = smem_u32(ring + s * kStage), sc = st + kTile + NT * 128;
                scales_to_tmem<NA>(tsw, scale_desc(sc));
                scales_to_tmem<NA * NH>(tsx, scale_desc(sc + NA * 512));
                umma_stage<BLOCK>(tmem + b * acc_cols(NT), sw128_desc(st), sw128_desc(st + kTile), idesc, tsw, tsx, 4 * NH,
                                  kb != w.kb0);
                umma_commit(empty + s);
                if (++s == NS)
                    s = 0, ph ^= 1;
            }
            umma_commit(tfull + b);
            if (++b == kAcc)
                b = 0, tph ^= 1;
        }
    issued:;
    } else if (warp > kOutWarps + 1) {
        // ------------------------------------------------------------ scales
        constexpr int AHEAD = NH == 1 ? 4 : 2;  // stages of this warp under way in registers
        using Row = typename std::conditional<BLOCK == 16, uint4, uint2>::type;  // a row's scales of a stage
        const int me = warp - kOutWarps - 2;
        Row v[AHEAD][4 * NH];
        int fu = w.first, fkb = w.kb0 + me;  // what is fetched next
        Unit U{};
        if (fu < w.n_units)
            U = unit_of<NT>(a, w, fu);
        auto fetch = [&](Row (&d)[4 * NH]) {
            while (fu < w.n_units && fkb >= w.kb1) {  // (a unit's stages run on into the next one's)
                fkb -= w.kb1 - w.kb0;
                fu += w.step;
                if (fu < w.n_units)
                    U = unit_of<NT>(a, w, fu);
            }
            if (fu >= w.n_units)
                return;
            // (plain loads: the read-only path must not be used by a launch that began before its
            // predecessor's end)
            const Row *p = reinterpret_cast<const Row *>(a.sx) + (int64_t)fkb * a.rows;
#pragma unroll
            for (int i = 0; i < 4 * NH; ++i)
                if (32 * i < NT && 32 * i < U.n)  // (a row behind the last: its own column alone, or none)
                    d[i] = p[min(U.tok0 + 32 * i + lane, a.rows - 1)];
            fkb += kScaleWarps;
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
#pragma unroll
            for (int j = 0; j < 4 * NH; ++j)
                v[i][j] = Row{};
            fetch(v[i]);
        }
        const int units = w.first < w.n_units ? (w.n_units - w.first + w.step - 1) / w.step : 0;
        const int64_t total = (int64_t)(w.kb1 - w.kb0) * units;
        int s = me % NS;
        uint32_t ph = 1;
        bool ok = true;
        for (int64_t it = me; it < total && ok;) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (it >= total)
                    break;
                ok = wwait(empty + s, ph, a.err, abort);
                if (!ok)
                    break;
                uint4 *to = reinterpret_cast<uint4 *>(ring + s * kStage + kTile + NT * 128 + NA * 512) + lane;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    uint32_t r[4][NA];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Row x = v[i][4 * h + j];
                        r[j][0] = x.x, r[j][1] = x.y;
                        if constexpr (NA == 4)
                            r[j][2] = x.z, r[j][3] = x.w;
                    }
#pragma unroll
                    for (int k = 0; k < NA; ++k)
                        to[(k * NH + h) * 32] = make_uint4(r[0][k], r[1][k], r[2][k], r[3][k]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the tensor core's copies read them)
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(full + s);
                fetch(v[i]);
                it += kScaleWarps;
                s += kScaleWarps;
                if (s >= NS)
                    s -= NS, ph ^= 1;
            }
        }
    } else {
        // ----------------------------------------------------------- results
        const int quad = warp & 3;
        const uint32_t ta = tmem + ((uint32_t)quad << 21);
        const float tx = a.tx ? *a.tx : 1.0f;
        uint8_t *mine = tail + T.out + warp * 1024;
        const int es = a.out_bf16 ? 2 : 4;
        const int64_t pitch = a.ldo * es;
        int b = 0;
        uint32_t tph = 0;
        for (int u = w.first; u < w.n_units; u += w.step) {
            const Unit U = unit_of<NT>(a, w, u);
            const float tw = a.tw ? a.tw[U.e] : 1.0f;
            if (!wwait(tfull + b, tph, a.err, abort))
                break;
            fence_after();
            const uint32_t tb = ta + b * acc_cols(NT);
            const int row = quad * 32 + lane, o0 = U.f * 128 + quad * 32, o = o0 + lane;
            float *part = reinterpret_cast<float *>(ring);
            const bool whole = cl == 1 && a.out_bf16 && a.out_vec && o0 + 32 <= a.N;
            const Factors f = factors_of(tx, tw);
            const float f1 = f.a, f2 = f.b;
#pragma unroll 1
            for (int c0 = (warp >> 2) * 16; c0 < U.n; c0 += 32) {
                const int n = U.n - c0;  // tokens of these columns
                char *to = static_cast<char *>(a.out) + (int64_t)(U.tok0 + c0) * pitch + (int64_t)o0 * es;
                if (whole) {
                    // A token's 32 rows are to be neighbours, and are lanes of TMEM: fragments of 8 rows x 8 tokens go to
                    // shared memory transposed, four of them an instruction.  (Row by row in 2-byte stores
                    // 4096 x 4096 x 704 took 13.9 us instead of 13.0; whole lines by way of four warps' buffer 13.3.)  A token's four pieces of 16 bytes are rotated against bank conflicts.
                    uint32_t r[2][8];
                    tmem_ld_frag(tb + c0, r[0]);
                    tmem_ld_frag(tb + c0 + (16u << 16), r[1]);
                    tmem_wait();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int token = 8 * k + (lane & 7), piece = (lane >> 3) ^ ((token >> 1) & 3);
                        store_transposed(smem_u32(mine) + token * 64 + piece * 16,
                                         scaled_bf16(r[0][4 * k], r[0][4 * k + 1], f1, f2),
                                         scaled_bf16(r[0][4 * k + 2], r[0][4 * k + 3], f1, f2),
                                         scaled_bf16(r[1][4 * k], r[1][4 * k + 1], f1, f2),
                                         scaled_bf16(r[1][4 * k + 2], r[1][4 * k + 3], f1, f2));
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int token = i * 8 + (lane >> 2), piece = (lane & 3) ^ ((token >> 1) & 3);
                        const uint4 v = reinterpret_cast<const uint4 *>(mine)[token * 4 + piece];
                        if (token < n)
                            *reinterpret_cast<uint4 *>(to + token * pitch + (lane & 3) * 16) = v;
                    }
                    __syncwarp();
                    continue;
                }
                uint32_t r[16];
                tmem_ld16(tb + c0, r);
                tmem_wait();
                float y[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    y[j] = tmem_value(r[j]) * f1 * f2;
                if (cl > 1) {  // one unit; every operand has been read
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        part[(c0 + j) * 128 + row] = y[j];
                } else if (o < a.N) {
                    to += lane * es;
#pragma unroll
                    for (int j = 0; j < 16; ++j, to += pitch)
                        if (j < n) {
                            if (a.out_bf16)
                                *reinterpret_cast<uint16_t *>(to) = f2bf(y[j]);
                            else
                                *reinterpret_cast<float *>(to) = y[j];
                        }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(tempty + b);
            if (++b == kAcc)
                b = 0, tph ^= 1;
        }
    }

    if (cl > 1) {
        __syncwarp();
        cluster_sync();
        if (warp < kOutWarps && w.first < w.n_units && !*abort) {
            const Unit U = unit_of<NT>(a, w, w.first);
            // column n of the tile: CTA n % cl of the cluster, over all ranks in order
            for (int n = rank + cl * warp; n < U.n; n += cl * kOutWarps) {
                const uint32_t col = smem_u32(reinterpret_cast<float *>(ring) + n * 128);
                const int64_t to = (int64_t)(U.tok0 + n) * a.ldo + U.f * 128;
                if (a.out_vec) {  // four neighbouring rows to a lane
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                    for (int r = 0; r < cl; ++r) {
                        const float4 p = ld_cluster(mapa(col + 16 * lane, r));
                        v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
                    }
                    const float y[4] = {v.x, v.y, v.z, v.w};
                    const int64_t at = to + 4 * lane;
                    const int left = a.N - U.f * 128 - 4 * lane;
                    if (left >= 4 && a.out_bf16)
                        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
                            make_uint2(f2bf(y[0]) | (uint32_t)f2bf(y[1]) << 16, f2bf(y[2]) | (uint32_t)f2bf(y[3]) << 16);
                    else if (left >= 4)
                        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = v;
                    else
#pragma unroll
                        for (int i = 0; i < 3; ++i)
                            if (i < left) {
                                if (a.out_bf16)
                                    static_cast<uint16_t *>(a.out)[at + i] = f2bf(y[i]);
                                else
                                    static_cast<float *>(a.out)[at + i] = y[i];
                            }
                } else {  // neighbouring rows to neighbouring lanes
                    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
                    for (int r = 0; r < cl; ++r) {
                        const uint32_t at = mapa(col + 4 * lane, r);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            y[i] += ld_cluster1(at + 128 * i);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 32 * i + lane;
                        if (U.f * 128 + row < a.N) {
                            if (a.out_bf16)
                                static_cast<uint16_t *>(a.out)[to + row] = f2bf(y[i]);
                            else
                                static_cast<float *>(a.out)[to + row] = y[i];
                        }
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
    if (warp == kOutWarps + 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
}

// One 16-byte line of a piece to a thread.
__global__ void __launch_bounds__(256) pack_kernel(const PackArgs a)
{
    const int NA = atoms_of(a.block), stages = (a.nb + 4 * NA - 1) / (4 * NA), FT = (a.rows + 127) / 128;
    const int64_t lines = (int64_t)a.count * FT * stages * NA * 32;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < lines; i += (int64_t)gridDim.x * blockDim.x) {
        const int line = (int)(i % 32);
        int64_t x = i / 32;
        const int b0 = (int)(x % ((int64_t)stages * NA)) * 4;  // first of four blocks
        x /= (int64_t)stages * NA;
        const int f = (int)(x % FT), e = (int)(x / FT);
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = f * 128 + 32 * j + line;
            v[j] = 0;
            for (int k = 0; k < 4; ++k)
                if (row < a.rows && b0 + k < a.nb)
                    v[j] |= (uint32_t)__ldg(a.scales + ((int64_t)e * a.rows + row) * a.ld + b0 + k) << (8 * k);
        }
        reinterpret_cast<uint4 *>(a.out)[i] = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

template <int NT, int BLOCK>
cudaError_t launch_t(const GemmArgs &a, int grid, cudaStream_t s)
{
    const size_t smem = gemm_smem(BLOCK, NT, a.stages);
    cudaError_t e = smem_optin((const void *)gemm_kernel<NT, BLOCK>, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[2];
    unsigned n = 0;
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
    if (a.cl > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim = {(unsigned)a.cl, 1, 1};
        ++n;
    }
    c.attrs = at;
    c.numAttrs = n;
    return cudaLaunchKernelEx(&c, gemm_kernel<NT, BLOCK>, a);
}

}  // namespace

cudaError_t launch_pack(const PackArgs &a, cudaStream_t s)
{
    pack_kernel<<<1024, 256, 0, s>>>(a);
    return cudaGetLastError();
}

size_t gemm_smem(int block, int nt, int stages)
{
    return 1024 + (size_t)stages * stage_bytes(block, nt) + tail_of().total;
}

cudaError_t launch_gemm(int block, int nt, const GemmArgs &a, int grid, cudaStream_t s)
{
    static_assert(kMaxStages * 2 * 8 + 4 * 8 + 8 <= 512, "barriers");
    if (a.stages > kMaxStages)
        return cudaErrorInvalidValue;
#define MX_CASE(N)                                                                              \
    if (nt == N)                                                                                \
        return block == 16 ? launch_t<N, 16>(a, grid, s) : launch_t<N, 32>(a, grid, s)
    MX_CASE(16);
    MX_CASE(32);
    MX_CASE(64);
    MX_CASE(128);
    MX_CASE(224);
#undef MX_CASE
    return cudaErrorInvalidValue;
}

}  // namespace fp4
}  // namespace mx
