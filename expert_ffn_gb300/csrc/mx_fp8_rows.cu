// mx_fp8_rows.cu -- the FP8 products for many rows: tokens on the M side of the
// MMA, weights on its N side.
//
//   y[m, o] = sum_b (sx[m, b] * sw[o / 128, b]) * sum_{k in block b} qx[m, k] qw[o, k]
//
// Same mathematics as mx_fp8_gemm.cu, the other way round.  There the scale of a
// token belongs to a TMEM column, so the summing warps read a vector of factors
// from shared memory for every block (2 wavefronts per 16 bytes, measured), and
// under a busy tensor core, which itself reads 96 of the 128 bytes a cycle that
// shared memory delivers, that took 9 cycles a column.  Here a token is a TMEM
// lane: its scale is one register, its factor for a block one product, and the
// sums cost a TMEM load and half an FMA instruction a column.
//
// A CTA walks tiles of 128 tokens x BN weight rows (kGateUp: 128 gate and the
// same 128 up rows).  Warps:
//   0-7   sums: two warpgroups, each half of the tile's columns; a thread keeps
//         BN / 2 running sums of its token in registers (216 after setmaxnreg)
//   8     TMA producer: token and weight tiles (SWIZZLE_128B), 4 stages of 128
//         columns
//   9     MMA: one lane, four tcgen05.mma (K = 32) a block, two TMEM buffers
// Results pass through 2 KB of shared memory a warp, 64 bytes of each of its 32
// rows at a time, so that they leave in 16-byte pieces of whole sectors; no
// barrier between warps is involved.
#include "mx_fp8_tc.cuh"

namespace mx {
namespace fp8 {

namespace {

constexpr int kSumWarps = 8, kWarps = 12, kThreads = kWarps * 32;
constexpr uint32_t kTile = 128 * 128;
constexpr int kStages(int bn) { return bn == 256 ? 4 : 6; }
constexpr uint32_t stage_bytes(int bn) { return kTile + bn * 128; }

// Dynamic shared memory after the ring.
struct RowTail {
    int out, am, tab, bars, total;
};
__host__ __device__ constexpr RowTail row_tail()
{
    RowTail t{};
    int o = 0;
    t.out = o;  // a warp's results on their way out
    o += kSumWarps * 2048;
    t.am = o;  // largest hidden value of each token in each half of the columns
    o += 2 * 128 * 4;
    t.tab = o;
    o += (3 * kMaxExperts + 16) * 4;
    t.bars = o;
    o += 256;
    t.total = o;
    return t;
}

struct Tile {
    int e, f, tok0, n;
};

struct RowWalk {
    int n_units, FT;
    const int *tt, *lo, *len;
};

// Tile u: the matrix, then its weight tile, then the token tile, so that the
// token tiles of one weight tile are worked on at the same time.
__device__ __forceinline__ Tile tile_at(const GemmArgs &a, const RowWalk &w, int u)
{
    int lo = 0, hi = a.E;
    while (lo + 1 < hi) {
        const int mid = (lo + hi) >> 1;
        if (w.tt[mid] * w.FT <= u)
            lo = mid;
        else
            hi = mid;
    }
    const int t = w.tt[lo + 1] - w.tt[lo], v = u - w.tt[lo] * w.FT;
    Tile T;
    T.e = lo;
    T.f = v / t;
    const int r = 128 * (v - T.f * t);
    T.tok0 = w.lo[lo] + r;
    T.n = min(128, w.len[lo] - r);
    return T;
}

__device__ __forceinline__ void tmem_ld32(uint32_t ta, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : MX_R16(r, 0), MX_R16(r, 16)
                 : "r"(ta)
                 : "memory");
}

#define MX_W16O(r, o)                                                                                               \
    "+r"(r[o + 0]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), "+r"(r[o + 6]), \
        "+r"(r[o + 7]), "+r"(r[o + 8]), "+r"(r[o + 9]), "+r"(r[o + 10]), "+r"(r[o + 11]), "+r"(r[o + 12]),          \
        "+r"(r[o + 13]), "+r"(r[o + 14]), "+r"(r[o + 15])

__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : MX_W16O(r, 0), MX_W16O(r, 16)::"memory");
}

// 16-byte piece c (0..3) of row r in a warp's 2 KB: 32 rows of 64 bytes, pieces
// rotated so that neither a row per lane nor four lanes per row conflict.
__device__ __forceinline__ int piece(int r, int c) { return r * 4 + (c ^ ((r >> 1) & 3)); }

template <int MODE, int BN>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const __grid_constant__ GemmArgs a)
{
    constexpr int NS = kStages(BN), NC = BN / 2, NH = NC / 32;  // columns of a thread, loads of 32
    constexpr uint32_t kStage = stage_bytes(BN);
    constexpr RowTail RT = row_tail();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *tail = ring + NS * kStage;
    float *am = reinterpret_cast<float *>(tail + RT.am);
    int *tab = reinterpret_cast<int *>(tail + RT.tab);
    uint64_t *full = reinterpret_cast<uint64_t *>(tail + RT.bars), *empty = full + 8;
    uint64_t *tfull = empty + 8, *tempty = tfull + 2;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(tempty + 2);
    volatile int *abort = reinterpret_cast<volatile int *>(tslot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + i, 1);
            mbar_init(tempty + i, kSumWarps);
        }
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                     "r"(2 * BN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    RowWalk w;
    {
        int *tt = tab, *lo = tab + kMaxExperts + 1, *len = lo + kMaxExperts;
        if (warp == 0)
            group_table(a, 128, lane, tt, lo, len);
        w.tt = tt;
        w.lo = lo;
        w.len = len;
        w.FT = MODE == kGateUp ? blocks(a.N) : (a.N + BN - 1) / BN;
    }
    fence_before();
    __syncthreads();
    fence_after();
    w.n_units = w.tt[a.E] * w.FT;
    const uint32_t tmem = *tslot;
    const int KB = blocks(a.K), NB = blocks(a.N);

    if (warp >= kSumWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8 && lane == 0) {
            // -------------------------------------------------- TMA producer
            int s = 0;
            uint32_t ph = 1;
            for (int u = blockIdx.x; u < w.n_units; u += gridDim.x) {
                const Tile T = tile_at(a, w, u);
                const int xr = (T.n + a.xbox - 1) / a.xbox * a.xbox;
                // (rows of the second half behind the matrix: no copy, its columns are not stored)
                const bool two = BN == 256 && (MODE == kGateUp || T.f * BN + 128 < a.N);
                for (int kb = 0; kb < KB; ++kb) {
                    if (!bwait(empty + s, ph, a.err, abort))
                        goto produced;
                    uint8_t *st = ring + s * kStage;
                    mbar_arrive_expect_tx(full + s, xr * 128 + (two ? 2 : 1) * kTile);
                    for (int r = 0; r < T.n; r += a.xbox)
                        tma_2d(st + r * 128, &a.xm, kb * kBlk, T.tok0 + r, full + s);
                    if (MODE == kGateUp) {
                        tma_3d(st + kTile, &a.wa, kb * kBlk, T.f * kBlk, T.e, full + s);
                        tma_3d(st + 2 * kTile, &a.wb, kb * kBlk, T.f * kBlk, T.e, full + s);
                    } else {
                        tma_3d(st + kTile, &a.wa, kb * kBlk, T.f * BN, T.e, full + s);
                        if (two)
                            tma_3d(st + 2 * kTile, &a.wa, kb * kBlk, T.f * BN + 128, T.e, full + s);
                    }
                    if (++s == NS)
                        s = 0, ph ^= 1;
                }
            }
        produced:;
        } else if (warp == 9 && lane == 0) {
            // ----------------------------------------------------------- MMA
            int s = 0, b = 0;
            uint32_t ph = 0, tph = 1;
            const uint32_t idesc = idesc_e4m3(BN);
            for (int u = blockIdx.x; u < w.n_units; u += gridDim.x)
                for (int kb = 0; kb < KB; ++kb) {
                    if (!bwait(tempty + b, tph, a.err, abort) || !bwait(full + s, ph, a.err, abort))
                        goto issued;
                    fence_after();
                    const uint32_t st = smem_u32(ring + s * kStage);
                    const uint64_t xd = sw128_desc(st), wd = sw128_desc(st + kTile);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f8(tmem + b * BN, xd + 2 * k, wd + 2 * k, idesc, k > 0);
                    umma_commit(empty + s);
                    umma_commit(tfull + b);
                    if (++s == NS)
                        s = 0, ph ^= 1;
                    if (++b == 2)
                        b = 0, tph ^= 1;
                }
        issued:;
        }
    } else {
        // -------------------------------------------------------------- sums
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int wg = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t ta = tmem + ((uint32_t)quad << 21);
        uint4 *mine = reinterpret_cast<uint4 *>(tail + RT.out + warp * 2048);
        int b = 0;
        uint32_t tph = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < w.n_units && ok; u += gridDim.x) {
            const Tile T = tile_at(a, w, u);
            const bool live = quad * 32 < T.n;  // (a warp without tokens only releases the buffers)
            uint64_t acc[NC / 2];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i)
                acc[i] = 0;
            // scales of this token and of the weight blocks of this half: for kGateUp both matrices'
            const float *sx = a.sx + (int64_t)(T.tok0 + min(row, T.n - 1)) * a.sx_r;
            const int blk = MODE == kGateUp ? T.f : min(T.f * (BN / 128) + (BN == 256 ? wg : 0), NB - 1);
            const float *s0 = a.swa + ((int64_t)T.e * NB + blk) * KB;
            const float *s1 = MODE == kGateUp ? a.swb + ((int64_t)T.e * NB + blk) * KB : s0;
            float x0 = sx[0], w0 = __ldg(s0), v0 = MODE == kGateUp ? __ldg(s1) : 0.0f;
            for (int kb = 0; kb < KB; ++kb) {
                const int nx = min(kb + 1, KB - 1);  // the next block's scales, ahead of their use
                const float x1 = sx[nx * a.sx_b], w1 = __ldg(s0 + nx), v1 = MODE == kGateUp ? __ldg(s1 + nx) : 0.0f;
                ok = wwait(tfull + b, tph, a.err, abort);
                if (!ok)
                    break;
                fence_after();
                const float f0 = x0 * w0, f1 = MODE == kGateUp ? x0 * v0 : f0;
                if (live) {
                    const uint32_t tb = ta + b * BN + (MODE == kGateUp ? wg * 64 : wg * NC);
                    // kGateUp: 64 gate columns, then the 64 up columns 128 further on
                    auto at = [&](int h) { return tb + (MODE == kGateUp && h >= NH / 2 ? 128 - NC / 2 : 0) + 32 * h; };
                    uint32_t r[2][32];
                    tmem_ld32(at(0), r[0]);
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        tmem_wait32(r[h & 1]);
                        if (h + 1 < NH)
                            tmem_ld32(at(h + 1), r[(h + 1) & 1]);
                        const float f = MODE == kGateUp && h >= NH / 2 ? f1 : f0;
                        const uint64_t ff = pair_f32(f, f);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            fma_f32x2(acc[h * 16 + j],
                                      pair_f32(__uint_as_float(r[h & 1][2 * j]), __uint_as_float(r[h & 1][2 * j + 1])),
                                      ff);
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(tempty + b);
                if (++b == 2)
                    b = 0, tph ^= 1;
                x0 = x1, w0 = w1, v0 = v1;
            }

            if constexpr (MODE == kGateUp) {
                float hv[NC / 2];
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < NC / 4; ++i) {
                    float g0, g1, u0, u1;
                    unpair_f32(acc[i], g0, g1);
                    unpair_f32(acc[NC / 4 + i], u0, u1);
                    hv[2 * i] = act_of(g0, a.act) * u0;
                    hv[2 * i + 1] = act_of(g1, a.act) * u1;
                    m = max(m, max(__float_as_uint(hv[2 * i]) & 0x7FFFFFFFu, __float_as_uint(hv[2 * i + 1]) & 0x7FFFFFFFu));
                }
                am[wg * 128 + row] = __uint_as_float(m);
                // both halves of a token's hidden block; the eight warps give up together
                __syncwarp();
                ok = named_and(1, 256, ok);
                if (!ok)
                    break;
                m = max(m, __float_as_uint(am[(wg ^ 1) * 128 + row]));
                const float s = scale_of(__uint_as_float(m), 0);
                // (by a reciprocal: h is a rounded sum, on no border between two e4m3 numbers)
                const float inv = __frcp_rn(s);
                uint32_t e[NC / 8];
#pragma unroll
                for (int i = 0; i < NC / 8; ++i)
                    e[i] = e4m3_x2(hv[4 * i] * inv, hv[4 * i + 1] * inv) |
                           e4m3_x2(hv[4 * i + 2] * inv, hv[4 * i + 3] * inv) << 16;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    mine[piece(lane, c)] = make_uint4(e[4 * c], e[4 * c + 1], e[4 * c + 2], e[4 * c + 3]);
                if (wg == 0 && row < T.n)
                    a.hs[(int64_t)T.f * a.hs_ld + T.tok0 + row] = s;
                __syncwarp();
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 8 + (lane >> 2), t = quad * 32 + r;
                    if (t < T.n)
                        *reinterpret_cast<uint4 *>(a.h + (int64_t)(T.tok0 + t) * a.ldh + T.f * kBlk + wg * 64 +
                                                   (lane & 3) * 16) = mine[piece(r, lane & 3)];
                }
                // (am of this tile is read before the next tile's barrier, after which it may be overwritten)
                ok = named_and(2, 256, ok);
            } else {
                if (!ok)
                    break;
                if (!live)
                    continue;
                const int o0 = T.f * BN + wg * NC;
                // passes of 64 bytes a row: 32 bf16 or 16 fp32 columns
                auto flush = [&](int c0, int per) {
                    __syncwarp();
                    for (int i = 0; i < 4; ++i) {
                        const int r = i * 8 + (lane >> 2), t = quad * 32 + r, o = o0 + c0 + (lane & 3) * per;
                        const uint4 v = mine[piece(r, lane & 3)];
                        if (t >= T.n || o >= a.N)
                            continue;
                        const int64_t at = (int64_t)(T.tok0 + t) * a.ldo + o;
                        if (a.out_bf16) {
                            uint16_t *p = reinterpret_cast<uint16_t *>(a.out) + at;
                            if (a.out_vec && o + 8 <= a.N) {
                                *reinterpret_cast<uint4 *>(p) = v;
                            } else {
                                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    if (o + k < a.N)
                                        p[k] = (uint16_t)(x[k >> 1] >> (16 * (k & 1)));
                            }
                        } else {
                            uint32_t *p = reinterpret_cast<uint32_t *>(a.out) + at;
                            if (a.out_vec && o + 4 <= a.N) {
                                *reinterpret_cast<uint4 *>(p) = v;
                            } else {
                                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (o + k < a.N)
                                        p[k] = x[k];
                            }
                        }
                    }
                    __syncwarp();
                };
                auto bf2 = [](uint64_t v) {
                    float lo, hi;
                    unpair_f32(v, lo, hi);
                    uint32_t r;
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
                    return r;
                };
                if (a.out_bf16) {
#pragma unroll
                    for (int p = 0; p < NC / 32; ++p) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            mine[piece(lane, c)] = make_uint4(bf2(acc[16 * p + 4 * c]), bf2(acc[16 * p + 4 * c + 1]),
                                                              bf2(acc[16 * p + 4 * c + 2]), bf2(acc[16 * p + 4 * c + 3]));
                        flush(32 * p, 8);
                    }
                } else {
#pragma unroll
                    for (int p = 0; p < NC / 16; ++p) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            float y0, y1, y2, y3;
                            unpair_f32(acc[8 * p + 2 * c], y0, y1);
                            unpair_f32(acc[8 * p + 2 * c + 1], y2, y3);
                            mine[piece(lane, c)] = make_uint4(__float_as_uint(y0), __float_as_uint(y1),
                                                              __float_as_uint(y2), __float_as_uint(y3));
                        }
                        flush(16 * p, 4);
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
    fence_after();
    __syncwarp();
    if (warp == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN) : "memory");
}

template <int MODE, int BN>
cudaError_t launch_t(const GemmArgs &a, int grid, cudaStream_t s)
{
    const size_t smem = 1024 + kStages(BN) * stage_bytes(BN) + row_tail().total;
    const cudaError_t e = smem_optin((const void *)rows_kernel<MODE, BN>, smem);
    if (e != cudaSuccess)
        return e;
    rows_kernel<MODE, BN><<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows(Mode mode, int bn, const GemmArgs &a, int grid, cudaStream_t s)
{
    if (mode == kGateUp)
        return launch_t<kGateUp, 256>(a, grid, s);
    return bn == 256 ? launch_t<kProduct, 256>(a, grid, s) : launch_t<kProduct, 128>(a, grid, s);
}

}  // namespace fp8
}  // namespace mx
