// mx_fp8_rows.cu -- the FP8 products for many rows: tokens on the M side of the
// MMA, weights on its N side.
//
//   y[m, o] = sum_b (sx[m, b] * sw[o / 128, b]) * sum_{k in block b} qx[m, k] qw[o, k]
//
// Same mathematics as mx_fp8_gemm.cu, the other way round.  There the scale of a
// token belongs to a TMEM column, so the summing warps read a vector of factors
// from shared memory for every block, beside a tensor core that reads its operands
// there.  Here a token is a TMEM lane and its factor for a block one register.
//
// A tile is 128 tokens x BN weight rows (kGateUp: 128 gate and the same 128 up rows).
// Warps:
//   0-7   sums: two warpgroups, each 64 columns of each 128; a thread keeps BN / 2
//         running sums of its token in registers (232 after setmaxnreg)
//   8     TMA producer: token and weight tiles (SWIZZLE_128B)
//   9     MMA: four tcgen05.mma (K = 32) a block, two TMEM buffers of BN columns
//   10    factors: sx * sw of a block for each token (and 128 weight rows) into shared
//         memory, beside the TMEM buffer, so that the summing threads wait for no load from
//         global memory
// A 16-byte load of shared memory takes a warp 110 to 220 cycles beside the MMAs' own reads and
// 73 without, so a buffer has one barrier for its products and its factors, and one for its
// release.
// Results pass through 2 KB of shared memory a warp, 16 of its 32 rows at a time, so
// that they leave as whole lines.
//
// A launch may hold two problems, the routed experts' and the shared expert's: the
// first is bound by HBM, the second by the tensor cores, and their tiles alternate.
//
// What bounds it: a block of 128 x 256 x 128 takes the tensor core 512 cycles (four MMAs of
// 128); the summing warps follow it, two sums to an FMA instruction, but a tile's end is
// theirs, and the two buffers let the MMAs run only two blocks ahead of it.  4096 x 4096 x 4096
// takes 58 us, 2.35 PFLOP/s: 512 tiles on 152 SMs are four rounds for 3.4 of work, 34 us of
// MMAs; without the sums it takes 54.  32768 rows of 256 experts x 1024 x 4096 take 210 us, 6.1
// TB/s; gate/up and down of 4096 tokens of top-8 of those, with a shared expert of 4096, 480
// and 330 us.  Tried and slower: a CTA pair (141 us at 4096^3: each block's hand-over crosses
// the pair), 128 columns a tile in four buffers (104 us), sixteen summing warps (66 us).
#include "mx_fp8_tc.cuh"

namespace mx {
namespace fp8 {

namespace {

constexpr int kSumWarps = 8, kWarps = 12, kThreads = kWarps * 32;
constexpr uint32_t kTile = 128 * 128;

constexpr int kAcc = 2;  // TMEM buffers of BN columns

constexpr uint32_t stage_bytes(int bn) { return kTile + bn * 128; }
constexpr int stages_of(int bn) { return (int)(196608 / stage_bytes(bn)); }

// Dynamic shared memory after the ring.
struct RowTail {
    int out, am, fac, tab, bars, total;
};
__host__ __device__ constexpr RowTail row_tail()
{
    RowTail t{};
    int o = 0;
    t.out = o;  // a warp's results on their way out
    o += kSumWarps * 2048;
    t.am = o;  // largest hidden value of each token in each half of the columns
    o += 2 * 128 * 4;
    t.fac = o;  // [buffer][half or matrix][token]
    o += kAcc * 2 * 128 * 4;
    t.tab = o;
    o += (3 * kMaxExperts + 16) * 4;
    t.bars = o;
    o += 384;
    t.total = o;
    return t;
}

struct Tile {
    int p;  // problem
    int e, f, tok0, n;
};

struct RowWalk {
    int n0, n;   // units of the first problem, of both
    int ft0, ft1;
    const int *tt, *lo, *len;  // groups of the first problem
};

// Unit v of the launch.  The second problem's units are spread evenly among the
// first's.  Within a problem: the matrix, then its weight tile, then the token
// tile, so that the token tiles of one weight tile are worked on at one time.
__device__ __forceinline__ Tile tile_at(const RowsArgs &a, const RowWalk &w, int v)
{
    Tile T;
    const int n1 = w.n - w.n0;
    const int s = n1 ? (int)((int64_t)v * n1 / w.n) : 0;
    if (n1 && (int)((int64_t)(v + 1) * n1 / w.n) > s) {
        const int t = (a.p[1].rows + 128 - 1) / (128);
        T.p = 1;
        T.e = 0;
        T.f = s / t;
        T.tok0 = 128 * (s - T.f * t);
        T.n = min(128, a.p[1].rows - T.tok0);
        return T;
    }
    const int u = v - s;
    int lo = 0, hi = a.p[0].E;
    while (lo + 1 < hi) {
        const int mid = (lo + hi) >> 1;
        if (w.tt[mid] * w.ft0 <= u)
            lo = mid;
        else
            hi = mid;
    }
    const int t = w.tt[lo + 1] - w.tt[lo], x = u - w.tt[lo] * w.ft0;
    T.p = 0;
    T.e = lo;
    T.f = x / t;
    const int r = 128 * (x - T.f * t);
    T.tok0 = w.lo[lo] + r;
    T.n = min(128, w.len[lo] - r);
    return T;
}

// Request 32 columns of this warp's TMEM lanes; r holds them after tmem_wait.
__device__ __forceinline__ void tmem_get32(uint32_t ta, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : MX_R16(r, 0), MX_R16(r, 16)
                 : "r"(ta)
                 : "memory");
}

// 16-byte piece c (0..3) of row r in a warp's 2 KB: 32 rows of 64 bytes, pieces
// rotated so that neither a row per lane nor four lanes per row conflict.
__device__ __forceinline__ int piece(int r, int c) { return r * 4 + (c ^ ((r >> 1) & 3)); }

// The same for 16 rows of 128 bytes.
__device__ __forceinline__ int line_piece(int r, int c) { return r * 8 + (c ^ (r & 7)); }

__device__ __forceinline__ uint32_t bf16_x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t f16_x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int MODE, int BN>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const __grid_constant__ RowsArgs a)
{
    constexpr int NS = stages_of(BN), NSUB = BN / 128, NC = BN / 2;  // buffers of a block, columns of a thread
    constexpr uint32_t kStage = stage_bytes(BN);
    constexpr RowTail RT = row_tail();
    static_assert(NS <= 12, "barriers");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *tail = ring + NS * kStage;
    float *am = reinterpret_cast<float *>(tail + RT.am);
    float *fac = reinterpret_cast<float *>(tail + RT.fac);
    int *tab = reinterpret_cast<int *>(tail + RT.tab);
    uint64_t *full = reinterpret_cast<uint64_t *>(tail + RT.bars), *empty = full + 12;
    uint64_t *tfull = empty + 12, *tempty = tfull + kAcc;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(tempty + kAcc);
    volatile int *abort = reinterpret_cast<volatile int *>(tslot + 1);
    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < kAcc; ++i) {
            mbar_init(tfull + i, 2);  // products, factors
            mbar_init(tempty + i, kSumWarps);
        }
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                     "r"(kAcc * BN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    RowWalk w;
    {
        int *tt = tab, *lo = tab + kMaxExperts + 1, *len = lo + kMaxExperts;
        if (warp == 0)
            group_table(a.p[0].offsets, a.p[0].E, a.p[0].rows, 128, lane, tt, lo, len);
        w.tt = tt;
        w.lo = lo;
        w.len = len;
        w.ft0 = MODE == kGateUp ? blocks(a.p[0].N) : (a.p[0].N + BN - 1) / BN;
        w.ft1 = MODE == kGateUp ? blocks(a.p[1].N) : (a.p[1].N + BN - 1) / BN;
    }
    fence_before();
    __syncthreads();
    fence_after();
    w.n0 = w.tt[a.p[0].E] * w.ft0;
    w.n = w.n0 + (a.p[1].rows + 128 - 1) / (128) * w.ft1;
    const uint32_t tmem = *tslot;

    if (warp >= kSumWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        // (TMA and MMA: the whole warp walks the loop and one elected lane issues.  Behind `lane ==
        // 0` the compiler does not know that one lane is left and issues each in a loop over lanes.)
        if (warp == 8) {
            // -------------------------------------------------- TMA producer
            int s = 0;
            uint32_t ph = 1;
            for (int u = blockIdx.x; u < w.n; u += gridDim.x) {
                const Tile T = tile_at(a, w, u);
                const RowsProblem &P = a.p[T.p];
                const int KB = blocks(P.K), xr = (T.n + kRowsBox - 1) / kRowsBox * kRowsBox;
                const int row0 = MODE == kGateUp ? T.f * kBlk : T.f * BN;
                // (rows of the second half behind the matrix: no copy, their columns are not stored)
                const bool two = NSUB == 2 && (MODE == kGateUp || row0 + 128 < P.N);
                for (int kb = 0; kb < KB; ++kb) {
                    if (!wwait(empty + s, ph, a.err, abort))
                        goto produced;
                    uint8_t *st = ring + s * kStage;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(full + s, xr * 128 + (two ? 2 : 1) * kTile);
                        for (int r = 0; r < T.n; r += kRowsBox)
                            tma_2d(st + r * 128, &P.xm, kb * kBlk, T.tok0 + r, full + s);
                        tma_3d(st + kTile, &P.wa, kb * kBlk, row0, T.e, full + s);
                        if (two)
                            tma_3d(st + 2 * kTile, MODE == kGateUp ? &P.wb : &P.wa, kb * kBlk,
                                   MODE == kGateUp ? row0 : row0 + 128, T.e, full + s);
                    }
                    __syncwarp();
                    if (++s == NS)
                        s = 0, ph ^= 1;
                }
            }
        produced:;
        } else if (warp == 9) {
            // ----------------------------------------------------------- MMA
            int s = 0, b = 0;
            uint32_t ph = 0, tph = 1;
            const uint32_t idesc = idesc_e4m3(BN);
            for (int u = blockIdx.x; u < w.n; u += gridDim.x) {
                const int KB = blocks(a.p[tile_at(a, w, u).p].K);
                for (int kb = 0; kb < KB; ++kb) {
                    if (!wwait(full + s, ph, a.err, abort) || !wwait(tempty + b, tph, a.err, abort))
                        goto issued;
                    fence_after();
                    const uint32_t st = smem_u32(ring + s * kStage);
                    const uint64_t xd = sw128_desc(st), wd = sw128_desc(st + kTile);
                    umma_block(tmem + b * BN, xd, wd, idesc);
                    umma_commit2(tfull + b, empty + s);
                    if (++b == kAcc)
                        b = 0, tph ^= 1;
                    if (++s == NS)
                        s = 0, ph ^= 1;
                }
            }
        issued:;
        } else if (warp == 10) {
            // ------------------------------------------------------- factors
            constexpr int BATCH = 2;
            int b = 0;
            uint32_t ph = 1;
            bool ok = true;
            for (int u = blockIdx.x; u < w.n && ok; u += gridDim.x) {
                const Tile T = tile_at(a, w, u);
                const RowsProblem &P = a.p[T.p];
                const int KB = blocks(P.K), NB = blocks(P.N);
                const int blk = MODE == kGateUp ? T.f : T.f * (BN / 128);
                const int64_t at = ((int64_t)T.e * NB + blk) * KB;
                const float *s0 = P.swa + at;
                const float *s1 = MODE == kGateUp ? P.swb + at : blk + 1 < NB ? s0 + KB : s0;
                const float *sx[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sx[j] = P.sx + (int64_t)(T.tok0 + min(lane + 32 * j, T.n - 1)) * P.sx_r;
                for (int kb0 = 0; kb0 < KB && ok; kb0 += BATCH) {
                    float x[BATCH][4], w0[BATCH], w1[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int kb = min(kb0 + i, KB - 1);
                        w0[i] = __ldg(s0 + kb);
                        w1[i] = __ldg(s1 + kb);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[i][j] = __ldg(sx[j] + kb * P.sx_b);
                    }
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        if (kb0 + i >= KB)
                            break;
                        ok &= wwait(tempty + b, ph, a.err, abort);
                        float *o = fac + b * 256 + lane;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            o[32 * j] = x[i][j] * w0[i];
                            o[128 + 32 * j] = x[i][j] * w1[i];
                        }
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(tfull + b);
                        if (++b == kAcc)
                            b = 0, ph ^= 1;
                    }
                }
            }
        }
    } else {
        // -------------------------------------------------------------- sums
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int wg = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t ta = tmem + ((uint32_t)quad << 21);
        uint4 *mine = reinterpret_cast<uint4 *>(tail + RT.out + warp * 2048);
        int b = 0;
        uint32_t tph = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < w.n && ok; u += gridDim.x) {
            const Tile T = tile_at(a, w, u);
            const RowsProblem &P = a.p[T.p];
            const int KB = blocks(P.K);
            const int n = T.n, tok0 = T.tok0;
            const bool live = quad * 32 < n;  // (a warp without tokens only releases the buffers)
            uint64_t acc2[NC / 2];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i)
                acc2[i] = 0;
            // (a warp without tokens has a loop of its own, and a wait that gave up does not leave
            // the loop early: either made the compiler copy the sums in every block)
            auto release = [&]() {
                fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(tempty + b);
                if (++b == kAcc)
                    b = 0, tph ^= 1;
            };
            if (!live)
                for (int kb = 0; kb < KB; ++kb) {
                    ok &= bwait(tfull + b, tph, a.err, abort);
                    release();
                }
            else
                for (int kb = 0; kb < KB; ++kb) {
                    ok &= bwait(tfull + b, tph, a.err, abort);
                    fence_after();
                    // 64 columns of each half of the buffer, 32 at a time, the next 32 on their way
                    const uint32_t tb = ta + b * BN + wg * 64;
                    uint32_t r[2][32];
                    tmem_get32(tb, r[0]);
                    const float f[2] = {fac[b * 256 + row], fac[b * 256 + 128 + row]};
#pragma unroll
                    for (int h = 0; h < 2 * NSUB; ++h) {
                        tmem_wait();
                        if (h + 1 < 2 * NSUB)
                            tmem_get32(tb + ((h + 1) >> 1) * 128 + ((h + 1) & 1) * 32, r[(h + 1) & 1]);
                        else
                            release();  // (the columns and the factors are in registers)
                        const uint64_t ff = pair_f32(f[h >> 1], f[h >> 1]);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            fma_after(acc2[h * 16 + i], r[h & 1][2 * i], r[h & 1][2 * i + 1], ff);
                    }
                }
            ok = __all_sync(0xFFFFFFFFu, ok);
            float acc[NC];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i)
                unpair_f32(acc2[i], acc[2 * i], acc[2 * i + 1]);

            if constexpr (MODE == kGateUp) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) {
                    acc[i] = act_of(acc[i], a.act) * acc[NC / 2 + i];
                    m = max(m, __float_as_uint(acc[i]) & 0x7FFFFFFFu);
                }
                am[wg * 128 + row] = __uint_as_float(m);
                // both halves of a token's hidden block; the eight warps give up together
                __syncwarp();
                ok = named_and(1, 256, ok);
                if (!ok)
                    break;
                m = max(m, __float_as_uint(am[(wg ^ 1) * 128 + row]));
                const float s = scale_of(__uint_as_float(m), 0);
                const Quotient q(__uint_as_float(m), s);
                if (q.m != 1.0f)
#pragma unroll
                    for (int i = 0; i < NC / 2; ++i)
                        acc[i] *= q.m;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t e[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float *h = acc + 16 * c + 4 * i;
                        e[i] = q.e4m3_of(h[0], h[1]) | q.e4m3_of(h[2], h[3]) << 16;
                    }
                    mine[piece(lane, c)] = make_uint4(e[0], e[1], e[2], e[3]);
                }
                if (wg == 0 && row < n)
                    P.hs[(int64_t)T.f * P.hs_ld + tok0 + row] = s;
                __syncwarp();
                uint8_t *h = P.h + (int64_t)(tok0 + quad * 32 + (lane >> 2)) * P.ldh + T.f * kBlk + wg * 64 + (lane & 3) * 16;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (quad * 32 + i * 8 + (lane >> 2) < n)
                        *reinterpret_cast<uint4 *>(h + i * 8 * P.ldh) = mine[piece(i * 8 + (lane >> 2), lane & 3)];
                // (am of this tile is read before the next tile's barrier, after which it may be overwritten)
                __syncwarp();
                ok = named_and(2, 256, ok);
            } else {
                if (!ok)
                    break;
                if (!live)
                    continue;
                // (this thread's columns: 64 of each buffer of 128)
                const int o0 = T.f * BN + wg * 64;
                const int es = P.out_kind == kOutF32 ? 4 : 2, per = 16 / es;
                if (P.out_kind == kOutF16) {
                    // FP16 of y 2^-k, k such that the row's largest finite of 64 columns is below 2^15, and
                    // 2^k beside it: 11 significant bits at half the bytes.  Under a bf16 result, whose 8 bits
                    // are what is left of them: the layer of 4096 tokens takes 994 us, with fp32 rows 1110; of
                    // 700 tokens it is off by 1.675e-3 of its norm, with fp32 rows by 1.662e-3.
                    // (2^-112 counts as the smallest: 2^k and 2^-k stay normal.)  The maximum is taken on the
                    // bits one exponent up, where infinities and NaN, which keep themselves, are negative.
#pragma unroll
                    for (int j = 0; j < NSUB; ++j) {
                        int m = 16 << 23;
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            m = max(m, (int)((__float_as_uint(acc[j * 64 + i]) & 0x7FFFFFFFu) + (1u << 23)));
                        const int k = (m >> 23) - 1 - (127 + 14);
                        const float down = __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            acc[j * 64 + i] *= down;
                        if (row < n && o0 + j * 128 < P.N)
                            P.out_scale[(int64_t)(tok0 + row) * P.out_scale_ld + (o0 >> 6) + 2 * j] =
                                __uint_as_float((uint32_t)(127 + k) << 23);
                    }
                }
                // Passes of 16 rows x 128 bytes (64 two-byte or 32 four-byte columns): whole lines leave.
                const int prow = lane >> 3, col = (lane & 7) * per;  // this lane's row of four, and column
                char *base = static_cast<char *>(P.out) + ((int64_t)(tok0 + quad * 32 + prow) * P.ldo + o0 + col) * es;
                const int64_t rstep = 4 * P.ldo * es;
                // rows r0 .. r0 + 15, columns c0 on; x: this lane's row, eight pieces of 16 bytes
                auto pass = [&](int r0, int c0, auto &&x) {
                    if ((lane >> 4) == (r0 >> 4))
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            mine[line_piece(lane & 15, c)] = x(c);
                    __syncwarp();
                    const int o = o0 + c0 + col, rows = n - quad * 32 - r0 - prow;  // (rows 0, 4, 8, 12 below it)
                    char *to = base + (r0 >> 2) * rstep + c0 * es;
                    if (!P.out_vec) {
                        // a row at a time, one word of it to a lane
                        const int left = P.N - o0 - c0, nr = n - quad * 32 - r0, c = lane * 4 / es;
                        const uint32_t *word = reinterpret_cast<const uint32_t *>(mine);
                        char *p = static_cast<char *>(P.out) + ((int64_t)(tok0 + quad * 32 + r0) * P.ldo + o0 + c0 + c) * es;
#pragma unroll 8
                        for (int i = 0; i < 16; ++i, p += P.ldo * es) {
                            const uint32_t v = word[line_piece(i, lane >> 2) * 4 + (lane & 3)];
                            if (i < nr && c < left) {
                                if (es == 4) {
                                    *reinterpret_cast<uint32_t *>(p) = v;
                                } else {
                                    reinterpret_cast<uint16_t *>(p)[0] = (uint16_t)v;
                                    if (c + 1 < left)
                                        reinterpret_cast<uint16_t *>(p)[1] = (uint16_t)(v >> 16);
                                }
                            }
                        }
                    } else if (o + per <= P.N) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (4 * i < rows)
                                *reinterpret_cast<uint4 *>(to + i * rstep) = mine[line_piece(4 * i + prow, lane & 7)];
                    } else {
                        for (int i = 0; i < 4 && 4 * i < rows; ++i) {
                            const uint4 v = mine[line_piece(4 * i + prow, lane & 7)];
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                            char *p = to + i * rstep;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                if (k >= per || o + k >= P.N)
                                    break;
                                if (es == 2)
                                    reinterpret_cast<uint16_t *>(p)[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
                                else
                                    reinterpret_cast<uint32_t *>(p)[k] = w[k & 3];
                            }
                        }
                    }
                    __syncwarp();
                };
#pragma unroll
                for (int j = 0; j < NSUB; ++j) {
                    const float *y = acc + 64 * j;
                    if (P.out_kind == kOutF32) {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int r0 = 0; r0 < 32; r0 += 16)
                                pass(r0, 128 * j + 32 * q, [&](int c) {
                                    const float *z = y + 32 * q + 4 * c;
                                    return make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]),
                                                      __float_as_uint(z[3]));
                                });
                    } else {
                        uint32_t h[32];
                        if (P.out_kind == kOutF16) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                h[i] = f16_x2(y[2 * i], y[2 * i + 1]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                h[i] = bf16_x2(y[2 * i], y[2 * i + 1]);
                        }
#pragma unroll
                        for (int r0 = 0; r0 < 32; r0 += 16)
                            pass(r0, 128 * j,
                                 [&](int c) { return make_uint4(h[4 * c], h[4 * c + 1], h[4 * c + 2], h[4 * c + 3]); });
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
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kAcc * BN) : "memory");
}

template <int MODE, int BN>
cudaError_t launch_t(const RowsArgs &a, int grid, cudaStream_t s)
{
    const size_t smem = 1024 + stages_of(BN) * stage_bytes(BN) + row_tail().total;
    const cudaError_t e = smem_optin((const void *)rows_kernel<MODE, BN>, smem);
    if (e != cudaSuccess)
        return e;
    rows_kernel<MODE, BN><<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows(Mode mode, int bn, const RowsArgs &a, int grid, cudaStream_t s)
{
    if (mode == kGateUp)
        return launch_t<kGateUp, 256>(a, grid, s);
    return bn == 256 ? launch_t<kProduct, 256>(a, grid, s) : launch_t<kProduct, 128>(a, grid, s);
}

}  // namespace fp8
}  // namespace mx
