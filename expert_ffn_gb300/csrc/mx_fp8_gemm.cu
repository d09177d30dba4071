// mx_fp8_gemm.cu -- products of e4m3 rows with block-scaled e4m3 matrices on the
// 5th-generation tensor cores (tcgen05, accumulators in TMEM).
//
//   y[m, o] = sum_b (sx[m, b] * sw[o / 128, b]) * sum_{k in block b} qx[m, k] qw[o, k]
//
// The tensor core sums one block of 128 columns; the block's scales are applied
// in fp32 by CUDA cores, which keep the running sums in registers.  The weights
// take the M side of the MMA (128 rows = one block of weight scales, so the
// weight scale is one number per MMA tile and block) and the tokens its N side
// (16 to 64): a single token then costs the smallest N, a group of tokens is
// padded to 16 rather than to 128, and weights stream from HBM straight into
// the MMA's operand layout without passing through a thread.
//
// A CTA walks units (128 weight rows x one token tile, or what Mode says).  Warps:
//   0-3  sums: tcgen05.ld of a block's products (lane quadrant = warp % 4), packed
//        two-lane FMA by the block's factors, and the epilogue
//   4    TMA producer: weight tiles 128 x 128 bytes and token tiles (SWIZZLE_128B)
//        into a ring of stages
//   5    MMA: four tcgen05.mma (K = 32) per matrix and block into a ring of TMEM buffers
//   6    factors: sx * sw of a block for each token into a ring in shared memory, so that
//        the summing warps read them as broadcast vectors
// Few units: a cluster of `cl` CTAs splits the inner dimension of one unit; each CTA
// sums every cl-th token column over the partial sums in all their shared memories,
// in rank order, so the result does not depend on timing; which block is whose goes by
// the sizes alone (first_block), so it does not depend on the other tokens' experts either.
//
// What bounds it: an MMA of 128 weight rows x 32 columns takes 47 cycles up to N = 32 and 53
// at 64, so an SM could stream 77 bytes of weights a cycle, three times its share of HBM: few
// tokens are bound by HBM where there are enough units, and by the chain (launch, tables,
// pipeline fill, eight blocks, cluster) where there are not.  64 x 4096 x 4096 takes 8.5 us (HBM
// 2.6); the layer of 31 tokens of top-8 of 128 experts 48 us, of which the first 5 pass before
// the quantised tokens are there.
//
// Every wait is bounded: a wait that gives up sets the caller's error word and
// ends the CTA's work.
#include "mx_fp8_tc.cuh"

namespace mx {
namespace fp8 {

namespace {

constexpr uint32_t kTile = 128 * 128;  // bytes of one weight tile
constexpr int kFacRing = 8;            // blocks of factors in flight
// Few tokens: the factor of a hidden block of an expert that the token did not choose.
constexpr uint32_t kNotChosen = 0x80000000u;  // -0; a chosen one's has 0 added, which makes a -0 of it +0

constexpr int kSumWarps = 4, kThreads = (kSumWarps + 3) * 32;
constexpr int n_mats(int mode) { return mode == kFewGateUp ? 2 : 1; }
// TMEM buffers: at most 256 columns (two CTAs of an SM share 512).
constexpr int n_acc(int mode, int nt)
{
    const int cols = n_mats(mode) * nt;
    return 256 / cols > 4 ? 4 : 256 / cols;
}
constexpr uint32_t tmem_cols(int mode, int nt)
{
    uint32_t c = 32;
    while (c < (uint32_t)(n_acc(mode, nt) * n_mats(mode) * nt))
        c *= 2;
    return c;
}
constexpr uint32_t stage_bytes(int mode, int nt) { return n_mats(mode) * kTile + nt * 128; }

// Token columns of one pass of the epilogue.  (A cluster, whose one unit is done by
// then, leaves all its columns in the ring instead.)
constexpr int pass_cols(int mode, int nt)
{
    return mode == kFewDown ? 16 : n_mats(mode) * nt > 64 ? 32 : nt;
}

// CTAs that share an SM.
constexpr int per_sm(int mode, int nt) { return mode == kFewDown && nt <= 32 ? 2 : 1; }

// Dynamic shared memory after the ring (byte offsets from its end).
struct Tail {
    int fac, stage, tab, bars, total;
};
__host__ __device__ constexpr Tail tail_of(int mode, int nt)
{
    Tail t{};
    int o = 0;
    t.stage = o;  // sums on their way out: [matrix][column][128 rows] fp32
    o += n_mats(mode) * pass_cols(mode, nt) * 512;
    t.fac = o;
    o += kFacRing * n_mats(mode) * nt * 4;
    t.tab = o;  // expert tables; few tokens: active experts, their bits, routing indices and weights
    o += mode == kFewGateUp || mode == kFewDown ? (kMaxExperts + kMaxExperts / 32 + 2 * nt * kMaxTopK) * 4
                                                : (3 * kMaxExperts + 16) * 4;
    t.bars = o;
    o += 640;
    t.total = o;
    return t;
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
    int kb0, kb1;              // blocks of the inner dimension; kFewDown: 0 and this rank's number
    int FT, n_act;
    int n_routed, sh0, rank;   // kFewDown: of these the routed experts', the first of the shared expert
    const uint32_t *list;      // and the routed ones, as far as they fit (see block_of)
    const int *tt, *lo, *len;  // by tokens: token-tile offsets [E + 1], group starts and lengths [E]
    const int *act;            // few tokens: active experts
    const int *idx;            // their routing: [T][topk] experts and weights
    const float *wts;
};

template <int MODE, int NT>
__device__ __forceinline__ Unit unit_of(const GemmArgs &a, const Walk &w, int u)
{
    Unit U{};
    if (MODE == kProduct) {
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

// kFewDown: a cluster's ranks share the inner blocks of all active experts and the shared one.
// Block c of expert e (the shared one counts as the one behind the last) is rank (e IB + c) mod
// cl's, so that a token's sums are the same whichever experts the other tokens choose: their
// blocks add zeros.  (An even cut of the active experts' blocks moved with those.  This one is
// uneven where few are active: 2 tokens of top-8 of 128 experts 28.2 us, cut evenly 27.4.)
__device__ __forceinline__ int div_cl(const GemmArgs &a, int x)  // (exact: x cl < 2^32)
{
    return a.cl > 1 ? (int)__umulhi((unsigned)x, a.cl_inv) : x;
}

__device__ __forceinline__ int first_block(const GemmArgs &a, int e, int rank)
{
    const int x = e * a.IB, c = rank - (x - div_cl(a, x) * a.cl);
    return c < 0 ? c + a.cl : c;
}

// Entries of Walk::list that there is room for, behind the active experts and their bits.
constexpr int list_room(int nt) { return 2 * nt * kMaxTopK - kMaxExperts / 32; }

// A list entry: expert, its place among the active ones, block.
__device__ __forceinline__ uint32_t list_entry(int e, int at, int c) { return (uint32_t)e | at << 10 | (uint32_t)c << 19; }

// The entry of this rank's routed block kb when there is no room for it in the list: the last
// active expert whose first block comes at kb or before.
__device__ __noinline__ uint32_t far_block(const GemmArgs &a, const int *act, int n_act, int rank, int kb)
{
    const int q = div_cl(a, a.IB);
    int lo = 0, hi = n_act;
    while (lo + 1 < hi) {
        const int mid = (lo + hi) >> 1;
        if (q * mid + (act[mid] >> 16) <= kb)
            lo = mid;
        else
            hi = mid;
    }
    const int e = act[lo] & 0xFFFF;
    return list_entry(e, lo, first_block(a, e, rank) + (kb - q * lo - (act[lo] >> 16)) * a.cl);
}

// Block kb of a unit: matrix (-1: shared), block column; kFewDown: hidden block among all experts'.
struct Block {
    int e, c, item;
};
template <int MODE, int NT>
__device__ __forceinline__ Block block_of(const GemmArgs &a, const Walk &w, const Unit &U, int kb)
{
    if (MODE != kFewDown)
        return Block{U.e, kb, kb};
    if (kb >= w.n_routed) {
        const int c = w.sh0 + (kb - w.n_routed) * a.cl;
        return Block{-1, c, w.n_act * a.IB + c};
    }
    const uint32_t v = kb < list_room(NT) ? w.list[kb] : far_block(a, w.act, w.n_act, w.rank, kb);
    const int c = (int)(v >> 19);
    return Block{(int)(v & 1023), c, (int)(v >> 10 & 511) * a.IB + c};
}
static_assert(kMaxExperts <= 512, "list entries");

// Results of token column n of a unit: 128 weight rows, four to a lane.
template <int MODE, int NT>
__device__ __forceinline__ void emit(const GemmArgs &a, const Walk &w, const Unit &U, int n,
                                     const float4 (&v)[n_mats(MODE)], int lane)
{
    constexpr int NMAT = n_mats(MODE);
    if constexpr (NMAT == 2) {
        // few tokens: the routing weight joins the scale; a token that did not choose the
        // expert (most do not: found out first) has zeros and is marked
        float wt = 1.0f;
        bool in = true;
        if (U.e >= 0) {
            const bool mine = lane < a.topk && w.idx[n * a.topk + lane] == U.e;
            wt = mine ? w.wts[n * a.topk + lane] : 0.0f;
            in = __any_sync(0xFFFFFFFFu, mine);
        }
        uint32_t e = 0;
        float sc = __uint_as_float(kNotChosen);
        if (in) {
            if (U.e >= 0)
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    wt += __shfl_xor_sync(0xFFFFFFFFu, wt, o);
            const float h[4] = {act_of(v[0].x, a.act) * v[NMAT - 1].x, act_of(v[0].y, a.act) * v[NMAT - 1].y,
                                act_of(v[0].z, a.act) * v[NMAT - 1].z, act_of(v[0].w, a.act) * v[NMAT - 1].w};
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mx = max(mx, __float_as_uint(h[i]) & 0x7FFFFFFFu);
            const float top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, mx)), s = scale_of(top, 0);
            const Quotient q(top, s);
            e = q.e4m3_of(h[0] * q.m, h[1] * q.m) | q.e4m3_of(h[2] * q.m, h[3] * q.m) << 16;
            sc = s * wt + 0.0f;
        }
        const int64_t at = (int64_t)U.item * NT + n;
        reinterpret_cast<uint32_t *>(a.h + at * kBlk)[lane] = e;
        if (lane == 0)
            a.hs[at] = sc;
    } else {
        const int o = U.f * kBlk + 4 * lane;
        const int64_t at = (int64_t)(U.tok0 + n) * a.ldo + o;
        float y[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
        if (MODE == kFewDown) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (o + i < a.N)
                    y[i] = fmaf(a.lam, y[i],
                                a.residual ? load_act(a.residual, at + i, a.out_kind == kOutBf16) : 0.0f);
        }
        if (a.out_vec && o + 4 <= a.N) {
            if (a.out_kind == kOutBf16)
                *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(a.out) + at) =
                    make_uint2(f2bf(y[0]) | (uint32_t)f2bf(y[1]) << 16, f2bf(y[2]) | (uint32_t)f2bf(y[3]) << 16);
            else
                *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + at) =
                    make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (o + i < a.N) {
                    if (a.out_kind == kOutBf16)
                        reinterpret_cast<uint16_t *>(a.out)[at + i] = f2bf(y[i]);
                    else
                        reinterpret_cast<float *>(a.out)[at + i] = y[i];
                }
        }
    }
}

// Down of few tokens once more, for a unit with NaN or infinities in its first two columns: block by
// block, each column with the experts that its token chose alone.  (The weights of an expert
// meet the other tokens' zeros too, and zero times a NaN, or a factor of zero times an infinite
// scale, is NaN.)  Columns that were right come out the same, bit for bit.  Apart from the
// kernel's loops, where every instruction counts: with a predicate for each column 64 tokens of
// top-8 of 128 experts took 189 us instead of 153, with a test in the factors alone 31 tokens
// 127 instead of 115; looking at two columns' sums at the unit's end costs 0.4 us at most.
// Leaves the sums [column][128 rows] in `stage`, of a cluster, or as results.  `bars`: three
// barriers; parity: that of the next wait for them, which is returned.
template <int NT>
__device__ __noinline__ uint32_t redo_down(const GemmArgs &a, int f, int n_blocks, int n_routed, const int *act,
                                           const uint32_t *list, int n_act, int sh0, int rank, uint8_t *ring,
                                           float *stage, uint64_t *bars, uint32_t parity, uint32_t tmem,
                                           volatile int *abort)
{
    constexpr int GC = pass_cols(kFewDown, NT);
    Walk w{};
    w.n_routed = n_routed;
    w.act = act;
    w.list = list;
    w.n_act = n_act;
    w.sh0 = sh0;
    w.rank = rank;
    w.FT = blocks(a.N);
    const Unit U = unit_of<kFewDown, NT>(a, w, f);
    const int warp = warp_index(), lane = threadIdx.x & 31, row = (warp & 3) * 32 + lane;
    float acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        acc[n] = 0.0f;
    for (int kb = 0; kb < n_blocks; ++kb) {
        const Block B = block_of<kFewDown, NT>(a, w, U, kb);
        const int e = B.e, c = B.c;
        if (warp == kSumWarps) {
            if (elect_one()) {
                mbar_arrive_expect_tx(bars, kTile + NT * 128);
                tma_3d(ring, e < 0 ? &a.sa : &a.wa, c * kBlk, U.f * kBlk, e < 0 ? 0 : e, bars);
                tma_2d(ring + kTile, &a.xm, 0, B.item * NT, bars);
            }
            __syncwarp();
        }
        bool ok = wwait(bars, parity, a.err, abort);
        if (warp == kSumWarps + 1 && ok) {
            umma_block(tmem, sw128_desc(smem_u32(ring)), sw128_desc(smem_u32(ring + kTile)),
                       idesc_e4m3((U.n + 15) & ~15));
            umma_commit2(bars + 1, bars + 2);
        }
        ok = ok && wwait(bars + 1, parity, a.err, abort);
        fence_after();
        if (warp < kSumWarps && ok) {
            const float sw = e < 0 ? __ldg(a.ssa + (int64_t)U.f * a.SB + c)
                                   : __ldg(a.swa + ((int64_t)e * w.FT + U.f) * a.IB + c);
#pragma unroll
            for (int ch = 0; ch < NT / 16; ++ch) {
                uint32_t r[16];
                tmem_ld16(tmem + ((uint32_t)warp << 21) + ch * 16, r);
                tmem_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int n = ch * 16 + j;
                    const float x = n < U.n ? a.hs[(int64_t)B.item * NT + n] : __uint_as_float(kNotChosen);
                    if (__float_as_uint(x) != kNotChosen)
                        acc[n] = fmaf(tmem_value(r[j]), x * sw + 0.0f, acc[n]);
                }
            }
        }
        fence_before();
        parity ^= 1;
        if (!__syncthreads_and(ok))
            return parity;
        fence_after();
    }
    if (a.cl > 1) {
        if (warp < kSumWarps)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                stage[n * 128 + row] = acc[n];
        return parity;
    }
#pragma unroll
    for (int ps = 0; ps < NT / GC; ++ps) {
        if (ps * GC >= U.n)
            break;
        if (warp < kSumWarps)
#pragma unroll
            for (int j = 0; j < GC; ++j)
                stage[j * 128 + row] = acc[ps * GC + j];
        __syncthreads();
        if (warp < kSumWarps)
            for (int j = warp; j < GC && ps * GC + j < U.n; j += 4) {
                const float4 v[1] = {reinterpret_cast<const float4 *>(stage + j * 128)[lane]};
                emit<kFewDown, NT>(a, w, U, ps * GC + j, v, lane);
            }
        __syncthreads();
    }
    return parity;
}

template <int MODE, int NT>
__global__ void __launch_bounds__(kThreads, per_sm(MODE, NT)) gemm_kernel(const __grid_constant__ GemmArgs a)
{
    constexpr int NMAT = n_mats(MODE), EW = kSumWarps, NB = n_acc(MODE, NT), NCH = NT / 16;
    constexpr uint32_t kStage = stage_bytes(MODE, NT), kCols = NMAT * NT, kTmem = tmem_cols(MODE, NT);
    constexpr bool FEW = MODE == kFewGateUp || MODE == kFewDown;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // (the same offset in every CTA of the cluster: remote addresses rely on it)
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const int NS = a.stages, cl = a.cl;
    uint8_t *tail = ring + NS * kStage;
    constexpr Tail T = tail_of(MODE, NT);
    constexpr int GC = pass_cols(MODE, NT);
    float *stage = reinterpret_cast<float *>(cl > 1 ? ring : tail + T.stage);
    float *fac = reinterpret_cast<float *>(tail + T.fac);
    int *tab = reinterpret_cast<int *>(tail + T.tab);
    uint64_t *full = reinterpret_cast<uint64_t *>(tail + T.bars), *empty = full + 16;
    uint64_t *tfull = empty + 16, *tempty = tfull + 4, *ffull = tempty + 4, *fempty = ffull + kFacRing;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(fempty + kFacRing);
    volatile int *abort = reinterpret_cast<volatile int *>(tslot + 1);
    volatile uint64_t *redo = reinterpret_cast<volatile uint64_t *>(tslot + 2);  // kFewDown: units to do again
    uint32_t *any_redo = tslot + 4;                                              // some of the cluster's
    volatile int *sh0 = reinterpret_cast<volatile int *>(tslot + 5);             // Walk::sh0
    uint64_t *rbars = reinterpret_cast<uint64_t *>(tslot + 6);                   // and the barriers of that
    const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
    const uint32_t rank = cl > 1 ? cluster_rank() : 0;

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
        if (MODE == kFewDown)
            for (int i = 0; i < 3; ++i)
                mbar_init(rbars + i, 1);
        *redo = 0;
        *any_redo = 0;
        if (MODE == kFewDown)
            *sh0 = first_block(a, a.E, rank);
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
        int *act = tab, *idx = tab + kMaxExperts + kMaxExperts / 32;
        float *wts = reinterpret_cast<float *>(idx + NT * kMaxTopK);
        if (tid < kMaxExperts / 32)
            mask[tid] = 0;
        __syncthreads();
        for (int s = tid; s < a.T * a.topk; s += kThreads) {
            const int e = __ldg(a.idx + s);
            if (MODE == kFewGateUp) {
                idx[s] = e;
                wts[s] = __ldg(a.wts + s);
            }
            if (e >= 0 && e < a.E)
                atomicOr(mask + (e >> 5), 1u << (e & 31));
        }
        __syncthreads();
        int n = 0;
        for (int i = 0; i < kMaxExperts / 32; ++i)
            n += __popc(mask[i]);
        auto place = [&](const uint32_t *bits, int e) {  // of expert e among those with a bit
            int at = __popc(bits[e >> 5] & ((1u << (e & 31)) - 1));
            for (int i = 0; i < e >> 5; ++i)
                at += __popc(bits[i]);
            return at;
        };
        if (MODE == kFewGateUp) {
            for (int e = tid; e < a.E; e += kThreads)
                if (mask[e >> 5] >> (e & 31) & 1)
                    act[place(mask, e)] = e;
        } else {
            // of an expert's IB blocks this rank has q, or q + 1 where its first one is below IB - q cl
            const int q = div_cl(a, a.IB), more = a.IB - q * cl;
            uint32_t *extra = mask + kMaxExperts / 32, *list = extra + kMaxExperts / 32;
            for (int i = warp; i < kMaxExperts / 32; i += kThreads / 32) {
                const uint32_t v = __ballot_sync(0xFFFFFFFFu, first_block(a, i * 32 + lane, rank) < more);
                if (lane == 0)
                    extra[i] = v & mask[i];
            }
            __syncthreads();
            for (int e = tid; e < a.E; e += kThreads)
                if (mask[e >> 5] >> (e & 31) & 1) {
                    const int at = place(mask, e), before = place(extra, e);
                    int c = first_block(a, e, rank), to = q * at + before;
                    act[at] = e | before << 16;
                    for (; c < a.IB && to < list_room(NT); c += cl)
                        list[to++] = list_entry(e, at, c);
                }
            w.n_routed = q * n;
            for (int i = 0; i < kMaxExperts / 32; ++i)
                w.n_routed += __popc(extra[i]);
            w.rank = rank;
            w.list = list;
        }
        w.n_act = n;
        w.act = act;
        w.idx = idx;
        w.wts = wts;
        w.n_units = MODE == kFewGateUp ? n * a.IB + a.SB : w.FT;
    } else {
        int *tt = tab, *lo = tab + kMaxExperts + 1, *len = lo + kMaxExperts;
        if (warp == 0)
            group_table(a.offsets, a.E, a.rows, NT, lane, tt, lo, len);
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
    if (MODE == kFewDown) {
        // (by way of shared memory: known to be the same in all threads, it made 64 tokens of top-8 of 256
        // experts take 485 us instead of 462)
        w.sh0 = *sh0;
        w.kb1 = w.n_routed + (w.sh0 < a.SB ? div_cl(a, a.SB - w.sh0 + cl - 1) : 0);
    } else {
        w.kb0 = KB * rank / cl;
        w.kb1 = KB * (rank + 1) / cl;
    }
    const uint32_t tmem = *tslot;

    if (warp == EW) {
        // ------------------------------------------------------ TMA producer
        {
            // (the whole warp walks the loop and one elected lane issues: behind `lane == 0` the
            // compiler issues each copy, or MMA, in a loop over lanes)
            auto weights = [&](const Unit &U, int kb, int s) {
                uint8_t *st = ring + s * kStage;
                const Block B = block_of<MODE, NT>(a, w, U, kb);
                const bool sh = FEW && B.e < 0;
                tma_3d(st, sh ? &a.sa : &a.wa, B.c * kBlk, U.f * kBlk, sh ? 0 : B.e, full + s);
                if (NMAT == 2)
                    tma_3d(st + kTile, sh ? &a.sb : &a.wb, B.c * kBlk, U.f * kBlk, sh ? 0 : B.e, full + s);
            };
            auto tokens = [&](const Unit &U, int kb, int s) {
                uint8_t *st = ring + s * kStage + NMAT * kTile;
                const Block B = block_of<MODE, NT>(a, w, U, kb);
                if (MODE == kFewDown)
                    tma_2d(st, &a.xm, 0, B.item * NT, full + s);
                else
                    tma_2d(st, &a.xm, B.c * kBlk, U.tok0, full + s);
            };
            constexpr uint32_t bytes = NMAT * kTile + NT * 128;
            int early = 0;  // stages whose weights were requested before the launch's inputs were complete
            if (FEW) {
                for (int u = w.first; u < w.n_units && early < NS; u += w.step) {
                    const Unit U = unit_of<MODE, NT>(a, w, u);
                    for (int kb = w.kb0; kb < w.kb1 && early < NS; ++kb, ++early) {
                        if (elect_one()) {
                            mbar_arrive_expect_tx(full + early, bytes);
                            weights(U, kb, early);
                        }
                        __syncwarp();
                    }
                }
                pdl_wait();
            }
            int it = 0, s = 0;
            uint32_t ph = 1;
            for (int u = w.first; u < w.n_units; u += w.step) {
                const Unit U = unit_of<MODE, NT>(a, w, u);
                for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    if (it >= early && !wwait(empty + s, ph, a.err, abort))
                        goto produced;
                    if (elect_one()) {
                        if (it >= early) {
                            mbar_arrive_expect_tx(full + s, bytes);
                            weights(U, kb, s);
                        }
                        tokens(U, kb, s);
                    }
                    __syncwarp();
                    if (++s == NS)
                        s = 0, ph ^= 1;
                }
            }
        }
    produced:;
    } else if (warp == EW + 1) {
        // --------------------------------------------------------------- MMA
        if (FEW)
            pdl_wait();  // (the launch before is not on this one's bounded waits' time)
        {
            int s = 0, b = 0;
            uint32_t ph = 0, tph = 1;
            for (int u = w.first; u < w.n_units; u += w.step) {
                const Unit U = unit_of<MODE, NT>(a, w, u);
                const uint32_t idesc = idesc_e4m3((U.n + 15) & ~15);
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!wwait(tempty + b, tph, a.err, abort) || !wwait(full + s, ph, a.err, abort))
                        goto issued;
                    fence_after();
                    const uint32_t st = smem_u32(ring + s * kStage);
                    const uint64_t xd = sw128_desc(st + NMAT * kTile);
#pragma unroll
                    for (int m = 0; m < NMAT; ++m)
                        umma_block(tmem + b * kCols + m * NT, sw128_desc(st + m * kTile), xd, idesc);
                    umma_commit2(empty + s, tfull + b);
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
        constexpr int NL = (NT + 31) / 32, BATCH = 4;
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
                        const Block B = block_of<MODE, NT>(a, w, U, kb);
                        const int e = B.e, c = B.c;
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
                                x[i][j] = MODE == kFewDown ? a.hs[(int64_t)B.item * NT + n]
                                                           : a.sx[(U.tok0 + n) * a.sx_r + c * a.sx_b];
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
        if (FEW)
            pdl_wait();
        const int row = warp * 32 + lane;
        const uint32_t ta = tmem + ((uint32_t)warp << 21);
        int b = 0, q = 0;
        uint32_t tph = 0, fph = 0;
        bool ok = true;
        for (int u = w.first, k = 0; u < w.n_units && ok; u += w.step, ++k) {
            const Unit U = unit_of<MODE, NT>(a, w, u);
            const int nch = (U.n + 15) / 16;
            uint64_t acc[NMAT][NT / 2];
#pragma unroll
            for (int m = 0; m < NMAT; ++m)
#pragma unroll
                for (int i = 0; i < NT / 2; ++i)
                    acc[m][i] = 0;
            // (a wait that gave up does not leave the loop early: the sums stay in place)
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                ok &= bwait(ffull + q, fph, a.err, abort);
                ok &= bwait(tfull + b, tph, a.err, abort);
                fence_after();
                const float4 *f = reinterpret_cast<const float4 *>(fac + q * NMAT * NT);
                const uint32_t tb = ta + b * kCols;
                // chunk by chunk, the next one's columns on their way while one is summed
                uint32_t r[2][16];
                tmem_ld16(tb, r[0]);
#pragma unroll
                for (int i = 0; i < NCH * NMAT; ++i) {
                    const int ch = i / NMAT, m = i % NMAT;
                    if (ch < nch) {
                        const int nx = i + 1;
                        tmem_wait();
                        if (nx < NCH * NMAT && nx / NMAT < nch)
                            tmem_ld16(tb + (nx % NMAT) * NT + nx / NMAT * 16, r[nx & 1]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 v = f[(m * NT + ch * 16) / 4 + j];
                            const uint32_t *p = r[i & 1] + 4 * j;
                            fma_after(acc[m][ch * 8 + 2 * j], p[0], p[1], pair_f32(v.x, v.y));
                            fma_after(acc[m][ch * 8 + 2 * j + 1], p[2], p[3], pair_f32(v.z, v.w));
                        }
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
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (MODE == kFewDown) {
                // a NaN in a row's weights, or an infinite scale of theirs, is in the sums of every
                // column; one of a token's own in that column alone
                float first, second;
                unpair_f32(acc[0][0], first, second);
                const bool good = __all_sync(0xFFFFFFFFu, U.n < 2 || fabsf(first) < INFINITY || fabsf(second) < INFINITY);
                if (cl > 1) {
                    if (!good) {
                        *redo = 1;
                        if (lane < cl)
                            asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(mapa(smem_u32(any_redo), lane))
                                         : "memory");
                    }
                } else if (!named_and(1, 128, good)) {
                    if (tid == 0)
                        *redo = *redo | 1ull << k;  // (54 units to a CTA at most)
                    __syncwarp();
                    ok = named_and(1, 128, ok);  // (the four warps give up together)
                    continue;
                }
            }

            // The sums leave in passes of GC columns through shared memory, where a
            // warp takes a whole column (128 rows, four to a lane): its stores are
            // contiguous, the largest |h| of a hidden block is one warp maximum, and
            // the code stays small -- unrolled over the registers it ran at the rate
            // of its instruction fetches (64 columns: 5 us for the stores alone).
            if (cl > 1) {  // one unit: the rest follows the cluster's barrier
#pragma unroll
                for (int m = 0; m < NMAT; ++m)
#pragma unroll
                    for (int j = 0; j < NT / 2; ++j) {
                        float lo, hi;
                        unpair_f32(acc[m][j], lo, hi);
                        stage[(m * NT + 2 * j) * 128 + row] = lo;
                        stage[(m * NT + 2 * j + 1) * 128 + row] = hi;
                    }
                break;
            }
#pragma unroll
            for (int ps = 0; ps < NT / GC; ++ps) {
                if (ps * GC >= U.n)
                    break;
#pragma unroll
                for (int m = 0; m < NMAT; ++m)
#pragma unroll
                    for (int j = 0; j < GC / 2; ++j) {
                        float lo, hi;
                        unpair_f32(acc[m][ps * GC / 2 + j], lo, hi);
                        stage[(m * GC + 2 * j) * 128 + row] = lo;
                        stage[(m * GC + 2 * j + 1) * 128 + row] = hi;
                    }
                // (the four warps give up together: none is left at a barrier)
                __syncwarp();
                ok = named_and(1, 128, ok);
                if (!ok)
                    break;
                for (int j = warp; j < GC && ps * GC + j < U.n; j += 4) {
                    float4 v[NMAT];
#pragma unroll
                    for (int m = 0; m < NMAT; ++m)
                        v[m] = reinterpret_cast<const float4 *>(stage + (m * GC + j) * 128)[lane];
                    emit<MODE, NT>(a, w, U, ps * GC + j, v, lane);
                }
                __syncwarp();
                ok = named_and(1, 128, ok);
                if (!ok)
                    break;
            }
        }
    }
    auto do_again = [&]() {
        if constexpr (MODE == kFewDown) {
            fence_after();
            const uint64_t todo = *abort ? 0 : *redo;
            uint32_t parity = 0;
            for (int u = w.first, k = 0; u < w.n_units && !*abort; u += w.step, ++k)
                if (todo >> k & 1)
                    parity = redo_down<NT>(a, u, w.kb1, w.n_routed, w.act, w.list, w.n_act, w.sh0, rank, ring, stage, rbars,
                                           parity, tmem, abort);
        }
    };
    if (MODE == kFewDown && cl == 1) {
        __syncthreads();
        if (*redo)
            do_again();
    }
    if (cl > 1) {
        __syncwarp();
        cluster_sync();
        if (MODE == kFewDown && *static_cast<volatile uint32_t *>(any_redo)) {  // (the same in the whole cluster)
            do_again();
            cluster_sync();
        }
        if (warp < kSumWarps && w.first < w.n_units && !*abort) {
            const Unit U = unit_of<MODE, NT>(a, w, w.first);
            // column n of the tile: CTA n % cl of the cluster, over all ranks in order
            for (int n = rank + cl * warp; n < U.n; n += cl * 4) {
                float4 v[NMAT];
#pragma unroll
                for (int m = 0; m < NMAT; ++m) {
                    const uint32_t at = smem_u32(stage + (m * NT + n) * 128 + 4 * lane);
                    v[m] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                    for (int r = 0; r < cl; ++r) {
                        const float4 p = ld_cluster(mapa(at, r));
                        v[m].x += p.x, v[m].y += p.y, v[m].z += p.z, v[m].w += p.w;
                    }
                }
                emit<MODE, NT>(a, w, U, n, v, lane);
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
    const size_t smem = gemm_smem((Mode)MODE, NT, a.stages);
    cudaError_t e = smem_optin((const void *)gemm_kernel<MODE, NT>, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(kThreads);
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

size_t gemm_smem(Mode mode, int nt, int stages)
{
    return 1024 + (size_t)stages * stage_bytes(mode, nt) + tail_of(mode, nt).total;
}

cudaError_t launch_gemm(Mode mode, int nt, const GemmArgs &a, int grid, cudaStream_t s)
{
#define MX_CASE(M, N)            \
    if (mode == M && nt == N)    \
        return launch_t<M, N>(a, grid, s)
    MX_CASE(kProduct, 16);
    MX_CASE(kProduct, 32);
    MX_CASE(kProduct, 64);
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
