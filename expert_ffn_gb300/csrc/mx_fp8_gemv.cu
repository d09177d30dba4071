// mx_fp8_gemv.cu -- the FP8 products for one to eight rows, and the MoE layer of
// one token in two launches.
//
// These read every weight once and do next to nothing with it, so what counts is
// that all SMs have loads in flight from the first moment to the last, and how
// long the chain before and behind them is.  A tile of 16 weight rows is one CTA
// (or several: no persistence, the scheduler evens them out); its warps split the
// inner dimension.  A lane loads 16-byte pieces of rows straight into the operand
// registers of mma.sync m16n8k32 (e4m3) -- in the layer by way of shared memory, where
// more of them can be under way: four lanes cover 64 consecutive bytes of
// a row, and since any order of k serves a dot product, the four words of a piece
// are used as they come, against the tokens' bytes in the same order.  No barrier or
// tensor memory stands between HBM and the MMA; through the tcgen05 kernel the 2112 x
// 2816 product of one row takes 5.8 us, most of it set-up, pipeline fill and cluster
// reduction, here 3.5.  The MMA's eight columns are the tokens.
//
// The layer, of one token: gate/up quantises its slice of x in each warp while the
// weights are under way, and leaves the hidden blocks in e4m3; down sums over all slots
// and the shared expert in a fixed order, so no scratch output and no third launch are
// needed.  Its first weights are requested before the gate/up launch has ended.  With 128
// experts, top-8, d_model 2816: 18.6 us for 65 MB, 3.5 TB/s.  Of them gate/up takes 11 (x
// quantised after 5, the sums done at 9, the cluster's largest |h| at 10 to 11.5), down's
// CTAs find room when gate/up's leave, and its 22 MB come in the 6.5 us after that.  Two
// tokens and more are faster by mx_fp8_gemm.cu (128 experts, top-8: 2 tokens 28 us and 44
// here, 8 tokens 61 and 316, where the same expert's blocks made long chains).
#include "mx_fp8.cuh"

#include <mutex>

namespace mx {
namespace fp8 {

namespace {

constexpr int kN = 8;  // MMA columns: tokens

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The bytes of v below `n` of 16 (n may be negative or above).
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int n)
{
    auto m = [n](uint32_t w, int at) {
        const int k = n - at;
        return k >= 4 ? w : k <= 0 ? 0u : w & ((1u << (8 * k)) - 1u);
    };
    return make_uint4(m(v.x, 0), m(v.y, 4), m(v.z, 8), m(v.w, 12));
}

// One matrix tile of 16 rows as a lane sees it: its two rows.
struct Rows2 {
    const uint8_t *r0, *r1;
};

__device__ __forceinline__ Rows2 rows_of(const uint8_t *w, int64_t ld, int row0, int n, int lane)
{
    const int g = row0 + (lane >> 2);
    return Rows2{w + (int64_t)min(g, n - 1) * ld, w + (int64_t)min(g + 8, n - 1) * ld};
}

// Block b (128 columns) of both rows: words 0-3 of each half of 64 columns.
struct Piece {
    uint4 a[2], c[2];
};

__device__ __forceinline__ Piece load_block(const Rows2 &r, int b, int cols, int lane)
{
    Piece p;
    const int o = b * kBlk + (lane & 3) * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int k = o + 64 * j;
        p.a[j] = p.c[j] = make_uint4(0, 0, 0, 0);
        if (k < cols) {  // (a row's last 16 bytes are its own: the pitch is a multiple of 16)
            p.a[j] = ld_stream_u4(r.r0 + k);
            p.c[j] = ld_stream_u4(r.r1 + k);
        }
    }
    return p;
}

// The same into four 16-byte places of shared memory, `gap` apart, asynchronously; a
// piece behind the last column is left out.
__device__ __forceinline__ void copy_block(uint8_t *to, int gap, const Rows2 &r, int b, int cols, int lane)
{
    const int o = b * kBlk + (lane & 3) * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (o + 64 * j < cols) {
            cp_async16(to + 2 * j * gap, r.r0 + o + 64 * j);
            cp_async16(to + (2 * j + 1) * gap, r.r1 + o + 64 * j);
        }
}

__device__ __forceinline__ Piece copied(const uint8_t *from, int gap)
{
    Piece p;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        p.a[j] = *reinterpret_cast<const uint4 *>(from + 2 * j * gap);
        p.c[j] = *reinterpret_cast<const uint4 *>(from + (2 * j + 1) * gap);
    }
    return p;
}

// What lies behind the last column is not the caller's data: make it zero.
__device__ __forceinline__ void trim(Piece &p, int b, int cols, int lane)
{
    if ((b + 1) * kBlk <= cols)
        return;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int n = cols - (b * kBlk + (lane & 3) * 16 + 64 * j);
        p.a[j] = keep_bytes(p.a[j], n);
        p.c[j] = keep_bytes(p.c[j], n);
    }
}

// acc += (block's product) * (sx of columns 2 tig, 2 tig + 1) * sw
__device__ __forceinline__ void add_block(float (&acc)[4], const Piece &p, const uint4 (&x)[2], float f0, float f1)
{
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        mma_e4m3(d, p.a[j].x, p.c[j].x, p.a[j].y, p.c[j].y, x[j].x, x[j].y);
        mma_e4m3(d, p.a[j].z, p.c[j].z, p.a[j].w, p.c[j].w, x[j].z, x[j].w);
    }
    acc[0] = fmaf(d[0], f0, acc[0]);
    acc[1] = fmaf(d[1], f1, acc[1]);
    acc[2] = fmaf(d[2], f0, acc[2]);
    acc[3] = fmaf(d[3], f1, acc[3]);
}

// A warp's sums [16 rows][8 tokens] to its place in `part`.
__device__ __forceinline__ void put_sums(float *part, const float (&acc)[4], int lane)
{
    const int g = lane >> 2, c = 2 * (lane & 3);
    *reinterpret_cast<float2 *>(part + g * kN + c) = make_float2(acc[0], acc[1]);
    *reinterpret_cast<float2 *>(part + (g + 8) * kN + c) = make_float2(acc[2], acc[3]);
}

// Quantise 128 values of a token (four to a lane) into `q`; every lane gets the scale.
__device__ __forceinline__ float quantize128(const float (&v)[4], uint8_t *q, int lane)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const uint64_t p[2] = {pair_f32(v[0], v[1]), pair_f32(v[2], v[3])};
    uint32_t e[2];
    const float s = quantize_pairs(p, __reduce_max_sync(0xFFFFFFFFu, m), 0, e);
    reinterpret_cast<uint32_t *>(q)[lane] = e[0] | e[1] << 16;
    return s;
}

// ------------------------------------------------------------------- product

constexpr int kMmWarps = 8, kMmBatch = 4;

__global__ void __launch_bounds__(kMmWarps * 32, 2) gemv_kernel(const GemvArgs a)
{
    __shared__ __align__(16) float part[kMmWarps][16 * kN];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = blockIdx.x * 16, KB = blocks(a.K);
    const Rows2 r = rows_of(a.w, a.ldw, row0, a.N, lane);
    const int b0 = KB * warp / kMmWarps, b1 = KB * (warp + 1) / kMmWarps;
    const float *sw = a.sw + (int64_t)(row0 / kBlk) * KB;
    const int n = min(lane >> 2, a.T - 1), c0 = min(2 * (lane & 3), a.T - 1), c1 = min(2 * (lane & 3) + 1, a.T - 1);
    const uint8_t *xr = a.q + n * a.ldq;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = b0; b < b1; b += kMmBatch) {
        Piece p[kMmBatch];
        uint4 x[kMmBatch][2];
        float f0[kMmBatch], f1[kMmBatch], s[kMmBatch];
#pragma unroll
        for (int i = 0; i < kMmBatch; ++i)
            if (b + i < b1)
                p[i] = load_block(r, b + i, a.K, lane);
#pragma unroll
        for (int i = 0; i < kMmBatch; ++i)
            if (b + i < b1) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = (b + i) * kBlk + (lane & 3) * 16 + 64 * j;
                    x[i][j] = k < a.K ? ldg_u4(xr + k) : make_uint4(0, 0, 0, 0);
                }
                s[i] = __ldg(sw + b + i);
                f0[i] = __ldg(a.sx + c0 * a.sx_r + (b + i) * a.sx_b);
                f1[i] = __ldg(a.sx + c1 * a.sx_r + (b + i) * a.sx_b);
            }
#pragma unroll
        for (int i = 0; i < kMmBatch; ++i)
            if (b + i < b1) {
                trim(p[i], b + i, a.K, lane);
                if ((b + i + 1) * kBlk > a.K)  // (nor are a row of x's last bytes)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        x[i][j] = keep_bytes(x[i][j], a.K - ((b + i) * kBlk + (lane & 3) * 16 + 64 * j));
                add_block(acc, p[i], x[i], f0[i] * s[i], f1[i] * s[i]);
            }
    }
    put_sums(part[warp], acc, lane);
    __syncthreads();
    const int t = threadIdx.x >> 4, o = threadIdx.x & 15;
    if (t < a.T && row0 + o < a.N) {
        float y = 0.0f;
#pragma unroll
        for (int k = 0; k < kMmWarps; ++k)
            y += part[k][o * kN + t];
        const int64_t at = t * a.ldo + row0 + o;
        if (a.out_bf16)
            reinterpret_cast<uint16_t *>(a.out)[at] = f2bf(y);
        else
            reinterpret_cast<float *>(a.out)[at] = y;
    }
}

// --------------------------------------------------------------------- layer

// Four neighbouring values of the token, as they lie in memory: nothing here
// waits for them.  A lane behind the last column reads the last four.
__device__ __forceinline__ uint4 load4(const void *p, int c, int n, int bf16)
{
    uint4 r = make_uint4(0, 0, 0, 0);
    if (n % 4 == 0) {
        const int k = min(c, n - 4);
        if (bf16) {
            const uint2 h = __ldg(reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + k));
            r.x = h.x, r.y = h.y;
        } else {
            r = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint32_t *>(p) + k));
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = min(c + i, n - 1);
            w[i] = bf16 ? __ldg(reinterpret_cast<const uint16_t *>(p) + k) : __ldg(reinterpret_cast<const uint32_t *>(p) + k);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return r;
}

// Their numbers, zeros from column n on.
__device__ __forceinline__ void values4(const uint4 &r, int c, int n, int bf16, float (&v)[4])
{
    uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if (bf16) {
        const bool pairs = n % 4 == 0;
        w[3] = pairs ? r.y & 0xFFFF0000u : r.w << 16;
        w[2] = pairs ? r.y << 16 : r.z << 16;
        w[1] = pairs ? r.x & 0xFFFF0000u : r.y << 16;
        w[0] = r.x << 16;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = c + i < n ? __uint_as_float(w[i]) : 0.0f;
}

constexpr int kGuWarps = 4, kGuDepth = 3, kGuX = 6, kGuCluster = kBlk / 16, kGuGap = kGuWarps * 32 * 16;
constexpr int kGuRing = kGuDepth * 8 * kGuGap;  // bytes: [kGuDepth][gate, up][4][thread] pieces under way

// Hidden blocks: h8[block][128] in e4m3 and their factors (scale times routing weight);
// block = the shared expert's, then (slot, block): an expert may come twice, an index may
// be none of the experts.  A CTA has 16 hidden rows, gate and up; the eight CTAs of a
// block form a cluster and tell each other their largest |h|.  Weights go through shared
// memory asynchronously, each lane's pieces to its own places: in registers two blocks a
// warp could be under way, and the token's loads came behind them (the launch took 13.5 us
// and not 11).
__global__ void __launch_bounds__(kGuWarps * 32, 4) gemv_gate_up(const GemvArgs a)
{
    extern __shared__ __align__(16) uint8_t gu[];
    // a warp's sums, in its own first two places of the ring when all has been read
    auto part = [&](int w, int m) { return reinterpret_cast<float *>(gu + m * kGuGap + w * 512); };
    __shared__ float am[kGuCluster];
    pdl_trigger();
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // (this CTA runs: its memory may be written)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int KB = blocks(a.K), SB = blocks(a.S), IB = blocks(a.I);
    const int rank = blockIdx.x % kGuCluster, blk = blockIdx.x / kGuCluster;
    const int slot = blk < SB ? -1 : (blk - SB) / IB;
    const int e = slot < 0 ? -1 : __ldg(a.idx + slot);
    // the warp's slice of x: its first kGuX blocks' loads before those of weights
    const int b0 = KB * warp / kGuWarps, b1 = KB * (warp + 1) / kGuWarps, nx = b1 - b0;
    uint4 raw[kGuX];
    auto load_x = [&](int q) {
#pragma unroll
        for (int i = 0; i < kGuX; ++i)
            raw[i] = load4(a.x, (b0 + min(q + i, nx - 1)) * kBlk + 4 * lane, a.K, a.bf16);
    };
    if (nx > 0)
        load_x(0);
    int f = blk, rows = a.S;
    const uint8_t *wg = a.sw_gate, *wu = a.sw_up;
    const float *sg = a.ss_gate, *su = a.ss_up;
    int64_t lg = a.ld_sgate, lu = a.ld_sup;
    if (slot >= 0) {
        if (e < 0 || e >= a.E)
            return;
        f = blk - SB - slot * IB;
        rows = a.I;
        wg = a.w_gate + (int64_t)e * a.I * a.ld_gate;
        wu = a.w_up + (int64_t)e * a.I * a.ld_up;
        lg = a.ld_gate;
        lu = a.ld_up;
        sg = a.s_gate + (int64_t)e * IB * KB;
        su = a.s_up + (int64_t)e * IB * KB;
    }
    const int row0 = f * kBlk + rank * 16;
    sg += (int64_t)f * KB;
    su += (int64_t)f * KB;
    if (row0 < rows) {
        const Rows2 rg = rows_of(wg, lg, row0, rows, lane), ru = rows_of(wu, lu, row0, rows, lane);
        // behind the ring the slices of x, e4m3, and their scales
        const int slice = (KB + kGuWarps - 1) / kGuWarps;
        uint8_t *x = gu + kGuRing + warp * slice * kBlk;
        float *fx = reinterpret_cast<float *>(gu + kGuRing + kGuWarps * slice * kBlk) + warp * slice;
        float ag[4] = {0.0f, 0.0f, 0.0f, 0.0f}, au[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        // kGuDepth blocks of both matrices are under way at any time
        uint8_t *mine = gu + threadIdx.x * 16;
        float s0[kGuDepth], s1[kGuDepth];
        auto load = [&](int i, int b) {
            copy_block(mine + 8 * i * kGuGap, kGuGap, rg, b, a.K, lane);
            copy_block(mine + (8 * i + 4) * kGuGap, kGuGap, ru, b, a.K, lane);
            s0[i] = __ldg(sg + b);
            s1[i] = __ldg(su + b);
        };
#pragma unroll
        for (int i = 0; i < kGuDepth; ++i) {
            if (b0 + i < b1)
                load(i, b0 + i);
            cp_async_commit();
        }
        for (int q = 0; q < nx; q += kGuX) {
            if (q)
                load_x(q);
#pragma unroll
            for (int i = 0; i < kGuX; ++i)
                if (q + i < nx) {
                    float v[4];
                    values4(raw[i], (b0 + q + i) * kBlk + 4 * lane, a.K, a.bf16, v);
                    const float s = quantize128(v, x + (q + i) * kBlk, lane);
                    if (lane == 0)
                        fx[q + i] = s;
                }
        }
        __syncwarp();
        const uint8_t *xb = x + (lane & 3) * 16;  // (all eight columns of the MMA: the token)
        for (int b = b0; b < b1; b += kGuDepth)
#pragma unroll
            for (int i = 0; i < kGuDepth; ++i)
                if (b + i < b1) {
                    const uint4 xv[2] = {*reinterpret_cast<const uint4 *>(xb), *reinterpret_cast<const uint4 *>(xb + 64)};
                    const float fv = fx[b + i - b0];
                    xb += kBlk;
                    cp_async_wait<kGuDepth - 1>();
                    Piece pg = copied(mine + 8 * i * kGuGap, kGuGap), pu = copied(mine + (8 * i + 4) * kGuGap, kGuGap);
                    trim(pg, b + i, a.K, lane);
                    trim(pu, b + i, a.K, lane);
                    add_block(ag, pg, xv, fv * s0[i], fv * s0[i]);
                    add_block(au, pu, xv, fv * s1[i], fv * s1[i]);
                    if (b + i + kGuDepth < b1)
                        load(i, b + i + kGuDepth);
                    cp_async_commit();
                }
        __syncwarp();
        put_sums(part(warp, 0), ag, lane);
        put_sums(part(warp, 1), au, lane);
    }
    __syncthreads();
    const int r = threadIdx.x;  // the CTA's hidden row, of the first 16 threads
    float h = 0.0f;
    if (r < 16 && row0 + r < rows) {
        float g = 0.0f, v = 0.0f;
#pragma unroll
        for (int k = 0; k < kGuWarps; ++k) {
            g += part(k, 0)[r * kN];
            v += part(k, 1)[r * kN];
        }
        h = (a.act == MX_SILU ? __fdividef(g, 1.0f + __expf(-g)) : gelu_fast(g)) * v;
    }
    uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h) & 0x7FFFFFFFu);
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (r < kGuCluster) {
        uint32_t at;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&am[rank])), "r"(r));
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(m) : "memory");
    }
    // (the other CTAs' maxima come with the barrier; none writes here after it)
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (r >= 16)
        return;
    m = 0;
#pragma unroll
    for (int k = 0; k < kGuCluster; ++k)
        m = max(m, __float_as_uint(am[k]));
    const float s = scale_of(__uint_as_float(m), 0);
    const Quotient q(__uint_as_float(m), s);
    a.h8[(int64_t)blk * kBlk + rank * 16 + r] = (uint8_t)q.e4m3_of(h * q.m, 0.0f);
    if (rank == 0 && r == 0)  // (the routing weight joins the scale)
        a.hf[blk] = slot < 0 ? s : s * __ldg(a.wts + slot);
}

constexpr int kDnWarps = 8, kDnDepth = 6, kDnX = 3, kDnGap = kDnWarps * 32 * 16;

// 16 output columns: all hidden blocks of the shared expert and of the slots, split over
// the warps in order.
__global__ void __launch_bounds__(kDnWarps * 32, 2) gemv_down(const GemvArgs a)
{
    extern __shared__ __align__(16) uint8_t dn[];  // [kDnDepth][4][thread] pieces under way
    __shared__ __align__(16) float part[kDnWarps][16 * kN];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int IB = blocks(a.I), SB = blocks(a.S), DB = blocks(a.K);
    const int row0 = blockIdx.x * 16;
    const int items = SB + a.topk * IB;
    const int b0 = (int)((int64_t)items * warp / kDnWarps), b1 = (int)((int64_t)items * (warp + 1) / kDnWarps);
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    // the next item to request: its slot (-1: the shared expert), block and rows
    int lj = b0 < SB ? -1 : (b0 - SB) / IB, lc = b0 < SB ? b0 : (b0 - SB) - lj * IB;
    Rows2 lr;
    const float *ls;
    bool lok;
    auto locate = [&]() {
        const int e = lj < 0 ? 0 : lj < a.topk ? __ldg(a.idx + lj) : -1;
        lok = e >= 0 && (lj < 0 || e < a.E);
        if (!lok)
            return;
        lr = lj < 0 ? rows_of(a.sw_down, a.ld_sdown, row0, a.K, lane)
                    : rows_of(a.w_down + (int64_t)e * a.K * a.ld_down, a.ld_down, row0, a.K, lane);
        ls = lj < 0 ? a.ss_down + (int64_t)(row0 / kBlk) * SB : a.s_down + ((int64_t)e * DB + row0 / kBlk) * IB;
    };
    uint8_t *mine = dn + threadIdx.x * 16;
    float sw[kDnDepth];
    int left[kDnDepth];  // columns from the block's first to the matrix's last; 0: no expert
    auto load = [&](int i) {
        const int cols = lj < 0 ? a.S : a.I;
        left[i] = 0;
        if (lok) {
            left[i] = cols - lc * kBlk;
            copy_block(mine + 4 * i * kDnGap, kDnGap, lr, lc, cols, lane);
            sw[i] = __ldg(ls + lc);
        }
        if (++lc == (lj < 0 ? SB : IB)) {
            lc = 0;
            ++lj;
            locate();
        }
    };
    locate();
#pragma unroll
    for (int i = 0; i < kDnDepth; ++i) {
        if (b0 + i < b1)
            load(i);
        cp_async_commit();
    }
    const int o = threadIdx.x, at = row0 + o;
    const bool writes = o < 16 && at < a.K;
    const float res = writes && a.residual ? load_act(a.residual, at, a.bf16) : 0.0f;
    pdl_wait();  // the hidden blocks, behind the first requests for weights
    // (written by the launch before: not through the read-only path)
    const uint8_t *xb = a.h8 + (int64_t)b0 * kBlk + (lane & 3) * 16;
    const float *fb = a.hf + b0;
    uint4 x[kDnX][2];
    float f[kDnX];
    auto hidden = [&](int i, int item) {
        const int at = min(item, items - 1) - b0;  // (behind the warp's last: read, not used)
        x[i][0] = *reinterpret_cast<const uint4 *>(xb + (int64_t)at * kBlk);
        x[i][1] = *reinterpret_cast<const uint4 *>(xb + (int64_t)at * kBlk + 64);
        f[i] = fb[at];
    };
    if (b0 < b1)
#pragma unroll
        for (int i = 0; i < kDnX; ++i)
            hidden(i, b0 + i);
    for (int b = b0; b < b1; b += kDnDepth) {
#pragma unroll
        for (int i = 0; i < kDnDepth; ++i) {
            if (b + i < b1) {
                cp_async_wait<kDnDepth - 1>();
                if (left[i]) {
                    Piece p = copied(mine + 4 * i * kDnGap, kDnGap);
                    if (left[i] < kBlk) {  // what lies behind the last column is nobody's: neither operand's
                        const int at = (lane & 3) * 16;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            p.a[j] = keep_bytes(p.a[j], left[i] - at - 64 * j);
                            p.c[j] = keep_bytes(p.c[j], left[i] - at - 64 * j);
                            x[i % kDnX][j] = keep_bytes(x[i % kDnX][j], left[i] - at - 64 * j);
                        }
                    }
                    add_block(acc, p, x[i % kDnX], f[i % kDnX] * sw[i], f[i % kDnX] * sw[i]);
                }
                hidden(i % kDnX, b + i + kDnX);
                if (b + i + kDnDepth < b1)
                    load(i);
                cp_async_commit();
            }
        }
    }
    put_sums(part[warp], acc, lane);
    __syncthreads();
    if (writes) {
        float y = 0.0f;
#pragma unroll
        for (int k = 0; k < kDnWarps; ++k)
            y += part[k][o * kN];
        y = fmaf(a.lam, y, res);
        if (a.bf16)
            reinterpret_cast<uint16_t *>(a.out)[at] = f2bf(y);
        else
            reinterpret_cast<float *>(a.out)[at] = y;
    }
}

}  // namespace

cudaError_t launch_gemv(const GemvArgs &a, cudaStream_t s)
{
    gemv_kernel<<<(a.N + 15) / 16, kMmWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

namespace {

// Gate/up of one token: a cluster for each of n hidden blocks.
cudaError_t gate_up_config(int K, int n, cudaLaunchConfig_t &c, cudaLaunchAttribute &at)
{
    c = cudaLaunchConfig_t{};
    c.gridDim = dim3(n * kGuCluster);
    c.blockDim = dim3(kGuWarps * 32);
    c.dynamicSmemBytes = kGuRing + kGuWarps * ((blocks(K) + kGuWarps - 1) / kGuWarps) * (kBlk + 4);
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim = {kGuCluster, 1, 1};
    c.attrs = &at;
    c.numAttrs = 1;
    return smem_optin((const void *)gemv_gate_up, c.dynamicSmemBytes);
}

}  // namespace

int gemv_moe_blocks(int K)
{
    constexpr int kDevices = 64, kSlices = kGemvMoeCols / kBlk / kGuWarps + 1;
    static std::mutex mu;
    static int16_t cache[kDevices][kSlices] = {{0}};  // plus one
    const int slice = (blocks(K) + kGuWarps - 1) / kGuWarps;
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices || slice >= kSlices)
        return 0;
    std::lock_guard<std::mutex> g(mu);
    if (!cache[dev][slice]) {
        cudaLaunchConfig_t c;
        cudaLaunchAttribute at;
        if (gate_up_config(K, 1, c, at) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, gemv_gate_up, &c) != cudaSuccess)
            return 0;
        cache[dev][slice] = (int16_t)(n + 1);
    }
    return cache[dev][slice] - 1;
}

cudaError_t launch_gemv_moe(const GemvArgs &a, cudaStream_t s)
{
    cudaLaunchConfig_t c;
    cudaLaunchAttribute at;
    cudaError_t e = gate_up_config(a.K, blocks(a.S) + a.topk * blocks(a.I), c, at);
    if (e != cudaSuccess)
        return e;
    c.stream = s;
    if ((e = cudaLaunchKernelEx(&c, gemv_gate_up, a)) != cudaSuccess)
        return e;
    c.gridDim = dim3((a.K + 15) / 16);
    c.blockDim = dim3(kDnWarps * 32);
    c.dynamicSmemBytes = kDnDepth * 4 * kDnGap;
    if ((e = smem_optin((const void *)gemv_down, c.dynamicSmemBytes)) != cudaSuccess)
        return e;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&c, gemv_down, a);
}

}  // namespace fp8
}  // namespace mx
