// mx_fp8_api.cu -- the FP8 block-scaled entry points of include/mx_moe.h:
// argument validation (all of it on the host, before any CUDA call), the
// workspace plan, and the choice of tile, split and grid for each launch.
#include "mx_fp8.cuh"
#include "mx_host.h"

#include <algorithm>
#include <cmath>
#include <mutex>

using namespace mx;
using namespace mx::fp8;

namespace mx {

int num_sms()
{
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 148;
    std::lock_guard<std::mutex> g(mu);
    if (!cache[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 148;
        cache[dev] = n;
    }
    return cache[dev];
}

}  // namespace mx

namespace {

constexpr int kMaxCols = 1 << 20, kMaxRows = 1 << 28;
constexpr int kSmem = 227 * 1024;      // shared memory of a CTA alone on its SM
constexpr int kSmemHalf = 113 * 1024;  // of one of two

// ---------------------------------------------------------------- validation

mx_status check_matrix(const mx_fp8_matrix *m, const char *name)
{
    if (!m)
        return fail(MX_ERR_INVALID_ARG, "%s is NULL", name);
    if (!m->w || !m->scales)
        return fail(MX_ERR_INVALID_ARG, "%s has a NULL pointer", name);
    if (m->rows < 1 || m->cols < 1 || m->rows > kMaxCols || m->cols > kMaxCols)
        return fail(MX_ERR_UNSUPPORTED, "%s: shape [%d, %d] must be within [1, %d]", name, m->rows, m->cols, kMaxCols);
    if (m->count < 1 || m->count > kMaxExperts)
        return fail(MX_ERR_UNSUPPORTED, "%s: %d matrices, at most %d are supported", name, m->count, kMaxExperts);
    if (m->ld < m->cols)
        return fail(MX_ERR_INVALID_ARG, "%s: row pitch %lld is below its %d columns", name, (long long)m->ld, m->cols);
    if (m->ld > 4 * (int64_t)kMaxCols)
        return fail(MX_ERR_UNSUPPORTED, "%s: row pitch %lld is above %d", name, (long long)m->ld, 4 * kMaxCols);
    if (!aligned(m->w, 16) || m->ld % 16)
        return fail(MX_ERR_ALIGNMENT, "%s: address and row pitch must be multiples of 16 bytes", name);
    if (!aligned(m->scales, 4))
        return fail(MX_ERR_ALIGNMENT, "%s: scales must be 4-byte aligned", name);
    return MX_OK;
}

mx_status check_rows(const mx_fp8_rows *r, const char *name, bool operand)
{
    if (!r)
        return fail(MX_ERR_INVALID_ARG, "%s is NULL", name);
    if (r->rows < 0 || r->rows > kMaxRows)
        return fail(MX_ERR_INVALID_ARG, "%s: %d rows must be within [0, %d]", name, r->rows, kMaxRows);
    if (r->cols < 1 || r->cols > kMaxCols)
        return fail(MX_ERR_UNSUPPORTED, "%s: %d columns must be within [1, %d]", name, r->cols, kMaxCols);
    if (r->ld < r->cols)
        return fail(MX_ERR_INVALID_ARG, "%s: row pitch %lld is below its %d columns", name, (long long)r->ld, r->cols);
    if (r->ld > ((int64_t)1 << 36))
        return fail(MX_ERR_UNSUPPORTED, "%s: row pitch %lld is too large", name, (long long)r->ld);
    if (r->scale_row < 0 || r->scale_block < 0)
        return fail(MX_ERR_INVALID_ARG, "%s: negative scale strides", name);
    if (r->rows == 0)
        return MX_OK;
    if (!r->q || !r->scales)
        return fail(MX_ERR_INVALID_ARG, "%s has a NULL pointer", name);
    if (operand && (!aligned(r->q, 16) || r->ld % 16))
        return fail(MX_ERR_ALIGNMENT, "%s: address and row pitch must be multiples of 16 bytes", name);
    if (!aligned(r->scales, 4))
        return fail(MX_ERR_ALIGNMENT, "%s: scales must be 4-byte aligned", name);
    return MX_OK;
}

mx_status check_layer(const mx_fp8_layer *L)
{
    mx_status st;
    if (!L)
        return fail(MX_ERR_INVALID_ARG, "layer is NULL");
    if ((st = check_matrix(&L->gate, "gate")) != MX_OK || (st = check_matrix(&L->up, "up")) != MX_OK ||
        (st = check_matrix(&L->down, "down")) != MX_OK)
        return st;
    const int D = L->gate.cols, I = L->gate.rows, E = L->gate.count;
    if (L->up.rows != I || L->up.cols != D || L->up.count != E || L->down.rows != D || L->down.cols != I ||
        L->down.count != E)
        return fail(MX_ERR_INVALID_ARG, "up must be %d x [%d, %d] and down %d x [%d, %d]", E, I, D, E, D, I);
    if (L->shared_gate.w) {
        if ((st = check_matrix(&L->shared_gate, "shared_gate")) != MX_OK ||
            (st = check_matrix(&L->shared_up, "shared_up")) != MX_OK ||
            (st = check_matrix(&L->shared_down, "shared_down")) != MX_OK)
            return st;
        const int S = L->shared_gate.rows;
        if (L->shared_gate.cols != D || L->shared_gate.count != 1 || L->shared_up.rows != S ||
            L->shared_up.cols != D || L->shared_up.count != 1 || L->shared_down.rows != D ||
            L->shared_down.cols != S || L->shared_down.count != 1)
            return fail(MX_ERR_INVALID_ARG, "the shared expert must be [%d, %d], [%d, %d] and [%d, %d]", S, D, S, D, D,
                        S);
    }
    if (L->top_k < 1 || L->top_k > kMaxTopK)
        return fail(MX_ERR_INVALID_ARG, "top_k %d must be in [1, %d]", L->top_k, kMaxTopK);
    if ((st = check_dtype(L->act_dtype, "act_dtype")) != MX_OK)
        return st;
    if (L->activation != MX_GELU_TANH && L->activation != MX_SILU)
        return fail(MX_ERR_INVALID_ARG, "activation %d is not MX_GELU_TANH or MX_SILU", L->activation);
    return MX_OK;
}

// -------------------------------------------------------------- launch choice

// Ring depth that fits `bytes` of shared memory, at most `want`.
int fit_stages(Mode mode, int nt, int bytes, int want)
{
    int s = std::min(want, 16);
    while (s > 2 && gemm_smem(mode, nt, s) > (size_t)bytes)
        --s;
    return s;
}

// Token tile for `n` rows: the smallest that holds them.
int tile_for(int n, int most)
{
    int nt = 16;
    while (nt < most && nt < n)
        nt *= 2;
    return nt;
}

mx_status weight_map(CUtensorMap *m, const mx_fp8_matrix &w)
{
    const cudaError_t e =
        tma_map_bytes(m, w.w, TmaBytes{(uint64_t)w.cols, (uint64_t)w.rows, (uint64_t)w.count, (uint64_t)w.ld, 128});
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "tensor map of a weight");
}

mx_status rows_map(CUtensorMap *m, const void *q, int64_t rows, int64_t cols, int64_t ld, int box)
{
    const cudaError_t e =
        tma_map_bytes(m, q, TmaBytes{(uint64_t)cols, (uint64_t)rows, 0, (uint64_t)ld, (uint32_t)box});
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "tensor map of the activations");
}

// CTAs that share the `items` inner blocks of each of `units` units, out of `ctas` that
// run at once; they form a cluster.  More than `most` gain nothing over whole clusters
// left waiting (clusters of eight with an SM to a CTA: a GPC holds one or two).
int split_of(int64_t units, double items, int ctas, int most)
{
    const int64_t n = std::min<int64_t>(units <= 8 ? 8 : most, ctas / units);
    return items < 8 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(n, (int64_t)(items / 2)));
}

// (Times here and below are device times of calls in a graph that take three sets of inputs in
// turn; what is below 40 MB stays in the L2 cache.)

// Rows of a group from which on the tokens take the MMA's M side (mx_fp8_rows.cu).
// The two sides' times cross there: 128 matrices [2112, 2816] with a quarter, one, eight
// and 24 rows each 33 | 72 | 119 | 126 us on the N side and 33 | 76 | 119 | 123 on the M
// side, and when a few matrices have most of the rows 24 | 55 | 120 | 139 and 27 | 60 |
// 112 | 129.  Four rows to a matrix: evenly 158 us (N) and 163 (M) for 256 matrices [1024,
// 4096], all of them to one 33 and 19; two rows: 139 and 143, 20 and 19.
constexpr double kManyRows = 3.0;

// One matrix: the N side up to a tile of 64 rows, and for more as long as clusters can
// split its units: 128 x 2112 x 2816 in four 8.0 us (M side 9.9), 256 x 1024 x 4096 in four
// 8.7 (12.1), 128 x 4096 x 14336 in two 25.7 (38.4); but 192 x 2112 x 2816 in two 11.0 (9.9).
bool many_rows(int rows, const mx_fp8_matrix &w)
{
    const int KB = blocks(w.cols);
    const int cl = split_of((int64_t)((rows + 63) / 64) * blocks(w.rows), KB, num_sms(), 4);
    return rows > 64 && cl < (KB >= 32 ? 2 : 3);
}

// One launch of one or two products by mx_fp8_rows.cu; p[i].xm is encoded here from
// its rows at q[i].
mx_status run_rows(Mode mode, RowsArgs &g, const void *const *q, const int64_t *ldq, const double *avg, cudaStream_t s)
{
    const int sms = num_sms();
    mx_status st;
    double wide = 0;  // tiles of 128 x 256
    for (int i = 0; i < 2; ++i) {
        RowsProblem &p = g.p[i];
        if (p.rows == 0)
            continue;
        // (a group that is expected to have `avg` rows)
        const double tiles = !p.offsets ? (p.rows + 127) / 128 : p.E * (avg[i] <= 100 ? 1.0 : avg[i] / 128 + 0.5);
        wide += tiles * (mode == kGateUp ? blocks(p.N) : (p.N + 255) / 256);
        if ((st = rows_map(&p.xm, q[i], p.rows, p.K, ldq[i], kRowsBox)) != MX_OK)
            return st;
    }
    // Narrower tiles while each finds an SM of its own: 256 x 4096 x 4096, 64 of them, 12.8 us
    // and by wide ones 16.7; 600 rows, 160 or 80, 21.5 and 17.9.  (A factor for each 64 columns
    // wants a thread to have them.)
    const int bn = mode == kGateUp || g.p[0].out_kind == kOutF16 || 2 * wide > sms ? 256 : 128;
    const cudaError_t e = launch_rows(mode, bn, g, sms, s);
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "FP8 product");
}

// One product launch by mx_fp8_gemm.cu over rows grouped by matrix (offsets NULL: one
// group).  Tokens take the MMA's N side, in a tile that holds them, of 64 at most; groups,
// of kManyRows on average at most, in tiles of 16.
mx_status run_product(GemmArgs &g, const void *q, int64_t ldq, cudaStream_t s)
{
    const int sms = num_sms(), FT = blocks(g.N), KB = blocks(g.K);
    const int nt = g.offsets ? 16 : tile_for(g.rows, 64);
    const int64_t tiles = g.offsets ? g.E : (g.rows + nt - 1) / nt;
    mx_status st;
    // (64 x 4096 x 4096: 15.5 us whole, 12.5 in two, 9.5 in four or more; 64 x 704 x 2816
    // 12.8, 7.9 in four, 6.9 in eight)
    g.cl = g.offsets ? 1 : split_of(tiles * FT, KB, sms, 4);
    g.stages = fit_stages(kProduct, nt, kSmem, std::max(2, KB));
    if ((st = rows_map(&g.xm, q, g.rows, g.K, ldq, nt)) != MX_OK)
        return st;
    const int64_t units = g.offsets ? ((int64_t)g.rows / nt + g.E) * FT : tiles * FT;
    const cudaError_t e = launch_gemm(kProduct, nt, g, (int)std::min<int64_t>(sms / g.cl, units) * g.cl, s);
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "FP8 product");
}

mx_status product(const mx_fp8_rows *x, const int32_t *offsets, const mx_fp8_matrix *w, void *out, int64_t ldo,
                  int out_dtype, void *stream, void *ws, size_t ws_bytes)
{
    mx_status st;
    if ((st = check_rows(x, "x", true)) != MX_OK || (st = check_matrix(w, "w")) != MX_OK ||
        (st = check_dtype(out_dtype, "out_dtype")) != MX_OK)
        return st;
    if (x->cols != w->cols)
        return fail(MX_ERR_INVALID_ARG, "x has %d columns, w has %d", x->cols, w->cols);
    if (ldo < w->rows)
        return fail(MX_ERR_INVALID_ARG, "output row pitch %lld is below its %d columns", (long long)ldo, w->rows);
    if (x->rows == 0)
        return MX_OK;
    if (!out)
        return fail(MX_ERR_INVALID_ARG, "out is NULL");
    if (!aligned(out, out_dtype == MX_BF16 ? 2 : 4))
        return fail(MX_ERR_ALIGNMENT, "out is misaligned");
    if ((st = check_ws(ws, ws_bytes, kErrBytes)) != MX_OK)
        return st;
    // Weights straight into registers while they are few: one and eight rows by 2112 x 2816
    // take 3.6, 3.9 us (the tcgen05 kernel 5.8, 5.9), by 4096 x 4096 6.4, 6.9 (6.9, 7.4), by
    // 14336 x 4096 17.8, 19.1 (13.7, 13.9).
    if (!offsets && x->rows <= kGemvRows && (int64_t)w->rows * w->cols <= 1 << 25) {
        GemvArgs v{};
        v.T = x->rows;
        v.K = w->cols;
        v.N = w->rows;
        v.q = static_cast<const uint8_t *>(x->q);
        v.ldq = x->ld;
        v.sx = x->scales;
        v.sx_r = x->scale_row;
        v.sx_b = x->scale_block;
        v.w = static_cast<const uint8_t *>(w->w);
        v.ldw = w->ld;
        v.sw = w->scales;
        v.out = out;
        v.ldo = ldo;
        v.out_bf16 = out_dtype == MX_BF16;
        const cudaError_t e = launch_gemv(v, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? MX_OK : cuda_fail(e, "FP8 product");
    }
    const double avg = offsets ? (double)x->rows / w->count : x->rows;
    if (offsets ? avg > kManyRows : many_rows(x->rows, *w)) {
        RowsArgs r{};
        RowsProblem &p = r.p[0];
        p.rows = x->rows;
        p.K = w->cols;
        p.N = w->rows;
        p.E = w->count;
        p.offsets = offsets;
        p.sx = x->scales;
        p.sx_r = x->scale_row;
        p.sx_b = x->scale_block;
        p.swa = w->scales;
        p.out = out;
        p.ldo = ldo;
        p.out_kind = out_dtype == MX_BF16 ? kOutBf16 : kOutF32;
        p.out_vec = vec16(out, ldo, out_dtype == MX_BF16);
        r.err = static_cast<unsigned *>(ws);
        if ((st = weight_map(&p.wa, *w)) != MX_OK)
            return st;
        const void *q[1] = {x->q};
        return run_rows(kProduct, r, q, &x->ld, &avg, static_cast<cudaStream_t>(stream));
    }
    GemmArgs g{};
    g.rows = x->rows;
    g.K = w->cols;
    g.N = w->rows;
    g.E = w->count;
    g.offsets = offsets;
    g.sx = x->scales;
    g.sx_r = x->scale_row;
    g.sx_b = x->scale_block;
    g.swa = w->scales;
    g.out = out;
    g.ldo = ldo;
    g.out_kind = out_dtype == MX_BF16 ? kOutBf16 : kOutF32;
    g.out_vec = vec16(out, ldo, out_dtype == MX_BF16);
    g.err = static_cast<unsigned *>(ws);
    if ((st = weight_map(&g.wa, *w)) != MX_OK)
        return st;
    return run_product(g, x->q, x->ld, static_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------------ the layer

struct Plan {
    // all paths: e4m3 activations and their scales [blocks(D)][T]
    size_t xq, sx;
    // up to kFewTokens tokens: hidden tiles [item][nt][128] and factors [item][nt]
    size_t h, hs;
    size_t h8, hf;  // one token: the same for the two-launch form, by slot
    int nt, items;
    // more: grouping, gathered rows, hidden rows, per-slot outputs
    size_t counts, cursor, offsets, pos, xr, sr, hr, hrs, hsh, hshs, y, ys, yf, ysf;
    size_t total;
};

Plan make_plan(const mx_fp8_layer *L, int T)
{
    const int64_t D = L->gate.cols, I = L->gate.rows, E = L->gate.count, K = L->top_k;
    const int64_t S = L->shared_gate.w ? L->shared_gate.rows : 0;
    const int64_t IB = blocks((int)I), SB = blocks((int)S), DB = blocks((int)D), n = T * K;
    Plan p{};
    size_t o = kErrBytes;
    auto take = [&](int64_t bytes) {
        const size_t at = o;
        o += up256((size_t)bytes);
        return at;
    };
    p.xq = take(T * up16(D));
    p.sx = take(DB * T * 4);
    if (T <= kFewTokens) {
        p.nt = tile_for(T, kFewTokens);
        p.items = (int)(std::min(n, E) * IB + SB);
        p.h = take((int64_t)p.items * p.nt * kBlk);
        p.hs = take((int64_t)p.items * p.nt * 4);
        const int64_t slots = T == 1 ? K * IB + SB : 0;
        p.h8 = take(slots * kBlk);
        p.hf = take(slots * 4);
    } else {
        p.counts = take(2 * E * 4);
        p.cursor = p.counts + E * 4;
        p.offsets = take((E + 1) * 4);
        p.pos = take(n * 4);
        p.xr = take(n * up16(D));
        p.sr = take(DB * n * 4);
        p.hr = take(n * IB * kBlk);
        p.hrs = take(IB * n * 4);
        p.hsh = take(T * SB * kBlk);
        p.hshs = take(SB * T * 4);
        // (FP16 with a factor for each 64 columns under a bf16 result, else fp32)
        const int es = L->act_dtype == MX_BF16 ? 2 : 4;
        p.y = take(n * D * es);
        p.ys = take(S ? T * D * es : 0);
        p.yf = take(es == 2 ? n * ((D + 63) / 64) * 4 : 0);
        p.ysf = take(es == 2 && S ? T * ((D + 63) / 64) * 4 : 0);
    }
    p.total = o;
    return p;
}

void matrices(GemmArgs &g, const mx_fp8_matrix &a, const mx_fp8_matrix *b)
{
    g.K = a.cols;
    g.N = a.rows;
    g.E = a.count;
    g.swa = a.scales;
    g.swb = b ? b->scales : nullptr;
}

// One token by two launches (mx_fp8_gemv.cu), when all hidden blocks are worked on at one time
// (four CTAs to an SM up to d_model 7680, then three, two from 15 K on), and while each CTA's
// own quantisation of the token is short: d_model 2816, 65 blocks, take 18.6 us and by the
// few-token form 21.7, 4096 and 72 blocks 25.2 and 28.1, 5120 and 72 32.2 and 32.3, 76 39.0 and
// 33.2; 7168, 40 blocks 30.8 and 31.8, 56 38.5 and 35.7; 16384, 32 blocks 47.6 and 55.7, 40
// 60.9 and 59.2, 56 87 and 69; 32768, 32 blocks 88.9 and 99.9, 40 137 and 104.  256 experts of
// 1024 with a shared one of 4096, d_model 4096, are 96 blocks, 32.5 and 32.8.
bool one_token(const mx_fp8_layer *L, int T)
{
    const int64_t D = L->gate.cols;
    const int64_t n = L->top_k * (int64_t)blocks(L->gate.rows) + (L->shared_gate.w ? blocks(L->shared_gate.rows) : 0);
    return T == 1 && D <= kGemvMoeCols && n <= (D <= 5120 ? 76 : 40) && n <= gemv_moe_blocks((int)D);
}

mx_status run_gemv(const void *x, const int32_t *idx, const float *wts, const mx_fp8_layer *L,
                   const void *residual, void *out, cudaStream_t s, uint8_t *ws)
{
    auto bytes = [](const mx_fp8_matrix &m) { return static_cast<const uint8_t *>(m.w); };
    GemvArgs v{};
    v.T = 1;
    v.K = L->gate.cols;
    v.x = x;
    v.bf16 = L->act_dtype == MX_BF16;
    v.act = L->activation;
    v.topk = L->top_k;
    v.E = L->gate.count;
    v.I = L->gate.rows;
    v.idx = idx;
    v.wts = wts;
    v.w_gate = bytes(L->gate), v.w_up = bytes(L->up), v.w_down = bytes(L->down);
    v.ld_gate = L->gate.ld, v.ld_up = L->up.ld, v.ld_down = L->down.ld;
    v.s_gate = L->gate.scales, v.s_up = L->up.scales, v.s_down = L->down.scales;
    if (L->shared_gate.w) {
        v.S = L->shared_gate.rows;
        v.sw_gate = bytes(L->shared_gate), v.sw_up = bytes(L->shared_up), v.sw_down = bytes(L->shared_down);
        v.ld_sgate = L->shared_gate.ld, v.ld_sup = L->shared_up.ld, v.ld_sdown = L->shared_down.ld;
        v.ss_gate = L->shared_gate.scales, v.ss_up = L->shared_up.scales, v.ss_down = L->shared_down.scales;
    }
    const Plan p = make_plan(L, 1);
    v.h8 = ws + p.h8;
    v.hf = reinterpret_cast<float *>(ws + p.hf);
    v.out = out;
    v.residual = residual;
    v.lam = L->layer_scalar;
    const cudaError_t e = launch_gemv_moe(v, s);
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "FP8 layer");
}

// Up to kFewTokens tokens: quantise, then gate/up and down over the active
// experts, each launched while its predecessor still runs so that its weights
// are on their way when its operand is ready.
mx_status run_few(const void *x, int T, const int32_t *idx, const float *wts, const mx_fp8_layer *L,
                  const void *residual, void *out, cudaStream_t s, uint8_t *ws)
{
    const Plan p = make_plan(L, T);
    const int D = L->gate.cols, I = L->gate.rows, E = L->gate.count, K = L->top_k, sms = num_sms();
    const bool shared = L->shared_gate.w != nullptr;
    const int IB = blocks(I), SB = shared ? blocks(L->shared_gate.rows) : 0;
    mx_status st;
    cudaError_t e;

    QuantArgs q{};
    q.x = x;
    q.rows = T;
    q.ldx = D;
    q.cols = D;
    q.bf16 = L->act_dtype == MX_BF16;
    q.q = ws + p.xq;
    q.ldq = up16(D);
    q.scales = reinterpret_cast<float *>(ws + p.sx);
    q.s_r = 1;
    q.s_b = T;
    q.pdl = 1;
    if ((e = launch_quantize(q, num_sms(), s)) != cudaSuccess)
        return cuda_fail(e, "FP8 quantisation");

    GemmArgs g{};
    matrices(g, L->gate, &L->up);
    g.rows = T;
    g.sx = q.scales;
    g.sx_r = 1;
    g.sx_b = T;
    g.h = ws + p.h;
    g.hs = reinterpret_cast<float *>(ws + p.hs);
    g.act = L->activation;
    g.idx = idx;
    g.wts = wts;
    g.T = T;
    g.topk = K;
    g.IB = IB;
    g.SB = SB;
    g.err = reinterpret_cast<unsigned *>(ws);
    g.pdl = 1;
    if ((st = weight_map(&g.wa, L->gate)) != MX_OK || (st = weight_map(&g.wb, L->up)) != MX_OK ||
        (st = rows_map(&g.xm, ws + p.xq, T, D, up16(D), p.nt)) != MX_OK)
        return st;
    if (shared) {
        g.ssa = L->shared_gate.scales;
        g.ssb = L->shared_up.scales;
        if ((st = weight_map(&g.sa, L->shared_gate)) != MX_OK || (st = weight_map(&g.sb, L->shared_up)) != MX_OK)
            return st;
    }
    // experts that T tokens are expected to select, each on its own draw of K
    const double active = E * (1.0 - std::pow(1.0 - std::min(1.0, (double)K / E), (double)T));
    const int DB = blocks(D);
    // (one CTA to an SM with all its memory for loads in flight)
    g.cl = 1;
    g.stages = fit_stages(kFewGateUp, p.nt, kSmem, 16);
    if ((e = launch_gemm(kFewGateUp, p.nt, g, std::max(1, std::min(sms, p.items)), s)) != cudaSuccess)
        return cuda_fail(e, "FP8 gate/up");

    GemmArgs d = g;
    matrices(d, L->down, nullptr);
    d.out = out;
    d.ldo = D;
    d.out_kind = L->act_dtype == MX_BF16 ? kOutBf16 : kOutF32;
    d.out_vec = vec16(out, D, L->act_dtype == MX_BF16);
    d.residual = residual;
    d.lam = L->layer_scalar;
    d.pdl = 0;
    if ((st = weight_map(&d.wa, L->down)) != MX_OK ||
        (st = rows_map(&d.xm, ws + p.h, (int64_t)p.items * p.nt, kBlk, kBlk, p.nt)) != MX_OK)
        return st;
    if (shared) {
        d.ssa = L->shared_down.scales;
        if ((st = weight_map(&d.sa, L->shared_down)) != MX_OK)
            return st;
    }
    const double items = active * IB + SB;
    // Two CTAs to an SM take more blocks than SMs: 8, 31 tokens of top-8 of 128 experts
    // (d_model 2816, 22 units) in four 73, 143 us for the layer, in six 63, 123, in eight 61,
    // 115; 256 experts with d_model 4096 (32 units, six at most) in four 126, 338, in six 122,
    // 313.  A tile of 64 tokens wants an SM: 64 tokens in three 192 us, in four 170, in six 151.
    const bool two = p.nt <= 32;
    d.cl = two ? split_of(DB, items, sms * 4 / 3, 8) : split_of(DB, items, sms, 6);
    d.cl_inv = d.cl > 1 ? (unsigned)(((1ull << 32) + d.cl - 1) / d.cl) : 0;
    d.stages = fit_stages(kFewDown, p.nt, two ? kSmemHalf : kSmem, 16);
    const int grid = d.cl > 1 ? DB * d.cl : std::min(two ? 2 * sms : sms, DB);
    if ((e = launch_gemm(kFewDown, p.nt, d, grid, s)) != cudaSuccess)
        return cuda_fail(e, "FP8 down");
    return MX_OK;
}

mx_status run_many(const void *x, int T, const int32_t *idx, const float *wts, const mx_fp8_layer *L,
                   const void *residual, void *out, cudaStream_t s, uint8_t *ws)
{
    const Plan p = make_plan(L, T);
    const int D = L->gate.cols, I = L->gate.rows, E = L->gate.count, K = L->top_k, n = T * K;
    const bool shared = L->shared_gate.w != nullptr;
    const int IB = blocks(I), S = shared ? L->shared_gate.rows : 0, SB = blocks(S);
    auto f32 = [&](size_t o) { return reinterpret_cast<float *>(ws + o); };
    auto i32 = [&](size_t o) { return reinterpret_cast<int32_t *>(ws + o); };
    mx_status st;
    cudaError_t e;

    if ((e = launch_group(idx, n, E, i32(p.counts), i32(p.cursor), i32(p.offsets), i32(p.pos), s)) != cudaSuccess)
        return cuda_fail(e, "grouping");
    QuantArgs q{};
    q.x = x;
    q.rows = T;
    q.ldx = D;
    q.cols = D;
    q.bf16 = L->act_dtype == MX_BF16;
    q.q = shared ? ws + p.xq : nullptr;
    q.ldq = up16(D);
    q.scales = f32(p.sx);
    q.s_r = 1;
    q.s_b = T;
    q.pos = i32(p.pos);
    q.topk = K;
    q.qr = ws + p.xr;
    q.sr = f32(p.sr);
    q.sr_b = n;
    if ((e = launch_quantize(q, num_sms(), s)) != cudaSuccess)
        return cuda_fail(e, "FP8 quantisation");

    // The routed and the shared expert's products in one launch each, tokens on the M side
    // whatever their number to an expert: 100 tokens of top-8 of 128 experts 175 us, on the
    // N side and the shared expert by itself 179; when a few experts have most of them 87 and 117.
    const double avg[2] = {(double)n / E, (double)T};
    const bool half = L->act_dtype == MX_BF16;
    const int64_t ldx[2] = {up16(D), up16(D)}, ldh[2] = {(int64_t)IB * kBlk, (int64_t)SB * kBlk};
    const void *xq[2] = {ws + p.xr, ws + p.xq}, *hq[2] = {ws + p.hr, ws + p.hsh};
    RowsArgs gu{}, dn{};
    gu.act = L->activation;
    gu.err = dn.err = reinterpret_cast<unsigned *>(ws);
    for (int sh = 0; sh < (shared ? 2 : 1); ++sh) {
        const mx_fp8_matrix &wg = sh ? L->shared_gate : L->gate, &wu = sh ? L->shared_up : L->up;
        const mx_fp8_matrix &wd = sh ? L->shared_down : L->down;
        RowsProblem &g = gu.p[sh], &d = dn.p[sh];
        g.rows = d.rows = sh ? T : n;
        g.offsets = d.offsets = sh ? nullptr : i32(p.offsets);
        g.K = D;
        g.N = wg.rows;
        g.E = d.E = wg.count;
        g.sx = f32(sh ? p.sx : p.sr);
        g.sx_r = d.sx_r = 1;
        g.sx_b = d.sx_b = g.rows;
        g.swa = wg.scales;
        g.swb = wu.scales;
        g.h = ws + (sh ? p.hsh : p.hr);
        g.ldh = ldh[sh];
        g.hs = f32(sh ? p.hshs : p.hrs);
        g.hs_ld = g.rows;
        d.K = wd.cols;
        d.N = D;
        d.sx = g.hs;
        d.swa = wd.scales;
        d.out = ws + (sh ? p.ys : p.y);
        d.ldo = D;
        d.out_kind = half ? kOutF16 : kOutF32;
        d.out_vec = vec16(d.out, D, half);
        d.out_scale = f32(sh ? p.ysf : p.yf);
        d.out_scale_ld = (D + 63) / 64;
        if ((st = weight_map(&g.wa, wg)) != MX_OK || (st = weight_map(&g.wb, wu)) != MX_OK ||
            (st = weight_map(&d.wa, wd)) != MX_OK)
            return st;
    }
    if ((st = run_rows(kGateUp, gu, xq, ldx, avg, s)) != MX_OK || (st = run_rows(kProduct, dn, hq, ldh, avg, s)) != MX_OK)
        return st;

    CombineArgs c{};
    c.Y = ws + p.y;
    c.Yf = half ? f32(p.yf) : nullptr;
    c.Ys = shared ? ws + p.ys : nullptr;
    c.Ysf = half ? f32(p.ysf) : nullptr;
    c.pos = i32(p.pos);
    c.wts = wts;
    c.residual = residual;
    c.out = out;
    c.T = T;
    c.D = D;
    c.topk = K;
    c.bf16 = L->act_dtype == MX_BF16;
    c.lam = L->layer_scalar;
    if ((e = launch_combine(c, s)) != cudaSuccess)
        return cuda_fail(e, "combine");
    return MX_OK;
}

}  // namespace

extern "C" {

mx_status mx_fp8_quantize(const void *x, int64_t ldx, int dtype, int pow2, const mx_fp8_rows *out, void *stream)
{
    mx_status st;
    if ((st = check_rows(out, "out", false)) != MX_OK || (st = check_dtype(dtype, "dtype")) != MX_OK)
        return st;
    if (pow2 != 0 && pow2 != 1)
        return fail(MX_ERR_INVALID_ARG, "pow2 %d is not 0 or 1", pow2);
    if (ldx < out->cols)
        return fail(MX_ERR_INVALID_ARG, "input row pitch %lld is below its %d columns", (long long)ldx, out->cols);
    if (out->rows == 0)
        return MX_OK;
    if (!x)
        return fail(MX_ERR_INVALID_ARG, "x is NULL");
    if (!aligned(x, dtype == MX_BF16 ? 2 : 4))
        return fail(MX_ERR_ALIGNMENT, "x is misaligned");
    QuantArgs q{};
    q.x = x;
    q.rows = out->rows;
    q.ldx = ldx;
    q.cols = out->cols;
    q.bf16 = dtype == MX_BF16;
    q.pow2 = pow2;
    q.q = static_cast<uint8_t *>(out->q);
    q.ldq = out->ld;
    q.scales = out->scales;
    q.s_r = out->scale_row;
    q.s_b = out->scale_block;
    const cudaError_t e = launch_quantize(q, num_sms(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "FP8 quantisation");
}

size_t mx_fp8_matmul_workspace_bytes(const mx_fp8_matrix *w, int rows)
{
    return check_matrix(w, "w") == MX_OK && rows >= 0 ? kErrBytes : 0;
}

mx_status mx_fp8_matmul(const mx_fp8_rows *x, const mx_fp8_matrix *w, void *out, int64_t ldo, int out_dtype,
                        void *stream, void *ws, size_t ws_bytes)
{
    if (w && w->count != 1)
        return fail(MX_ERR_INVALID_ARG, "w holds %d matrices, one is wanted", w->count);
    return product(x, nullptr, w, out, ldo, out_dtype, stream, ws, ws_bytes);
}

mx_status mx_fp8_grouped_matmul(const mx_fp8_rows *x, const int32_t *offsets, const mx_fp8_matrix *w, void *out,
                                int64_t ldo, int out_dtype, void *stream, void *ws, size_t ws_bytes)
{
    if (!offsets)
        return fail(MX_ERR_INVALID_ARG, "offsets is NULL");
    if (!aligned(offsets, 4))
        return fail(MX_ERR_ALIGNMENT, "offsets must be 4-byte aligned");
    return product(x, offsets, w, out, ldo, out_dtype, stream, ws, ws_bytes);
}

size_t mx_fp8_moe_workspace_bytes(const mx_fp8_layer *layer, int T_max)
{
    if (check_layer(layer) != MX_OK || T_max < 0 || (int64_t)T_max * layer->top_k > kMaxRows)
        return 0;
    const int t = std::max(T_max, 1);
    // (for any number of tokens up to t: each form grows with them)
    size_t n = std::max(make_plan(layer, 1).total, make_plan(layer, std::min(t, kFewTokens)).total);
    if (t > kFewTokens)
        n = std::max(n, make_plan(layer, t).total);
    return n;
}

mx_status mx_fp8_moe_forward(const void *x, int T, const int32_t *topk_idx, const float *topk_w,
                             const mx_fp8_layer *layer, const void *residual, void *out, void *stream, void *ws,
                             size_t ws_bytes)
{
    mx_status st;
    if ((st = check_layer(layer)) != MX_OK)
        return st;
    if (T < 0 || (int64_t)T * layer->top_k > kMaxRows)
        return fail(MX_ERR_INVALID_ARG, "T = %d must be >= 0 and T * top_k <= %d", T, kMaxRows);
    if (T == 0)
        return MX_OK;
    if (!x || !topk_idx || !topk_w || !out)
        return fail(MX_ERR_INVALID_ARG, "x, topk_idx, topk_w and out must not be NULL");
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(residual, 16) || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
        return fail(MX_ERR_ALIGNMENT, "x, out and residual must be 16-byte aligned, topk_idx and topk_w 4-byte");
    if ((st = check_ws(ws, ws_bytes, make_plan(layer, T).total)) != MX_OK)
        return st;
    const size_t bytes = (size_t)T * layer->gate.cols * (layer->act_dtype == MX_BF16 ? 2 : 4);
    const void *ins[2] = {x, residual};
    for (const void *in : ins) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
        if (in && a != b && a < b + bytes && b < a + bytes)
            return fail(MX_ERR_INVALID_ARG, "out overlaps an input without being it");
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *w = static_cast<uint8_t *>(ws);
    if (one_token(layer, T))
        return run_gemv(x, topk_idx, topk_w, layer, residual, out, s, w);
    return T <= kFewTokens ? run_few(x, T, topk_idx, topk_w, layer, residual, out, s, w)
                           : run_many(x, T, topk_idx, topk_w, layer, residual, out, s, w);
}

}  // extern "C"
