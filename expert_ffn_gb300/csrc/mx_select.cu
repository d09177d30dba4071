// mx_select.cu -- routing from logits: scores, groups, top-k, weights, and the
// grouping of slots by expert.
//
// One warp per token; lane i holds the P = E / 32 neighbouring experts from i P
// on in registers, so that a lane's order is the experts' order and ties go to the
// lower index by the first lane and the first register.  Scores are computed
// in fp32.  The choice compares 32-bit keys (the score's bits, made to order as
// unsigned integers; 0: no longer there), k times a maximum over registers and one
// warp reduction.
//
// Exactness.  Where an fp32 score (with a bias, or the sum of a run's two best)
// decides, everything within its error bound of the maximum is a candidate; a
// second candidate, about one token in a thousand, sends the comparison to fp64, for
// the candidates alone.  Without a bias experts compare by their logits, which no
// rounding has touched.
//
// What bounds it: 4096 x 256 fp32 logits are 4 MB, 0.6 us of HBM; a token takes a warp
// some 700 instructions, most of them the k rounds' maxima, and the launches (two where
// slots are grouped and more than one block works on them) the rest.
#include "mx_common.cuh"
#include "mx_host.h"
#include "mx_internal.h"
#include "mx_moe.h"

#include <algorithm>
#include <cmath>

namespace mx {
namespace sel {

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kMaxBlocks = 256;  // blocks whose counts the grouping adds up

struct Args {
    const void *logits;
    int64_t ld;
    int bf16, T, E, K;
    int vec;               // a lane's logits are one aligned piece
    int score, n_groups, topk_groups, best, renorm;
    float scale;
    const float *bias;
    int32_t *idx;
    float *w;
    int32_t *counts, *offsets, *perm;  // nullable together
    int32_t *bc;           // [blocks][E] counts of each block's tokens
    int per;               // tokens of a block
};

__device__ __forceinline__ uint32_t ordered(float f)
{
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float unordered(uint32_t o)
{
    return __uint_as_float(o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
}

__device__ __forceinline__ float load1(const Args &a, int64_t at)
{
    return a.bf16 ? bf2f(__ldg(reinterpret_cast<const uint16_t *>(a.logits) + at))
                  : __ldg(reinterpret_cast<const float *>(a.logits) + at);
}

// ------------------------------------------------------- comparisons in fp64

__device__ double warp_max(double v)
{
    for (int o = 16; o; o >>= 1) {
        const double y = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = y > v ? y : v;
    }
    return v;
}

// Normaliser of a token's softmax: 1 / sum exp(l - m), with its largest logit m (the whole warp).
struct Soft64 {
    double inv;
    float m;
};
__device__ __noinline__ Soft64 soft64(const Args &a, int t)
{
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32)
        m = fmaxf(m, load1(a, (int64_t)t * a.ld + e));  // (a NaN is left out)
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    double z = 0.0;
    for (int e = lane; e < a.E; e += 32) {
        const float l = load1(a, (int64_t)t * a.ld + e);
        if (l == l)
            z += l == m ? 1.0 : exp((double)l - (double)m);
    }
    for (int o = 16; o; o >>= 1)
        z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    return Soft64{z > 0.0 ? 1.0 / z : 0.0, m};
}

// The score that expert e of token t is chosen by.
__device__ double choice64(const Args &a, int t, int e, const Soft64 &S)
{
    const float l = load1(a, (int64_t)t * a.ld + e);
    double s = a.score == MX_SIGMOID ? 1.0 / (1.0 + exp(-(double)l))
                                     : (l == S.m ? 1.0 : exp((double)l - (double)S.m)) * S.inv;
    if (!(l == l))
        s = 0.0;
    double c = a.bias ? s + (double)__ldg(a.bias + e) : s;
    return l == l && c == c ? c : -INFINITY;
}

// Of the candidates (bit j of a lane's mask: expert lane P + j) the one with the highest score,
// the lowest of equal ones.
__device__ __noinline__ int best64(const Args &a, int t, uint32_t mask, int P)
{
    const int lane = threadIdx.x & 31;
    Soft64 S{};
    if (a.score == MX_SOFTMAX)
        S = soft64(a, t);
    double top = -INFINITY;
    int at = 1 << 20;
    for (uint32_t left = mask; left; left &= left - 1) {
        const int e = lane * P + __ffs(left) - 1;
        const double c = choice64(a, t, e, S);
        if (at == 1 << 20 || c > top)
            top = c, at = e;
    }
    const double all = warp_max(top);
    return (int)__reduce_min_sync(0xFFFFFFFFu, (unsigned)(top == all ? at : 1 << 20));
}

// The same of runs: bit g of `mask` (one for the warp).
__device__ __noinline__ int best_group64(const Args &a, int t, uint32_t mask)
{
    const int lane = threadIdx.x & 31, size = a.E / a.n_groups;
    Soft64 S{};
    if (a.score == MX_SOFTMAX)
        S = soft64(a, t);
    double top = -INFINITY;
    int at = -1;
    for (uint32_t left = mask; left; left &= left - 1) {
        const int g = __ffs(left) - 1;
        double c1 = -INFINITY, c2 = -INFINITY;
        for (int i = lane; i < size; i += 32) {
            const double c = choice64(a, t, g * size + i, S);
            if (c > c1)
                c2 = c1, c1 = c;
            else if (c > c2)
                c2 = c;
        }
        for (int o = 16; o; o >>= 1) {
            const double y1 = __shfl_xor_sync(0xFFFFFFFFu, c1, o), y2 = __shfl_xor_sync(0xFFFFFFFFu, c2, o);
            c2 = y1 > c1 ? (c1 > y2 ? c1 : y2) : (y1 > c2 ? y1 : c2);
            c1 = y1 > c1 ? y1 : c1;
        }
        double c = a.best == 2 ? c1 + c2 : c1;
        c = c == c ? c : -INFINITY;
        if (at < 0 || c > top)
            top = c, at = g;
    }
    return at;
}

// ------------------------------------------------------------------ selection

// The key that the warp chooses next: the lane that holds it, or several candidates.
template <int P>
__device__ __forceinline__ void load_logits(const Args &a, int t, int lane, float (&l)[P])
{
    const int64_t at = (int64_t)t * a.ld + lane * P;
    if (a.vec) {
        if (a.bf16) {
            uint32_t r[P < 2 ? 1 : P / 2];
            const uint16_t *p = reinterpret_cast<const uint16_t *>(a.logits) + at;
            if constexpr (P == 1)
                r[0] = __ldg(p);
            else if constexpr (P == 2)
                r[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
            else if constexpr (P == 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
                r[0] = v.x, r[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < P / 8; ++i) {
                    const uint4 v = ldg_u4(p + 8 * i);
                    r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
                }
            }
#pragma unroll
            for (int j = 0; j < P; ++j)
                l[j] = __uint_as_float((j & 1) ? r[j / 2] & 0xFFFF0000u : r[j / 2] << 16);
        } else {
            const float *p = reinterpret_cast<const float *>(a.logits) + at;
            if constexpr (P == 1)
                l[0] = __ldg(p);
            else if constexpr (P == 2) {
                const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
                l[0] = v.x, l[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < P / 4; ++i) {
                    const float4 v = __ldg(reinterpret_cast<const float4 *>(p) + i);
                    l[4 * i] = v.x, l[4 * i + 1] = v.y, l[4 * i + 2] = v.z, l[4 * i + 3] = v.w;
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j)
            l[j] = lane * P + j < a.E ? load1(a, at + j) : 0.0f;
    }
}

// One token by one warp.  row: E floats of shared memory (for groups).  Lane k < K returns
// the k-th choice and its weight.
template <int P>
__device__ __forceinline__ void select_token(const Args &a, int t, int lane, float *row, int &my_idx, float &my_w)
{
    constexpr uint32_t FULL = 0xFFFFFFFFu;
    float l[P], s[P];
    load_logits<P>(a, t, lane, l);
    const int here = min(max(a.E - lane * P, 0), P);  // experts of this lane

    // scores (a NaN logit: 0)
    float smax = 0.0f;
    if (a.score == MX_SIGMOID) {
#pragma unroll
        for (int j = 0; j < P; ++j)
            s[j] = j < here && l[j] == l[j] ? 1.0f / (1.0f + expf(-l[j])) : 0.0f;
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < P; ++j)
            m = fmaxf(m, j < here ? l[j] : -INFINITY);
        m = unordered(__reduce_max_sync(FULL, ordered(m)));
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            s[j] = j < here && l[j] == l[j] ? (l[j] == m ? 1.0f : expf(l[j] - m)) : 0.0f;
            z += s[j];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            z += __shfl_xor_sync(FULL, z, o);
        const float inv = z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
        for (int j = 0; j < P; ++j)
            s[j] *= inv;
    }

    // keys of the choice.  eps: more than any |fp32 score - exact one|.  A sigmoid is right to
    // 2^-22 of itself (expf 2 ulp, two roundings), a softmax to 2^-19 of the largest (its sum has up to 21
    // roundings, its arguments' shift by d is worth d e^-d); a bias adds one rounding of c.
    uint32_t key[P];
    float eps = 0.0f;
    if (a.bias) {
        float cmax = 0.0f;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float c = -INFINITY;
            if (j < here) {
                c = s[j] + __ldg(a.bias + lane * P + j);
                c = l[j] == l[j] && c == c ? c : -INFINITY;
                if (fabsf(c) < INFINITY)
                    cmax = fmaxf(cmax, fabsf(c));
                smax = fmaxf(smax, s[j]);
            }
            key[j] = j < here ? ordered(c + 0.0f) : 0u;
        }
        eps = 1.9073486e-6f * __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(smax))) +
              1.1920929e-7f * __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(cmax)));
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j)
            key[j] = j < here ? ordered((l[j] == l[j] ? l[j] : -INFINITY) + 0.0f) : 0u;
    }

    if (a.topk_groups < a.n_groups) {
        // Runs: 32 / n_groups lanes (a power of two) each go over a part of one run's scores.
        const int size = a.E / a.n_groups;
        const bool by_score = a.best == 2 && !a.bias;  // (sums of scores; else the keys' own order)
        float geps = a.best == 2 ? 2.0f * eps : eps;
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (j < here)
                row[lane * P + j] = by_score ? (l[j] == l[j] ? s[j] : -INFINITY) : unordered(key[j]);
        if (by_score) {
#pragma unroll
            for (int j = 0; j < P; ++j)
                smax = fmaxf(smax, s[j]);
            geps = 2.0f * 1.9073486e-6f * __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(smax)));
        }
        __syncwarp();
        int per = 1;
        while (2 * per * a.n_groups <= 32)
            per *= 2;
        const int g = lane / per, part = lane & (per - 1);
        float c1 = -INFINITY, c2 = -INFINITY;
        if (g < a.n_groups)
            for (int i = part; i < size; i += per) {
                // (each run starts at another place: runs are often 32 banks apart)
                int at = i + g * per;
                at = at < size ? at : at % size;
                const float c = row[g * size + at];
                c2 = fmaxf(c2, fminf(c1, c));
                c1 = fmaxf(c1, c);
            }
        for (int o = per >> 1; o; o >>= 1) {
            const float y1 = __shfl_xor_sync(FULL, c1, o), y2 = __shfl_xor_sync(FULL, c2, o);
            c2 = fmaxf(fminf(c1, y1), fmaxf(c2, y2));
            c1 = fmaxf(c1, y1);
        }
        __syncwarp();
        float gs = a.best == 2 ? c1 + c2 : c1;
        if (a.best == 2 && geps > 0.0f && fabsf(gs) < INFINITY)
            geps += 1.1920929e-7f * fabsf(gs);  // (the sum's own rounding; made the warp's largest below)
        geps = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(geps)));
        gs = gs == gs ? gs : -INFINITY;
        uint32_t gkey = part == 0 && g < a.n_groups ? ordered(gs + 0.0f) : 0u;
        uint32_t kept = 0;
        for (int k = 0; k < a.topk_groups; ++k) {
            const uint32_t m = __reduce_max_sync(FULL, gkey);
            uint32_t cand = __ballot_sync(FULL, gkey == m);
            int win = (__ffs(cand) - 1) / per;
            if (geps > 0.0f) {
                const float mf = unordered(m), lo = mf - 2.0f * geps;
                cand = __ballot_sync(FULL, gkey != 0u && unordered(gkey) >= lo);
                if (cand & (cand - 1)) {
                    uint32_t groups = 0;
                    for (uint32_t left = cand; left; left &= left - 1)
                        groups |= 1u << ((__ffs(left) - 1) / per);
                    win = best_group64(a, t, groups);
                }
            }
            kept |= 1u << win;
            if (g == win)
                gkey = 0u;
        }
        int r = lane * P % size, gg = lane * P / size;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            if (j < here && !(kept >> gg & 1u))
                key[j] = 0u;
            if (++r == size)
                r = 0, ++gg;
        }
    }

    my_idx = 0;
    my_w = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        uint32_t top = key[0];
#pragma unroll
        for (int j = 1; j < P; ++j)
            top = max(top, key[j]);
        const uint32_t m = __reduce_max_sync(FULL, top);
        int win = -1;
        if (eps > 0.0f) {
            const uint32_t lo = ordered(unordered(m) - 2.0f * eps);
            uint32_t mask = 0;
#pragma unroll
            for (int j = 0; j < P; ++j)
                mask |= key[j] >= lo && key[j] != 0u ? 1u << j : 0u;
            const uint32_t lanes = __ballot_sync(FULL, mask != 0u), more = __ballot_sync(FULL, (mask & (mask - 1)) != 0u);
            if ((lanes & (lanes - 1)) || more)
                win = best64(a, t, mask, P);
        }
        if (win < 0) {
            const int src = __ffs(__ballot_sync(FULL, top == m)) - 1;
            int j0 = 0;
#pragma unroll
            for (int j = P - 1; j >= 0; --j)
                if (key[j] == m)
                    j0 = j;
            win = __shfl_sync(FULL, lane * P + j0, src);
        }
        const int src = win / P;
        float sv = 0.0f;
        if (lane == src) {
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (src * P + j == win) {
                    sv = s[j];
                    key[j] = 0u;
                }
        }
        sv = __shfl_sync(FULL, sv, src);
        if (lane == k) {
            my_idx = win;
            my_w = sv;
        }
    }
    if (a.renorm) {
        float sum = my_w;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum += __shfl_xor_sync(FULL, sum, o);
        my_w = sum > 0.0f ? my_w / sum : 0.0f;
    }
    my_w *= a.scale;
}

// ------------------------------------------------------------------- grouping

// Slots [lo, hi) of a block to their places, in ascending order within an expert: h[w][e] starts
// as the place of warp w's first slot of expert e.
__device__ __forceinline__ void warp_counts(const int32_t *idx, int lo, int hi, int lane, int *mine)
{
    for (int s0 = lo; s0 < hi; s0 += 32) {
        const int s = s0 + lane, e = s < hi ? idx[s] : -1;
        const unsigned m = __match_any_sync(0xFFFFFFFFu, e);
        if (e >= 0 && lane == __ffs(m) - 1)
            mine[e] += __popc(m);
        __syncwarp();
    }
}

// Block b's slots into perm.  base[e]: place of its first slot of expert e; h: kWarps * E.
__device__ void place_slots(const Args &a, int b, const int *base, int *h)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = (int64_t)b * a.per;
    const int n = (int)min((int64_t)a.per, a.T - first) * a.K, part = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int32_t *idx = a.idx + first * a.K;
    const int lo = min(warp * part, n), hi = min(lo + part, n);
    for (int i = threadIdx.x; i < kWarps * a.E; i += kThreads)
        h[i] = 0;
    __syncthreads();
    int *mine = h + warp * a.E;
    warp_counts(idx, lo, hi, lane, mine);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        int run = base[e];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int c = h[w * a.E + e];
            h[w * a.E + e] = run;
            run += c;
        }
    }
    __syncthreads();
    const unsigned lt = (1u << lane) - 1u;
    for (int s0 = lo; s0 < hi; s0 += 32) {
        const int s = s0 + lane, e = s < hi ? idx[s] : -1;
        const unsigned m = __match_any_sync(0xFFFFFFFFu, e);
        if (e >= 0)
            a.perm[mine[e] + __popc(m & lt)] = (int)(first * a.K) + s;
        __syncwarp();
        if (e >= 0 && lane == __ffs(m) - 1)
            mine[e] += __popc(m);
        __syncwarp();
    }
}

// Exclusive sum of v over the block's threads i < kMaxExperts, two values to a thread: in place
// over cnt[E]; total into cnt[E].
__device__ void scan_counts(int *cnt, int E)
{
    __shared__ int wsum[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int v0 = 2 * tid < E ? cnt[2 * tid] : 0, v1 = 2 * tid + 1 < E ? cnt[2 * tid + 1] : 0;
    int incl = v0 + v1;
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
    const int ex = before + incl - v0 - v1;
    if (2 * tid < E)
        cnt[2 * tid] = ex;
    if (2 * tid + 1 < E)
        cnt[2 * tid + 1] = ex + v0;
    if (tid == kThreads - 1)
        cnt[E] = ex + v0 + v1;
    __syncthreads();
}
static_assert(2 * kThreads >= kMaxExperts, "two experts to a thread");

// Dynamic shared memory: rows for groups [kWarps][E] floats, later the warps' counts; then counts [E + 1].
size_t smem_bytes(int E) { return (size_t)(kWarps * E + E + 1) * 4; }

template <int P>
__global__ void __launch_bounds__(kThreads) select_kernel(const Args a)
{
    extern __shared__ __align__(16) float sm[];
    int *cnt = reinterpret_cast<int *>(sm + kWarps * a.E);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.counts) {
        pdl_trigger();  // (the placing kernel waits for this one's end)
        for (int e = threadIdx.x; e < a.E; e += kThreads)
            cnt[e] = 0;
        __syncthreads();
    }
    const int64_t first = (int64_t)blockIdx.x * a.per;
    const int last = (int)min((int64_t)a.T, first + a.per);
    for (int t = (int)first + warp; t < last; t += kWarps) {
        int i;
        float w;
        select_token<P>(a, t, lane, sm + warp * a.E, i, w);
        if (lane < a.K) {
            a.idx[(int64_t)t * a.K + lane] = i;
            a.w[(int64_t)t * a.K + lane] = w;
            if (a.counts)
                atomicAdd(cnt + i, 1);
        }
        __syncwarp();
    }
    if (!a.counts)
        return;
    __syncthreads();
    if (gridDim.x > 1) {
        for (int e = threadIdx.x; e < a.E; e += kThreads)
            a.bc[(int64_t)blockIdx.x * a.E + e] = cnt[e];
        return;
    }
    for (int e = threadIdx.x; e < a.E; e += kThreads)
        a.counts[e] = cnt[e];
    __syncthreads();
    scan_counts(cnt, a.E);
    for (int e = threadIdx.x; e <= a.E; e += kThreads)
        a.offsets[e] = cnt[e];
    place_slots(a, 0, cnt, reinterpret_cast<int *>(sm));
}

// More than one block: each adds up all blocks' counts itself (an eighth of them to a warp)
// and places its own slots.
__global__ void __launch_bounds__(kThreads) place_kernel(const Args a)
{
    extern __shared__ __align__(16) int smi[];
    int *h = smi, *cnt = smi + kWarps * a.E;
    const int nb = gridDim.x, me = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ int below[kMaxExperts];
    for (int e = tid; e < a.E; e += kThreads)
        cnt[e] = below[e] = 0;
    __syncthreads();
    pdl_wait();
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        if (e < a.E) {
            int all = 0, low = 0;
#pragma unroll 8
            for (int b = warp; b < nb; b += kWarps) {
                const int c = a.bc[(int64_t)b * a.E + e];
                all += c;
                low += b < me ? c : 0;
            }
            atomicAdd(cnt + e, all);
            atomicAdd(below + e, low);
        }
    }
    __syncthreads();
    if (me == 0)
        for (int e = tid; e < a.E; e += kThreads)
            a.counts[e] = cnt[e];
    __syncthreads();
    scan_counts(cnt, a.E);
    if (me == 0)
        for (int e = tid; e <= a.E; e += kThreads)
            a.offsets[e] = cnt[e];
    for (int e = tid; e < a.E; e += kThreads)
        below[e] += cnt[e];
    place_slots(a, me, below, h);
}

// Blocks that share T tokens whose slots are grouped: eight tokens to a block (a warp each), more
// where that would be above kMaxBlocks.
int tokens_of_block(int T) { return std::max(kWarps, ((T + kMaxBlocks - 1) / kMaxBlocks + kWarps - 1) / kWarps * kWarps); }

template <int P>
cudaError_t launch(const Args &a, int grid, cudaStream_t s)
{
    const size_t smem = smem_bytes(a.E);
    select_kernel<P><<<grid, kThreads, smem, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.counts && grid > 1)
        e = launch_dependent(place_kernel, grid, kThreads, smem, s, a);
    return e;
}

mx_status check_router(const mx_router *r)
{
    if (!r)
        return fail(MX_ERR_INVALID_ARG, "router is NULL");
    if (r->n_experts < 1 || r->n_experts > kMaxExperts)
        return fail(MX_ERR_UNSUPPORTED, "n_experts %d must be in [1, %d]", r->n_experts, kMaxExperts);
    if (r->n_groups < 1 || r->n_groups > 32 || r->n_experts % r->n_groups)
        return fail(MX_ERR_INVALID_ARG, "n_groups %d must be in [1, 32] and divide %d", r->n_groups, r->n_experts);
    if (r->topk_groups < 1 || r->topk_groups > r->n_groups)
        return fail(MX_ERR_INVALID_ARG, "topk_groups %d must be in [1, %d]", r->topk_groups, r->n_groups);
    const int size = r->n_experts / r->n_groups, most = std::min(size * r->topk_groups, kMaxTopK);
    if (r->top_k < 1 || r->top_k > most)
        return fail(MX_ERR_INVALID_ARG, "top_k %d must be in [1, %d]", r->top_k, most);
    if (r->score != MX_SOFTMAX && r->score != MX_SIGMOID)
        return fail(MX_ERR_INVALID_ARG, "score %d is not MX_SOFTMAX or MX_SIGMOID", r->score);
    if (r->group_best != 1 && r->group_best != 2)
        return fail(MX_ERR_INVALID_ARG, "group_best %d is not 1 or 2", r->group_best);
    if (r->group_best == 2 && size < 2)
        return fail(MX_ERR_INVALID_ARG, "group_best 2 needs runs of at least two experts");
    if (r->renormalise != 0 && r->renormalise != 1)
        return fail(MX_ERR_INVALID_ARG, "renormalise %d is not 0 or 1", r->renormalise);
    if (!std::isfinite(r->scale))
        return fail(MX_ERR_INVALID_ARG, "scale must be finite");
    if (!aligned(r->bias, 4))
        return fail(MX_ERR_ALIGNMENT, "bias must be 4-byte aligned");
    return MX_OK;
}

size_t ws_bytes_of(int E, int T)
{
    const int per = tokens_of_block(T), nb = (T + per - 1) / per;
    return kErrBytes + up256(nb > 1 ? (size_t)nb * E * 4 : 0);
}

}  // namespace
}  // namespace sel
}  // namespace mx

using namespace mx;

extern "C" size_t mx_route_logits_workspace_bytes(const mx_router *router, int T_max)
{
    if (sel::check_router(router) != MX_OK)
        return 0;
    if (T_max < 0) {
        fail(MX_ERR_INVALID_ARG, "T_max %d is negative", T_max);
        return 0;
    }
    // (fewer tokens never need more: blocks and tokens of a block both grow with T, up to the rounding
    // of the tokens of a block, which kMaxBlocks blocks bound)
    return std::max(sel::ws_bytes_of(router->n_experts, T_max),
                    T_max > sel::kWarps * sel::kMaxBlocks ? kErrBytes + up256((size_t)sel::kMaxBlocks * router->n_experts * 4)
                                                          : (size_t)0);
}

extern "C" mx_status mx_route_logits(const void *logits, int64_t ld, int dtype, int T, const mx_router *router,
                                     int32_t *topk_idx, float *topk_w, int32_t *counts, int32_t *offsets, int32_t *perm,
                                     void *stream, void *ws, size_t ws_bytes)
{
    mx_status st;
    if ((st = sel::check_router(router)) != MX_OK || (st = check_dtype(dtype, "dtype")) != MX_OK)
        return st;
    const int E = router->n_experts, K = router->top_k;
    if (T < 0 || (int64_t)T * K > 0x7FFFFFFF)
        return fail(MX_ERR_INVALID_ARG, "T %d must be at least 0, T * top_k below 2^31", T);
    if (ld < E)
        return fail(MX_ERR_INVALID_ARG, "row pitch %lld is below the %d experts", (long long)ld, E);
    if (ld > ((int64_t)1 << 31))
        return fail(MX_ERR_UNSUPPORTED, "row pitch %lld is too large", (long long)ld);
    const bool group = counts || offsets || perm;
    if (group && (!counts || !offsets || (!perm && T > 0)))
        return fail(MX_ERR_INVALID_ARG, "counts, offsets and perm come together");
    if (T > 0 && (!logits || !topk_idx || !topk_w))
        return fail(MX_ERR_INVALID_ARG, "logits, topk_idx and topk_w must not be NULL");
    if (!aligned(logits, dtype_bytes(dtype)) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(counts, 4) ||
        !aligned(offsets, 4) || !aligned(perm, 4))
        return fail(MX_ERR_ALIGNMENT, "a pointer is misaligned");
    if (group && (st = check_ws(ws, ws_bytes, sel::ws_bytes_of(E, T))) != MX_OK)
        return st;
    if (T == 0 && !group)
        return MX_OK;
    sel::Args a{};
    a.logits = logits;
    a.ld = ld;
    a.bf16 = dtype == MX_BF16;
    a.T = T;
    a.E = E;
    a.K = K;
    a.score = router->score;
    a.n_groups = router->n_groups;
    a.topk_groups = router->topk_groups;
    a.best = router->group_best;
    a.renorm = router->renormalise;
    a.scale = router->scale;
    a.bias = router->bias;
    a.idx = topk_idx;
    a.w = topk_w;
    if (group) {
        a.counts = counts;
        a.offsets = offsets;
        a.perm = perm;
        a.bc = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + kErrBytes);
    }
    a.per = group ? sel::tokens_of_block(T) : sel::kWarps;
    const int grid = std::max<int64_t>(1, ((int64_t)T + a.per - 1) / a.per);
    int P = 1;
    while (32 * P < E)
        P *= 2;
    const size_t piece = std::min<size_t>(16, P * dtype_bytes(dtype));
    a.vec = E == 32 * P && aligned(logits, piece) && ld * dtype_bytes(dtype) % piece == 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = P == 1   ? sel::launch<1>(a, grid, s)
                          : P == 2 ? sel::launch<2>(a, grid, s)
                          : P == 4 ? sel::launch<4>(a, grid, s)
                          : P == 8 ? sel::launch<8>(a, grid, s)
                                   : sel::launch<16>(a, grid, s);
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "routing");
}
