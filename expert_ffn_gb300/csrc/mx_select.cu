// mx_select.cu -- routing from logits: scores, groups, top-k, weights, and the
// grouping of slots by expert.
//
// One warp per token; lane i holds the P = E / 32 neighbouring experts from i P
// on in registers, so that a lane's order is the experts' order and ties go to the
// lower index by the first lane and the first register.  Scores are computed
// in fp32, and only where the choice needs them: without a bias experts are compared by
// their logits, and the chosen ones' weights are worked out at the end, a lane each.
// The choice compares 32-bit keys (a number's bits, made to order as
// unsigned integers; 0: no longer there): each lane sorts its own, then k times the
// highest of the 32 heads is taken off by one warp reduction; which expert a key was, lane k finds
// at the end among the winning lane's keys in shared memory.
//
// Exactness.  Where an fp32 score (with a bias, or the sum of a run's two best)
// decides, the chosen ones and the next are looked at once more: any two neighbours
// within their error bounds send the token to a loop that compares the candidates in fp64.
// With random biases that is about one token in a thousand of fp32 logits with sigmoids; but bf16 logits
// are often equal, and with a bias of zeros, as a balance bias begins, some third of the tokens go there: 4096 x 256
// without runs, slots grouped, sigmoid 16.6 us (random biases 14.3), softmax 29.4 (21.4).  Without
// a bias experts compare by their logits, which no rounding has touched (12.5).
//
// Grouping.  One selecting block (up to eight tokens) puts its slots in order itself; of few the last to end those of
// all.  Of more each leaves its tokens' counts by expert, and the placing kernel's blocks each add up all of them (bytes, an expert's
// neighbouring, so that 4096 tokens of 256 experts are 32 KB and four blocks' one dp4a) and put
// their own tokens' slots in order.
//
// What bounds it: 4096 x 256 fp32 logits are 4 MB, 0.6 us of HBM.  Choosing takes 9.0 us of the whole 15.4: a warp's chain
// of some 1170 instructions a token (31 % of the issue slots, 48 % of the warps), then the placing launch.
#include "mx_common.cuh"
#include "mx_host.h"
#include "mx_internal.h"
#include "mx_moe.h"

#include <algorithm>
#include <cmath>

namespace mx {
namespace sel {

namespace {

// Warps of a selecting block: eight.  When many tokens' slots are grouped 32 (16 for more than 256 experts,
// whose keys take more registers), so that the placing blocks have fewer counts to add up: 4096 x 256 in runs
// 15.4 us (by eight 18.9), 2048 13; but 32 warps on one SM take each other's time: 333 x 60 by eight 6.8 us, by
// 32 8.1.
constexpr int kWarps = 8;
constexpr int many_warps(int P) { return P <= 8 ? 32 : 16; }
constexpr int kManyTokens = 2048;
constexpr int kRuns = 512;    // selecting blocks when many tokens' slots are grouped, as long as kMaxRun allows
constexpr int kMaxRun = 224;  // tokens of a block at most (its counts are bytes)
constexpr int kPlaceWarps = 16, kPlaceBlocks = 128;
constexpr int kMaxTokens = 1 << 30;
// Slots up to which the last selecting block places them all: one launch less.  That is for single calls, which the host
// bounds (2.5 us a launch; 333 x 60 top-4 7.9 us a call instead of 10.3); in a captured graph it costs up to 0.9 us of the
// device's time: 9 tokens 5.4 us instead of 5.6, 333 x 60 top-4 6.8 instead of 6.5, 256 x 256 top-8 9.4 instead of 8.5
// (512 x 256 top-8 15.0 instead of 8.9).
constexpr int kLastSlots = 2048;

struct Args {
    const void *logits;
    int64_t ld;
    int bf16, T, E, K;
    int vec, vec_bias;     // a lane's logits, its biases are aligned pieces
    int score, n_groups, topk_groups, best, renorm;
    float scale;
    const float *bias;
    int32_t *idx;
    float *w;
    int32_t *counts, *offsets, *perm;  // nullable together
    int words;             // of 32 tokens each, where the last selecting block places all slots; else 0
    unsigned *ticket;      // such blocks that have ended; 0 between calls
    uint8_t *bc;           // [E][pitch] counts of the selecting blocks' tokens
    int per, runs, join;   // tokens of a selecting block, such blocks, how many of them a placing block joins
    int pitch, run_lanes;  // runs rounded up to a multiple of 16; lanes that share an expert's, a power of two
    int lanes;             // lanes of a run of experts, a power of two; 0: it does not end with lanes
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

// A logit; a NaN counts as -inf (fmaxf leaves it out), and -0 as 0.
__device__ __forceinline__ float tidy(float l) { return fmaxf(l + 0.0f, -INFINITY); }

__device__ __forceinline__ float load1(const Args &a, int64_t at)
{
    return tidy(a.bf16 ? bf2f(reinterpret_cast<const uint16_t *>(a.logits)[at])
                       : reinterpret_cast<const float *>(a.logits)[at]);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
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
        m = fmaxf(m, load1(a, (int64_t)t * a.ld + e));
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    double z = 0.0;
    for (int e = lane; e < a.E; e += 32) {
        const float l = load1(a, (int64_t)t * a.ld + e);
        z += l == m ? 1.0 : exp((double)l - (double)m);
    }
    for (int o = 16; o; o >>= 1)
        z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    return Soft64{1.0 / z, m};
}

// The score that expert e of token t is chosen by.
__device__ double choice64(const Args &a, int t, int e, const Soft64 &S)
{
    const float l = load1(a, (int64_t)t * a.ld + e);
    const double s = a.score == MX_SIGMOID ? 1.0 / (1.0 + exp(-(double)l))
                                           : (l == S.m ? 1.0 : exp((double)l - (double)S.m)) * S.inv;
    const double c = a.bias ? s + (double)a.bias[e] : s;
    return c == c ? c : -INFINITY;
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

// A bound of a score's rounding: relative to it, on top of the score's own error `off`.
constexpr float kRel = 2.3841858e-7f;  // 2^-22

// The chosen runs (a bit each) where fp32 leaves them open.  gs, ge: this lane's run's score and its error bound;
// leader: a lane that speaks for run g.
__device__ __noinline__ uint32_t exact_groups(const Args &a, int t, float gs, float ge, bool leader, int g)
{
    uint32_t kept = 0;
    for (int k = 0; k < a.topk_groups; ++k) {
        const bool in = leader && !(kept >> g & 1u);
        const uint32_t low = __reduce_max_sync(0xFFFFFFFFu, in ? ordered(gs - ge) : 0u);
        const uint32_t all = __reduce_or_sync(0xFFFFFFFFu, in && ordered(gs + ge) >= low ? 1u << g : 0u);
        kept |= 1u << (all & (all - 1) ? best_group64(a, t, all) : __ffs(all) - 1);
    }
    return kept;
}

// The chosen experts, lane k the k-th, where fp32 leaves their order open.  keys: of all experts, in shared memory.
template <int P>
__device__ __noinline__ int exact_experts(const Args &a, int t, const uint32_t *keys, float off)
{
    const int lane = threadIdx.x & 31;
    uint32_t key[P];
#pragma unroll
    for (int j = 0; j < P; ++j)
        key[j] = lane * P + j < a.E ? keys[lane * P + j] : 0u;
    int mine = 0;
    for (int k = 0; k < a.K; ++k) {
        uint32_t top = key[0];
#pragma unroll
        for (int j = 1; j < P; ++j)
            top = max(top, key[j]);
        const uint32_t mk = __reduce_max_sync(0xFFFFFFFFu, top);
        const float f = unordered(mk);
        const uint32_t lo = fabsf(f) < INFINITY ? ordered(f - 2.0f * (off + kRel * fabsf(f))) : mk;
        uint32_t mask = 0;
#pragma unroll
        for (int j = 0; j < P; ++j)
            mask |= key[j] >= lo ? 1u << j : 0u;
        const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, mask != 0u);
        int e;
        if ((lanes & (lanes - 1)) | __ballot_sync(0xFFFFFFFFu, (mask & (mask - 1)) != 0u))
            e = best64(a, t, mask, P);
        else
            e = __shfl_sync(0xFFFFFFFFu, lane * P + __ffs(mask) - 1, __ffs(lanes) - 1);
#pragma unroll
        for (int j = 0; j < P; ++j)
            key[j] = lane * P + j == e ? 0u : key[j];
        if (lane == k)
            mine = e;
    }
    return mine;
}

// ------------------------------------------------------------------ selection

// Sorts descending (Batcher's odd-even merge sort).
template <int P>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[P])
{
#pragma unroll
    for (int p = 1; p < P; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < P; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (j + i + q < P && (j + i) / (2 * p) == (j + i + q) / (2 * p)) {
                        const uint32_t x = k[j + i], y = k[j + i + q];
                        k[j + i] = max(x, y);
                        k[j + i + q] = min(x, y);
                    }
}

// The lane's logits; behind the last expert -inf.
template <int P>
__device__ __forceinline__ void load_logits(const Args &a, int t, int lane, float (&l)[P])
{
    const int64_t at = (int64_t)t * a.ld + lane * P;
    if (a.vec) {
        if (a.bf16) {
            uint32_t r[P < 2 ? 1 : P / 2];
            const uint16_t *p = reinterpret_cast<const uint16_t *>(a.logits) + at;
            if constexpr (P == 1)
                r[0] = *p;
            else if constexpr (P == 2)
                r[0] = *reinterpret_cast<const uint32_t *>(p);
            else if constexpr (P == 4) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                r[0] = v.x, r[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < P / 8; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(p + 8 * i);
                    r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
                }
            }
#pragma unroll
            for (int j = 0; j < P; ++j)
                l[j] = __uint_as_float((j & 1) ? r[j / 2] & 0xFFFF0000u : r[j / 2] << 16);
        } else {
            const float *p = reinterpret_cast<const float *>(a.logits) + at;
            if constexpr (P == 1)
                l[0] = *p;
            else if constexpr (P == 2) {
                const float2 v = *reinterpret_cast<const float2 *>(p);
                l[0] = v.x, l[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < P / 4; ++i) {
                    const float4 v = reinterpret_cast<const float4 *>(p)[i];
                    l[4 * i] = v.x, l[4 * i + 1] = v.y, l[4 * i + 2] = v.z, l[4 * i + 3] = v.w;
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j)
            l[j] = lane * P + j < a.E ? load1(a, at + j) : -INFINITY;
        return;
    }
#pragma unroll
    for (int j = 0; j < P; ++j)
        l[j] = tidy(l[j]);
}

// One token by one warp.  row: E words of shared memory.  Lane k < K returns the k-th choice and its
// weight.
template <int P>
__device__ __forceinline__ void select_token(const Args &a, int t, int lane, uint32_t *row, int &my_idx, float &my_w)
{
    constexpr uint32_t FULL = 0xFFFFFFFFu;
    float l[P];
    load_logits<P>(a, t, lane, l);
    const int here = min(max(a.E - lane * P, 0), P);  // experts of this lane
    const bool groups = a.topk_groups < a.n_groups;
    const bool by_score = groups && a.best == 2 && !a.bias;  // runs by sums of scores (else by what experts go by)
    const bool soft = a.score == MX_SOFTMAX;

    // c: what experts are chosen by.  off: more than the error of any score in it.  A sigmoid by the fast exponential
    // (2 + 1.16 |l| ulp) is off by s (1 - s) of that, 0.62 2^-23 at most, and two roundings; a softmax by expf (2 ulp)
    // by the arguments' shift, worth d e^-d ulp, and up to 25 roundings of its sum, below 2^-19 of the largest.
    float c[P], s[P], m = 0.0f, z = 1.0f, off = 0.0f;
    if (soft) {
        m = l[0];
#pragma unroll
        for (int j = 1; j < P; ++j)
            m = fmaxf(m, l[j]);
        m = unordered(__reduce_max_sync(FULL, ordered(m)));
        if (a.bias || by_score || !a.renorm) {  // (the weights' own sum replaces it otherwise)
            z = 0.0f;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                s[j] = j >= here ? 0.0f : l[j] == m ? 1.0f : expf(l[j] - m);
                z += s[j];
            }
            z = warp_sum(z);
            const float inv = 1.0f / z;
#pragma unroll
            for (int j = 0; j < P; ++j)
                s[j] *= inv;
            off = 1.9073486e-6f * inv;
        }
    } else if (a.bias || by_score) {
#pragma unroll
        for (int j = 0; j < P; ++j)
            s[j] = __fdividef(1.0f, 1.0f + __expf(-l[j]));
        off = 2.9802322e-7f;
    }
    if (a.bias) {
        if (P >= 4 && a.vec_bias) {
#pragma unroll
            for (int i = 0; i < P / 4; ++i) {
                const float4 v = reinterpret_cast<const float4 *>(a.bias + lane * P)[i];
                c[4 * i] = v.x, c[P >= 4 ? 4 * i + 1 : 0] = v.y, c[P >= 4 ? 4 * i + 2 : 0] = v.z, c[P >= 4 ? 4 * i + 3 : 0] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j)
                c[j] = j < here ? a.bias[lane * P + j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < P; ++j)
            c[j] = fmaxf(s[j] + c[j], -INFINITY);  // (a NaN, by the bias, ranks as -inf; a sum of -0 and a score is not -0)
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j)
            c[j] = l[j];
    }

    uint32_t kept = FULL;
    int per = a.lanes;
    if (groups) {
        // The two highest of each run: `per` lanes go over one run's scores.
        const int size = a.E / a.n_groups;
        float c1 = -INFINITY, c2 = -INFINITY;
        if (per) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float x = j >= here ? -INFINITY : by_score ? s[j] : c[j];
                c2 = fmaxf(c2, fminf(c1, x));
                c1 = fmaxf(c1, x);
            }
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (j < here)
                    row[lane * P + j] = __float_as_uint(by_score ? s[j] : c[j]);
            __syncwarp();
            per = 1;
            while (2 * per * a.n_groups <= 32)
                per *= 2;
            if (lane / per < a.n_groups)
                for (int i = lane & (per - 1); i < size; i += per) {
                    const float x = __uint_as_float(row[lane / per * size + i]);
                    c2 = fmaxf(c2, fminf(c1, x));
                    c1 = fmaxf(c1, x);
                }
            __syncwarp();
        }
        const int shift = __ffs(per) - 1, g = lane >> shift;
        for (int o = per >> 1; o; o >>= 1) {
            const float y1 = __shfl_xor_sync(FULL, c1, o), y2 = __shfl_xor_sync(FULL, c2, o);
            c2 = fmaxf(fminf(c1, y1), fmaxf(c2, y2));
            c1 = fmaxf(c1, y1);
        }
        const bool leader = (lane & (per - 1)) == 0 && g < a.n_groups;
        float gs = a.best == 2 ? fmaxf(c1 + c2, -INFINITY) : c1;  // (a NaN ranks as -inf)
        uint32_t gkey = leader ? ordered(gs + 0.0f) : 0u;
        kept = 0;
        for (int k = 0; k < a.topk_groups; ++k) {
            const uint32_t mk = __reduce_max_sync(FULL, gkey);
            const int src = __ffs(__ballot_sync(FULL, gkey == mk)) - 1;
            kept |= 1u << (src >> shift);
            if (lane == src)
                gkey = 0u;
        }
        if (off > 0.0f && (a.best == 2 || a.bias)) {
            // open, unless the chosen runs are above the others by more than their errors
            const bool finite = fabsf(gs) < INFINITY;
            const float ge = !finite ? 0.0f : a.best == 2 ? 2.0f * off + kRel * (fabsf(c1) + fabsf(c2)) : off + kRel * fabsf(gs);
            const bool in = kept >> g & 1u;
            const uint32_t low = __reduce_min_sync(FULL, leader && in ? ordered(gs - ge) : FULL);
            const uint32_t high = __reduce_max_sync(FULL, leader && !in ? ordered(gs + ge) : 0u);
            if (high >= low)
                kept = exact_groups(a, t, gs, ge, leader, g);
        }
        if (a.lanes && !(kept >> (g & 31) & 1u))  // (a lane behind the last run has no experts)
            per = -1;
    }

    // Keys, and a copy of them in shared memory.
    uint32_t key[P];
    if (groups && !a.lanes) {
        const int size = a.E / a.n_groups;
        int r = lane * P % size, g = lane * P / size;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            key[j] = j < here && (kept >> g & 1u) ? ordered(c[j]) : 0u;
            if (++r == size)
                r = 0, ++g;
        }
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j)
            key[j] = j < here && per >= 0 ? ordered(c[j]) : 0u;
    }
    if (P >= 4 && a.E == 32 * P) {
#pragma unroll
        for (int i = 0; i < P / 4; ++i)
            reinterpret_cast<uint4 *>(row + lane * P)[i] =
                make_uint4(key[4 * i], key[P >= 4 ? 4 * i + 1 : 0], key[P >= 4 ? 4 * i + 2 : 0], key[P >= 4 ? 4 * i + 3 : 0]);
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (j < here)
                row[lane * P + j] = key[j];
    }
    __syncwarp();
    sort_keys(key);

    // The highest heads, one after another; with scores that carry an error one more than the call wants.
    const bool open = a.bias != nullptr;
    uint32_t my_key = 0, mk = 0;
    int my_src = 0;
    for (int k = 0; k < a.K + (open ? 1 : 0); ++k) {
        mk = __reduce_max_sync(FULL, key[0]);
        const int src = __ffs(__ballot_sync(FULL, key[0] == mk)) - 1;
        if (lane == k) {
            my_key = mk;
            my_src = src;
        }
        if (lane == src) {
#pragma unroll
            for (int j = 0; j + 1 < P; ++j)
                key[j] = key[j + 1];
            key[P - 1] = 0u;
        }
    }
    bool close = false;
    if (open) {
        uint32_t next = __shfl_down_sync(FULL, my_key, 1);
        if (lane == a.K - 1)
            next = mk;
        const float f = unordered(my_key);
        close = lane < a.K && fabsf(f) < INFINITY && next >= ordered(f - 2.0f * (off + kRel * fabsf(f)));
        close = __any_sync(FULL, close);
    }
    if (close) {
        my_idx = exact_experts<P>(a, t, row, off);
    } else {
        // the key's place among the winning lane's (equal keys of a lane were taken in their order)
        const unsigned long long who = lane < a.K ? (unsigned long long)my_src << 32 | my_key : ~(unsigned long long)lane;
        int skip = __popc(__match_any_sync(FULL, who) & ((1u << lane) - 1u));
        my_idx = 0;
        if (lane < a.K) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int e = my_src * P + j;
                if (e < a.E && row[e] == my_key && skip-- == 0)
                    my_idx = e;
            }
        }
    }
    __syncwarp();

    // The weights of the chosen, a lane each, from their logits.  (A renormalised softmax goes by the largest
    // chosen one, which in runs need not be the largest of all.  So do renormalised sigmoids below 1/2, as e^(l - m) / (1 + e^l):
    // by themselves fp32 would lose them from -88 on, whatever they are to the largest.)
    float w = 0.0f;
    const float x = lane < a.K ? load1(a, (int64_t)t * a.ld + my_idx) : -INFINITY;
    bool by_exp = soft;
    if (a.renorm) {
        const float top = unordered(__reduce_max_sync(FULL, ordered(x)));
        by_exp = soft || (top < 0.0f && top > -700.0f);
        if (by_exp)
            m = top;
    }
    if (lane < a.K) {
        w = !by_exp ? 1.0f / (1.0f + expf(-x)) : x == m ? 1.0f : expf(x - m);
        if (by_exp && !soft)
            w /= 1.0f + expf(x);
    }
    if (a.renorm)
        z = warp_sum(w);
    if (soft || a.renorm)
        w = z > 0.0f ? w / z : 0.0f;
    my_w = w * a.scale;
}

// ------------------------------------------------------------------- grouping
//
// A token chooses an expert once at most, so the slots of 32 tokens are a word of bits for each expert: a slot's
// rank among its expert's is the number of bits below its token's.

// Exclusive sum of cnt[E] over the experts, in place, by the block; the total into cnt[E].
template <int WARPS>
__device__ __forceinline__ void scan_counts(int *cnt, int E)
{
    constexpr int PER = 32 * WARPS >= kMaxExperts ? 1 : kMaxExperts / (32 * WARPS);
    static_assert(PER * 32 * WARPS >= kMaxExperts, "experts of a thread");
    __shared__ int wsum[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int v[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v[i] = PER * tid + i < E ? cnt[PER * tid + i] : 0;
        sum += v[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o)
            incl += y;
    }
    if (lane == 31)
        wsum[warp] = incl;
    __syncthreads();
    int run = incl - sum + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? wsum[lane] : 0);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (PER * tid + i < E)
            cnt[PER * tid + i] = run;
        run += v[i];
    }
    if (tid == 32 * WARPS - 1)
        cnt[E] = run;
    __syncthreads();
}

// Dynamic shared memory of a selecting block: the warps' keys [warps][E], bits [E], counts [E + 1]; `words`: and for the
// last block's placing bits and places [E][words].
size_t smem_bytes(int warps, int E, int words = 0) { return (size_t)(warps * E + 2 * E + 1 + 2 * words * E) * 4; }

// All tokens' slots, at most kLastSlots, by one block of THREADS threads, the other blocks' choices among them.  cnt
// [E + 1], bits and places [E][a.words]: shared memory.
template <int THREADS>
__device__ __forceinline__ void place_all(const Args &a, int *cnt, uint32_t *bits, int *places)
{
    constexpr int EACH = kLastSlots / THREADS;  // slots of a thread
    static_assert(EACH * THREADS == kLastSlots, "slots");
    const int tid = threadIdx.x, n = a.T * a.K, W = a.words;
    int e[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        e[i] = tid + i * THREADS < n ? __ldcg(a.idx + tid + i * THREADS) : -1;
    for (int i = tid; i < a.E * W; i += THREADS)
        bits[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (e[i] >= 0) {
            const int t = (tid + i * THREADS) / a.K;
            atomicOr(bits + e[i] * W + (t >> 5), 1u << (t & 31));
        }
    __syncthreads();
    for (int x = tid; x < a.E; x += THREADS) {
        int run = 0;
        for (int w = 0; w < W; ++w) {
            places[x * W + w] = run;
            run += __popc(bits[x * W + w]);
        }
        cnt[x] = run;
        a.counts[x] = run;
    }
    __syncthreads();
    scan_counts<THREADS / 32>(cnt, a.E);
    for (int x = tid; x <= a.E; x += THREADS)
        a.offsets[x] = cnt[x];
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (e[i] >= 0) {
            const int s = tid + i * THREADS, t = s / a.K, at = e[i] * W + (t >> 5);
            a.perm[cnt[e[i]] + places[at] + __popc(bits[at] & ((1u << (t & 31)) - 1u))] = s;
        }
}

template <int P, int WARPS, bool GROUP>
__global__ void __launch_bounds__(32 * WARPS, many_warps(P) / WARPS) select_kernel(const Args a)
{
    constexpr int THREADS = 32 * WARPS;
    extern __shared__ __align__(16) uint32_t sm[];
    uint32_t *bits = sm + WARPS * a.E;
    int *cnt = reinterpret_cast<int *>(bits + a.E);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (the launch behind may set itself up; it waits for this one's end.  Plain loads: the read-only path is
    // not for a launch that began before its predecessor's end)
    pdl_trigger();
    if (GROUP) {
        for (int e = threadIdx.x; e < a.E; e += THREADS)
            bits[e] = cnt[e] = 0;
        __syncthreads();
    }
    const int64_t first = (int64_t)blockIdx.x * a.per;
    const int last = (int)min((int64_t)a.T, first + a.per);
    pdl_wait();
    int i = 0;
    for (int t = (int)first + warp; t < last; t += WARPS) {
        float w;
        select_token<P>(a, t, lane, sm + warp * a.E, i, w);
        if (lane < a.K) {
            a.idx[(int64_t)t * a.K + lane] = i;
            a.w[(int64_t)t * a.K + lane] = w;
            if (GROUP && !a.words)
                atomicAdd(cnt + i, 1);
            if (GROUP && a.runs <= 1)
                atomicOr(bits + i, 1u << warp);
        }
        __syncwarp();
    }
    if (!GROUP)
        return;
    if constexpr (WARPS == kWarps)  // (more warps are for more tokens than those)
        if (a.words) {
            // the last block to come here puts all slots in order
            __shared__ bool last_block;
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                last_block = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
                if (last_block)
                    *a.ticket = 0;  // (as the next call finds it)
            }
            __syncthreads();
            if (!last_block)
                return;
            __threadfence();
            uint32_t *all = reinterpret_cast<uint32_t *>(cnt + a.E + 1);
            place_all<THREADS>(a, cnt, all, reinterpret_cast<int *>(all + a.words * a.E));
            return;
        }
    __syncthreads();
    if (a.runs > 1) {
        for (int e = threadIdx.x; e < a.E; e += THREADS)
            a.bc[(int64_t)e * a.pitch + blockIdx.x] = (uint8_t)cnt[e];
        return;
    }
    // a warp a token, and no more than these
    for (int e = threadIdx.x; e < a.E; e += THREADS)
        a.counts[e] = cnt[e];
    scan_counts<WARPS>(cnt, a.E);
    for (int e = threadIdx.x; e <= a.E; e += THREADS)
        a.offsets[e] = cnt[e];
    if (warp < a.T && lane < a.K)
        a.perm[cnt[i] + __popc(bits[i] & ((1u << warp) - 1u))] = warp * a.K + lane;
}

__global__ void __launch_bounds__(32 * kPlaceWarps) place_kernel(const Args a)
{
    constexpr int THREADS = 32 * kPlaceWarps, SLOTS = 32 * kMaxTopK / THREADS;  // slots of a thread, of 32 tokens
    __shared__ uint32_t bits[kMaxExperts];
    __shared__ int cnt[kMaxExperts + 1], place[kMaxExperts];
    const int me = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int e = tid; e < a.E; e += THREADS)
        bits[e] = 0;
    const int64_t t0 = (int64_t)me * a.join * a.per, t1 = min((int64_t)a.T, t0 + (int64_t)a.join * a.per);
    pdl_wait();
    // slot tid + i * THREADS of the 32 tokens from t on
    int expert_of[SLOTS];
    auto load_slots = [&](int64_t t) {
        const int n = (int)min((int64_t)32, t1 - t) * a.K;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            expert_of[i] = tid + i * THREADS < n ? __ldcg(a.idx + t * a.K + tid + i * THREADS) : -1;
    };
    load_slots(t0);
    // All blocks' counts, and those of the blocks before this one's: `lanes` neighbouring lanes have an expert, a lane sixteen
    // neighbouring blocks at a time.  Each begins with another expert: in one order all met at the same lines
    // (4096 x 256: 20 us instead of 11).
    constexpr int BATCH = 4;
    const int mine = me * a.join, lanes = a.run_lanes, each = 32 / lanes, part = lane & (lanes - 1);
    const int turn = (int)((int64_t)me * a.E / gridDim.x);
    auto expert = [&](int i) { return i + turn < a.E ? i + turn : i + turn - a.E; };
    for (int i0 = warp * each + lane / lanes; i0 - lane / lanes < a.E; i0 += BATCH * kPlaceWarps * each) {
        unsigned all[BATCH] = {}, low[BATCH] = {};
        for (int r = 16 * part; r < a.runs; r += 16 * lanes) {
            uint4 v[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int i = i0 + b * kPlaceWarps * each;
                v[b] = make_uint4(0, 0, 0, 0);
                if (i < a.E)
                    v[b] = *reinterpret_cast<const uint4 *>(a.bc + (int64_t)expert(i) * a.pitch + r);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                auto ones = [&](int n) {  // a one for each of a word's first n bytes
                    return n >= 4 ? 0x01010101u : n > 0 ? 0x01010101u >> (8 * (4 - n)) : 0u;
                };
                const uint32_t in = ones(a.runs - r - 4 * i), under = ones(mine - r - 4 * i);
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    const uint32_t x = i == 0 ? v[b].x : i == 1 ? v[b].y : i == 2 ? v[b].z : v[b].w;
                    all[b] = __dp4a(x, in, all[b]);
                    low[b] = __dp4a(x, under, low[b]);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            for (int o = lanes >> 1; o; o >>= 1) {
                all[b] += __shfl_xor_sync(0xFFFFFFFFu, all[b], o);
                low[b] += __shfl_xor_sync(0xFFFFFFFFu, low[b], o);
            }
            const int i = i0 + b * kPlaceWarps * each;
            if (part == 0 && i < a.E) {
                cnt[expert(i)] = (int)all[b];
                place[expert(i)] = (int)low[b];
            }
        }
    }
    __syncthreads();
    if (me == 0)
        for (int e = tid; e < a.E; e += THREADS)
            a.counts[e] = cnt[e];
    if (me == 0)
        __syncthreads();
    scan_counts<kPlaceWarps>(cnt, a.E);
    if (me == 0)
        for (int e = tid; e <= a.E; e += THREADS)
            a.offsets[e] = cnt[e];
    for (int64_t t = t0; t < t1; t += 32) {
        int token[SLOTS];
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            token[i] = (tid + i * THREADS) / a.K;
            if (expert_of[i] >= 0)
                atomicOr(bits + expert_of[i], 1u << token[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int e = expert_of[i];
            if (e >= 0)
                a.perm[cnt[e] + place[e] + __popc(bits[e] & ((1u << token[i]) - 1u))] = (int)(t * a.K) + tid + i * THREADS;
        }
        if (t + 32 >= t1)
            break;
        load_slots(t + 32);
        __syncthreads();
        for (int e = tid; e < a.E; e += THREADS) {
            place[e] += __popc(bits[e]);
            bits[e] = 0;
        }
        __syncthreads();
    }
}

// Registers of a lane for E experts.
int width_of(int E)
{
    int P = 1;
    while (32 * P < E)
        P *= 2;
    return P;
}

// Warps and tokens of a selecting block when slots are grouped.
int group_warps(int T, int E)
{
    return T > kManyTokens ? many_warps(width_of(E)) : kWarps;
}
int run_tokens(int T, int E)
{
    const int warps = group_warps(T, E);
    if (warps == kWarps)
        return warps;
    const int64_t per = ((int64_t)T + kRuns - 1) / kRuns;
    return (int)std::min<int64_t>(kMaxRun, std::max<int64_t>(warps, (per + warps - 1) / warps * warps));
}
int runs_of(int T, int E) { return (int)(((int64_t)T + run_tokens(T, E) - 1) / run_tokens(T, E)); }

template <int P, int WARPS>
cudaError_t launch_grouped(const Args &a, cudaStream_t s)
{
    const size_t smem = smem_bytes(WARPS, a.E, a.words);
    cudaError_t e = smem_optin((const void *)select_kernel<P, WARPS, true>, smem);
    if (e != cudaSuccess)
        return e;
    e = launch_dependent(select_kernel<P, WARPS, true>, std::max(1, a.runs), 32 * WARPS, smem, s, a);
    if (e == cudaSuccess && a.runs > 1 && !a.words)
        e = launch_dependent(place_kernel, (a.runs + a.join - 1) / a.join, 32 * kPlaceWarps, 0, s, a);
    return e;
}

template <int P>
cudaError_t launch(const Args &a, cudaStream_t s)
{
    if (a.counts)
        return group_warps(a.T, a.E) == kWarps ? launch_grouped<P, kWarps>(a, s) : launch_grouped<P, many_warps(P)>(a, s);
    const int grid = (int)(((int64_t)a.T + kWarps - 1) / kWarps);
    return launch_dependent(select_kernel<P, kWarps, false>, grid, 32 * kWarps, smem_bytes(kWarps, a.E), s, a);
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

int pitch_of(int runs) { return (runs + 15) / 16 * 16; }

size_t ws_bytes_of(int E, int T)
{
    const int runs = runs_of(T, E);
    return kErrBytes + up256(runs > 1 ? (size_t)pitch_of(runs) * E : 0);
}

}  // namespace
}  // namespace sel
}  // namespace mx

using namespace mx;

extern "C" size_t mx_route_logits_workspace_bytes(const mx_router *router, int T_max)
{
    if (sel::check_router(router) != MX_OK)
        return 0;
    if (T_max < 0 || T_max > sel::kMaxTokens) {
        fail(MX_ERR_INVALID_ARG, "T_max %d must be in [0, 2^30]", T_max);
        return 0;
    }
    // (any number of tokens up to T_max: there are the more blocks the more tokens there are, up to kManyTokens and
    // from there to kRuns whole blocks and again when those are full)
    const int E = router->n_experts;
    return std::max({sel::ws_bytes_of(E, T_max), sel::ws_bytes_of(E, std::min(T_max, sel::kManyTokens)),
                     sel::ws_bytes_of(E, std::min(T_max, sel::kRuns * sel::many_warps(sel::width_of(E))))});
}

extern "C" mx_status mx_route_logits(const void *logits, int64_t ld, int dtype, int T, const mx_router *router,
                                     int32_t *topk_idx, float *topk_w, int32_t *counts, int32_t *offsets, int32_t *perm,
                                     void *stream, void *ws, size_t ws_bytes)
{
    mx_status st;
    if ((st = sel::check_router(router)) != MX_OK || (st = check_dtype(dtype, "dtype")) != MX_OK)
        return st;
    const int E = router->n_experts, K = router->top_k;
    if (T < 0 || T > sel::kMaxTokens || (int64_t)T * K > 0x7FFFFFFF)
        return fail(MX_ERR_INVALID_ARG, "T %d must be in [0, 2^30], T * top_k below 2^31", T);
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
        a.bc = static_cast<uint8_t *>(ws) + kErrBytes;
        a.ticket = static_cast<unsigned *>(ws) + 16;  // (of the error word's 256 bytes)
        a.runs = sel::runs_of(T, E);
        a.words = T > sel::kWarps && (int64_t)T * K <= sel::kLastSlots && T <= 512 ? (T + 31) / 32 : 0;  // (bits of 512 tokens)
        a.pitch = sel::pitch_of(a.runs);
        // (32 tokens to a placing block, more from kPlaceBlocks on)
        a.join = std::max(32 / sel::run_tokens(T, E), (a.runs + sel::kPlaceBlocks - 1) / sel::kPlaceBlocks);
        a.run_lanes = 1;
        while (a.run_lanes < 32 && 16 * a.run_lanes < a.runs)
            a.run_lanes *= 2;
    }
    a.per = group ? sel::run_tokens(T, E) : sel::kWarps;
    const int P = sel::width_of(E);
    const int size = E / a.n_groups, lanes = size / P;
    a.lanes = size % P == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    const size_t piece = std::min<size_t>(16, P * dtype_bytes(dtype));
    a.vec = E == 32 * P && aligned(logits, piece) && ld * dtype_bytes(dtype) % piece == 0;
    a.vec_bias = E == 32 * P && aligned(a.bias, 16);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = P == 1   ? sel::launch<1>(a, s)
                          : P == 2 ? sel::launch<2>(a, s)
                          : P == 4 ? sel::launch<4>(a, s)
                          : P == 8 ? sel::launch<8>(a, s)
                                   : sel::launch<16>(a, s);
    return e == cudaSuccess ? MX_OK : cuda_fail(e, "routing");
}
