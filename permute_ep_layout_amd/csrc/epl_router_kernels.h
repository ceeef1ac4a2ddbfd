// Device kernels of the router and its gradient for gfx950 (CDNA4): scores,
// the choice of top-k experts (with a bias and groups), their weights; and
// the gradient of the logits from the weights'.
//
// The choice needs an exact order, so every candidate is one binary64 key:
// its choice score with the low 11 bits of the significand replaced by the
// expert's index, such that of two equal scores the lower index has the
// larger key. Keys are then all different, one v_max_f64 both compares and
// carries the index, and the selection is a sorting network on registers.
// Without a bias (and without sums of two) the score is the logit itself,
// which orders the experts as any score does and leaves the low 29 bits of a
// binary64 free: the order is exact. With them scores are compared as
// binary64 numbers, good to about 2^-44, to 41 bits. They are first computed
// in binary32; where two that matter lie within its error of each other, the
// choice is done again in binary64: 1 or 2 tokens in a thousand with binary32
// logits, but every third where scores tie, as those of bf16 logits do with a
// bias of zero (65536 tokens, 256 experts: 94 us, not 28; of 4 of 8 groups 115,
// not 35). Equal logits with equal biases would need no second look.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epl.h"

namespace epl_router_k {

constexpr int kMaxExperts = 2048;
constexpr int kMaxTopk = 64;
constexpr int kMaxGroups = 64;
constexpr int kThreads = 256;
constexpr uint64_t kIndexMask = 2047;

struct Args {
    const void *logits;
    const float *bias;             // [E] or null
    const uint8_t *mask;           // [T] or null
    int64_t *idx;                  // [T, K]
    float *w;                      // [T, K]
    int64_t T;
    int K, E, G, topk_groups, group_top;
    int per_log;                   // log2 of a group's pieces of 8 experts (route_kernel)
    bool softmax, renorm, bf16, need_scores, vec, bias_vec;
    float scale;
};

struct GradArgs {
    const void *logits;
    const int64_t *idx;
    const float *g;                // [T, K] d weights
    void *out;                     // [T, E] d logits
    int64_t T;
    int K, E;
    bool softmax, renorm, bf16, vec;
    float scale;
};

// exp(x) in binary64 to a few units of 2^-47: x = n ln 2 + r with |r| <=
// ln 2 / 2 (ln 2 in the two words of fdlibm's e_exp.c), the Taylor polynomial
// of degree 11 in r (its remainder is below 2^-47), and an exponent shift.
__device__ __forceinline__ double exp64(double x)
{
    x = fmin(fmax(x, -700.0), 700.0);
    const double n = __builtin_rint(x * 1.4426950408889634074);
    double r = fma(n, -6.93147180369123816490e-01, x);
    r = fma(n, -1.90821492927058770002e-10, r);
    double p = 1.0 / 39916800.0;
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}

// 1 / d for finite positive d: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double rcp64(double d)
{
    double y = __builtin_amdgcn_rcp(d);
    y = fma(fma(-d, y, 1.0), y, y);
    return fma(fma(-d, y, 1.0), y, y);
}

// 0 below -700, where exp64 stops growing. (No branch: a select of the
// finished value. A branch an element made the choice twice as slow.)
__device__ __forceinline__ double sigmoid64(double x)
{
    const double s = rcp64(1.0 + exp64(-x));
    return x < -700.0 ? 0.0 : s;
}

// +inf competes as the largest finite logit; a NaN stays one.
__device__ __forceinline__ float no_inf(float v) { return v > 3.402823466e+38f ? 3.402823466e+38f : v; }

__device__ __forceinline__ float load_logit(const void *p, bool bf16, int64_t at)
{
    return no_inf(bf16 ? (float)static_cast<const __bf16 *>(p)[at]
                       : static_cast<const float *>(p)[at]);
}

// Keys at or below it are no candidates; every score's key is above it, the
// lowest finite binary32 too.
constexpr double kNone = -1e300;

// The key of a score, or one that is no candidate.
__device__ __forceinline__ double make_key(double score, int index, bool candidate)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, score + 0.0);      // -0 becomes +0
    const uint32_t hi = (uint32_t)(u >> 32);
    // of a negative score the larger index has the larger magnitude
    const uint32_t flip = (uint32_t)((int32_t)hi >> 31) & (uint32_t)kIndexMask;
    const uint32_t lo = ((uint32_t)u & ~(uint32_t)kIndexMask) |
                        (((uint32_t)kIndexMask - (uint32_t)index) ^ flip);
    return __builtin_bit_cast(double, ((uint64_t)(candidate ? hi : 0xffefffffu) << 32) | lo);
}

__device__ __forceinline__ int key_index(double key)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, key);
    const int tail = (int)(u & kIndexMask);
    return (u >> 63) ? tail : (int)kIndexMask - tail;
}

// What orders the experts: the logits themselves, or scores (with a bias, or
// summed over groups).
enum Order { kLogits, kSigmoid, kSoftmax };

// Whether an expert may be chosen, by its logit and its bias.
__device__ __forceinline__ bool usable(float l, float bias) { return l > -INFINITY && bias > -INFINITY; }

// Choice score of a logit. `m` and `inv` are the row's largest logit and 1 /
// sum of exponentials.
template <Order ORDER>
__device__ __forceinline__ double exact_score(float l, float bias, double m, double inv)
{
    if constexpr (ORDER == kLogits)
        return (double)l;
    else if constexpr (ORDER == kSoftmax)
        return exp64((double)l - m) * inv + (double)no_inf(bias);
    else
        return sigmoid64((double)l) + (double)no_inf(bias);
}

// The key of the choice score in binary32, which make_key would give for it,
// in fewer instructions: the score's binary64 has its low 29 bits clear, and a
// sum with a score that is not negative is never -0. Of sigmoids `l` may be
// +inf, which gives the same 1 as the largest finite logit.
template <Order ORDER>
__device__ __forceinline__ double fast_key(float l, float bias, float m, float inv, int index)
{
    float s;
    bool candidate = l > -INFINITY;
    if constexpr (ORDER == kLogits) {
        s = l + 0.0f;                                                // -0 becomes +0
    } else {
        const float p = ORDER == kSoftmax ? __expf(l - m) * inv
                                          : __builtin_amdgcn_rcpf(1.0f + __expf(-l));
        const float sum = p + bias;
        candidate &= sum > -INFINITY;                                // a NaN of either neither
        s = __builtin_amdgcn_fmed3f(sum, -3.402823466e+38f, 3.402823466e+38f);
    }
    const uint64_t u = __builtin_bit_cast(uint64_t, (double)s);
    const uint32_t hi = (uint32_t)(u >> 32);
    const uint32_t flip = (uint32_t)((int32_t)hi >> 31) & (uint32_t)kIndexMask;
    const uint32_t lo = (uint32_t)u | (((uint32_t)kIndexMask - (uint32_t)index) ^ flip);
    return __builtin_bit_cast(double, ((uint64_t)(candidate ? hi : 0xffefffffu) << 32) | lo);
}

// How far two choice scores in binary32 must lie apart for their order to be
// sure, given the larger one's magnitude and the row's largest score s. Of a
// sigmoid: exp and the reciprocal are good to a step each and the argument's
// rounding passes on s (1 - s) |l| < 1/4 of a step, in all below 4 2^-24 s,
// for either score; a softmax's exponentials are off by (2 |x| + 4) 2^-24 of
// themselves, below 5 2^-24 of the largest score, and their sum by 2 ln E + 4
// of that at most; the sum with the bias half a step. Doubled, and rounded up.
template <Order ORDER>
__device__ __forceinline__ double margin(double c, double top)
{
    return (ORDER == kSoftmax ? 0x1p-17 : 0x1p-20) * top + 0x1p-21 * fabs(c);
}

// ---- register sorting ------------------------------------------------------

__device__ __forceinline__ void desc(double &a, double &b)
{
    const double hi = fmax(a, b), lo = fmin(a, b);
    a = hi;
    b = lo;
}

// Batcher's odd-even merge sort of 8 keys, descending (19 exchanges).
__device__ __forceinline__ void sort8(double (&k)[8])
{
    desc(k[0], k[1]); desc(k[2], k[3]); desc(k[4], k[5]); desc(k[6], k[7]);
    desc(k[0], k[2]); desc(k[1], k[3]); desc(k[4], k[6]); desc(k[5], k[7]);
    desc(k[1], k[2]); desc(k[5], k[6]);
    desc(k[0], k[4]); desc(k[1], k[5]); desc(k[2], k[6]); desc(k[3], k[7]);
    desc(k[2], k[4]); desc(k[3], k[5]);
    desc(k[1], k[2]); desc(k[3], k[4]); desc(k[5], k[6]);
}

// The 8 largest of two descending lists, descending: the larger of a[i] and
// b[7 - i] over i is a bitonic sequence of the 8 largest.
__device__ __forceinline__ void merge8(double (&a)[8], const double (&b)[8])
{
    double c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c[i] = fmax(a[i], b[7 - i]);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d))
                desc(c[i], c[i + d]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a[i] = c[i];
}

// The value of the lane `D` away (the lane number's bit D flipped, for lists
// that are alike within blocks of D lanes): DPP moves within 16 lanes, a
// permute above.
template <int D>
__device__ __forceinline__ int lane_swap(int v)
{
    if constexpr (D == 1)
        return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);          // quad_perm 1 0 3 2
    else if constexpr (D == 2)
        return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);          // quad_perm 2 3 0 1
    else if constexpr (D == 4)
        return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);         // row_half_mirror
    else if constexpr (D == 8)
        return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);         // row_mirror
    else
        return __shfl_xor(v, D);
}
template <int D>
__device__ __forceinline__ float lane_swap(float v)
{
    return __builtin_bit_cast(float, lane_swap<D>(__builtin_bit_cast(int, v)));
}
template <int D>
__device__ __forceinline__ double lane_swap(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)lane_swap<D>((int)(uint32_t)u);
    const uint32_t hi = (uint32_t)lane_swap<D>((int)(uint32_t)(u >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// f(v, v of the other half) over blocks of L lanes: all lanes get the same.
template <int L, int D = 1, typename V, typename F>
__device__ __forceinline__ V all_lanes(V v, F f)
{
    if constexpr (D < L)
        return all_lanes<L, D * 2>(f(v, lane_swap<D>(v)), f);
    else
        return v;
}
template <int L, typename V>
__device__ __forceinline__ V lane_max(V v)
{
    return all_lanes<L>(v, [](V a, V b) { return a > b ? a : b; });
}
template <int L, typename V>
__device__ __forceinline__ V lane_sum(V v)
{
    return all_lanes<L>(v, [](V a, V b) { return a + b; });
}

template <int L, int D = 1>
__device__ __forceinline__ void merge_lanes(double (&k)[8])
{
    if constexpr (D < L) {
        double o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = lane_swap<D>(k[i]);
        merge8(k, o);
        merge_lanes<L, D * 2>(k);
    }
}

__device__ __forceinline__ void two_best(double &a, double &b, double c, double d)
{
    const double lo = fmin(a, c);
    a = fmax(a, c);
    b = fmax(lo, fmax(b, d));
}

// A group's score from its two best keys (a group of one candidate has that
// one, a group of none -infinity), and how far another's must lie from it, as
// the low and the high half of 8 bytes. (As a struct it went through memory.)
// The error of a sum follows its terms, not the sum: biases may cancel in it.
// Both are halved where scores add, so that no sum leaves binary32; the
// rounding of the sum fits into the margins, which are twice the errors.
template <Order ORDER>
__device__ __forceinline__ double group_score(const Args &a, double best, double next, double top)
{
    const bool two = a.group_top == 2 && next > kNone;
    const double half = ORDER == kLogits ? 1.0 : 0.5;
    const double sum = two ? best + next : best;
    const double near = margin<ORDER>(best, top) + (two ? margin<ORDER>(next, top) : 0.0);
    const uint32_t lo = __builtin_bit_cast(uint32_t, (float)(half * sum));
    const uint32_t hi = __builtin_bit_cast(uint32_t, best > kNone ? (float)(half * near) : 0.0f);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float score_half(double g)
{
    return __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(uint64_t, g));
}
__device__ __forceinline__ float near_half(double g)
{
    return __builtin_bit_cast(float, (uint32_t)(__builtin_bit_cast(uint64_t, g) >> 32));
}

// A finite score to 40 significant bits, to nearest even: what binary64 and the
// order of a sum leave uncertain of equal sums is far below.
__device__ __forceinline__ double round40(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (u + 0xfff + ((u >> 13) & 1)) & ~(uint64_t)0x1fff);
}

// LDS operations of one wave are in order: this keeps the compiler's order.
__device__ __forceinline__ void wave_lds() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local"); }

// Logits of 8 neighbouring experts; -inf past the row's end. CLAMP: no_inf.
template <bool CLAMP = true>
__device__ __forceinline__ void load8(const void *p, bool bf16, bool vec, int64_t row, int E, int e0,
                                      float (&v)[8])
{
    const int64_t at = row * E + e0;
    if (vec && e0 + 8 <= E) {
        if (bf16) {
            typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
            const bf16x8 r = *reinterpret_cast<const bf16x8 *>(static_cast<const __bf16 *>(p) + at);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = CLAMP ? no_inf((float)r[i]) : (float)r[i];
        } else {
            const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
            const float4 y = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at + 4);
            const float t[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = CLAMP ? no_inf(t[i]) : t[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = e0 + i < E ? load_logit(p, bf16, at + i) : -INFINITY;
}

// A logit that takes part: NaN counts as -inf.
__device__ __forceinline__ float usable(float l) { return l > -INFINITY ? l : -INFINITY; }

// Weights of the chosen experts in lanes k = 0 .. K - 1 of a block of at
// least K lanes: `l` is the chosen logit (-inf: no expert).
template <int L>
__device__ __forceinline__ float weight_of(const Args &a, float l, double m, double inv)
{
    double s;
    if (a.softmax) {
        // the row's sum drops out of renormalised weights: the chosen
        // logits' own maximum keeps their ratios from underflowing
        const double top = a.renorm ? (double)lane_max<L>(l) : m;
        s = l > -INFINITY ? exp64((double)l - top) : 0.0;
        if (!a.renorm)
            s *= inv;
    } else {
        s = l > -INFINITY ? sigmoid64((double)l) : 0.0;
    }
    if (a.renorm) {
        const double d = lane_sum<L>(s);
        s = d > 0.0 ? s / d : 0.0;
    }
    return (float)(s * (double)a.scale);
}

// ---- any top-k, any groups: a wave a token, its keys in LDS ----------------
//
// Scores in binary64; K rounds, each the largest key below the last round's.
// For sizes that the kernel below does not cover (K above 8, groups that end
// inside a piece), and for its tokens whose choice binary32 leaves in doubt.
// 16384 tokens, top-10 of 512 experts: 107 - 110 us; top-6 of 160 in 8 groups:
// 49 - 55 us; by the K rounds over LDS and the binary64 scores.
__device__ __forceinline__ void route_token(const Args &a, int64_t t, int lane, double *key,
                                            double *score)
{
    double m = 0.0, inv = 1.0;
    if (a.softmax) {
        float mx = -INFINITY;
        for (int e = lane; e < a.E; e += 64)
            mx = fmaxf(mx, usable(load_logit(a.logits, a.bf16, t * a.E + e)));
        mx = lane_max<64>(mx);
        m = mx > -INFINITY ? (double)mx : 0.0;
        double s = 0.0;
        for (int e = lane; e < a.E; e += 64) {
            const float l = load_logit(a.logits, a.bf16, t * a.E + e);
            const double x = exp64((double)l - m);
            s += l > -INFINITY ? x : 0.0;
        }
        s = lane_sum<64>(s);
        inv = s > 0.0 ? 1.0 / s : 0.0;
    }
    const auto score_of = [&](float l, float bias) {
        return !a.need_scores ? exact_score<kLogits>(l, bias, m, inv)
               : a.softmax    ? exact_score<kSoftmax>(l, bias, m, inv)
                              : exact_score<kSigmoid>(l, bias, m, inv);
    };
    if (a.G == 1) {
        for (int e = lane; e < a.E; e += 64) {
            const float b = a.bias ? a.bias[e] : 0.0f;
            const float l = load_logit(a.logits, a.bf16, t * a.E + e);
            key[e] = make_key(score_of(l, b), e, usable(l, b));
        }
        wave_lds();
    } else {
        // `per` lanes a group, a power of two: the two best of its scores,
        // which are full ones yet (keys drop their low bits)
        const int per = 1 << (31 - __builtin_clz(64 / a.G)), size = a.E / a.G;
        const int g = lane / per, first = lane % per, e0 = g * size;
        double x = 2.0 * kNone, y = x;
        int ex = 0, ey = 0;
        const auto take = [&](double c, int e) {
            const bool best = c > x, next = c > y;
            y = best ? x : next ? c : y;
            ey = best ? ex : next ? e : ey;
            x = best ? c : x;
            ex = best ? e : ex;
        };
        if (g < a.G)
            for (int i = first; i < size; i += per) {
                const int e = e0 + i;
                const float b = a.bias ? a.bias[e] : 0.0f;
                const float l = load_logit(a.logits, a.bf16, t * a.E + e);
                const double c = usable(l, b) ? score_of(l, b) : 2.0 * kNone;
                key[e] = c;
                take(c, e);
            }
        for (int d = 1; d < per; d <<= 1) {
            const double ox = __shfl_xor(x, d), oy = __shfl_xor(y, d);
            const int oex = __shfl_xor(ex, d), oey = __shfl_xor(ey, d);
            take(ox, oex);
            take(oy, oey);
        }
        double own = x;
        if (a.group_top == 2 && y > kNone) {
            // scores and biases apart: two groups may hold the same ones
            // paired otherwise, and these sums are equal then
            const double bias = a.bias ? (double)no_inf(a.bias[ex]) + (double)no_inf(a.bias[ey]) : 0.0;
            own = (score_of(load_logit(a.logits, a.bf16, t * a.E + ex), 0.0f) +
                   score_of(load_logit(a.logits, a.bf16, t * a.E + ey), 0.0f)) + bias;
        }
        if (a.need_scores)
            own = round40(own);
        if (g < a.G && first == 0)
            score[g] = own;
        wave_lds();
        own = score[g];              // (lanes may have summed equal scores differently)
        // a total order, so that topk_groups of them stay whatever lies close
        int before = 0;
        for (int o = first; o < a.G; o += per)
            before += score[o] > own || (score[o] == own && o < g) ? 1 : 0;
        for (int d = 1; d < per; d <<= 1)
            before += __shfl_xor(before, d);
        if (g < a.G)
            for (int e = e0 + first; e < e0 + size; e += per)
                key[e] = make_key(key[e], e, before < a.topk_groups && key[e] > kNone);
        wave_lds();
    }
    const bool live = !a.mask || a.mask[t] != 0;
    double last = INFINITY;
    int mine = -1;
    for (int k = 0; k < a.K; ++k) {
        double x = 2.0 * kNone;
        for (int e = lane; e < a.E; e += 64) {
            const double v = key[e];
            x = v < last && v > x ? v : x;
        }
        last = lane_max<64>(x);
        mine = lane == k && live && last > kNone ? key_index(last) : mine;
    }
    const float l = mine >= 0 ? load_logit(a.logits, a.bf16, t * a.E + mine) : -INFINITY;
    const float w = weight_of<64>(a, l, m, inv);
    if (lane < a.K) {
        a.idx[t * a.K + lane] = mine;
        a.w[t * a.K + lane] = mine >= 0 ? w : 0.0f;
    }
    wave_lds();
}

__global__ __launch_bounds__(64) void route_any_kernel(Args a)
{
    __shared__ double key[kMaxExperts];
    __shared__ double score[kMaxGroups];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x)
        route_token(a, t, threadIdx.x, key, score);
}

// ---- top-k of at most 8, L lanes a token, CH pieces of 8 experts a lane ----
//
// Piece c of lane i holds experts (c L + i) 8 .. + 7. Each lane sorts its
// pieces, merges them to its 8 best, and log2(L) merges across lanes leave
// the token's 8 best, in order, in every lane. Bound by its vector
// instructions: 65536 tokens x 256 experts in binary32 take 20 us by sigmoid
// (3.6 TB/s) and 35 us with a bias and 4 of 8 groups besides (2.1 TB/s), 1600
// instructions a wave of 8 tokens, which issue in 84% of its cycles.

// The token's 8 best keys in every lane; false, on one of its lanes at least,
// where the error of binary32 leaves their order in doubt. `groups` (of
// group_score) and `gone`: the token's LDS, of kMaxGroups each.
template <int L, int CH, Order ORDER>
__device__ __forceinline__ bool choose(const Args &a, const float (&l)[CH][8], int lane, float m,
                                       float inv, double *groups, int *gone, double (&best)[8])
{
    const double top = ORDER == kSoftmax ? (double)inv : 1.0;
    double key[CH][8];
    bool sure = true;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int e0 = (c * L + lane) * 8;
        float b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (a.bias) {
            if (e0 + 8 <= a.E && a.bias_vec) {
                const float4 x = *reinterpret_cast<const float4 *>(a.bias + e0);
                const float4 y = *reinterpret_cast<const float4 *>(a.bias + e0 + 4);
                b[0] = x.x, b[1] = x.y, b[2] = x.z, b[3] = x.w;
                b[4] = y.x, b[5] = y.y, b[6] = y.z, b[7] = y.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    b[i] = e0 + i < a.E ? a.bias[e0 + i] : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            key[c][i] = fast_key<ORDER>(l[c][i], b[i], m, inv, e0 + i);
        sort8(key[c]);
    }
    if (a.G > 1) {
        // pieces lie within groups of `per` pieces (a power of two): the two
        // best keys of a group by exchanges; lane g then ranks group g
        const int per = 1 << a.per_log;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            double x = key[c][0], y = key[c][1];
            if (per > 1) { two_best(x, y, lane_swap<1>(x), lane_swap<1>(y)); }
            if (per > 2) { two_best(x, y, lane_swap<2>(x), lane_swap<2>(y)); }
            if constexpr (L > 4)
                if (per > 4) { two_best(x, y, lane_swap<4>(x), lane_swap<4>(y)); }
            if constexpr (L > 8)
                if (per > 8) { two_best(x, y, lane_swap<8>(x), lane_swap<8>(y)); }
            if constexpr (L > 16)
                if (per > 16) { two_best(x, y, lane_swap<16>(x), lane_swap<16>(y)); }
            if constexpr (L > 32)
                if (per > 32) { two_best(x, y, lane_swap<32>(x), lane_swap<32>(y)); }
            const int piece = c * L + lane;
            if ((piece & (per - 1)) == 0 && piece >> a.per_log < a.G)
                groups[piece >> a.per_log] = group_score<ORDER>(a, x, y, top);
        }
        wave_lds();
        for (int g = lane; g < a.G; g += L) {
            const float own = score_half(groups[g]), near = near_half(groups[g]);
            int before = 0, close = 0;
            for (int o = 0; o < a.G; ++o) {
                const float s = score_half(groups[o]), far = near_half(groups[o]);
                before += (int)(s > own) | ((int)(s == own) & (int)(o < g));
                if (ORDER != kLogits)
                    close += (int)(fabsf(s - own) <= fmaxf(near, far));
            }
            gone[g] = before >= a.topk_groups;
            // the last group that stays must stand clear of the others
            if (ORDER != kLogits)
                sure &= !(before == a.topk_groups - 1 && close > 1 && own > -INFINITY);
        }
        wave_lds();
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            // (a sum: half the instructions of a select)
            const double out = gone[min((c * L + lane) >> a.per_log, a.G - 1)] ? -1e308 : 0.0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                key[c][i] += out;
        }
        wave_lds();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        best[i] = key[0][i];
#pragma unroll
    for (int c = 1; c < CH; ++c)
        merge8(best, key[c]);
    merge_lanes<L>(best);
    if (ORDER == kLogits)
        return true;

    // The chosen stand clear of each other and, counted, of the rest.
    double last = 0.0;
    int over = 0, want = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool is = i < a.K && best[i] > kNone;
        if (i > 0)
            sure &= !is || best[i > 0 ? i - 1 : 0] - best[i] > margin<ORDER>(best[i > 0 ? i - 1 : 0], top);
        last = is ? best[i] : last;
        want += (int)is;
    }
    const double bar = last - margin<ORDER>(last, top);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            over += (int)(key[c][i] >= bar);
    const int all = lane_sum<L>(over);
    return sure & (want == 0 || all == want);
}

template <int L, int CH, Order ORDER>
__global__ __launch_bounds__(kThreads) void route_kernel(Args a)
{
    constexpr int TOK = kThreads / L;
    __shared__ double groups[TOK][kMaxGroups];
    __shared__ int gone[TOK][kMaxGroups];
    __shared__ double again[ORDER == kLogits ? 1 : kThreads / 64][ORDER == kLogits ? 1 : L * CH * 8];
    const int lane = threadIdx.x % L, slot = threadIdx.x / L;
    const int64_t t = (int64_t)blockIdx.x * TOK + slot;
    const bool in = t < a.T;
    const int64_t row = in ? t : a.T - 1;

    float l[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c)
        load8<ORDER != kSigmoid>(a.logits, a.bf16, a.vec, row, a.E, (c * L + lane) * 8, l[c]);

    float m = 0.0f, inv = 1.0f;
    double over = 1.0;
    if (ORDER == kSoftmax || (ORDER == kLogits && a.softmax && !a.renorm)) {
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                mx = fmaxf(mx, l[c][i]);             // (fmaxf passes over a NaN)
        mx = lane_max<L>(mx);
        m = mx > -INFINITY ? mx : 0.0f;
        // Exponentials in binary32, by pieces; the pieces' sums and the inverse
        // in binary64, so that the weights are rounded once: what errors of
        // some steps leave of a sum of many terms is a fraction of a step.
        double s = 0.0;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = l[c][i] > -INFINITY ? __expf(l[c][i] - m) : 0.0f;
            s += (double)(((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7])));
        }
        s = lane_sum<L>(s);
        over = s > 0.0 ? rcp64(s) : 0.0;
        inv = (float)over;
    }

    double best[8];
    const bool sure = choose<L, CH, ORDER>(a, l, lane, m, inv, groups[slot], gone[slot], best);

    // lane k keeps the k-th best
    double mine = 2.0 * kNone;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        mine = lane == i ? best[i] : mine;
    const bool live = in && lane < a.K && (!a.mask || a.mask[row] != 0);
    const bool found = live && mine > kNone;
    const int e = found ? key_index(mine) : -1;
    const float chosen = found ? load_logit(a.logits, a.bf16, row * a.E + e) : -INFINITY;
    const float w = weight_of<L>(a, chosen, (double)m, over);
    constexpr uint64_t lanes = L == 64 ? ~0ull : (1ull << (L % 64)) - 1;      // of a token
    uint64_t doubt = ORDER == kLogits ? 0 : __builtin_amdgcn_ballot_w64(!sure && in);
    if (in && lane < a.K && ((doubt >> (threadIdx.x % 64 - lane)) & lanes) == 0) {
        a.idx[t * a.K + lane] = e;
        a.w[t * a.K + lane] = found ? w : 0.0f;
    }
    if constexpr (ORDER != kLogits) {
        // tokens in doubt, one after the other, by the whole wave
        const int wave = threadIdx.x / 64;
        const int64_t t0 = (int64_t)blockIdx.x * TOK + wave * (64 / L);
        while (doubt != 0) {
            const int which = __builtin_ctzll(doubt) / L;
            doubt &= ~(lanes << (which * L % 64));
            route_token(a, t0 + which, threadIdx.x % 64, again[wave], groups[wave * (64 / L)]);
        }
    }
}

// ---- gradient of the logits ------------------------------------------------
//
// With p the scores, chosen experts i_k, g_k = scale * d w_k:
//   renormalised: h_k = g_k - sum_j (p_j / D) g_j over the chosen, D their sum
//       softmax: d l_{i_k} = (p_k / D) h_k, zero elsewhere (the sum over all
//                experts drops out of the ratios)
//       sigmoid: d l_{i_k} = (p_k / D) (1 - p_k) h_k, zero elsewhere
//   plain: sigmoid: d l_{i_k} = p_k (1 - p_k) g_k
//          softmax: d l_i = p_i (d p_i - sum_j p_j d p_j) for every expert
// Slots that name the same expert add up. L lanes a token: each lane makes a
// share of the K slots' values, puts them in LDS, and writes its pieces of 8
// experts by comparing their indices with the slots'. Bound by memory:
// 65536 x 256 in binary32, 23 us (4.7 TB/s); 16384 x 256 in bf16, 8.6 us, of
// which 4 are its start and the two dependent reads. (A row built up in LDS
// took 23.4 us for the first, and 34.8 against 29.5 for the dense softmax.)
template <int L, int CH>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(GradArgs a)
{
    constexpr int TOK = kThreads / L;
    __shared__ float val[TOK][kMaxTopk], grad[TOK][kMaxTopk];
    __shared__ int who[TOK][kMaxTopk];
    const int lane = threadIdx.x % L, slot = threadIdx.x / L;
    const int64_t t = (int64_t)blockIdx.x * TOK + slot;
    const bool in = t < a.T;
    const int64_t row = in ? t : a.T - 1;
    const bool dense = a.softmax && !a.renorm;

    float p[CH][8];
    float m = 0.0f, inv = 0.0f;
    if (dense) {
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            load8(a.logits, a.bf16, a.vec, row, a.E, (c * L + lane) * 8, p[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                mx = fmaxf(mx, usable(p[c][i]));
        }
        mx = lane_max<L>(mx);
        m = mx > -INFINITY ? mx : 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[c][i] = p[c][i] > -INFINITY ? __expf(p[c][i] - m) : 0.0f;
                s += p[c][i];
            }
        s = lane_sum<L>(s);
        inv = s > 0.0f ? 1.0f / s : 0.0f;
    }

    // The slots' logits and gradients, read once; and the chosen logits'
    // maximum, from which the scores of a renormalised choice are taken: only
    // their ratios matter, and scores that all leave binary32 (sigmoids of
    // logits below -87) have some too.
    float top = -INFINITY;
    const float floor = a.softmax ? -INFINITY : -700.0f;       // scores below it are 0 (sigmoid64)
    const auto scored = [&](float l) { return l > -INFINITY && l >= floor; };
    for (int k = lane; k < a.K; k += L) {
        const int64_t e = a.idx[row * a.K + k];
        const bool live = e >= 0 && e < a.E;
        const float l = live ? load_logit(a.logits, a.bf16, row * a.E + e) : -INFINITY;
        who[slot][k] = live ? (int)e : -1;
        val[slot][k] = l;
        grad[slot][k] = live ? a.g[row * a.K + k] * a.scale : 0.0f;
        top = fmaxf(top, scored(l) ? l : -INFINITY);
    }
    if (a.renorm)
        top = lane_max<L>(top);
    // The score of a chosen logit; of a renormalised choice over that of
    // `top` (a sigmoid's: over exp(top) where that is below 1). A sigmoid is
    // exp(min(l, 0)) / (1 + exp(-|l|)).
    const float from = !a.renorm || top == -INFINITY ? 0.0f : a.softmax ? top : fminf(top, 0.0f);
    const auto share = [&](float l) {
        return a.softmax ? __expf(l - from)
                         : __expf(fminf(l, 0.0f) - from) / (1.0f + __expf(-fabsf(l)));
    };
    float sum = 0.0f, dot = 0.0f;
    for (int k = lane; k < a.K; k += L) {
        const float l = val[slot][k];
        float s = 0.0f;
        if (scored(l))
            s = dense ? __expf(l - m) * inv : share(l);
        sum += s;
        dot += s * grad[slot][k];
    }
    sum = lane_sum<L>(sum);
    dot = lane_sum<L>(dot);
    const float over = a.renorm ? (sum > 0.0f ? 1.0f / sum : 0.0f) : 1.0f;
    const float mean = a.renorm ? dot * over : 0.0f;
    for (int k = lane; k < a.K; k += L) {
        const float l = val[slot][k];
        float d = 0.0f;
        if (scored(l)) {
            d = grad[slot][k] - mean;
            if (!dense) {
                d *= share(l) * over;
                if (!a.softmax)
                    d /= 1.0f + __expf(l);                  // 1 - s without cancellation
            }
        }
        val[slot][k] = d;
    }
    __syncthreads();
    if (!in)
        return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int e0 = (c * L + lane) * 8;
        if (e0 >= a.E)
            break;
        float d[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int k = 0; k < a.K; ++k) {
            const int at = who[slot][k] - e0;
            const float v = val[slot][k];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] += at == i ? v : 0.0f;
        }
        if (dense)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] = p[c][i] * inv * (d[i] - dot);
        const int64_t at = t * a.E + e0;
        if (a.vec && e0 + 8 <= a.E) {
            if (a.bf16) {
                typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
                bf16x8 r;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] = (__bf16)d[i];
                *reinterpret_cast<bf16x8 *>(static_cast<__bf16 *>(a.out) + at) = r;
            } else {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at);
                o[0] = make_float4(d[0], d[1], d[2], d[3]);
                o[1] = make_float4(d[4], d[5], d[6], d[7]);
            }
        } else {
            for (int i = 0; i < 8 && e0 + i < a.E; ++i) {
                if (a.bf16)
                    static_cast<__bf16 *>(a.out)[at + i] = (__bf16)d[i];
                else
                    static_cast<float *>(a.out)[at + i] = d[i];
            }
        }
    }
}

}  // namespace epl_router_k
