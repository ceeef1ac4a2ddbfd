// Device kernels of the experts' matrix products for gfx950 (CDNA4): the
// product of each expert's block of rows with that expert's weight, and its
// gradients.
//
// All of them are one contraction per expert,
//     out[m, n] = sum_k P[m, k] * Q[n, k],   n contiguous in memory,
// and differ in which operand has its contraction index contiguous:
//     forward        P = rows [M, K]             Q = weight [N, K]
//     data gradient  P = rows [M, K]             Q = weight [K, N]  (strided)
//     weight grad.   P = d rows [K, M] (strided) Q = rows [K, N]    (strided)
// The matrix instruction is v_mfma_f32_16x16x32_bf16: products of bf16 are
// exact in binary32 and sums are kept in binary32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "epl.h"

namespace epl_product {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kMaxExperts = 2048;
constexpr int kTileK = 64;             // contraction depth of one LDS stage
constexpr int kNumXcd = 8;
constexpr int kMaxParts = 16;          // parts that a tile's contraction is split into, at most

// Waves along m and n of a tile's workgroup: a wave has half of its rows and
// 64 of its columns. Tiles of 256 x 256 take 8 waves, those of 128 x 128 four
// and two of their workgroups fit a CU.
constexpr int kWavesM = 2;
constexpr int waves_n(int bn) { return bn / 64; }
constexpr int tile_threads(int bn) { return kWavesM * waves_n(bn) * 64; }
constexpr int tile_groups(int bn) { return 512 / tile_threads(bn); }    // a CU

struct Args {
    const __bf16 *p;          // rows (forward, data gradient) or d rows (weight gradient)
    const __bf16 *q;          // weights, or rows (weight gradient)
    const float *bias;        // [E, N] or null
    const __bf16 *residual;   // [rows, cols of y] or null
    __bf16 *pre;              // [rows, .] or null: written by forward activations, read by gradient ones
    void *y;                  // output
    const int32_t *start, *count;
    int64_t rows;             // rows of the ragged buffers
    int E;
    int K;                    // contraction (columns of x); weight gradient: columns of x = output columns
    int N;                    // columns of the product; weight gradient: columns of d = output rows
    int act;                  // EPL_ACT_*
    int out_f32;
    int accumulate;           // weight gradient: add to y
    int *header;              // workspace: its first word is the number of tiles split
    f32x4 *ws;                // and behind it the partial tiles, or null
    int max_parts;            // parts that a tile's contraction is split into, at most
    int stages;               // steps of kTileK of a contraction (on average)
};

// f(0), f(1), .. f(N - 1) with the index a constant from the start: an array
// of 128 accumulators indexed by an unrolled loop stays in scratch memory.
template <typename F, int... I>
__device__ __forceinline__ void each_of(F &&f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F &&f)
{
    each_of(f, std::make_integer_sequence<int, N>{});
}

// An expert's block, cut to the buffer: [lo, lo + n).
template <typename A>
__device__ __forceinline__ int block_of(const A &a, int e, int64_t &lo)
{
    const int64_t s = a.start[e], c = a.count[e];
    lo = s < 0 ? 0 : s > a.rows ? a.rows : s;
    int64_t hi = c <= 0 ? lo : s + c;
    hi = hi > a.rows ? a.rows : hi;
    return hi > lo ? (int)(hi - lo) : 0;
}

// ------------------------------------------------------------- epilogue --

template <int C>
__device__ __forceinline__ void load_bf16(const __bf16 *p, float (&v)[C])
{
    typedef __bf16 vec __attribute__((ext_vector_type(C)));
    const vec r = *reinterpret_cast<const vec *>(p);
#pragma unroll
    for (int i = 0; i < C; ++i)
        v[i] = (float)r[i];
}

// One rounding to nearest even, of the finished binary32 value. PAST: past
// the caches.
template <int C, bool PAST = false>
__device__ __forceinline__ void store_bf16(__bf16 *p, const float (&v)[C])
{
    typedef __bf16 vec __attribute__((ext_vector_type(C)));
    vec r;
#pragma unroll
    for (int i = 0; i < C; ++i)
        r[i] = (__bf16)v[i];
    if (PAST)
        __builtin_nontemporal_store(r, reinterpret_cast<vec *>(p));
    else
        *reinterpret_cast<vec *>(p) = r;
}

template <int C, bool PAST = false>
__device__ __forceinline__ void store_out(const Args &a, int64_t at, const float (&v)[C])
{
    if (a.out_f32) {
        float *y = static_cast<float *>(a.y) + at;
#pragma unroll
        for (int i = 0; i < C; i += 4) {
            const f32x4 r = {v[i], v[i + 1], v[i + 2], v[i + 3]};
            if (PAST)
                __builtin_nontemporal_store(r, reinterpret_cast<f32x4 *>(y + i));
            else
                *reinterpret_cast<f32x4 *>(y + i) = r;
        }
    } else {
        store_bf16<C, PAST>(static_cast<__bf16 *>(a.y) + at, v);
    }
}

// 1 / (1 + exp(-z)): exp overflows to infinity for z below -88, where the
// quotient is its limit 0. The hardware's reciprocal is good to one step.
__device__ __forceinline__ float sigmoidf(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// z * sigmoid(z); -inf gives the limit 0 rather than -inf * 0.
__device__ __forceinline__ float silu(float z) { return z == -INFINITY ? 0.0f : z * sigmoidf(z); }

__device__ __forceinline__ float silu_slope(float z)
{
    const float p = sigmoidf(z);
    return fabsf(z) > 80.0f ? (z > 0.0f ? 1.0f : 0.0f) : p * (1.0f + z * (1.0f - p));
}

// The normal distribution function at -a, 0 <= a <= 14 (where it leaves
// binary32), and g = exp(-a^2 / 2), both to a few steps of their own size. With
// t = 1 / (1 + p a) the first is t P(t) g, P the polynomial of degree 7 with
// the least relative error (9.3e-8), fitted in binary64 by reweighted least
// squares to erfc(a / sqrt 2) / 2 over g. The exponent -a^2 log2(e) / 2 is kept
// in two words, y and yl: rounded to one it would cost 2^-24 a^2 of the result,
// 25 u at 5. (The constant's own error is in P.) 12288 x 2048 outputs of 64
// experts take 290 us; with a formula of the same cost less 5 instructions that
// is good to 1.5e-7 absolute, and so to 1e-3 in the tail, 286.
__device__ __forceinline__ float normal_tail(float a, float &g)
{
    const float h = a * a, c = 0.721347511f;
    const float y = -c * h, yl = fmaf(-c, fmaf(a, a, -h), fmaf(-c, h, -y));
    g = __builtin_amdgcn_exp2f(y);
    g = fmaf(g * 0.693147181f, yl, g);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.234f, a, 1.0f));
    float p = fmaf(-0.0663837567f, t, 0.222562999f);
    p = fmaf(p, t, -0.164247572f);
    p = fmaf(p, t, 0.194947466f);
    p = fmaf(p, t, 0.0281724539f);
    p = fmaf(p, t, 0.0995916724f);
    p = fmaf(p, t, 0.0919290408f);
    p = fmaf(p, t, 0.0934276506f);
    return p * t * g;
}

// z times its distribution function: max(z, 0) - |z| tail(|z|).
__device__ __forceinline__ float gelu(float z)
{
    float g;
    const float a = fminf(fabsf(z), 14.0f);
    return fmaf(-a, normal_tail(a, g), z < 0.0f ? 0.0f : z);
}

__device__ __forceinline__ float gelu_slope(float z)
{
    float g;
    const float tail = normal_tail(fminf(fabsf(z), 14.0f), g);
    const float c = z < 0.0f ? tail : 1.0f - tail;
    return fabsf(z) > 15.0f ? (z > 0.0f ? 1.0f : 0.0f) : fmaf(z * 0.39894228040143268f, g, c);
}

// What the epilogue of C columns of a row reads besides the product, as it
// is in memory: of a gradient activation the saved columns (of the gated one
// the gate's and the up half's), of the others the residual.
template <int C>
struct Side {
    typedef __bf16 vec __attribute__((ext_vector_type(C)));
    vec x, y;
};

template <int C>
__device__ __forceinline__ Side<C> side_of(const Args &a, int64_t row, int n)
{
    typedef typename Side<C>::vec vec;
    Side<C> s = {};
    if (a.act == EPL_ACT_SWIGLU_GRAD) {
        s.x = *reinterpret_cast<const vec *>(a.pre + row * 2 * a.N + n);
        s.y = *reinterpret_cast<const vec *>(a.pre + row * 2 * a.N + a.N + n);
    } else if (a.act >= EPL_ACT_SILU_GRAD) {
        s.x = *reinterpret_cast<const vec *>(a.pre + row * a.N + n);
    } else if (a.residual) {
        s.x = *reinterpret_cast<const vec *>(a.residual + row * (a.act == EPL_ACT_SWIGLU ? a.N / 2 : a.N) + n);
    }
    return s;
}

// The bias of C columns, or zeros.
template <int C>
__device__ __forceinline__ void bias_of(const Args &a, int e, int n, float (&b)[C])
{
#pragma unroll
    for (int i = 0; i < C; i += 4) {
        f32x4 v = {0, 0, 0, 0};
        if (a.bias)
            v = *reinterpret_cast<const f32x4 *>(a.bias + (int64_t)e * a.N + n + i);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            b[i + j] = v[j];
    }
}

// C columns n .. n + C - 1 of one row of the finished product.
template <int C>
__device__ __forceinline__ void emit(const Args &a, int64_t row, int n, const float (&b)[C],
                                     const Side<C> &s, float (&z)[C])
{
    if (a.act == EPL_ACT_SWIGLU_GRAD) {
        // saved [rows, 2 N]: gate, up; y likewise
        float dg[C], du[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            dg[i] = z[i] * (float)s.y[i] * silu_slope((float)s.x[i]);
            du[i] = z[i] * silu((float)s.x[i]);
        }
        store_out<C>(a, row * 2 * a.N + n, dg);
        store_out<C>(a, row * 2 * a.N + a.N + n, du);
        return;
    }
    const int64_t at = row * a.N + n;
    if (a.act == EPL_ACT_SILU_GRAD) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            z[i] *= silu_slope((float)s.x[i]);
    } else if (a.act == EPL_ACT_GELU_GRAD) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            z[i] *= gelu_slope((float)s.x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            z[i] += b[i];
        if (a.pre)
            store_bf16<C, true>(a.pre + at, z);          // read by the backward pass, much later
        if (a.act == EPL_ACT_SILU) {
#pragma unroll
            for (int i = 0; i < C; ++i)
                z[i] = silu(z[i]);
        } else if (a.act == EPL_ACT_GELU) {
#pragma unroll
            for (int i = 0; i < C; ++i)
                z[i] = gelu(z[i]);
        }
        if (a.residual)
#pragma unroll
            for (int i = 0; i < C; ++i)
                z[i] += (float)s.x[i];
    }
    store_out<C>(a, at, z);
}

// The gated activation: columns f .. f + C - 1 of the gate half and of the up half.
template <int C>
__device__ __forceinline__ void emit_pair(const Args &a, int64_t row, int f, const float (&bg)[C],
                                          const float (&bu)[C], const Side<C> &s, float (&g)[C],
                                          float (&u)[C])
{
    const int F = a.N / 2;
    float v[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        g[i] += bg[i];
        u[i] += bu[i];
        v[i] = silu(g[i]) * u[i];
    }
    if (a.pre) {
        store_bf16<C, true>(a.pre + row * a.N + f, g);
        store_bf16<C, true>(a.pre + row * a.N + F + f, u);
    }
    if (a.residual)
#pragma unroll
        for (int i = 0; i < C; ++i)
            v[i] += (float)s.x[i];
    store_out<C>(a, row * F + f, v);
}

// C neighbouring elements of a weight gradient: past the caches, which hold
// the operands that tiles share (64 experts of 192 rows, 2048 x 4096 in
// binary32: 653 us through them, 584 past them; of 500 rows, 2048 x 2048: 415,
// 350). Whoever reads gradients of this size next finds them in memory anyway.
template <int C>
__device__ __forceinline__ void emit_weight(const Args &a, int64_t at, float (&v)[C])
{
    if (a.accumulate) {
        float old[C];
        if (a.out_f32) {
#pragma unroll
            for (int x = 0; x < C; ++x)
                old[x] = static_cast<const float *>(a.y)[at + x];
        } else {
            load_bf16<C>(static_cast<const __bf16 *>(a.y) + at, old);
        }
#pragma unroll
        for (int x = 0; x < C; ++x)
            v[x] += old[x];
    }
    store_out<C, true>(a, at, v);
}

// ----------------------------------------------------------- tile kernel --
//
// A workgroup of 8 (or 4) waves computes BM x BN outputs, 64 deep at a time,
// from two LDS stages that buffer loads fill directly (16 bytes a lane) while
// the other stage is multiplied. Q is the matrix instruction's A operand and
// P its B operand, so a lane's accumulator registers run along n, the
// contiguous index of the output: register quad (i, j) of lane 16 q + r holds
// row 16 i + r, columns 16 j + 4 q .. + 3 of the wave's part.
//
// LDS layouts (XOR swizzles on 16-byte pieces so that the 16 lanes of a read
// fall on different banks; a DMA writes LDS in lane order, so the swizzle is
// applied to the global address that the lane reads):
//   contiguous operand: [rows][64], piece c of row r at c ^ swz(r)
//   strided operand:    [64][cols], piece c of row k at c ^ swz_t(k), read
//                       with ds_read_b64_tr_b16, which hands lane r column r
//                       of a 4-row block, 4 consecutive k
//
// Bound by the matrix instructions and the clock they leave: 8 x 4096 rows,
// 7168 -> 4096, in 1.49 - 1.55 ms, 1.24 - 1.29 PFLOP/s (the same loop without
// its loads takes 1.11 ms); with few rows an expert by the weights' bytes:
// 64 x 192 rows, 4096 -> 2048, 289 - 294 us, 4.4 TB/s. Weight gradients: 29765
// rows, 4096 x 7168, 1.35 - 1.40 ms (1.25 - 1.29 PFLOP/s); 64 x 192 rows,
// 2048 x 4096 in binary32, 0.63 - 0.65 ms, by the 2.1 GB they write (into the
// same buffers every time 0.49 - 0.53).

__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swz_t(int k) { return ((k & 3) << 1) | (((k >> 3) & 1) << 3); }

// A buffer descriptor of `bytes` bytes from `base`: a lane that reads beyond
// them gets zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const char *base, int bytes)
{
    // scalar registers, whatever the compiler can prove: a descriptor in
    // vector registers costs a loop at every use
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(((uint64_t)hi << 32) | lo), 0,
                                             __builtin_amdgcn_readfirstlane(max(bytes, 0)), 0x00020000);
}

// All of this wave's loads into LDS and reads of it are done, and the other
// waves' too.
__device__ __forceinline__ void landed()
{
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// 16 bytes a lane into 1 KB of LDS.
__device__ __forceinline__ void dma(__amdgpu_buffer_rsrc_t r, uint32_t off, uint16_t *lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)lds, 16, (int)off, 0, 0, 0);
}

// 8 consecutive k of one column from a strided operand's stage [64][COLS]:
// two 4-row transposing reads.
template <int COLS>
__device__ __forceinline__ bf16x8 read_tr(const uint16_t *at)
{
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(at + 4 * COLS));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// `elements` behind the lane's byte offset into a stage.
__device__ __forceinline__ const uint16_t *at(const uint16_t *stage, int bytes, int elements)
{
    return reinterpret_cast<const uint16_t *>(reinterpret_cast<const char *>(stage) + bytes) + elements;
}

// offset ^= by, in place: the compiler must not keep a register for every value
// (with those the weight gradient's loop spills: 1.86 ms against 1.35 for
// 29765 rows of 7168 x 4096). Left outside the loops: 2 vector registers of the
// data gradient's 256 x 256 tile, and scalar ones, which go to lanes of a vector
// register.
__device__ __forceinline__ void walk(int &offset, int by)
{
    offset ^= by;
    asm("" : "+v"(offset));
}

enum Form { kForward, kDataGrad, kWeightGrad };

// The m tiles of the experts before each expert, and of all of them: never
// more than blocks apart from each other have, so that no sum overflows where
// bad ones share rows. rows_of(e, first row) is an expert's number of rows.
template <int BM, int THREADS, typename F>
__device__ __forceinline__ void tile_prefix(int E, int64_t rows, F &&rows_of, int32_t *pre,
                                            int32_t *sums)
{
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int most = (int)(rows / BM) + E;
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += THREADS) {
        const int e = e0 + t;
        int64_t lo;
        const int own = e < E ? (rows_of(e, lo) + BM - 1) / BM : 0;
        int up = own;
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(up, d);
            up += lane >= d ? v : 0;
        }
        if (lane == 63)
            sums[wave] = up;
        __syncthreads();
        int before = base;
        for (int w = 0; w < THREADS / 64; ++w) {
            before = min(before + (w < wave ? sums[w] : 0), most);
            base = min(base + sums[w], most);
        }
        if (e < E)
            pre[e] = min(before + up - own, most);
        __syncthreads();
    }
    if (t == 0)
        pre[E] = base;
    __syncthreads();
}
template <int BM, int THREADS>
__device__ __forceinline__ void tile_prefix(const Args &a, int32_t *pre, int32_t *sums)
{
    tile_prefix<BM, THREADS>(
        a.E, a.rows, [&](int e, int64_t &lo) { return block_of(a, e, lo); }, pre, sums);
}

// The last expert with pre[e] <= m tile `t`, the same for a whole wave.
__device__ __forceinline__ int expert_of_tile(const int32_t *pre, int E, int t)
{
    int l = 0, h = E;
    while (h - l > 1) {
        const int mid = (l + h) >> 1;
        if (pre[mid] <= t)
            l = mid;
        else
            h = mid;
    }
    return __builtin_amdgcn_readfirstlane(l);
}

// Into how many parts to split the contraction of the `left` tiles of a round
// of `grid` workgroups: as many as there are workgroups for, if that pays. It
// saves stages (1 - 1 / parts) steps of 1.55 us (128 x 128: 1.1) and costs
// 0.09 us (0.026) a part, which writes its sums and has them read: 128 tiles
// of 256 x 256 over 512, 1024, 2048, 4096, 7168 in two parts each took 40, 46,
// 58, 81, 132 us, whole 30, 41, 61, 102, 187.
__host__ __device__ inline int parts_of(int left, int grid, int max_parts, int stages, int side)
{
    const int parts = left > 0 ? (grid / left < max_parts ? grid / left : max_parts) : 1;
    const int64_t saved = (int64_t)stages * (parts - 1) * (side == 256 ? 17 : 42);
    return parts > 1 && saved > (int64_t)left * parts * parts ? parts : 1;
}

// Which tiles are computed whole, and into how many parts the contraction of
// the rest is split. A round is one tile for every workgroup; a last round
// that would leave half of them or more without one can be shared out: each
// of its `left` tiles among `parts` workgroups, whose sums join_kernel adds in
// order.
struct Plan {
    int64_t whole;
    int left, parts;
};

template <int BM>
__device__ __forceinline__ Plan plan_of(const Args &a, int64_t tiles, int grid)
{
    Plan p{tiles, 0, 1};
    const int left = (int)(tiles % grid);
    const int parts = a.ws ? parts_of(left, grid, a.max_parts, a.stages, BM) : 1;
    if (parts > 1)
        p = Plan{tiles - left, left, parts};
    return p;
}

struct Tile {
    int64_t lo;               // first row of the expert's block
    int e, cnt, tm, tn;
};

template <Form FORM>
__device__ __forceinline__ Tile locate(const Args &a, const int32_t *pre, int64_t t, int ntm, int ntn)
{
    Tile x;
    int64_t in_e;
    int ntm_e = ntm;
    if (FORM == kWeightGrad) {
        x.e = (int)(t / ((int64_t)ntm * ntn));
        in_e = t - (int64_t)x.e * ntm * ntn;
    } else {
        int l = 0, h = a.E;                 // last expert with pre[e] * ntn <= t
        while (h - l > 1) {
            const int mid = (l + h) >> 1;
            if ((int64_t)pre[mid] * ntn <= t)
                l = mid;
            else
                h = mid;
        }
        x.e = __builtin_amdgcn_readfirstlane(l);
        const int first = __builtin_amdgcn_readfirstlane(pre[x.e]);
        in_e = t - (int64_t)first * ntn;
        ntm_e = __builtin_amdgcn_readfirstlane(pre[x.e + 1]) - first;
    }
    x.cnt = block_of(a, x.e, x.lo);
    // within an expert: bands of up to 8 m tiles, m fastest, so that the
    // tiles in flight on an XCD share both operands in its L2
    const int band = (int)(in_e / (8 * (int64_t)ntn));
    const int bh = min(8, ntm_e - band * 8);
    const int rest = (int)(in_e - (int64_t)band * 8 * ntn);
    x.tm = band * 8 + rest % bh;
    x.tn = rest / bh;
    return x;
}

// A register quad of a wave's rows into its part of LDS, [rows][64] with
// 16-byte pieces swizzled by row.
__device__ __forceinline__ void put(float *mine, int row, int piece, f32x4 v)
{
    *reinterpret_cast<f32x4 *>(mine + row * 64 + (piece ^ (row & 15)) * 4) = v;
}

template <int C>
__device__ __forceinline__ void take(const float *mine, int row, int col, float (&v)[C])
{
#pragma unroll
    for (int i = 0; i < C; i += 4) {
        const f32x4 x =
            *reinterpret_cast<const f32x4 *>(mine + row * 64 + (((col + i) / 4) ^ (row & 15)) * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[i + j] = x[j];
    }
}

// The epilogue of `rows` rows of 64 columns that a wave holds in its part of
// LDS: a lane takes 8 neighbouring columns, or 8 of the gate and 8 of the up
// half, or 4 of a weight gradient in binary32, so that rows leave in whole
// lines. m0: the first of them in the tile's block; n0: the first column in
// the tile's columns.
template <int BN, Form FORM>
__device__ __forceinline__ void emit_rows(const Args &a, const Tile &x, const float *mine, int rows,
                                          int m0, int n0, int lane)
{
    const bool paired = a.act == EPL_ACT_SWIGLU;
    const bool four = FORM == kWeightGrad && a.out_f32;
    const int lanes = four ? 16 : paired ? 4 : 8;             // a row
    const int last = FORM == kWeightGrad ? a.N : x.cnt;
    const int c = (lane % lanes) * (64 / lanes), n = x.tn * BN + n0 + c, step = 64 / lanes;
    if (FORM == kWeightGrad) {
        if (n >= a.K)
            return;
#pragma unroll 1
        for (int row = lane / lanes; row < rows && m0 + row < last; row += step) {
            const int64_t at = ((int64_t)x.e * a.N + m0 + row) * a.K + n;
            if (four) {
                float v[4];
                take<4>(mine, row, c, v);
                emit_weight<4>(a, at, v);
            } else {
                float v[8];
                take<8>(mine, row, c, v);
                emit_weight<8>(a, at, v);
            }
        }
        return;
    }
    if (n >= a.N)
        return;
    const int f = paired ? n / 2 : n;                         // column of y
    float b[8], bu[8];
    bias_of<8>(a, x.e, f, b);
    bias_of<8>(a, x.e, paired ? a.N / 2 + f : f, bu);
    // what four rows read is on its way before the first is finished (one at
    // a time, the product of 64 experts with bias, activation and residual
    // took 300 us, not 290)
    constexpr int ahead = 4;
#pragma unroll 1
    for (int row0 = lane / lanes; row0 < rows && m0 + row0 < last; row0 += ahead * step) {
        Side<8> s[ahead];
#pragma unroll
        for (int i = 0; i < ahead; ++i)
            s[i] = side_of<8>(a, x.lo + min(m0 + row0 + i * step, last - 1), f);
#pragma unroll
        for (int i = 0; i < ahead; ++i) {
            const int row = row0 + i * step;
            if (row >= rows || m0 + row >= last)
                break;
            float v[8], u[8];
            take<8>(mine, row, c, v);
            if (paired) {
                take<8>(mine, row, c + 8, u);
                emit_pair<8>(a, x.lo + m0 + row, f, b, bu, s[i], v, u);
            } else {
                emit<8>(a, x.lo + m0 + row, n, b, s[i], v);
            }
        }
    }
}

template <int BM, int BN, Form FORM>
__global__ __launch_bounds__(tile_threads(BN), 2) void tile_kernel(Args a)
{
    constexpr bool PT = FORM == kWeightGrad;             // P strided
    constexpr bool QT = FORM != kForward;                // Q strided
    constexpr int WN = waves_n(BN), WM = kWavesM, WAVES = WM * WN;
    constexpr int IP = BM / WM / 16;                     // 16-row pieces of P a wave
    constexpr int ROWS = WAVES * 8;                      // rows of a contiguous operand a DMA
    constexpr int ISP = BM / ROWS, ISQ = BN / ROWS;      // DMAs a stage
    constexpr int KP = WAVES * 512 / BM, KQ = WAVES * 512 / BN;    // rows of a strided one
    __shared__ __align__(1024) uint16_t sp0[BM * kTileK], sp1[BM * kTileK];
    __shared__ __align__(1024) uint16_t sq0[BN * kTileK], sq1[BN * kTileK];
    __shared__ int32_t pre[FORM == kWeightGrad ? 1 : kMaxExperts + 1];
    __shared__ int32_t sums[8];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, r = lane & 15, q = lane >> 4;
    const bool paired = a.act == EPL_ACT_SWIGLU;

    // The lane's LDS offsets (bytes) of its first pieces; the others lie at
    // fixed distances, since the swizzles use none of the bits that the piece
    // and (for strided operands) the 32-deep half change; those of a strided
    // operand by an exclusive or, for which the offset walks from piece to
    // piece and comes back to the first.
    int aq[2], ap[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int n = wn * 64 + r, m = wm * (BM / WM) + r;
        const int k = q * 8 + (r >> 2), c = (r & 3) >> 1;
        aq[h] = 2 * (QT ? k * BN + ((wn * 8 + c) ^ swz_t(k)) * 8 + (r & 1) * 4
                        : n * kTileK + ((h * 4 + q) ^ swz(n)) * 8);
        ap[h] = 2 * (PT ? k * BM + ((wm * (BM / WM / 8) + c) ^ swz_t(k)) * 8 + (r & 1) * 4
                        : m * kTileK + ((h * 4 + q) ^ swz(m)) * 8);
    }

    // tiles along m and n, over all experts
    const int ntn = FORM == kWeightGrad ? (a.K + BN - 1) / BN : (a.N + BN - 1) / BN;
    int ntm = 0;
    int64_t total;
    if (FORM == kWeightGrad) {
        ntm = (a.N + BM - 1) / BM;
        total = (int64_t)a.E * ntm * ntn;
    } else {
        tile_prefix<BM, WAVES * 64>(a, pre, sums);
        total = (int64_t)pre[a.E] * ntn;
    }

    // workgroups of one XCD (every eighth) take neighbouring tiles
    const int grid = gridDim.x;
    int64_t first = blockIdx.x;
    if (grid % kNumXcd == 0)
        first = (first % kNumXcd) * (grid / kNumXcd) + first / kNumXcd;
    const Plan plan = plan_of<BM>(a, total, grid);
    const int64_t items = plan.whole + plan.left * plan.parts;
    if (a.ws && blockIdx.x == 0 && tid == 0)
        a.header[0] = plan.left;

    for (int64_t item = first; item < items; item += grid) {
        const bool split = item >= plan.whole;
        // parts of the same place in the contraction are neighbours
        const int o = split ? (int)(item - plan.whole) : 0;
        const int part = split ? o / plan.left : 0, rest = split ? o % plan.left : 0;
        const Tile x = locate<FORM>(a, pre, split ? plan.whole + rest : item, ntm, ntn);
        const int e = x.e, cnt = x.cnt, tm = x.tm, tn = x.tn;
        const int64_t lo = x.lo;

        // opaque: what is derived from the lane for one tile is not kept for the next
        int own = tid;
        asm volatile("" : "+v"(own));
        // Operands: base, the lane's offset, and the bytes between the DMAs of
        // a stage. Their ends: a strided operand ends with its rows of the
        // contraction; a contiguous one with its last row, and pieces beyond
        // the contraction are sent past it by the offset's top bit.
        const int whole = FORM == kWeightGrad ? cnt : a.K;
        const int steps = (whole + kTileK - 1) / kTileK;
        const int s0 = split ? steps * part / plan.parts : 0;
        const int s1 = split ? steps * (part + 1) / plan.parts : steps;
        // Experts start at different places of the contraction and come round:
        // rows lie a power of two or so apart, and tiles that all read the
        // same columns would meet on the same memory channels (64 experts of
        // 192 rows, 4096 -> 2048: 293 us without, 264 with). Tiles of one
        // expert stay together, for what they share in L2.
        const int turns = s1 - s0;
        const int rot = turns > 0 ? (int)((uint32_t)(e * 13) % (uint32_t)turns) : 0;
        const int qcols = FORM == kWeightGrad ? a.K : a.N;
        const char *bp, *bq;
        uint32_t op, oq;
        int np = 0, nq = 0;                  // bytes of a contiguous operand
        int kp = 0, kq = 0;                  // contraction index of the lane's piece
        const int ip = PT ? KP * a.N * 2 : ROWS * a.K * 2;
        const int iq = QT ? KQ * qcols * 2 : (paired ? ROWS / 2 : ROWS) * a.K * 2;
        if (PT) {
            const int k = (own * 8) / BM, c = ((own * 8 % BM) / 8) ^ swz_t(k);
            op = ((uint32_t)k * a.N + tm * BM + c * 8) * 2;
            bp = reinterpret_cast<const char *>(a.p + lo * a.N);
        } else {
            const int row = own >> 3, c = (own & 7) ^ swz(row);
            op = ((uint32_t)row * a.K + c * 8) * 2;
            kp = c * 8;
            bp = reinterpret_cast<const char *>(a.p + (lo + (int64_t)tm * BM) * a.K);
            np = min(cnt - tm * BM, BM) * a.K * 2;
        }
        if (QT) {
            const int k = (own * 8) / BN, c = ((own * 8 % BN) / 8) ^ swz_t(k);
            const int col = paired ? tn * (BN / 2) + (c >> 1) * 8 + (c & 1) * (a.N / 2)
                                   : tn * BN + c * 8;
            oq = ((uint32_t)k * qcols + col) * 2;
            bq = reinterpret_cast<const char *>(
                FORM == kWeightGrad ? a.q + lo * qcols : a.q + (int64_t)e * a.K * a.N);
        } else {
            const int row = own >> 3, c = (own & 7) ^ swz(row);
            const int n = paired ? tn * (BN / 2) + (row >> 4) * 8 + (row & 7) + (row & 8 ? a.N / 2 : 0)
                                 : tn * BN + row;
            oq = ((uint32_t)n * a.K + c * 8) * 2;
            kq = c * 8;
            bq = reinterpret_cast<const char *>(a.q + (int64_t)e * a.K * a.N);
            nq = a.N * a.K * 2;
        }

        f32x4 acc[IP * 4];
        each<IP * 4>([&](auto i) { acc[i] = f32x4{0, 0, 0, 0}; });

        struct Stage {
            __amdgpu_buffer_rsrc_t rp, rq;
            uint32_t op, oq;
        };
        auto stage = [&](int s) {
            const int v = s + rot, k0 = (v < s1 ? v : v - turns) * kTileK;
            const int left = s < s1 ? min(whole - k0, kTileK) : 0;
            Stage f;
            f.rp = PT ? rsrc(bp + (int64_t)k0 * a.N * 2, left * a.N * 2) : rsrc(bp + k0 * 2, np - k0 * 2);
            f.rq = QT ? rsrc(bq + (int64_t)k0 * qcols * 2, left * qcols * 2)
                      : rsrc(bq + k0 * 2, nq - k0 * 2);
            f.op = !PT && kp >= left ? op | 0x80000000u : op;
            f.oq = !QT && kq >= left ? oq | 0x80000000u : oq;
            return f;
        };
        // DMA number x of a stage: those of P, then those of Q
        auto fetch_one = [&](const Stage &f, uint16_t *lp, uint16_t *lq, auto x) {
            if constexpr (x < ISP)
                dma(f.rp, f.op + x * ip, lp + x * WAVES * 512 + wave * 512);
            else
                dma(f.rq, f.oq + (x - ISP) * iq, lq + (x - ISP) * WAVES * 512 + wave * 512);
        };
        auto fetch = [&](int s, uint16_t *lp, uint16_t *lq) {
            const Stage f = stage(s);
            each<ISP + ISQ>([&](auto x) { fetch_one(f, lp, lq, x); });
        };
        auto read_q = [&](bf16x8 (&f)[4], const uint16_t *lq, auto kb) {
            each<4>([&](auto j) {
                f[j] = QT ? read_tr<BN>(at(lq, aq[0] ^ (j * 32), kb * 32 * BN))
                          : *reinterpret_cast<const bf16x8 *>(at(lq, aq[kb], j * 16 * kTileK));
            });
        };
        bf16x8 fp[4], qa[4], qb[4];
        auto read_p = [&](const uint16_t *lp, auto g) {      // piece g of a stage's 2 IP
            constexpr int i = g % IP, kb = g / IP;
            if constexpr (PT) {
                fp[g % 4] = read_tr<BM>(at(lp, ap[0], kb * 32 * BM));
                walk(ap[0], (i ^ ((i + 1) % IP)) * 32);
            } else {
                fp[g % 4] = *reinterpret_cast<const bf16x8 *>(at(lp, ap[kb], i * 16 * kTileK));
            }
        };
        auto multiply = [&](const bf16x8 (&fq)[4], auto g) {
            constexpr int i = g % IP;
            each<4>([&](auto j) {
                acc[i * 4 + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[j], fp[g % 4],
                                                                         acc[i * 4 + j], 0, 0, 0);
            });
        };
        // One stage: 2 IP groups of 4 products, one piece of P each, the
        // second half of them with the second half's Q. After a group the
        // piece 4 further on is read into its registers, so reads run under
        // the products all the time. One barrier a stage, a group behind the
        // last read of it: it says both that every wave has read all of this
        // stage, which the DMA of the stage after the next may now overwrite,
        // and that the next stage, whose first pieces are read from then on,
        // has landed.
        using Zero = std::integral_constant<int, 0>;
        using One = std::integral_constant<int, 1>;
        auto turn = [&](int s, uint16_t *cp, uint16_t *cq, uint16_t *xp, uint16_t *xq) {
            constexpr int all = 2 * IP, meet = all - 4, dmas = ISP + ISQ;
            Stage f;
            each<all>([&](auto g) {
                if constexpr (g < IP)
                    multiply(qa, g);
                else
                    multiply(qb, g);
                if constexpr (g == 0)
                    read_q(qb, cq, One{});
                if constexpr (g < meet)
                    read_p(cp, std::integral_constant<int, g + 4>{});
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (g == meet) {
                    landed();
                    f = stage(s + 2);
                    read_q(qa, xq, Zero{});      // after the last stage: not used
                }
                if constexpr (g >= meet)
                    read_p(xp, std::integral_constant<int, g - meet>{});
                if constexpr (g >= meet) {       // the DMAs, over the groups that are left
                    constexpr int part = g - meet, per = (dmas + 3) / 4;
                    each<per>([&](auto u) {
                        constexpr std::integral_constant<int, part * per + decltype(u)::value> x{};
                        if constexpr (x < dmas)
                            fetch_one(f, cp, cq, x);
                    });
                    __builtin_amdgcn_sched_barrier(0);
                }
            });
        };
        // Pairs of stages, without a branch inside: a stage past the last is
        // filled with zeros, by descriptors that hold no bytes.
        fetch(s0, sp0, sq0);
        landed();
        fetch(s0 + 1, sp1, sq1);
        read_q(qa, sq0, Zero{});
        each<4>([&](auto g) { read_p(sp0, g); });
        for (int s = s0; s < s1; s += 2) {
            turn(s, sp0, sq0, sp1, sq1);
            turn(s + 1, sp1, sq1, sp0, sq0);
        }
        landed();                            // (what was fetched past the end too)
        if (PT)
            walk(ap[0], 4 % IP * 32);        // back from the 4 pieces read ahead

        const int m0 = tm * BM + wm * (BM / WM), n0 = wn * 64;
        own = tid & 63;
        asm volatile("" : "+v"(own));
        const int er = own & 15, eq = own >> 4;
        if (split) {
            // registers as they are; join_kernel reads them alike
            f32x4 *slot = a.ws + (int64_t)(rest * plan.parts + part) * (BM * BN / 4);
            each<IP * 4>([&](auto y) { slot[((y / 4 * WAVES + wave) * 4 + y % 4) * 64 + own] = acc[y]; });
        } else {
            // Two passes of half the wave's rows through its own part of the
            // stages: the epilogue's code is there once a pass, not once an
            // accumulator (43 000 instructions otherwise).
            constexpr int half = IP / 2 * 16;
            constexpr int share = WAVES / 4;       // waves to a stage array
            uint16_t *const stages = wave < share       ? sp0
                                     : wave < 2 * share ? sp1
                                     : wave < 3 * share ? sq0
                                                        : sq1;
            float *const mine = reinterpret_cast<float *>(stages) + wave % share * half * 64;
            each<2>([&](auto h) {
                each<IP / 2>([&](auto i) {
                    each<4>([&](auto j) {
                        put(mine, i * 16 + er, j * 4 + eq, acc[(h * (IP / 2) + i) * 4 + j]);
                    });
                });
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
                emit_rows<BN, FORM>(a, x, mine, half, m0 + h * half, n0, own);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
            });
            __syncthreads();       // the next tile's stages overwrite the other waves' parts
        }
    }
}

// Adds the parts of the tiles that tile_kernel<BM, BN, FORM> split, in order,
// and runs their epilogue. A workgroup takes one 16-row piece of each wave
// (blockIdx.x) of tiles blockIdx.y, + gridDim.y, ..; `grid` is the tile
// kernel's.
template <int BM, int BN, Form FORM>
__global__ __launch_bounds__(tile_threads(BN)) void join_kernel(Args a, int grid)
{
    constexpr int WN = waves_n(BN), WM = kWavesM, WAVES = WM * WN;
    __shared__ __align__(16) float rows[WAVES * 16 * 64];
    __shared__ int32_t pre[FORM == kWeightGrad ? 1 : kMaxExperts + 1];
    __shared__ int32_t sums[8];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
    if (a.header[0] == 0)          // (found from the counts: 16 experts of 500 rows, 512 ->
        return;                    // 640, took 24 us rather than 22; 64 of 192 290, not 285)
    const int i = blockIdx.x;
    const int ntn = FORM == kWeightGrad ? (a.K + BN - 1) / BN : (a.N + BN - 1) / BN;
    const int ntm = FORM == kWeightGrad ? (a.N + BM - 1) / BM : 0;
    if (FORM != kWeightGrad)
        tile_prefix<BM, WAVES * 64>(a, pre, sums);
    const Plan plan = plan_of<BM>(
        a, FORM == kWeightGrad ? (int64_t)a.E * ntm * ntn : (int64_t)pre[a.E] * ntn, grid);
    for (int l = blockIdx.y; l < plan.left; l += gridDim.y) {
        const Tile x = locate<FORM>(a, pre, plan.whole + l, ntm, ntn);
        const f32x4 *slot = a.ws + (int64_t)l * plan.parts * (BM * BN / 4) + ((i * WAVES + wave) * 4) * 64 + lane;
        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = slot[j * 64];
        for (int p = 1; p < plan.parts; ++p) {
            slot += BM * BN / 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j] += slot[j * 64];
        }
        const int m0 = x.tm * BM + wm * (BM / WM) + i * 16, n0 = wn * 64;
        float *mine = rows + wave * 16 * 64;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            put(mine, r, j * 4 + q, acc[j]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        emit_rows<BN, FORM>(a, x, mine, 16, m0, n0, lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    }
}

// ------------------------------------------------------ few-rows kernel --
//
// For experts with a few rows the weights' bytes are the cost: each is read
// once for 32 rows, straight into the registers of the matrix instruction (an
// expert of many among experts of few has its weights read that much oftener:
// 768 rows over 64 experts, 4096 -> 2048, evenly 221 us, with 705 of them in
// one expert 429). A workgroup
// of WAVES waves takes 32 columns of one expert; the waves share the
// contraction (128 deep a turn each) and add their sums through LDS in wave
// order. Workgroups start at different places of the contraction and come
// round, so that those under way at one time read different columns of their
// rows, which lie on different memory channels (64 experts of one row, 4096
// -> 2048: 231 us without, 178 with).

constexpr int kFewCols = 32;            // two matrix instructions wide
// (64 columns, which read x half as often: 8 experts of 1, 8, 14 rows, 7168 ->
// 4096, 93, 98, 103 us against 87, 98, 108; more rows go to the tiles.)

template <int WAVES, int MT>
__device__ __forceinline__ void few_rows(const Args &a, int e, int64_t row0, int left, int nb,
                                         f32x4 *red)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, q = lane >> 4;
    const bool paired = a.act == EPL_ACT_SWIGLU;
    constexpr int J = kFewCols / 16;
    const int F = a.N / 2;
    const __bf16 *w = a.q + (int64_t)e * a.N * a.K;
    const __bf16 *pw[J], *px[MT];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        // lane q holds 8 neighbouring columns, or 4 of the gate and the same 4 of the up half
        const int n = paired ? min(nb * 16 + r, F - 1) + j * F
                             : min(nb * 32 + (r >> 2) * 8 + j * 4 + (r & 3), a.N - 1);
        pw[j] = w + (int64_t)n * a.K + q * 8;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
        px[i] = a.p + (row0 + min(i * 16 + r, left - 1)) * a.K + q * 8;
    f32x4 acc[MT][J];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
            acc[i][j] = f32x4{0, 0, 0, 0};

    const bf16x8 zero = {};
    const int turns = (a.K + 127) / 128;
    int at = (int)((uint32_t)(e * 13 + nb * 3 + wave) % (uint32_t)turns);
    for (int t = wave; t < turns; t += WAVES) {
        bf16x8 fw[4][J], fx[4][MT];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = at * 128 + u * 32;
            const bool in = k + q * 8 < a.K;
#pragma unroll
            for (int j = 0; j < J; ++j)
                fw[u][j] = in ? *reinterpret_cast<const bf16x8 *>(pw[j] + k) : zero;
#pragma unroll
            for (int i = 0; i < MT; ++i)
                fx[u][i] = in ? *reinterpret_cast<const bf16x8 *>(px[i] + k) : zero;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[u][j], fx[u][i],
                                                                        acc[i][j], 0, 0, 0);
        at += WAVES;
        while (at >= turns)
            at -= turns;
    }

    __syncthreads();           // red may still be read for the rows before
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
            red[((wave * MT + i) * J + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    if (wave >= MT)
        return;
    float v[J * 4];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        f32x4 sum = red[(wave * J + j) * 64 + lane];
#pragma unroll
        for (int o = 1; o < WAVES; ++o)
            sum += red[((o * MT + wave) * J + j) * 64 + lane];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            v[j * 4 + x] = sum[x];
    }
    const int64_t row = row0 + wave * 16 + r;
    if (wave * 16 + r >= left)
        return;
    if (paired) {
        const int f = nb * 16 + q * 4;
        if (f < F) {
            float bg[4], bu[4], g[4], u[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
                g[x] = v[x], u[x] = v[4 + x];
            bias_of<4>(a, e, f, bg);
            bias_of<4>(a, e, F + f, bu);
            emit_pair<4>(a, row, f, bg, bu, side_of<4>(a, row, f), g, u);
        }
    } else {
        const int n = nb * 32 + q * 8;
        if (n < a.N) {
            float b[8];
            bias_of<8>(a, e, n, b);
            emit<8>(a, row, n, b, side_of<8>(a, row, n), v);
        }
    }
}

template <int WAVES>
__global__ __launch_bounds__(WAVES * 64, WAVES == 4 ? 2 : 4) void few_rows_kernel(Args a)
{
    __shared__ f32x4 red[WAVES * 2 * (kFewCols / 16) * 64];
    const int e = blockIdx.y, nb = blockIdx.x;
    int64_t lo;
    const int cnt = block_of(a, e, lo);
    for (int m = 0; m < cnt; m += 32) {
        if (cnt - m <= 16)
            few_rows<WAVES, 1>(a, e, lo + m, cnt - m, nb, red);
        else
            few_rows<WAVES, 2>(a, e, lo + m, cnt - m, nb, red);
    }
}

}  // namespace epl_product
