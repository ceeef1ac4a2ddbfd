// Device kernels of the experts' matrix products on 8-bit rows and weights for
// gfx950 (CDNA4): e4m3 codes with a scale for each 128 columns of a row and
// for each 128 x 128 block of a weight,
//     z[p, n] = sum_b sx[p, b] sw[n / 128, b] sum_{k in block b} x[p, k] w[n, k],
// with the epilogue of the bf16 products, and the result as codes and scales
// as well.
//
// The matrix instruction is v_mfma_f32_16x16x128_f8f6f4, one block of the
// contraction: its sum starts from zero, and is multiplied by its scales and
// added to the accumulators in binary32. The instruction itself adds the
// products in groups of 8 neighbours and drops, of each product, the bits below
// 2^-13 of the largest one's power of two (towards zero; measured); the groups
// are added in binary32. Against exact sums that is about 2^-16 of the result
// for normal data, and it is what twice the rate of bf16 costs: the codes
// themselves are off by up to 2^-4.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epl.h"
#include "epl_cast_kernels.h"
#include "epl_product_kernels.h"

namespace epl_product8 {

using epl_cast::Factor;
using epl_cast::Scales;
using epl_product::bias_of;
using epl_product::block_of;
using epl_product::Side;
using epl_product::side_of;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kGroup = epl_cast::kGroup;

struct Args : epl_product::Args {
    const uint8_t *x8, *w8;
    Scales xs;                // of x
    const void *ws;           // of the weight: [E, blocks of out, blocks of in] as it lies
    int ws_bytes;             // exponents, one byte each, rather than fp32
    int in_out;               // weight [E, K, N]
    uint8_t *codes;           // the result as codes, or null
    Scales cs;                // and their scales
};

__device__ __forceinline__ int blocks_of(int n) { return (n + kGroup - 1) / kGroup; }

// Columns of y.
__device__ __forceinline__ int out_cols(const Args &a)
{
    return a.act == EPL_ACT_SWIGLU ? a.N / 2 : a.act == EPL_ACT_SWIGLU_GRAD ? 2 * a.N : a.N;
}

// The scale of column n's block and block b of the contraction.
__device__ __forceinline__ float weight_scale(const Args &a, int e, int n, int b)
{
    const int nb = blocks_of(a.N), kb = blocks_of(a.K);
    const int64_t at = (int64_t)e * nb * kb + (a.in_out ? b * nb + n / kGroup : n / kGroup * kb + b);
    return a.ws_bytes ? epl_cast::power_of(static_cast<const uint8_t *>(a.ws)[at])
                      : static_cast<const float *>(a.ws)[at];
}

// The finished values of C columns n .. of one row, from the product z: z is
// column n of y, and u column N + n (gradient of the gated activation). Of the
// gated activation z and u are the gate's and the up half's product, and z the
// result.
template <int C>
__device__ __forceinline__ void finish(const Args &a, int64_t row, int n, const float (&b)[C],
                                       const float (&bu)[C], const Side<C> &s, float (&z)[C],
                                       float (&u)[C])
{
    using namespace epl_product;
    if (a.act == EPL_ACT_SWIGLU_GRAD) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            u[i] = z[i] * silu((float)s.x[i]);
            z[i] = z[i] * (float)s.y[i] * silu_slope((float)s.x[i]);
        }
        return;
    }
    if (a.act == EPL_ACT_SILU_GRAD || a.act == EPL_ACT_GELU_GRAD) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            z[i] *= a.act == EPL_ACT_SILU_GRAD ? silu_slope((float)s.x[i]) : gelu_slope((float)s.x[i]);
        return;
    }
    const bool paired = a.act == EPL_ACT_SWIGLU;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        z[i] += b[i];
        u[i] += bu[i];
    }
    if (a.pre) {                                   // read by the backward pass, much later
        store_bf16<C, true>(a.pre + row * a.N + n, z);
        if (paired)
            store_bf16<C, true>(a.pre + row * a.N + a.N / 2 + n, u);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (paired)
            z[i] = silu(z[i]) * u[i];
        else if (a.act == EPL_ACT_SILU)
            z[i] = silu(z[i]);
        else if (a.act == EPL_ACT_GELU)
            z[i] = gelu(z[i]);
        if (a.residual)
            z[i] += (float)s.x[i];
    }
}

template <int C>
__device__ __forceinline__ float largest(const float (&v)[C])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i)
        m = fmaxf(m, fabsf(v[i]));
    return m;
}

// C codes of one row.
template <int C>
__device__ __forceinline__ void store_codes(const Args &a, int64_t at, const float (&v)[C],
                                            const Factor &f)
{
    typedef uint32_t vec __attribute__((ext_vector_type(C / 4)));
    uint32_t w[C / 4];
    epl_cast::codes_of(v, f, w);
    vec r;
#pragma unroll
    for (int i = 0; i < C / 4; ++i)
        r[i] = w[i];
    *reinterpret_cast<vec *>(a.codes + at) = r;
}

// ------------------------------------------------------ few-rows kernel --
//
// A workgroup of 8 waves takes 128 columns of y for an expert, a wave 16 of
// them (of the gated activation 16 of each half) over the whole contraction.

constexpr int kFewThreads = 512;

// 32 codes of a row's or column's block at k: pieces q and q + 4 of it.
__device__ __forceinline__ i32x8 piece(const uint8_t *row, int k, int q, int K)
{
    i32x4 lo = {}, hi = {};
    if (k + q * 16 < K)
        lo = *reinterpret_cast<const i32x4 *>(row + k + q * 16);
    if (k + q * 16 + 64 < K)
        hi = *reinterpret_cast<const i32x4 *>(row + k + q * 16 + 64);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The same of a column of a weight [K, N].
__device__ __forceinline__ i32x8 column(const uint8_t *col, int k, int q, int K, int N)
{
    i32x8 r = {};
    for (int i = 0; i < 32; ++i) {
        const int at = k + q * 16 + (i & 15) + (i >> 4) * 64;
        if (at < K)
            r[i / 4] |= (int)((uint32_t)col[(int64_t)at * N] << (8 * (i & 3)));
    }
    return r;
}

template <bool PAIRED>
__global__ __launch_bounds__(kFewThreads) void few_rows_kernel(Args a)
{
    __shared__ float most[2][8][16];
    const int e = blockIdx.y, nb = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, q = lane >> 4;
    const int F = PAIRED ? a.N / 2 : a.N;
    const int n = nb * kGroup + wave * 16;           // first column of the wave
    constexpr int J = PAIRED ? 2 : 1;
    int64_t lo;
    const int cnt = block_of(a, e, lo);
    const int nq = min(n + q * 4, F - 4);            // first column of the lane's quad
    const bool in = n + q * 4 < F;
    const uint8_t *w[J];
    for (int j = 0; j < J; ++j) {
        const int64_t c = min(n + r, F - 1) + j * F;
        w[j] = a.w8 + (int64_t)e * a.N * a.K + (a.in_out ? c : c * a.K);
    }
    float b[4], bu[4] = {0, 0, 0, 0};
    bias_of<4>(a, e, nq, b);
    if (PAIRED)
        bias_of<4>(a, e, F + nq, bu);
    for (int m = 0; m < cnt; m += 16) {
        const int64_t row = lo + min(m + r, cnt - 1);
        const bool live = m + r < cnt && in;
        f32x4 acc[J];
        for (int j = 0; j < J; ++j)
            acc[j] = f32x4{0, 0, 0, 0};
        for (int g = 0; g < blocks_of(a.K); ++g) {
            const i32x8 fx = piece(a.x8 + row * a.K, g * kGroup, q, a.K);
            const float sx = epl_cast::load_scale(a.xs, row, g);
            for (int j = 0; j < J; ++j) {
                const i32x8 fw = a.in_out ? column(w[j], g * kGroup, q, a.K, a.N)
                                          : piece(w[j], g * kGroup, q, a.K);
                const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    fw, fx, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
                const float s = sx * weight_scale(a, e, j * F + nq, g);
                for (int i = 0; i < 4; ++i)
                    acc[j][i] = fmaf(part[i], s, acc[j][i]);
            }
        }
        float z[4], u[4] = {0, 0, 0, 0};
        for (int i = 0; i < 4; ++i) {
            z[i] = acc[0][i];
            if (PAIRED)
                u[i] = acc[J - 1][i];
        }
        const bool two = a.act == EPL_ACT_SWIGLU_GRAD;
        const int cols = out_cols(a);
        if (live) {
            finish<4>(a, row, nq, b, bu, side_of<4>(a, row, nq), z, u);
            if (a.y) {
                epl_product::store_out<4>(a, row * cols + nq, z);
                if (two)
                    epl_product::store_out<4>(a, row * cols + F + nq, u);
            }
        }
        if (!a.codes)
            continue;
        for (int h = 0; h < (two ? 2 : 1); ++h) {
            float v = in ? largest(h ? u : z) : 0.0f;
            v = fmaxf(v, __shfl_xor(v, 16));
            v = fmaxf(v, __shfl_xor(v, 32));
            most[h][wave][r] = v;
        }
        __syncthreads();
        for (int h = 0; h < (two ? 2 : 1); ++h) {
            float v = 0.0f;
            for (int i = 0; i < 8; ++i)
                v = fmaxf(v, most[h][i][r]);
            const Factor f = epl_cast::factor_of(v, a.cs.format == EPL_SCALE_UE8M0);
            if (live)
                store_codes<4>(a, row * cols + h * F + nq, h ? u : z, f);
            if (live && wave == 0 && q == 0)
                epl_cast::store_scale(a.cs, row, (h * F + n) / kGroup, f);
        }
        __syncthreads();
    }
}

}  // namespace epl_product8
