// Device kernels of the 8-bit casts for gfx950 (CDNA4): rows and weights to
// e4m3 codes with a scale for each block of 128, and back.
//
//     fp32 scales   s = amax / 448,  code = e4m3(x * (448 / amax))
//     UE8M0         s = 2^k, the least with amax <= 448 s (k >= -126),
//                   code = e4m3(x * 2^-k)
// in binary32 steps, e4m3 to nearest even. Both directions are bound by the
// bytes of the rows: nothing is read twice. Measured: 32768 gated rows of 2 x 2048
// to codes 74 us, 29765 rows of 7168 back 141 us (4.5 TB/s both, a copy of 2 GiB
// 4.8-5.0), 8 weights of 4096 x 7168 135 us (5.2 TB/s). Few rows are a launch and
// two dependent reads: one row of 7168 3.5 us.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epl.h"
#include "epl_product_kernels.h"

namespace epl_cast {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kGroup = 128;            // columns (and rows of a weight) of a scale

// ------------------------------------------------------------- the cast --

// Scale and factor of a group whose largest magnitude is amax. A group with
// an infinity has factor 0 and an infinite (UE8M0: NaN) scale: its infinities
// become NaN codes. NaNs are no part of amax and become NaN codes.
struct Factor {
    float scale;              // fp32 scale
    uint32_t byte;            // or the exponent of a power of two, + 127
    float first, then;        // x * first * then is what is rounded
};
__device__ __forceinline__ Factor factor_of(float amax, bool power)
{
    Factor f;
    if (power) {
        // amax = m 2^e with 1 <= m < 2, 448 = 1.75 2^8
        const uint32_t u = __float_as_uint(amax);
        const uint32_t b = (u >> 23) + ((u & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
        f.byte = u >= 0x7F800000u ? 255u : b > 9u ? b - 8u : 1u;
        f.scale = 0.0f;
        f.first = 1.0f;
        f.then = f.byte == 255u ? 0.0f : __uint_as_float((254u - f.byte) << 23);
    } else {
        f.byte = 0;
        f.scale = amax / 448.0f;
        // 448 / amax leaves binary32 below 1.3e-36: such a group is first
        // scaled by 2^64, which changes no rounding
        f.first = amax < 0x1p-64f ? 0x1p64f : 1.0f;
        f.then = amax > 0.0f ? 448.0f / (amax * f.first) : 0.0f;
    }
    return f;
}

// Four codes in a word. |v| <= 448 (1 + 2^-22), which rounds to 448 at most.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Codes of N values (N % 4 == 0).
template <int N>
__device__ __forceinline__ void codes_of(const float (&v)[N], const Factor &f, uint32_t (&c)[N / 4])
{
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        c[i] = codes4(v[4 * i] * f.first * f.then, v[4 * i + 1] * f.first * f.then,
                      v[4 * i + 2] * f.first * f.then, v[4 * i + 3] * f.first * f.then);
}

// The value of an exponent byte: 0 stands for 2^-127, 255 for NaN.
__device__ __forceinline__ float power_of(uint32_t byte)
{
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Where the scales of rows lie (EPL_SCALE_*): fp32 [rows, groups], UE8M0 int32
// [ceil(groups / 4), rows], or fp32 [rows / cap, groups, cap].
struct Scales {
    void *at;
    int format;
    int groups;
    int cap;
    int64_t rows;
};

__device__ __forceinline__ int64_t scale_index(const Scales &s, int64_t row, int g)
{
    if (s.format == EPL_SCALE_F32_RECT) {
        const int64_t e = row / s.cap;
        return (e * s.groups + g) * s.cap + row - e * s.cap;
    }
    return row * s.groups + g;
}

__device__ __forceinline__ float load_scale(const Scales &s, int64_t row, int g)
{
    if (s.format == EPL_SCALE_UE8M0)
        return power_of(static_cast<const uint8_t *>(s.at)[((int64_t)(g >> 2) * s.rows + row) * 4 + (g & 3)]);
    return static_cast<const float *>(s.at)[scale_index(s, row, g)];
}

// The bytes behind the last group's in its word are zeros.
__device__ __forceinline__ void store_scale(const Scales &s, int64_t row, int g, const Factor &f)
{
    if (s.format == EPL_SCALE_UE8M0) {
        uint8_t *const at = static_cast<uint8_t *>(s.at) + ((int64_t)(g >> 2) * s.rows + row) * 4;
        at[g & 3] = (uint8_t)f.byte;
        if (g == s.groups - 1)
            for (int i = (g & 3) + 1; i < 4; ++i)
                at[i] = 0;
    } else {
        static_cast<float *>(s.at)[scale_index(s, row, g)] = f.scale;
    }
}

// Maximum over the 8 lanes 8m .. 8m + 7, all of which are active.
__device__ __forceinline__ float max8(float v)
{
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false)));
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false)));
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false)));
}

// ----------------------------------------------------------------- rows --

struct Args {
    const void *x;            // values (quantize)
    void *y;                  // values (dequantize)
    uint8_t *codes;
    Scales scales;
    const int32_t *start, *count;     // blocks of rows, or null: all rows
    int64_t rows;
    int E;                    // blocks; 1 without
    int C;                    // columns of the codes
};

// A workgroup of 4 waves takes tiles of kRows rows by kCols columns: 8 lanes to
// a group of 128 columns, 16 each, so that a wave reads and writes whole lines
// of up to 8 groups.
constexpr int kThreads = 256;
constexpr int kRows = 16;
constexpr int kCols = 8 * kGroup;
constexpr int kGrid = 2048;            // workgroups that the GPU holds at once

__device__ __forceinline__ void load16(const __bf16 *p, float (&v)[16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const u32x4 r = reinterpret_cast<const u32x4 *>(p)[h];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[8 * h + 2 * i] = __uint_as_float(r[i] << 16);
            v[8 * h + 2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ void load16(const float *p, float (&v)[16])
{
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const f32x4 r = reinterpret_cast<const f32x4 *>(p)[h];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[4 * h + i] = r[i];
    }
}

__device__ __forceinline__ void store16(__bf16 *p, const float (&v)[16])
{
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        bf16x8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r[i] = (__bf16)v[8 * h + i];
        reinterpret_cast<bf16x8 *>(p)[h] = r;
    }
}

__device__ __forceinline__ void store16(float *p, const float (&v)[16])
{
#pragma unroll
    for (int h = 0; h < 4; ++h)
        reinterpret_cast<f32x4 *>(p)[h] = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
}

// Calls item(row, group, lane of the group's 8, live) for every group of every
// owned row; the 8 lanes of a group come together, whether live or not.
template <typename F>
__device__ __forceinline__ void each_group(const Args &a, F &&item)
{
    __shared__ int32_t pre[epl_product::kMaxExperts + 1];
    __shared__ int32_t sums[8];
    const int S = a.scales.groups, chunks = (S + 7) / 8;
    auto rows_of = [&](int e, int64_t &lo) {
        lo = 0;
        return a.start ? epl_product::block_of(a, e, lo) : (int)a.rows;
    };
    epl_product::tile_prefix<kRows, kThreads>(a.E, a.rows, rows_of, pre, sums);
    const int64_t tiles = (int64_t)pre[a.E] * chunks;
    const int team = threadIdx.x >> 3, lane = threadIdx.x & 7;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int mt = (int)(t / chunks), chunk = (int)(t % chunks);
        const int e = epl_product::expert_of_tile(pre, a.E, mt);
        int64_t lo;
        const int cnt = rows_of(e, lo);
        const int m0 = (mt - pre[e]) * kRows;
        const int rows = min(cnt - m0, kRows), groups = min(S - chunk * 8, 8);
        const int items = rows * groups;
        const int by = 65536 / groups + 1;     // i / groups = i * by >> 16, i < 128, groups <= 8
#pragma unroll 2
        for (int i0 = team; i0 < ((items + 31) & ~31); i0 += 32) {
            const int i = min(i0, items - 1), row = i * by >> 16;
            item(lo + m0 + row, chunk * 8 + i - row * groups, lane, i0 < items);
        }
    }
}

template <typename T, bool GATED>
__global__ __launch_bounds__(kThreads) void quantize_kernel(Args a)
{
    const bool power = a.scales.format == EPL_SCALE_UE8M0;
    each_group(a, [&](int64_t row, int g, int lane, bool live) {
        const int c = g * kGroup + lane * 16;
        float v[16];
        if (c < a.C) {
            const T *x = static_cast<const T *>(a.x) + row * a.C * (GATED ? 2 : 1) + c;
            load16(x, v);
            if (GATED) {
                float u[16];
                load16(x + a.C, u);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] = epl_product::silu(v[i]) * u[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = 0.0f;
        }
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            amax = fmaxf(amax, fabsf(v[i]));
        const Factor f = factor_of(max8(amax), power);
        uint32_t w[4];
        codes_of(v, f, w);
        if (live && c < a.C)
            *reinterpret_cast<u32x4 *>(a.codes + row * a.C + c) = u32x4{w[0], w[1], w[2], w[3]};
        if (live && lane == 0)
            store_scale(a.scales, row, g, f);
    });
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(Args a)
{
    each_group(a, [&](int64_t row, int g, int lane, bool live) {
        const int c = g * kGroup + lane * 16;
        if (!live || c >= a.C)
            return;
        const float s = load_scale(a.scales, row, g);
        const u32x4 w = *reinterpret_cast<const u32x4 *>(a.codes + row * a.C + c);
        float v[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
            v[4 * i] = lo[0] * s, v[4 * i + 1] = lo[1] * s;
            v[4 * i + 2] = hi[0] * s, v[4 * i + 3] = hi[1] * s;
        }
        store16(static_cast<T *>(a.y) + row * a.C + c, v);
    });
}

// -------------------------------------------------------------- weights --
//
// A workgroup takes blocks of 128 x 128, which its registers hold between the
// maximum and the rounding: one block, but where there are more of them than a
// launch may have workgroups (2^32 threads), as of 2048 weights of 2^20 columns.

struct WeightArgs {
    const void *w;            // [E, N, K]
    uint8_t *codes;
    void *scale;              // [E, N / 128, K / 128] fp32 or uint8
    int N, K, power;
    int64_t blocks;
};

constexpr int kWeightGrid = 1 << 23;   // workgroups at most

template <typename T>
__device__ __forceinline__ void quantize_block(const WeightArgs &a, int b, float *most)
{
    const int kb = (a.K + kGroup - 1) / kGroup, nb = (a.N + kGroup - 1) / kGroup;
    const int64_t e = b / (nb * kb);
    const int n0 = b / kb % nb * kGroup, k0 = b % kb * kGroup;
    const int tid = threadIdx.x, k = k0 + (tid & 7) * 16, n = n0 + (tid >> 3);
    const int64_t at = (e * a.N + n) * a.K + k;
    float v[4][16];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (k < a.K && n + 32 * i < a.N) {
            load16(static_cast<const T *>(a.w) + at + (int64_t)32 * i * a.K, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[i][j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
            amax = fmaxf(amax, fabsf(v[i][j]));
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        amax = fmaxf(amax, __shfl_xor(amax, d));
    if ((tid & 63) == 0)
        most[tid >> 6] = amax;
    __syncthreads();
    const Factor f = factor_of(fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])), a.power);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (k < a.K && n + 32 * i < a.N) {
            uint32_t c[4];
            codes_of(v[i], f, c);
            *reinterpret_cast<u32x4 *>(a.codes + at + (int64_t)32 * i * a.K) =
                u32x4{c[0], c[1], c[2], c[3]};
        }
    }
    if (tid == 0) {
        if (a.power)
            static_cast<uint8_t *>(a.scale)[b] = (uint8_t)f.byte;
        else
            static_cast<float *>(a.scale)[b] = f.scale;
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_weight_kernel(WeightArgs a)
{
    __shared__ float most[4];
    for (int64_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
        if (b != blockIdx.x)
            __syncthreads();           // the block before has been rounded
        quantize_block<T>(a, (int)b, most);
    }
}

}  // namespace epl_cast
