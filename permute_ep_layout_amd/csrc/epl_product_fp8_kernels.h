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
// 2^(E - 13) (towards zero; measured), E the largest sum of two codes' exponents
// among the group's products that are not zero, a subnormal code's being -6; the
// groups are added in binary32. The product of E is at least 2^E, or with a
// subnormal code 2^(E - 3) (with two, products are multiples of 2^-18 and lose
// nothing), so that the seven others lose at most 7 2^-13, or 7 2^-10, of the sum
// of the magnitudes. Against exact sums that is about 2^-16 of the result for
// normal data, and it is what twice the rate of bf16 costs: the codes themselves
// are off by up to 2^-4.
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
    const void *wscale;       // of the weight: [E, blocks of out, blocks of in] as it lies
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

// The scale of block nb of an expert's columns and block b of the contraction
// (weight [E, N, K]).
__device__ __forceinline__ float weight_scale(const Args &a, int e, int nb, int b)
{
    const int64_t at = ((int64_t)e * blocks_of(a.N) + nb) * blocks_of(a.K) + b;
    return a.ws_bytes ? epl_cast::power_of(static_cast<const uint8_t *>(a.wscale)[at])
                      : static_cast<const float *>(a.wscale)[at];
}

// The finished values of C columns n .. of one row, from z, product and bias: z is
// column n of y, and u column N + n (gradient of the gated activation). Of the
// gated activation z and u are the gate's and the up half's product, and z the
// result. kept: what the backward pass is left of both.
template <int C>
struct Kept {
    typedef __bf16 vec __attribute__((ext_vector_type(C)));
    vec z, u;
};

template <int C, bool PAIRED>
__device__ __forceinline__ void finish(const Args &a, const Side<C> &s, float (&z)[C], float (&u)[C],
                                       Kept<C> &kept)
{
    using namespace epl_product;
    if (!PAIRED && a.act == EPL_ACT_SWIGLU_GRAD) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            u[i] = z[i] * silu((float)s.x[i]);
            z[i] = z[i] * (float)s.y[i] * silu_slope((float)s.x[i]);
        }
        return;
    }
    if (!PAIRED && a.act >= EPL_ACT_SILU_GRAD) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            z[i] *= a.act == EPL_ACT_SILU_GRAD ? silu_slope((float)s.x[i]) : gelu_slope((float)s.x[i]);
        return;
    }
    if (a.pre) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            kept.z[i] = (__bf16)z[i];
            if (PAIRED)
                kept.u[i] = (__bf16)u[i];
        }
    }
    if (PAIRED) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            z[i] = silu(z[i]) * u[i];
    } else if (a.act == EPL_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            z[i] = silu(z[i]);
    } else if (a.act == EPL_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            z[i] = gelu(z[i]);
    }
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            z[i] += (float)s.x[i];
    }
}

// What finish() leaves, to memory: the kept product past the caches (it is
// read by the backward pass, much later), and y.
template <int C, bool PAIRED>
__device__ __forceinline__ void store_row(const Args &a, int64_t row, int n, const float (&z)[C],
                                          const float (&u)[C], const Kept<C> &kept)
{
    typedef typename Kept<C>::vec vec;
    if (a.pre && a.act <= EPL_ACT_SWIGLU) {
        __builtin_nontemporal_store(kept.z, reinterpret_cast<vec *>(a.pre + row * a.N + n));
        if (PAIRED)
            __builtin_nontemporal_store(kept.u, reinterpret_cast<vec *>(a.pre + row * a.N + a.N / 2 + n));
    }
    if (a.y) {
        const int64_t at = row * out_cols(a) + n;
        epl_product::store_out<C>(a, at, z);
        if (!PAIRED && a.act == EPL_ACT_SWIGLU_GRAD)
            epl_product::store_out<C>(a, at + a.N, u);
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

// ----------------------------------------------------------- tile kernel --
//
// The tile kernel of the bf16 products on bytes: a workgroup of 8 (or 4) waves
// computes BM x BN outputs, one block of 128 of the contraction at a time, from
// two LDS stages that buffer loads fill while the other is multiplied. The
// weight is the matrix instruction's A operand and the rows its B operand, so
// that a lane's quad (i, j) holds row 16 i + r of the wave's rows (lane 16 q +
// r) and columns 16 j + 4 q .. + 3: one scale of x for the quad, and one of the
// weight. A lane's 32 k of an instruction are the 16-byte pieces q and q + 4 of
// the block, for both operands alike.
//
// LDS: a contiguous operand as there (128 bytes a row, pieces swizzled by row);
// a strided weight [128][BN] with piece c of row k at c ^ swz_t8(k), read with
// ds_read_b64_tr_b8, which hands lane r of 16 column r of 8 rows, so that the 8
// rows of two such groups fall on different banks.
//
// The scales of a block (of BM rows and of BN / 8 pieces of 8 columns) come
// through registers: a thread loads one of them two stages ahead, and writes it
// to LDS, as a number, before the barrier that ends the wait for it.
//
// Columns of the gated activation alternate by 16, gate and up.
//
// Measured: 8 x 4096 rows, 7168 -> 4096, 1045-1070 us, 1.8 PFLOP/s (gated and cast
// 930, powers of two as scales 915-925), where a library's product with one scale
// reaches 2.5-2.7: a tile of 56 blocks 131 us, of 16 43. The matrix units are busy for
// 45% of the cycles at 2.1 GHz. What bounds it is x's loads, with one block's products
// to arrive under, and the epilogue, 8 to 10 us a tile: before weights were loaded early
// it took 1080 us, then without its loads 800, with all of them in L2 950, without its
// epilogue 1000. LDS holds no third stage of 64 KB, and smaller tiles load more. Loads
// of a further block into L2 alone gained 2% then, starts of the XCDs 10 to 20 us apart
// nothing; the epilogue's passes as one loop (less code, but spilled sums) lost 5 to 9%.
// Start, launch and epilogue of one round of large tiles (256 tiles, over 8 to 56 blocks,
// extrapolated to none): 20 us, transposed 22, with a cast 45, gated gradient 34, and with
// its cast 70.

using epl_product::at;
using epl_product::dma;
using epl_product::each;
using epl_product::landed;
using epl_product::Plan;
using epl_product::put;
using epl_product::rsrc;
using epl_product::swz;
using epl_product::take;
using epl_product::Tile;
using epl_product::tile_threads;
using epl_product::waves_n;

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;

constexpr int kWavesM = epl_product::kWavesM;

template <int BN>
__device__ __forceinline__ int swz_t8(int k)
{
    return BN == 256 ? (k & 7) | ((k >> 4 & 1) << 3) : (k >> 1 & 3) | ((k >> 4 & 1) << 2);
}

// Column of the product (in [0, N) or beyond) of column c of tile tn.
template <int BN>
__device__ __forceinline__ int column_of(const Args &a, int tn, int c)
{
    return a.act == EPL_ACT_SWIGLU ? tn * (BN / 2) + (c >> 5) * 16 + (c & 15) + (c >> 4 & 1) * (a.N / 2)
                                   : tn * BN + c;
}

// 32 codes of one column from a strided weight's stage [128][BN].
template <int BN>
__device__ __forceinline__ i32x8 read_tr8(const uint16_t *at)
{
    const uint8_t *p = reinterpret_cast<const uint8_t *>(at);
    const i32x2 a = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2 *)p);
    const i32x2 b = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2 *)(p + 8 * BN));
    const i32x2 c = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2 *)(p + 64 * BN));
    const i32x2 d = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2 *)(p + 72 * BN));
    return i32x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The epilogue of ROWS rows of 64 columns that a wave holds in its part of LDS
// (as epl_product::emit_rows): a lane takes 8 neighbouring columns of y. m0:
// the first row in the tile's block. With CODES every wave of the workgroup
// comes here together, and the values stay in registers until the waves that
// share a group of 128 columns have exchanged their largest.
template <int BN, int ROWS, bool CODES, bool PAIRED>
__device__ __forceinline__ void emit_rows(const Args &a, const Tile &x, const float *mine, int m0,
                                          int lane, int wm, int wn, float *most)
{
    constexpr int LANES = PAIRED ? 4 : 8, STEP = 64 / LANES, TURNS = ROWS / STEP;
    constexpr int WN = waves_n(BN), SHARE = PAIRED ? 4 : 2;        // waves of a group
    const int c = lane % LANES * 8;
    const int n = PAIRED ? x.tn * (BN / 2) + wn * 32 + c : x.tn * BN + wn * 64 + c;
    const int at = PAIRED ? (c >> 4) * 32 + (c & 15) : c;          // column in LDS
    const int F = PAIRED ? a.N / 2 : a.N, cols = out_cols(a);
    const bool in = n < F, two = !PAIRED && a.act == EPL_ACT_SWIGLU_GRAD;
    if (!CODES && !in)
        return;
    float b[8] = {}, bu[8] = {};
    if (in) {
        bias_of<8>(a, x.e, n, b);
        if (PAIRED)
            bias_of<8>(a, x.e, F + n, bu);
    }
    constexpr int AHEAD = CODES ? TURNS : TURNS < 4 ? TURNS : 4;
#pragma unroll 1
    for (int t0 = 0; t0 < TURNS; t0 += AHEAD) {
        Side<8> s[AHEAD];
        float v[AHEAD][8], u[AHEAD][8];
        if (in) {
#pragma unroll
            for (int t = 0; t < AHEAD; ++t)
                s[t] = side_of<8>(a, x.lo + min(m0 + (t0 + t) * STEP + lane / LANES, x.cnt - 1), n);
        }
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) {
            const int row = (t0 + t) * STEP + lane / LANES;
            const int64_t p = x.lo + m0 + row;
            const bool live = in && m0 + row < x.cnt;
            take<8>(mine, row, at, v[t]);
            if (PAIRED)
                take<8>(mine, row, at + 16, u[t]);
            if (live) {
                Kept<8> kept;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[t][i] += b[i];
                    if (PAIRED)
                        u[t][i] += bu[i];
                }
                finish<8, PAIRED>(a, s[t], v[t], u[t], kept);
                store_row<8, PAIRED>(a, p, n, v[t], u[t], kept);
            }
            if (CODES) {
                for (int h = 0; h < (two ? 2 : 1); ++h) {
                    float m = largest(h ? u[t] : v[t]);
#pragma unroll
                    for (int d = 1; d < LANES; d <<= 1)
                        m = fmaxf(m, __shfl_xor(m, d));
                    if (lane % LANES == 0)
                        most[((h * kWavesM + wm) * ROWS + row) * WN + wn] = m;
                }
            }
        }
        if (CODES) {
            __syncthreads();
#pragma unroll
            for (int t = 0; t < AHEAD; ++t) {
                const int row = (t0 + t) * STEP + lane / LANES;
                const int64_t p = x.lo + m0 + row;
                for (int h = 0; h < (two ? 2 : 1); ++h) {
                    const float *of = most + ((h * kWavesM + wm) * ROWS + row) * WN + wn / SHARE * SHARE;
                    float m = fmaxf(of[0], of[1]);
                    if (PAIRED)
                        m = fmaxf(m, fmaxf(of[2], of[3]));
                    const Factor f = epl_cast::factor_of(m, a.cs.format == EPL_SCALE_UE8M0);
                    if (in && m0 + row < x.cnt) {
                        store_codes<8>(a, p * cols + h * F + n, h ? u[t] : v[t], f);
                        if (wn % SHARE == 0 && lane % LANES == 0)
                            epl_cast::store_scale(a.cs, p, (h * F + n) / kGroup, f);
                    }
                }
            }
            __syncthreads();                   // the next rows' maxima overwrite these
        }
    }
}

template <int BN, int ROWS, bool CODES>
__device__ __forceinline__ void emit_any(const Args &a, const Tile &x, const float *mine, int m0,
                                         int lane, int wm, int wn, float *most)
{
    if (a.act == EPL_ACT_SWIGLU) {
        if constexpr (!CODES || BN == 256)
            emit_rows<BN, ROWS, CODES, true>(a, x, mine, m0, lane, wm, wn, most);
    } else {
        emit_rows<BN, ROWS, CODES, false>(a, x, mine, m0, lane, wm, wn, most);
    }
}

// All loads are done but the last N that this wave began.
template <int N>
__device__ __forceinline__ void all_but()
{
    static_assert(N < 64, "the counter's width");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0070);       // (and lgkmcnt(0))
}

// All waves of the workgroup have come here, and (N >= 0) what each loaded into LDS
// but its last N loads has landed, and what it wrote. (A fence would wait for
// all loads.)
template <int N = -1>
__device__ __forceinline__ void met()
{
    asm volatile("" ::: "memory");
    if constexpr (N >= 0)
        all_but<N>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// acc + by * sum, each rounded once. (by, a row's scale times a weight's, comes
// first: by * sum with the scales in turn would be three more instructions a quad,
// and where one order leaves binary32 the other may too.)
__device__ __forceinline__ f32x4 scaled(f32x4 sum, float by, f32x4 acc)
{
    return __builtin_elementwise_fma(sum, f32x4{by, by, by, by}, acc);
}

// Rows of a wave that the epilogue takes at a time.
template <bool CODES>
constexpr int epilogue_rows(int bm) { return bm / kWavesM / (CODES && bm == 256 ? 4 : 2); }

template <int BM, int BN, bool QT, bool CODES>
__global__ __launch_bounds__(tile_threads(BN), 2) void tile_kernel(Args a)
{
    constexpr int WN = waves_n(BN), WM = kWavesM, WAVES = WM * WN;
    constexpr int IP = BM / WM / 16;                     // 16-row pieces of x a wave
    constexpr int ROWS = WAVES * 8;                      // rows of a contiguous operand a DMA
    constexpr int ISP = BM / ROWS, ISQ = BN / ROWS;      // DMAs a stage
    constexpr int KQ = WAVES * 1024 / BN;                // rows of a strided one
    constexpr int BYTES = 128;                           // of a row in a stage
    constexpr int SCALES = BM + BN / 8;
    constexpr int EROWS = epilogue_rows<CODES>(BM);
    __shared__ __align__(1024) uint16_t sp0[BM * 64], sp1[BM * 64];
    __shared__ __align__(1024) uint16_t sq0[BN * 64], sq1[BN * 64];
    __shared__ float sc0[SCALES], sc1[SCALES];
    __shared__ float most[CODES ? 2 * WM * EROWS * WN : 1];
    __shared__ int32_t pre[epl_product::kMaxExperts + 1];
    __shared__ int32_t sums[8];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, r = lane & 15, q = lane >> 4;

    // the lane's LDS offsets (bytes) of its first pieces
    int aq[2], ap[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int n = wn * 64 + r, m = wm * (BM / WM) + r, k = q * 16 + (r >> 1);
        aq[h] = QT ? k * BN + ((wn * 4) ^ swz_t8<BN>(k)) * 16 + (r & 1) * 8
                   : n * BYTES + ((h * 4 + q) ^ swz(n)) * 16;
        ap[h] = m * BYTES + ((h * 4 + q) ^ swz(m)) * 16;
    }
    const int asx = wm * (BM / WM) + r, asw = BM + wn * 8 + (q >> 1);

    const int ntn = (a.N + BN - 1) / BN;
    epl_product::tile_prefix<BM, WAVES * 64>(a, pre, sums);
    const int64_t total = (int64_t)pre[a.E] * ntn;

    // workgroups of one XCD (every eighth) take neighbouring tiles
    const int grid = gridDim.x;
    int64_t first = blockIdx.x;
    if (grid % epl_product::kNumXcd == 0)
        first = (first % epl_product::kNumXcd) * (grid / epl_product::kNumXcd) + first / epl_product::kNumXcd;
    const Plan plan = epl_product::plan_of<BM>(a, total, grid);
    const int64_t items = plan.whole + plan.left * plan.parts;
    if (a.ws && blockIdx.x == 0 && tid == 0)
        a.header[0] = plan.left;

    for (int64_t item = first; item < items; item += grid) {
        const bool split = item >= plan.whole;
        const int o = split ? (int)(item - plan.whole) : 0;
        const int part = split ? o / plan.left : 0, rest = split ? o % plan.left : 0;
        const Tile x = epl_product::locate<epl_product::kForward>(a, pre, split ? plan.whole + rest : item,
                                                                  0, ntn);
        const int e = x.e, cnt = x.cnt, tm = x.tm, tn = x.tn;
        const int64_t lo = x.lo;

        // opaque: what is derived from the lane for one tile is not kept for the next
        int own = tid;
        asm volatile("" : "+v"(own));
        const int steps = blocks_of(a.K);
        const int s0 = split ? steps * part / plan.parts : 0;
        const int s1 = split ? steps * (part + 1) / plan.parts : steps;
        // experts start at different places of the contraction (epl_product::tile_kernel)
        const int turns = s1 - s0;
        const int rot = turns > 0 ? (int)((uint32_t)(e * 13) % (uint32_t)turns) : 0;
        const char *bp, *bq;
        uint32_t op, oq;
        int np, nq = 0, kp, kq = 0;
        const int ip = ROWS * a.K;
        const int iq = QT ? KQ * a.N : (a.act == EPL_ACT_SWIGLU ? ROWS / 2 : ROWS) * a.K;
        {
            const int row = own >> 3, c = (own & 7) ^ swz(row);
            op = (uint32_t)row * a.K + c * 16;
            kp = c * 16;
            bp = reinterpret_cast<const char *>(a.x8 + (lo + (int64_t)tm * BM) * a.K);
            np = min(cnt - tm * BM, BM) * a.K;
        }
        bq = reinterpret_cast<const char *>(a.w8 + (int64_t)e * a.K * a.N);
        if (QT) {
            const int k = own * 16 / BN, c = (own * 16 % BN / 16) ^ swz_t8<BN>(k);
            oq = (uint32_t)k * a.N + column_of<BN>(a, tn, c * 16);
        } else {
            const int row = own >> 3, c = (own & 7) ^ swz(row);
            oq = (uint32_t)column_of<BN>(a, tn, row) * a.K + c * 16;
            kq = c * 16;
            nq = a.N * a.K;
        }
        // the thread's scale: of row tm BM + tid, or of 8 columns
        const bool of_x = wave < BM / 64;    // (the same for a wave)
        const char *scale = nullptr;
        bool small = false;                  // an exponent byte
        int64_t per_block = 0;               // bytes to the next block's, or 4 blocks'
        if (of_x) {
            const int64_t p = lo + min(tm * BM + own, cnt - 1);
            const char *base = static_cast<const char *>(a.xs.at);
            if (a.xs.format == EPL_SCALE_UE8M0) {
                scale = base + p * 4;
                per_block = a.rows * 4;
                small = true;
            } else {
                scale = base + epl_cast::scale_index(a.xs, p, 0) * 4;
                per_block = a.xs.format == EPL_SCALE_F32_RECT ? (int64_t)a.xs.cap * 4 : 4;
            }
        } else if (own < SCALES) {
            const int n = min(column_of<BN>(a, tn, (own - BM) * 8), a.N - 1);
            const int nb = blocks_of(a.N), kb = blocks_of(a.K), size = a.ws_bytes ? 1 : 4;
            scale = static_cast<const char *>(a.wscale) +
                    ((int64_t)e * nb * kb + (int64_t)(n / kGroup) * (QT ? 1 : kb)) * size;
            per_block = (QT ? nb : 1) * size;
            small = a.ws_bytes;
        }

        f32x4 acc[IP * 4];
        each<IP * 4>([&](auto i) { acc[i] = f32x4{0, 0, 0, 0}; });

        struct Stage {
            __amdgpu_buffer_rsrc_t r;
            uint32_t o;
        };
        auto block_at = [&](int s) { const int v = s + rot; return v < s1 ? v : v - turns; };
        auto stage_p = [&](int s) {
            const int k0 = block_at(s) * kGroup, left = s < s1 ? min(a.K - k0, kGroup) : 0;
            return Stage{rsrc(bp + k0, np - k0), kp >= left ? op | 0x80000000u : op};
        };
        auto stage_q = [&](int s) {
            const int k0 = block_at(s) * kGroup, left = s < s1 ? min(a.K - k0, kGroup) : 0;
            if (QT)
                return Stage{rsrc(bq + (int64_t)k0 * a.N, left * a.N), oq};
            return Stage{rsrc(bq + k0, nq - k0), kq >= left ? oq | 0x80000000u : oq};
        };
        auto fetch_p = [&](const Stage &f, uint16_t *l, auto i) {
            dma(f.r, f.o + i * ip, l + i * WAVES * 512 + wave * 512);
        };
        auto fetch_q = [&](const Stage &f, uint16_t *l, auto i) {
            dma(f.r, f.o + i * iq, l + i * WAVES * 512 + wave * 512);
        };
        auto load_scale = [&](int s) {
            uint32_t v = 0;
            if (scale && s < s1) {
                const int b = block_at(s);
                if (small && of_x)
                    v = *reinterpret_cast<const uint8_t *>(scale + (b >> 2) * per_block + (b & 3));
                else if (small)
                    v = *reinterpret_cast<const uint8_t *>(scale + b * per_block);
                else
                    v = *reinterpret_cast<const uint32_t *>(scale + b * per_block);
            }
            return v;
        };
        auto write_scale = [&](float *sc, uint32_t v) {
            if (own < SCALES)
                sc[own] = small ? epl_cast::power_of(v) : __uint_as_float(v);
        };

        i32x8 fq[4], fp[2];
        float sx[2], sw[4];
        f32x4 sum[4];                        // blocks' sums on their way, and their scales
        float by[4];
        each<4>([&](auto i) { sum[i] = f32x4{0, 0, 0, 0}, by[i] = 0.0f; });
        auto pair = [&](const uint16_t *l, const int (&o2)[2], int rows) {
            const i32x4 l0 = *reinterpret_cast<const i32x4 *>(at(l, o2[0], rows * 64));
            const i32x4 l1 = *reinterpret_cast<const i32x4 *>(at(l, o2[1], rows * 64));
            return __builtin_shufflevector(l0, l1, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        auto read_q = [&](const uint16_t *lq, auto j) {
            if constexpr (QT)
                fq[j] = read_tr8<BN>(at(lq, aq[0] ^ (j * 16), 0));
            else
                fq[j] = pair(lq, aq, j * 16);
        };
        auto read_p = [&](const uint16_t *lp, const float *sc, auto g) {
            fp[g % 2] = pair(lp, ap, g * 16);
            sx[g % 2] = sc[asx + g * 16];
        };
        // Quad t = 4 g + j of a block: its sum starts; the sum that started three
        // instructions before, which is done by now, is added to its accumulators.
        auto multiply = [&](auto t) {
            constexpr int g = t / 4, j = t % 4, old = (t + 4 * IP - 3) % (4 * IP);
            sum[t % 4] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                fq[j], fp[g % 2], f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
            by[t % 4] = sx[g % 2] * sw[j];
            acc[old] = scaled(sum[old % 4], by[old % 4], acc[old]);
            // here, and not after the loop: the sums would have to wait in memory
            asm volatile("" : "+v"(acc[old]));
        };
        // One block: IP groups of 4 products, one piece of x each. A group's
        // reads of the next piece run under its products. The weight's part of a
        // stage has been read by all waves when they meet in the second group
        // (its codes wait in registers), and loads of the next stage but one
        // begin to overwrite it there; x's has when they meet before the last
        // group, where the next stage has landed too. The last group's products
        // free the weight's registers one by one for the next stage's. So weights
        // have nearly two blocks' products to arrive under, and x one (8 x 4096
        // rows, 7168 -> 4096, gated and cast: 930 us; both begun before and after the
        // last group, with one meeting, 970; all of them there 1000).
        constexpr int kNow = ISP / 2, per = (ISQ + IP - 4) / (IP - 3);
        static_assert((IP - 2) * per >= ISQ, "all of the weight's loads begin before the last group");
        Stage afterp;                        // the next stage's x
        uint32_t coming = 0;                 // the thread's scale of the next stage
        auto turn = [&](int s, uint16_t *cp, uint16_t *cq, float *cs, uint16_t *xp, uint16_t *xq,
                        float *xs) {
            Stage afterq;
            each<IP>([&](auto g) {
                if constexpr (g + 1 < IP)
                    read_p(cp, cs, std::integral_constant<int, g + 1>{});
                if constexpr (g == IP - 1) {
                    write_scale(xs, coming);
                    met<ISQ>();
                    afterp = stage_p(s + 2);
                    coming = load_scale(s + 2);
                }
                if constexpr (g == 0)
                    each<ISP - kNow>([&](auto i) {
                        fetch_p(afterp, xp, std::integral_constant<int, kNow + decltype(i)::value>{});
                    });
                if constexpr (g == 1) {
                    met();
                    afterq = stage_q(s + 2);
                }
                if constexpr (g >= 1 && g < IP - 1) {
                    each<per>([&](auto i) {
                        constexpr std::integral_constant<
                            int, (decltype(g)::value - 1) * per + decltype(i)::value> d{};
                        if constexpr (d < ISQ)
                            fetch_q(afterq, cq, d);
                    });
                }
                each<4>([&](auto j) {
                    multiply(std::integral_constant<int, g * 4 + j>{});
                    if constexpr (g == IP - 1) {
                        read_q(xq, j);
                        if constexpr (j < kNow)
                            fetch_p(afterp, cp, j);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                });
                if constexpr (g == IP - 1) {
                    read_p(xp, xs, std::integral_constant<int, 0>{});
                    each<4>([&](auto j) { sw[j] = xs[asw + j * 2]; });
                }
            });
        };
        coming = load_scale(s0);
        {
            const Stage p0 = stage_p(s0), q0 = stage_q(s0);
            each<ISP>([&](auto i) { fetch_p(p0, sp0, i); });
            each<ISQ>([&](auto i) { fetch_q(q0, sq0, i); });
        }
        write_scale(sc0, coming);
        landed();
        {
            const Stage q1 = stage_q(s0 + 1);
            each<ISQ>([&](auto i) { fetch_q(q1, sq1, i); });
        }
        afterp = stage_p(s0 + 1);
        each<kNow>([&](auto i) { fetch_p(afterp, sp1, i); });
        coming = load_scale(s0 + 1);
        each<4>([&](auto j) {
            read_q(sq0, j);
            sw[j] = sc0[asw + j * 2];
        });
        read_p(sp0, sc0, std::integral_constant<int, 0>{});
        for (int s = s0; s < s1; s += 2) {
            turn(s, sp0, sq0, sc0, sp1, sq1, sc1);
            turn(s + 1, sp1, sq1, sc1, sp0, sq0, sc0);
        }
        each<3>([&](auto i) {                // the last three sums
            constexpr int old = 4 * IP - 3 + i;
            acc[old] = scaled(sum[old % 4], by[old % 4], acc[old]);
        });
        landed();                            // (what was fetched past the end too)

        own = tid & 63;
        asm volatile("" : "+v"(own));
        const int er = own & 15, eq = own >> 4;
        if (split) {
            // registers as they are; join_kernel reads them alike
            f32x4 *slot = a.ws + (int64_t)(rest * plan.parts + part) * (BM * BN / 4);
            each<IP * 4>([&](auto y) { slot[((y / 4 * WAVES + wave) * 4 + y % 4) * 64 + own] = acc[y]; });
        } else {
            // some of the wave's rows at a time through its part of the stages
            constexpr int share = WAVES / 4;       // waves to a stage array
            uint16_t *const stages = wave < share       ? sp0
                                     : wave < 2 * share ? sp1
                                     : wave < 3 * share ? sq0
                                                        : sq1;
            float *const mine = reinterpret_cast<float *>(stages) + wave % share * EROWS * 64;
            constexpr int pieces = EROWS / 16;
            each<IP / pieces>([&](auto h) {
                each<pieces>([&](auto i) {
                    each<4>([&](auto j) {
                        put(mine, i * 16 + er, j * 4 + eq, acc[(h * pieces + i) * 4 + j]);
                    });
                });
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
                emit_any<BN, EROWS, CODES>(a, x, mine, tm * BM + wm * (BM / WM) + h * EROWS, own, wm, wn, most);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
            });
            __syncthreads();       // the next tile's stages overwrite the other waves' parts
        }
    }
}

// Adds the parts of the tiles that tile_kernel split, in order, and runs their
// epilogue (as epl_product::join_kernel).
template <int BM, int BN, bool CODES>
__global__ __launch_bounds__(tile_threads(BN)) void join_kernel(Args a, int grid)
{
    constexpr int WN = waves_n(BN), WM = kWavesM, WAVES = WM * WN;
    __shared__ __align__(16) float rows[WAVES * 16 * 64];
    __shared__ float most[CODES ? 2 * WM * 16 * WN : 1];
    __shared__ int32_t pre[epl_product::kMaxExperts + 1];
    __shared__ int32_t sums[8];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
    if (a.header[0] == 0)
        return;
    const int i = blockIdx.x, ntn = (a.N + BN - 1) / BN;
    epl_product::tile_prefix<BM, WAVES * 64>(a, pre, sums);
    const Plan plan = epl_product::plan_of<BM>(a, (int64_t)pre[a.E] * ntn, grid);
    for (int l = blockIdx.y; l < plan.left; l += gridDim.y) {
        const Tile x = epl_product::locate<epl_product::kForward>(a, pre, plan.whole + l, 0, ntn);
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
        float *mine = rows + wave * 16 * 64;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            put(mine, r, j * 4 + q, acc[j]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        emit_any<BN, 16, CODES>(a, x, mine, x.tm * BM + wm * (BM / WM) + i * 16, lane, wm, wn, most);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    }
}

// ------------------------------------------------------ few-rows kernel --
//
// For experts with a few rows the weights' bytes are the cost: each is read
// once for 16 or 32 rows, straight into the registers of the matrix
// instruction. A workgroup takes G times 16 columns of y for an expert (of the
// gated activation as many of each half), a wave 16 of them; the KS waves of
// the same columns take every KS-th block of the contraction each and add
// their sums through LDS in order. The rows and all scales come through LDS,
// where the G waves share them (from memory into each wave's registers 8 x 8
// rows, 7168 -> 4096 took 61 us, 8 x 1 48: their bytes are few but go through
// the same caches G times). Workgroups start at different places of the
// contraction and come round, as those of the bf16 products.
//
// Measured: 8 x 8 rows, 7168 -> 4096, gated, 47 us: 5.0 TB/s of weights (cast as well
// 54); 64 x 1, 4096 -> 2048, 93 us, 5.8 TB/s; 8 x 24 as the first 55.
//
// An expert's rows are taken 32 at a time, in turn, by the same workgroup: 64 experts,
// 4096 -> 2048, 1536 rows, 112 us evenly spread, 304 with half of them at one expert
// (tiles 134).
//
// A CU reads no more than some 35 GB/s in this way. Where the columns are too
// few for a workgroup on every CU, `parts` workgroups share the contraction,
// and few_join_kernel adds their sums in order.

template <int WAVES>
constexpr int few_threads() { return WAVES * 64; }

// Blocks of the contraction that LDS holds the rows of at a time: 128 KB of
// them, or 64 KB where two workgroups share a CU. A thread loads one scale of
// the rows for each time.
template <int WAVES, int MT>
constexpr int few_blocks() { return WAVES * 4 / MT; }

// Rows of an expert up to which its contraction is shared.
constexpr int kFewMost = 32;

struct FewShared {
    uint8_t *x;               // [blocks][16 MT][128], pieces swizzled by row
    float *sx, *sw;           // [blocks + 1][16 MT], [blocks + 1][4], zeros last
    f32x4 *red;               // in x, when that has been read
    float *most;
};

// The epilogue of row tile i (16 rows from row0 + 16 i on) by the G waves of a
// workgroup that hold its sums. All waves of the workgroup come here; `mine`:
// this one holds sums.
template <bool PAIRED, int G, int MT>
__device__ __forceinline__ void few_finish(const Args &a, int e, int64_t row0, int left, int nb, int g, int i,
                                           bool mine, const f32x4 (&sum)[PAIRED ? 2 : 1], float *most)
{
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int F = PAIRED ? a.N / 2 : a.N, n0 = (nb * G + g) * 16, nq = min(n0 + q * 4, F - 4);
    const int64_t row = row0 + min(i * 16 + r, left - 1);
    const bool live = mine && i * 16 + r < left && n0 + q * 4 < F;
    const bool two = !PAIRED && a.act == EPL_ACT_SWIGLU_GRAD;
    const int cols = out_cols(a);
    float z[4] = {}, u[4] = {};
    if (mine) {
        float b[4], bu[4];
        bias_of<4>(a, e, nq, b);
        bias_of<4>(a, e, PAIRED ? F + nq : nq, bu);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            z[k] = sum[0][k] + b[k];
            if (PAIRED)
                u[k] = sum[PAIRED ? 1 : 0][k] + bu[k];
        }
        Kept<4> kept;
        finish<4, PAIRED>(a, side_of<4>(a, row, nq), z, u, kept);
        if (live)
            store_row<4, PAIRED>(a, row, nq, z, u, kept);
    }
    if constexpr (G == 8) {
        if (!a.codes)
            return;
        if (mine) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v = largest(h ? u : z);
                v = fmaxf(v, __shfl_xor(v, 16));
                v = fmaxf(v, __shfl_xor(v, 32));
                if (q == 0)
                    most[((h * MT + i) * G + g) * 16 + r] = v;
            }
        }
        __syncthreads();
        if (live) {
            for (int h = 0; h < (two ? 2 : 1); ++h) {
                float v = 0.0f;
#pragma unroll
                for (int k = 0; k < G; ++k)
                    v = fmaxf(v, most[((h * MT + i) * G + k) * 16 + r]);
                const Factor f = epl_cast::factor_of(v, a.cs.format == EPL_SCALE_UE8M0);
                store_codes<4>(a, row * cols + h * F + nq, h ? u : z, f);
                if (g == 0 && q == 0)
                    epl_cast::store_scale(a.cs, row, (h * F + nq) / kGroup, f);
            }
        }
    }
}

// Where the sums of a shared contraction wait: quad j of the wave of columns g,
// row tile i, of part z.
template <int J, int G>
__device__ __forceinline__ f32x4 *few_slot(const Args &a, int z, int e, int nb, int groups, int i, int g)
{
    return a.ws + (((((int64_t)z * a.E + e) * groups + nb) * 2 + i) * G + g) * J * 64;
}

template <bool PAIRED, int G, int WAVES, int MT>
__device__ __forceinline__ void few_rows(const Args &a, int e, int64_t row0, int left, int nb, bool shared,
                                         const FewShared &l)
{
    constexpr int J = PAIRED ? 2 : 1, KS = WAVES / G, M = 16 * MT;
    // blocks at a time, two times of them on their way: more spill (8 x 24 rows,
    // 7168 -> 4096: 56 us with 4, 52 with 2; gated and cast 64 with 2, 54 with 1)
    constexpr int U = PAIRED ? 1 : MT == 2 ? 2 : 4;
    constexpr int SEG = few_blocks<WAVES, MT>();
    static_assert(KS >= MT, "a row tile's epilogue has waves of its own");
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = wave % G, ks = wave / G;
    const int F = PAIRED ? a.N / 2 : a.N, kb = blocks_of(a.K), nblocks = blocks_of(a.N);
    const int n0 = (nb * G + g) * 16;                       // the wave's first column
    const int nq = min(n0 + q * 4, F - 4);                  // first column of the lane's quad
    f32x4 *const red = l.red;
    const auto rw = rsrc(reinterpret_cast<const char *>(a.w8 + (int64_t)e * a.N * a.K), a.N * a.K);
    const auto rx = rsrc(reinterpret_cast<const char *>(a.x8 + row0 * a.K), left * a.K);
    uint32_t ow[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
        ow[j] = (uint32_t)(min(n0 + r, F - 1) + j * F) * a.K + q * 16;
    // scales of the weight: of the workgroup's block of columns, and of the two
    // that the up half's columns may lie in
    const int wb0 = nb * G * 16 / kGroup, ub0 = (F + nb * G * 16) / kGroup;
    const int at_u = PAIRED ? 1 + (F + nq) / kGroup - ub0 : 0;
    f32x4 acc[MT][J];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
            acc[i][j] = f32x4{0, 0, 0, 0};

    // this workgroup's part of the blocks
    const int z = shared ? (int)blockIdx.z : 0, parts = shared ? (int)gridDim.z : 1;
    const int first = kb * z / parts, own = kb * (z + 1) / parts - first;
    const int start = (int)((uint32_t)(e * 13 + nb * 3) % (uint32_t)max(own, 1));
    auto block_at = [&](int v) { return first + (v + start < own ? v + start : v + start - own); };
    struct Chunk {
        i32x4 w[U][J][2];
    };
    for (int v0 = 0; v0 < own; v0 += SEG) {
        const int v1 = min(v0 + SEG, own);
        // weights of the positions p, p + KS, .. of this segment
        auto load = [&](int p) {
            Chunk c;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int v = p + u * KS, k = block_at(min(v, own - 1)) * kGroup;
                const bool lo = v < v1 && k + q * 16 < a.K, hi = v < v1 && k + q * 16 + 64 < a.K;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    c.w[u][j][0] = __builtin_bit_cast(
                        i32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, (int)(lo ? ow[j] : 0x80000000u), k, 0));
                    c.w[u][j][1] = __builtin_bit_cast(
                        i32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, (int)(hi ? ow[j] + 64 : 0x80000000u), k, 0));
                }
            }
            return c;
        };
        auto multiply = [&](const Chunk &c, int p) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // beyond the segment: no weights and no scales (an infinite one times
                // nothing would be NaN)
                const int at = min(p + u * KS, v1 - 1) - v0, as = p + u * KS < v1 ? at : SEG;
                const float *sw = l.sw + as * 4;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint8_t *row = l.x + (at * M + i * 16 + r) * 128;
                    const i32x4 x0 = *reinterpret_cast<const i32x4 *>(row + (q ^ swz(r)) * 16);
                    const i32x4 x1 = *reinterpret_cast<const i32x4 *>(row + ((4 + q) ^ swz(r)) * 16);
                    const i32x8 x = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
                    const float sx = l.sx[as * M + i * 16 + r];
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const i32x8 w = __builtin_shufflevector(c.w[u][j][0], c.w[u][j][1], 0, 1, 2, 3, 4, 5, 6, 7);
                        const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            w, x, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
                        acc[i][j] = scaled(part, sx * sw[j ? at_u : 0], acc[i][j]);
                    }
                }
            }
        };
        __syncthreads();                     // the segment, and the rows, before have been read
        for (int i = wave; i < (v1 - v0) * (M / 8); i += WAVES) {
            const int v = i / (M / 8), row = i % (M / 8) * 8 + (lane >> 3), p = (lane & 7) ^ swz(row);
            const int k = block_at(v0 + v) * kGroup;
            dma(rx, k + p * 16 < a.K ? (uint32_t)row * a.K + k + p * 16 : 0x80000000u,
                reinterpret_cast<uint16_t *>(l.x + i * 1024));
        }
        float sx = 0.0f, sw = 0.0f;
        if (tid / M < v1 - v0 && tid % M < left)
            sx = epl_cast::load_scale(a.xs, row0 + tid % M, block_at(v0 + tid / M));
        if (tid / 4 < v1 - v0) {
            const int n = tid % 4 == 0 ? wb0 : ub0 + tid % 4 - 1;
            if (tid % 4 < (PAIRED ? 3 : 1) && n < nblocks)
                sw = weight_scale(a, e, n, block_at(v0 + tid / 4));
        }
        // the first weights are on their way while the rows are waited for: they are
        // the last loads that begin before the wait, and none of them begins after
        int p = v0 + ks;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        Chunk c = load(p), d = load(p + KS * U);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        l.sx[tid] = sx;
        if (tid < SEG * 4)
            l.sw[tid] = sw;
        if (tid < M)
            l.sx[SEG * M + tid] = 0.0f;
        if (tid < 4)
            l.sw[SEG * 4 + tid] = 0.0f;
        all_but<4 * U * J>();
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
        for (; p < v1; p += 2 * KS * U) {
            multiply(c, p);
            c = load(p + 2 * KS * U);
            multiply(d, p + KS * U);
            d = load(p + 3 * KS * U);
        }
    }

    __syncthreads();           // red lies where other waves may still read x
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
            red[((ks * MT + i) * J + j) * G * 64 + g * 64 + lane] = acc[i][j];
    __syncthreads();
    // waves ks = 0 .. MT - 1 finish a row tile each
    f32x4 sum[J] = {};
    if (ks < MT) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            sum[j] = red[(ks * J + j) * G * 64 + g * 64 + lane];
#pragma unroll
            for (int o = 1; o < KS; ++o)
                sum[j] += red[((o * MT + ks) * J + j) * G * 64 + g * 64 + lane];
        }
    }
    if (shared) {
        if (ks < MT) {
            f32x4 *const to = few_slot<J, G>(a, z, e, nb, gridDim.x, ks, g) + lane;
#pragma unroll
            for (int j = 0; j < J; ++j)
                to[j * 64] = sum[j];
        }
        return;
    }
    few_finish<PAIRED, G, MT>(a, e, row0, left, nb, g, ks, ks < MT, sum, l.most);
}

template <bool PAIRED, int G, int WAVES>
__global__ __launch_bounds__(few_threads<WAVES>(), 4) void few_rows_kernel(Args a)
{
    constexpr int SEG = few_blocks<WAVES, 1>();
    __shared__ __align__(1024) uint8_t x[SEG * 16 * 128];
    __shared__ float sx[SEG * 16 + 32], sw[SEG * 4 + 4];
    static_assert(sizeof(x) >= WAVES * 2 * (PAIRED ? 2 : 1) * 64 * sizeof(f32x4), "the sums fit x");
    __shared__ float most[G == 8 ? 2 * 2 * G * 16 : 1];
    const int e = blockIdx.y, nb = blockIdx.x;
    const FewShared l{x, sx, sw, reinterpret_cast<f32x4 *>(x), most};
    int64_t lo;
    const int cnt = block_of(a, e, lo);
    const bool shared = gridDim.z > 1 && cnt <= kFewMost;
    if (!shared && blockIdx.z > 0)
        return;                              // (an expert of many rows: the first part takes it all)
    for (int m = 0; m < cnt; m += 32) {
        if (cnt - m <= 16)
            few_rows<PAIRED, G, WAVES, 1>(a, e, lo + m, cnt - m, nb, shared, l);
        else
            few_rows<PAIRED, G, WAVES, 2>(a, e, lo + m, min(cnt - m, 32), nb, shared, l);
    }
}

// Adds the parts of shared contractions, in order, and runs their epilogue: a
// workgroup of 2 G waves takes what one of few_rows_kernel's takes.
template <bool PAIRED, int G>
__global__ __launch_bounds__(G * 128) void few_join_kernel(Args a, int parts)
{
    constexpr int J = PAIRED ? 2 : 1;
    __shared__ float most[G == 8 ? 2 * 2 * G * 16 : 1];
    const int e = blockIdx.y, nb = blockIdx.x, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = wave % G, i = wave / G;
    int64_t lo;
    const int cnt = block_of(a, e, lo);
    if (cnt == 0 || cnt > kFewMost)
        return;
    const bool mine = i * 16 < cnt;
    f32x4 sum[J] = {};
    if (mine) {
        for (int z = 0; z < parts; ++z) {
            const f32x4 *from = few_slot<J, G>(a, z, e, nb, gridDim.x, i, g) + lane;
#pragma unroll
            for (int j = 0; j < J; ++j)
                sum[j] += from[j * 64];
        }
    }
    few_finish<PAIRED, G, 2>(a, e, lo, cnt, nb, g, i, mine, sum, most);
}

}  // namespace epl_product8
