// libepl.so host side of the experts' products on 8-bit rows: argument checks
// and launches of epl_expert_product_fp8 (include/epl.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "epl.h"
#include "epl_product_fp8_kernels.h"
#include "epl_product_host.h"

namespace {

namespace P = epl_product8;
namespace H = epl_product_host;

using namespace H;

constexpr int64_t kMaxWeight = int64_t(1) << 30;     // bytes of an expert's

int out_cols(const epl_product_fp8_desc &p)
{
    return p.activation == EPL_ACT_SWIGLU        ? p.out_cols / 2
           : p.activation == EPL_ACT_SWIGLU_GRAD ? p.out_cols * 2
                                                 : p.out_cols;
}

bool desc_ok(const epl_product_fp8_desc *p)
{
    if (!p || p->reserved != 0 || p->reserved2 != 0)
        return false;
    if (p->num_experts < 1 || p->num_experts > epl_product::kMaxExperts)
        return false;
    if (p->num_rows < 0 || p->num_rows > kMaxRows || p->expected_rows < 0)
        return false;
    if (p->in_cols < 16 || p->in_cols % 16 != 0 || p->in_cols > kMaxCols || p->out_cols < 16 ||
        p->out_cols % 16 != 0 || p->out_cols > kMaxCols)
        return false;
    if ((int64_t)p->in_cols * p->out_cols > kMaxWeight)
        return false;
    if (p->activation < EPL_ACT_NONE || p->activation > EPL_ACT_SWIGLU_GRAD)
        return false;
    if (p->out_type != EPL_OUT_F32 && p->out_type != EPL_OUT_BF16)
        return false;
    if (p->weight_layout != EPL_WEIGHT_OUT_IN && p->weight_layout != EPL_WEIGHT_IN_OUT)
        return false;
    if (p->weight_scale_format != EPL_SCALE_F32 && p->weight_scale_format != EPL_SCALE_UE8M0)
        return false;
    // codes come in whole groups of 128 columns of each half
    const bool two = p->activation == EPL_ACT_SWIGLU_GRAD;
    if (p->codes_scale_format != EPL_SCALE_NONE &&
        ((p->codes_scale_format != EPL_SCALE_F32 && p->codes_scale_format != EPL_SCALE_UE8M0) ||
         (two ? p->out_cols : out_cols(*p)) % 128 != 0))
        return false;
    if (p->scale_format == EPL_SCALE_F32_RECT)
        return p->rows_per_expert >= 1 && p->num_rows % p->rows_per_expert == 0;
    return p->rows_per_expert == 0 &&
           (p->scale_format == EPL_SCALE_F32 || p->scale_format == EPL_SCALE_UE8M0);
}

// Rows an expert, on average, up to which the weights are read straight from
// memory, once for every 32 rows of an expert. Measured (this way, tiles), us: 8
// experts of 24 rows, 7168 -> 4096: 52, 63, gated with its cast 55, 76; 64 of 24,
// 4096 -> 2048: 108, 106; 8 of 32, none of them more, 7168 -> 4096: 53, 63; but where
// counts scatter about 32 half of the experts' weights are read twice. The counts are on
// the GPU: an uneven batch of few rows on average takes this way too, and longer.
constexpr int64_t kFewRows = 24;

// Large tiles take 2.2 us a stage for four times what a small one, two of them on
// a CU, takes 1.4 for. Measured (large, small), us: 8 experts of 4096 rows, 7168 ->
// 4096: 1056, 1330; of 512: 124, 161; of 256: 93, 83; 64 of 192, 4096 -> 2048: 159,
// 204; of 128: 149, 135; 1 of 4096, 2048 -> 2048: 51, 36.
constexpr Cost cost_of(Kind k) { return k == kLarge ? Cost{7.0, 2.2} : Cost{4.0, 1.4}; }

int max_parts(int64_t depth) { return H::max_parts(depth, P::kGroup); }

int64_t average_rows(const epl_product_fp8_desc &p)
{
    const int64_t rows = p.expected_rows > 0 ? std::min(p.expected_rows, p.num_rows) : p.num_rows;
    return (rows + p.num_experts - 1) / p.num_experts;
}

Kind kind_of(const epl_product_fp8_desc &p)
{
    const int64_t avg = average_rows(p);
    if (p.weight_layout == EPL_WEIGHT_OUT_IN && avg <= kFewRows)
        return kFew;
    // a small tile holds half a group of 128 columns of the gated activation
    if (p.activation == EPL_ACT_SWIGLU && p.codes_scale_format != EPL_SCALE_NONE)
        return kLarge;
    auto time = [&](Kind k) {
        return tiles_time(k, avg, p.out_cols, p.num_experts, p.in_cols, P::kGroup, cost_of(k));
    };
    return time(kLarge) <= time(kSmall) ? kLarge : kSmall;
}

int64_t tiles_of(const epl_product_fp8_desc &p, Kind k)
{
    return product_tiles(p.num_rows, p.num_experts, p.out_cols, k);
}

// Columns of y of a workgroup of the few-rows kernel: a whole group where the
// result is cast, else half of one.
int few_columns(const epl_product_fp8_desc &p) { return p.codes_scale_format != EPL_SCALE_NONE ? 128 : 64; }

int64_t few_groups(const epl_product_fp8_desc &p)
{
    const int cols = p.activation == EPL_ACT_SWIGLU ? p.out_cols / 2 : p.out_cols;
    return (cols + few_columns(p) - 1) / few_columns(p);
}

// Parts that its contraction is shared out to: so many that every CU has a
// workgroup, of eight blocks each at least, and where a workgroup's weights, at
// 35 KB a us, would take so much longer that the join's launch (5 us) pays: 1 expert
// of one row, 7168 -> 4096, gated: 19 us in 8 parts, 55 whole; 2048 -> 7168: 17 in
// two, 14 whole.
int few_parts(const epl_product_fp8_desc &p)
{
    const int64_t groups = few_groups(p) * p.num_experts, blocks = (p.in_cols + 127) / 128;
    const int64_t parts = std::min<int64_t>(kCus / std::max<int64_t>(groups, 1), blocks / 8);
    const int64_t bytes = (int64_t)few_columns(p) * (p.activation == EPL_ACT_SWIGLU ? 2 : 1) * p.in_cols;
    return parts > 1 && bytes - bytes / parts > 5 * 35000 ? (int)parts : 1;
}

size_t few_workspace(const epl_product_fp8_desc &p)
{
    const int parts = few_parts(p);
    const int paired = p.activation == EPL_ACT_SWIGLU ? 2 : 1;
    return parts < 2 ? 0
                     : kHeaderBytes + (size_t)parts * p.num_experts * few_groups(p) * P::kFewMost *
                                          few_columns(p) * paired * sizeof(float);
}

template <bool PAIRED, int G>
int launch_few(const P::Args &a, unsigned groups, int parts, hipStream_t s)
{
    constexpr int waves = 2 * G;
    const dim3 grid(groups, (unsigned)a.E);
    hipLaunchKernelGGL((P::few_rows_kernel<PAIRED, G, waves>), dim3(groups, (unsigned)a.E, (unsigned)parts),
                       dim3(P::few_threads<waves>()), 0, s, a);
    int rc = launch_status();
    if (rc == EPL_OK && parts > 1) {
        hipLaunchKernelGGL((P::few_join_kernel<PAIRED, G>), grid, dim3(G * 128), 0, s, a, parts);
        rc = launch_status();
    }
    return rc;
}

template <int SIDE, bool QT, bool CODES>
int launch_tiles(const P::Args &a, int64_t tiles, hipStream_t s)
{
    const bool split = a.ws && a.max_parts > 1;
    const int grid = tile_grid(a, tiles, SIDE, split);
    constexpr int threads = P::tile_threads(SIDE);
    hipLaunchKernelGGL((P::tile_kernel<SIDE, SIDE, QT, CODES>), dim3((unsigned)grid), dim3(threads), 0, s, a);
    int rc = launch_status();
    if (rc == EPL_OK && split) {
        constexpr int pieces = SIDE / P::kWavesM / 16;
        hipLaunchKernelGGL((P::join_kernel<SIDE, SIDE, CODES>), dim3(pieces, join_grid(tiles, grid)),
                           dim3(threads), 0, s, a, grid);
        rc = launch_status();
    }
    return rc;
}

template <bool QT, bool CODES>
int launch_kind(Kind k, const P::Args &a, int64_t tiles, hipStream_t s)
{
    return k == kSmall ? launch_tiles<128, QT, CODES>(a, tiles, s) : launch_tiles<256, QT, CODES>(a, tiles, s);
}

}  // namespace

extern "C" {

int epl_product_fp8_validate(const epl_product_fp8_desc *p)
{
    return desc_ok(p) ? EPL_OK : EPL_EINVAL;
}

size_t epl_product_fp8_workspace_bytes(const epl_product_fp8_desc *p)
{
    if (!desc_ok(p))
        return 0;
    const Kind k = kind_of(*p);
    return k == kFew ? few_workspace(*p) : tile_workspace(k, tiles_of(*p, k), max_parts(p->in_cols));
}

int epl_expert_product_fp8(const epl_product_fp8_desc *p, const uint8_t *x, const void *x_scale,
                           const uint8_t *weight, const void *weight_scale, const float *bias,
                           const uint16_t *residual, const int32_t *expert_start_loc,
                           const int32_t *num_tokens_per_expert, uint16_t *pre, void *y,
                           uint8_t *codes, void *codes_scale, void *workspace, void *stream)
{
    if (!desc_ok(p))
        return EPL_EINVAL;
    const bool grad = is_grad(p->activation);
    if (grad && (bias || residual))
        return EPL_EINVAL;
    const size_t ws_align = p->weight_scale_format == EPL_SCALE_UE8M0 ? 1 : 4;
    if (!weight || !aligned(weight, 16) || !weight_scale || !aligned(weight_scale, ws_align) ||
        !expert_start_loc || !aligned(expert_start_loc, 4) || !num_tokens_per_expert ||
        !aligned(num_tokens_per_expert, 4) || !aligned(bias, 16) || !aligned(residual, 16) ||
        !aligned(pre, 16) || !aligned(y, 16) || !aligned(codes, 16) || !aligned(codes_scale, 4) ||
        !aligned(workspace, 256))
        return EPL_EINVAL;
    const bool quantized = p->codes_scale_format != EPL_SCALE_NONE;
    if (!quantized && (codes || codes_scale))
        return EPL_EINVAL;
    if (p->num_rows == 0)
        return EPL_OK;
    if (!x || !aligned(x, 16) || !x_scale || !aligned(x_scale, 4) || (grad && !pre) ||
        (quantized ? !codes || !codes_scale : !y))
        return EPL_EINVAL;
    P::Args a{};
    a.x8 = x;
    a.w8 = weight;
    a.xs = P::Scales{const_cast<void *>(x_scale), p->scale_format, (p->in_cols + 127) / 128,
                     p->rows_per_expert, p->num_rows};
    a.wscale = weight_scale;
    a.ws_bytes = p->weight_scale_format == EPL_SCALE_UE8M0;
    a.in_out = p->weight_layout == EPL_WEIGHT_IN_OUT;
    a.codes = codes;
    a.cs = P::Scales{codes_scale, p->codes_scale_format, out_cols(*p) / 128, 0, p->num_rows};
    a.bias = bias;
    a.residual = reinterpret_cast<const __bf16 *>(residual);
    a.pre = reinterpret_cast<__bf16 *>(pre);
    a.y = y;
    a.start = expert_start_loc;
    a.count = num_tokens_per_expert;
    a.rows = p->num_rows;
    a.E = p->num_experts;
    a.K = p->in_cols;
    a.N = p->out_cols;
    a.act = p->activation;
    a.out_f32 = p->out_type == EPL_OUT_F32;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Kind k = kind_of(*p);
    if (k == kFew) {
        use_workspace(a, workspace);
        const unsigned groups = (unsigned)few_groups(*p);
        const int parts = workspace ? few_parts(*p) : 1;
        if (p->activation == EPL_ACT_SWIGLU)
            return quantized ? launch_few<true, 8>(a, groups, parts, s) : launch_few<true, 4>(a, groups, parts, s);
        return quantized ? launch_few<false, 8>(a, groups, parts, s) : launch_few<false, 4>(a, groups, parts, s);
    }
    a.max_parts = max_parts(a.K);
    a.stages = stages_of(a.K, P::kGroup);
    use_workspace(a, a.max_parts > 1 ? workspace : nullptr);
    const int64_t tiles = tiles_of(*p, k);
    if (a.in_out)
        return quantized ? launch_kind<true, true>(k, a, tiles, s) : launch_kind<true, false>(k, a, tiles, s);
    return quantized ? launch_kind<false, true>(k, a, tiles, s) : launch_kind<false, false>(k, a, tiles, s);
}

}  // extern "C"
