// libepl.so host side of the experts' products on 8-bit rows: argument checks
// and launches of epl_expert_product_fp8 (include/epl.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "epl.h"
#include "epl_product_fp8_kernels.h"

namespace {

namespace P = epl_product8;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launch_status() { return hipGetLastError() == hipSuccess ? EPL_OK : EPL_EHIP; }

// Offsets within one expert's weight and within a tile are 32-bit, and so are
// counts of rows, stepped through by up to a tile.
constexpr int32_t kMaxCols = 1 << 20;
constexpr int64_t kMaxWeight = int64_t(1) << 30;
constexpr int64_t kMaxRows = INT32_MAX - 1023;

bool is_grad(int act)
{
    return act == EPL_ACT_SILU_GRAD || act == EPL_ACT_GELU_GRAD || act == EPL_ACT_SWIGLU_GRAD;
}

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

}  // namespace

extern "C" {

int epl_product_fp8_validate(const epl_product_fp8_desc *p)
{
    return desc_ok(p) ? EPL_OK : EPL_EINVAL;
}

size_t epl_product_fp8_workspace_bytes(const epl_product_fp8_desc *) { return 0; }

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
    a.ws = weight_scale;
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
    const bool paired = p->activation == EPL_ACT_SWIGLU;
    const int cols = paired ? a.N / 2 : a.N;
    const dim3 grid((unsigned)((cols + 127) / 128), (unsigned)a.E);
    if (paired)
        hipLaunchKernelGGL((P::few_rows_kernel<true>), grid, dim3(P::kFewThreads), 0, s, a);
    else
        hipLaunchKernelGGL((P::few_rows_kernel<false>), grid, dim3(P::kFewThreads), 0, s, a);
    return launch_status();
}

}  // extern "C"
